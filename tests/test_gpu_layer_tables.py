"""Malformed tables of lengths and slots at the operators around a recurrence: recorded, nothing read or written out of range,
zeros in the rows of no request."""
import pytest
import torch

import kda_gated_delta_gb300 as kda
from tests.test_gpu_layer import BF16, DEV, F32, gen, idx, no_device_error, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def table(cu):
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


# tables in which a request's first row lies before the stretch that its rows begin with, and by fewer rows than a window has
BEHIND = [(4, [0, 2, 1, 30]), (4, [0, 1, 1, 0, 30]), (3, [0, 1, 0, 30]), (4, [0, 13, 12, 30]), (4, [0, 2, 0, 30])]


@pytest.mark.parametrize("W,cu", BEHIND, ids=str)
@pytest.mark.parametrize("dtype,C", [(BF16, 64), (BF16, 13), (F32, 64), (F32, 5)])
def test_conv_reads_no_row_before_a_request(W, cu, dtype, C):
    """x lies between rows of NaN, which reach no output and no state."""
    g = gen(40)
    T, n = 30, len(cu) - 1
    rows = torch.full((T + 16, C), float("nan"), dtype=dtype, device=DEV)
    x = rows[8:8 + T]
    x.copy_(normal(g, T, C, dtype=dtype))
    pool, w = normal(g, n, W - 1, C, dtype=dtype), normal(g, C, W)
    y = kda.causal_conv(x, w, pool, idx(list(range(n))), table(cu))
    assert kda.check_device_errors() == 2
    assert bool(y.isfinite().all()) and bool(pool.isfinite().all())
