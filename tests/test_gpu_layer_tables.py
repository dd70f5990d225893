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


# tables that decrease, in front, in the middle and behind, by steps that the walk over the rows goes over; with requests
# before the first row and behind the last
UNSOUND = [[0, 20, 10, 30], [0, 2, 1, 30], [0, 30, 0, 30], [0, 10, 10, 9, 30], [0, 5, 3, 3, 30], [0, 29, 30, 29, 30], [0, 30, 77], [0, 30, 30, 31],
           [-5, 0, 30], [-5, -7, 0, 30], [0, 17, -3, 17, 30], [30, 0], [12, 30, 0]]


@pytest.mark.parametrize("cu", UNSOUND, ids=str)
@pytest.mark.parametrize("W,dtype,C", [(4, BF16, 64), (4, BF16, 9), (2, F32, 64)])
def test_conv_records_tables(cu, W, dtype, C):
    """Recorded, and nothing outside is touched: NaN around x, slots of no request, and values around the outputs."""
    g = gen(41)
    T, n = 30, len(cu) - 1
    rows = torch.full((T + 2000, C), float("nan"), dtype=dtype, device=DEV)
    x = rows[1000:1000 + T]
    x.copy_(normal(g, T, C, dtype=dtype))
    pool, w = normal(g, n + 1, W - 1, C, dtype=dtype), normal(g, C, W)
    before = pool[n].clone()
    out = torch.full((T + 2000, C), 7.0, dtype=dtype, device=DEV)
    y = kda.causal_conv(x, w, pool, idx(list(range(n))), table(cu), out=out[1000:1000 + T])
    assert kda.check_device_errors() == 2
    assert bool(y.isfinite().all()) and bool(pool.isfinite().all()) and torch.equal(pool[n], before)
    assert bool((out[:1000] == 7).all()) and bool((out[1000 + T:] == 7).all())
    assert kda.check_device_errors() == 0


@pytest.mark.parametrize("many", [1, 700])
@pytest.mark.parametrize("bad", [None, 0, 1, 300, 698])
def test_conv_tables_of_many_requests(many, bad):
    """One pair out of order among 700 requests without tokens, before or behind the rows; the sound table records nothing."""
    g = gen(42)
    T, C = 40, 2056
    for front in (True, False):
        cu = [0] * many + [T] if front else [0] + [T] * many
        if bad is not None and bad + 1 < len(cu):
            cu[bad] += 1 if front else -1
        sound = all(a <= b for a, b in zip(cu, cu[1:])) and cu[0] == 0 and cu[-1] == T
        x, w, pool = normal(g, T, C, dtype=BF16), normal(g, C, 4), normal(g, many, 3, C, dtype=BF16)
        y = kda.causal_conv(x, w, pool, idx(list(range(many))), table(cu))
        assert kda.check_device_errors() == (0 if sound else 2)
        assert bool(y.isfinite().all())


@pytest.mark.parametrize("cu", UNSOUND, ids=str)
@pytest.mark.parametrize("scale,dtype,P,N", [(10, BF16, 64, 128), (1, BF16, 64, 128), (1, F32, 32, 16)])
def test_ssm_records_tables(cu, scale, dtype, P, N):
    """The same of the recurrence, in chunks (300 rows), and token by token."""
    cu = [c * scale for c in cu]
    H, G, T, n = 2, 1, 30 * scale, len(cu) - 1
    g = gen(43)
    rows = torch.full((T + 400, H * P + 2 * G * N), float("nan"), dtype=dtype, device=DEV)
    mine = rows[200:200 + T]
    mine.copy_(normal(g, *mine.shape, dtype=dtype))
    x, B, C = (t.unflatten(1, s) for t, s in zip(mine.split([H * P, G * N, G * N], 1), ((H, P), (G, N), (G, N))))
    dt, A_log, pool = normal(g, T, H), torch.rand(H, generator=g, device=DEV), normal(g, n + 1, H, P, N)
    before = pool[n].clone()
    out = torch.zeros((T + 400, H, P), dtype=dtype, device=DEV)
    out[:200] = out[200 + T:] = 7
    kda.ssm_prefill(x, dt, B, C, A_log, table(cu), pool, idx(list(range(n))), out=out[200:200 + T])
    assert kda.check_device_errors() == 2
    assert bool(out.isfinite().all()) and bool(pool.isfinite().all()) and torch.equal(pool[n], before)
    assert bool((out[:200] == 7).all()) and bool((out[200 + T:] == 7).all())
    assert kda.check_device_errors() == 0


def ssm_call(g, T, dtype, H, P, N, tail=0):
    """Inputs of a recurrence over T rows, and an output that holds sevens."""
    ins = (normal(g, T, H, P, dtype=dtype), normal(g, T, H), normal(g, T, 1, N, dtype=dtype), normal(g, T, 1, N, dtype=dtype), torch.rand(H, generator=g, device=DEV))
    return ins, torch.full((T, H, P), 7.0, dtype=dtype, device=DEV)


# scale 10: in chunks
FORMS = [(10, BF16, 64, 128), (1, BF16, 64, 128), (1, F32, 32, 16), (1, BF16, 64, 256)]


@pytest.mark.parametrize("scale,dtype,P,N", FORMS)
@pytest.mark.parametrize("cu,taken", [([0, 10, 77], [0]), ([-5, 10, 30], [1]), ([-5, 10, 20, 77], [1]), ([-9, -5, 4, 30], [2]), ([0, 12, 40, 77], [0]),
                                      ([4, 10, 25], [0, 1]), ([-5, 77], []), ([-5, -5], []), ([77, 77], []), ([0, 0, 0], [0, 1]), ([30, 30], [0])], ids=str)
def test_ssm_rows_of_no_request_get_zeros(cu, taken, scale, dtype, P, N):
    """Requests that reach past either end are taken by nobody: zeros in their rows, their states as they were, and the other
    requests' outputs and states are those of a sound call."""
    H, T, n = 2, 30 * scale, len(cu) - 1
    cu = [c * scale for c in cu]
    g = gen(44)
    ins, out = ssm_call(g, T, dtype, H, P, N)
    pool = normal(g, n, H, P, N)
    before = pool.clone()
    kda.ssm_prefill(*ins, table(cu), pool, idx(list(range(n))), out=out)
    assert kda.check_device_errors() == 2
    want, state = torch.zeros_like(out), before.clone()
    for b in taken:
        lo, hi = cu[b], cu[b + 1]
        if lo < hi:
            one = before[b:b + 1].clone()
            want[lo:hi] = kda.ssm_prefill(*[t[lo:hi] for t in ins[:4]], ins[4], table([0, hi - lo]), one, idx([0]))
            state[b] = one[0]
    assert torch.equal(out, want) and torch.equal(pool, state)


@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_slots_of_requests_without_tokens(at):
    """A slot past the pool is recorded whether its request has tokens or not, in every form."""
    g = gen(45)
    cu, slots = [0, 0, 200, 200, 200], [0, 1, 2, 3]
    slots[at] = 4
    x, w, pool = normal(g, 200, 64), normal(g, 64, 4), normal(g, 4, 3, 64)
    kda.causal_conv(x, w, pool, idx(slots), table(cu))
    assert kda.check_device_errors() == 1
    for dtype, P, N in ((BF16, 64, 128), (F32, 32, 16)):
        for n in (4, 3):                                 # 50 tokens a request: with short ones apart; 66: without
            if n == 3 and at == 3:
                continue
            ins, out = ssm_call(g, 200, dtype, 2, P, N)
            kda.ssm_prefill(*ins, table(cu[:n + 1]), normal(g, 4, 2, P, N), idx(slots[:n]), out=out)
            assert kda.check_device_errors() == 1


def test_codes_of_two_units_at_once():
    """A check gives one code and clears them all."""
    g = gen(46)
    for _ in range(3):
        kda.causal_conv(normal(g, 30, 8), normal(g, 8, 4), normal(g, 2, 3, 8), idx([0, 1]), table([0, 20, 31]))
        kda.selftest_wait_timeout(100)
        assert kda.check_device_errors() == 3 and kda.check_device_errors() == 0
