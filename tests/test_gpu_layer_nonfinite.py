"""Non-finite inputs of the selective recurrence: what its definition makes non-finite, and nothing else, in every form."""
import pytest
import torch

import kda_gated_delta_gb300 as kda
from tests import layer_reference as ref
from tests.test_gpu_layer import BF16, DEV, F32, gen, idx, no_device_error, normal, on_tensor_cores, ssm_bounds, ssm_inputs  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

# in chunks (heads of 64, pairs of heads, a head in two slices, few states), token by token, in segments of either
FORMS = [(BF16, 3, 64, 128, 1, 300), (BF16, 4, 64, 128, 2, 300), (BF16, 2, 128, 64, 2, 300), (BF16, 2, 64, 16, 1, 300), (BF16, 2, 32, 16, 1, 300),
         (F32, 2, 64, 64, 2, 300), (BF16, 1, 64, 128, 1, 4500), (F32, 1, 32, 64, 1, 4500)]


def inputs(seed, dtype, H, P, N, G, T):
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(seed, [T], H, P, N, G, dtype)
    return dict(x=x, dt=dt, B=B, C=C, A_log=A_log - 2, dt_bias=dt_bias, D=D)


def prefill(i, pool, T):
    p = pool.clone()
    y = kda.ssm_prefill(i["x"], i["dt"], i["B"], i["C"], i["A_log"], ref.lengths_to_cu([T], DEV), p, idx([0]), dt_bias=i["dt_bias"], D=i["D"])
    return y, p[0]


@pytest.mark.parametrize("dtype,H,P,N,G,T", FORMS)
@pytest.mark.parametrize("name", ["A_log", "dt_bias"])
def test_nan_parameter_of_a_head(name, dtype, H, P, N, G, T):
    """All outputs and the state of that head are NaN, and the others' bits are those of a clean call."""
    i = inputs(50, dtype, H, P, N, G, T)
    pool = normal(gen(51), 1, H, P, N)
    want, state = prefill(i, pool, T)
    i[name] = i[name].clone()
    i[name][H - 1] = NAN
    y, s = prefill(i, pool, T)
    assert bool(y[:, H - 1].isnan().all()) and bool(s[H - 1].isnan().all())
    assert torch.equal(y[:, :H - 1], want[:, :H - 1]) and torch.equal(s[:H - 1], state[:H - 1])
    p = pool.clone()
    y = kda.ssm_decode(*(i[k][:1] for k in ("x", "dt", "B", "C")), i["A_log"], p, idx([0]), dt_bias=i["dt_bias"], D=i["D"])
    assert bool(y[0, H - 1].isnan().all()) and bool(p[0, H - 1].isnan().all()) and bool(y[0, :H - 1].isfinite().all())


@pytest.mark.parametrize("dtype,H,P,N,G,T", FORMS)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("at", [0, 77, 128, 299])
def test_step_of_a_token(at, value, dtype, H, P, N, G, T):
    """From that token on the head's outputs are not finite; those before are within their bounds; other heads keep theirs."""
    i = inputs(52, dtype, H, P, N, G, T)
    pool = normal(gen(53), 1, H, P, N)
    want, state = prefill(i, pool, T)
    n = min(T, 300)
    ref_y, _, mag, _ = ref.ssm(i["x"][:n], i["dt"][:n], i["B"][:n], i["C"][:n], i["A_log"], pool, [0], [n], i["dt_bias"], i["D"])
    i["dt"] = i["dt"].clone()
    i["dt"][at, H - 1] = value
    y, s = prefill(i, pool, T)
    assert torch.equal(y[:, :H - 1], want[:, :H - 1]) and torch.equal(s[:H - 1], state[:H - 1])
    assert not bool(y[at:, H - 1].isfinite().any()) and not bool(s[H - 1].isfinite().any())
    yb, _ = ssm_bounds(ref_y, mag, mag[0], n, N, dtype, on_tensor_cores(dtype, P, N))
    ref.within(y[:at, H - 1], ref_y[:at, H - 1], yb[:at, H - 1])


@pytest.mark.parametrize("dtype,H,P,N,G,T", FORMS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 77, 128, 299])
def test_b_and_c_of_a_token(at, value, dtype, H, P, N, G, T):
    """A non-finite B reaches its group's outputs from its token on, a non-finite C those of its token; all others keep their
    bits."""
    i = inputs(54, dtype, H, P, N, G, T)
    pool = normal(gen(55), 1, H, P, N)
    want, state = prefill(i, pool, T)
    clean, mine, n = dict(i), H - H // G, N - 3
    i["B"] = i["B"].clone()
    i["B"][at, G - 1, n] = value
    y, s = prefill(i, pool, T)
    assert torch.equal(y[:at], want[:at]) and torch.equal(y[:, :mine], want[:, :mine]) and not bool(y[at:, mine:].isfinite().any())
    others = torch.arange(N, device=DEV) != n
    assert torch.equal(s[:mine], state[:mine]) and torch.equal(s[..., others], state[..., others]) and not bool(s[mine:, :, n].isfinite().any())
    i = dict(clean, C=clean["C"].clone())
    i["C"][at, G - 1, n] = value
    y, s = prefill(i, pool, T)
    keep = torch.arange(T, device=DEV) != at
    assert torch.equal(s, state) and torch.equal(y[keep], want[keep]) and torch.equal(y[at, :mine], want[at, :mine])
    assert not bool(y[at, mine:].isfinite().any())


@pytest.mark.parametrize("dtype,H,P,N,G,T", FORMS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [(0,), (77,), (128,), (299,), (40, 33, 127, 255)], ids=str)
def test_x_of_a_token(at, value, dtype, H, P, N, G, T):
    """A non-finite x reaches its own channel from its token on, and its channel's states; all else keeps its bits."""
    i = inputs(56, dtype, H, P, N, G, T)
    pool = normal(gen(57), 1, H, P, N)
    want, state = prefill(i, pool, T)
    i["x"] = i["x"].clone()
    touched, spoilt = torch.zeros(T, H, P, dtype=torch.bool, device=DEV), torch.zeros(H, P, dtype=torch.bool, device=DEV)
    for k, t in enumerate(at):
        h, c = (H - 1 - k) % H, (P - 7 + 5 * k) % P
        i["x"][t, h, c] = value
        touched[t:, h, c] = True
        spoilt[h, c] = True
    y, s = prefill(i, pool, T)
    assert torch.equal(y[~touched], want[~touched]) and torch.equal(s[~spoilt], state[~spoilt])
    assert not bool(y[touched].isfinite().any()) and not bool(s[spoilt].isfinite().any())


@pytest.mark.parametrize("out", [BF16, F32])
def test_x_not_finite_behind_a_request(out):
    """Rows of x that are not finite behind a request's last, inside its last chunk, and a request that is nothing but NaN."""
    H, P, N, G, lens = 2, 64, 128, 1, [300, 60, 100]
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(58, lens, H, P, N, G, BF16)
    pool = normal(gen(59), 3, H, P, N)
    calls = []
    for bad in (False, True):
        p = pool.clone()
        if bad:
            x = x.clone()
            x[300:360] = NAN
        calls.append((kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), p, idx([0, 1, 2]), dt_bias=dt_bias, D=D, out_dtype=out), p))
    (want, state), (y, s) = calls
    assert torch.equal(y[:300], want[:300]) and torch.equal(y[360:], want[360:]) and torch.equal(s[[0, 2]], state[[0, 2]])
    assert bool(y[300:360].isnan().all()) and bool(s[1].isnan().all())
