"""Short convolution, selective recurrence and group norm against their 64-bit forms.

Bounds, element by element.  A sum of n products in fp32 is off by at most (n + 1) half steps of the sum of their
magnitudes; a sigmoid by the special-function unit's exponential and reciprocal by 2^-18 of itself (argument up to 16:
16 / ln 2 half steps in the exponent, 2^-19.5, and the two functions' own 2^-22); a result is then rounded once to its
type."""
import pytest
import torch

import kda_gated_delta_gb300 as kda
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
SIGMOID = 2.0 ** -18


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0, std, generator=g)


def idx(slots):
    return torch.tensor(slots, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def no_device_error():
    kda.check_device_errors()
    yield
    assert kda.check_device_errors() == 0


# ---- convolution --------------------------------------------------------------------------------------

def conv_bound(want, mag, W, dtype, silu):
    # d silu / dx <= 1.1; the last rounding is of the computed value, hence the share of the bound itself
    b = (1.1 if silu else 1.0) * (W + 2) * ref.F32 * mag + (SIGMOID * want.abs() if silu else 0)
    return b + ref.half_step(dtype) * (want.abs() + b) + 1e-40


LENS = [[1], [40], [3, 1, 2, 0, 33, 64, 5], [31, 1, 2, 31, 1, 1, 30, 2], [0, 0, 7, 0], [1] * 40, [97, 128, 31]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("W,dtype,C,silu,bias", [(4, BF16, 64, True, False), (4, BF16, 2056, True, True), (3, F32, 20, False, True),
                                                 (2, BF16, 13, True, False), (4, F32, 37, True, True), (2, F32, 1, False, False)])
def test_conv_rows(lens, W, dtype, C, silu, bias):
    g = gen(1)
    T, slots = sum(lens), [5 + len(lens) - i for i in range(len(lens))]
    if len(lens) > 2:
        slots[1] = -1
    x, w = normal(g, T, C, dtype=dtype), normal(g, C, W, std=0.5)
    b = normal(g, C) if bias else None
    pool = normal(g, len(lens) + 6, W - 1, C, dtype=dtype)
    want, state, mag = ref.conv(x, w, pool, slots, lens, b, silu)
    y = kda.causal_conv(x, w, pool, idx(slots), ref.lengths_to_cu(lens, DEV), bias=b, activation="silu" if silu else None)
    ref.within(y, want, conv_bound(want, mag, W, dtype, silu))
    assert torch.equal(pool.double().cpu(), state)


@pytest.mark.parametrize("W,dtype,C", [(4, BF16, 264), (3, BF16, 9), (2, F32, 8), (4, F32, 5)])
def test_conv_decode_continues_a_prompt(W, dtype, C):
    """A prompt at once, in parts, and token by token: the same outputs and states, bit for bit."""
    g = gen(2)
    n, T = 3, 70
    x, w = normal(g, n, T, C, dtype=dtype), normal(g, C, W)
    slots = idx([2, 0, 3])
    pools = [torch.zeros(4, W - 1, C, dtype=dtype, device=DEV) for _ in range(3)]
    cu = ref.lengths_to_cu([T] * n, DEV)
    whole = kda.causal_conv(x.flatten(0, 1), w, pools[0], slots, cu, activation="silu").view(n, T, C)
    parts = []
    for a, b in ((0, 1), (1, 3), (3, 36), (36, 70)):
        parts.append(kda.causal_conv(x[:, a:b].flatten(0, 1), w, pools[1], slots, ref.lengths_to_cu([b - a] * n, DEV), activation="silu").view(n, b - a, C))
    single = torch.stack([kda.causal_conv(x[:, t].contiguous(), w, pools[2], slots, activation="silu") for t in range(T)], 1)
    assert torch.equal(whole, torch.cat(parts, 1)) and torch.equal(whole, single)
    assert torch.equal(pools[0], pools[1]) and torch.equal(pools[0], pools[2])


@pytest.mark.parametrize("split", [(64, 64, 64), (72, 8, 112), (191, 1), (1, 2, 3, 186)])
@pytest.mark.parametrize("cu", [True, False])
def test_conv_parts_of_a_strided_projection(split, cu):
    g = gen(3)
    lens = [5, 40, 1] if cu else [1] * 6
    T, C = sum(lens), sum(split)
    rows = normal(g, T, C + 72, dtype=BF16)
    x, w = rows[:, 8:8 + C], normal(g, C, 4)
    slots = [1, -1, 0] if cu else [3, 1, -1, 0, 2, 4]
    pool = normal(g, 6, 3, C, dtype=BF16)
    want, state, mag = ref.conv(x, w, pool, slots, lens)
    got = kda.causal_conv(x, w, pool, idx(slots), ref.lengths_to_cu(lens, DEV) if cu else None, split=split)
    assert [tuple(t.shape) for t in got] == [(T, n) for n in split] and all(t.is_contiguous() for t in got)
    ref.within(torch.cat(got, 1), want, conv_bound(want, mag, 4, BF16, False))
    assert torch.equal(pool.double().cpu(), state)


def test_conv_keeps_requests_apart():
    """NaN in a request's rows, in its state, in padding rows and in unused slots stays there."""
    g = gen(4)
    lens, C = [20, 9, 40], 16
    x, w, pool = normal(g, 69, C), normal(g, C, 4), normal(g, 5, 3, C)
    clean, before = x.clone(), pool.clone()
    x[20:29] = float("nan")
    pool[4] = pool[1] = float("nan")
    y = kda.causal_conv(x, w, pool, idx([0, 1, 2]), ref.lengths_to_cu(lens, DEV))
    want = kda.causal_conv(clean, w, before, idx([0, -1, 2]), ref.lengths_to_cu(lens, DEV))
    assert torch.equal(y[:20], want[:20]) and torch.equal(y[29:], want[29:]) and bool(y[20:29].isnan().all())
    assert torch.equal(pool[[0, 2, 3]], before[[0, 2, 3]])
    y = kda.causal_conv(x, w, pool, idx([0, -1, 2]), ref.lengths_to_cu(lens, DEV))
    assert not bool(y[20:29].any()) and not bool(y.isnan().any())


# ---- selective recurrence -------------------------------------------------------------------------------

def ssm_inputs(seed, lens, H, P, N, G, dtype, dt_dtype=F32, strided=False, big_steps=False):
    g = gen(seed)
    T = sum(lens)
    rows = normal(g, T, H * P + 2 * G * N + 16 * strided, dtype=dtype)
    if not strided:
        rows = rows.contiguous()
    x, B, C = rows[:, :H * P].unflatten(1, (H, P)), rows[:, H * P:H * P + G * N].unflatten(1, (G, N)), rows[:, H * P + G * N:H * P + 2 * G * N].unflatten(1, (G, N))
    if not strided:
        x, B, C = x.contiguous(), B.contiguous(), C.contiguous()
    dt = normal(g, T, H + 3, dtype=dt_dtype)[:, :H] if strided else normal(g, T, H, dtype=dt_dtype)
    A_log = torch.log(1 + 15 * torch.rand(H, generator=g, device=DEV))
    dt_bias = normal(g, H, std=2.0) + (30 if big_steps else -3)
    return x, dt, B, C, A_log, dt_bias, normal(g, H)


# Bounds of the recurrence in fp32: a step adds at most 6 half steps to a state (decay's own error 3, the product,
# the sum, dt's share), a result's sum N + 2 half steps and dt x B's own error some 8, all of the sums of magnitudes.
# On the tensor-core form (bf16 inputs, dims of 64 or 128, up to 128 states) a state's increments are products of
# halves of 16 bits together, 2^-16, and the factors of a result are rounded to bf16 once, 2^-8, of the magnitudes; an
# exponent inside 32 tokens is the difference of two sums of up to 32 steps of at most 128 each: six additions of half
# a step of 4096, 6 * 2^-13, twice, 1.5e-3 or 1.0e-3 of a factor (times ln 2).

def on_tensor_cores(dtype, P, N):
    return dtype is BF16 and P in (64, 128) and N <= 128


def ssm_bounds(want, y_mag, mags, longest, N, out, tc):
    tau = (6 * longest + N + 16) * ref.F32
    b = (tau + (ref.half_step(BF16) + 2.0 ** -9.9 if tc else 0)) * y_mag
    return b + ref.half_step(out) * (want.abs() + b) + 1e-40, (tau + (2.0 ** -16 if tc else 0)) * mags + 1e-40


SSM_LENS = [[1], [50], [130, 1, 0, 64, 3], [16, 17, 15, 128, 129], [0, 5], [300]]


@pytest.mark.parametrize("lens", SSM_LENS, ids=str)
@pytest.mark.parametrize("H,P,N,G,dtype,out", [(4, 64, 128, 2, BF16, BF16), (3, 64, 128, 1, BF16, F32), (2, 128, 128, 1, BF16, BF16), (4, 64, 64, 4, BF16, F32),
                                               (2, 32, 16, 1, BF16, BF16), (3, 64, 128, 3, F32, F32), (2, 16, 32, 2, F32, F32), (2, 128, 64, 1, F32, BF16),
                                               (1, 64, 256, 1, BF16, F32), (5, 64, 64, 1, BF16, BF16), (2, 64, 256, 2, F32, F32),
                                                   (4, 64, 16, 2, BF16, BF16), (2, 128, 32, 2, BF16, F32)])
def test_ssm_rows(lens, H, P, N, G, dtype, out):
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(5, lens, H, P, N, G, dtype, strided=len(lens) > 1)
    slots = [2 * len(lens) - i for i in range(len(lens))]
    if len(lens) > 3:
        slots[1] = -1
    pool = normal(gen(6), 2 * len(lens) + 2, H, P, N)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, slots, lens, dt_bias, D)
    got = kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), pool, idx(slots), dt_bias=dt_bias, D=D, out_dtype=out)
    assert got.dtype is out
    yb, sb = ssm_bounds(want, y_mag, mags, max(lens), N, out, on_tensor_cores(dtype, P, N))
    ref.within(got, want, yb)
    ref.within(pool, state, sb)


@pytest.mark.parametrize("H,P,N,G,dtype,out", [(4, 64, 128, 2, BF16, BF16), (3, 128, 128, 3, F32, F32), (2, 32, 16, 1, BF16, F32), (2, 16, 32, 1, F32, BF16),
                                               (6, 64, 256, 2, BF16, BF16), (40, 64, 64, 8, BF16, BF16), (32, 128, 128, 1, BF16, BF16)])
@pytest.mark.parametrize("batch", [1, 7, 64])
def test_ssm_decode(H, P, N, G, dtype, out, batch):
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(7, [1] * batch, H, P, N, G, dtype, dt_dtype=BF16, strided=True)
    slots = [(i * 3 + 1) % (batch + 2) if (batch + 2) % 3 else i for i in range(batch)]
    if batch > 1:
        slots[batch // 2] = -1
    pool = normal(gen(8), batch + 2, H, P, N)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, slots, [1] * batch, dt_bias, D)
    got = kda.ssm_decode(x, dt, B, C, A_log, pool, idx(slots), dt_bias=dt_bias, D=D, out_dtype=out)
    yb, sb = ssm_bounds(want, y_mag, mags, 1, N, out, False)
    ref.within(got, want, yb)
    ref.within(pool, state, sb)


@pytest.mark.parametrize("lens", [[2300], [700, 3333, 0, 1, 2048, 4100]], ids=str)
@pytest.mark.parametrize("H,P,N,G,dtype", [(3, 64, 128, 1, BF16), (1, 128, 64, 1, BF16), (4, 64, 16, 2, BF16), (2, 64, 64, 1, F32), (3, 16, 16, 3, F32), (2, 32, 128, 1, BF16)])
def test_ssm_requests_in_segments(lens, H, P, N, G, dtype):
    """Long requests of few heads are cut into segments that start from chained states; the pool is updated in place."""
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(20, lens, H, P, N, G, dtype)
    A_log = A_log - 3                                       # states that last over thousands of tokens
    slots = [len(lens) - i for i in range(len(lens))]
    pool = normal(gen(21), len(lens) + 2, H, P, N)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, slots, lens, dt_bias, D)
    kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), pool.clone(), idx(slots), dt_bias=dt_bias, D=D)
    got = kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), pool, idx(slots), dt_bias=dt_bias, D=D)
    yb, sb = ssm_bounds(want, y_mag, mags, max(lens), N, dtype, on_tensor_cores(dtype, P, N))
    ref.within(got, want, yb)
    ref.within(pool, state, sb)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ssm_without_bias_and_skip_and_large_steps(dtype):
    """Steps so large that a state is forgotten within a token: decays of zero, no infinities."""
    lens, H, P, N, G = [140, 3], 2, 64, 128, 1
    x, dt, B, C, A_log, dt_bias, _ = ssm_inputs(9, lens, H, P, N, G, dtype, big_steps=True)
    pool = normal(gen(10), 3, H, P, N)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, [0, 2], lens, dt_bias)
    got = kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), pool, idx([0, 2]), dt_bias=dt_bias)
    yb, sb = ssm_bounds(want, y_mag, mags, max(lens), N, dtype, on_tensor_cores(dtype, P, N))
    ref.within(got, want, yb)
    ref.within(pool, state, sb)
    pool = normal(gen(10), 3, H, P, N)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, [0, 2], lens)
    got = kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), pool, idx([0, 2]))
    yb, sb = ssm_bounds(want, y_mag, mags, max(lens), N, dtype, on_tensor_cores(dtype, P, N))
    ref.within(got, want, yb)
    ref.within(pool, state, sb)


@pytest.mark.parametrize("dtype,P,N", [(BF16, 64, 128), (F32, 64, 64)])
def test_ssm_decode_continues_a_prompt(dtype, P, N):
    """A prompt in parts and its last tokens one at a time: within both forms' bounds of the 64-bit recurrence."""
    H, G, n, T = 4, 2, 2, 150
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(11, [T] * n, H, P, N, G, dtype)
    pool = torch.zeros(n, H, P, N, device=DEV)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, [0, 1], [T] * n, dt_bias, D)
    rows = [t.view(n, T, *t.shape[1:]) for t in (x, dt, B, C)]
    got = []
    for a, b in ((0, 100), (100, 133), (133, 146)):
        part = [t[:, a:b].flatten(0, 1).contiguous() for t in rows]
        got.append(kda.ssm_prefill(*part, A_log, ref.lengths_to_cu([b - a] * n, DEV), pool, idx([0, 1]), dt_bias=dt_bias, D=D).view(n, b - a, H, P))
    for t in range(146, T):
        got.append(kda.ssm_decode(*[r[:, t].contiguous() for r in rows], A_log, pool, idx([0, 1]), dt_bias=dt_bias, D=D)[:, None])
    yb, sb = ssm_bounds(want, y_mag, mags, T, N, dtype, on_tensor_cores(dtype, P, N))
    ref.within(torch.cat(got, 1).flatten(0, 1), want, yb)
    ref.within(pool, state, sb)


@pytest.mark.parametrize("dtype,P,N", [(BF16, 64, 128), (BF16, 128, 64), (F32, 32, 16)])
def test_ssm_keeps_requests_apart(dtype, P, N):
    """NaN in a request's rows, in its state and in unused slots reaches no other request."""
    H, G, lens = 2, 1, [20, 9, 140, 3]
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(12, lens, H, P, N, G, dtype)
    pool = normal(gen(13), 6, H, P, N)
    clean = [t.clone() for t in (x, dt, B, C)]
    before = pool.clone()
    cu = ref.lengths_to_cu(lens, DEV)
    for t in (x, dt, B, C):
        t[20:29] = float("nan")
    pool[4] = pool[1] = float("nan")
    y = kda.ssm_prefill(x, dt, B, C, A_log, cu, pool, idx([0, 1, 2, 5]), dt_bias=dt_bias, D=D)
    want = kda.ssm_prefill(*clean, A_log, cu, before, idx([0, -1, 2, 5]), dt_bias=dt_bias, D=D)
    assert torch.equal(y[:20], want[:20]) and torch.equal(y[29:], want[29:]) and not bool(want[20:29].any())
    assert torch.equal(pool[[0, 2, 3, 5]], before[[0, 2, 3, 5]])


# ---- group norm -----------------------------------------------------------------------------------------

def norm_bound(want, seen, center, w, b, mag, out, eps, gate_first):
    """`seen`: what is normalised, in 64 bits; `mag`: the gate behind the norm.  In units of the root mean square, a
    centered value is off by some (log2 n + 8) half steps of the group's largest, and the root by as many of itself; a gate
    before the norm adds a sigmoid's share to both, one behind it or an activation (of slope 1.1 at most) to the result."""
    m = seen.mean(-1, keepdim=True) if center else 0
    rms = torch.sqrt((seen - m).square().mean(-1, keepdim=True) + eps)
    share = 2 * (seen.shape[-1].bit_length() + 8) * ref.F32 + (2 * SIGMOID if gate_first else 0)
    e = share * (seen.abs().amax(-1, keepdim=True) / rms) * (1 if w is None else w.double().cpu().abs())
    e = e + (0 if b is None else 2 * ref.F32 * b.double().cpu().abs())
    e = 1.1 * e * mag + SIGMOID * want.abs()
    return e + ref.half_step(out) * (want.abs() + e) + 1e-40


NORMS = [dict(), dict(w=1, b=1, activation="silu"), dict(w=1, center=False, gate=1, activation="sigmoid"), dict(gate=1, b=1),
         dict(w=1, gate=1, activation="silu", gate_first=True, center=False, eps=1e-6), dict(activation="sigmoid", center=False)]


@pytest.mark.parametrize("T,G,n", [(1, 1, 1), (5, 3, 7), (33, 2, 33), (64, 4, 64), (17, 8, 128), (3, 1, 256), (9, 5, 333), (4, 2, 512),
                                   (3, 1, 4096), (2, 3, 5000), (2, 1, 16384), (1, 2, 16383)])
@pytest.mark.parametrize("io,out", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
def test_norm(T, G, n, io, out):
    g = gen(14 + n)
    x = (normal(g, T, G * n + 8, dtype=io) + 0.5)[:, :G * n].unflatten(1, (G, n))
    weight, shift = normal(g, G, n), normal(g, G, n)
    gates = normal(g, T, G * n + 16, dtype=out)[:, 16:].unflatten(1, (G, n))
    for case in NORMS:
        kw = dict(case)
        w, b = weight if kw.pop("w", 0) else None, shift if kw.pop("b", 0) else None
        gate = gates if kw.pop("gate", 0) else None
        want = ref.norm(x, w, b, gate=gate, **kw)
        got = kda.group_norm(x, w, b, gate=gate, out_dtype=out, **kw)
        assert got.dtype is out
        z = 1.0 if gate is None else ref.act(gate.double().cpu(), kw.get("activation"))
        first = kw.get("gate_first", False)
        seen = x.double().cpu() * (z if first else 1)
        mag = 1.0 if gate is None or first else z.abs()
        ref.within(got, want, norm_bound(want, seen, kw.get("center", True), w, b, mag, out, kw.get("eps", 1e-5), first))


def test_norm_keeps_rows_apart():
    g = gen(15)
    x, gate = normal(g, 9, 3, 128, dtype=BF16), normal(g, 9, 3, 128, dtype=BF16)
    want = kda.group_norm(x, gate=gate, activation="silu")
    x[4, 1, 5] = float("nan")
    gate[7, 2, 0] = float("inf")
    got = kda.group_norm(x, gate=gate, activation="silu")
    same = torch.ones(9, 3, dtype=torch.bool, device=DEV)
    same[4, 1] = same[7, 2] = False
    assert torch.equal(got[same], want[same]) and bool(got[4, 1].isnan().all()) and torch.equal(got[7, 2, 1:], want[7, 2, 1:])


# ---- all together ---------------------------------------------------------------------------------------

def layer(proj, p, slots, cu, new_conv, new_state):
    """Convolution, recurrence and gated norm of one layer as a model calls them, from one fused projection row."""
    H, P, G, N = 4, 64, 2, 128
    z, xbc, dt = proj.split([H * P, H * P + 2 * G * N, H], 1)
    x, B, C = kda.causal_conv(xbc, p["w"], new_conv, slots, cu, activation="silu", split=(H * P, G * N, G * N))
    x, B, C = x.unflatten(1, (H, P)), B.unflatten(1, (G, N)), C.unflatten(1, (G, N))
    if cu is None:
        y = kda.ssm_decode(x, dt, B, C, p["A_log"], new_state, slots, dt_bias=p["dt_bias"], D=p["D"])
    else:
        y = kda.ssm_prefill(x, dt, B, C, p["A_log"], cu, new_state, slots, dt_bias=p["dt_bias"], D=p["D"])
    return kda.group_norm(y.view(-1, G, H * P // G), p["g"], gate=z.unflatten(1, (G, H * P // G)), activation="silu", gate_first=True, center=False), y, (x, B, C, dt)


def layer_weights(g):
    H, P, G, N = 4, 64, 2, 128
    return dict(w=normal(g, H * P + 2 * G * N, 4, std=0.5), A_log=torch.rand(H, generator=g, device=DEV), dt_bias=normal(g, H) - 3, D=normal(g, H),
                g=normal(g, G, H * P // G))


def test_a_layer_decoded_as_prefilled():
    """The three together: prompts and then single tokens.  Each operator's result against its 64-bit form on the inputs
    that the operator before it gave."""
    g = gen(16)
    H, P, G, N, n, T = 4, 64, 2, 128, 3, 45
    p = layer_weights(g)
    proj = normal(g, n, T, 2 * H * P + 2 * G * N + H, dtype=BF16)
    conv_pool, state_pool = torch.zeros(n, 3, H * P + 2 * G * N, dtype=BF16, device=DEV), torch.zeros(n, H, P, N, device=DEV)
    slots = idx([2, 0, 1])
    calls = [layer(proj[:, :40].flatten(0, 1), p, slots, ref.lengths_to_cu([40] * n, DEV), conv_pool, state_pool)]
    calls[0] = [t.unflatten(0, (n, 40)) for t in (*calls[0][:2], *calls[0][2])]
    for t in range(40, T):
        o, y, ins = layer(proj[:, t], p, slots, None, conv_pool, state_pool)
        calls.append([v[:, None] for v in (o, y, *ins)])
    o, y, x, B, C, dt = (torch.cat([c[i] for c in calls], 1).flatten(0, 1) for i in range(6))
    xbc = proj[..., H * P:2 * H * P + 2 * G * N].flatten(0, 1)
    zero = torch.zeros_like(conv_pool)
    want, _, mag = ref.conv(xbc, p["w"], zero, [2, 0, 1], [T] * n, silu=True)
    ref.within(torch.cat([x.flatten(1), B.flatten(1), C.flatten(1)], 1), want, conv_bound(want, mag, 4, BF16, True))
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, p["A_log"], torch.zeros_like(state_pool), [2, 0, 1], [T] * n, p["dt_bias"], p["D"])
    yb, sb = ssm_bounds(want, y_mag, mags, T, N, BF16, True)
    ref.within(y, want, yb)
    ref.within(state_pool, state, sb)
    z = proj[..., :H * P].flatten(0, 1).unflatten(1, (G, -1))
    want = ref.norm(y.reshape(n * T, G, -1), p["g"], gate=z, activation="silu", gate_first=True, center=False)
    seen = y.reshape(n * T, G, -1).double().cpu() * ref.act(z.double().cpu(), "silu")
    ref.within(o, want, norm_bound(want, seen, False, p["g"], None, 1.0, BF16, 1e-5, True))


def test_captured_layer_and_other_stream():
    """A decode step and a prompt captured into a graph and replayed, and a call on another stream: the bits of plain calls."""
    g = gen(17)
    H, P, G, N = 4, 64, 2, 128
    p = layer_weights(g)
    for cu, T, n in ((None, 5, 5), (ref.lengths_to_cu([200, 1, 30], DEV), 231, 3)):
        proj = normal(g, T, 2 * H * P + 2 * G * N + H, dtype=BF16)
        pools = [normal(g, n, 3, H * P + 2 * G * N, dtype=BF16), normal(g, n, H, P, N)]
        slots = idx(list(range(n)))

        def fresh():
            return [t.clone() for t in pools]

        a = fresh()
        want = layer(proj, p, slots, cu, *a)[0]
        b = fresh()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = layer(proj, p, slots, cu, *b)[0]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want) and all(torch.equal(u, v) for u, v in zip(a, b))
        c = fresh()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = layer(proj, p, slots, cu, *c)[0]
        for t, u in zip(c, pools):
            t.copy_(u)
        graph.replay()
        assert torch.equal(got, want) and all(torch.equal(u, v) for u, v in zip(a, c))
        for t, u in zip(c, pools):
            t.copy_(u)
        graph.replay()
        assert torch.equal(got, want) and all(torch.equal(u, v) for u, v in zip(a, c))


def test_places_past_32_bits():
    """States, rows and outputs whose offsets pass 2^31 elements."""
    g = gen(22)
    H, P, N, G = 16, 64, 128, 1
    slots = 16500                                            # 2^31.01 states
    pool = torch.empty(slots, H, P, N, device=DEV)
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(23, [140, 3], H, P, N, G, BF16)
    for s in (0, slots - 1):
        pool[s] = normal(gen(s), H, P, N)
    small = torch.stack([pool[0], pool[-1]])
    cu = ref.lengths_to_cu([140, 3], DEV)
    want = kda.ssm_prefill(x, dt, B, C, A_log, cu, small, idx([0, 1]), dt_bias=dt_bias, D=D)
    got = kda.ssm_prefill(x, dt, B, C, A_log, cu, pool, idx([0, slots - 1]), dt_bias=dt_bias, D=D)
    assert torch.equal(got, want) and torch.equal(pool[0], small[0]) and torch.equal(pool[-1], small[1])
    want = kda.ssm_decode(x[:2], dt[:2], B[:2], C[:2], A_log, small, idx([1, 0]), dt_bias=dt_bias, D=D)
    got = kda.ssm_decode(x[:2], dt[:2], B[:2], C[:2], A_log, pool, idx([slots - 1, 0]), dt_bias=dt_bias, D=D)
    assert torch.equal(got, want) and torch.equal(pool[0], small[0]) and torch.equal(pool[-1], small[1])
    del pool
    T, C_, wide = 70000, 64, 32768                           # 2^31.1 elements of rows
    rows = torch.empty(T, wide, dtype=BF16, device=DEV)
    rows[:, :C_] = normal(g, T, C_, dtype=BF16)
    w, state = normal(g, C_, 4), torch.zeros(2, 3, C_, dtype=BF16, device=DEV)
    cu = ref.lengths_to_cu([69000, 1000], DEV)
    want = kda.causal_conv(rows[:, :C_].contiguous(), w, state.clone(), idx([0, 1]), cu)
    assert torch.equal(kda.causal_conv(rows[:, :C_], w, state, idx([0, 1]), cu), want)
    x = rows[:, :C_].unflatten(1, (2, 32))
    assert torch.equal(kda.group_norm(x), kda.group_norm(x.contiguous()))
    rows[-3:] = normal(g, 3, wide, dtype=BF16)
    y = kda.group_norm(rows.view(T, 64, 512)[-3:])
    assert torch.equal(kda.group_norm(rows.view(T, 64, 512), out=rows.view(T, 64, 512).clone())[-3:], y)


@pytest.mark.parametrize("lens", [[5, 400, 0, 32, 33, 1, 2, 3, 4, 5, 6, 7], [1] * 30 + [300], [32] * 6], ids=str)
def test_ssm_short_requests_beside_long_ones(lens):
    """Requests of few tokens go token by token, the others of the same call in chunks; rows of no request get zeros."""
    H, P, N, G = 2, 64, 128, 1
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(24, lens + [9], H, P, N, G, BF16)
    slots = list(range(len(lens)))
    slots[1], slots[3] = -1, -1
    pool = normal(gen(25), len(lens), H, P, N)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, slots + [-1], lens + [9], dt_bias, D)
    got = kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), pool, idx(slots), dt_bias=dt_bias, D=D)
    assert kda.check_device_errors() == 2                      # nine rows behind the last request
    yb, sb = ssm_bounds(want, y_mag, mags, max(lens), N, BF16, True)
    ref.within(got, want, yb)
    ref.within(pool, state, sb)


def test_ssm_many_requests():
    """More requests than the planning CTA has threads, in no order of length."""
    H, P, N, G = 1, 64, 64, 1
    lens = [50 + (37 * i) % 61 for i in range(1100)]            # 80 on average: all in chunks
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(30, lens, H, P, N, G, BF16)
    slots = [(7 * i + 3) % 1103 for i in range(1100)]
    pool = normal(gen(31), 1103, H, P, N)
    want, state, y_mag, mags = ref.ssm(x, dt, B, C, A_log, pool, slots, lens, dt_bias, D)
    got = kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), pool, idx(slots), dt_bias=dt_bias, D=D)
    yb, sb = ssm_bounds(want, y_mag, mags, max(lens), N, BF16, True)
    ref.within(got, want, yb)
    ref.within(pool, state, sb)


@pytest.mark.parametrize("lens", [[5000, 40, 3000], [9, 31, 140, 2]], ids=str)
def test_ssm_same_call_same_bits(lens):
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(32, lens, 2, 64, 128, 1, BF16)
    pool = normal(gen(33), len(lens), 2, 64, 128)
    first = None
    for _ in range(10):
        p = pool.clone()
        y = kda.ssm_prefill(x, dt, B, C, A_log, ref.lengths_to_cu(lens, DEV), p, idx(list(range(len(lens)))), dt_bias=dt_bias, D=D)
        first = first or (y, p)
        assert torch.equal(y, first[0]) and torch.equal(p, first[1])


def test_overlapping_requests_are_recorded():
    """A table whose requests share rows has more segments and states than the workspace holds: recorded, nothing written
    outside the outputs and slots."""
    g = gen(34)
    T, n, H, P, N = 6000, 20, 1, 64, 128
    x, dt, B, C, A_log, dt_bias, D = ssm_inputs(35, [T], H, P, N, 1, BF16)
    cu = torch.tensor([0, T] * (n // 2) + [T], dtype=torch.int32, device=DEV)
    need = kda.ssm_prefill_workspace_size(H, P, N, 1, n, T)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    pool = normal(g, n + 1, H, P, N)
    before = pool.clone()
    kda.ssm_prefill(x, dt, B, C, A_log, cu, pool, idx(list(range(n))), dt_bias=dt_bias, D=D, workspace=ws[:need])
    assert kda.check_device_errors() == 2
    assert bool((ws[need:] == 77).all()) and torch.equal(pool[n], before[n])


def test_calls_on_two_streams_at_once():
    """Two layers' prompts side by side, each with its own workspace and states."""
    lens, H, P, N, G = [700, 90], 4, 64, 128, 1
    ins = [ssm_inputs(26 + i, lens, H, P, N, G, BF16) for i in range(2)]
    cu = ref.lengths_to_cu(lens, DEV)
    pools = [normal(gen(28 + i), 2, H, P, N) for i in range(2)]
    alone = []
    for v, p in zip(ins, pools):
        q = p.clone()
        alone.append((kda.ssm_prefill(*v[:5], cu, q, idx([0, 1]), dt_bias=v[5], D=v[6]), q))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for v, p, s in zip(ins, pools, streams):
            with torch.cuda.stream(s):
                q = p.clone()
                got.append((kda.ssm_prefill(*v[:5], cu, q, idx([0, 1]), dt_bias=v[5], D=v[6]), q))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(got, alone) for a, b in zip(x, y))


def test_bad_tables_are_recorded():
    """Slots past the pool, rows of no request and lengths past the tokens: zeros and a code, no access out of range."""
    g = gen(18)
    H, P, G, N, C = 2, 64, 1, 128, 24
    x, dt, B, Cc, A_log, dt_bias, D = ssm_inputs(19, [30], H, P, N, G, BF16)
    xc, w = normal(g, 30, C), normal(g, C, 4)
    for cu, slots, code, zero in (([0, 10, 30], [0, 9], 1, slice(10, 30)), ([4, 10, 30], [0, 1], 2, slice(0, 4)), ([0, 10, 25], [0, 1], 2, slice(25, 30)),
                                  ([0, 10, 77], [0, 1], 2, slice(10, 30)), ([-5, 10, 30], [0, 1], 2, slice(0, 10))):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        pool, state = torch.zeros(3, 3, C, device=DEV), torch.zeros(3, H, P, N, device=DEV)
        y = kda.causal_conv(xc, w, pool, idx(slots), cu)
        assert kda.check_device_errors() == code and not bool(y[zero].any()) and bool((y.isfinite()).all())
        y = kda.ssm_prefill(x, dt, B, Cc, A_log, cu, state, idx(slots), out=torch.full((30, H, P), 7.0, dtype=BF16, device=DEV))
        assert kda.check_device_errors() == code and not bool(state[2].any())
        if code == 1 or cu.tolist() in ([4, 10, 30], [0, 10, 25]):
            assert not bool(y[zero].any())
    y = kda.causal_conv(xc[:2].contiguous(), w, pool, idx([0, 3]))
    assert kda.check_device_errors() == 1 and not bool(y[1].any())
    y = kda.ssm_decode(x[:2], dt[:2], B[:2], Cc[:2], A_log, state, idx([5, 0]))
    assert kda.check_device_errors() == 1 and not bool(y[0].any())
