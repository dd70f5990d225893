"""Paged cache and attention on the GPU against plain 64-bit forms (tests/kv_reference.py)."""
import math

import pytest
import torch

import kda_gated_delta_gb300 as kda
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


def _bf(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def _filled_cache(batch, Hkv, D, dtype, seed, poison=True):
    """A cache whose tokens are random; with `poison`, every slot that holds none is NaN (4 bits: scale
    NaN).  Returns it on the device and k_of for the reference."""
    g = torch.Generator().manual_seed(seed)
    shape = (batch.num_pages, Hkv, batch.page)
    used = torch.zeros(batch.num_pages, batch.page, dtype=torch.bool)
    for i, n in enumerate(batch.lens.tolist()):
        for j in range(max(0, n)):
            page, row = batch.place(i, j)
            if page >= 0:
                used[page, row] = True
    hole = ~used[:, None, :, None].expand(*shape, 1)
    if dtype == "bf16":
        k, v = _bf(g, *shape, D), _bf(g, *shape, D)
        k64, v64 = k.double(), v.double()
        if poison:
            k, v = k.masked_fill(hole, NAN), v.masked_fill(hole, NAN)
        cache = kda.KVCache(k.to(DEV), v.to(DEV))
    else:
        parts, dense = [], []
        for _ in range(2):
            code = torch.randint(0, 16, (*shape, D), generator=g)
            s = ref.e4m3(torch.rand(*shape, D // 16, generator=g).double() * 0.5 + 0.01)
            dense.append(ref.dequantise(code, s))
            s8 = s.float().to(torch.float8_e4m3fn).view(torch.uint8)
            if poison:
                s8 = s8.masked_fill(hole, 0x7f)
            parts.append(((code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8).to(DEV), s8.to(DEV).view(torch.float8_e4m3fn)))
        (k64, v64) = dense
        cache = kda.KVCache(parts[0][0], parts[1][0], parts[0][1], parts[1][1])

    def k_of(i, positions):
        page = batch.table[i].long()[positions // batch.page]
        return k64[page, :, positions % batch.page], v64[page, :, positions % batch.page]

    return cache, k_of


def _attend(batch, Hq, Hkv, D, dtype, window=0, sinks=0, scale=None, seed=0, decode=False, q_pad=0, tight=True, q_std=2.0):
    g = torch.Generator().manual_seed(seed + 1)
    cache, k_of = _filled_cache(batch, Hkv, D, dtype, seed + 2)
    q = _bf(g, batch.T, Hq, D, std=q_std)
    table, lens, cu = batch.on(DEV)
    wide = torch.full((batch.T, Hq * D + q_pad), NAN, dtype=torch.bfloat16, device=DEV)
    qd = wide[:, :Hq * D].unflatten(1, (Hq, D))
    qd.copy_(q)
    kw = dict(max_len=max(1, int(batch.lens.max()))) if tight else {}
    out, lse = kda.paged_attention(qd, cache, table, lens, None if decode else cu, window=window, sinks=sinks, scale=scale,
                                   max_new=max(1, max(batch.new)) if tight else None, return_lse=True, **kw)
    torch.cuda.synchronize()
    assert kda.check_device_errors() == 0
    o, l, mag, big = ref.attention(q, k_of, batch, window, sinks, D ** -0.5 if scale is None else scale)
    tol_o, tol_l = ref.bounds(o, l, mag, big)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(out).all()
    err = (out - o).abs()
    assert (err <= tol_o).all(), float((err / tol_o).max())
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all() and (out[empty] == 0).all()
    assert ((lse - l).abs()[~empty] <= tol_l[~empty]).all(), float(((lse - l).abs() / tol_l)[~empty].max())
    return out


BOTH = pytest.mark.parametrize("dtype", ["bf16", "fp4"])


@BOTH
@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 8, 2, 64), (64, 6, 2, 16), (128, 5, 5, 128), (128, 16, 1, 32), (64, 7, 1, 64),
                                           (128, 20, 1, 16), (64, 24, 1, 32)])
def test_decode(dtype, D, Hq, Hkv, page):
    b = ref.Batch([1] * 6, [0, 1, 62, 63, 64, 400], page, seed=D + Hq)
    _attend(b, Hq, Hkv, D, dtype, decode=True)


@BOTH
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 0), (64, 4), (100, 130), (128, 0), (5000, 3)])
def test_decode_window(dtype, window, sinks):
    b = ref.Batch([1] * 5, [0, 15, 127, 300, 701], 16, seed=window, drop=(window, sinks))
    _attend(b, 8, 2, 128, dtype, window=window, sinks=sinks, decode=True)


@BOTH
def test_decode_long_is_split(dtype):
    b = ref.Batch([1, 1], [9000, 20000], 64, seed=3)
    _attend(b, 4, 1, 128, dtype, decode=True)
    _attend(b, 4, 1, 128, dtype, decode=True, tight=False)
    _attend(b, 4, 1, 128, dtype, decode=True, window=6000, sinks=300)


@BOTH
@pytest.mark.parametrize("past,D,window,sinks", [([3000, 100, -1], 128, 0, 0), ([900], 128, 0, 0), ([1700, 40, 650], 64, 0, 0), ([5000, 2049], 128, 1500, 70)])
def test_few_requests_join_in_clusters(dtype, past, D, window, sinks):
    """A few requests of some thousand tokens: up to eight parts, some of them empty, joined on the chip."""
    b = ref.Batch([1] * len(past), past, 32, seed=len(past), drop=(window, sinks))
    _attend(b, 8, 2, D, dtype, window=window, sinks=sinks, decode=True)
    if min(past) > 4:
        b = ref.Batch([3] * len(past), past, 32, seed=len(past), drop=(window, sinks))
        _attend(b, 10, 2, D, dtype, window=window, sinks=sinks)


@BOTH
@pytest.mark.parametrize("new,G,D", [(2, 4, 128), (4, 4, 128), (3, 5, 64), (16, 1, 128), (16, 8, 64), (9, 16, 128)])
def test_verify(dtype, new, G, D):
    b = ref.Batch([new] * 4, [0, 13, 130, 511], 32, seed=new)
    _attend(b, 2 * G, 2, D, dtype)


@BOTH
def test_verify_long_is_split(dtype):
    b = ref.Batch([4, 4], [5000, 9001], 64, seed=5)
    _attend(b, 8, 1, 128, dtype)
    _attend(b, 8, 1, 128, dtype, window=3000, sinks=70)


@BOTH
@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 4, 1, 64), (64, 4, 2, 16), (128, 3, 1, 128), (128, 1, 1, 32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 0), (130, 5), (1, 2)])
def test_prompts(dtype, D, Hq, Hkv, page, window, sinks):
    b = ref.Batch([1, 130, 257, 64, 0, 300], [0, 5, 0, 131, 40, 100], page, seed=D + page, drop=(window, sinks))
    _attend(b, Hq, Hkv, D, dtype, window=window, sinks=sinks)


@BOTH
def test_mixed_lengths_and_padding(dtype):
    """Padding rows (kv_lens <= 0), requests without new tokens, tokens before position 0, loose bounds."""
    b = ref.Batch([1, 5, 0, 40, 3, 2], [9, 0, 10, 70, -3, -1], 16, seed=9)
    assert b.lens.tolist() == [10, 5, 10, 110, 0, 1]
    _attend(b, 8, 2, 128, dtype)
    _attend(b, 8, 2, 128, dtype, tight=False)
    d = ref.Batch([1, 1, 1], [-1, 30, -6], 16, seed=10)
    _attend(d, 8, 2, 128, dtype, decode=True)


@BOTH
def test_strided_queries_and_scales(dtype):
    b = ref.Batch([3, 50], [20, 31], 16, seed=11)
    _attend(b, 4, 2, 64, dtype, q_pad=264, scale=0.3)
    _attend(b, 4, 2, 64, dtype, q_pad=8, scale=1.0, q_std=8.0)      # near one-hot weights


@BOTH
def test_large_and_small_queries(dtype):
    """Query magnitudes far from 1, in 16-bit formats' corners: the scores keep their fp32 accuracy."""
    b = ref.Batch([1, 20], [100, 100], 32, seed=12)
    _attend(b, 4, 2, 128, dtype, q_std=3e5, scale=1e-6)
    _attend(b, 4, 2, 128, dtype, q_std=1e-7, scale=1e6)
    _attend(b, 4, 2, 128, dtype, q_std=0.0)


def test_non_finite_keys_and_values_that_are_visible():
    """NaN in a visible key reaches exactly the queries that see it."""
    b = ref.Batch([1, 1], [40, 40], 16, seed=13)
    cache, _ = _filled_cache(b, 1, 128, "bf16", 1, poison=False)
    page, row = b.place(0, 7)
    cache.k[page, 0, row] = NAN
    table, lens, _ = b.on(DEV)
    q = _bf(torch.Generator().manual_seed(1), 2, 4, 128).to(DEV)
    out = kda.paged_attention(q, cache, table, lens)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


@BOTH
def test_repeated_calls_and_streams_give_the_same_bits(dtype):
    b = ref.Batch([4, 300, 1], [6000, 100, 20], 64, seed=14)
    cache, _ = _filled_cache(b, 2, 128, dtype, 3)
    table, lens, cu = b.on(DEV)
    q = _bf(torch.Generator().manual_seed(2), b.T, 8, 128).to(DEV)
    kw = dict(max_new=300, max_len=6004, return_lse=True)
    first = kda.paged_attention(q, cache, table, lens, cu, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = kda.paged_attention(q, cache, table, lens, cu, stream=side, **kw)
        side.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@BOTH
def test_step_in_a_graph(dtype):
    """Append and attend captured once and replayed with the lengths advanced on the device."""
    B, Hq, Hkv, D, page = 3, 8, 2, 128, 16
    g = torch.Generator().manual_seed(5)
    cache = kda.kv_cache(B * 8, Hkv, page, D, dtype, DEV)
    table = torch.randperm(B * 8, generator=g).to(torch.int32).view(B, 8).to(DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    rope = kda.rope_table(128, D, device=DEV)
    q, k, v = (_bf(g, B, h, D).to(DEV) for h in (Hq, Hkv, Hkv))
    qo, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(max(1, kda.attention_workspace_size(Hq, Hkv, D, page, B, B, 1, 128, dtype=dtype)), dtype=torch.uint8, device=DEV)

    def step():
        lens.add_(1)
        kda.kv_append(k, v, cache, table, lens, q=q, q_out=qo, rope=rope)
        kda.paged_attention(qo, cache, table, lens, max_len=128, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    got = []
    for i in range(20):
        for x in (q, k, v):
            x.copy_(_bf(g, *x.shape))
        graph.replay()
        got.append((out.clone(), q.clone()))
    assert lens.tolist() == [21] * B and kda.check_device_errors() == 0
    b = ref.Batch([1] * B, [20] * B, page)
    b.table = table.cpu()
    cu = torch.arange(0, 21 * B + 1, 21, dtype=torch.int32, device=DEV)
    kk, vv = kda.kv_read(cache, table, lens, cu, num_tokens=21 * B)
    kk, vv = kk.cpu().double(), vv.cpu().double()
    last = kda.kv_append(k, v, cache, table, lens, q=q, rope=rope).cpu()
    o, l, mag, big = ref.attention(last, lambda i, p: (kk[21 * i + p], vv[21 * i + p]), b, 0, 0, D ** -0.5)
    assert ((got[-1][0].cpu().double() - o).abs() <= ref.bounds(o, l, mag, big)[0]).all()


@BOTH
@pytest.mark.parametrize("new,past", [([1, 1], [9000, 20000]), ([1] * 40, [2000] * 40), ([1], [3000]), ([40, 3], [6000, 100]), ([300], [200])])
def test_every_form_in_a_graph(dtype, new, past):
    """Calls that are cut along the cache (joined by a kernel of their own or in a cluster) and prompts, captured:
    a replay gives the bits of the plain call, also after the inputs changed in place."""
    b = ref.Batch(new, past, 64, seed=21)
    cache, _ = _filled_cache(b, 1, 128, dtype, 4)
    table, lens, cu = b.on(DEV)
    g = torch.Generator().manual_seed(6)
    q = _bf(g, b.T, 4, 128).to(DEV)
    kw = dict(max_new=max(new), max_len=int(b.lens.max()), return_lse=True)
    kda.paged_attention(q, cache, table, lens, cu, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = kda.paged_attention(q, cache, table, lens, cu, **kw)
    for _ in range(2):
        q.copy_(_bf(g, *q.shape))
        graph.replay()
        want = kda.paged_attention(q, cache, table, lens, cu, **kw)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@BOTH
def test_limits_of_window_and_sinks(dtype):
    """The largest values mean: everything."""
    for new, past in (([1, 1], [100, 700]), ([40, 3], [100, 700])):
        b = ref.Batch(new, past, 16, seed=22)
        full = _attend(b, 8, 2, 128, dtype)
        for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
            assert torch.equal(_attend(b, 8, 2, 128, dtype, window=window, sinks=sinks), full)


@BOTH
def test_small_scales(dtype):
    """Factors of the scores that underflow: the weights are uniform over what is visible, masked tokens stay out."""
    b = ref.Batch([1, 40], [100, 100], 32, seed=33)
    _attend(b, 8, 2, 128, dtype, q_std=0.0, scale=1e-9)
    _attend(b, 8, 2, 128, dtype, q_std=1e-30, scale=1e-20)
    _attend(b, 8, 2, 128, dtype, window=30, sinks=2, scale=1e-30)


@BOTH
@pytest.mark.parametrize("new,past", [([2, 1], [3000, 20]), ([300, 40], [100, 9000]), ([5, 3, 4], [9, 40, 0])])
def test_bounds_that_bound_nothing(dtype, new, past):
    """Numbers whose product with the heads of a group passes 32 bits, and every other from all tokens up."""
    b = ref.Batch(new, past, 32, seed=30)
    cache, _ = _filled_cache(b, 2, 128, dtype, 5)
    table, lens, cu = b.on(DEV)
    q = _bf(torch.Generator().manual_seed(7), b.T, 8, 128).to(DEV)
    want = _attend(b, 8, 2, 128, dtype, tight=False)           # by default all tokens
    assert torch.isfinite(want).all()
    first = kda.paged_attention(q, cache, table, lens, cu, max_new=b.T, return_lse=True)
    for bound in (b.T + 1, 2 ** 29, 2 ** 30, 2 ** 31 - 1):
        out, lse = torch.full_like(q, NAN), torch.full((b.T, 8), NAN, device=DEV)
        kda.paged_attention(q, cache, table, lens, cu, max_new=bound, out=out, lse=lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert kda.check_device_errors() == 0


# ---- append and read ------------------------------------------------------------------------------------

def _append_case(new, past, Hq, Hkv, D, page, dtype, rot, interleaved, seed=0, pad=0, with_positions=False, scale=None, decode=False):
    g = torch.Generator().manual_seed(seed)
    b = ref.Batch(new, past, page, seed=seed)
    rope = kda.rope_table(4000, rot, device=DEV) if rot else None
    table, lens, cu = b.on(DEV)
    q, k, v = _bf(g, b.T, Hq, D), _bf(g, b.T, Hkv, D), _bf(g, b.T, Hkv, D)
    if scale is not None:
        k, v = k * scale, v * scale
    fused = torch.full((b.T, (Hq + 2 * Hkv) * D + pad), NAN, dtype=torch.bfloat16, device=DEV)
    cut = [0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D]
    qd, kd, vd = (fused[:, cut[i]:cut[i + 1]].unflatten(1, (-1, D)) for i in range(3))
    qd.copy_(q), kd.copy_(k), vd.copy_(v)
    positions = torch.randint(0, 4000, (b.T,), generator=g, dtype=torch.int32) if with_positions else None
    cache = kda.kv_cache(b.num_pages, Hkv, page, D, dtype, DEV)
    for t in cache:
        if t is not None:
            t.view(torch.uint8).fill_(0x55)
    qo = kda.kv_append(kd, vd, cache, table, lens, None if decode else cu, q=qd, rope=rope, interleaved=interleaved,
                       positions=None if positions is None else positions.to(DEV))
    assert kda.check_device_errors() == 0
    where = []                                               # (token, page, row, position)
    for i in range(len(new)):
        for r in range(new[i]):
            pos = int(b.lens[i]) - new[i] + r
            t = int(b.cu[i]) + r
            where.append((t, *b.place(i, pos), pos) if pos >= 0 and b.lens[i] > 0 else (t, -1, 0, -1))

    def turned(x, t, pos):
        if not rot:
            return x[t].double()
        return ref.rotate(x[t], pos if positions is None else int(positions[t]), rope.cpu(), interleaved)

    return b, cache, qo.cpu(), q, k, v, where, turned, (table, lens, None if decode else cu)


SHAPES = [(8, 2, 128, 64, 128, False), (6, 3, 64, 16, 32, False), (4, 4, 128, 128, 64, True), (1, 1, 64, 32, 64, True), (5, 1, 128, 16, 0, False),
          (32, 8, 128, 64, 96, False)]


@pytest.mark.parametrize("Hq,Hkv,D,page,rot,interleaved", SHAPES)
@pytest.mark.parametrize("with_positions", [False, True])
def test_append_bf16(Hq, Hkv, D, page, rot, interleaved, with_positions):
    if with_positions and not rot:
        pytest.skip("nothing to rotate")
    b, cache, qo, q, k, v, where, turned, _ = _append_case([1, 70, 0, 3, 2], [0, 10, 4, 63, -1], Hq, Hkv, D, page, "bf16", rot,
                                                           interleaved, pad=8, with_positions=with_positions)
    kc, vc = cache.k.cpu(), cache.v.cpu()
    touched = torch.zeros(b.num_pages, page, dtype=torch.bool)
    for t, pg, row, pos in where:
        if pos < 0:
            assert (qo[t] == 0).all()
            continue
        touched[pg, row] = True
        for got, x in ((qo[t], q), (kc[pg, :, row], k)):
            want = turned(x, t, pos)
            # one rounding to bf16 of a sum that fp32 rounds once
            assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -14) + 2.0 ** -23 * x[t].double().abs().max()).all()
        assert torch.equal(vc[pg, :, row], v[t])
    for c in (kc, vc):                                       # nothing else was written
        rest = c.view(torch.int16).permute(0, 2, 1, 3)[~touched]
        assert (rest == 0x5555).all()


@pytest.mark.parametrize("Hq,Hkv,D,page,rot,interleaved", SHAPES)
@pytest.mark.parametrize("scale", [None, 0.0, 1e-4, 2e5])
def test_append_fp4(Hq, Hkv, D, page, rot, interleaved, scale):
    """Codes and scales equal the definition, from the same keys that a bf16 cache gets."""
    args = ([1, 70, 0, 3, 2], [0, 10, 4, 63, -1], Hq, Hkv, D, page)
    b, cache, qo, q, k, v, where, turned, tables = _append_case(*args, "fp4", rot, interleaved, pad=8, scale=scale)
    _, full, qo2, *_ = _append_case(*args, "bf16", rot, interleaved, pad=8, scale=scale)
    assert torch.equal(qo, qo2)
    kd, vd = kda.kv_read(cache, *tables, num_tokens=b.T)
    for side, (c, s, dense, out) in enumerate(((cache.k, cache.k_scale, full.k, kd), (cache.v, cache.v_scale, full.v, vd))):
        c, s, dense, out = c.cpu(), s.cpu(), dense.cpu(), out.cpu()
        touched = torch.zeros(b.num_pages, page, dtype=torch.bool)
        for t, pg, row, pos in where:
            if pos < 0:
                assert (out[t] == 0).all()
                continue
            touched[pg, row] = True
            code, scales = ref.quantise(dense[pg, :, row])
            got_s = s[pg, :, row].float().double()
            assert torch.equal(got_s, scales), (side, t)
            got = ref.unpack(c[pg, :, row])
            assert torch.equal(ref.dequantise(got, got_s), ref.dequantise(code, scales)), (side, t)
            assert torch.equal(out[t].double(), ref.dequantise(code, scales))
        assert (c.permute(0, 2, 1, 3)[~touched] == 0x55).all()
        assert (s.view(torch.uint8).permute(0, 2, 1, 3)[~touched] == 0x55).all()


def test_append_fp4_ties():
    """Every bf16 significand against every scale: exact ties of codes and scales go to even."""
    D, T = 128, 512
    x = torch.zeros(T, 1, D)
    frac = 1 + torch.arange(128) / 128
    for t in range(T):
        x[t, 0] = frac.roll(t % 128)[:D] * 2.0 ** ((torch.arange(D) + t // 128) % 4 - 2.0)
        x[t, 0, ::16] = 6.0 * float(frac[(t * 7) % 128])
    x = x.to(torch.bfloat16)
    cache = kda.kv_cache(8, 1, 64, D, "fp4", DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    kda.kv_append(x.to(DEV), x.to(DEV), cache, table, lens, cu)
    code, s = ref.quantise(x)
    for out in kda.kv_read(cache, table, lens, cu, num_tokens=T):
        assert torch.equal(out.cpu().double(), ref.dequantise(code, s))


@pytest.mark.parametrize("D,rot,interleaved", [(128, 0, False), (128, 128, False), (128, 64, True), (64, 32, False)])
def test_append_fp4_non_finite(D, rot, interleaved):
    """A NaN in a key or value makes its group NaN, as it would a bf16 cache; infinities saturate."""
    T, inf = 40, math.inf
    g = torch.Generator().manual_seed(9)
    k, v = _bf(g, T, 2, D), _bf(g, T, 2, D)
    for x in (k, v):
        x[3, 0, 5], x[4, 1, D - 1], x[5, 0, :] = NAN, NAN, NAN
        x[6, 1, 17], x[7, 0, 30], x[8, 1, :] = inf, -inf, inf
        x[9, 0, 2], x[9, 0, 3] = inf, NAN
        x[10, 1, 0:16] = torch.tensor([inf, 5000.0] + 14 * [300.0])
    rope = kda.rope_table(100, rot, device=DEV) if rot else None
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    lens, cu = torch.tensor([T], dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)
    full, cache = kda.kv_cache(4, 2, 16, D, "bf16", DEV), kda.kv_cache(4, 2, 16, D, "fp4", DEV)
    for c in (full, cache):
        kda.kv_append(k.to(DEV), v.to(DEV), c, table, lens, cu, rope=rope, interleaved=interleaved)
    for x, got in zip(kda.kv_read(full, table, lens, cu, num_tokens=T), kda.kv_read(cache, table, lens, cu, num_tokens=T)):
        x, got = x.cpu().unflatten(-1, (-1, 16)), got.cpu().double().unflatten(-1, (-1, 16))
        bad = torch.isnan(x).any(-1)
        assert bad.any() and torch.isnan(got[bad]).all()
        code, s = ref.quantise(x.clamp(-2688, 2688).nan_to_num(0.0).flatten(-2))
        want = ref.dequantise(code, s).unflatten(-1, (-1, 16))
        assert torch.equal(got[~bad], want[~bad])
    q = _bf(g, 1, 4, D).to(DEV)                               # both kv heads hold a NaN that the last token sees
    assert torch.isnan(kda.paged_attention(q, cache, table, lens)).all()
    assert kda.check_device_errors() == 0


@BOTH
def test_append_decode_form_and_in_place_queries(dtype):
    for B in (1, 37):
        b, cache, qo, q, k, v, where, turned, _ = _append_case([1] * B, list(range(0, 3 * B, 3)), 8, 2, 128, 16, dtype, 128, False, decode=True)
        for t, pg, row, pos in where:
            want = turned(q, t, pos)
            assert ((qo[t].double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -14) + 2.0 ** -23 * q[t].double().abs().max()).all()
    x = q.to(DEV)
    table, lens, _ = b.on(DEV)
    same = kda.kv_append(k.to(DEV), v.to(DEV), cache, table, lens, q=x, q_out=x, rope=kda.rope_table(4000, 128, device=DEV))
    assert same.data_ptr() == x.data_ptr() and torch.equal(x.cpu(), qo)


@BOTH
def test_slots_past_4_gb(dtype):
    """Cache rows whose element and byte offsets pass 32 bits, written, read back and attended over."""
    Hkv, page, D = 8, 128, 128
    pages = (2 ** 31 // (Hkv * page * D) + 9) * (1 if dtype == "bf16" else 4)
    shape = (pages, Hkv, page)
    if dtype == "bf16":
        cache = kda.KVCache(*(torch.empty(*shape, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    else:
        cache = kda.KVCache(*(torch.empty(*shape, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)),
                            *(torch.empty(*shape, D // 16, dtype=torch.uint8, device=DEV) for _ in range(2)))
    g = torch.Generator().manual_seed(1)
    T = 300
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    k, v, q = _bf(g, T, Hkv, D), _bf(g, T, Hkv, D), _bf(g, T, 2 * Hkv, D)
    kda.kv_append(k.to(DEV), v.to(DEV), cache, table, lens, cu)
    kk, vv = (x.cpu() for x in kda.kv_read(cache, table, lens, cu, num_tokens=T))
    for got, x in ((kk, k), (vv, v)):
        assert torch.equal(got, x) if dtype == "bf16" else torch.equal(got.double(), ref.dequantise(*ref.quantise(x)))
    b = ref.Batch([T], [0], page)
    kk, vv = kk.double(), vv.double()
    for n in (T, 1):
        b.new, b.past, b.cu = [n], [T - n], torch.tensor([0, n], dtype=torch.int32)
        o, l, mag, big = ref.attention(q[:n], lambda i, p: (kk[p], vv[p]), b, 0, 0, D ** -0.5)
        out = kda.paged_attention(q[:n].contiguous().to(DEV), cache, table, lens, b.cu.to(DEV))
        assert ((out.cpu().double() - o).abs() <= ref.bounds(o, l, mag, big)[0]).all()


# ---- device-side checks: bad tables are recorded and never followed ------------------------------------------

def _small(dtype="bf16", new=1):
    b = ref.Batch([new, new], [40, 20], 16, seed=1)
    cache, _ = _filled_cache(b, 2, 128, dtype, 1, poison=False)
    g = torch.Generator().manual_seed(3)
    q, k = _bf(g, b.T, 8, 128).to(DEV), _bf(g, b.T, 2, 128).to(DEV)
    return b, cache, q, k, *b.on(DEV)


@BOTH
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("what,code", [("page", 6), ("negative", 6), ("length", 8), ("cu", 2), ("position", 7)])
def test_bad_tables_are_recorded(dtype, new, what, code):
    b, cache, q, k, table, lens, cu = _small(dtype, new)
    rope = kda.rope_table(200, 128, device=DEV)
    before = [None if t is None else t.clone() for t in cache]
    positions = None
    if what == "page":
        table[0, :] = b.num_pages
    elif what == "negative":
        table[0, :] = -5
    elif what == "length":
        lens[0] = 10 ** 6
    elif what == "cu":
        cu[1] = -3
    else:
        positions = torch.full((b.T,), 200, dtype=torch.int32, device=DEV)
    kda.kv_append(k, k, cache, table, lens, cu, rope=rope, positions=positions)
    assert kda.check_device_errors() == code
    if what == "position":
        assert all(x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(cache, before))
        return
    kda.paged_attention(q, cache, table, lens, cu, max_new=new)
    assert kda.check_device_errors() == code
    b, cache, q, k, table, lens, cu = _small(dtype, new)       # and the next call is as ever
    kda.paged_attention(q, cache, table, lens, cu)
    assert kda.check_device_errors() == 0


@BOTH
@pytest.mark.parametrize("new,G,bound", [([600, 100], 1, 100), ([30, 700, 5, 64], 4, 64), ([300, 17, 17], 8, 17)])
def test_a_request_above_the_bound_leaves_the_others(dtype, new, G, bound):
    """Its own outputs are unspecified, every other request's are right."""
    b = ref.Batch(new, [50] * len(new), 32, seed=31)
    cache, k_of = _filled_cache(b, 2, 128, dtype, 5)
    table, lens, cu = b.on(DEV)
    q = _bf(torch.Generator().manual_seed(7), b.T, 2 * G, 128)
    out = torch.full((b.T, 2 * G, 128), NAN, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((b.T, 2 * G), NAN, device=DEV)
    kda.paged_attention(q.to(DEV), cache, table, lens, cu, max_new=bound, max_len=int(b.lens.max()), out=out, lse=lse)
    assert kda.check_device_errors() == 8
    o, l, mag, big = ref.attention(q, k_of, b, 0, 0, 128 ** -0.5)
    tol_o, tol_l = ref.bounds(o, l, mag, big)
    for i, n in enumerate(new):
        if n <= bound:
            at = slice(int(b.cu[i]), int(b.cu[i + 1]))
            assert ((out[at].cpu().double() - o[at]).abs() <= tol_o[at]).all()
            assert ((lse[at].cpu().double() - l[at]).abs() <= tol_l[at]).all()


@BOTH
@pytest.mark.parametrize("new,past,max_new", [([1, 1], [20, 30], 1), ([2, 1], [3000, 2000], 2), ([2, 2], [9000, 20000], 2), ([40, 30], [100, 20], 40),
                                              ([40, 30], [6000, 900], 40)])
def test_rows_that_no_request_owns(dtype, new, past, max_new):
    """Rows before cu_seqlens[0] and from cu_seqlens[-1] on: recorded, with zeros, in uncut calls, clusters and cut calls
    of both forms; append and read agree."""
    b = ref.Batch(new, past, 64, seed=32)
    cache, k_of = _filled_cache(b, 2, 128, dtype, 6)
    table, lens, cu = b.on(DEV)
    q = _bf(torch.Generator().manual_seed(8), b.T, 8, 128)
    o, l, mag, big = ref.attention(q, k_of, b, 0, 0, 128 ** -0.5)
    tol_o, tol_l = ref.bounds(o, l, mag, big)
    for front, back in ((0, 5), (3, 0), (2, 70)):
        T = front + b.T + back
        qd = torch.full((T, 8, 128), NAN, dtype=torch.bfloat16, device=DEV)
        qd[front:front + b.T] = q.to(DEV)
        out, lse = torch.full_like(qd, NAN), torch.full((T, 8), NAN, device=DEV)
        kda.paged_attention(qd, cache, table, lens, cu + front, max_new=max_new, max_len=int(b.lens.max()), out=out, lse=lse)
        assert kda.check_device_errors() == 2
        kda.paged_attention(qd, cache, table, lens, cu + front, max_new=max_new, max_len=int(b.lens.max()))   # without lse
        assert kda.check_device_errors() == 2
        own = torch.zeros(T, dtype=torch.bool)
        own[front:front + b.T] = True
        out, lse = out.cpu(), lse.cpu()
        assert (out[~own] == 0).all() and (lse[~own] == -math.inf).all()
        assert ((out[own].double() - o).abs() <= tol_o).all()
        assert ((lse[own].double() - l).abs() <= tol_l).all()
        k = _bf(torch.Generator().manual_seed(10), T, 2, 128).to(DEV)
        scratch = kda.kv_cache(b.num_pages, 2, 64, 128, dtype, DEV)
        qo = kda.kv_append(k, k, scratch, table, lens, cu + front, q=qd)
        assert kda.check_device_errors() == 2 and (qo.cpu()[~own] == 0).all() and torch.equal(qo.cpu()[own], q)
        for x in kda.kv_read(scratch, table, lens, cu + front, num_tokens=T):
            assert (x.cpu()[~own] == 0).all()
        assert kda.check_device_errors() == 2
