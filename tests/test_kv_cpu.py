"""Paged cache and attention, host side (no GPU): argument checks that return before any work is
enqueued, defaults, the struct mirror, and the 4-bit format's reference against its definition."""
import ctypes

import pytest
import torch

import kda_gated_delta_gb300 as kda
from kda_gated_delta_gb300 import binding, build
from tests import kv_reference as ref

FAKE = 1 << 20
MIS = FAKE + 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def _p(**kw):
    p = binding.KvParams()
    binding.lib().kda_kv_params_init(ctypes.byref(p), kw.pop("Hq", 8), kw.pop("Hkv", 2), kw.pop("D", 128), kw.pop("page", 64))
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_defaults(L):
    p = _p()
    assert (p.num_q_heads, p.num_kv_heads, p.head_dim, p.page_size) == (8, 2, 128, 64)
    assert (p.cache_dtype, p.rot_dim, p.rope_interleaved, p.window, p.num_sinks, p.softmax_scale) == (0, 128, 0, 0, 0, 0.0)


def _append(L, p=None, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, rope=FAKE, rows=100, pos=None, cu=FAKE, lens=FAKE,
            table=FAKE, n=2, mp=4, T=5, kc=FAKE, vc=FAKE, ksc=None, vsc=None, pages=8, qo=FAKE + (1 << 16)):
    p = _p() if p is None else p
    return L.kda_kv_append(ctypes.byref(p), q, qs, k, ks, v, vs, rope, rows, pos, cu, lens, table, n, mp, T, kc, vc, ksc,
                           vsc, pages, qo, None)


def _attend(L, p=None, q=FAKE, qs=1024, kc=FAKE, vc=FAKE, ksc=None, vsc=None, pages=8, cu=FAKE, lens=FAKE, table=FAKE, n=2,
            mp=4, T=5, new=4, length=256, out=FAKE, ws=FAKE, wsb=1 << 40):
    p = _p() if p is None else p
    return L.kda_paged_attention(ctypes.byref(p), q, qs, kc, vc, ksc, vsc, pages, cu, lens, table, n, mp, T, new, length,
                                 out, None, ws, wsb, None)


@pytest.mark.parametrize("call", [_append, _attend])
def test_shared_checks(L, call):
    assert call(L, p=_p(Hq=7)) == -1                       # not a multiple of the kv heads
    assert call(L, p=_p(window=-1)) == -1
    assert call(L, p=_p(num_sinks=-1)) == -1
    assert call(L, p=_p(softmax_scale=float("nan"))) == -1
    assert call(L, p=_p(D=96)) == -2
    assert call(L, p=_p(page=48)) == -2
    assert call(L, p=_p(page=256)) == -2
    assert call(L, p=_p(cache_dtype=2)) == -2
    assert call(L, p=_p(rot_dim=16)) == -2
    assert call(L, p=_p(rot_dim=160)) == -2
    assert call(L, p=_p(Hq=258, Hkv=2), qs=258 * 128) == -2
    assert call(L, p=_p(Hq=1032, Hkv=129), qs=1032 * 128) == -2
    assert call(L, n=1 << 29) == -2
    assert call(L, n=-1) == -1 and call(L, T=-1) == -1 and call(L, mp=0) == -1
    assert call(L, cu=None) == -1                          # one token per request: T must equal n
    assert call(L, lens=None) == -1 and call(L, table=None) == -1
    assert call(L, kc=None) == -1 and call(L, kc=MIS) == -3 and call(L, vc=MIS) == -3
    assert call(L, p=_p(cache_dtype=1)) == -1              # scales missing
    assert call(L, p=_p(cache_dtype=1), ksc=FAKE, vsc=MIS) == -3
    assert call(L, q=MIS) == -3
    assert call(L, qs=1000) == -1 and call(L, qs=1028) == -1
    assert call(L, T=1 << 22) == -2 and call(L, pages=1 << 27) == -2
    assert call(L, T=0) == 0 and call(L, n=0) == 0


@pytest.mark.parametrize("call", [_append, _attend])
def test_page_counts_whose_product_passes_64_bits(L, call):
    """A caller without a bound on its pages gets a refusal, not a call that takes every page index for good."""
    for pages in (1 << 27, 1 << 31, 1 << 47, 1 << 57, (1 << 62) + 1, (1 << 63) - 1):
        assert call(L, pages=pages) == -2
        assert call(L, pages=pages, p=_p(Hq=1, Hkv=1), qs=128) == -2 or pages == 1 << 27
    assert call(L, pages=-1) == -1


def test_append_checks(L):
    assert _append(L, k=None) == -1 and _append(L, v=None) == -1
    assert _append(L, q=None) == -1 and _append(L, qo=None) == -1
    assert _append(L, rope=None) == -1 and _append(L, rope=MIS) == -3
    assert _append(L, ks=248) == -1 and _append(L, vs=260) == -1
    assert _append(L, qs=1032, qo=FAKE) == -1              # in place needs contiguous queries
    assert _append(L, k=MIS) == -3 and _append(L, qo=MIS) == -3


def test_read_checks(L):
    def read(ko=FAKE, vo=FAKE, T=5):
        return L.kda_kv_read(ctypes.byref(_p()), FAKE, FAKE, None, None, 8, FAKE, FAKE, FAKE, 2, 4, T, ko, vo, None)
    assert read(ko=None) == -1 and read(vo=MIS) == -3 and read(T=0) == 0


def test_attention_checks(L):
    assert _attend(L, out=None) == -1 and _attend(L, out=MIS) == -3
    assert _attend(L, new=0) == -1 and _attend(L, length=0) == -1 and _attend(L, length=257) == -1
    assert _attend(L, cu=None, T=2, new=2) == -1
    size = L.kda_paged_attention_workspace_size
    p = _p()
    assert size(ctypes.byref(p), 2, 2, 0, 256) == 0 and size(ctypes.byref(_p(D=96)), 2, 2, 1, 256) == 0
    # a single request over a long history is split, and its parts need a workspace
    need = size(ctypes.byref(p), 1, 1, 1, 65536)
    if need:
        args = dict(cu=None, T=1, n=1, new=1, mp=1024, length=65536, pages=1024)
        assert _attend(L, ws=None, **args) == -4 and _attend(L, wsb=need - 1, **args) == -4
        assert _attend(L, ws=FAKE + 16, **args) == -4


@pytest.mark.parametrize("fp4", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,new", [(1, 1), (4, 4), (40, 40), (300, 300)])
def test_cut_calls_need_their_workspace(L, T, new, D, fp4):
    """One request over a long history is cut into more parts than a cluster joins, with few and with many query rows."""
    p = _p(D=D, cache_dtype=fp4)
    need = L.kda_paged_attention_workspace_size(ctypes.byref(p), 1, T, new, 65536)
    assert need > 8 * T * 8 * (D + 1) * 4                  # more than eight parts of 8 heads, in fp32
    args = dict(p=p, qs=8 * D, ksc=FAKE, vsc=FAKE, T=T, n=1, new=new, mp=1024, length=65536, pages=1024)
    if new == 1:
        args["cu"] = None
    assert _attend(L, ws=None, **args) == -4 and _attend(L, wsb=need - 1, **args) == -4 and _attend(L, ws=FAKE + 16, **args) == -4


def test_any_large_bound_on_new_tokens_means_all_tokens(L):
    """The form and its workspace go by one bound, whose products with the heads of a group stay whole numbers."""
    size = L.kda_paged_attention_workspace_size
    for Hq, Hkv, n, T, length in ((8, 2, 1, 3, 65536), (32, 8, 2, 5, 65536), (128, 1, 1, 40, 65536), (32, 8, 8, 16384, 4096), (5, 5, 1, 16, 70000)):
        p = _p(Hq=Hq, Hkv=Hkv)
        want = size(ctypes.byref(p), n, T, T, length)
        for new in (T + 1, (1 << 24) + 1, 1 << 25, 1 << 28, 1 << 29, 1 << 30, (1 << 31) - 1):
            assert size(ctypes.byref(p), n, T, new, length) == want, (Hq, T, new)
    args = dict(T=3, n=1, mp=1024, length=65536, pages=1024)    # 12 rows a kv head
    need = size(ctypes.byref(_p()), 1, 3, 3, 65536)
    assert need > 0
    for new in (3, 1 << 29, (1 << 31) - 1):
        assert _attend(L, new=new, wsb=need - 1, **args) == -4 and _attend(L, new=new, ws=None, **args) == -4


def test_python_numbers_past_32_bits(L, monkeypatch):
    """They are not taken modulo 2^32: a window of 2^32 + 5 is no window of 5."""
    def seen(**kw):
        return binding._kv_params(8, 2, 128, 64, False, **kw)._obj

    for big in (2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70):
        p = seen(window=big, sinks=big)
        assert p.window == p.num_sinks == 2 ** 31 - 1
        assert seen(window=-big).window < 0 and seen(sinks=-big).num_sinks < 0       # refused by the library
        size = kda.attention_workspace_size
        assert size(8, 2, 128, 64, 1, 3, big, 65536) == size(8, 2, 128, 64, 1, 3, 3, 65536) > 0
        assert size(8, 2, 128, 64, 1, 1, 1, -big) == size(8, 2, 128, 64, 1, 1, -big, 256) == 0
    p = seen(window=2 ** 31 - 1, sinks=5)
    assert (p.window, p.num_sinks) == (2 ** 31 - 1, 5)


def test_workspace_of_an_unknown_cache_type(L):
    for dtype in ("int8", "FP4", torch.bfloat16, None):       # none of them means bf16
        with pytest.raises(ValueError):
            kda.attention_workspace_size(8, 2, 128, 64, 1, 1, 1, 65536, dtype=dtype)
    assert kda.attention_workspace_size(8, 2, 128, 64, 1, 1, 1, 65536) > 0
    assert kda.attention_workspace_size(8, 2, 128, 64, 1, 1, 1, 65536, dtype="fp4") > 0


def test_python_refusals():
    with pytest.raises(ValueError):
        kda.kv_cache(4, 2, 64, 128, dtype="int8", device="cpu")
    c = kda.kv_cache(4, 2, 64, 128, device="cpu")
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):                        # CPU tensors
        kda.kv_append(x, x, c, i[:, None], i)
    with pytest.raises(ValueError):
        kda.paged_attention(x, c, i[:, None], i)


def test_rope_table():
    t = kda.rope_table(1000, 64, device="cpu")
    assert t.shape == (1000, 64) and t.dtype == torch.float32
    f = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    a = torch.arange(1000, dtype=torch.float64)[:, None] * f
    exact = torch.cat([a.cos(), a.sin()], 1)
    assert ((t.double() - exact).abs() <= 2.0 ** -16 * exact.abs() * 1.001).all()
    assert (t.view(torch.int32) & 0xff == 0).all()          # 16 significant bits: products with bf16 are exact


def test_four_bit_reference():
    s = ref.e4m3(torch.tensor([0.0, 2.0 ** -10, 2.0 ** -9, 1.0, 1.0625, 1.1875, 500.0], dtype=torch.float64))
    assert s.tolist() == [0.0, 0.0, 2.0 ** -9, 1.0, 1.0, 1.25, 448.0]
    x = torch.zeros(16, dtype=torch.bfloat16)
    x[:9] = torch.tensor([6.0, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, -5.0, 0.3])
    code, s = ref.quantise(x)
    assert s.item() == 1.0
    assert ref.dequantise(code, s)[:9].tolist() == [6.0, 0.0, 1.0, -1.0, 2.0, 2.0, 4.0, -4.0, 0.5]
