"""Convolution, selective recurrence and group norm, host side (no GPU): argument checks that return before any work is
enqueued, defaults, the structs' mirrors, and the Python calls' own refusals."""
import ctypes

import pytest
import torch

import kda_gated_delta_gb300 as kda
from kda_gated_delta_gb300 import binding, build
from tests.test_device_guard_cpu import BF, I32, on, reached  # noqa: F401

FAKE = 1 << 20
MIS = FAKE + 4
F32 = torch.float32


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def _conv(L, C=64, W=4, io=1, act=1, x=FAKE, xs=None, w=FAKE, b=None, cu=FAKE, n=2, T=5, pool=FAKE, slots=4, idx=FAKE, outs=(FAKE,), parts=None, m=None):
    parts = [C] if parts is None else parts
    p = binding.ConvParams(C, W, io, act)
    return L.kda_causal_conv(ctypes.byref(p), x, C if xs is None else xs, w, b, cu, n, T, pool, slots, idx, (ctypes.c_void_p * len(outs))(*outs),
                             (ctypes.c_int32 * len(parts))(*parts), len(parts) if m is None else m, None)


def test_conv_checks(L):
    for kw in (dict(C=0), dict(n=-1), dict(T=-1), dict(slots=-1), dict(cu=None), dict(parts=[60]), dict(parts=[64, 0], outs=(FAKE, FAKE)), dict(m=0),
               dict(x=None), dict(w=None), dict(pool=None), dict(idx=None), dict(xs=63), dict(outs=(None,)), dict(parts=[1 << 30, 1 << 30, 1 << 30, (1 << 30) + 64], outs=(FAKE,) * 4)):
        assert _conv(L, **kw) == -1, kw
    assert _conv(L, parts=[16] * 4 + [0], outs=(FAKE,) * 5) == -1
    for kw in (dict(W=1), dict(W=5), dict(io=2), dict(act=2), dict(act=-1), dict(C=(1 << 20) + 1), dict(T=2 ** 31), dict(xs=1 << 31), dict(n=1 << 30)):
        assert _conv(L, **kw) == -2, kw
    for kw in (dict(x=FAKE + 1), dict(pool=FAKE + 1), dict(w=FAKE + 2), dict(b=FAKE + 2), dict(outs=(FAKE + 1,)), dict(io=0, x=FAKE + 2)):
        assert _conv(L, **kw) == -3, kw
    assert _conv(L, T=0) == 0 and _conv(L, n=0) == 0 and _conv(L, T=0, x=None, pool=None) == 0


def _p(**kw):
    p = binding.SsmParams()
    binding.lib().kda_ssm_params_init(ctypes.byref(p), kw.pop("H", 4), kw.pop("P", 64), kw.pop("N", 128), kw.pop("G", 2))
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _rows(p, x=FAKE, xs=256, dt=FAKE, ds=4, B=FAKE, bs=256, C=FAKE, cs=256, A=FAKE):
    return ctypes.byref(p), x, xs, dt, ds, B, bs, C, cs, A, None, None


def _prefill(L, p=None, cu=FAKE, n=2, T=5, pool=FAKE, slots=4, idx=FAKE, out=FAKE, ws=FAKE, wsb=1 << 40, **kw):
    return L.kda_ssm_prefill(*_rows(_p() if p is None else p, **kw), cu, n, T, pool, slots, idx, out, ws, wsb, None)


def _decode(L, p=None, n=2, T=None, pool=FAKE, slots=4, idx=FAKE, out=FAKE, **kw):
    return L.kda_ssm_decode(*_rows(_p() if p is None else p, **kw), n if T is None else T, pool, slots, idx, out, None)


def test_ssm_defaults(L):
    p = _p()
    assert (p.num_heads, p.head_dim, p.state_dim, p.num_groups) == (4, 64, 128, 2)
    assert (p.io_dtype, p.dt_dtype, p.out_dtype, p.softplus_threshold) == (binding.KDA_BF16, binding.KDA_F32, binding.KDA_BF16, 20.0)


@pytest.mark.parametrize("call", [_prefill, _decode])
def test_ssm_checks(L, call):
    for kw in (dict(H=0), dict(G=0), dict(H=3), dict(softplus_threshold=float("nan")), dict(softplus_threshold=-1.0)):
        assert call(L, p=_p(**kw)) == -1, kw
    for kw in (dict(P=48), dict(P=256), dict(P=8), dict(N=8), dict(N=96), dict(N=512), dict(io_dtype=2), dict(dt_dtype=-1), dict(out_dtype=3)):
        assert call(L, p=_p(**kw)) == -2, kw
    assert call(L, p=_p(H=4100, G=1), xs=4100 * 64, ds=4100) == -2
    for kw in (dict(n=-1), dict(slots=-1), dict(x=None), dict(dt=None), dict(B=None), dict(C=None), dict(A=None), dict(pool=None), dict(idx=None), dict(out=None),
               dict(xs=248), dict(xs=260), dict(bs=248), dict(cs=257), dict(ds=3)):
        assert call(L, **kw) == -1, kw
    for kw in (dict(x=MIS), dict(B=MIS), dict(C=MIS), dict(pool=MIS), dict(out=MIS), dict(dt=FAKE + 2)):
        assert call(L, **kw) == -3, kw
    for kw in (dict(T=2 ** 31 - 1), dict(xs=1 << 31), dict(ds=1 << 31), dict(bs=1 << 31), dict(cs=1 << 31)):
        assert call(L, **kw) == -2, kw
    assert call(L, T=0) == 0 and call(L, n=0) == 0


def test_ssm_prefill_checks(L):
    assert _prefill(L, cu=None) == -1 and _prefill(L, T=-1) == -1 and _prefill(L, n=1 << 29) == -2
    size = L.kda_ssm_prefill_workspace_size
    assert size(ctypes.byref(_p(P=48)), 2, 5) == 0 and size(ctypes.byref(_p()), 0, 5) == 0 and size(ctypes.byref(_p()), 2, -1) == 0
    for p, n, T in ((_p(), 1, 100000), (_p(H=64, G=8), 8, 16412)):
        need = size(ctypes.byref(p), n, T)
        if need:
            kw = dict(xs=p.num_heads * 64, ds=p.num_heads, bs=p.num_groups * 128, cs=p.num_groups * 128)
            assert _prefill(L, p=p, n=n, T=T, ws=None, **kw) == -4 and _prefill(L, p=p, n=n, T=T, wsb=need - 1, **kw) == -4
            assert _prefill(L, p=p, n=n, T=T, ws=FAKE + 16, **kw) == -4


def _norm(L, G=4, n=128, io=1, od=1, act=0, first=0, eps=1e-5, x=FAKE, xs=512, gate=None, gs=0, w=None, b=None, T=5, out=FAKE):
    p = binding.NormParams(G, n, io, od, act, first, 1, eps)
    return L.kda_group_norm(ctypes.byref(p), x, xs, gate, gs, w, b, T, out, None)


def test_norm_checks(L):
    for kw in (dict(G=0), dict(n=0), dict(T=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(first=1), dict(x=None), dict(out=None), dict(xs=511),
               dict(gate=FAKE, gs=511)):
        assert _norm(L, **kw) == -1, kw
    for kw in (dict(io=2), dict(od=2), dict(act=3), dict(act=-1), dict(n=16385, xs=1 << 20), dict(T=1 << 31), dict(T=1 << 29), dict(xs=1 << 31), dict(gate=FAKE, gs=1 << 31)):
        assert _norm(L, **kw) == -2, kw
    for kw in (dict(x=FAKE + 1), dict(out=FAKE + 1), dict(gate=FAKE + 1, gs=512), dict(w=FAKE + 2), dict(b=FAKE + 2), dict(io=0, x=FAKE + 2)):
        assert _norm(L, **kw) == -3, kw
    assert _norm(L, T=0) == 0 and _norm(L, T=0, x=None) == 0


# ---- the Python calls ---------------------------------------------------------------------------------

def calls(at):
    """name -> (call, its tensors by name), everything on cuda:`at`."""
    t = dict(xc=on(at, 4, 64, dtype=BF), w=on(at, 64, 4), bc=on(at, 64), pc=on(at, 3, 3, 64, dtype=BF), idx=on(at, 2, dtype=I32), cu=on(at, 3, dtype=I32),
             o1=on(at, 4, 48, dtype=BF), o2=on(at, 4, 16, dtype=BF),
             x=on(at, 4, 2, 64, dtype=BF), dt=on(at, 4, 2), B=on(at, 4, 1, 128, dtype=BF), C=on(at, 4, 1, 128, dtype=BF), A=on(at, 2), db=on(at, 2), D=on(at, 2),
             pool=on(at, 3, 2, 64, 128), out=on(at, 4, 2, 64, dtype=BF), ws=on(at, 1 << 20, dtype=torch.uint8), i4=on(at, 4, dtype=I32),
             g=on(at, 2, 64), b=on(at, 2, 64), gate=on(at, 4, 2, 64, dtype=BF))
    ssm = ["x", "dt", "B", "C", "A", "pool", "db", "D", "out"]
    return t, {
        "kda_causal_conv": (lambda t: kda.causal_conv(t["xc"], t["w"], t["pc"], t["idx"], t["cu"], bias=t["bc"], activation="silu", split=(48, 16), out=(t["o1"], t["o2"])),
                            ["xc", "w", "pc", "idx", "cu", "bc", "o1", "o2"]),
        "kda_ssm_prefill": (lambda t: kda.ssm_prefill(t["x"], t["dt"], t["B"], t["C"], t["A"], t["cu"], t["pool"], t["idx"], dt_bias=t["db"], D=t["D"], out=t["out"],
                                                      workspace=t["ws"]), ssm + ["idx", "cu", "ws"]),
        "kda_ssm_decode": (lambda t: kda.ssm_decode(t["x"], t["dt"], t["B"], t["C"], t["A"], t["pool"], t["i4"], dt_bias=t["db"], D=t["D"], out=t["out"]), ssm + ["i4"]),
        "kda_group_norm": (lambda t: kda.group_norm(t["x"], t["g"], t["b"], gate=t["gate"], out=t["out"]), ["x", "g", "b", "gate", "out"]),
    }


NAMES = ["kda_causal_conv", "kda_ssm_prefill", "kda_ssm_decode", "kda_group_norm"]


@pytest.mark.parametrize("name", NAMES)
def test_devices(reached, name):  # noqa: F811
    base, table = calls(0)
    call, used = table[name]
    call(base)
    assert reached == [name]
    for one in used:
        other = dict(base)
        other[one] = base[one].clone()
        other[one].at = 1
        with pytest.raises(ValueError, match="cuda:"):
            call(other)
        other[one] = base[one].as_subclass(torch.Tensor)          # a CPU tensor
        with pytest.raises(ValueError):
            call(other)
    with pytest.raises(ValueError, match="current device"):
        call(calls(1)[0])
    assert reached == [name]


@pytest.mark.parametrize("name", NAMES)
def test_types_and_shapes(reached, name):  # noqa: F811
    base, table = calls(0)
    call, used = table[name]
    for one in used:
        t = base[one]
        with pytest.raises((TypeError, ValueError)):
            call({**base, one: on(0, *t.shape, dtype=torch.float16)})
        if one != "ws":
            with pytest.raises(ValueError):
                call({**base, one: on(0, *t.shape, 2, dtype=t.dtype)})
        if one not in ("ws", "pc", "pool") and t.dim() > 0:
            with pytest.raises(ValueError):
                call({**base, one: on(0, t.shape[0] + 1, *t.shape[1:], dtype=t.dtype)})
    assert reached == []


def test_refusals_of_their_own(reached):  # noqa: F811
    t, _ = calls(0)
    conv = lambda **kw: kda.causal_conv(t["xc"], t["w"], t["pc"], t["idx"], t["cu"], **kw)  # noqa: E731
    for kw in (dict(activation="sigmoid"), dict(activation="gelu"), dict(split=(32, 31)), dict(split=(65, -1)), dict(split=()), dict(split=(16,) * 3 + (8, 8)),
               dict(split=(32, 32), out=(t["o1"],))):
        with pytest.raises(ValueError):
            conv(**kw)
    with pytest.raises(ValueError):
        kda.causal_conv(t["xc"], t["w"], t["pc"], t["idx"])                          # two requests, four tokens
    with pytest.raises(ValueError):
        kda.causal_conv(t["xc"].t(), t["w"], t["pc"], t["idx"], t["cu"])              # channels apart
    with pytest.raises(ValueError):
        kda.causal_conv(t["xc"][:1].expand(4, 64), t["w"], t["pc"], t["idx"], t["cu"])  # one row four times
    with pytest.raises(ValueError):
        kda.ssm_decode(t["x"], t["dt"], t["B"], t["C"], t["A"], t["pool"], t["idx"])
    with pytest.raises(ValueError):
        kda.ssm_prefill(t["x"], t["dt"], t["B"], t["C"], t["A"], on(0, 1, dtype=I32), t["pool"], on(0, 0, dtype=I32))
    for kw in (dict(activation="gelu"), dict(gate_first=True)):
        with pytest.raises(ValueError):
            kda.group_norm(t["x"], **kw)
    with pytest.raises(TypeError):
        kda.group_norm(t["x"], gate=t["gate"], out_dtype=F32)                           # a gate of another type than the output
    assert reached == []
    conv(split=(48, 16), out=(t["o1"], t["o2"]), activation="silu")
    kda.causal_conv(on(0, 4, 80, dtype=BF)[:, 16:], t["w"], t["pc"], t["idx"], t["cu"], out=on(0, 4, 64, dtype=BF))
    assert reached == ["kda_causal_conv"] * 2


def test_element_alignment(L):
    """fp32 parameters and the int32 tables need their elements' alignment: a kernel that read them elsewhere would fault."""
    for at in (1, 2, 3):
        off = FAKE + at
        for kw in (dict(cu=off), dict(idx=off)):
            assert _conv(L, **kw) == -3, kw
        assert _conv(L, cu=None, T=2, idx=off) == -3
        for call in (_prefill, _decode):
            assert call(L, A=off) == -3 and call(L, idx=off) == -3
        assert _prefill(L, cu=off) == -3
        p = ctypes.byref(_p())
        head = (p, FAKE, 256, FAKE, 4, FAKE, 256, FAKE, 256, FAKE)
        for bias, D in ((off, None), (None, off)):
            assert L.kda_ssm_prefill(*head, bias, D, FAKE, 2, 5, FAKE, 4, FAKE, FAKE, FAKE, 1 << 40, None) == -3
            assert L.kda_ssm_decode(*head, bias, D, 2, FAKE, 4, FAKE, FAKE, None) == -3


def test_numbers_given_as_tensors(reached, monkeypatch):  # noqa: F811
    """A scalar that changes in place between two calls is not answered with its old value."""
    t, table = calls(0)
    seen = []

    def fn(name):
        def call(p, *args):
            p = p._obj
            seen.append(p.eps if name == "kda_group_norm" else p.softmax_scale if name == "kda_paged_attention" else p.softplus_threshold)
            return 0
        return call

    monkeypatch.setattr(binding, "_fn", fn)
    number = torch.tensor(0.5)
    cache = on(0, 8, 2, 16, 64, dtype=BF), on(0, 8, 2, 16, 64, dtype=BF)
    q, pages, lens = on(0, 2, 4, 64, dtype=BF), on(0, 2, 4, dtype=I32), on(0, 2, dtype=I32)
    for value in (0.5, 0.25):
        number.fill_(value)
        kda.group_norm(t["x"], eps=number)
        kda.ssm_prefill(t["x"], t["dt"], t["B"], t["C"], t["A"], t["cu"], t["pool"], t["idx"], softplus_threshold=number, workspace=t["ws"])
        kda.ssm_decode(t["x"], t["dt"], t["B"], t["C"], t["A"], t["pool"], t["i4"], softplus_threshold=number)
        kda.paged_attention(q, (*cache, None, None), pages, lens, scale=number)
        assert seen == [value] * 4
        seen.clear()


def test_workspace_by_device(reached, monkeypatch):  # noqa: F811
    """A call's workspace is that of its device: another device's size, looked up earlier, is not taken for it."""
    at, given = [0], []

    class Lib:
        def kda_ssm_prefill_workspace_size(self, p, n, T):
            return 1000 + at[0]

    monkeypatch.setattr(binding, "lib", lambda: Lib())
    monkeypatch.setattr(binding, "_device", lambda: at[0])
    monkeypatch.setattr(binding, "_fn", lambda name: lambda *args: given.append(args[-2]) or 0)
    for dev in (0, 1, 0):
        at[0] = dev
        t, _ = calls(dev)
        kda.ssm_prefill(t["x"], t["dt"], t["B"], t["C"], t["A"], t["cu"], t["pool"], t["idx"], out=t["out"], softplus_threshold=7.0)
    assert given == [1000, 1001, 1000]
