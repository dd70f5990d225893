"""Every Python call refuses tensors that are not on the current device, where its kernels would be launched.
On the CPU: tensors that claim a device, a current device by decree, and a library that records what reaches it."""
import types

import pytest
import torch

import kda_gated_delta_gb300 as kda
from kda_gated_delta_gb300 import binding


class Claims(torch.Tensor):
    """A CPU tensor that says it is on cuda:`at`."""
    at = 0
    is_cuda = True

    def get_device(self):
        return self.at


def on(at, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Claims)
    t.at = at
    return t


@pytest.fixture
def reached(monkeypatch):
    """Names of the entry points that were called; the current device is 0."""
    names = []

    def fn(name):
        def call(*args):
            names.append(name)
            return 0
        return call

    real = binding.lib()

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name) if name.endswith("_init") or name.endswith("_size") else fn(name)

    monkeypatch.setattr(binding, "lib", lambda: Lib())
    monkeypatch.setattr(binding, "_fn", fn)
    monkeypatch.setattr(binding, "_attention_workspace", lambda *a: 0)
    monkeypatch.setattr(binding, "_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0, device_index=0))
    return names


BF, I32 = torch.bfloat16, torch.int32


def kv_calls(at):
    """name -> (call, its tensors by name); everything on cuda:`at` but what is replaced."""
    def cache(t):
        return t["ck"], t["cv"], t["ks"], t["vs"]

    base = dict(k=on(at, 2, 2, 128, dtype=BF), v=on(at, 2, 2, 128, dtype=BF), q=on(at, 2, 4, 128, dtype=BF), table=on(at, 2, 4, dtype=I32),
                lens=on(at, 2, dtype=I32), cu=on(at, 3, dtype=I32), rope=on(at, 10, 128), pos=on(at, 2, dtype=I32),
                qo=on(at, 2, 4, 128, dtype=BF), out=on(at, 2, 4, 128, dtype=BF), lse=on(at, 2, 4), ws=on(at, 512, dtype=torch.uint8),
                ko=on(at, 2, 2, 128, dtype=BF), vo=on(at, 2, 2, 128, dtype=BF),
                ck=on(at, 8, 2, 16, 64, dtype=torch.uint8), cv=on(at, 8, 2, 16, 64, dtype=torch.uint8),
                ks=on(at, 8, 2, 16, 8, dtype=torch.uint8), vs=on(at, 8, 2, 16, 8, dtype=torch.uint8))
    cached = ["ck", "cv", "ks", "vs", "table", "lens", "cu"]
    return base, {
        "kda_kv_append": (lambda t: kda.kv_append(t["k"], t["v"], cache(t), t["table"], t["lens"], t["cu"], q=t["q"], q_out=t["qo"],
                                                  rope=t["rope"], positions=t["pos"]), cached + ["k", "v", "q", "qo", "rope", "pos"]),
        "kda_kv_read": (lambda t: kda.kv_read(cache(t), t["table"], t["lens"], t["cu"], num_tokens=2, out=(t["ko"], t["vo"])), cached + ["ko", "vo"]),
        "kda_paged_attention": (lambda t: kda.paged_attention(t["q"], cache(t), t["table"], t["lens"], t["cu"], out=t["out"], lse=t["lse"],
                                                              workspace=t["ws"]), cached + ["q", "out", "lse", "ws"]),
    }


@pytest.mark.parametrize("name", ["kda_kv_append", "kda_kv_read", "kda_paged_attention"])
def test_cache_calls(reached, name):
    base, calls = kv_calls(0)
    call, used = calls[name]
    call(base)
    assert reached == [name]
    for one in used:                                         # one tensor elsewhere
        other = dict(base)
        other[one] = base[one].clone()
        other[one].at = 1
        with pytest.raises(ValueError, match="cuda:"):
            call(other)
    with pytest.raises(ValueError, match="current device"):    # all of them elsewhere
        call(kv_calls(1)[0])
    assert reached == [name]


@pytest.mark.parametrize("name", ["kda_kv_append", "kda_kv_read", "kda_paged_attention"])
def test_shapes_of_the_tables(reached, name):
    """One length and one table row per request: further entries would be read as other requests'."""
    base, calls = kv_calls(0)
    call, _ = calls[name]
    for bad in (dict(lens=on(0, 2, 3, dtype=I32)), dict(lens=on(0, dtype=I32)), dict(lens=on(0, 1, dtype=I32)), dict(table=on(0, 8, dtype=I32)),
                dict(cu=on(0, 3, 2, dtype=I32)), dict(cu=on(0, dtype=I32)), dict(cu=on(0, 2, dtype=I32)),
                dict(lens=on(0, 0, dtype=I32), table=on(0, 0, 4, dtype=I32), cu=on(0, 1, dtype=I32))):
        with pytest.raises(ValueError):
            call({**base, **bad})
    assert reached == []
    call({**base, "lens": on(0, 2, 1, dtype=I32)})
    assert reached == [name]


def test_bounds_past_32_bits(reached, monkeypatch):
    base, calls = kv_calls(0)
    got = []
    monkeypatch.setattr(binding, "_fn", lambda name: lambda *args: got.append(args[14:16]) or 0)
    for new, length in ((2 ** 32 + 1, 2 ** 32 + 64), (2 ** 63, 2 ** 31), (-2 ** 32 + 1, -2 ** 32 + 64)):
        kda.paged_attention(base["q"], (base["ck"], base["cv"], base["ks"], base["vs"]), base["table"], base["lens"], base["cu"],
                            max_new=new, max_len=length)
    top = 2 ** 31 - 1
    assert got == [(top, top), (top, top), (-top, -top)]


def state_calls(at):
    H, D, B = 2, 128, 2
    x = [on(at, B, H, D, dtype=BF) for _ in range(3)]
    gates = [on(at, B, H, D), on(at, B, H), on(at, H), on(at, H, D)]
    pool, idx, cu = on(at, 4, H, D, D), on(at, B, dtype=I32), on(at, B + 1, dtype=I32)
    inter, out = on(at, B, 1, H, D, D), on(at, B, H, D, dtype=BF)
    rings, cursor = [on(at, 4, H, 8, D) for _ in range(3)], on(at, B, dtype=I32)
    ws = on(at, 1 << 20, dtype=torch.uint8)
    return {
        "kda_chunk_prefill": (lambda a: kda.chunk_prefill(*a[:10], out=a[10], workspace=a[11]), [*x, *gates, cu, pool, idx, out, ws]),
        "kda_recurrent_decode": (lambda a: kda.recurrent_decode(*a[:9], out=a[9]), [*x, *gates, pool, idx, out]),
        "kda_recurrent_verify": (lambda a: kda.recurrent_verify(*a[:9], 1, inter=a[9], out=a[10]), [*x, *gates, pool, idx, inter, out]),
        "kda_replay_decode": (lambda a: kda.replay_decode(*a[:9], tuple(a[9:12]), a[12], out=a[13]), [*x, *gates, pool, idx, *rings, cursor, out]),
        "kda_commit_verified_states": (lambda a: kda.commit_verified_states(*a), [inter, cursor, pool, idx]),
    }


@pytest.mark.parametrize("name", ["kda_chunk_prefill", "kda_recurrent_decode", "kda_recurrent_verify", "kda_replay_decode", "kda_commit_verified_states"])
def test_state_calls(reached, name):
    call, tensors = state_calls(0)[name]
    call(tensors)
    assert reached == [name]
    for i in range(len(tensors)):
        other = list(tensors)
        other[i] = tensors[i].clone()
        other[i].at = 1
        with pytest.raises(ValueError, match="current device"):
            call(other)
    assert reached == [name]


def test_stream_of_another_device(reached):
    call, tensors = state_calls(0)["kda_recurrent_decode"]
    stream = types.SimpleNamespace(cuda_stream=0, device_index=1)
    with pytest.raises(ValueError, match="stream"):
        kda.recurrent_decode(*tensors[:9], out=tensors[9], stream=stream)
    assert reached == []
