"""Thin ctypes binding of libkda (include/kda.h).

Argument marshalling only: every step of the computation runs in the CUDA kernels behind the
C ABI.  PyTorch supplies device memory and the current stream.  There is no fallback: if
``libkda.so`` has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import NamedTuple

import torch

from . import build as _build

KDA_OK = 0
KDA_F32, KDA_BF16 = 0, 1
CACHE_BF16, CACHE_FP4 = 0, 1
GATE_PER_CHANNEL, GATE_PER_HEAD = 0, 1

_STATUS = {
    0: "KDA_OK", -1: "KDA_ERR_INVALID_ARG", -2: "KDA_ERR_UNSUPPORTED", -3: "KDA_ERR_MISALIGNED",
    -4: "KDA_ERR_WORKSPACE", -5: "KDA_ERR_CUDA", -6: "KDA_ERR_DEVICE_CHECK", -7: "KDA_ERR_SCRATCH_LIMIT",
}


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS.get(status, status)} ({status_string(status)})")


class Params(ctypes.Structure):
    """Mirror of ``kda_params``."""
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("gate_kind", ctypes.c_int32),
        ("chunk_size", ctypes.c_int32),
        ("use_lower_bound", ctypes.c_int32),
        ("lower_bound", ctypes.c_float),
        ("scale", ctypes.c_float),
        ("l2_eps", ctypes.c_float),
        ("softplus_threshold", ctypes.c_float),
    ]


class KvParams(ctypes.Structure):
    """Mirror of ``kda_kv_params``."""
    _fields_ = [
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("cache_dtype", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32),
        ("rope_interleaved", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("num_sinks", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
    ]


class ConvParams(ctypes.Structure):
    """Mirror of ``kda_conv_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_channels", "width", "io_dtype", "activation")]


class SsmParams(ctypes.Structure):
    """Mirror of ``kda_ssm_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_heads", "head_dim", "state_dim", "num_groups", "io_dtype", "dt_dtype", "out_dtype")]
    _fields_ += [("softplus_threshold", ctypes.c_float)]


class NormParams(ctypes.Structure):
    """Mirror of ``kda_norm_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_groups", "group_size", "io_dtype", "out_dtype", "activation", "gate_first", "center")]
    _fields_ += [("eps", ctypes.c_float)]


_P = ctypes.c_void_p
_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libkda.so (built by ``kda_gated_delta_gb300.build``); raise if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libkda.so is not built ({path}); run python -m kda_gated_delta_gb300.build")
        L = ctypes.CDLL(path)
        L.kda_params_init.restype = None
        L.kda_params_init.argtypes = [ctypes.POINTER(Params), ctypes.c_int32, ctypes.c_int32]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_status_string.argtypes = [ctypes.c_int32]
        L.kda_chunk_prefill_workspace_size.restype = ctypes.c_size_t
        L.kda_chunk_prefill_workspace_size.argtypes = [ctypes.POINTER(Params), ctypes.c_int32, ctypes.c_int64]
        L.kda_chunk_prefill.restype = ctypes.c_int32
        L.kda_chunk_prefill.argtypes = [ctypes.POINTER(Params), _P, _P, _P, _P, _P, _P, _P, _P,
                                        ctypes.c_int32, ctypes.c_int64, _P, ctypes.c_int64, _P, _P,
                                        _P, ctypes.c_size_t, _P]
        L.kda_chunk_prefill_timed.restype = ctypes.c_int32
        L.kda_chunk_prefill_timed.argtypes = L.kda_chunk_prefill.argtypes + [ctypes.POINTER(ctypes.c_void_p)]
        L.kda_recurrent_decode.restype = ctypes.c_int32
        L.kda_recurrent_decode.argtypes = [ctypes.POINTER(Params), _P, _P, _P, _P, _P, _P, _P,
                                           ctypes.c_int32, _P, ctypes.c_int64, _P, _P, _P]
        L.kda_recurrent_verify.restype = ctypes.c_int32
        L.kda_recurrent_verify.argtypes = [ctypes.POINTER(Params), _P, _P, _P, _P, _P, _P, _P,
                                           ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_int64, _P,
                                           _P, _P, _P]
        L.kda_chunk_prefill_snapshots.restype = ctypes.c_int32
        L.kda_chunk_prefill_snapshots.argtypes = L.kda_chunk_prefill.argtypes[:-1] + [_P, ctypes.c_int64, _P]
        L.kda_replay_decode.restype = ctypes.c_int32
        L.kda_replay_decode.argtypes = [ctypes.POINTER(Params), _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32,
                                        _P, ctypes.c_int64, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P]
        L.kda_commit_verified_states.restype = ctypes.c_int32
        L.kda_commit_verified_states.argtypes = [ctypes.POINTER(Params), _P, ctypes.c_int32, ctypes.c_int32, _P,
                                                 _P, ctypes.c_int64, _P, _P]
        L.kda_check_device_errors.restype = ctypes.c_int32
        L.kda_check_device_errors.argtypes = [_P, ctypes.POINTER(ctypes.c_int32)]
        L.kda_selftest_wait_timeout.restype = ctypes.c_int32
        L.kda_selftest_wait_timeout.argtypes = [ctypes.c_uint32, _P, _P]
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        KP, cache, batch = ctypes.POINTER(KvParams), [_P, _P, _P, _P], [_P, _P, _P, i32, i32, i64]
        L.kda_kv_params_init.restype = None
        L.kda_kv_params_init.argtypes = [KP, i32, i32, i32, i32]
        L.kda_kv_append.restype = i32
        L.kda_kv_append.argtypes = [KP, _P, i64, _P, i64, _P, i64, _P, i64, _P, *batch, *cache, i64, _P, _P]
        L.kda_kv_read.restype = i32
        L.kda_kv_read.argtypes = [KP, *cache, i64, *batch, _P, _P, _P]
        L.kda_paged_attention_workspace_size.restype = ctypes.c_size_t
        L.kda_paged_attention_workspace_size.argtypes = [KP, i32, i64, i32, i32]
        L.kda_paged_attention.restype = i32
        L.kda_paged_attention.argtypes = [KP, _P, i64, *cache, i64, *batch, i32, i32, _P, _P, _P, ctypes.c_size_t, _P]
        CP, SP, NP = ctypes.POINTER(ConvParams), ctypes.POINTER(SsmParams), ctypes.POINTER(NormParams)
        L.kda_causal_conv.restype = i32
        L.kda_causal_conv.argtypes = [CP, _P, i64, _P, _P, _P, i32, i64, _P, i64, _P, _P, _P, i32, _P]
        L.kda_ssm_params_init.restype = None
        L.kda_ssm_params_init.argtypes = [SP, i32, i32, i32, i32]
        L.kda_ssm_prefill_workspace_size.restype = ctypes.c_size_t
        L.kda_ssm_prefill_workspace_size.argtypes = [SP, i32, i64]
        rows = [SP, _P, i64, _P, i64, _P, i64, _P, i64, _P, _P, _P]
        L.kda_ssm_prefill.restype = i32
        L.kda_ssm_prefill.argtypes = rows + [_P, i32, i64, _P, i64, _P, _P, _P, ctypes.c_size_t, _P]
        L.kda_ssm_decode.restype = i32
        L.kda_ssm_decode.argtypes = rows + [i32, _P, i64, _P, _P, _P]
        L.kda_group_norm.restype = i32
        L.kda_group_norm.argtypes = [NP, _P, i64, _P, i64, _P, _P, i64, _P, _P]
        _lib = L
        return L


def status_string(status: int) -> str:
    try:
        return lib().kda_status_string(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return KDA_F32
    if dt == torch.bfloat16:
        return KDA_BF16
    raise TypeError(f"unsupported dtype {dt}")


def make_params(num_heads: int, head_dim: int, io_dtype=torch.bfloat16, out_dtype=None,
                gate: str = "kda", chunk_size: int = 64, lower_bound=None, scale=None,
                l2_eps: float = 1e-6, softplus_threshold: float = 20.0) -> Params:
    p = Params()
    lib().kda_params_init(ctypes.byref(p), int(num_heads), int(head_dim))
    p.io_dtype = _dtype_code(io_dtype)
    p.out_dtype = _dtype_code(io_dtype if out_dtype is None else out_dtype)
    p.gate_kind = GATE_PER_CHANNEL if gate == "kda" else GATE_PER_HEAD
    p.chunk_size = int(chunk_size)
    p.use_lower_bound = 0 if lower_bound is None else 1
    p.lower_bound = 0.0 if lower_bound is None else float(lower_bound)
    p.scale = 0.0 if scale is None else float(scale)
    p.l2_eps = float(l2_eps)
    p.softplus_threshold = float(softplus_threshold)
    return p


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


# The current device: kernels are launched there, whatever the tensors' device, so the two must agree.
_device = torch._C._cuda_getDevice


def _dev(t, name, dtype=None):
    if t is None:
        return
    at = t.get_device() if isinstance(t, torch.Tensor) else -1
    if at < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if at != _device():
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    elif stream.device_index != _device():
        raise ValueError(f"stream is of cuda:{stream.device_index}, the current device is cuda:{_device()}")
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, what: str):
    if rc != KDA_OK:
        raise KdaError(rc, what)


def prefill_workspace_size(params: Params, num_seqs: int, total_tokens: int) -> int:
    return int(lib().kda_chunk_prefill_workspace_size(ctypes.byref(params), int(num_seqs), int(total_tokens)))


PREFILL_PHASE_EVENTS = 4
PREFILL_PHASES = ("chunk_table", "chunk_intra", "chunk_state")


def chunk_prefill(q, k, v, g_raw, b_raw, A_log, dt_bias, cu_seqlens, state_pool, state_idx,
                  out=None, *, params: Params | None = None, workspace=None, stream=None,
                  events=None, chunk_states=None, **kw):
    """kda_chunk_prefill on torch tensors; returns ``out`` ([T, H, D]).  ``state_pool`` is
    updated in place.  ``kw`` are forwarded to :func:`make_params` when ``params`` is None.
    With ``events`` (4 recorded-once ``torch.cuda.Event``), kda_chunk_prefill_timed records them
    around the chunk-table, intra-chunk and state-pass kernels.  With ``chunk_states``
    ([num_chunks, H, D, D] fp32), kda_chunk_prefill_snapshots also writes the state after every
    chunk (chunks numbered by sequence, then position)."""
    T, H, D = q.shape
    if params is None:
        params = make_params(H, D, io_dtype=q.dtype, **kw)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    _dev(g_raw, "g_raw", torch.float32)
    _dev(b_raw, "b_raw", torch.float32)
    _dev(A_log, "A_log", torch.float32)
    _dev(dt_bias, "dt_bias", torch.float32)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    _dev(state_pool, "state_pool", torch.float32)
    _dev(state_idx, "state_idx", torch.int32)
    n = state_idx.numel()
    if out is None:
        out = torch.empty((T, H, D), device=q.device,
                          dtype=torch.float32 if params.out_dtype == KDA_F32 else torch.bfloat16)
    _dev(out, "out")
    need = prefill_workspace_size(params, n, T)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _dev(workspace, "workspace", torch.uint8)
    args = (ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(b_raw), _ptr(A_log),
            _ptr(dt_bias), _ptr(cu_seqlens), n, T, _ptr(state_pool), state_pool.shape[0], _ptr(state_idx),
            _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    if chunk_states is not None:
        if events is not None:
            raise ValueError("events and chunk_states cannot be combined")
        _dev(chunk_states, "chunk_states", torch.float32)
        rc = lib().kda_chunk_prefill_snapshots(*args[:-1], _ptr(chunk_states), chunk_states.shape[0], args[-1])
        _check(rc, "kda_chunk_prefill_snapshots")
        return out
    if events is None:
        rc = lib().kda_chunk_prefill(*args)
    else:
        if len(events) != PREFILL_PHASE_EVENTS:
            raise ValueError("events must hold 4 CUDA events")
        handles = (ctypes.c_void_p * PREFILL_PHASE_EVENTS)(*[ctypes.c_void_p(e.cuda_event) for e in events])
        rc = lib().kda_chunk_prefill_timed(*args, handles)
    _check(rc, "kda_chunk_prefill")
    return out


def recurrent_decode(q, k, v, g_raw, b_raw, A_log, dt_bias, state_pool, state_idx, out=None, *,
                     params: Params | None = None, stream=None, **kw):
    """kda_recurrent_decode: one token per request ([B, H, D] inputs); pool updated in place."""
    B, H, D = q.shape
    if params is None:
        params = make_params(H, D, io_dtype=q.dtype, **kw)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    for name, t in (("g_raw", g_raw), ("b_raw", b_raw), ("A_log", A_log), ("dt_bias", dt_bias),
                    ("state_pool", state_pool)):
        _dev(t, name, torch.float32)
    _dev(state_idx, "state_idx", torch.int32)
    if out is None:
        out = torch.empty((B, H, D), device=q.device,
                          dtype=torch.float32 if params.out_dtype == KDA_F32 else torch.bfloat16)
    _dev(out, "out")
    rc = lib().kda_recurrent_decode(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw),
                                    _ptr(b_raw), _ptr(A_log), _ptr(dt_bias), B, _ptr(state_pool),
                                    state_pool.shape[0], _ptr(state_idx), _ptr(out), _stream(stream))
    _check(rc, "kda_recurrent_decode")
    return out


def recurrent_verify(q, k, v, g_raw, b_raw, A_log, dt_bias, state_pool, state_idx, t_draft,
                     inter=None, out=None, *, params: Params | None = None, stream=None, **kw):
    """kda_recurrent_verify: ``t_draft`` tokens per request (request-major rows).  Returns
    ``(out, inter)`` with inter [B, t_draft, H, D, D] fp32; the pool is not modified."""
    TT, H, D = q.shape
    B = state_idx.numel()
    if TT != B * t_draft:
        raise ValueError("q must hold batch * t_draft rows")
    if params is None:
        params = make_params(H, D, io_dtype=q.dtype, **kw)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    for name, t in (("g_raw", g_raw), ("b_raw", b_raw), ("A_log", A_log), ("dt_bias", dt_bias),
                    ("state_pool", state_pool)):
        _dev(t, name, torch.float32)
    _dev(state_idx, "state_idx", torch.int32)
    if inter is None:
        inter = torch.empty((B, t_draft, H, D, D), device=q.device, dtype=torch.float32)
    if out is None:
        out = torch.empty((TT, H, D), device=q.device,
                          dtype=torch.float32 if params.out_dtype == KDA_F32 else torch.bfloat16)
    _dev(inter, "inter", torch.float32)
    _dev(out, "out")
    rc = lib().kda_recurrent_verify(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw),
                                    _ptr(b_raw), _ptr(A_log), _ptr(dt_bias), B, int(t_draft),
                                    _ptr(state_pool), state_pool.shape[0], _ptr(state_idx),
                                    _ptr(inter), _ptr(out), _stream(stream))
    _check(rc, "kda_recurrent_verify")
    return out, inter


def replay_rings(num_slots, num_heads, head_dim, ring_len, gate="kda", device="cuda"):
    """Allocate zeroed ReplaySSM rings (d, k, a) for kda_replay_decode."""
    d = torch.zeros(num_slots, num_heads, ring_len, head_dim, device=device)
    k = torch.zeros_like(d)
    a = torch.zeros_like(d) if gate == "kda" else torch.zeros(num_slots, num_heads, ring_len, device=device)
    return d, k, a


def replay_decode(q, k, v, g_raw, b_raw, A_log, dt_bias, state_pool, state_idx, rings, write_pos,
                  force_flush=None, out=None, *, params: Params | None = None, stream=None, **kw):
    """kda_replay_decode: one token per request against checkpoint + ring.  ``rings`` is the
    (ring_d, ring_k, ring_a) triple; ``write_pos`` [B] int32 is not advanced here."""
    B, H, D = q.shape
    ring_d, ring_k, ring_a = rings
    if params is None:
        params = make_params(H, D, io_dtype=q.dtype, **kw)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    for name, t in (("g_raw", g_raw), ("b_raw", b_raw), ("A_log", A_log), ("dt_bias", dt_bias),
                    ("state_pool", state_pool), ("ring_d", ring_d), ("ring_k", ring_k), ("ring_a", ring_a)):
        _dev(t, name, torch.float32)
    _dev(state_idx, "state_idx", torch.int32)
    _dev(write_pos, "write_pos", torch.int32)
    _dev(force_flush, "force_flush", torch.int32)
    if out is None:
        out = torch.empty((B, H, D), device=q.device,
                          dtype=torch.float32 if params.out_dtype == KDA_F32 else torch.bfloat16)
    _dev(out, "out")
    rc = lib().kda_replay_decode(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(b_raw),
                                 _ptr(A_log), _ptr(dt_bias), B, _ptr(state_pool), state_pool.shape[0],
                                 _ptr(state_idx), _ptr(ring_d), _ptr(ring_k), _ptr(ring_a), ring_d.shape[2],
                                 _ptr(write_pos), _ptr(force_flush), _ptr(out), _stream(stream))
    _check(rc, "kda_replay_decode")
    return out


def commit_verified_states(inter, accept_len, state_pool, state_idx, *, params: Params | None = None,
                           stream=None, **kw):
    """kda_commit_verified_states: copy inter[b, accept_len[b] - 1] into each accepted slot."""
    B, Td, H, D, _ = inter.shape
    if params is None:
        params = make_params(H, D, **kw)
    _dev(inter, "inter", torch.float32)
    _dev(accept_len, "accept_len", torch.int32)
    _dev(state_pool, "state_pool", torch.float32)
    _dev(state_idx, "state_idx", torch.int32)
    rc = lib().kda_commit_verified_states(ctypes.byref(params), _ptr(inter), B, Td, _ptr(accept_len),
                                          _ptr(state_pool), state_pool.shape[0], _ptr(state_idx), _stream(stream))
    _check(rc, "kda_commit_verified_states")
    return state_pool


# ---- the paged key/value cache and its attention ------------------------------------------------------

class KVCache(NamedTuple):
    """A paged cache: ``k`` and ``v`` [pages, kv heads, page size, head_dim] bf16, or uint8 with two
    4-bit channels a byte (last dimension head_dim / 2) and e4m3 scales [.., head_dim / 16].  Wherever
    a cache is taken, a plain (k, v, k_scale, v_scale) tuple will do."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None


def _is_fp4(dtype) -> bool:
    if dtype not in ("bf16", "fp4"):
        raise ValueError(f"dtype must be 'bf16' or 'fp4', got {dtype!r}")
    return dtype == "fp4"


def kv_cache(num_pages, num_kv_heads, page_size, head_dim, dtype="bf16", device="cuda") -> KVCache:
    """Allocate a zeroed cache; ``dtype`` "bf16" or "fp4"."""
    shape = (int(num_pages), int(num_kv_heads), int(page_size))
    if not _is_fp4(dtype):
        k = torch.zeros(*shape, int(head_dim), dtype=torch.bfloat16, device=device)
        return KVCache(k, torch.zeros_like(k))
    k = torch.zeros(*shape, head_dim // 2, dtype=torch.uint8, device=device)
    s = torch.zeros(*shape, head_dim // 16, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    return KVCache(k, torch.zeros_like(k), s, s.clone())


def rope_table(num_positions, rot_dim, theta=10000.0, device="cuda") -> torch.Tensor:
    """Rotation table [num_positions, rot_dim] fp32 for :func:`kv_append`: cos(p f_i), then sin(p f_i),
    f_i = theta^(-2i / rot_dim).  The angles are taken in fp64 and the entries kept to 16 significant
    bits (off by at most 2^-16 relative, far below the 2^-8 of the bf16 result), so that a product with a
    bf16 value is exact in fp32."""
    f = float(theta) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(num_positions, dtype=torch.float64, device=device)[:, None] * f
    m, e = torch.frexp(torch.cat([a.cos(), a.sin()], 1))
    return torch.ldexp(torch.round(m * 65536.0), e - 16).float().contiguous()


_TOP = 2 ** 31 - 1


def _clip(x):
    """x as an int32 argument.  ctypes would take it modulo 2^32; all numbers past either end mean the same here:
    more than any length, or an error."""
    return x if -_TOP <= x <= _TOP else _TOP if x > 0 else -_TOP


@functools.lru_cache(maxsize=256)
def _kv_params(Hq, Hkv, D, page, fp4, rot=0, interleaved=False, window=0, sinks=0, scale=None):
    p = KvParams(_clip(Hq), _clip(Hkv), _clip(D), _clip(page), CACHE_FP4 if fp4 else CACHE_BF16, _clip(rot), 1 if interleaved else 0,
                 _clip(window), _clip(sinks), 0.0 if scale is None else scale)
    return ctypes.byref(p)


# The calls below take a few microseconds, and a decode step makes them once a layer, so each argument is
# first looked at in one expression; only one that fails it goes through the checks that say what is wrong.
_BF16, _F32, _I32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn


def _need(t, name, dtype, dev):
    if not (t.dtype is dtype and t.get_device() == dev and t.is_contiguous()):
        _dev(t, name, dtype)
        raise ValueError(f"{name} must be on cuda:{dev}, with the cache")


def _kv_cache_args(cache):
    """(device, kv heads, page size, head_dim, 4-bit?, k, v, k_scale and v_scale pointers, pages)."""
    k, v, ks, vs = cache
    fp4 = k.dtype is _U8
    if not fp4 and k.dtype is not _BF16:
        raise TypeError(f"cache.k must be torch.bfloat16 or torch.uint8 (4 bits), got {k.dtype}")
    dev = k.get_device()
    if dev < 0:
        raise ValueError("cache.k must be a CUDA tensor")
    _need(k, "cache.k", k.dtype, dev)
    _need(v, "cache.v", k.dtype, dev)
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("cache.k and cache.v must be [pages, kv heads, page size, channels], of one shape")
    pages, Hkv, page, D = shape
    if not fp4:
        return dev, Hkv, page, D, False, k.data_ptr(), v.data_ptr(), None, None, pages
    for name, t in (("cache.k_scale", ks), ("cache.v_scale", vs)):
        if t is None:
            raise ValueError(f"{name} is missing")
        if t.dtype is not _E4M3 and t.dtype is not _U8:
            raise TypeError(f"{name} must be torch.float8_e4m3fn, got {t.dtype}")
        _need(t, name, t.dtype, dev)
        if t.shape != (pages, Hkv, page, D // 8):
            raise ValueError(f"{name} must be [pages, kv heads, page size, head_dim / 16]")
    return dev, Hkv, page, 2 * D, True, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages


def _kv_batch(cu_seqlens, kv_lens, block_table, T, dev):
    """(cu_seqlens, kv_lens, block_table pointers, requests, pages per request, tokens)."""
    _need(kv_lens, "kv_lens", _I32, dev)
    _need(block_table, "block_table", _I32, dev)
    n, shape = kv_lens.numel(), block_table.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError("block_table must be [requests, pages per request], with one entry of kv_lens per request")
    if cu_seqlens is None:
        if T != n:
            raise ValueError("without cu_seqlens there is one token per request")
        return None, kv_lens.data_ptr(), block_table.data_ptr(), n, shape[1], T
    _need(cu_seqlens, "cu_seqlens", _I32, dev)
    if cu_seqlens.numel() != n + 1:
        raise ValueError("cu_seqlens must have one entry more than kv_lens")
    if n == 0 and T > 0:
        raise ValueError("tokens without a request")           # the library would leave their outputs unwritten
    return cu_seqlens.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), n, shape[1], T


def _rows(t, name, heads, D, dev):
    """Pointer, token stride, tokens and heads of a bf16 [T, heads, D] tensor whose heads are contiguous (a
    slice of a fused projection will do)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on cuda:{dev}, with the cache")
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != D or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {D}], got {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1] * D, shape[0], shape[1]
    s = t.stride()
    if s[2] != 1 or (s[1] != D and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), s[0], shape[0], shape[1]


@functools.lru_cache(maxsize=None)
def _fn(name):
    """An entry point of the loaded library."""
    return getattr(lib(), name)


def _raw_stream(dev):
    """The current stream of the call's device, which has to be the current one."""
    if dev != _device():
        raise ValueError(f"the cache is on cuda:{dev}, the current device is cuda:{_device()}")
    return torch._C._cuda_getCurrentRawStream(dev)


def kv_append(k, v, cache, block_table, kv_lens, cu_seqlens=None, *, q=None, q_out=None, rope=None,
              interleaved=False, positions=None, stream=None):
    """kda_kv_append: write the new tokens' keys and values ([T, kv heads, D] bf16) into the cache, the
    keys rotated by the table ``rope`` ([positions, rot_dim], see :func:`rope_table`; None: no rotation).
    With ``q`` ([T, q heads, D]) returns it rotated (into ``q_out``, which may be ``q``)."""
    if stream is not None:                                    # what the call allocates belongs to its stream
        with torch.cuda.stream(stream):
            return kv_append(k, v, cache, block_table, kv_lens, cu_seqlens, q=q, q_out=q_out, rope=rope,
                             interleaved=interleaved, positions=positions)
    dev, Hkv, page, D, fp4, pk, pv, pks, pvs, pages = _kv_cache_args(cache)
    kp, k_stride, T, _ = _rows(k, "k", Hkv, D, dev)
    vp, v_stride, Tv, _ = _rows(v, "v", Hkv, D, dev)
    if Tv != T:
        raise ValueError("k and v must have the same number of tokens")
    pc, pl, pt, n, max_pages, _ = _kv_batch(cu_seqlens, kv_lens, block_table, T, dev)
    rot, rows, rp = 0, 0, None
    if rope is not None:
        _need(rope, "rope", _F32, dev)
        if rope.dim() != 2:
            raise ValueError("rope must be [positions, rot_dim]")
        rows, rot = rope.shape
        rp = rope.data_ptr()
    if positions is not None:
        _need(positions, "positions", _I32, dev)
        if positions.shape != (T,):
            raise ValueError("positions must hold one entry per token")
        positions = positions.data_ptr()
    Hq, qp, q_stride, qo = Hkv, None, 0, None
    if q is not None:
        qp, q_stride, Tq, Hq = _rows(q, "q", None, D, dev)
        if Tq != T:
            raise ValueError("q and k must have the same number of tokens")
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=_BF16, device=q.device)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
        else:
            _need(q_out, "q_out", _BF16, dev)
        qo = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = _fn("kda_kv_append")(_kv_params(Hq, Hkv, D, page, fp4, rot, interleaved), qp, q_stride, kp, k_stride, vp, v_stride,
                              rp, rows, positions, pc, pl, pt, n, max_pages, T, pk, pv, pks, pvs, pages, qo,
                              _raw_stream(dev))
    if rc:
        _check(rc, "kda_kv_append")
    return q_out


def kv_read(cache, block_table, kv_lens, cu_seqlens=None, *, num_tokens=None, out=None, stream=None):
    """kda_kv_read: the last tokens of each request, as many as ``cu_seqlens`` gives it (None: one each),
    as bf16 (k, v) [T, kv heads, D].  ``num_tokens`` = cu_seqlens[-1] is needed with ``cu_seqlens``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_read(cache, block_table, kv_lens, cu_seqlens, num_tokens=num_tokens, out=out)
    dev, Hkv, page, D, fp4, pk, pv, pks, pvs, pages = _kv_cache_args(cache)
    T = kv_lens.numel() if cu_seqlens is None else num_tokens
    if T is None:
        raise ValueError("num_tokens is needed with cu_seqlens")
    batch = _kv_batch(cu_seqlens, kv_lens, block_table, int(T), dev)
    if out is None:
        k_out = torch.empty((T, Hkv, D), dtype=_BF16, device=kv_lens.device)
        out = k_out, torch.empty_like(k_out)
    else:
        for name, t in (("out[0]", out[0]), ("out[1]", out[1])):
            _need(t, name, _BF16, dev)
            if t.shape != (T, Hkv, D):
                raise ValueError(f"{name} must be [{T}, {Hkv}, {D}]")
    rc = _fn("kda_kv_read")(_kv_params(Hkv, Hkv, D, page, fp4), pk, pv, pks, pvs, pages, *batch, out[0].data_ptr(),
                            out[1].data_ptr(), _raw_stream(dev))
    if rc:
        _check(rc, "kda_kv_read")
    return out


@functools.lru_cache(maxsize=4096)
def _attention_workspace(p, n, T, max_new, max_len):
    return int(lib().kda_paged_attention_workspace_size(p, _clip(n), T, _clip(max_new), _clip(max_len)))


def paged_attention(q, cache, block_table, kv_lens, cu_seqlens=None, *, window=0, sinks=0, scale=None,
                    max_new=None, max_len=None, out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """kda_paged_attention: ``q`` [T, q heads, D] bf16 over the cache; returns ``out`` (or ``(out, lse)``).

    ``window`` 0: all tokens up to a query's own; w: the last w of them and the first ``sinks``.
    ``max_new`` bounds the new tokens of a request (default: all T; 1 without ``cu_seqlens``), ``max_len``
    bounds kv_lens (default: what block_table can hold): host numbers, the tighter the better."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return paged_attention(q, cache, block_table, kv_lens, cu_seqlens, window=window, sinks=sinks, scale=scale,
                                   max_new=max_new, max_len=max_len, out=out, lse=lse, return_lse=return_lse,
                                   workspace=workspace)
    dev, Hkv, page, D, fp4, pk, pv, pks, pvs, pages = _kv_cache_args(cache)
    qp, q_stride, T, Hq = _rows(q, "q", None, D, dev)
    batch = _kv_batch(cu_seqlens, kv_lens, block_table, T, dev)
    if max_new is None or cu_seqlens is None:
        max_new = 1 if cu_seqlens is None else max(T, 1)
    if max_len is None:
        max_len = batch[4] * page
    if out is None:
        out = torch.empty((T, Hq, D), dtype=_BF16, device=q.device)
    else:
        _need(out, "out", _BF16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    if lse is not None:
        _need(lse, "lse", _F32, dev)
        if lse.shape != (T, Hq):
            raise ValueError("lse must be [tokens, q heads]")
    elif return_lse:
        lse = torch.empty((T, Hq), dtype=_F32, device=q.device)
    p = _kv_params(Hq, Hkv, D, page, fp4, 0, False, window, sinks, None if scale is None else float(scale))
    need = _attention_workspace(p, batch[3], T, max_new, max_len)
    ws = None
    if workspace is not None:
        _need(workspace, "workspace", _U8, dev)
        need = workspace.numel()
    elif need:
        workspace = torch.empty(need, dtype=_U8, device=q.device)
    if workspace is not None:
        ws = workspace.data_ptr()
    rc = _fn("kda_paged_attention")(p, qp, q_stride, pk, pv, pks, pvs, pages, *batch, _clip(max_new), _clip(max_len), out.data_ptr(),
                                    None if lse is None else lse.data_ptr(), ws, need, _raw_stream(dev))
    if rc:
        _check(rc, "kda_paged_attention")
    return out if lse is None else (out, lse)


def attention_workspace_size(num_q_heads, num_kv_heads, head_dim, page_size, num_seqs, num_tokens, max_new, max_len, *,
                             dtype="bf16", window=0, sinks=0) -> int:
    """Bytes of ``workspace`` that :func:`paged_attention` needs for these sizes (it allocates them itself
    when none is given)."""
    p = _kv_params(num_q_heads, num_kv_heads, head_dim, page_size, _is_fp4(dtype), 0, False, window, sinks)
    return _attention_workspace(p, num_seqs, num_tokens, max_new, max_len)


# ---- around a recurrence: short convolution, selective recurrence, group norm ---------------------------

_CODES = {_F32: KDA_F32, _BF16: KDA_BF16}
_ACTIVATIONS = {None: 0, "silu": 1, "sigmoid": 2}


def _code(dtype, name):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")
    return code


def _tokens(t, name, shape, dtype, dev):
    """Pointer and token stride of a [T, ...] tensor of which one token's values are contiguous (a slice of a fused
    projection will do).  ``shape``: what follows T."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on cuda:{dev}, with x")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape[1:] != shape:
        raise ValueError(f"{name} must be [tokens, {', '.join(map(str, shape))}], got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), math.prod(shape)
    s, n = t.stride(), 1
    for i in range(len(shape), 0, -1):
        if shape[i - 1] > 1 and s[i] != n:
            raise ValueError(f"{name}: the values of a token must be contiguous")
        n *= shape[i - 1]
    if t.shape[0] > 1 and s[0] < n:
        raise ValueError(f"{name}: the rows of two tokens overlap")
    return t.data_ptr(), max(s[0], n)


def _need_with_x(t, name, dtype, dev, shape):
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    _dev(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, with x")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _here(t, name):
    """The device of x, which has to be the current one."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_device()}")
    return dev


@functools.lru_cache(maxsize=256)
def _conv_params(C, W, code, act):
    return ctypes.byref(ConvParams(_clip(C), _clip(W), code, act))


@functools.lru_cache(maxsize=256)
def _conv_split(parts, C):
    """(channel counts as the library takes them, type of its array of pointers)."""
    if not 1 <= len(parts) <= 4 or min(parts) < 1 or sum(parts) != C:
        raise ValueError(f"split must be one to four channel counts with the sum {C}, got {parts}")
    return (ctypes.c_int32 * len(parts))(*(_clip(n) for n in parts)), ctypes.c_void_p * len(parts)


def causal_conv(x, weight, state_pool, state_idx, cu_seqlens=None, *, bias=None, activation=None, split=None, out=None, stream=None):
    """kda_causal_conv: short causal convolution of each channel of ``x`` ([T, C] bf16 or fp32, rows may be strided) with
    ``weight`` ([C, W] fp32, W 2 to 4); ``activation`` None or "silu".  ``state_pool`` ([slots, W - 1, C], the type of x)
    holds each request's last inputs and is updated in place; without ``cu_seqlens`` there is one token per request.

    Returns [T, C], or with ``split`` (channel counts, up to four) a tuple of contiguous [T, n]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return causal_conv(x, weight, state_pool, state_idx, cu_seqlens, bias=bias, activation=activation, split=split, out=out)
    dev = _here(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [tokens, channels]")
    T, C = shape
    dtype = x.dtype
    code = _code(dtype, "x")
    if x.is_contiguous():
        xp, x_stride = x.data_ptr(), C
    else:
        xp, x_stride = _tokens(x, "x", shape[1:], dtype, dev)
    if weight.dim() != 2:
        raise ValueError(f"weight must be [{C}, width]")
    W = weight.shape[1]
    wp = _need_with_x(weight, "weight", _F32, dev, (C, W))
    bp = None if bias is None else _need_with_x(bias, "bias", _F32, dev, (C,))
    if state_pool.dim() != 3:
        raise ValueError(f"state_pool must be [slots, {W - 1}, {C}]")
    slots = state_pool.shape[0]
    pool = _need_with_x(state_pool, "state_pool", dtype, dev, (slots, W - 1, C))
    n = state_idx.numel()
    idx = _need_with_x(state_idx, "state_idx", _I32, dev, (n,))
    cu = None
    if cu_seqlens is not None:
        cu = _need_with_x(cu_seqlens, "cu_seqlens", _I32, dev, (n + 1,))
        if n == 0 and T > 0:
            raise ValueError("tokens without a request")
    elif T != n:
        raise ValueError("without cu_seqlens there is one token per request")
    act = _ACTIVATIONS.get(activation, -1)
    if act < 0 or act > 1:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    parts = (C,) if split is None else tuple(split)
    counts, pointers = _conv_split(parts, C)
    if out is None:
        device = x.device
        outs = [torch.empty((T, m), dtype=dtype, device=device) for m in parts]
    else:
        outs = [out] if split is None else list(out)
        if len(outs) != len(parts):
            raise ValueError("out must have one tensor per part")
        for i, (o, m) in enumerate(zip(outs, parts)):
            _need_with_x(o, f"out[{i}]", dtype, dev, (T, m))
    rc = _fn("kda_causal_conv")(_conv_params(C, W, code, act), xp, x_stride, wp, bp, cu, n, T, pool, slots, idx,
                                pointers(*[o.data_ptr() for o in outs]), counts, len(parts), torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "kda_causal_conv")
    return outs[0] if split is None else tuple(outs)


@functools.lru_cache(maxsize=256)
def _ssm_params(H, P, N, G, io, dt, out, threshold):
    return ctypes.byref(SsmParams(_clip(H), _clip(P), _clip(N), _clip(G), io, dt, out, threshold))


@functools.lru_cache(maxsize=4096)
def _ssm_workspace(p, n, T, dev):
    """For device `dev`, which is the current one: requests are cut by its number of SMs."""
    return int(lib().kda_ssm_prefill_workspace_size(p, _clip(n), T))


def ssm_prefill_workspace_size(num_heads, head_dim, state_dim, num_groups, num_seqs, num_tokens, *, dtype=torch.bfloat16,
                               out_dtype=None) -> int:
    """Bytes of ``workspace`` that :func:`ssm_prefill` needs for these sizes on the current device (it allocates them itself
    when none is given)."""
    io = _code(dtype, "dtype")
    p = _ssm_params(num_heads, head_dim, state_dim, num_groups, io, KDA_F32, io if out_dtype is None else _code(out_dtype, "out_dtype"), 20.0)
    return _ssm_workspace(p, num_seqs, num_tokens, _device() if torch.cuda.is_available() else -1)


def _ssm_args(x, dt, B, C, A_log, state_pool, state_idx, dt_bias, D, out, out_dtype, threshold):
    """(device, params, the entry points' shared pointers, requests, pool, slots, indices, out)."""
    dev = _here(x, "x")
    shape, b_shape = x.shape, B.shape
    if len(shape) != 3 or len(b_shape) != 3:
        raise ValueError("x must be [tokens, heads, head_dim], B and C [tokens, groups, states]")
    T, H, P = shape
    _, G, N = b_shape
    dtype = x.dtype
    code = _code(dtype, "x")
    xp, xs = _tokens(x, "x", shape[1:], dtype, dev)
    bp, bs = _tokens(B, "B", b_shape[1:], dtype, dev)
    cp, cs = _tokens(C, "C", b_shape[1:], dtype, dev)
    dt_code = _code(dt.dtype, "dt")
    dp, ds = _tokens(dt, "dt", (H,), dt.dtype, dev)
    if not T == b_shape[0] == C.shape[0] == dt.shape[0]:
        raise ValueError("x, dt, B and C must have the same number of tokens")
    heads = (H,)
    al = _need_with_x(A_log, "A_log", _F32, dev, heads)
    db = None if dt_bias is None else _need_with_x(dt_bias, "dt_bias", _F32, dev, heads)
    dd = None if D is None else _need_with_x(D, "D", _F32, dev, heads)
    if state_pool.dim() != 4:
        raise ValueError(f"state_pool must be [slots, {H}, {P}, {N}]")
    slots = state_pool.shape[0]
    pool = _need_with_x(state_pool, "state_pool", _F32, dev, (slots, H, P, N))
    n = state_idx.numel()
    idx = _need_with_x(state_idx, "state_idx", _I32, dev, (n,))
    if out is None:
        out_dtype = dtype if out_dtype is None else out_dtype
        out_code = _code(out_dtype, "out_dtype")
        out = torch.empty((T, H, P), dtype=out_dtype, device=x.device)
    else:
        out_code = _code(out.dtype, "out")
        _need_with_x(out, "out", out.dtype, dev, (T, H, P))
    p = _ssm_params(H, P, N, G, code, dt_code, out_code, float(threshold))
    return dev, T, p, (p, xp, xs, dp, ds, bp, bs, cp, cs, al, db, dd), n, (pool, slots, idx, out.data_ptr()), out


def ssm_prefill(x, dt, B, C, A_log, cu_seqlens, state_pool, state_idx, *, dt_bias=None, D=None, out=None, out_dtype=None,
                softplus_threshold=20.0, workspace=None, stream=None):
    """kda_ssm_prefill: selective state space recurrence over packed prompts.  ``x`` [T, H, P], ``B``, ``C`` [T, G, N] (bf16
    or fp32), ``dt`` [T, H] (bf16 or fp32, before softplus); rows may be strided.  ``state_pool`` [slots, H, P, N] fp32
    is updated in place.  Returns ``out`` [T, H, P]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_prefill(x, dt, B, C, A_log, cu_seqlens, state_pool, state_idx, dt_bias=dt_bias, D=D, out=out, out_dtype=out_dtype,
                               softplus_threshold=softplus_threshold, workspace=workspace)
    dev, T, p, rows, n, state, out = _ssm_args(x, dt, B, C, A_log, state_pool, state_idx, dt_bias, D, out, out_dtype, softplus_threshold)
    cu = _need_with_x(cu_seqlens, "cu_seqlens", _I32, dev, (n + 1,))
    if n == 0 and T > 0:
        raise ValueError("tokens without a request")
    need, ws = _ssm_workspace(p, n, T, dev), None
    if workspace is not None:
        need = workspace.numel()
        ws = _need_with_x(workspace, "workspace", _U8, dev, (need,))
    elif need:
        workspace = torch.empty(need, dtype=_U8, device=x.device)
        ws = workspace.data_ptr()
    rc = _fn("kda_ssm_prefill")(*rows, cu, n, T, *state, ws, need, torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "kda_ssm_prefill")
    return out


def ssm_decode(x, dt, B, C, A_log, state_pool, state_idx, *, dt_bias=None, D=None, out=None, out_dtype=None,
               softplus_threshold=20.0, stream=None):
    """kda_ssm_decode: one token per request (row b is request b's), see :func:`ssm_prefill`."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_decode(x, dt, B, C, A_log, state_pool, state_idx, dt_bias=dt_bias, D=D, out=out, out_dtype=out_dtype,
                              softplus_threshold=softplus_threshold)
    dev, T, p, rows, n, state, out = _ssm_args(x, dt, B, C, A_log, state_pool, state_idx, dt_bias, D, out, out_dtype, softplus_threshold)
    if T != n:
        raise ValueError("there must be one token per request")
    rc = _fn("kda_ssm_decode")(*rows, n, *state, torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "kda_ssm_decode")
    return out


@functools.lru_cache(maxsize=256)
def _norm_params(G, n, io, out, act, first, center, eps):
    return ctypes.byref(NormParams(_clip(G), _clip(n), io, out, act, first, center, eps))


def group_norm(x, weight=None, bias=None, *, gate=None, activation=None, gate_first=False, center=True, eps=1e-5, out=None,
               out_dtype=None, stream=None):
    """kda_group_norm: norm of each group of a token's channels.  ``x`` [T, G, n] (bf16 or fp32, rows may be strided),
    ``weight`` and ``bias`` [G, n] fp32 or None; ``center`` False: by the root mean square only.  ``activation`` None, "silu"
    or "sigmoid" is applied to the result, or with ``gate`` ([T, G, n], the type of the output) to the gate, which multiplies
    the result, or x before the norm (``gate_first``).  Returns ``out`` [T, G, n] (default: the type of x)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_norm(x, weight, bias, gate=gate, activation=activation, gate_first=gate_first, center=center, eps=eps, out=out,
                              out_dtype=out_dtype)
    dev = _here(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [tokens, groups, channels]")
    shape = x.shape
    T, G, n = shape
    code = _code(x.dtype, "x")
    xp, xs = _tokens(x, "x", shape[1:], x.dtype, dev)
    wp = None if weight is None else _need_with_x(weight, "weight", _F32, dev, shape[1:])
    bp = None if bias is None else _need_with_x(bias, "bias", _F32, dev, shape[1:])
    if out is None:
        out_dtype = x.dtype if out_dtype is None else out_dtype
        out_code = _code(out_dtype, "out_dtype")
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
    else:
        out_dtype = out.dtype
        out_code = _code(out_dtype, "out")
        _need_with_x(out, "out", out_dtype, dev, shape)
    gp, gs = None, 0
    if gate is not None:
        if gate.shape != shape:
            raise ValueError("gate must have the shape of x")
        gp, gs = _tokens(gate, "gate", shape[1:], out_dtype, dev)
    elif gate_first:
        raise ValueError("gate_first without gate")
    act = _ACTIVATIONS.get(activation, -1)
    if act < 0:
        raise ValueError(f"activation must be None, 'silu' or 'sigmoid', got {activation!r}")
    rc = _fn("kda_group_norm")(_norm_params(G, n, code, out_code, act, 1 if gate_first else 0, 1 if center else 0, float(eps)), xp, xs, gp, gs, wp, bp,
                               T, out.data_ptr(), torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "kda_group_norm")
    return out


def selftest_wait_timeout(polls: int, result=None, stream=None) -> None:
    """Enqueue the bounded-wait self-test (a wait that cannot complete; see kda.h).

    result: None or a device int32 tensor of 2 elements that receives (first wait completed,
    drain completed).  The timeout is then reported by check_device_errors() as code 3."""
    if result is not None:
        _dev(result, "result", torch.int32)
        if result.numel() < 2:
            raise ValueError("result must hold 2 int32 elements")
    rc = lib().kda_selftest_wait_timeout(int(polls), _ptr(result) if result is not None else None,
                                         _stream(stream))
    _check(rc, "kda_selftest_wait_timeout")


def check_device_errors(stream=None) -> int:
    """Synchronise and return the device error code recorded by the kernels (0 = none)."""
    code = ctypes.c_int32(0)
    rc = lib().kda_check_device_errors(_stream(stream), ctypes.byref(code))
    if rc not in (KDA_OK, -6):
        _check(rc, "kda_check_device_errors")
    return int(code.value)
