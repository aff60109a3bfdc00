"""ctypes binding of the C ABI in include/attn_jvp.h and include/attn_paged.h.

Argument marshalling only: shapes, strides and raw pointers of torch
tensors are handed to ``libattn_jvp.so``; every arithmetic step runs in its
CUDA kernels.  Outputs are allocated with torch (device memory plumbing).
CPU (host) inputs of the attention entry points are staged through the
device: the host->device copies, the kernel and the device->host copies all
run on the current stream.  (The rotation and the paged cache take CUDA
tensors only.)

There is no fallback: if the library is missing or the GPU is absent the
call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from array import array
from typing import Optional

import torch

from . import build as _build

EXPORTS = (
    "attn_fwd_jvp",
    "attn_fwd",
    "attn_fwd_jvp_f16",
    "attn_fwd_f16",
    "attn_fwd_f8",
    "attn_fwd_jvp_noalloc",
    "attn_bwd",
    "attn_bwd_f16",
    "attn_bwd_stages",
    "attn_sync_check",
    "attn_status_string",
    "attn_launch_count",
    "attn_set_wait_timeout_ns",
    "attn_debug_skip_first_load",
    "attn_rope",
    "attn_rope_f16",
    "attn_rope_freqs",
    "attn_rope_steps",
    "attn_paged_append",
    "attn_paged_append_f16",
    "attn_paged_decode",
    "attn_paged_decode_f16",
    "attn_paged_decode_workspace",
)

STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED",
          3: "ATTN_ERR_MISALIGNED", 4: "ATTN_ERR_CUDA", 5: "ATTN_ERR_TIMEOUT",
          6: "ATTN_ERR_PAGE"}


class AttnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("M", ctypes.c_int32),
                ("N", ctypes.c_int32), ("Dqk", ctypes.c_int32), ("Dv", ctypes.c_int32),
                ("T", ctypes.c_int64), ("max_seq_len", ctypes.c_int32)]


class AttnBias(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_int64 * 4),
                ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64 * 4)]


class AttnRopeSpec(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("out_scale", ctypes.c_float)]


class AttnRopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("H", ctypes.c_int32),
                ("x_stride", ctypes.c_int64 * 3), ("y_stride", ctypes.c_int64 * 3)]


class AttnRopeFreq(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("orig_len", ctypes.c_double), ("low_turns", ctypes.c_double),
                ("high_turns", ctypes.c_double)]


class AttnPagedCache(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("Dqk", ctypes.c_int32),
                ("Dv", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("seq_lens", ctypes.c_void_p)]


class AttnPagedNew(ctypes.Structure):
    # (attn_paged_append below writes it as 64-bit words, in this order)
    _fields_ = [("T", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("Hq", ctypes.c_int32),
                ("k_stride", ctypes.c_int64 * 2), ("v_stride", ctypes.c_int64 * 2), ("q_stride", ctypes.c_int64 * 2),
                ("q_out_stride", ctypes.c_int64 * 2)]


class AttnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_LIB = None


def lib() -> ctypes.CDLL:
    """Open the library (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with attention_forward_jvp_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.attn_fwd_jvp.restype = i32
    L.attn_fwd_jvp.argtypes = [ctypes.POINTER(AttnShape), vp, vp, vp, vp, vp, vp, vp,
                               ctypes.POINTER(AttnBias), i32, f32, vp, vp, vp, vp]
    L.attn_fwd_jvp_noalloc.restype = i32
    L.attn_fwd_jvp_noalloc.argtypes = L.attn_fwd_jvp.argtypes
    L.attn_fwd_jvp_f16.restype = i32
    L.attn_fwd_jvp_f16.argtypes = L.attn_fwd_jvp.argtypes
    L.attn_fwd.restype = i32
    L.attn_fwd.argtypes = [ctypes.POINTER(AttnShape), vp, vp, vp, vp,
                           ctypes.POINTER(AttnBias), i32, f32, vp, vp, vp]
    L.attn_fwd_f16.restype = i32
    L.attn_fwd_f16.argtypes = L.attn_fwd.argtypes
    L.attn_bwd.restype = i32
    L.attn_bwd.argtypes = [ctypes.POINTER(AttnShape), vp, vp, vp, vp, vp, vp, vp,
                           ctypes.POINTER(AttnBias), i32, f32, vp, vp, vp, vp, vp]
    L.attn_bwd_f16.restype = i32
    L.attn_bwd_f16.argtypes = L.attn_bwd.argtypes
    L.attn_bwd_stages.restype = i32
    L.attn_bwd_stages.argtypes = [ctypes.POINTER(AttnShape), vp, vp, vp, vp, vp, vp, vp,
                                  ctypes.POINTER(AttnBias), i32, f32, vp, vp, vp, vp, i32,
                                  ctypes.c_uint, vp]
    L.attn_fwd_f8.restype = i32
    L.attn_fwd_f8.argtypes = [ctypes.POINTER(AttnShape), vp, vp, vp, i32, f32, vp, vp, vp]
    L.attn_sync_check.restype = i32
    L.attn_sync_check.argtypes = [vp]
    L.attn_status_string.restype = ctypes.c_char_p
    L.attn_status_string.argtypes = [i32]
    L.attn_launch_count.restype = ctypes.c_uint64
    L.attn_launch_count.argtypes = []
    L.attn_set_wait_timeout_ns.restype = None
    L.attn_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    L.attn_debug_skip_first_load.restype = None
    L.attn_debug_skip_first_load.argtypes = [i32]
    i64, sz = ctypes.c_int64, ctypes.c_size_t
    for f in (L.attn_rope, L.attn_rope_f16):
        f.restype = i32
        f.argtypes = [ctypes.c_int32, i64, ctypes.c_int32, ctypes.POINTER(AttnRopeSpec), vp, ctypes.c_int32, vp, vp,
                      vp, ctypes.c_int32, i32, vp]
    L.attn_rope_freqs.restype = i32
    L.attn_rope_freqs.argtypes = [ctypes.POINTER(AttnRopeFreq), vp]
    L.attn_rope_steps.restype = i32
    L.attn_rope_steps.argtypes = [vp, ctypes.c_int32, vp]
    for f in (L.attn_paged_append, L.attn_paged_append_f16):
        f.restype = i32
        f.argtypes = [ctypes.POINTER(AttnPagedCache), vp, ctypes.POINTER(AttnRopeSpec), vp]
    L.attn_paged_decode_workspace.restype = sz
    L.attn_paged_decode_workspace.argtypes = [ctypes.POINTER(AttnPagedCache), ctypes.c_int32]
    for f in (L.attn_paged_decode, L.attn_paged_decode_f16):
        f.restype = i32
        f.argtypes = [ctypes.POINTER(AttnPagedCache), ctypes.c_int32, vp, vp, f32, vp, vp, vp, sz, vp]
    _LIB = L
    return L


def _check(status: int):
    if status != 0:
        raise AttnError(status, lib().attn_status_string(status).decode())


def status_string(status: int) -> str:
    return lib().attn_status_string(status).decode()


def launch_count() -> int:
    return int(lib().attn_launch_count())


def sync_check(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise and return the device error status (0 = ok)."""
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(lib().attn_sync_check(ctypes.c_void_p(s.cuda_stream)))


def set_wait_timeout_ns(ns: int):
    lib().attn_set_wait_timeout_ns(int(ns))


def debug_skip_first_load(enable: bool):
    lib().attn_debug_skip_first_load(1 if enable else 0)


def _elem_type(q: torch.Tensor):
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"inputs must be bfloat16 or float16, got {q.dtype}")
    return q.dtype


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, dev):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _need_out(t: torch.Tensor, name: str, shape, dtype, dev):
    """A caller-given output: the library writes its whole extent, so it
    must be exactly the shape, dtype and device the call produces, and
    contiguous."""
    _need(t, name, dtype, dev)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _describe(q, k, v, offsets, max_seq_len, bias, mask):
    """Shape struct + bias struct (with the tensors kept alive)."""
    sh = AttnShape()
    keep = []
    if offsets is None:
        if q.dim() != 4:
            raise ValueError("dense q must be [B, H, M, Dqk]")
        B, H, M, Dqk = q.shape
        N, Dv = k.shape[2], v.shape[3]
        if tuple(k.shape) != (B, H, N, Dqk) or tuple(v.shape) != (B, H, N, Dv):
            raise ValueError("k must be [B, H, N, Dqk] and v [B, H, N, Dv]")
        sh.B, sh.H, sh.M, sh.N, sh.Dqk, sh.Dv, sh.T, sh.max_seq_len = B, H, M, N, Dqk, Dv, 0, 0
        out_shape = (B, H, M, Dv)
    else:
        if q.dim() != 3:
            raise ValueError("jagged q must be [H, T, Dqk]")
        if max_seq_len is None:
            raise ValueError("jagged inputs need max_seq_len")
        H, T, Dqk = q.shape
        Dv = v.shape[2]
        if tuple(k.shape) != (H, T, Dqk) or tuple(v.shape) != (H, T, Dv):
            raise ValueError("k must be [H, T, Dqk] and v [H, T, Dv]")
        sh.B, sh.H, sh.M, sh.N, sh.Dqk, sh.Dv = offsets.numel() - 1, H, 0, 0, Dqk, Dv
        sh.T, sh.max_seq_len = T, int(max_seq_len)
        out_shape = (H, T, Dv)
    bs = None
    if bias is not None or mask is not None:
        if offsets is not None:
            raise ValueError("bias / mask are supported for dense inputs only")
        bs = AttnBias()
        full = (sh.B, sh.H, sh.M, sh.N)
        if bias is not None:
            if bias.dtype != torch.float32 or bias.device != q.device:
                raise TypeError("bias must be float32 on the inputs' device")
            be = bias.expand(full)
            bs.bias = be.data_ptr()
            bs.bias_stride = (ctypes.c_int64 * 4)(*be.stride())
            keep.append(be)
        if mask is not None:
            if mask.dtype == torch.bool:
                mask = mask.view(torch.uint8)
            if mask.dtype != torch.uint8 or mask.device != q.device:
                raise TypeError("mask must be bool/uint8 on the inputs' device")
            me = mask.expand(full)
            bs.mask = me.data_ptr()
            bs.mask_stride = (ctypes.c_int64 * 4)(*me.stride())
            keep.append(me)
    return sh, bs, out_shape, keep


def _scale(sm_scale):
    return float("nan") if sm_scale is None else float(sm_scale)


def attn_fwd_jvp(q, k, v, tq, tk, tv, causal: bool = False, sm_scale: Optional[float] = None,
                 offsets: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
                 bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                 out=None):
    """Attention forward + JVP in one pass.  Returns (o, to, lse).

    Dense: q, tq [B, H, M, Dqk]; k, tk [B, H, N, Dqk]; v, tv [B, H, N, Dv].
    Jagged: [H, T, D] with int32 ``offsets`` [B + 1] and ``max_seq_len``.
    ``bias`` (fp32) and ``mask`` (bool/uint8, True = attend) broadcast to
    [B, H, M, N].  CPU inputs are copied to the current CUDA device and the
    outputs copied back (the end-to-end path); CUDA inputs stay on device.
    """
    if q.device.type == "cpu":
        return _host_call(attn_fwd_jvp, (q, k, v, tq, tk, tv), dict(
            causal=causal, sm_scale=sm_scale, offsets=offsets, max_seq_len=max_seq_len,
            bias=bias, mask=mask), n_out=3)
    dev = q.device
    dt = _elem_type(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("tq", tq), ("tk", tk), ("tv", tv)):
        _need(t, name, dt, dev)
    if tq.shape != q.shape or tk.shape != k.shape or tv.shape != v.shape:
        raise ValueError("tangents must have the primals' shapes")
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, dev)
    sh, bs, out_shape, keep = _describe(q, k, v, offsets, max_seq_len, bias, mask)
    if out is None:
        o = torch.empty(out_shape, dtype=dt, device=dev)
        to = torch.empty(out_shape, dtype=dt, device=dev)
        lse = torch.empty(out_shape[:-1], dtype=torch.float32, device=dev)
    else:
        o, to, lse = out
        _need_out(o, "o", out_shape, dt, dev)
        _need_out(to, "to", out_shape, dt, dev)
        _need_out(lse, "lse", out_shape[:-1], torch.float32, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    fn = lib().attn_fwd_jvp_f16 if dt == torch.float16 else lib().attn_fwd_jvp
    st = fn(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(tq), _ptr(tk),
                            _ptr(tv), _ptr(offsets), ctypes.byref(bs) if bs is not None else None,
                            1 if causal else 0, _scale(sm_scale), _ptr(o), _ptr(to), _ptr(lse),
                            ctypes.c_void_p(stream))
    del keep
    _check(st)
    return o, to, lse


def attn_fwd(q, k, v, causal: bool = False, sm_scale: Optional[float] = None,
             offsets: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
             bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None, out=None):
    """Attention forward only.  Returns (o, lse)."""
    if q.device.type == "cpu":
        return _host_call(attn_fwd, (q, k, v), dict(
            causal=causal, sm_scale=sm_scale, offsets=offsets, max_seq_len=max_seq_len,
            bias=bias, mask=mask), n_out=2)
    dev = q.device
    dt = _elem_type(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, dt, dev)
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, dev)
    sh, bs, out_shape, keep = _describe(q, k, v, offsets, max_seq_len, bias, mask)
    if out is None:
        o = torch.empty(out_shape, dtype=dt, device=dev)
        lse = torch.empty(out_shape[:-1], dtype=torch.float32, device=dev)
    else:
        o, lse = out
        _need_out(o, "o", out_shape, dt, dev)
        _need_out(lse, "lse", out_shape[:-1], torch.float32, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    fn = lib().attn_fwd_f16 if dt == torch.float16 else lib().attn_fwd
    st = fn(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(offsets),
                        ctypes.byref(bs) if bs is not None else None, 1 if causal else 0,
                        _scale(sm_scale), _ptr(o), _ptr(lse), ctypes.c_void_p(stream))
    del keep
    _check(st)
    return o, lse


BWD_DELTA, BWD_DQ, BWD_DKDV, BWD_ALL = 1, 2, 4, 7


def attn_bwd(q, k, v, o, lse, do, causal: bool = False, sm_scale: Optional[float] = None,
             offsets: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
             bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
             out=None, stages: int = BWD_ALL):
    """Attention backward.  Takes the forward's inputs (with its ``bias`` /
    ``mask``, dense only; the bias gets no gradient), its output ``o`` and
    log-sum-exp ``lse`` and the gradient ``do`` of O; returns
    (dq, dk, dv, delta), delta = rowsum(do o o) in float32.  Dense
    ``[B, H, M|N, D]`` or jagged ``[H, T, D]`` with int32 ``offsets`` and
    ``max_seq_len`` (tokens past a sequence's cap get zero gradients).
    ``stages`` (an OR of BWD_DELTA, BWD_DQ, BWD_DKDV) runs a subset of the
    launches; the others leave their outputs as given."""
    if q.device.type == "cpu":
        return _host_call(attn_bwd, (q, k, v, o, lse, do),
                          dict(causal=causal, sm_scale=sm_scale, offsets=offsets,
                               max_seq_len=max_seq_len, bias=bias, mask=mask), n_out=4)
    dev = q.device
    dt = _elem_type(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _need(t, name, dt, dev)
    _need(lse, "lse", torch.float32, dev)
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, dev)
    sh, bs, out_shape, keep = _describe(q, k, v, offsets, max_seq_len, bias, mask)
    if tuple(o.shape) != out_shape or tuple(do.shape) != out_shape or tuple(lse.shape) != out_shape[:-1]:
        raise ValueError("o and do must be shaped like the forward's output and lse like its log-sum-exp")
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        delta = torch.empty(out_shape[:-1], dtype=torch.float32, device=dev)
    else:
        dq, dk, dv, delta = out
        _need_out(dq, "dq", q.shape, dt, dev)
        _need_out(dk, "dk", k.shape, dt, dev)
        _need_out(dv, "dv", v.shape, dt, dev)
        _need_out(delta, "delta", out_shape[:-1], torch.float32, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    if stages == BWD_ALL:
        fn = lib().attn_bwd_f16 if dt == torch.float16 else lib().attn_bwd
        st = fn(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(offsets),
                ctypes.byref(bs) if bs is not None else None, 1 if causal else 0, _scale(sm_scale),
                _ptr(dq), _ptr(dk), _ptr(dv), _ptr(delta), ctypes.c_void_p(stream))
    else:
        st = lib().attn_bwd_stages(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do),
                                   _ptr(lse), _ptr(offsets), ctypes.byref(bs) if bs is not None else None,
                                   1 if causal else 0, _scale(sm_scale),
                                   _ptr(dq), _ptr(dk), _ptr(dv), _ptr(delta),
                                   1 if dt == torch.float16 else 0, int(stages), ctypes.c_void_p(stream))
    del keep
    _check(st)
    return dq, dk, dv, delta


def attn_fwd_f8(q, k, vt, causal: bool = False, sm_scale: Optional[float] = None, out=None):
    """FP8 (e5m2) forward: q [B, H, M, D], k [B, H, N, D] and the transposed
    value vt [B, H, D, N], all torch.float8_e5m2.  Returns (o, lse): o e5m2
    [B, H, M, D], lse float32 [B, H, M]."""
    if q.device.type == "cpu":
        return _host_call(attn_fwd_f8, (q, k, vt), dict(causal=causal, sm_scale=sm_scale), n_out=2)
    dev = q.device
    dt = torch.float8_e5m2
    for name, t in (("q", q), ("k", k), ("vt", vt)):
        _need(t, name, dt, dev)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, M, D]")
    B, H, M, D = q.shape
    N = k.shape[2]
    if tuple(k.shape) != (B, H, N, D) or tuple(vt.shape) != (B, H, D, N):
        raise ValueError("k must be [B, H, N, D] and vt [B, H, D, N]")
    sh = AttnShape()
    sh.B, sh.H, sh.M, sh.N, sh.Dqk, sh.Dv, sh.T, sh.max_seq_len = B, H, M, N, D, D, 0, 0
    if out is None:
        o = torch.empty((B, H, M, D), dtype=dt, device=dev)
        lse = torch.empty((B, H, M), dtype=torch.float32, device=dev)
    else:
        o, lse = out
        _need_out(o, "o", (B, H, M, D), dt, dev)
        _need_out(lse, "lse", (B, H, M), torch.float32, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    st = lib().attn_fwd_f8(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(vt), 1 if causal else 0,
                           _scale(sm_scale), _ptr(o), _ptr(lse), ctypes.c_void_p(stream))
    _check(st)
    return o, lse


_STREAMS = {}


def _chunk_streams(dev, n=4):
    """Streams of the chunked host path (per device, created once)."""
    key = dev.index
    if key not in _STREAMS:
        _STREAMS[key] = [torch.cuda.Stream(dev) for _ in range(n)]
    return _STREAMS[key]


def _slab_chunks(fn, tensors, kw) -> int:
    """How many chunks of whole (batch, head) slabs the host path of a dense
    forward call is cut into: with at least 8 slabs, every tensor contiguous
    and every chunk boundary keeping the 16-byte alignment of the lse rows
    (M a multiple of 4), 4 when the inputs are 128 MB or more and 2 below
    (each chunk costs host time to issue; on a GB300 the copies of a step
    this small finish sooner in two chunks); else 1."""
    if fn not in (attn_fwd_jvp, attn_fwd):
        return 1
    if any(kw.get(k) is not None for k in ("offsets", "bias", "mask")):
        return 1
    q = tensors[0]
    if q.dim() != 4 or any(t.dim() != 4 or t.shape[:2] != q.shape[:2] or not t.is_contiguous()
                           for t in tensors):
        return 1
    if q.shape[0] * q.shape[1] < 8 or q.shape[2] % 4 != 0:
        return 1
    nbytes = sum(t.numel() * t.element_size() for t in tensors)
    return 4 if nbytes >= (128 << 20) else 2


def _host_call(fn, tensors, kw, n_out):
    """End-to-end path for host tensors: copy in, compute, copy out.

    A dense forward without bias or mask is cut into chunks of whole
    (batch, head) slabs, each an independent problem computed by its own
    call of the C entry point (the whole problem is validated once, then
    each chunk passes its slab pointers); a chunk's input copies, kernel and
    output copies run in order on a stream of its own, so the copies of one
    chunk overlap the kernel of another.  The results are those of one call
    over the whole batch."""
    dev = torch.device("cuda", torch.cuda.current_device())
    n = _slab_chunks(fn, tensors, kw)
    if n == 1:
        dt = [t.to(dev, non_blocking=True) for t in tensors]
        for key in ("offsets", "bias", "mask"):
            if kw.get(key) is not None:
                kw[key] = kw[key].to(dev, non_blocking=True)
        outs = fn(*dt, **kw)
        host = tuple(torch.empty(o.shape, dtype=o.dtype, pin_memory=True) for o in outs)
        for h, o in zip(host, outs):
            h.copy_(o, non_blocking=True)
        torch.cuda.current_stream(dev).synchronize()
        return host[:n_out]

    q, v = tensors[0], tensors[2]
    B, H, M = q.shape[0], q.shape[1], q.shape[2]
    S = B * H
    shapes = [(B, H, M, v.shape[3])] * (n_out - 1) + [(B, H, M)]
    dtypes = [q.dtype] * (n_out - 1) + [torch.float32]
    d_in = [torch.empty(t.shape, dtype=t.dtype, device=dev) for t in tensors]
    d_out = [torch.empty(sh, dtype=dt, device=dev) for sh, dt in zip(shapes, dtypes)]
    h_out = [torch.empty(sh, dtype=dt, pin_memory=True) for sh, dt in zip(shapes, dtypes)]

    def slab(t, a, b):  # slabs [a, b) of a [B, H, ...] tensor, as [1, b - a, ...]
        return t.view(S, *t.shape[2:])[a:b].view(1, b - a, *t.shape[2:])

    # the whole problem through the binding's checks once (shapes, dtypes,
    # devices), with no launch: the chunks below skip them
    jvp = fn is attn_fwd_jvp
    f16 = _elem_type(q) == torch.float16
    for name, t in zip(("q", "k", "v", "tq", "tk", "tv"), d_in):
        _need(t, name, q.dtype, dev)
    if jvp and (tensors[3].shape != q.shape or tensors[4].shape != tensors[1].shape
                or tensors[5].shape != v.shape):
        raise ValueError("tangents must have the primals' shapes")
    sh, _, _, _ = _describe(d_in[0], d_in[1], d_in[2], None, None, None, None)
    L = lib()
    cfn = (L.attn_fwd_jvp_f16 if f16 else L.attn_fwd_jvp) if jvp else (L.attn_fwd_f16 if f16 else L.attn_fwd)
    scale = _scale(kw.get("sm_scale"))
    causal = 1 if kw.get("causal") else 0
    per_in = [t.numel() // S * t.element_size() for t in d_in]      # bytes per slab
    per_out = [t.numel() // S * t.element_size() for t in d_out]
    cur = torch.cuda.current_stream(dev)
    streams = _chunk_streams(dev)
    for st in streams:
        st.wait_stream(cur)
    try:
        for c in range(n):
            a, b = S * c // n, S * (c + 1) // n
            st = streams[c % len(streams)]
            with torch.cuda.stream(st):
                for h, d in zip(tensors, d_in):
                    slab(d, a, b).copy_(slab(h, a, b), non_blocking=True)
                csh = AttnShape()
                csh.B, csh.H, csh.M, csh.N, csh.Dqk, csh.Dv = 1, b - a, sh.M, sh.N, sh.Dqk, sh.Dv
                pin = [ctypes.c_void_p(d.data_ptr() + a * pb) for d, pb in zip(d_in, per_in)]
                pout = [ctypes.c_void_p(o.data_ptr() + a * pb) for o, pb in zip(d_out, per_out)]
                # (q, k, v[, tq, tk, tv], offsets, bias, causal, scale, o[, to], lse, stream)
                _check(cfn(ctypes.byref(csh), *pin, None, None, causal, scale, *pout,
                           ctypes.c_void_p(st.cuda_stream)))
                for ho, o in zip(h_out, d_out):
                    slab(ho, a, b).copy_(slab(o, a, b), non_blocking=True)
    finally:
        # also when a chunk's call raises: no copy may still be running
        # when the device buffers are released
        for st in streams:
            st.synchronize()
    return tuple(h_out[:n_out])


# ------------------------------------------- rotary positions, paged cache


def _need_cuda(t: torch.Tensor, name: str, dtype, dev=None):
    """A CUDA tensor of this type (on this device), its last dimension contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dim() == 0:
        raise ValueError(f"{name} must have dimensions, got a single number")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _call_on(dev, fn, *args):
    """fn(*args, stream) with `dev` current; its status raised."""
    i = dev.index
    # (the handle alone: torch.cuda.current_stream builds an object around it,
    # at two thirds of the cost of the call)
    stream = torch._C._cuda_getCurrentRawStream(i)
    if torch._C._cuda_getDevice() == i:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != 0:
        _check(st)


_ROPE_SCALING = {None: 0, "linear": 1, "base": 2, "by_parts": 3}


class Rope:
    """A rotation by position: what a program keeps of its position encoding.

    Pair i of the first ``rot_dim`` elements of a head turns by
    ``p * inv_freq[i]`` at position p, with ``inv_freq[i] = base ** (-2 i /
    rot_dim)``; pairs are (i, i + rot_dim / 2), or (2i, 2i + 1) when
    ``interleaved``; the result is multiplied by ``out_scale``.  ``scaling``
    stretches the frequencies for contexts longer than those trained on:

      None        as they are
      "linear"    all divided by ``factor``
      "base"      the base times ``factor ** (rot_dim / (rot_dim - 2))``
      "by_parts"  divided by ``factor`` where a pair makes fewer than
                  ``low_turns`` turns over ``orig_len`` positions, kept where
                  it makes more than ``high_turns``, blended in between

    or ``inv_freq`` (rot_dim / 2 numbers, float64) gives them outright.
    ``inv_freq`` holds the frequencies (float64, CPU) and ``steps`` the
    device array of the kernels (turns per position times 2^64)."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: Optional[str] = None,
                 factor: float = 1.0, orig_len: float = 0, low_turns: float = 1.0, high_turns: float = 32.0,
                 out_scale: float = 1.0, inv_freq=None, device=None):
        rot_dim = int(rot_dim)
        if rot_dim <= 0 or rot_dim % 2:
            raise ValueError("rot_dim must be even and positive")
        if scaling not in _ROPE_SCALING:
            raise ValueError(f"scaling must be one of {list(_ROPE_SCALING)}, got {scaling!r}")
        if not math.isfinite(out_scale):
            raise ValueError("out_scale must be finite")
        if inv_freq is None:
            freq = AttnRopeFreq(rot_dim, _ROPE_SCALING[scaling], base, factor, orig_len, low_turns, high_turns)
            f = torch.empty(rot_dim // 2, dtype=torch.float64)
            _check(lib().attn_rope_freqs(ctypes.byref(freq), f.data_ptr()))
        else:
            if scaling is not None:
                raise ValueError("inv_freq gives the frequencies outright: no scaling with it")
            f = torch.as_tensor(inv_freq, dtype=torch.float64).detach().cpu().contiguous().clone()
            if tuple(f.shape) != (rot_dim // 2,):
                raise ValueError(f"inv_freq must hold {rot_dim // 2} numbers")
        steps = torch.empty(rot_dim // 2, dtype=torch.int64)
        _check(lib().attn_rope_steps(f.data_ptr(), rot_dim // 2, steps.data_ptr()))
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError(f"the rotation runs on a CUDA device, got {dev}")
        self.rot_dim, self.interleaved, self.out_scale = rot_dim, bool(interleaved), float(out_scale)
        self.inv_freq = f
        self.steps = steps.to(dev)
        self._spec = AttnRopeSpec(self.steps.data_ptr(), rot_dim, 1 if interleaved else 0, out_scale)
        self._ref = ctypes.byref(self._spec)


def attn_rope(tensors, rope: Rope, positions: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
              inverse: bool = False, out=None):
    """Rotate up to four tensors by position, in one launch.  Returns a tuple
    of them.

    Dense: [B, H, N, D], equal but for H (q, k, their tangents, or gradients
    with ``inverse``, which turns back: the transpose of the rotation).
    ``positions`` int32 [B, N] or [N], default 0 .. N - 1.  Jagged:
    [H, T, D] with int32 ``offsets`` [B + 1]; ``positions`` int32 [T],
    default the place in the sequence; rows at offsets[B] and behind are not
    written.  Any strides with contiguous rows of D (a transposed view of a
    [B, N, H, D] projection); rows on 16-byte boundaries with D and rot_dim
    multiples of 16 run at speed, others element by element.  ``out``: one
    tensor for each, of its own, or the input itself to rotate in place (a
    tensor given twice then is refused); by default new contiguous ones."""
    tensors = tuple(tensors)
    n = len(tensors)
    if not 1 <= n <= 4:
        raise ValueError("attn_rope takes one to four tensors")
    x0 = tensors[0]
    dev, dt, nd = x0.device, _elem_type(x0), x0.dim()
    jagged = offsets is not None
    if nd != (3 if jagged else 4):
        raise ValueError("tensors must be [B, H, N, D], or [H, T, D] with offsets")
    _need_cuda(x0, "every tensor", dt)
    s0 = x0.shape
    B, H0, N, D = (1, *s0) if jagged else s0
    if rope.rot_dim > D:
        raise ValueError(f"rot_dim {rope.rot_dim} exceeds the head dim {D}")
    if rope.steps.device != dev:
        raise ValueError(f"the rotation is on {rope.steps.device}, the tensors on {dev}")
    if out is not None:
        out = tuple(out)
        if len(out) != n:
            raise ValueError("out must hold one tensor for each input")
        for x, y in zip(tensors, out):
            _need_cuda(y, "out", dt, dev)
            if y.shape != x.shape:
                raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(y.shape)}")
    words = []  # of an array of AttnRopeTensor (H's upper half is padding; the hosts are little-endian)
    made = []
    for i, x in enumerate(tensors):
        xs, H = x.stride(), H0
        if x is not x0:
            if x.dtype is not dt or x.device != dev or xs[-1:] != (1,):
                _need_cuda(x, "every tensor", dt, dev)
            sx = x.shape
            if sx != s0 and (len(sx) != nd or sx[-2:] != s0[-2:] or (not jagged and sx[0] != B)):
                raise ValueError("the tensors must agree in all but their heads")
            H = sx[nd - 3]
        if out is None:
            if x.is_contiguous():
                y, ys = torch.empty_like(x), xs
            else:
                y = torch.empty(x.shape, dtype=dt, device=dev)
                ys = y.stride()
            made.append(y)
        else:
            y = out[i]
            ys = y.stride()
        if jagged:
            words += (x.data_ptr(), y.data_ptr(), H, 0, xs[0], xs[1], 0, ys[0], ys[1])
        else:
            words += (x.data_ptr(), y.data_ptr(), H, xs[0], xs[1], xs[2], ys[0], ys[1], ys[2])
    if out is None:
        out = tuple(made)
    arr = array("q", words)
    pos = ps = off = None
    n_seq = 0
    if positions is not None:
        if positions.dtype != torch.int32 or positions.device != dev:
            raise TypeError("positions must be int32 on the tensors' device")
        want = (N,) if jagged or positions.dim() == 1 else (B, N)
        if tuple(positions.shape) != want:
            raise ValueError(f"positions must have shape {want}, got {tuple(positions.shape)}")
        st = positions.stride()
        strides = array("q", st if len(st) == 2 else (0, st[0]))
        ps = strides.buffer_info()[0]
        pos = positions.data_ptr()
    if jagged:
        _need(offsets, "offsets", torch.int32, dev)
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be [B + 1]")
        off, n_seq = offsets.data_ptr(), offsets.numel() - 1
    L = lib()
    _call_on(dev, L.attn_rope_f16 if dt == torch.float16 else L.attn_rope, B, N, D, rope._ref, arr.buffer_info()[0],
             n, pos, ps, off, n_seq, 1 if inverse else 0)
    return out


class PagedCache:
    """A paged key-value cache, as a serving program holds it: pools
    ``k`` [pages, Hkv, page_size, Dqk] and ``v`` [pages, Hkv, page_size, Dv]
    (any strides with contiguous rows: pass ``pool.transpose(1, 2)`` of a
    token-major one), int32 ``page_table`` [B, max_pages] and ``seq_lens``
    [B].  Position p of sequence b is token p % page_size of page
    page_table[b, p // page_size]; seq_lens[b] counts the tokens of sequence
    b, those being appended in the same step included, and is 0 for an idle
    place of the batch.  The tensors are the caller's, read by the kernels
    when they run: change their contents between calls, not the tensors."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor):
        dt, dev = _elem_type(k), k.device
        _need_cuda(k, "k", dt)
        _need_cuda(v, "v", dt, dev)
        _need_cuda(page_table, "page_table", torch.int32, dev)
        _need_cuda(seq_lens, "seq_lens", torch.int32, dev)
        if k.dim() != 4 or v.dim() != 4 or k.shape[:3] != v.shape[:3]:
            raise ValueError("k must be [pages, Hkv, page_size, Dqk] and v [pages, Hkv, page_size, Dv]")
        if page_table.dim() != 2 or seq_lens.dim() != 1 or seq_lens.shape[0] != page_table.shape[0]:
            raise ValueError("page_table must be [B, max_pages] and seq_lens [B]")
        self.k, self.v, self.page_table, self.seq_lens = k, v, page_table, seq_lens
        self.B, self.max_pages = page_table.shape
        self.n_pages, self.Hkv, self.page_size, self.Dqk = k.shape
        self.Dv = v.shape[3]
        self.device, self.dtype = dev, dt
        c = AttnPagedCache()
        c.B, c.max_pages, c.n_pages, c.page_size = self.B, self.max_pages, self.n_pages, self.page_size
        c.Hkv, c.Dqk, c.Dv = self.Hkv, self.Dqk, self.Dv
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.k_stride[:], c.v_stride[:] = k.stride()[:3], v.stride()[:3]
        c.page_table, c.table_stride, c.seq_lens = page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr()
        self._struct, self._ref = c, ctypes.byref(c)
        self._workspace = {}  # bytes a decode needs, by query heads

    def _workspace_bytes(self, Hq: int) -> int:
        with torch.cuda.device(self.device):
            n = self._workspace[Hq] = int(lib().attn_paged_decode_workspace(self._ref, Hq))
        return n


def attn_paged_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, rope: Optional[Rope] = None,
                      q: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None):
    """Write the keys k [T, Hkv, Dqk] and values v [T, Hkv, Dv] of new tokens
    into their pages, the keys rotated to their positions by ``rope``, and
    return the queries q [T, Hq, Dqk] rotated beside them (in ``out``, which
    may be q itself; None without q).

    Without ``offsets`` T = B and token b is the last of sequence b; with
    int32 offsets [B + 1], tokens offsets[b] .. offsets[b + 1] are the last
    of sequence b (rows behind offsets[B] are left alone).  An idle place
    writes nothing to the cache and zeros to its query row.  Any strides with
    contiguous rows; a jagged [H, T, D] tensor goes in as its transpose(0, 1)."""
    dev, dt = cache.device, cache.dtype
    for name, t in (("k", k), ("v", v), ("q", q)):
        if t is not None and (t.dtype is not dt or t.device != dev or t.stride()[-1:] != (1,)):
            _need_cuda(t, name, dt, dev)
    T = k.shape[0]
    if k.shape != (T, cache.Hkv, cache.Dqk) or v.shape != (T, cache.Hkv, cache.Dv):
        raise ValueError(f"k must be [T, {cache.Hkv}, {cache.Dqk}] and v [T, {cache.Hkv}, {cache.Dv}]")
    off = 0
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, dev)
        if offsets.shape != (cache.B + 1,):
            raise ValueError(f"offsets must be [{cache.B + 1}]")
        off = offsets.data_ptr()
    elif T != cache.B:
        raise ValueError(f"without offsets there is one token for each of the {cache.B} sequences, got {T}")
    ks, vs, qs, os_ = k.stride(), v.stride(), (0, 0), (0, 0)
    qp = op = Hq = 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != cache.Dqk:
            raise ValueError(f"q must be [{T}, Hq, {cache.Dqk}]")
        if out is None:
            out = torch.empty(q.shape, dtype=dt, device=dev)
        else:
            _need_cuda(out, "out", dt, dev)
            if out.shape != q.shape:
                raise ValueError(f"out must have shape {tuple(q.shape)}, got {tuple(out.shape)}")
        qp, op, Hq, qs, os_ = q.data_ptr(), out.data_ptr(), q.shape[1], q.stride(), out.stride()
    elif out is not None:
        raise ValueError("out holds the rotated q: there is none without q")
    a = array("q", (T, off, k.data_ptr(), v.data_ptr(), qp, op, Hq, ks[0], ks[1], vs[0], vs[1], qs[0], qs[1],
                    os_[0], os_[1]))
    if rope is not None:
        if rope.rot_dim > cache.Dqk:
            raise ValueError(f"rot_dim {rope.rot_dim} exceeds the head dim {cache.Dqk}")
        if rope.steps.device != dev:
            raise ValueError(f"the rotation is on {rope.steps.device}, the cache on {dev}")
    L = lib()
    _call_on(dev, L.attn_paged_append_f16 if dt == torch.float16 else L.attn_paged_append, cache._ref,
             a.buffer_info()[0], rope._ref if rope is not None else None)
    return out


def attn_paged_decode(cache: PagedCache, q: torch.Tensor, sm_scale: Optional[float] = None, out=None):
    """Attention of one query token per sequence over the paged cache:
    q [B, Hq, Dqk], Hq a multiple of the cache's key heads (query head h
    reads key head h // (Hq / Hkv)).  Returns (o [B, Hq, Dv], lse [B, Hq]
    float32, natural log).  An idle place (length 0) gets o = 0, lse = -inf."""
    dev, dt, B = cache.device, cache.dtype, cache.B
    qs, sq = q.stride(), q.shape
    if q.dtype is not dt or q.device != dev or qs[-1:] != (1,):
        _need_cuda(q, "q", dt, dev)
    if len(sq) != 3 or sq[0] != B or sq[2] != cache.Dqk:
        raise ValueError(f"q must be [{B}, Hq, {cache.Dqk}]")
    Hq = sq[1]
    if cache.Hkv == 0 or Hq % cache.Hkv:
        raise ValueError(f"the cache's {cache.Hkv} key heads must divide the {Hq} query heads")
    if out is None:
        o = torch.empty((B, Hq, cache.Dv), dtype=dt, device=dev)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    else:
        o, lse = out
        _need_out(o, "o", (B, Hq, cache.Dv), dt, dev)
        _need_out(lse, "lse", (B, Hq), torch.float32, dev)
    n = cache._workspace.get(Hq)
    if n is None:
        n = cache._workspace_bytes(Hq)
    # of this call alone: a graph's is its own, calls on two streams have two
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    strides = array("q", qs)
    L = lib()
    _call_on(dev, L.attn_paged_decode_f16 if dt == torch.float16 else L.attn_paged_decode, cache._ref, Hq,
             q.data_ptr(), strides.buffer_info()[0], _scale(sm_scale), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), n)
    return o, lse
