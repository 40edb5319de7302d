"""Thin ctypes binding over libplx.so (argument marshalling only).

Every function here has the name of the C entry point it calls (declared in
include/plx.h) and does nothing but check tensor shapes/dtypes/devices, pass
``data_ptr()`` values and the current CUDA stream, and turn a non-OK status
into an exception. All arithmetic runs in the library's kernels; there is no
fallback: if libplx.so is missing or fails to load, every call raises.
PyTorch supplies device memory and streams only. What a call allocates itself
(results not given, workspaces) comes in the order of its stream, as under
``torch.cuda.stream``: with ``stream=`` given, use a result on another stream
as one made there.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libplx.so")

PLX_OK = 0
PLX_ERR_INVALID_ARG = 1
PLX_ERR_UNSUPPORTED = 2
PLX_ERR_CUDA = 3
PLX_ERR_DEVICE_TIMEOUT = 4
PLX_ERR_BOUNDS = 5

# Current device and raw handle of its current stream. torch.cuda.current_stream
# builds a Stream object around the handle, which costs 2 us of a 17 us call; it
# serves where a torch version lacks the inner names.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

# Every symbol the header declares, with its ctypes signature.
_vp, _i, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
SIGNATURES = {
    "plx_prefill_fwd": (_i, [_vp] * 6 + [_i] * 5 + [_vp]),
    "plx_prefill_fwd_f32": (_i, [_vp] * 6 + [_i] * 5 + [_vp]),
    "plx_prefill_fwd_chunk": (_i, [_vp] * 6 + [_i] * 6 + [_vp]),
    "plx_prefill_fwd_cor": (_i, [_vp] * 7 + [_i] * 6 + [_vp]),
    "plx_prefill_fwd_train": (_i, [_vp] * 8 + [_i] * 5 + [_vp]),
    "plx_prefill_bwd": (_i, [_vp] * 13 + [_i] * 5 + [_vp]),
    "plx_qkvr_proj": (_i, [_vp] * 6 + [_i] * 6 + [_vp]),
    "plx_decode_fwd": (_i, [_vp] * 6 + [_i] * 4 + [_vp]),
    "plx_decode_fwd_ex": (_i, [_vp] * 6 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_decode_fwd_noalloc": (_i, [_vp] * 6 + [_i] * 4 + [_vp]),
    "plx_decode_fwd_cor": (_i, [_vp] * 7 + [_i] * 4 + [_vp]),
    "plx_decode_workspace_bytes": (_sz, [_i] * 5),
    "plx_decode_default_nsplit": (_i, [_i] * 2),
    "plx_kv_append": (_i, [_vp] * 2 + [_ll] * 2 + [_vp] * 7 + [_i] * 7 + [_vp]),
    "plx_kv_read": (_i, [_vp] * 8 + [_i] * 7 + [_vp]),
    "plx_decode_fwd_paged": (_i, [_vp] * 9 + [_i] * 7 + [_vp, _sz, _vp]),
    "plx_decode_paged_workspace_bytes": (_sz, [_i] * 4),
    "plx_prefill_fwd_paged": (_i, [_vp] * 2 + [_ll] * 2 + [_vp] * 8 + [_ll] * 2 + [_vp] + [_i] * 8
                              + [_vp, _sz, _vp]),
    "plx_prefill_paged_workspace_bytes": (_sz, [_i] * 5),
    "plx_decode_fwd_shared": (_i, [_vp] * 11 + [_i] * 8 + [_vp, _sz, _vp]),
    "plx_decode_shared_workspace_bytes": (_sz, [_i] * 4),
    "plx_kv_update": (_i, [_vp] * 12 + [_i] * 6 + [_vp, _sz, _vp]),
    "plx_kv_update_workspace_bytes": (_sz, [_i] * 3),
    "plx_kv_compact": (_i, [_vp] * 11 + [_i] * 6 + [_vp, _sz, _vp]),
    "plx_kv_compact_workspace_bytes": (_sz, [_i]),
    "plx_rotary_fwd": (_i, [_vp] * 11 + [ctypes.c_double] + [_i] * 9 + [_vp]),
    "plx_rotary_bwd": (_i, [_vp] * 11 + [ctypes.c_double] + [_i] * 9 + [_vp]),
    "plx_rotary_freqs": (_i, [_vp] * 2 + [_i, ctypes.c_double, _i] + [ctypes.c_double] * 4),
    "plx_check_device_error": (_i, [_vp]),
    "plx_debug_timeout_probe": (_i, [_ll, _vp]),
    "plx_status_string": (ctypes.c_char_p, [_i]),
    "plx_last_error_message": (ctypes.c_char_p, []),
}


class PlxError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


_lib = None
_lock = threading.Lock()


def lib():
    """Load libplx.so (built by ``build.build()``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libplx.so not built ({LIB_PATH}); run "
                    "python -m parametrized_local_linear_gb300.build")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def load_debug_lib():
    """libplx_debug.so, the build with device-side bounds checks (see
    include/plx.h), loaded with the same signatures; built if missing."""
    from . import build
    L = ctypes.CDLL(build.build(debug_bounds=True))
    for name, (res, args) in SIGNATURES.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


def _check(status: int):
    if status != PLX_OK:
        msg = lib().plx_last_error_message().decode(errors="replace")
        raise PlxError(status, msg or lib().plx_status_string(status).decode())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, dev, stream):
    """Memory for a result, in the order of the call's stream: from the current
    stream's pool, another stream would write what work queued here may still use."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _need(t, name, dtype, ndim, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _prefill(fn, dtype, q, k, v, r, out, lse, stream):
    _need(q, "q", dtype, 4)
    dev = q.device
    for name, t in (("k", k), ("v", v), ("r", r)):
        _need(t, name, dtype, 4, dev)
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if tuple(r.shape) != tuple(q.shape):
        raise ValueError("r must have the shape of q")
    if tuple(k.shape) != (B, Hkv, L, d) or tuple(v.shape) != (B, Hkv, L, d):
        raise ValueError("k and v must be [B, Hkv, L, d] matching q")
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    _need(out, "out", dtype, 4, dev)
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have the shape of q")
    if lse is not None:
        _need(lse, "lse", torch.float32, 3, dev)
        if tuple(lse.shape) != (B, Hq, L):
            raise ValueError("lse must be [B, Hq, L]")
    with torch.cuda.device(dev):
        st = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(), out.data_ptr(),
                lse.data_ptr() if lse is not None else None, B, Hq, Hkv, L, d,
                _stream(stream, dev))
    _check(st)
    return out, lse


def plx_prefill_fwd(q, k, v, r, out=None, lse=None, stream=None):
    """Causal Parallax prefill, bf16 (see include/plx.h). Returns (out, lse)."""
    return _prefill(lib().plx_prefill_fwd, torch.bfloat16, q, k, v, r, out, lse, stream)


def plx_prefill_fwd_chunk(q, k, v, r, out=None, lse=None, stream=None):
    """Chunked causal prefill (see include/plx.h): q, r [B, Hq, Lq, d] are the
    last Lq positions of k, v [B, Hkv, Lk, d]. Returns (out, lse)."""
    out, lse, _ = _prefill_chunk(q, k, v, r, out, lse, None, stream)
    return out, lse


def plx_prefill_fwd_cor(q, k, v, r, out=None, lse=None, cor=None, stream=None):
    """Chunked causal prefill that also writes the correction-to-output ratio
    |Sigma rho| / |o| per row (see include/plx.h). ``cor`` is fp32
    [B, Hq, Lq] (allocated if None). Returns (out, lse, cor)."""
    if cor is None:
        cor = _empty(q.shape[:3], torch.float32, q.device, stream)
    return _prefill_chunk(q, k, v, r, out, lse, cor, stream)


def _prefill_chunk(q, k, v, r, out, lse, cor, stream):
    _need(q, "q", torch.bfloat16, 4)
    dev = q.device
    for name, t in (("k", k), ("v", v), ("r", r)):
        _need(t, name, torch.bfloat16, 4, dev)
    B, Hq, Lq, d = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    if tuple(r.shape) != tuple(q.shape):
        raise ValueError("r must have the shape of q")
    if tuple(k.shape) != (B, Hkv, Lk, d) or tuple(v.shape) != (B, Hkv, Lk, d):
        raise ValueError("k and v must be [B, Hkv, Lk, d] matching q")
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    _need(out, "out", torch.bfloat16, 4, dev)
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have the shape of q")
    for name, t in (("lse", lse), ("cor", cor)):
        if t is not None:
            _need(t, name, torch.float32, 3, dev)
            if tuple(t.shape) != (B, Hq, Lq):
                raise ValueError(f"{name} must be [B, Hq, Lq]")
    lse_ptr = lse.data_ptr() if lse is not None else None
    with torch.cuda.device(dev):
        if cor is None:
            st = lib().plx_prefill_fwd_chunk(q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(),
                                             out.data_ptr(), lse_ptr, B, Hq, Hkv, Lq, Lk, d,
                                             _stream(stream, dev))
        else:
            st = lib().plx_prefill_fwd_cor(q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(),
                                           out.data_ptr(), lse_ptr, cor.data_ptr(), B, Hq, Hkv, Lq,
                                           Lk, d, _stream(stream, dev))
    _check(st)
    return out, lse, cor


def plx_prefill_fwd_train(q, k, v, r, out=None, lse=None, o1=None, sbar=None, stream=None):
    """Training forward (see include/plx.h): returns (out, lse, o1, sbar), the
    last three being what plx_prefill_bwd needs."""
    _need(q, "q", torch.bfloat16, 4)
    dev = q.device
    for name, t in (("k", k), ("v", v), ("r", r)):
        _need(t, name, torch.bfloat16, 4, dev)
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if tuple(r.shape) != tuple(q.shape) or tuple(k.shape) != (B, Hkv, L, d) or v.shape != k.shape:
        raise ValueError("r must match q; k and v must be [B, Hkv, L, d]")
    out = _empty(q.shape, q.dtype, dev, stream) if out is None else out
    o1 = _empty(q.shape, q.dtype, dev, stream) if o1 is None else o1
    lse = _empty((B, Hq, L), torch.float32, dev, stream) if lse is None else lse
    sbar = _empty((B, Hq, L), torch.float32, dev, stream) if sbar is None else sbar
    for name, t in (("out", out), ("o1", o1)):
        _need(t, name, torch.bfloat16, 4, dev)
        if tuple(t.shape) != tuple(q.shape):
            raise ValueError(f"{name} must have the shape of q")
    for name, t in (("lse", lse), ("sbar", sbar)):
        _need(t, name, torch.float32, 3, dev)
        if tuple(t.shape) != (B, Hq, L):
            raise ValueError(f"{name} must be [B, Hq, L]")
    with torch.cuda.device(dev):
        st = lib().plx_prefill_fwd_train(q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(),
                                         out.data_ptr(), lse.data_ptr(), o1.data_ptr(),
                                         sbar.data_ptr(), B, Hq, Hkv, L, d, _stream(stream, dev))
    _check(st)
    return out, lse, o1, sbar


def plx_prefill_bwd(q, k, v, r, out, o1, lse, sbar, dout, dq=None, dk=None, dv=None, dr=None,
                    stream=None):
    """Backward of the causal prefill (see include/plx.h). Returns
    (dq, dk, dv, dr), bf16, shaped like q, k, v, r."""
    _need(q, "q", torch.bfloat16, 4)
    dev = q.device
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    for name, t in (("k", k), ("v", v)):
        _need(t, name, torch.bfloat16, 4, dev)
        if tuple(t.shape) != (B, Hkv, L, d):
            raise ValueError(f"{name} must be [B, Hkv, L, d]")
    dq = _empty(q.shape, q.dtype, dev, stream) if dq is None else dq
    dr = _empty(q.shape, q.dtype, dev, stream) if dr is None else dr
    dk = _empty(k.shape, k.dtype, dev, stream) if dk is None else dk
    dv = _empty(v.shape, v.dtype, dev, stream) if dv is None else dv
    for name, t, like in (("r", r, q), ("out", out, q), ("o1", o1, q), ("dout", dout, q),
                          ("dq", dq, q), ("dr", dr, q), ("dk", dk, k), ("dv", dv, k)):
        _need(t, name, torch.bfloat16, 4, dev)
        if tuple(t.shape) != tuple(like.shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    for name, t in (("lse", lse), ("sbar", sbar)):
        _need(t, name, torch.float32, 3, dev)
        if tuple(t.shape) != (B, Hq, L):
            raise ValueError(f"{name} must be [B, Hq, L]")
    with torch.cuda.device(dev):
        st = lib().plx_prefill_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(),
                                   out.data_ptr(), o1.data_ptr(), lse.data_ptr(), sbar.data_ptr(),
                                   dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                   dr.data_ptr(), B, Hq, Hkv, L, d, _stream(stream, dev))
    _check(st)
    return dq, dk, dv, dr


def plx_qkvr_proj(x, w, B, L, Hq, Hkv, d=128, q=None, k=None, v=None, r=None, stream=None):
    """Fused [W_Q; W_K; W_V; W_R] x projection (see include/plx.h): x bf16
    [B * L, D], w bf16 [(2 Hq + 2 Hkv) d, D]. Returns (q, k, v, r) in the
    attention layouts [B, H, L, d]."""
    _need(x, "x", torch.bfloat16, 2)
    dev = x.device
    _need(w, "w", torch.bfloat16, 2, dev)
    T, D = x.shape
    if T != B * L or tuple(w.shape) != ((2 * Hq + 2 * Hkv) * d, D):
        raise ValueError("x must be [B * L, D] and w [(2 Hq + 2 Hkv) d, D]")
    shapes = {"q": (B, Hq, L, d), "k": (B, Hkv, L, d), "v": (B, Hkv, L, d), "r": (B, Hq, L, d)}
    outs = {}
    for name, t in (("q", q), ("k", k), ("v", v), ("r", r)):
        if t is None:
            t = _empty(shapes[name], torch.bfloat16, dev, stream)
        _need(t, name, torch.bfloat16, 4, dev)
        if tuple(t.shape) != shapes[name]:
            raise ValueError(f"{name} must be {shapes[name]}")
        outs[name] = t
    with torch.cuda.device(dev):
        st = lib().plx_qkvr_proj(x.data_ptr(), w.data_ptr(), outs["q"].data_ptr(),
                                 outs["k"].data_ptr(), outs["v"].data_ptr(), outs["r"].data_ptr(),
                                 B, L, D, Hq, Hkv, d, _stream(stream, dev))
    _check(st)
    return outs["q"], outs["k"], outs["v"], outs["r"]


def plx_prefill_fwd_f32(q, k, v, r, out=None, lse=None, stream=None):
    """Causal Parallax prefill, fp32 (see include/plx.h). Returns (out, lse)."""
    return _prefill(lib().plx_prefill_fwd_f32, torch.float32, q, k, v, r, out, lse, stream)


def _decode_shapes(q, r, kcache, vcache, seqlens, out=None, cor=None):
    """Shape checks shared by every decode call, made before any device check
    or launch: a short ``seqlens``, ``out`` or ``cor`` would otherwise let the
    kernels read or write past the end of a buffer."""
    if q.dim() != 3:
        raise ValueError(f"q must be [B, Hq, d], got shape {tuple(q.shape)}")
    B, Hq, d = q.shape
    if tuple(r.shape) != tuple(q.shape):
        raise ValueError(f"r has shape {tuple(r.shape)}, expected the shape of q {tuple(q.shape)}")
    if kcache.dim() != 3 or kcache.shape[2] != d:
        raise ValueError(f"kcache must be [T, Hkv, {d}], got shape {tuple(kcache.shape)}")
    if tuple(vcache.shape) != tuple(kcache.shape):
        raise ValueError(f"vcache has shape {tuple(vcache.shape)}, expected the shape of kcache "
                         f"{tuple(kcache.shape)}")
    if seqlens.dim() != 1 or seqlens.shape[0] != B:
        raise ValueError(f"seqlens must have shape ({B},), got {tuple(seqlens.shape)}")
    if out is not None and tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected the shape of q {tuple(q.shape)}")
    if cor is not None and tuple(cor.shape) != (B, Hq):
        raise ValueError(f"cor has shape {tuple(cor.shape)}, expected ({B}, {Hq})")


def _decode_tensors(q, r, kcache, vcache, seqlens, out, cor=None):
    _decode_shapes(q, r, kcache, vcache, seqlens, out, cor)
    _need(q, "q", torch.bfloat16, 3)
    dev = q.device
    for name, t in (("r", r), ("kcache", kcache), ("vcache", vcache)):
        _need(t, name, torch.bfloat16, 3, dev)
    _need(seqlens, "seqlens", torch.int32, 1, dev)
    if out is not None:
        _need(out, "out", torch.bfloat16, 3, dev)
    if cor is not None:
        _need(cor, "cor", torch.float32, 2, dev)
    return dev


def plx_decode_fwd(q, r, kcache, vcache, seqlens, out=None, nsplit=0, workspace=None,
                   stream=None):
    """Parallax decode over a packed ragged KV cache (see include/plx.h).

    q, r: bf16 [B, Hq, d]; kcache, vcache: bf16 [sum(seqlens), Hkv, d];
    seqlens: int32 [B] on the device. ``nsplit``/``workspace`` select
    plx_decode_fwd_ex; the defaults call plx_decode_fwd. Returns out.
    """
    dev = _decode_tensors(q, r, kcache, vcache, seqlens, out)
    B, Hq, d = q.shape
    Hkv = kcache.shape[1]
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    L = lib()
    with torch.cuda.device(dev):
        s = _stream(stream, dev)
        if nsplit == 0 and workspace is None:
            st = L.plx_decode_fwd(q.data_ptr(), r.data_ptr(), kcache.data_ptr(), vcache.data_ptr(),
                                  seqlens.data_ptr(), out.data_ptr(), B, Hq, Hkv, d, s)
        else:
            ws_ptr, ws_bytes = None, 0
            if workspace is not None:
                if not workspace.is_cuda or workspace.device != dev:
                    raise ValueError("workspace must be on the device of q")
                ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
            st = L.plx_decode_fwd_ex(q.data_ptr(), r.data_ptr(), kcache.data_ptr(),
                                     vcache.data_ptr(), seqlens.data_ptr(), out.data_ptr(), B, Hq,
                                     Hkv, d, int(nsplit), ws_ptr, ws_bytes, s)
    _check(st)
    return out


def plx_decode_fwd_noalloc(q, r, kcache, vcache, seqlens, out, stream=None):
    """Decode through the entry point that allocates nothing (see include/plx.h):
    the partial records go to the library's fixed device array. ``out`` must be
    given (bf16 [B, Hq, d]); returns it."""
    if out is None:
        raise ValueError("out must be given: this entry point allocates nothing")
    dev = _decode_tensors(q, r, kcache, vcache, seqlens, out)
    B, Hq, d = q.shape
    with torch.cuda.device(dev):
        st = lib().plx_decode_fwd_noalloc(q.data_ptr(), r.data_ptr(), kcache.data_ptr(),
                                          vcache.data_ptr(), seqlens.data_ptr(), out.data_ptr(),
                                          B, Hq, kcache.shape[1], d, _stream(stream, dev))
    _check(st)
    return out


def plx_decode_fwd_cor(q, r, kcache, vcache, seqlens, out=None, cor=None, stream=None):
    """Decode that also writes the correction-to-output ratio |Sigma rho| / |o|
    per (sequence, head) (see include/plx.h). ``cor`` is fp32 [B, Hq]
    (allocated if None). Returns (out, cor)."""
    dev = _decode_tensors(q, r, kcache, vcache, seqlens, out, cor)
    B, Hq, d = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    if cor is None:
        cor = _empty((B, Hq), torch.float32, dev, stream)
    with torch.cuda.device(dev):
        st = lib().plx_decode_fwd_cor(q.data_ptr(), r.data_ptr(), kcache.data_ptr(),
                                      vcache.data_ptr(), seqlens.data_ptr(), out.data_ptr(),
                                      cor.data_ptr(), B, Hq, kcache.shape[1], d,
                                      _stream(stream, dev))
    _check(st)
    return out, cor


def plx_decode_workspace_bytes(B, Hq, Hkv, d, nsplit) -> int:
    return int(lib().plx_decode_workspace_bytes(B, Hq, Hkv, d, nsplit))


def plx_decode_default_nsplit(B, Hkv) -> int:
    return int(lib().plx_decode_default_nsplit(B, Hkv))


def _is(t, dtype, shape, index):
    """Whether t is a contiguous tensor of this type and shape on CUDA device
    `index`. The paged calls check up to ten tensors, and a decode step waits
    for them: this reads the fewest attributes, and only a tensor that fails it
    goes through the checks that say why."""
    return (t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous())


def _like(t, name, dtype, shape, dev):
    """_need with the whole shape."""
    if _is(t, dtype, shape, dev.index):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _need(t, name, dtype, len(shape), dev)


def _given(name, t):
    """For tensors that only some of the paged calls can do without."""
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")


def _check_pages(kpages, vpages, kscale, vscale, block_table, seqlens, dev):
    """Raises for what is wrong with the tensors of a paged cache."""
    shape = kpages.shape
    if len(shape) != 4:
        raise ValueError(f"kpages must be [num_pages, Hkv, page_size, d], got shape {tuple(shape)}")
    if block_table.dim() != 2 or block_table.shape[0] < 1:
        raise ValueError(f"block_table must be [B, max_pages], got shape {tuple(block_table.shape)}")
    B, width = block_table.shape
    fp8 = kscale is not None or vscale is not None
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    if fp8:
        for name, t in (("kscale", kscale), ("vscale", vscale)):
            if t is None or t.shape != shape[:3]:
                raise ValueError(f"{name} must be given with shape {tuple(shape[:3])}")
    if vpages.shape != shape:
        raise ValueError(f"vpages has shape {tuple(vpages.shape)}, expected {tuple(shape)}")
    if seqlens is not None and seqlens.shape != (B,):
        raise ValueError(f"seqlens must have shape ({B},), got {tuple(seqlens.shape)}")
    if kpages.dtype is not dtype or vpages.dtype is not dtype:
        name, t = ("kpages", kpages) if kpages.dtype is not dtype else ("vpages", vpages)
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dev.type != "cuda":
        raise ValueError("kpages must be a CUDA tensor" if kpages.device.type != "cuda" else
                         "all tensors must be CUDA tensors")
    _like(kpages, "kpages", dtype, shape, dev)
    _like(vpages, "vpages", dtype, shape, dev)
    _like(block_table, "block_table", torch.int32, (B, width), dev)
    if seqlens is not None:
        _like(seqlens, "seqlens", torch.int32, (B,), dev)
    if fp8:
        _like(kscale, "kscale", torch.uint8, shape[:3], dev)
        _like(vscale, "vscale", torch.uint8, shape[:3], dev)


def _pages(kpages, vpages, kscale, vscale, block_table, seqlens, dev):
    """Checks of a paged cache and of the int32 [B] lengths (or None) that go
    with it; returns the pointers (kpages, vpages, kscale, vscale, block_table)
    and the sizes (B, Hkv, d, num_pages, page_size, max_pages)."""
    shape, entries, index = kpages.shape, block_table.shape, dev.index
    fp8 = kscale is not None and vscale is not None
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    if not (len(shape) == 4 and len(entries) == 2 and entries[0] >= 1
            and (fp8 or kscale is vscale)
            and _is(kpages, dtype, shape, index) and _is(vpages, dtype, shape, index)
            and _is(block_table, torch.int32, entries, index)
            and (seqlens is None or _is(seqlens, torch.int32, entries[:1], index))
            and (not fp8 or (_is(kscale, torch.uint8, shape[:3], index)
                             and _is(vscale, torch.uint8, shape[:3], index)))):
        _check_pages(kpages, vpages, kscale, vscale, block_table, seqlens, dev)
    B, width = entries
    n, Hkv, page, d = shape
    return (kpages.data_ptr(), vpages.data_ptr(), kscale.data_ptr() if fp8 else None,
            vscale.data_ptr() if fp8 else None, block_table.data_ptr()), (B, Hkv, d, n, page, width)


def _packed(t, name, heads, d, dev):
    """(token, head) strides of packed rows [T, heads, d]; only a row's d
    values must be contiguous."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != d or shape[1] != heads:
        raise ValueError(f"{name} must be [T, {heads}, {d}], got shape {tuple(shape)}")
    if t.get_device() != dev.index:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    ts, hs, ds = t.stride()
    if ds != 1 and d != 1:
        raise ValueError(f"{name} must have its last dimension contiguous")
    # A dimension of size one has no stride of its own.
    if heads == 1:
        hs = d
    if shape[0] == 1:
        ts = max(d, hs * heads)
    return ts, hs


def _launch(fn, dev, stream, args):
    """fn(*args, stream) on the device of the tensors; raises on a bad status."""
    if _current_device() == dev.index:
        status = fn(*args, _raw_stream(dev.index) if stream is None else stream.cuda_stream)
        if status != PLX_OK:
            _check(status)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, _stream(stream, dev)))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(sizer, sizes, index):
    """What the library's size function says on that device (it goes by its SM count)."""
    with torch.cuda.device(index):
        return getattr(lib(), sizer)(*sizes)


def _workspace(workspace, sizer, sizes, stream, dev):
    """(tensor, pointer, bytes) of the caller's workspace, or of one of the
    needed size from torch's caching allocator, in the order of the call's stream (a
    stream-ordered allocation by the library would give its memory back to the
    driver whenever the GPU idles: 200 us for a call after a synchronize)."""
    if workspace is None:
        need = _workspace_bytes(sizer, sizes, dev.index)
        workspace = _empty(need, torch.uint8, dev, stream)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_cuda or workspace.device != dev:
        raise ValueError("workspace must be on the device of q")
    if not workspace.is_contiguous() or workspace.numel() == 0:
        raise ValueError("workspace must be contiguous and not empty")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def plx_kv_append(k, v, kpages, vpages, block_table, seqlens, cu_q=None, kscale=None, vscale=None,
                  stream=None):
    """Write new tokens into a paged KV cache (see include/plx.h): k, v bf16
    [T, Hkv, d] with any token and head strides (the projection's [Hkv, T, d]
    transposed will do); pages bf16, or torch.float8_e4m3fn with uint8
    ``kscale`` / ``vscale``. ``cu_q=None``: one new token a sequence. Returns
    (kpages, vpages)."""
    if k.dim() != 3:
        raise ValueError(f"k must be [T, Hkv, d], got shape {tuple(k.shape)}")
    if v.shape != k.shape:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected the shape of k {tuple(k.shape)}")
    _given("seqlens", seqlens)
    dev = k.device
    ptrs, (B, Hkv, d, n, page, width) = _pages(kpages, vpages, kscale, vscale, block_table, seqlens,
                                               dev)
    strides = _packed(k, "k", Hkv, d, dev)
    if _packed(v, "v", Hkv, d, dev) != strides:
        raise ValueError("k and v must have the same strides")
    T = k.shape[0]
    if cu_q is not None:
        _like(cu_q, "cu_q", torch.int32, (B + 1,), dev)
    elif T != B:
        raise ValueError(f"without cu_q, k must have one row for each of the {B} sequences, got {T}")
    _launch(lib().plx_kv_append, dev, stream,
            (k.data_ptr(), v.data_ptr(), *strides, *ptrs, seqlens.data_ptr(),
             cu_q.data_ptr() if cu_q is not None else None, T, B, Hkv, d, n, page, width))
    return kpages, vpages


def plx_kv_read(kpages, vpages, block_table, cu_k, T, kscale=None, vscale=None, k=None, v=None,
                stream=None):
    """Read sequences of a paged KV cache back (see include/plx.h): the first
    cu_k[b + 1] - cu_k[b] tokens of sequence b at rows cu_k[b] .. of bf16
    [T, Hkv, d], the packed cache of plx_decode_fwd. Returns (k, v)."""
    _given("cu_k", cu_k)
    dev = kpages.device
    T = int(T)
    if T < 0:
        raise ValueError(f"T must be >= 0, got {T}")
    ptrs, (B, Hkv, d, n, page, width) = _pages(kpages, vpages, kscale, vscale, block_table, None, dev)
    _like(cu_k, "cu_k", torch.int32, (B + 1,), dev)
    if k is None:
        k = _empty((T, Hkv, d), torch.bfloat16, dev, stream)
    else:
        _like(k, "k", torch.bfloat16, (T, Hkv, d), dev)
    if v is None:
        v = _empty((T, Hkv, d), torch.bfloat16, dev, stream)
    else:
        _like(v, "v", torch.bfloat16, (T, Hkv, d), dev)
    _launch(lib().plx_kv_read, dev, stream,
            (*ptrs, cu_k.data_ptr(), k.data_ptr(), v.data_ptr(), T, B, Hkv, d, n, page, width))
    return k, v


def plx_decode_fwd_paged(q, r, kpages, vpages, block_table, seqlens, kscale=None, vscale=None,
                         out=None, workspace=None, stream=None):
    """Decode over a paged KV cache (see include/plx.h): q, r bf16 [B, Hq, d].
    Returns out."""
    if q.dim() != 3:
        raise ValueError(f"q must be [B, Hq, d], got shape {tuple(q.shape)}")
    _given("seqlens", seqlens)
    dev = q.device
    B, Hq, d = shape = q.shape
    if B != block_table.shape[0] or d != kpages.shape[-1]:
        raise ValueError(f"q must be ({block_table.shape[0]}, {Hq}, {kpages.shape[-1]}), got shape "
                         f"{tuple(shape)}")
    rows = [("q", q), ("r", r)] + ([("out", out)] if out is not None else [])
    good = all([_is(t, torch.bfloat16, shape, dev.index) for _, t in rows])
    if not good:
        for name, t in rows:
            if t.shape != shape:
                raise ValueError(f"{name} must be {tuple(shape)}, got shape {tuple(t.shape)}")
    ptrs, (B, Hkv, d, n, page, width) = _pages(kpages, vpages, kscale, vscale, block_table, seqlens,
                                               dev)
    if not good:
        for name, t in rows:
            _like(t, name, torch.bfloat16, shape, dev)
    if out is None:
        out = _empty(shape, torch.bfloat16, dev, stream)
    ws, ws_ptr, ws_bytes = _workspace(workspace, "plx_decode_paged_workspace_bytes", (B, Hq, Hkv, d),
                                      stream, dev)
    _launch(lib().plx_decode_fwd_paged, dev, stream,
            (q.data_ptr(), r.data_ptr(), *ptrs, seqlens.data_ptr(), out.data_ptr(), B, Hq, Hkv, d, n,
             page, width, ws_ptr, ws_bytes))
    return out


def plx_prefill_fwd_paged(q, r, kpages, vpages, block_table, seqlens, cu_q, kscale=None,
                          vscale=None, out=None, lse=None, workspace=None, stream=None):
    """Causal prefill of a ragged batch of chunks over a paged KV cache (see
    include/plx.h): q, r bf16 [T, Hq, d] with any token and head strides, the
    same for both. ``lse`` is fp32 [T, Hq] or None. Returns (out, lse)."""
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, d], got shape {tuple(q.shape)}")
    if r.shape != q.shape:
        raise ValueError(f"r has shape {tuple(r.shape)}, expected the shape of q {tuple(q.shape)}")
    _given("seqlens", seqlens)
    _given("cu_q", cu_q)
    dev = q.device
    ptrs, (B, Hkv, d, n, page, width) = _pages(kpages, vpages, kscale, vscale, block_table, seqlens,
                                               dev)
    T, Hq, _ = q.shape
    strides = _packed(q, "q", Hq, d, dev)
    if _packed(r, "r", Hq, d, dev) != strides:
        raise ValueError("q and r must have the same strides")
    _like(cu_q, "cu_q", torch.int32, (B + 1,), dev)
    if out is None:
        out, out_strides = _empty((T, Hq, d), torch.bfloat16, dev, stream), (Hq * d, d)
    else:
        if out.shape != q.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(q.shape)}")
        out_strides = _packed(out, "out", Hq, d, dev)
    if lse is not None:
        _like(lse, "lse", torch.float32, (T, Hq), dev)
    ws, ws_ptr, ws_bytes = _workspace(workspace, "plx_prefill_paged_workspace_bytes",
                                      (T, B, Hq, Hkv, d), stream, dev)
    _launch(lib().plx_prefill_fwd_paged, dev, stream,
            (q.data_ptr(), r.data_ptr(), *strides, *ptrs, seqlens.data_ptr(), cu_q.data_ptr(),
             out.data_ptr(), *out_strides, lse.data_ptr() if lse is not None else None, T, B, Hq, Hkv,
             d, n, page, width, ws_ptr, ws_bytes))
    return out, lse


def _shared_checks(q, r, kpages, block_table, seqlens, cu_g, prefix_lens, out):
    """Raises for what is wrong with the shapes of a shared decode; returns its groups."""
    if q.dim() != 3:
        raise ValueError(f"q must be [B, Hq, d], got shape {tuple(q.shape)}")
    for name, t in (("seqlens", seqlens), ("cu_g", cu_g), ("prefix_lens", prefix_lens)):
        _given(name, t)
    B, Hq, d = shape = q.shape
    if B != block_table.shape[0] or d != kpages.shape[-1]:
        raise ValueError(f"q must be ({block_table.shape[0]}, {Hq}, {kpages.shape[-1]}), got shape "
                         f"{tuple(shape)}")
    if prefix_lens.dim() != 1 or prefix_lens.shape[0] < 1:
        raise ValueError(f"prefix_lens must be [ngroups], got shape {tuple(prefix_lens.shape)}")
    groups = prefix_lens.shape[0]
    for name, t in (("r", r), ("out", out)):
        if t is not None and t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got shape {tuple(t.shape)}")
    if cu_g.shape != (groups + 1,):
        raise ValueError(f"cu_g must have shape ({groups + 1},), got {tuple(cu_g.shape)}")
    return groups


def plx_decode_fwd_shared(q, r, kpages, vpages, block_table, seqlens, cu_g, prefix_lens, kscale=None,
                          vscale=None, out=None, workspace=None, stream=None):
    """Decode over a paged KV cache for groups of sequences that share their first
    keys (see include/plx.h): q, r bf16 [B, Hq, d]; group g is the sequences
    cu_g[g] .. cu_g[g + 1] - 1, whose first prefix_lens[g] keys are read for all of them
    together, through the pages of the first one that has keys. Returns out."""
    dev, shape, bf16, i32 = q.device, q.shape, torch.bfloat16, torch.int32
    index = dev.index
    good = (seqlens is not None and cu_g is not None and prefix_lens is not None
            and len(shape) == 3 and shape[0] == block_table.shape[0]
            and shape[2] == kpages.shape[-1] and len(prefix_lens.shape) == 1
            and prefix_lens.shape[0] >= 1)
    if good:
        groups = prefix_lens.shape[0]
        good = (_is(q, bf16, shape, index) and _is(r, bf16, shape, index)
                and (out is None or _is(out, bf16, shape, index))
                and _is(cu_g, i32, (groups + 1,), index) and _is(prefix_lens, i32, (groups,), index))
    if not good:
        groups = _shared_checks(q, r, kpages, block_table, seqlens, cu_g, prefix_lens, out)
    Hq = shape[1]
    ptrs, (B, Hkv, d, n, page, width) = _pages(kpages, vpages, kscale, vscale, block_table, seqlens,
                                               dev)
    if not good:
        for name, t in (("q", q), ("r", r)) + ((("out", out),) if out is not None else ()):
            _like(t, name, bf16, shape, dev)
        _like(cu_g, "cu_g", i32, (groups + 1,), dev)
        _like(prefix_lens, "prefix_lens", i32, (groups,), dev)
    if out is None:
        out = _empty(shape, bf16, dev, stream)
    ws, ws_ptr, ws_bytes = _workspace(workspace, "plx_decode_shared_workspace_bytes",
                                      (B, Hq, Hkv, d), stream, dev)
    _launch(lib().plx_decode_fwd_shared, dev, stream,
            (q.data_ptr(), r.data_ptr(), *ptrs, seqlens.data_ptr(), cu_g.data_ptr(),
             prefix_lens.data_ptr(), out.data_ptr(), groups, B, Hq, Hkv, d, n, page, width, ws_ptr,
             ws_bytes))
    return out


def plx_kv_update(kpages, vpages, block_table, seqlens, page_refs, lens, src=None, kscale=None,
                  vscale=None, block_table_out=None, seqlens_out=None, page_refs_out=None,
                  workspace=None, stream=None):
    """Forks, reorders, cuts, grows and empties the rows of a paged KV cache's block
    table (see include/plx.h): row b takes over the first min(lens[b], its length)
    tokens of old row src[b] (its own without ``src``, none for -1) and gets pages for
    lens[b]. int32 tensors: seqlens, lens, src [B], page_refs [num_pages]. In place, or
    into all three of ``block_table_out``, ``seqlens_out``, ``page_refs_out``. Returns
    (block_table, seqlens, page_refs) as they are afterwards."""
    outs = (block_table_out, seqlens_out, page_refs_out)
    for name, t in (("seqlens", seqlens), ("page_refs", page_refs), ("lens", lens)):
        _given(name, t)
    dev = kpages.device
    ptrs, (B, Hkv, d, n, page, width) = _pages(kpages, vpages, kscale, vscale, block_table, seqlens,
                                               dev)
    if block_table_out is None or seqlens_out is None or page_refs_out is None:
        if not (block_table_out is None and seqlens_out is None and page_refs_out is None):
            raise ValueError("block_table_out, seqlens_out and page_refs_out must be given all or none")
        outs = block_table, seqlens, page_refs
    i32, index = torch.int32, dev.index
    if not (_is(page_refs, i32, (n,), index) and _is(lens, i32, (B,), index)
            and (src is None or _is(src, i32, (B,), index)) and _is(outs[0], i32, (B, width), index)
            and _is(outs[1], i32, (B,), index) and _is(outs[2], i32, (n,), index)):
        _like(page_refs, "page_refs", i32, (n,), dev)
        _like(lens, "lens", i32, (B,), dev)
        if src is not None:
            _like(src, "src", i32, (B,), dev)
        _like(outs[0], "block_table_out", i32, (B, width), dev)
        _like(outs[1], "seqlens_out", i32, (B,), dev)
        _like(outs[2], "page_refs_out", i32, (n,), dev)
    ws, ws_ptr, ws_bytes = _workspace(workspace, "plx_kv_update_workspace_bytes", (B, n, width),
                                      stream, dev)
    _launch(lib().plx_kv_update, dev, stream,
            (*ptrs, seqlens.data_ptr(), page_refs.data_ptr(),
             src.data_ptr() if src is not None else None, lens.data_ptr(), outs[0].data_ptr(),
             outs[1].data_ptr(), outs[2].data_ptr(), B, Hkv, d, n, page, width, ws_ptr, ws_bytes))
    return outs


def plx_kv_compact(kpages, vpages, block_table, seqlens, page_refs, kscale=None, vscale=None,
                   block_table_out=None, page_refs_out=None, page_map=None, used=None,
                   workspace=None, stream=None):
    """Moves the used pages of a paged KV cache to the front of the pool (see
    include/plx.h), in place or into ``block_table_out`` and ``page_refs_out``. Returns
    (block_table, page_refs, page_map, used): ``page_map`` int32 [num_pages] has every
    used page's new number, -1 for a free one, ``used`` int32 [1] how many are used."""
    outs = (block_table_out, page_refs_out)
    for name, t in (("seqlens", seqlens), ("page_refs", page_refs)):
        _given(name, t)
    dev = kpages.device
    ptrs, (B, Hkv, d, n, page, width) = _pages(kpages, vpages, kscale, vscale, block_table, seqlens,
                                               dev)
    if block_table_out is None or page_refs_out is None:
        if not (block_table_out is None and page_refs_out is None):
            raise ValueError("block_table_out and page_refs_out must be given both or neither")
        outs = block_table, page_refs
    i32, index = torch.int32, dev.index
    if not (_is(page_refs, i32, (n,), index) and _is(outs[0], i32, (B, width), index)
            and _is(outs[1], i32, (n,), index) and (page_map is None or _is(page_map, i32, (n,), index))
            and (used is None or _is(used, i32, (1,), index))):
        _like(page_refs, "page_refs", i32, (n,), dev)
        _like(outs[0], "block_table_out", i32, (B, width), dev)
        _like(outs[1], "page_refs_out", i32, (n,), dev)
        if page_map is not None:
            _like(page_map, "page_map", i32, (n,), dev)
        if used is not None:
            _like(used, "used", i32, (1,), dev)
    if page_map is None:
        page_map = _empty((n,), i32, dev, stream)
    if used is None:
        used = _empty((1,), i32, dev, stream)
    ws, ws_ptr, ws_bytes = _workspace(workspace, "plx_kv_compact_workspace_bytes", (n,), stream, dev)
    _launch(lib().plx_kv_compact, dev, stream,
            (*ptrs, seqlens.data_ptr(), page_refs.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(),
             page_map.data_ptr(), used.data_ptr(), B, Hkv, d, n, page, width, ws_ptr, ws_bytes))
    return (*outs, page_map, used)


_ROTARY_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_ROTARY_KINDS = {None: 0, "linear": 1, "base": 2, "parts": 3}


def plx_rotary_freqs(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_len=0,
                     beta_slow=1.0, beta_fast=32.0, device=None):
    """Frequencies of rotary positions (see include/plx.h), for a context ``factor``
    times as long with ``scaling`` "linear", "base" or "parts". Returns (inv_freq fp64
    [rotary_dim / 2] on ``device``, scale)."""
    if scaling not in _ROTARY_KINDS:
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
    freqs, scale = (ctypes.c_double * (max(int(rotary_dim), 2) // 2))(), ctypes.c_double()
    _check(lib().plx_rotary_freqs(ctypes.addressof(freqs), ctypes.addressof(scale), int(rotary_dim), base,
                                  _ROTARY_KINDS[scaling], factor, original_len, beta_slow, beta_fast))
    return torch.tensor(list(freqs), dtype=torch.float64, device=device), scale.value


_strides = struct.Struct("18q").pack


def _rotary_checks(q, k, r, inv_freq, positions, seqlens, cu_q, outs):
    """Raises for what is wrong with the tensors of a rotary call."""
    for name, t, o in zip("qkr", (q, k, r), outs):
        if t is None and o is not None:
            raise ValueError(f"{name}_out without {name}")
    given = [(name, t, o) for name, t, o in zip("qkr", (q, k, r), outs) if t is not None]
    if not given:
        raise ValueError("q, k and r are all None")
    first, x = given[0][:2]
    dev, dtype, dims = x.device, x.dtype, x.dim()
    if dtype not in _ROTARY_DTYPES:
        raise TypeError(f"{first} must be torch.bfloat16 or torch.float32, got {dtype}")
    if dims not in (3, 4):
        raise ValueError(f"{first} must be [T, H, d] or [B, H, L, d], got shape {tuple(x.shape)}")
    packed = dims == 3
    B, L, d = (1, x.shape[0], x.shape[2]) if packed else (x.shape[0], x.shape[2], x.shape[3])
    heads = {}
    for name, t, o in given:
        H = t.shape[1] if t.dim() == dims else 0
        shape = (L, H, d) if packed else (B, H, L, d)
        if t.shape != shape or heads.setdefault(name == "k", H) != H:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, which does not go with {first}'s "
                             f"{tuple(x.shape)}")
        if H == 0:
            raise ValueError(f"{name} has no heads")
        if o is not None and o.shape != shape:
            raise ValueError(f"{name}_out has shape {tuple(o.shape)}, expected {tuple(shape)}")
    for name, t, o in given:
        for what, y in ((name, t), (name + "_out", o)):
            if y is None:
                continue
            if dev.type != "cuda" or y.get_device() != dev.index:
                raise ValueError(f"{what} must be a CUDA tensor on the device of {first} ({dev})")
            if y.dtype is not dtype:
                raise TypeError(f"{what} must be {dtype}, got {y.dtype}")
            if y.stride()[-1] != 1 and y.numel() > 0:
                raise ValueError(f"{what} must have its last dimension contiguous")
    _like(inv_freq, "inv_freq", torch.float64, (inv_freq.shape[0] if inv_freq.dim() == 1 else 0,), dev)
    if positions is not None:
        if seqlens is not None or cu_q is not None:
            raise ValueError("positions and seqlens / cu_q exclude each other")
        _like(positions, "positions", torch.int32, (L,) if packed else (B, L), dev)
    elif seqlens is not None:
        if not packed:
            raise ValueError("seqlens goes with packed rows [T, H, d]")
        nseq = seqlens.shape[0] if seqlens.dim() == 1 else 0
        _like(seqlens, "seqlens", torch.int32, (nseq,), dev)
        if cu_q is not None:
            _like(cu_q, "cu_q", torch.int32, (nseq + 1,), dev)
    elif cu_q is not None:
        raise ValueError("cu_q without seqlens")
    elif packed:
        raise ValueError("packed rows need positions, or seqlens (and cu_q)")


def _rotary(fn, q, k, r, inv_freq, positions, seqlens, cu_q, interleaved, scale, q_out, k_out, r_out,
            stream):
    # As for the paged calls: one lean pass over the tensors, and the checks that
    # say why only where it finds something.
    x = q if q is not None else k if k is not None else r
    if x is None:
        _rotary_checks(q, k, r, inv_freq, positions, seqlens, cu_q, (q_out, k_out, r_out))
    dev, dtype, shape = x.device, x.dtype, x.shape
    index, dims, nseq = x.get_device(), len(shape), 0
    packed = dims == 3
    good = (index >= 0 and dtype in _ROTARY_DTYPES and (packed or dims == 4)
            and inv_freq.dtype is torch.float64 and inv_freq.get_device() == index
            and inv_freq.dim() == 1 and inv_freq.is_contiguous())
    if good:
        B, L, d = (1, shape[0], shape[2]) if packed else (shape[0], shape[2], shape[3])
        if positions is not None:
            good = (seqlens is None and cu_q is None
                    and _is(positions, torch.int32, (L,) if packed else (B, L), index))
        elif seqlens is not None:
            nseq = seqlens.numel()
            good = (packed and _is(seqlens, torch.int32, (nseq,), index)
                    and (cu_q is None or _is(cu_q, torch.int32, (nseq + 1,), index)))
        else:
            good = cu_q is None and not packed
    Hq = Hkv = 0
    ptrs, outs, results = [], [], []  # pointers; (sequence, token, head) strides
    ins, to = [], []
    for t, o, kv in ((q, q_out, False), (k, k_out, True), (r, r_out, False)) if good else ():
        if t is None:
            good = good and o is None
            ptrs.append(None)
            outs.append(None)
            results.append(None)
            ins += 0, 0, 0
            to += 0, 0, 0
            continue
        ts, st = t.shape, t.stride()
        if len(ts) != dims:
            good = False
            break
        H = ts[1]
        if kv:
            Hkv = H
        else:
            good = good and (Hq == 0 or H == Hq)
            Hq = H
        good = (good and H > 0 and t.dtype is dtype and t.get_device() == index and st[-1] == 1
                and ts[0] == shape[0] and ts[-1] == d and (packed or ts[2] == L))
        ptrs.append(t.data_ptr())
        ins += (0, st[0], st[1]) if packed else (st[0], st[2], st[1])
        if o is None:
            o = _empty(ts, dtype, dev, stream)
            to += (0, H * d, d) if packed else (H * L * d, d, L * d)
        else:
            if o.shape != ts:
                good = False
                break
            st = o.stride()
            good = good and o.dtype is dtype and o.get_device() == index and st[-1] == 1
            to += (0, st[0], st[1]) if packed else (st[0], st[2], st[1])
        outs.append(o.data_ptr())
        results.append(o)
    if not good:
        _rotary_checks(q, k, r, inv_freq, positions, seqlens, cu_q, (q_out, k_out, r_out))
        raise ValueError("rotary tensors with strides that do not go with their last dimension")
    if B > 0 and L > 0:
        _launch(fn, dev, stream,
                (*ptrs, *outs, _strides(*ins, *to), None if positions is None else positions.data_ptr(),
                 None if seqlens is None else seqlens.data_ptr(),
                 None if cu_q is None else cu_q.data_ptr(), inv_freq.data_ptr(), scale, nseq, B, L,
                 Hq or 1, Hkv or 1, d, 2 * inv_freq.shape[0], 1 if interleaved else 0,
                 _ROTARY_DTYPES[dtype]))
    return tuple(results)


def plx_rotary_fwd(q, k, inv_freq, r=None, positions=None, seqlens=None, cu_q=None,
                   interleaved=False, scale=1.0, q_out=None, k_out=None, r_out=None, stream=None):
    """Rotary positions (see include/plx.h): q, r [B, Hq, L, d] and k [B, Hkv, L, d], or
    packed rows [T, H, d], bf16 or fp32 with any strides of the outer dimensions; the
    first 2 * len(inv_freq) values of each row are turned. Positions: int32
    ``positions`` [B, L] or [T], or those of plx_kv_append's new tokens from ``seqlens``
    and ``cu_q`` (packed), or 0 .. L - 1. q, k or r may be None; ``q_out=q`` works in
    place. With ``seqlens``, rows of padding and rows behind the last sequence are not
    written: an output that is given keeps what it held there, one that the call
    allocates holds anything there, NaN included (give a zeroed one where they are
    read, as in sums over rows). Returns (q, k, r) turned."""
    return _rotary(lib().plx_rotary_fwd, q, k, r, inv_freq, positions, seqlens, cu_q, interleaved,
                   scale, q_out, k_out, r_out, stream)


def plx_rotary_bwd(dq, dk, inv_freq, dr=None, positions=None, seqlens=None, cu_q=None,
                   interleaved=False, scale=1.0, dq_out=None, dk_out=None, dr_out=None,
                   stream=None):
    """Backward of plx_rotary_fwd (see include/plx.h): from the gradients of its outputs
    those of its inputs, with its other arguments; with ``seqlens``, rows that are not
    written are as there. Returns (dq, dk, dr)."""
    return _rotary(lib().plx_rotary_bwd, dq, dk, dr, inv_freq, positions, seqlens, cu_q, interleaved,
                   scale, dq_out, dk_out, dr_out, stream)


def plx_decode_shared_workspace_bytes(B, Hq, Hkv, d) -> int:
    return int(lib().plx_decode_shared_workspace_bytes(B, Hq, Hkv, d))


def plx_kv_update_workspace_bytes(B, num_pages, max_pages) -> int:
    return int(lib().plx_kv_update_workspace_bytes(B, num_pages, max_pages))


def plx_kv_compact_workspace_bytes(num_pages) -> int:
    return int(lib().plx_kv_compact_workspace_bytes(num_pages))


def plx_decode_paged_workspace_bytes(B, Hq, Hkv, d) -> int:
    return int(lib().plx_decode_paged_workspace_bytes(B, Hq, Hkv, d))


def plx_prefill_paged_workspace_bytes(T, B, Hq, Hkv, d) -> int:
    return int(lib().plx_prefill_paged_workspace_bytes(T, B, Hq, Hkv, d))


def plx_check_device_error(stream=None, device=None):
    """Synchronise the stream and raise PlxError if a bounded wait ran out."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        _check(lib().plx_check_device_error(_stream(stream, dev)))


def plx_debug_timeout_probe(limit_cycles=100000, stream=None):
    dev = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(lib().plx_debug_timeout_probe(int(limit_cycles), _stream(stream, dev)))
