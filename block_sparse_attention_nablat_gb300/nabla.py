"""Thin ctypes binding of the C ABI in include/nabla.h (libnabla.so).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  torch supplies device memory (outputs and the mask-builder
workspace are allocated here with torch when the caller passes none) and the
current CUDA stream.  A call given another `stream` allocates from that stream's
memory: its scratch is reused only behind its kernels, and its outputs may be read
on that stream and, once ordered behind it, on the stream that was current.  If the
library is missing, every call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnabla.so")

NABLA_OK = 0
NABLA_F32, NABLA_BF16 = 0, 1

_lib = None


class _Strides(ctypes.Structure):
    """nabla_strides of include/nabla.h, in elements."""
    _fields_ = [("batch", ctypes.c_int64), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class NablaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {nabla_status_string(status)} ({status})")


def load() -> ctypes.CDLL:
    """Load libnabla.so (built by __graft_entry__.build()); raise if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.nabla_abi_version.restype = i32
    lib.nabla_abi_version.argtypes = []
    lib.nabla_status_string.restype = ctypes.c_char_p
    lib.nabla_status_string.argtypes = [i32]
    lib.nabla_build_mask_workspace_bytes.restype = sz
    lib.nabla_build_mask_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.nabla_build_mask.restype = i32
    lib.nabla_build_mask.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, ctypes.c_double, vp,
                                     vp, vp, sz, vp]
    lib.nabla_build_mask_noalloc.restype = i32
    lib.nabla_build_mask_noalloc.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, ctypes.c_double,
                                             vp, vp, vp]
    lib.nabla_build_mask_topk.restype = i32
    lib.nabla_build_mask_topk.argtypes = [vp, vp, i32, i32, i32, i32, i32, ctypes.c_double, vp,
                                          vp, vp, sz, vp]
    lib.nabla_attn_fwd.restype = i32
    lib.nabla_attn_fwd.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, ctypes.c_float,
                                   vp, vp]
    lib.nabla_attn_bwd_workspace_bytes.restype = sz
    lib.nabla_attn_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.nabla_attn_bwd.restype = i32
    lib.nabla_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                   ctypes.c_float, vp, vp, vp, vp, sz, vp]
    lib.nabla_attn_fwd_lse.restype = i32
    lib.nabla_attn_fwd_lse.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                       ctypes.c_float, vp, vp, vp]
    lib.nabla_sta_mask.restype = i32
    lib.nabla_sta_mask.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp]
    for name in ("nabla_fractal_flatten", "nabla_fractal_unflatten"):
        fn = getattr(lib, name)
        fn.restype = i32
        fn.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    st, f32 = ctypes.POINTER(_Strides), ctypes.c_float
    qk = [vp, st, vp, st, i32, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp, i32, i32, i32, vp, f32]
    lib.nabla_qk_norm_rope.restype = i32
    lib.nabla_qk_norm_rope.argtypes = qk + [vp, st, vp, st, vp]
    lib.nabla_qk_norm_rope_bwd_workspace_bytes.restype = sz
    lib.nabla_qk_norm_rope_bwd_workspace_bytes.argtypes = [i32]
    lib.nabla_qk_norm_rope_bwd.restype = i32
    lib.nabla_qk_norm_rope_bwd.argtypes = qk + [vp, st, vp, st, vp, st, vp, st, vp, vp, vp, sz, vp]
    xs = [i32, i32, i32, i32, i32, i32, i32]  # dtype, B, Sq, Sk, h, hk, D
    lib.nabla_cross_attn_fwd_workspace_bytes.restype = sz
    lib.nabla_cross_attn_fwd_workspace_bytes.argtypes = xs
    lib.nabla_cross_attn_fwd.restype = i32
    lib.nabla_cross_attn_fwd.argtypes = [vp, st, vp, st, vp, st] + xs + [vp, f32, vp, vp, vp, sz, vp]
    lib.nabla_cross_attn_bwd_workspace_bytes.restype = sz
    lib.nabla_cross_attn_bwd_workspace_bytes.argtypes = xs
    lib.nabla_cross_attn_bwd.restype = i32
    lib.nabla_cross_attn_bwd.argtypes = ([vp, st, vp, st, vp, st, vp, st, vp, vp, st] + xs +
                                         [vp, f32, vp, vp, vp, vp, sz, vp])
    lib.nabla_diff_attn_fwd_workspace_bytes.restype = sz
    lib.nabla_diff_attn_fwd_workspace_bytes.argtypes = xs
    lib.nabla_diff_attn_fwd.restype = i32
    lib.nabla_diff_attn_fwd.argtypes = ([vp, st] * 3 + xs +
                                        [vp, i32, vp, f32, vp, vp, vp, vp, sz, vp])
    lib.nabla_diff_attn_bwd_workspace_bytes.restype = sz
    lib.nabla_diff_attn_bwd_workspace_bytes.argtypes = xs
    lib.nabla_diff_attn_bwd.restype = i32
    lib.nabla_diff_attn_bwd.argtypes = ([vp, st] * 5 + [vp, vp, st] + xs +
                                        [vp, i32, vp, f32, vp, vp, vp, vp, vp, sz, vp])
    i64 = ctypes.c_int64
    mods = [vp, i64, vp, i64]  # gate, scale
    lib.nabla_block_norm.restype = i32
    lib.nabla_block_norm.argtypes = ([vp, st, vp, st, i32, i32, i32, i32, i32, i32, vp, vp, i32] +
                                     mods + [vp, i64, i32, i32, f32, f32, vp, st, vp, st, vp])
    lib.nabla_block_norm_bwd_workspace_bytes.restype = sz
    lib.nabla_block_norm_bwd_workspace_bytes.argtypes = [i32, i32, i32]
    lib.nabla_block_norm_bwd.restype = i32
    lib.nabla_block_norm_bwd.argtypes = (
        [vp, st] * 4 + [i32, i32, i32, i32, i32, i32, vp, vp, i32] + mods +
        [i32, i32, f32, f32, vp, st, vp, st, vp, vp, vp, vp, vp, vp, sz, vp])
    lib.nabla_selftest_bounded_wait.restype = i32
    lib.nabla_selftest_bounded_wait.argtypes = [vp]
    lib.nabla_get_last_device_status.restype = i32
    lib.nabla_get_last_device_status.argtypes = [vp]
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream, device: torch.device) -> Optional[int]:
    """The cudaStream_t to launch on: the given one, else torch's current stream of
    the tensors' device (not of whichever device happens to be current)."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(device: torch.device, fn, *args) -> int:
    """Run one C-ABI call with the tensors' device current: the library launches on,
    and takes its per-device state from, the current device."""
    with torch.cuda.device(device):
        return fn(*args)


def _run(device: torch.device, stream, fn, where: str, *args) -> None:
    """One C-ABI call whose last argument is the stream, on the tensors' device, raising
    what it returns.  The device is switched only where another one is current, and the
    default stream is asked for by number: a small call is a few microseconds of GPU work,
    and both would cost it as much again."""
    index = device.index
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream = _stream(stream, device)
    if torch.cuda.current_device() == index:
        st = fn(*args, stream)
    else:
        st = _call(device, fn, *args, stream)
    if st != NABLA_OK:
        raise NablaError(st, where)


def _allocators(stream, device: torch.device):
    """torch.empty for the outputs and for the scratch of a call on `stream`.

    The caching allocator hands a freed block out again in the order of the stream it was
    allocated on.  A block of the current stream would go to the next allocation there,
    or to a call on a third stream, while this call's kernels on `stream` still use it
    (its scratch is dropped when the call returns), and might itself still be in use by
    work of the current stream.  So both come from `stream`, and the outputs, which the
    caller goes on using, are also kept until the current stream is done with them."""
    if stream is None or device.type != "cuda":
        return torch.empty, torch.empty
    handle = _stream(stream, device)
    current = torch.cuda.current_stream(device)
    if handle == current.cuda_stream:
        return torch.empty, torch.empty
    if handle in (0, 1):  # 1: cudaStreamLegacy, the default stream's other name
        stream = torch.cuda.default_stream(device)
    elif not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device)

    def scratch(*size, **kw):
        with torch.cuda.stream(stream):
            return torch.empty(*size, **kw)

    def outputs(*size, **kw):
        t = scratch(*size, **kw)
        t.record_stream(current)
        return t

    return outputs, scratch


def _like(t: torch.Tensor, empty) -> torch.Tensor:
    """A dense tensor of t's shape and type from `empty` (see _allocators)."""
    if empty is torch.empty:  # a microsecond less of a small call
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return empty(t.shape, dtype=t.dtype, device=t.device)


@functools.lru_cache(maxsize=1024)
def _bytes(name: str, *shape) -> int:
    """What the library's function `name` says of a shape, which alone it depends on."""
    return getattr(load(), name)(*shape)


def _dtype_code_of(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return NABLA_BF16
    if dtype == torch.float32:
        return NABLA_F32
    raise TypeError(f"unsupported dtype {dtype}")


def _dtype_code(t: torch.Tensor) -> int:
    return _dtype_code_of(t.dtype)


def _check(status: int, where: str) -> None:
    if status != NABLA_OK:
        raise NablaError(status, where)


def _shape(q: torch.Tensor) -> Tuple[int, int, int, int]:
    if q.dim() != 4:
        raise ValueError("q/k/v must be [B, S, h, D]")
    if not q.is_contiguous():
        raise ValueError("q/k/v must be contiguous [B, S, h, D]")
    return tuple(q.shape)


# The C ABI receives bare pointers and cannot see a buffer's size, element type
# or device, so every tensor handed to it is checked here first: a short or
# mistyped buffer, or one in host memory, would otherwise be read or written
# out of bounds by the kernels.
def _on(t: torch.Tensor, name: str, device: torch.device) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _buf(t: torch.Tensor, name: str, numel: int, dtype: torch.dtype,
         device: torch.device) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    _on(t, name, device)


def _rows(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype,
          device: torch.device) -> Optional[_Strides]:
    """Checks a [B, S, h, D] tensor that may be a view of a larger one, or lie in another
    order, and returns its strides for the C ABI."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.is_contiguous():
        return None  # dense
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"the columns of {name} must lie together")
    span = t.shape[3]
    for s, n in sorted((s, n) for s, n in zip(st[:3], t.shape) if n > 1):
        if s < span:
            raise ValueError(f"the rows of {name} must not overlap (an expanded tensor has to be "
                             "made contiguous)")
        span += s * (n - 1)
    return _Strides(*st[:3])


def _cuda(t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")


def _csr(kv_nb: torch.Tensor, kv_inds: torch.Tensor, B: int, h: int, s1: int,
         device: torch.device) -> None:
    _buf(kv_nb, "kv_nb", B * h * s1, torch.int32, device)
    _buf(kv_inds, "kv_inds", B * h * s1 * s1, torch.int32, device)


def nabla_abi_version() -> int:
    return load().nabla_abi_version()


def nabla_status_string(status: int) -> str:
    return load().nabla_status_string(int(status)).decode()


def nabla_build_mask_workspace_bytes(B: int, S: int, h: int, D: int) -> int:
    return load().nabla_build_mask_workspace_bytes(B, S, h, D)


def nabla_build_mask(q: torch.Tensor, k: torch.Tensor, sta: torch.Tensor, thr: float,
                     kv_nb: Optional[torch.Tensor] = None,
                     kv_inds: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """(q, k [B,S,h,D], sta [s1,s1] uint8, thr) -> (kv_nb [B,h,s1], kv_inds [B,h,s1,s1]) int32."""
    lib = load()
    B, S, h, D = _shape(q)
    if k.shape != q.shape or k.dtype != q.dtype:
        raise ValueError("k must match q")
    s1 = S // 64
    dev = q.device
    empty, scratch = _allocators(stream, dev)
    if kv_nb is None:
        kv_nb = empty((B, h, s1), dtype=torch.int32, device=dev)
    if kv_inds is None:
        kv_inds = empty((B, h, s1, s1), dtype=torch.int32, device=dev)
    _on(k, "k", dev)
    _buf(sta, "sta", s1 * s1, torch.uint8, dev)
    _csr(kv_nb, kv_inds, B, h, s1, dev)
    need = lib.nabla_build_mask_workspace_bytes(B, S, h, D)
    if workspace is None:
        workspace = scratch(max(need, 1), dtype=torch.uint8, device=dev)
    _on(workspace, "workspace", dev)
    _cuda(q)
    st = _call(dev, lib.nabla_build_mask, _ptr(q), _ptr(k), _dtype_code(q), B, S, h, D, _ptr(sta),
               float(thr), _ptr(kv_nb), _ptr(kv_inds), _ptr(workspace),
               workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check(st, "nabla_build_mask")
    return kv_nb, kv_inds


def nabla_build_mask_noalloc(q: torch.Tensor, k: torch.Tensor, sta: torch.Tensor, thr: float,
                             kv_nb: torch.Tensor, kv_inds: torch.Tensor, stream=None):
    """nabla_build_mask without a workspace: the library's fixed device scratch is
    used instead (see include/nabla.h); outputs must be preallocated by the caller."""
    B, S, h, D = _shape(q)
    if k.shape != q.shape or k.dtype != q.dtype:
        raise ValueError("k must match q")
    s1 = S // 64
    _on(k, "k", q.device)
    _buf(sta, "sta", s1 * s1, torch.uint8, q.device)
    _csr(kv_nb, kv_inds, B, h, s1, q.device)
    _cuda(q)
    st = _call(q.device, load().nabla_build_mask_noalloc, _ptr(q), _ptr(k), _dtype_code(q), B, S,
               h, D, _ptr(sta), float(thr), _ptr(kv_nb), _ptr(kv_inds), _stream(stream, q.device))
    _check(st, "nabla_build_mask_noalloc")
    return kv_nb, kv_inds


def nabla_build_mask_topk(q: torch.Tensor, k: torch.Tensor, topk_ratio: float,
                          kv_nb: Optional[torch.Tensor] = None,
                          kv_inds: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """Top-k block selector (sla.get_block_map): (q, k [B,S,h,D], topk_ratio) ->
    (kv_nb [B,h,s1], kv_inds [B,h,s1,s1]) int32, kept blocks ascending."""
    lib = load()
    B, S, h, D = _shape(q)
    if k.shape != q.shape or k.dtype != q.dtype:
        raise ValueError("k must match q")
    s1 = S // 64
    dev = q.device
    empty, scratch = _allocators(stream, dev)
    if kv_nb is None:
        kv_nb = empty((B, h, s1), dtype=torch.int32, device=dev)
    if kv_inds is None:
        kv_inds = empty((B, h, s1, s1), dtype=torch.int32, device=dev)
    _on(k, "k", dev)
    _csr(kv_nb, kv_inds, B, h, s1, dev)
    need = lib.nabla_build_mask_workspace_bytes(B, S, h, D)
    if workspace is None:
        workspace = scratch(max(need, 1), dtype=torch.uint8, device=dev)
    _on(workspace, "workspace", dev)
    _cuda(q)
    st = _call(dev, lib.nabla_build_mask_topk, _ptr(q), _ptr(k), _dtype_code(q), B, S, h, D,
               float(topk_ratio), _ptr(kv_nb), _ptr(kv_inds), _ptr(workspace),
               workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check(st, "nabla_build_mask_topk")
    return kv_nb, kv_inds


def nabla_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_nb: torch.Tensor,
                   kv_inds: torch.Tensor, scale: Optional[float] = None,
                   o: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Block-sparse attention over the kept 64x64 blocks; returns o [B,S,h,D]."""
    lib = load()
    B, S, h, D = _shape(q)
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k, v must match q")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if o is None:
        o = _allocators(stream, q.device)[0](q.shape, dtype=q.dtype, device=q.device)
    _on(k, "k", q.device)
    _on(v, "v", q.device)
    _csr(kv_nb, kv_inds, B, h, S // 64, q.device)
    _buf(o, "o", q.numel(), q.dtype, q.device)
    _cuda(q)
    st = _call(q.device, lib.nabla_attn_fwd, _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), B, S, h, D,
               _ptr(kv_nb), _ptr(kv_inds), float(scale), _ptr(o), _stream(stream, q.device))
    _check(st, "nabla_attn_fwd")
    return o


def nabla_attn_bwd_workspace_bytes(B: int, S: int, h: int, D: int) -> int:
    return load().nabla_attn_bwd_workspace_bytes(B, S, h, D)


def nabla_attn_fwd_lse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_nb: torch.Tensor,
                       kv_inds: torch.Tensor, scale: Optional[float] = None,
                       o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       stream=None):
    """nabla_attn_fwd that also returns the rows' base-2 log-sum-exp: (o, lse [B,h,S] fp32)."""
    lib = load()
    B, S, h, D = _shape(q)
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k, v must match q")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    empty, _ = _allocators(stream, q.device)
    o = empty(q.shape, dtype=q.dtype, device=q.device) if o is None else o
    lse = empty((B, h, S), dtype=torch.float32, device=q.device) if lse is None else lse
    _on(k, "k", q.device)
    _on(v, "v", q.device)
    _csr(kv_nb, kv_inds, B, h, S // 64, q.device)
    _buf(o, "o", q.numel(), q.dtype, q.device)
    _buf(lse, "lse", B * h * S, torch.float32, q.device)
    _cuda(q)
    st = _call(q.device, lib.nabla_attn_fwd_lse, _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), B, S,
               h, D, _ptr(kv_nb), _ptr(kv_inds), float(scale), _ptr(o), _ptr(lse),
               _stream(stream, q.device))
    _check(st, "nabla_attn_fwd_lse")
    return o, lse


def nabla_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                   dout: torch.Tensor, kv_nb: torch.Tensor, kv_inds: torch.Tensor,
                   scale: Optional[float] = None, dq: Optional[torch.Tensor] = None,
                   dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   stream=None):
    """Gradients of nabla_attn_fwd: returns (dq, dk, dv), each [B,S,h,D] in q's dtype.
    lse: the forward's log-sum-exp from nabla_attn_fwd_lse (computed here if None)."""
    lib = load()
    B, S, h, D = _shape(q)
    for t in (k, v, o, dout):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError("k, v, o, dout must match q")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    empty, scratch = _allocators(stream, q.device)
    dq, dk, dv = (empty(q.shape, dtype=q.dtype, device=q.device) if t is None else t
                  for t in (dq, dk, dv))
    for name, t in (("k", k), ("v", v), ("o", o), ("dout", dout)):
        _on(t, name, q.device)
    _csr(kv_nb, kv_inds, B, h, S // 64, q.device)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _buf(t, name, q.numel(), q.dtype, q.device)
    if lse is not None:
        _buf(lse, "lse", B * h * S, torch.float32, q.device)
    need = lib.nabla_attn_bwd_workspace_bytes(B, S, h, D)
    if workspace is None:
        workspace = scratch(max(need, 1), dtype=torch.uint8, device=q.device)
    _on(workspace, "workspace", q.device)
    _cuda(q)
    st = _call(q.device, lib.nabla_attn_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
               _ptr(dout), _dtype_code(q), B, S, h, D, _ptr(kv_nb), _ptr(kv_inds), float(scale),
               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
               workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    _check(st, "nabla_attn_bwd")
    return dq, dk, dv


def nabla_sta_mask(T: int, H: int, W: int, wt: int, wh: int, ww: int, device=None,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """STA window [s1, s1] uint8 on the (T, H, W) block grid."""
    lib = load()
    s1 = T * H * W
    if out is None:
        dev = torch.device(device or "cuda")
        out = _allocators(stream, dev)[0]((s1, s1), dtype=torch.uint8, device=dev)
    _buf(out, "out", s1 * s1, torch.uint8, out.device)
    _cuda(out)
    st = _call(out.device, lib.nabla_sta_mask, T, H, W, wt, wh, ww, _ptr(out),
               _stream(stream, out.device))
    _check(st, "nabla_sta_mask")
    return out


def nabla_fractal_flatten(x: torch.Tensor, P: int = 8, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """x [B, T, H, W, h, D] (raster token order) -> [B, T*H*W, h, D] in fractal order."""
    if x.dim() != 6 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [B, T, H, W, h, D] tensor")
    B, T, H, W, h, D = x.shape
    if out is None:
        out = _allocators(stream, x.device)[0]((B, T * H * W, h, D), dtype=x.dtype,
                                               device=x.device)
    _buf(out, "out", x.numel(), x.dtype, x.device)
    _cuda(x)
    st = _call(x.device, load().nabla_fractal_flatten, _ptr(x), _dtype_code(x), B, T, H, W, h, D,
               P, _ptr(out), _stream(stream, x.device))
    _check(st, "nabla_fractal_flatten")
    return out


def nabla_fractal_unflatten(y: torch.Tensor, T: int, H: int, W: int, P: int = 8,
                            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [B, T*H*W, h, D] in fractal order -> [B, T, H, W, h, D] in raster order."""
    if y.dim() != 4 or y.shape[1] != T * H * W or not y.is_contiguous():
        raise ValueError("y must be a contiguous [B, T*H*W, h, D] tensor")
    B, _, h, D = y.shape
    if out is None:
        out = _allocators(stream, y.device)[0]((B, T, H, W, h, D), dtype=y.dtype,
                                               device=y.device)
    _buf(out, "out", y.numel(), y.dtype, y.device)
    _cuda(y)
    st = _call(y.device, load().nabla_fractal_unflatten, _ptr(y), _dtype_code(y), B, T, H, W, h, D,
               P, _ptr(out), _stream(stream, y.device))
    _check(st, "nabla_fractal_unflatten")
    return out


def _qk_args(q, k, wq, wk, cos, sin, pos, interleaved, eps):
    """Checks what the query/key norm and its backward have in common and returns the
    C arguments up to eps, the two tensors' shapes and the weights' type."""
    if q.dim() != 4:
        raise ValueError("q must be [B, S, h, D]")
    B, S, hq, D = q_shape = q.shape
    dev, dtype = q.device, q.dtype
    hk, k_shape, k_ptr, k_st = 0, None, None, None
    q_st = _rows(q, "q", q_shape, dtype, dev)
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be [B, S, h, D]")
        k_shape = k.shape
        hk = k_shape[2]
        k_st = _rows(k, "k", (B, S, hk, D), dtype, dev)
        k_ptr = k.data_ptr()
    kind, wcode = torch.float32, NABLA_F32
    w = wq if wq is not None else wk
    if w is not None:
        kind, wcode = w.dtype, _dtype_code(w)
        for name, w in (("wq", wq), ("wk", wk)):
            if w is not None:
                _buf(w, name, D, kind, dev)
                if w.numel() != D:
                    raise ValueError(f"{name} must be [{D}], got {tuple(w.shape)}")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    R = n = 0
    if cos is not None:
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [rows, R / 2], of the same shape")
        n, half = cos.shape
        R = 2 * half
        _buf(cos, "cos", n * half, torch.float32, dev)
        _buf(sin, "sin", n * half, torch.float32, dev)
    if pos is not None:
        if cos is None or pos.shape != (B, S):
            raise ValueError(f"pos must be [{B}, {S}], with cos and sin")
        _buf(pos, "pos", B * S, torch.int32, dev)
    return (q.data_ptr(), q_st, k_ptr, k_st, _dtype_code(q), B, S, hq, hk, D, _ptr(wq), _ptr(wk),
            wcode, _ptr(cos), _ptr(sin), n, R, 1 if interleaved else 0, _ptr(pos),
            eps), q_shape, k_shape, kind


def nabla_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None,
                       wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None,
                       cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
                       pos: Optional[torch.Tensor] = None, interleaved: bool = True,
                       eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
                       k_out: Optional[torch.Tensor] = None, stream=None):
    """RMS norm of q [B,S,hq,D] and k [B,S,hk,D] (or q alone) per head with weights
    wq, wk [D] (None: 1) and, with cos, sin [rows, R/2] fp32, the position rotation of
    their first R columns; token s takes table row s, or pos[b, s].  interleaved:
    rotate columns (2i, 2i + 1), else (i, i + R/2).  q, k and the outputs may be views of
    larger tensors with their dimensions in any order in memory, as long as a row's columns
    lie together and no two rows overlap.  Returns (q_out, k_out)."""
    args, q_shape, k_shape, _ = _qk_args(q, k, wq, wk, cos, sin, pos, interleaved, eps)
    dev = q.device
    empty, _ = _allocators(stream, dev)
    qo = ko = None
    if q_out is None:
        q_out = empty(q_shape, dtype=q.dtype, device=dev)
    else:
        qo = _rows(q_out, "q_out", q_shape, q.dtype, dev)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
    elif k_out is None:
        k_out = empty(k_shape, dtype=q.dtype, device=dev)
    else:
        ko = _rows(k_out, "k_out", k_shape, q.dtype, dev)
    _cuda(q)
    _run(dev, stream, load().nabla_qk_norm_rope, "nabla_qk_norm_rope", *args, q_out.data_ptr(), qo,
         _ptr(k_out), ko)
    return q_out, k_out


def nabla_qk_norm_rope_bwd_workspace_bytes(D: int) -> int:
    return load().nabla_qk_norm_rope_bwd_workspace_bytes(D)


def nabla_qk_norm_rope_bwd(q: torch.Tensor, k: Optional[torch.Tensor],
                           wq: Optional[torch.Tensor], wk: Optional[torch.Tensor],
                           dq_out: torch.Tensor, dk_out: Optional[torch.Tensor] = None,
                           cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
                           pos: Optional[torch.Tensor] = None, interleaved: bool = True,
                           eps: float = 1e-6, dq: Optional[torch.Tensor] = None,
                           dk: Optional[torch.Tensor] = None, dwq: Optional[torch.Tensor] = None,
                           dwk: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of nabla_qk_norm_rope for the upstream gradients dq_out, dk_out of its
    outputs: returns (dq, dk, dwq, dwk); dwq, dwk [D] in the weights' type, None where
    the weight is None.  dq_out, dk_out, dq and dk may be views as there; an expanded
    gradient (that of a plain sum) has to be made contiguous first."""
    args, q_shape, k_shape, kind = _qk_args(q, k, wq, wk, cos, sin, pos, interleaved, eps)
    dev, dtype, D = q.device, q.dtype, q.shape[3]
    if dq_out is None or (k is None) != (dk_out is None):
        raise ValueError("dq_out and, with k, dk_out are needed")
    if k is None and (dk is not None or wk is not None):
        raise ValueError("dk or wk without k")
    zq, zk = _rows(dq_out, "dq_out", q_shape, dtype, dev), _rows(dk_out, "dk_out", k_shape, dtype,
                                                                 dev)
    empty, scratch = _allocators(stream, dev)
    oq = ok = None
    if dq is None:
        dq = empty(q_shape, dtype=dtype, device=dev)
    else:
        oq = _rows(dq, "dq", q_shape, dtype, dev)
    if k is not None:
        if dk is None:
            dk = empty(k_shape, dtype=dtype, device=dev)
        else:
            ok = _rows(dk, "dk", k_shape, dtype, dev)
    for name, d, w in (("dwq", dwq, wq), ("dwk", dwk, wk)):
        if d is not None:
            if w is None:
                raise ValueError(f"{name} without its weight")
            _buf(d, name, D, kind, dev)
    if dwq is None and wq is not None:
        dwq = empty(D, dtype=kind, device=dev)
    if dwk is None and wk is not None:
        dwk = empty(D, dtype=kind, device=dev)
    lib = load()
    if workspace is None and (dwq is not None or dwk is not None):
        workspace = scratch(lib.nabla_qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8,
                            device=dev)
    if workspace is not None:
        _on(workspace, "workspace", dev)
    _cuda(q)
    _run(dev, stream, lib.nabla_qk_norm_rope_bwd, "nabla_qk_norm_rope_bwd", *args,
         dq_out.data_ptr(), zq, _ptr(dk_out), zk, dq.data_ptr(), oq, _ptr(dk), ok, _ptr(dwq),
         _ptr(dwk), _ptr(workspace),
         0 if workspace is None else workspace.numel() * workspace.element_size())
    return dq, dk, dwq, dwk


def _cross_args(q, k, v, kv_len):
    """Checks q, k, v and kv_len of a cross attention; returns the C ABI's strides and
    its (dtype, B, Sq, Sk, h, hk, D)."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        name = "q" if q.dim() != 4 else "k" if k.dim() != 4 else "v"
        raise ValueError(f"{name} must be [B, S, h, D]")
    B, Sq, h, D = q.shape
    Sk, hk = k.shape[1:3]
    dev, dtype = q.device, q.dtype
    kv = (B, Sk, hk, D)
    strides = (_rows(q, "q", q.shape, dtype, dev), _rows(k, "k", kv, dtype, dev),
               _rows(v, "v", kv, dtype, dev))
    if kv_len is not None:
        if kv_len.shape != (B,):
            raise ValueError(f"kv_len must be [{B}], got {tuple(kv_len.shape)}")
        _buf(kv_len, "kv_len", B, torch.int32, dev)
    return strides, (_dtype_code(q), B, Sq, Sk, h, hk, D)


def nabla_cross_attn_fwd_workspace_bytes(dtype: torch.dtype, B: int, Sq: int, Sk: int, h: int,
                                         hk: int, D: int) -> int:
    code = NABLA_BF16 if dtype == torch.bfloat16 else NABLA_F32
    return load().nabla_cross_attn_fwd_workspace_bytes(code, B, Sq, Sk, h, hk, D)


def _cross_fwd(q, k, v, kv_len, scale, o, lse, with_lse, workspace, stream):
    strides, sizes = _cross_args(q, k, v, kv_len)
    dev = q.device
    empty, scratch = _allocators(stream, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(sizes[-1])
    if o is None:
        o = empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _buf(o, "o", q.numel(), q.dtype, dev)
    if lse is not None:
        _buf(lse, "lse", q.numel() // sizes[-1], torch.float32, dev)
    elif with_lse:
        lse = empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=dev)
    lib = load()
    if workspace is None:
        need = lib.nabla_cross_attn_fwd_workspace_bytes(*sizes)
        if need:
            workspace = scratch(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _on(workspace, "workspace", dev)
    _cuda(q)
    _run(dev, stream, lib.nabla_cross_attn_fwd, "nabla_cross_attn_fwd", q.data_ptr(), strides[0],
         k.data_ptr(), strides[1], v.data_ptr(), strides[2], *sizes, _ptr(kv_len), scale,
         o.data_ptr(), _ptr(lse), _ptr(workspace),
         0 if workspace is None else workspace.numel() * workspace.element_size())
    return o, lse


def nabla_cross_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         kv_len: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                         o: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of q [B,Sq,h,D] to the first kv_len[b] (int32 [B]; None: all) of the
    states k, v [B,Sk,hk,D], hk dividing h; q, k and v may be views of larger tensors with
    their dimensions in any order in memory, as long as a row's columns lie together and no
    two rows overlap.  Returns o [B,Sq,h,D], dense."""
    return _cross_fwd(q, k, v, kv_len, scale, o, None, False, workspace, stream)[0]


def nabla_cross_attn_fwd_lse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             kv_len: Optional[torch.Tensor] = None,
                             scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None):
    """nabla_cross_attn_fwd that also returns the rows' base-2 log-sum-exp:
    (o, lse [B,h,Sq] fp32)."""
    return _cross_fwd(q, k, v, kv_len, scale, o, lse, True, workspace, stream)


def nabla_cross_attn_bwd_workspace_bytes(dtype: torch.dtype, B: int, Sq: int, Sk: int, h: int,
                                         hk: int, D: int) -> int:
    code = NABLA_BF16 if dtype == torch.bfloat16 else NABLA_F32
    return load().nabla_cross_attn_bwd_workspace_bytes(code, B, Sq, Sk, h, hk, D)


def nabla_cross_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         lse: torch.Tensor, dout: torch.Tensor,
                         kv_len: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                         dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                         dv: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of nabla_cross_attn_fwd, from its inputs, the o and lse of
    nabla_cross_attn_fwd_lse and the upstream gradient dout of o: returns dq [B,Sq,h,D] and
    dk, dv [B,Sk,hk,D] (0 for states past kv_len), dense.  o and dout may be views as q, k
    and v may; an expanded dout (the gradient of a plain sum) has to be made contiguous
    first."""
    strides, sizes = _cross_args(q, k, v, kv_len)
    dev = q.device
    so, sg = _rows(o, "o", q.shape, q.dtype, dev), _rows(dout, "dout", q.shape, q.dtype, dev)
    _buf(lse, "lse", q.numel() // sizes[-1], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(sizes[-1])
    empty, scratch = _allocators(stream, dev)
    outs = []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, k)):
        if t is None:
            t = empty(like.shape, dtype=q.dtype, device=dev)
        else:
            _buf(t, name, like.numel(), q.dtype, dev)
        outs.append(t)
    dq, dk, dv = outs
    lib = load()
    if workspace is None:
        need = lib.nabla_cross_attn_bwd_workspace_bytes(*sizes)
        workspace = scratch(max(need, 1), dtype=torch.uint8, device=dev)
    _on(workspace, "workspace", dev)
    _cuda(q)
    _run(dev, stream, lib.nabla_cross_attn_bwd, "nabla_cross_attn_bwd", q.data_ptr(), strides[0],
         k.data_ptr(), strides[1], v.data_ptr(), strides[2], o.data_ptr(), so, lse.data_ptr(),
         dout.data_ptr(), sg, *sizes, _ptr(kv_len), scale, dq.data_ptr(), dk.data_ptr(),
         dv.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dq, dk, dv


def _lam(lam: torch.Tensor, h: int, device: torch.device) -> int:
    if lam.dim() != 1 or lam.numel() not in (1, h):
        raise ValueError(f"lam must be [{h}] or [1], got {list(lam.shape)}")
    _buf(lam, "lam", lam.numel(), torch.float32, device)
    return lam.numel()


def nabla_diff_attn_fwd_workspace_bytes(dtype: torch.dtype, B: int, Sq: int, Sk: int, h: int,
                                        hk: int, D: int) -> int:
    code = NABLA_BF16 if dtype == torch.bfloat16 else NABLA_F32
    return load().nabla_diff_attn_fwd_workspace_bytes(code, B, Sq, Sk, h, hk, D)


def _diff_fwd(q, k, v, lam, kv_len, scale, o, o2, lse, whole, workspace, stream):
    strides, sizes = _cross_args(q, k, v, kv_len)
    dev = q.device
    n = _lam(lam, sizes[4], dev)
    empty, scratch = _allocators(stream, dev)
    if scale is None:
        scale = math.sqrt(2.0 / sizes[-1])
    if o is None:
        o = _like(q, empty)
    else:
        _buf(o, "o", q.numel(), q.dtype, dev)
    if whole:
        if o2 is None:
            o2 = _like(q, empty)
        else:
            _buf(o2, "o2", q.numel(), q.dtype, dev)
        if lse is None:
            lse = empty((q.shape[0], q.shape[2], 2, q.shape[1]), dtype=torch.float32, device=dev)
        else:
            _buf(lse, "lse", 2 * q.numel() // sizes[-1], torch.float32, dev)
    lib = load()
    if workspace is None:
        need = _bytes("nabla_diff_attn_fwd_workspace_bytes", *sizes)
        if need:
            workspace = scratch(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _on(workspace, "workspace", dev)
    _cuda(q)
    _run(dev, stream, lib.nabla_diff_attn_fwd, "nabla_diff_attn_fwd", q.data_ptr(), strides[0],
         k.data_ptr(), strides[1], v.data_ptr(), strides[2], *sizes, lam.data_ptr(), n,
         _ptr(kv_len), scale, o.data_ptr(), _ptr(o2), _ptr(lse), _ptr(workspace),
         0 if workspace is None else workspace.numel() * workspace.element_size())
    return o, o2, lse


def nabla_diff_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
                        kv_len: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                        o: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Differential attention of q [B,Sq,h,D] to the first kv_len[b] (int32 [B]; None: all) of
    the states k, v [B,Sk,hk,D], hk dividing h: softmax of the scores of the first D / 2
    columns of q and k minus lam (fp32 [h] or [1]) times that of the last D / 2, times v.
    scale None: 1 / sqrt(D / 2).  q, k and v may be views as for nabla_cross_attn_fwd; heads
    2i and 2i + 1 of [B,S,2h,D/2] viewed as [B,S,h,D] are head i.  Returns o [B,Sq,h,D], dense."""
    return _diff_fwd(q, k, v, lam, kv_len, scale, o, None, None, False, workspace, stream)[0]


def nabla_diff_attn_fwd_lse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
                            kv_len: Optional[torch.Tensor] = None,
                            scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                            o2: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None):
    """nabla_diff_attn_fwd that also returns what its backward needs: (o, o2, lse) with the
    second map's rows o2 [B,Sq,h,D] and the maps' base-2 log-sum-exp lse [B,h,2,Sq] fp32."""
    return _diff_fwd(q, k, v, lam, kv_len, scale, o, o2, lse, True, workspace, stream)


def nabla_diff_attn_bwd_workspace_bytes(dtype: torch.dtype, B: int, Sq: int, Sk: int, h: int,
                                        hk: int, D: int) -> int:
    code = NABLA_BF16 if dtype == torch.bfloat16 else NABLA_F32
    return load().nabla_diff_attn_bwd_workspace_bytes(code, B, Sq, Sk, h, hk, D)


def nabla_diff_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
                        o: torch.Tensor, o2: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor,
                        kv_len: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                        dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                        dv: Optional[torch.Tensor] = None, dlam: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of nabla_diff_attn_fwd, from its inputs, what nabla_diff_attn_fwd_lse returned
    and the upstream gradient dout of o: returns dq [B,Sq,h,D], dk, dv [B,Sk,hk,D] (0 for states
    past kv_len), dense, and dlam in lam's shape.  o, o2 and dout may be views as q, k and v
    may; an expanded dout (the gradient of a plain sum) has to be made contiguous first."""
    strides, sizes = _cross_args(q, k, v, kv_len)
    dev = q.device
    n = _lam(lam, sizes[4], dev)
    so, s2, sg = (_rows(t, name, q.shape, q.dtype, dev)
                  for name, t in (("o", o), ("o2", o2), ("dout", dout)))
    _buf(lse, "lse", 2 * q.numel() // sizes[-1], torch.float32, dev)
    if scale is None:
        scale = math.sqrt(2.0 / sizes[-1])
    empty, scratch = _allocators(stream, dev)
    outs = []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, k), ("dlam", dlam, lam)):
        if t is None:
            t = _like(like, empty)
        else:
            _buf(t, name, like.numel(), like.dtype, dev)
        outs.append(t)
    lib = load()
    if workspace is None:
        workspace = scratch(_bytes("nabla_diff_attn_bwd_workspace_bytes", *sizes) or 1,
                            dtype=torch.uint8, device=dev)
    _on(workspace, "workspace", dev)
    _cuda(q)
    _run(dev, stream, lib.nabla_diff_attn_bwd, "nabla_diff_attn_bwd", q.data_ptr(), strides[0],
         k.data_ptr(), strides[1], v.data_ptr(), strides[2], o.data_ptr(), so, o2.data_ptr(), s2,
         lse.data_ptr(), dout.data_ptr(), sg, *sizes, lam.data_ptr(), n, _ptr(kv_len), scale,
         *(t.data_ptr() for t in outs), workspace.data_ptr(),
         workspace.numel() * workspace.element_size())
    return tuple(outs)


_NORMS = {None: 0, "rms": 1, "layer": 2}


def _plane(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype,
           device: torch.device) -> Optional[_Strides]:
    """_rows of a [B, S, C] tensor."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        if t.dim() != 3 or t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        return _rows(t.unsqueeze(2), name, (shape[0], shape[1], 1, shape[2]), dtype, device)
    return None


def _mod(t: torch.Tensor, name: str, B: int, S: int, C: int,
         device: torch.device) -> Tuple[int, int]:
    """Checks a modulation [C], [B, C] or [B, m, C] with m dividing S, which may be a view of
    a projection that holds several, and returns its number of rows and their distance."""
    shape = t.shape
    k = len(shape)
    if not 1 <= k <= 3 or shape[-1] != C or (k > 1 and shape[0] != B) or (
            k == 3 and (shape[1] < 1 or S % shape[1])):
        raise ValueError(f"{name} must be [{C}], [{B}, {C}] or [{B}, m, {C}] with m dividing {S}, "
                         f"got {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"the columns of {name} must lie together")
    if k == 1:
        return 1, C
    if k == 2:
        return B, st[0]
    m = shape[1]
    if B > 1 and m > 1 and st[0] != m * st[1]:
        raise ValueError(f"the rows of {name} must lie equally far apart (make it contiguous)")
    return B * m, st[1] if m > 1 else st[0]


def _norm_weight(w: torch.Tensor, name: str, C: int, kind, device: torch.device) -> int:
    _buf(w, name, C, w.dtype if kind is None else kind, device)
    if w.numel() != C:
        raise ValueError(f"{name} must be [{C}], got {list(w.shape)}")
    return w.data_ptr()


def _norm_args(like, u, gate, scale, shift, weight, post_weight, norm, post_norm, residual_scale,
               eps):
    """Checks what nabla_block_norm and its backward have in common; `like`: a [B, S, C]
    tensor.  Returns the shape, the C arguments from dt to the scale, the shift's two, and the
    rest to eps."""
    shape = like.shape
    if len(shape) != 3:
        raise ValueError("the tensors must be [B, S, C]")
    if norm not in _NORMS or post_norm not in _NORMS:
        name, n = ("norm", norm) if norm not in _NORMS else ("post_norm", post_norm)
        raise ValueError(f"{name} must be None, 'rms' or 'layer', got {n!r}")
    B, S, C = shape
    dev = like.device
    kind = w = pw = None
    if weight is not None:
        w = _norm_weight(weight, "weight", C, None, dev)
        kind = weight.dtype
    if post_weight is not None:
        pw = _norm_weight(post_weight, "post_weight", C, kind, dev)
        kind = post_weight.dtype
    if norm is None and (weight is not None or scale is not None or shift is not None):
        raise ValueError("weight, scale and shift need a norm")
    if post_norm is None and post_weight is not None:
        raise ValueError("post_weight needs a post_norm")
    if u is None and (gate is not None or post_norm is not None):
        raise ValueError("gate and post_norm need u")
    rows, first, at = 1, None, []
    for name, m in (("gate", gate), ("scale", scale), ("shift", shift)):
        if m is None:
            at.append((None, 0))
            continue
        if first is not None and (m.shape != first.shape or m.dtype != first.dtype):
            raise ValueError(f"{name} must be {list(first.shape)} {first.dtype} as the other "
                             f"modulations are, got {list(m.shape)} {m.dtype}")
        first = m
        rows, step = _mod(m, name, B, S, C, dev)
        at.append((m.data_ptr(), step))
    head = (_dtype_code(like), B, S, C, _NORMS[norm], _NORMS[post_norm], w, pw,
            NABLA_F32 if kind is None else _dtype_code_of(kind), *at[0], *at[1])
    return shape, head, at[2], (NABLA_F32 if first is None else _dtype_code(first), rows,
                                residual_scale, eps)


def nabla_block_norm(x: torch.Tensor, u: Optional[torch.Tensor] = None,
                     gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                     shift: Optional[torch.Tensor] = None,
                     weight: Optional[torch.Tensor] = None,
                     post_weight: Optional[torch.Tensor] = None, norm: Optional[str] = "layer",
                     post_norm: Optional[str] = None, residual_scale: float = 1.0,
                     eps: float = 1e-6, x_out: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None, stream=None):
    """The gated sum after a block's branch and the adaptive norm before the next:
    s = x + residual_scale * gate * N(u) * post_weight with post_norm's N, and
    y = N(s) * weight * (1 + scale) + shift with norm's; N is "rms", "layer" or None.
    x and u [B,S,C]; u None: s = x, the norm alone; norm None: the sum alone.  gate, scale and
    shift are all [C], [B,C] or [B,m,C] (a row for each of m equal runs of a batch's tokens),
    views of one projection if need be; weight and post_weight [C]; None: 1 (shift: 0).
    x_out may be x.  x, u and the outputs may be views whose columns lie together.
    Returns (s, y); s is x where u is None, y None where norm is."""
    shape, head, sh, rest = _norm_args(x, u, gate, scale, shift, weight, post_weight, norm, post_norm,
                                       residual_scale, eps)
    dev, dtype = x.device, x.dtype
    if u is None and norm is None:
        raise ValueError("neither u nor a norm: nothing to compute")
    x_st, u_st = _plane(x, "x", shape, dtype, dev), _plane(u, "u", shape, dtype, dev)
    empty, _ = _allocators(stream, dev)
    xo_st = y_st = None
    if u is None:
        if x_out is not None:
            raise ValueError("x_out without u")
    elif x_out is None:
        x_out = _like(x, empty)
    else:
        xo_st = _plane(x_out, "x_out", shape, dtype, dev)
    if norm is None:
        if y is not None:
            raise ValueError("y without a norm")
    elif y is None:
        y = _like(x, empty)
    else:
        y_st = _plane(y, "y", shape, dtype, dev)
    _cuda(x)
    _run(dev, stream, load().nabla_block_norm, "nabla_block_norm", x.data_ptr(), x_st, _ptr(u),
         u_st, *head, *sh, *rest, _ptr(x_out), xo_st, _ptr(y), y_st)
    return (x if u is None else x_out), y


def nabla_block_norm_bwd_workspace_bytes(B: int, S: int, C: int) -> int:
    return load().nabla_block_norm_bwd_workspace_bytes(B, S, C)


def nabla_block_norm_bwd(s: Optional[torch.Tensor], u: Optional[torch.Tensor],
                         dsum: Optional[torch.Tensor], dy: Optional[torch.Tensor],
                         gate: Optional[torch.Tensor] = None,
                         scale: Optional[torch.Tensor] = None,
                         shift: Optional[torch.Tensor] = None,
                         weight: Optional[torch.Tensor] = None,
                         post_weight: Optional[torch.Tensor] = None,
                         norm: Optional[str] = "layer", post_norm: Optional[str] = None,
                         residual_scale: float = 1.0, eps: float = 1e-6,
                         dx: Optional[torch.Tensor] = None, du: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of nabla_block_norm, from the sum s it returned, u, and the upstream
    gradients dsum of s (None: 0) and dy of y, with the forward's other arguments: returns
    (dx, du, dgate, dscale, dshift, dweight, dpost_weight), None for what was not given.  s and
    dy are not looked at (and may be None) where norm is None.  dx may be dsum; s, u, dsum, dy,
    dx and du may be views as there."""
    if norm is None:
        s = dy = None
    like = dsum if s is None else s
    if like is None:
        raise ValueError("s and dy, or dsum, are needed")
    shape, head, _, rest = _norm_args(like, u, gate, scale, shift, weight, post_weight, norm,
                                      post_norm, residual_scale, eps)
    if norm is not None and dy is None:
        raise ValueError("dy is needed with a norm")
    dev, dtype = like.device, like.dtype
    s_st, u_st = _plane(s, "s", shape, dtype, dev), _plane(u, "u", shape, dtype, dev)
    ds_st, dy_st = _plane(dsum, "dsum", shape, dtype, dev), _plane(dy, "dy", shape, dtype, dev)
    empty, scratch = _allocators(stream, dev)
    dx_st = du_st = None
    if dx is None:
        dx = _like(like, empty)
    else:
        dx_st = _plane(dx, "dx", shape, dtype, dev)
    if u is None:
        if du is not None:
            raise ValueError("du without u")
    elif du is None:
        du = _like(like, empty)
    else:
        du_st = _plane(du, "du", shape, dtype, dev)
    small = [None if t is None else _like(t, empty)
             for t in (gate, scale, shift, weight, post_weight)]
    if workspace is None and any(t is not None for t in small):
        workspace = scratch(_bytes("nabla_block_norm_bwd_workspace_bytes", *shape) or 1,
                            dtype=torch.uint8, device=dev)
    if workspace is not None:
        _on(workspace, "workspace", dev)
    _cuda(like)
    _run(dev, stream, load().nabla_block_norm_bwd, "nabla_block_norm_bwd", _ptr(s), s_st, _ptr(u),
         u_st, _ptr(dsum), ds_st, _ptr(dy), dy_st, *head, *rest, dx.data_ptr(), dx_st, _ptr(du),
         du_st, *map(_ptr, small), _ptr(workspace),
         0 if workspace is None else workspace.numel() * workspace.element_size())
    return (dx, du, *small)


def _stream_device(stream) -> torch.device:
    dev = getattr(stream, "device", None)
    return torch.device(dev) if dev is not None else torch.device(
        "cuda", torch.cuda.current_device())


def nabla_selftest_bounded_wait(stream=None) -> None:
    """Enqueue the bounded-wait probe (it must end as a recorded timeout)."""
    dev = _stream_device(stream)
    st = _call(dev, load().nabla_selftest_bounded_wait, _stream(stream, dev))
    _check(st, "nabla_selftest_bounded_wait")


def nabla_get_last_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status code."""
    dev = _stream_device(stream)
    return _call(dev, load().nabla_get_last_device_status, _stream(stream, dev))


def from_storage(a: np.ndarray, device) -> torch.Tensor:
    """numpy storage array (float32, or uint16 bf16 bit patterns) -> device tensor."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(a).to(device)
