"""Thin ctypes binding over libvattn.so: argument marshalling only.

Every function mirrors the C entry point of the same name in include/vattn.h.
Tensor arguments may be contiguous torch tensors (their data_ptr() is
passed; CUDA tensors for device pointers, host tensors for the host-buffer
entry point's q, k, v, o, lse) or raw integer addresses; `stream` defaults to
torch's current CUDA stream.
Every non-OK status raises VattnError.  There is no fallback: if the shared
library is missing the import of this module fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
# VATTN_DEBUG_BUILD=1 loads the debug build (device-side bounds checks; see
# build.py) instead of the default library.
LIB_PATH = os.path.join(_HERE, "libvattn_debug.so" if os.environ.get("VATTN_DEBUG_BUILD") == "1" else "libvattn.so")

VATTN_OK = 0
VATTN_ERR_INVALID_ARG = -1
VATTN_ERR_SHAPE = -2
VATTN_ERR_UNSUPPORTED = -3
VATTN_ERR_ALIGN = -4
VATTN_ERR_CUDA = -5
VATTN_ERR_DEVICE_TIMEOUT = -6
VATTN_ERR_WORKSPACE = -7
VATTN_ERR_DEVICE_BOUNDS = -8

VATTN_OP_DUAL_FWD = 1
VATTN_OP_STA_BWD = 2
VATTN_OP_DUAL_BWD = 3
VATTN_OP_DUAL_SYM_FWD = 4
VATTN_OP_DUAL_SYM_BWD = 5
VATTN_OP_STA_FWD_HOST = 6
VATTN_OP_HIER_FWD = 7
VATTN_OP_HIER_BWD = 8
VATTN_OP_STA_FWD_FP8 = 9
VATTN_OP_DUAL_FWD_FP8 = 10
VATTN_OP_DUAL_SYM_LEARNED_FWD = 11
VATTN_PLAN_OK = 0
VATTN_PLAN_NO_PAGES = 1
VATTN_PLAN_TABLE_FULL = 2
VATTN_PLAN_NO_SLOTS = 3
VATTN_PLAN_BAD_STATE = 4
VATTN_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024

VATTN_DEBUG_SKIP_ARRIVAL = 1


class VattnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"vattn error {code}: {msg}")
        self.code = code


class Geom(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("head_dim", ctypes.c_int64),
        ("T", ctypes.c_int32),
        ("H", ctypes.c_int32),
        ("W", ctypes.c_int32),
        ("tile", ctypes.c_int32 * 3),
        ("window", ctypes.c_int32 * 3),
        ("pool", ctypes.c_int32 * 3),
    ]


def make_geom(batch: int, heads: int, head_dim: int, grid: Sequence[int], tile: Sequence[int],
              window: Sequence[int], pool: Sequence[int] = (1, 1, 1)) -> Geom:
    g = Geom()
    g.batch, g.heads, g.head_dim = batch, heads, head_dim
    g.T, g.H, g.W = grid
    g.tile[:] = list(tile)
    g.window[:] = list(window)
    g.pool[:] = list(pool)
    return g


class CacheGeom(ctypes.Structure):
    _fields_ = [
        ("streams", ctypes.c_int64),
        ("q_heads", ctypes.c_int64),
        ("kv_heads", ctypes.c_int64),
        ("head_dim", ctypes.c_int64),
        ("pages", ctypes.c_int64),
        ("page_tokens", ctypes.c_int32),
        ("table_width", ctypes.c_int32),
        ("frame_tokens", ctypes.c_int32),
        ("window_frames", ctypes.c_int32),
    ]


def make_cache_geom(streams: int, q_heads: int, kv_heads: int, head_dim: int, pages: int, page_tokens: int,
                    table_width: int, frame_tokens: int = 0, window_frames: int = 0) -> CacheGeom:
    return CacheGeom(streams, q_heads, kv_heads, head_dim, pages, page_tokens, table_width, frame_tokens,
                     window_frames)


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_INT = ctypes.c_int
_GP = ctypes.POINTER(Geom)
_CP = ctypes.POINTER(CacheGeom)

_SIGS = {
    "vattn_tile_permute": [_GP, _P, _P, _I64, _P],
    "vattn_tile_unpermute": [_GP, _P, _P, _I64, _P],
    "vattn_kept_tiles": [_GP, _P, _P],
    "vattn_sta_fwd": [_GP, _P, _P, _P, _F, _P, _P, _P],
    "vattn_pool_kv": [_GP, _P, _P, _P, _P, _P],
    "vattn_global_fwd": [_GP, _P, _P, _P, _F, _P, _P, _P],
    "vattn_dual_fwd": [_GP, _P, _P, _P, _P, _F, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "vattn_sta_bwd": [_GP, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P],
    "vattn_dual_bwd": [_GP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _P, _SZ, _P],
    "vattn_dual_fwd_noalloc": [_GP, _P, _P, _P, _P, _F, _P, _P],
    "vattn_xwin_fwd": [_GP, _INT, _P, _P, _P, _F, _P, _P, _P],
    "vattn_hier_fwd": [_GP, _P, _P, _P, _F, _P, _P, _P, _SZ, _P],
    "vattn_hier_bwd": [_GP, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P],
    "vattn_sta_fwd_raster": [_GP, _P, _P, _P, _F, _P, _P, _P],
    "vattn_dual_fwd_fp8": [_GP, _P, _P, _P, _P, _F, _P, _P, _SZ, _P],
    "vattn_sta_fwd_fp8": [_GP, _P, _P, _P, _F, _P, _P, _P, _SZ, _P],
    "vattn_sta_fwd_host": [_GP, _P, _P, _P, _F, _P, _P, _I64, _P, _SZ, _P],
    "vattn_dual_sym_fwd": [_GP, _P, _P, _P, _P, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "vattn_dual_sym_learned_fwd": [_GP, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _SZ, _P],
    "vattn_dual_sym_bwd": [_GP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P],
    "vattn_xwin_bwd": [_GP, _INT, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P],
    "vattn_workspace_size": [_INT, _GP, ctypes.POINTER(_SZ)],
    "vattn_get_status": [_P],
    "vattn_last_error": [],
    "vattn_shutdown": [],
    "vattn_debug_set": [_INT, _I64],
    "vattn_debug_exp2": [_P, _P, _I64, _P],
    "vattn_debug_query_blocks": [_GP, _INT, _P, _I64, _P],
    "vattn_version": [],
}

# The 8-bit key/value cache (its geometry is a vattn_cache_geom).
_CACHE_SIGS = {
    "vattn_cache_plan": [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _P],
    "vattn_cache_append": [_CP, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P],
    "vattn_cache_fwd": [_CP, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _F, _I64, _I64, _P, _P, _P, _SZ, _P],
    "vattn_cache_workspace_size": [_CP, _I64, _I64, ctypes.POINTER(_SZ)],
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python video_dit_local_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, args in (*_SIGS.items(), *_CACHE_SIGS.items()):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name in ("vattn_last_error", "vattn_version") else ctypes.c_int
    return lib


lib = _load()


def _ptr(x) -> Optional[int]:
    """Device pointer argument: None, a raw address, or a contiguous CUDA tensor."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("a device pointer argument got a host tensor: pass a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (the library reads them as dense arrays)")
    return x.data_ptr()


def _hptr(x) -> Optional[int]:
    """Host pointer argument (vattn_sta_fwd_host's q, k, v, o, lse): None, a raw
    address, or a contiguous host tensor."""
    if x is None or isinstance(x, int):
        return x
    if x.is_cuda:
        raise ValueError("a host pointer argument got a CUDA tensor: pass host (ideally pinned) memory")
    if not x.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (the library reads them as dense arrays)")
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    if torch.cuda.is_available():
        return torch.cuda.current_stream().cuda_stream
    return None


def _check(code: int) -> None:
    if code != VATTN_OK:
        raise VattnError(code, lib.vattn_last_error().decode())


def _row_bytes(t) -> int:
    return t.shape[-1] * t.element_size() if t.dim() == 4 else t.element_size()


def vattn_tile_permute(geom: Geom, src, dst, row_bytes: Optional[int] = None, stream=None) -> None:
    rb = _row_bytes(src) if row_bytes is None else row_bytes
    _check(lib.vattn_tile_permute(ctypes.byref(geom), _ptr(src), _ptr(dst), rb, _stream(stream)))


def vattn_tile_unpermute(geom: Geom, src, dst, row_bytes: Optional[int] = None, stream=None) -> None:
    rb = _row_bytes(src) if row_bytes is None else row_bytes
    _check(lib.vattn_tile_unpermute(ctypes.byref(geom), _ptr(src), _ptr(dst), rb, _stream(stream)))


def vattn_kept_tiles(geom: Geom, out, stream=None) -> None:
    _check(lib.vattn_kept_tiles(ctypes.byref(geom), _ptr(out), _stream(stream)))


def vattn_sta_fwd(geom: Geom, q, k, v, scale: float, o, lse=None, stream=None) -> None:
    _check(lib.vattn_sta_fwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), scale, _ptr(o), _ptr(lse),
                             _stream(stream)))


def vattn_xwin_fwd(geom: Geom, shifted: int, q, k, v, scale: float, o, lse=None, stream=None) -> None:
    _check(lib.vattn_xwin_fwd(ctypes.byref(geom), int(shifted), _ptr(q), _ptr(k), _ptr(v), scale, _ptr(o), _ptr(lse),
                              _stream(stream)))


def vattn_xwin_bwd(geom: Geom, shifted: int, q, k, v, o, lse, dout, scale: float, dq, dk, dv, workspace,
                   ws_bytes: int = 0, stream=None) -> None:
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_xwin_bwd(ctypes.byref(geom), int(shifted), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                              _ptr(dout), scale, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes,
                              _stream(stream)))


def vattn_dual_sym_fwd(geom: Geom, q, k, v, g, scale: float, o, o_l=None, lse_l=None, qp=None, kp=None, vp=None,
                       o_p=None, lse_p=None, workspace=None, ws_bytes: int = 0, stream=None) -> None:
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_dual_sym_fwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(g), scale, _ptr(o), _ptr(o_l),
                                  _ptr(lse_l), _ptr(qp), _ptr(kp), _ptr(vp), _ptr(o_p), _ptr(lse_p), _ptr(workspace),
                                  ws_bytes, _stream(stream)))


def vattn_dual_sym_learned_fwd(geom: Geom, q, k, v, g, wq, wk, wv, w3, scale: float, o, workspace,
                               ws_bytes: int = 0, stream=None) -> None:
    """Learned compressed global branch (inference): weights fp32, taps-major
    ([heads, p_t*p_h*p_w, d] for wq/wk/wv, [heads, 27, d] for w3)."""
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_dual_sym_learned_fwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(wq), _ptr(wk),
                                          _ptr(wv), _ptr(w3), scale, _ptr(o), _ptr(workspace), ws_bytes,
                                          _stream(stream)))


def vattn_dual_sym_bwd(geom: Geom, q, k, v, g, o_l, lse_l, qp, kp, vp, o_p, lse_p, dout, scale: float, dq, dk, dv,
                       workspace, ws_bytes: int = 0, stream=None) -> None:
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_dual_sym_bwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o_l), _ptr(lse_l),
                                  _ptr(qp), _ptr(kp), _ptr(vp), _ptr(o_p), _ptr(lse_p), _ptr(dout), scale, _ptr(dq),
                                  _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_hier_fwd(geom: Geom, q, k, v, scale: float, o, lse=None, workspace=None, ws_bytes: int = 0,
                   stream=None) -> None:
    """Hierarchical local attention (geom.pool = the medium pool factor)."""
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_hier_fwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), scale, _ptr(o), _ptr(lse),
                              _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_hier_bwd(geom: Geom, q, k, v, o, lse, dout, scale: float, dq, dk, dv, workspace, ws_bytes: int = 0,
                   stream=None) -> None:
    """Backward of vattn_hier_fwd (geom.pool = the medium pool factor)."""
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_hier_bwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), scale,
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_sta_fwd_raster(geom: Geom, q, k, v, scale: float, o, lse=None, stream=None) -> None:
    """Sliding-tile forward on raster-order tensors (reorder fused into the kernel)."""
    _check(lib.vattn_sta_fwd_raster(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), scale, _ptr(o), _ptr(lse),
                                    _stream(stream)))


def vattn_dual_fwd_fp8(geom: Geom, q, k, v, g, scale: float, o, workspace, ws_bytes: int = 0, stream=None) -> None:
    """Dual forward with e4m3 Q*K^T in both branches (inference)."""
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_dual_fwd_fp8(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(g), scale, _ptr(o),
                                  _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_sta_fwd_fp8(geom: Geom, q, k, v, scale: float, o, lse=None, workspace=None, ws_bytes: int = 0,
                      stream=None) -> None:
    """Sliding-tile forward with e4m3 Q*K^T (per-head absmax scales), bf16 P*V."""
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_sta_fwd_fp8(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), scale, _ptr(o), _ptr(lse),
                                 _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_sta_fwd_host(geom: Geom, q, k, v, scale: float, o, lse, chunk_slices: int, workspace,
                       ws_bytes: int = 0, stream=None) -> None:
    """Host-buffer sliding-tile forward with copies overlapped by chunks of
    batch*head slices (q, k, v, o, lse: host tensors / addresses, raster)."""
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_sta_fwd_host(ctypes.byref(geom), _hptr(q), _hptr(k), _hptr(v), scale, _hptr(o), _hptr(lse),
                                  int(chunk_slices), _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_pool_kv(geom: Geom, k, v, kp, vp, stream=None) -> None:
    _check(lib.vattn_pool_kv(ctypes.byref(geom), _ptr(k), _ptr(v), _ptr(kp), _ptr(vp), _stream(stream)))


def vattn_global_fwd(geom: Geom, q, kp, vp, scale: float, o, lse=None, stream=None) -> None:
    _check(lib.vattn_global_fwd(ctypes.byref(geom), _ptr(q), _ptr(kp), _ptr(vp), scale, _ptr(o), _ptr(lse),
                                _stream(stream)))


def vattn_dual_fwd(geom: Geom, q, k, v, g, scale: float, o, o_l=None, lse_l=None, o_g=None, lse_g=None,
                   kp=None, vp=None, workspace=None, ws_bytes: int = 0, stream=None) -> None:
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_dual_fwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(g), scale, _ptr(o), _ptr(o_l),
                              _ptr(lse_l), _ptr(o_g), _ptr(lse_g), _ptr(kp), _ptr(vp), _ptr(workspace), ws_bytes,
                              _stream(stream)))


def vattn_dual_fwd_noalloc(geom: Geom, q, k, v, g, scale: float, o, stream=None) -> None:
    """vattn_dual_fwd for callers that cannot allocate: the workspace is the
    library's own static device scratch (VATTN_NOALLOC_SCRATCH_BYTES)."""
    _check(lib.vattn_dual_fwd_noalloc(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(g), scale, _ptr(o),
                                      _stream(stream)))


def vattn_sta_bwd(geom: Geom, q, k, v, o, lse, dout, scale: float, dq, dk, dv, workspace, ws_bytes: int = 0,
                  stream=None) -> None:
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_sta_bwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), scale,
                             _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_dual_bwd(geom: Geom, q, k, v, g, o_l, lse_l, o_g, lse_g, kp, vp, dout, scale: float, dq, dk, dv,
                   dg=None, workspace=None, ws_bytes: int = 0, stream=None) -> None:
    if workspace is not None and not ws_bytes:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.vattn_dual_bwd(ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o_l), _ptr(lse_l),
                              _ptr(o_g), _ptr(lse_g), _ptr(kp), _ptr(vp), _ptr(dout), scale, _ptr(dq), _ptr(dk),
                              _ptr(dv), _ptr(dg), _ptr(workspace), ws_bytes, _stream(stream)))


def vattn_workspace_size(op: int, geom: Geom) -> int:
    n = _SZ(0)
    _check(lib.vattn_workspace_size(op, ctypes.byref(geom), ctypes.byref(n)))
    return n.value


# The cache calls are short enough for their argument checks to matter, so each
# tensor is looked at once.
_torch = None
_I32 = _F32 = _BF16 = _BYTES = ()  # what an array's elements may be; known once a call has met a tensor


def _use_torch() -> None:
    global _torch, _I32, _F32, _BF16, _BYTES
    import torch
    _I32, _F32, _BF16 = (torch.int32,), (torch.float32,), (torch.bfloat16,)
    _BYTES = (torch.float8_e4m3fn, torch.uint8)
    _torch = torch


def _device(x) -> int:
    """The device of a call's first tensor; it must be the current one, on whose stream the kernels run."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError("a device pointer argument got a host tensor: pass a CUDA tensor")
    if _torch is None:
        _use_torch()
    cuda = _torch.cuda
    if cuda.is_initialized() and dev != cuda.current_device():
        raise ValueError(f"tensors on device {dev}: all must be on the current device")
    return dev


def _on(x, dev: int, what: str, kind, size: int) -> Optional[int]:
    """Address of a contiguous tensor on device `dev` of `size` bytes or more, its type one of `kind`; None and raw
    addresses pass."""
    try:
        if x.get_device() == dev and x.is_contiguous() and x.dtype in kind and x.nbytes >= size:
            return x.data_ptr()
    except AttributeError:  # no tensor
        pass
    if x is None or isinstance(x, int):
        return x
    if x.get_device() != dev:
        raise ValueError("a device pointer argument got a host tensor: pass a CUDA tensor" if x.get_device() < 0 else
                         f"tensors on devices {dev} and {x.get_device()}: all must be on the current device")
    if not x.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (the library reads them as dense arrays)")
    if hasattr(x, "dtype"):
        raise ValueError(f"{what}: {x.nbytes} bytes of {x.dtype}, but the call needs {size} of {kind[0]}")
    return x.data_ptr()


def _tokens(x, what: str, dev: int, heads: int, d: int):
    """(address, token stride, tokens) of a bf16 [tokens, heads, d] tensor whose tokens'
    rows are dense (a slice of a fused projection along dim 1 is)."""
    if x.get_device() != dev:
        raise ValueError(f"{what} is on another device than the call's other tensors")
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{what}: shape {tuple(shape)}, but the geometry says [tokens, {heads}, {d}]")
    if getattr(x, "dtype", _BF16[0]) not in _BF16:
        raise ValueError(f"{what}: {x.dtype}, but the call needs {_BF16[0]}")
    n = shape[0]
    token, head, channel = x.stride()
    if channel != 1 or (head != d and heads > 1):
        raise ValueError(f"{what}: heads and channels of a token must be contiguous")
    return x.data_ptr(), token if n > 1 else heads * d, n


def _current_stream(stream, dev: int) -> int:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _torch is None:
        _use_torch()
    return _torch._C._cuda_getCurrentRawStream(dev)


def vattn_cache_plan(geom: CacheGeom, new_tokens, kv_lens, block_table, free_pages, n_free, kv_lens_out, n_free_out,
                     q_starts, slots, result, max_tokens: Optional[int] = None, stream=None) -> None:
    """Pages and slots of one step's new tokens (int32 tensors; max_tokens defaults to the length of slots)."""
    dev = -1 if isinstance(new_tokens, int) else _device(new_tokens)
    if max_tokens is None:
        max_tokens = slots.numel()
    i32, lens = _I32, geom.streams * 4
    code = lib.vattn_cache_plan(geom, _on(new_tokens, dev, "new_tokens", i32, lens), _on(kv_lens, dev, "kv_lens", i32, lens),
                                _on(block_table, dev, "block_table", i32, lens * geom.table_width),
                                _on(free_pages, dev, "free_pages", i32, geom.pages * 4),
                                _on(n_free, dev, "n_free", i32, 4), _on(kv_lens_out, dev, "kv_lens_out", i32, lens),
                                _on(n_free_out, dev, "n_free_out", i32, 4), _on(q_starts, dev, "q_starts", i32, lens + 4),
                                _on(slots, dev, "slots", i32, max_tokens * 4), max_tokens,
                                _on(result, dev, "result", i32, 16), _current_stream(stream, dev))
    if code:
        _check(code)


def vattn_cache_append(geom: CacheGeom, k, v, slots, kcache, vcache, kscale, vscale, stream=None) -> None:
    """Quantise k, v [tokens, kv_heads, d] (bf16, may be slices of a fused projection) into their slots."""
    dev = _device(k)
    heads, d = geom.kv_heads, geom.head_dim
    kp, ks, n = _tokens(k, "k", dev, heads, d)
    vp, vs, nv = _tokens(v, "v", dev, heads, d)
    if nv != n or (not isinstance(slots, int) and slots.numel() < n):
        raise ValueError(f"{n} keys, {nv} values and {slots if isinstance(slots, int) else slots.numel()} slots")
    rows = geom.pages * heads * geom.page_tokens
    code = lib.vattn_cache_append(geom, kp, ks, vp, vs, _on(slots, dev, "slots", _I32, n * 4), n,
                                  _on(kcache, dev, "kcache", _BYTES, rows * d), _on(vcache, dev, "vcache", _BYTES, rows * d),
                                  _on(kscale, dev, "kscale", _F32, rows // 4), _on(vscale, dev, "vscale", _F32, rows // 4),
                                  _current_stream(stream, dev))
    if code:
        _check(code)


def vattn_cache_workspace_size(geom: CacheGeom, n_tokens: int, max_new: int) -> int:
    n = _SZ(0)
    _check(lib.vattn_cache_workspace_size(ctypes.byref(geom), n_tokens, max_new, ctypes.byref(n)))
    return n.value


def vattn_cache_fwd(geom: CacheGeom, q, q_starts, kv_lens, block_table, kcache, vcache, kscale, vscale, scale: float,
                    max_new: int, o, lse=None, workspace=None, ws_bytes: int = 0, stream=None) -> None:
    """Attention of q [tokens, q_heads, d] (bf16, may be a slice of a fused projection) over the cache."""
    dev = _device(q)
    if workspace is not None and not isinstance(workspace, int):
        size = workspace.numel() * workspace.element_size()
        if ws_bytes > size:
            raise ValueError(f"workspace: {size} bytes, but ws_bytes is {ws_bytes}")
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the call's device")
        workspace, ws_bytes = workspace.data_ptr(), ws_bytes or size
    heads, d, lens = geom.q_heads, geom.head_dim, geom.streams * 4
    qp, stride, n = _tokens(q, "q", dev, heads, d)
    rows = geom.pages * geom.kv_heads * geom.page_tokens
    code = lib.vattn_cache_fwd(geom, qp, stride, _on(q_starts, dev, "q_starts", _I32, lens + 4),
                               _on(kv_lens, dev, "kv_lens", _I32, lens),
                               _on(block_table, dev, "block_table", _I32, lens * geom.table_width),
                               _on(kcache, dev, "kcache", _BYTES, rows * d), _on(vcache, dev, "vcache", _BYTES, rows * d),
                               _on(kscale, dev, "kscale", _F32, rows // 4), _on(vscale, dev, "vscale", _F32, rows // 4),
                               scale, n, max_new, _on(o, dev, "o", _BF16, n * heads * d * 2),
                               _on(lse, dev, "lse", _F32, n * heads * 4), workspace, ws_bytes, _current_stream(stream, dev))
    if code:
        _check(code)


def vattn_get_status(stream=None) -> int:
    """Returns the status code (does not raise)."""
    return lib.vattn_get_status(_stream(stream))


def vattn_last_error() -> str:
    return lib.vattn_last_error().decode()


def vattn_shutdown() -> None:
    """Releases the host pipeline's library streams and events on every device."""
    _check(lib.vattn_shutdown())


def vattn_debug_set(flags: int, timeout_ns: int = 0) -> None:
    _check(lib.vattn_debug_set(flags, timeout_ns))


def vattn_debug_exp2(x, y, n: Optional[int] = None, stream=None) -> None:
    _check(lib.vattn_debug_exp2(_ptr(x), _ptr(y), x.numel() if n is None else n, _stream(stream)))


def vattn_debug_query_blocks(geom: Geom, window_mode: int):
    """Host-side query-block plan of the sliding-tile forward: an int32 tensor
    [n_blocks, 4] = (first tile-major row, rows that exist, straddle flag,
    tile of the key stream).  window_mode: 0 sliding, 1 partition, 2 shifted."""
    import torch
    n = ctypes.c_int64(0)
    _check(lib.vattn_debug_query_blocks(ctypes.byref(geom), window_mode, None, 0, ctypes.byref(n)))
    out = torch.empty((n.value, 4), dtype=torch.int32)
    _check(lib.vattn_debug_query_blocks(ctypes.byref(geom), window_mode, _hptr(out), n.value, ctypes.byref(n)))
    return out


def vattn_version() -> str:
    return lib.vattn_version().decode()
