"""Python binding of libfx (include/fx.h): argument marshalling only.

Every function here checks tensor dtypes/devices, allocates outputs and workspaces with PyTorch, and
calls the C entry point of the same name; all arithmetic runs in the library's CUDA kernels.  There is
no fallback: if libfx.so has not been built, or a CUDA tensor is missing, the call raises.

Build the library with ``python -m kv_cache_token_fx_gb300.build`` (or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
import threading

import torch

from . import build as _build

__all__ = [
    "FxError", "load_library", "library_path", "Workspace", "fx_focal_attn_scores", "fx_topk_select",
    "fx_focal_mass", "fx_choose_focal_layers", "fx_csfr_schedule", "FX_CSFR_FOCAL", "FX_CSFR_CURRENT",
    "FX_CSFR_PREVIOUS", "FX_CSFR_DENSE",
    "fx_sparse_gqa_decode", "fx_kv_compact", "fx_kv_append", "fx_kv_retain_per_layer", "fx_shared_prefix_decode",
    "fx_device_errors", "fx_focal_workspace_bytes", "fx_sparse_workspace_bytes", "fx_shared_prefix_workspace_bytes",
    "FX_DEVERR_LEN", "FX_DEVERR_INDEX", "FX_DEVERR_OFFSETS", "FX_DEVERR_CAPACITY", "FX_DEVERR_TIMEOUT",
    "FX_LAUNCH_PDL", "FX_LAUNCH_INPUTS_READY", "BranchPool",
    "PagedKV", "fx_paged_append", "fx_paged_gather", "fx_paged_decode", "fx_paged_importance",
    "fx_paged_decode_workspace_bytes", "FX_DEVERR_PAGE", "FX_PAGED_BF16", "FX_PAGED_E2M1",
]

FX_OK, FX_ERR_INVALID_ARG, FX_ERR_UNSUPPORTED, FX_ERR_WORKSPACE, FX_ERR_CUDA, FX_ERR_DEVICE = range(6)
FX_DEVERR_LEN, FX_DEVERR_INDEX, FX_DEVERR_OFFSETS, FX_DEVERR_CAPACITY, FX_DEVERR_TIMEOUT = 1, 2, 4, 8, 16
FX_DEVERR_PAGE = 32
FX_LAUNCH_PDL, FX_LAUNCH_INPUTS_READY = 1, 2
FX_PAGED_BF16, FX_PAGED_E2M1 = 0, 1
FX_CSFR_FOCAL, FX_CSFR_CURRENT, FX_CSFR_PREVIOUS, FX_CSFR_DENSE = range(4)
_STATUS = {0: "FX_OK", 1: "FX_ERR_INVALID_ARG", 2: "FX_ERR_UNSUPPORTED", 3: "FX_ERR_WORKSPACE",
           4: "FX_ERR_CUDA", 5: "FX_ERR_DEVICE"}

c_vp, c_i64, c_i32, c_int, c_float, c_size = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int,
                                              ctypes.c_float, ctypes.c_size_t)


class FxError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


class KVDesc(ctypes.Structure):
    _fields_ = [("k", c_vp), ("v", c_vp), ("len", c_vp), ("stride_b", c_i64), ("stride_h", c_i64),
                ("stride_t", c_i64), ("B", c_i32), ("Hkv", c_i32), ("Tcap", c_i32), ("d", c_i32)]


KVOutDesc = type("KVOutDesc", (ctypes.Structure,), {"_fields_": KVDesc._fields_})


class PrefixDesc(ctypes.Structure):
    _fields_ = [("k", c_vp), ("v", c_vp), ("stride_h", c_i64), ("stride_t", c_i64), ("P", c_i32),
                ("Hkv", c_i32), ("d", c_i32), ("len", c_vp)]


class BranchDesc(ctypes.Structure):
    _fields_ = [("suf_k", c_vp), ("suf_v", c_vp), ("suf_stride_h", c_i64), ("suf_stride_t", c_i64),
                ("suf_off", c_vp), ("suf_rows", c_i32), ("max_suffix", c_i32), ("draft_k", c_vp),
                ("draft_v", c_vp), ("draft_stride_b", c_i64), ("draft_stride_i", c_i64),
                ("draft_stride_h", c_i64), ("Br", c_i32), ("Mq", c_i32), ("suf_len", c_vp)]


class PagedDesc(ctypes.Structure):
    _fields_ = [("k", c_vp), ("v", c_vp), ("k_scale", c_vp), ("v_scale", c_vp), ("table", c_vp), ("len", c_vp),
                ("stride_page", c_i64), ("stride_h", c_i64), ("stride_t", c_i64), ("scale_stride_page", c_i64),
                ("scale_stride_h", c_i64), ("scale_stride_t", c_i64), ("table_stride", c_i64), ("format", c_i32),
                ("B", c_i32), ("Hkv", c_i32), ("d", c_i32), ("page_rows", c_i32), ("n_pages", c_i32),
                ("max_pages", c_i32), ("k_exp", c_i32), ("v_exp", c_i32)]


class PagedRows(ctypes.Structure):
    _fields_ = [("k", c_vp), ("v", c_vp), ("stride_n", c_i64), ("stride_h", c_i64), ("q", c_vp), ("q_out", c_vp),
                ("q_stride_n", c_i64), ("q_stride_h", c_i64), ("qo_stride_n", c_i64), ("qo_stride_h", c_i64),
                ("seq", c_vp), ("pos", c_vp), ("rope_pos", c_vp), ("cos_sin", c_vp), ("n", c_i32), ("Hq", c_i32),
                ("rot", c_i32), ("n_pos", c_i32), ("interleaved", c_i32)]


_lib = None
_lib_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load_library():
    """Load libfx.so (must have been built).  Raises FxError if it is missing."""
    global _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise FxError(FX_ERR_CUDA, f"{path} is not built; run `python -m kv_cache_token_fx_gb300.build`")
        lib = ctypes.CDLL(path)
        lib.fx_last_error.restype = ctypes.c_char_p
        lib.fx_abi_version.restype = c_int
        lib.fx_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint), c_vp]
        lib.fx_test_stall_wait.argtypes = [ctypes.c_uint]
        lib.fx_test_stall_wait.restype = None
        lib.fx_workspace_init.argtypes = [c_vp, c_size, c_vp]
        lib.fx_focal_workspace_bytes.argtypes = [c_int] * 5
        lib.fx_focal_workspace_bytes.restype = c_size
        c_uint = ctypes.c_uint
        lib.fx_focal_attn_scores.argtypes = [ctypes.POINTER(KVDesc), c_vp, c_int, c_int, c_int, c_float, c_int,
                                             c_int, c_vp, c_vp, c_vp, c_size, c_uint, c_vp]
        lib.fx_topk_select.argtypes = [c_vp, c_int, c_int, c_int, c_vp, c_vp, c_uint, c_vp]
        lib.fx_focal_mass.argtypes = [c_vp, c_int, c_int, c_int, c_int, c_vp, c_uint, c_vp]
        lib.fx_choose_focal_layers.argtypes = [ctypes.POINTER(ctypes.c_float), c_int, c_int,
                                               ctypes.POINTER(ctypes.c_int32)]
        lib.fx_csfr_schedule.argtypes = [c_int, ctypes.POINTER(ctypes.c_int32), c_int, c_int,
                                         ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
        lib.fx_sparse_workspace_bytes.argtypes = [c_int] * 6
        lib.fx_sparse_workspace_bytes.restype = c_size
        lib.fx_sparse_gqa_decode.argtypes = [ctypes.POINTER(KVDesc), c_vp, c_int, c_vp, c_int, c_int, c_float,
                                             c_vp, c_vp, c_size, c_uint, c_vp]
        lib.fx_kv_compact.argtypes = [ctypes.POINTER(KVDesc), c_i64, c_vp, c_i64, c_int, c_int,
                                      ctypes.POINTER(KVOutDesc), c_i64, c_int, c_uint, c_vp]
        lib.fx_kv_append.argtypes = [ctypes.POINTER(KVOutDesc), c_i64, c_int, c_vp, c_vp, c_vp, c_uint, c_vp]
        lib.fx_retain_workspace_bytes.argtypes = [c_int] * 6
        lib.fx_retain_workspace_bytes.restype = c_size
        lib.fx_kv_retain_per_layer.argtypes = [ctypes.POINTER(KVDesc), c_i64, c_int, c_vp, c_int, c_int, c_int,
                                               c_float, c_int, c_int, c_int, c_vp, ctypes.POINTER(KVOutDesc), c_i64,
                                               c_vp, c_size, ctypes.c_uint, c_vp]
        lib.fx_branch_pool_create.argtypes = [c_int, c_int, c_int]
        lib.fx_branch_pool_create.restype = c_vp
        lib.fx_branch_pool_destroy.argtypes = [c_vp]
        lib.fx_branch_pool_destroy.restype = None
        for name, args in (("extend_prefix", [c_vp, c_int]), ("fork", [c_vp]), ("append", [c_vp, c_int, c_int]),
                           ("release", [c_vp, c_int]), ("release_parent", [c_vp]), ("prefix_refs", [c_vp]),
                           ("prefix_len", [c_vp]), ("batch", [c_vp] + [ctypes.POINTER(ctypes.c_int32)] * 4)):
            f = getattr(lib, "fx_branch_pool_" + name)
            f.argtypes = args
            f.restype = c_int
        lib.fx_shared_prefix_workspace_bytes.argtypes = [c_int] * 6
        lib.fx_shared_prefix_workspace_bytes.restype = c_size
        lib.fx_shared_prefix_decode.argtypes = [ctypes.POINTER(PrefixDesc), ctypes.POINTER(BranchDesc), c_vp, c_int,
                                                c_vp, c_int, c_float, c_vp, c_vp, c_size, c_uint, c_vp]
        paged = c_vp   # the address of a PagedDesc
        lib.fx_paged_append.argtypes = [paged, ctypes.c_char_p, c_uint, c_vp]   # the bytes of a PagedRows
        lib.fx_paged_gather.argtypes = [paged, c_vp, c_vp, c_int, c_vp, c_vp, c_uint, c_vp]
        lib.fx_paged_decode_workspace_bytes.argtypes = [c_int] * 4
        lib.fx_paged_decode_workspace_bytes.restype = c_size
        lib.fx_paged_decode.argtypes = [paged, c_vp, c_i64, c_i64, c_i64, c_int, c_int, c_vp, c_int, c_vp, c_float,
                                        c_vp, c_vp, c_vp, c_size, c_uint, c_vp]
        lib.fx_paged_importance.argtypes = [paged, c_vp, c_i64, c_i64, c_i64, c_int, c_int, c_vp, c_float, c_int,
                                            c_int, c_vp, c_uint, c_vp]
        for name in ("fx_paged_append", "fx_paged_gather", "fx_paged_decode", "fx_paged_importance"):
            getattr(lib, name).restype = c_int
        for name in ("fx_device_errors", "fx_workspace_init", "fx_focal_attn_scores", "fx_topk_select",
                     "fx_focal_mass", "fx_choose_focal_layers", "fx_csfr_schedule",
                     "fx_sparse_gqa_decode", "fx_kv_compact", "fx_kv_append", "fx_kv_retain_per_layer",
                     "fx_shared_prefix_decode"):
            getattr(lib, name).restype = c_int
        _lib = lib
        return lib


def _check(status: int):
    if status != FX_OK:
        msg = load_library().fx_last_error().decode(errors="replace")
        raise FxError(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need_cuda(t, name, dtype):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise FxError(FX_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise FxError(FX_ERR_INVALID_ARG, f"{name} must be {dtype}, got {t.dtype}")


def _kv_desc(k, v, length):
    _need_cuda(k, "k", torch.bfloat16)
    _need_cuda(v, "v", torch.bfloat16)
    _need_cuda(length, "len", torch.int32)
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
        raise FxError(FX_ERR_INVALID_ARG, "k and v must be [B, Hkv, Tcap, d] views with equal strides, unit last stride")
    B, Hkv, Tcap, d = k.shape
    return KVDesc(k.data_ptr(), v.data_ptr(), length.data_ptr(), k.stride(0), k.stride(1), k.stride(2), B, Hkv,
                  Tcap, d)


def _default_scale(d):
    return 1.0 / math.sqrt(d)


# The handle of the per-thread default stream (cudaStreamPerThread): one number for another stream in every thread, so
# that neither a workspace nor allocated memory can be told by it.
_PER_THREAD = 2
_PER_THREAD_TEXT = "the per-thread default stream needs the caller's own outputs and workspace"


def _per_thread(stream):
    return stream is not None and (stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)) == _PER_THREAD


def _on_stream(device, stream):
    """Context in which memory is allocated for the stream that uses it."""
    if stream is None:
        return contextlib.nullcontext()
    if _per_thread(stream):
        raise FxError(FX_ERR_INVALID_ARG, _PER_THREAD_TEXT)
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        # (0 and 1 are the default stream; a stream object made of 0 would be some other one)
        stream = torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class Workspace:
    """A zero-initialised device scratch buffer reused across calls on one stream.

    ``ensure(nbytes)`` grows it (allocating a fresh zeroed buffer) when needed; a buffer that a CUDA
    graph has captured must not be grown afterwards, so size it before capture.  The buffer that it
    gives up stays reserved until the stream's work of that moment is done, and the fresh one is
    allocated for the stream.
    """

    def __init__(self, device=None, nbytes: int = 0):
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.buf = None
        if nbytes:
            self.ensure(nbytes)

    def ensure(self, nbytes: int, stream=None):
        if self.buf is None or self.buf.numel() < nbytes:
            # (a per-thread default stream: as the current stream's, which is all that is known of it)
            with contextlib.nullcontext() if _per_thread(stream) else _on_stream(self.device, stream):
                buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=self.device)
                if self.buf is not None:
                    self.buf.record_stream(torch.cuda.current_stream(self.device))
            _check(load_library().fx_workspace_init(_ptr(buf), buf.numel(), _stream(stream)))
            self.buf = buf   # (zeroed in the stream's order before another thread finds it)
        return self.buf


_default_ws = {}


def _workspace(ws, nbytes, device, stream):
    if ws is None:
        key = device.index if device.index is not None else torch.cuda.current_device()
        ws = _default_ws.get(key)
        if ws is None:
            ws = _default_ws[key] = Workspace(torch.device("cuda", key))
    buf = ws.ensure(nbytes, stream)
    return buf


def fx_focal_workspace_bytes(B, Hkv, Hq, Mq, Tcap) -> int:
    return int(load_library().fx_focal_workspace_bytes(B, Hkv, Hq, Mq, Tcap))


def fx_sparse_workspace_bytes(B, Hkv, Hq, k, tail_lo, Tcap) -> int:
    return int(load_library().fx_sparse_workspace_bytes(B, Hkv, Hq, k, tail_lo, Tcap))


def fx_shared_prefix_workspace_bytes(Br, Hkv, Hq, Mq, np_, max_suffix) -> int:
    return int(load_library().fx_shared_prefix_workspace_bytes(Br, Hkv, Hq, Mq, np_, max_suffix))


def fx_focal_attn_scores(k, v, length, q, *, q_pos0: int = -1, scale=None, cand=None, want_out=True,
                         want_scores=True, out=None, scores=None, ws=None, stream=None, flags: int = 0):
    """Focal layer: full attention + per-token importance.  Returns (out, scores) (None if not wanted).

    k, v [B, Hkv, Tcap, 128] bf16; length int32 [B]; q [B, Hq, Mq, 128] bf16 (contiguous).
    cand = (lo, hi) candidate range for the scores (default: the whole capacity).
    """
    lib = load_library()
    desc = _kv_desc(k, v, length)
    _need_cuda(q, "q", torch.bfloat16)
    if not q.is_contiguous() or q.dim() != 4:
        raise FxError(FX_ERR_INVALID_ARG, "q must be a contiguous [B, Hq, Mq, 128] tensor")
    B, Hkv, Tcap, d = k.shape
    _, Hq, Mq, _ = q.shape
    lo, hi = cand if cand is not None else (0, Tcap)
    if want_out and out is None:
        out = torch.empty((B, Hq, Mq, d), dtype=torch.float32, device=k.device)
    if want_scores and scores is None:
        scores = torch.empty((B, Hkv, hi - lo), dtype=torch.float32, device=k.device)
    if not want_out:
        out = None
    if not want_scores:
        scores = None
    nbytes = lib.fx_focal_workspace_bytes(B, Hkv, Hq, Mq, Tcap)
    buf = _workspace(ws, nbytes, k.device, stream)
    sc = _default_scale(d) if scale is None else float(scale)
    _check(lib.fx_focal_attn_scores(ctypes.byref(desc), _ptr(q), Hq, Mq, int(q_pos0), sc, int(lo), int(hi),
                                    _ptr(out), _ptr(scores), _ptr(buf), buf.numel(), int(flags), _stream(stream)))
    return out, scores


def fx_focal_mass(scores, R: int, *, mass=None, accumulate=False, stream=None, flags: int = 0):
    """Image-attention share per row: mass[r] (+)= sum_j scores[r, j] / R.  scores [..., n] fp32
    (contiguous, from fx_focal_attn_scores over the image tokens); returns mass [...] fp32."""
    lib = load_library()
    _need_cuda(scores, "scores", torch.float32)
    if not scores.is_contiguous():
        raise FxError(FX_ERR_INVALID_ARG, "scores must be contiguous")
    n = scores.shape[-1]
    rows = scores.numel() // n if n else 0
    if mass is None:
        if accumulate:
            raise FxError(FX_ERR_INVALID_ARG, "accumulate needs a mass tensor")
        mass = torch.empty(scores.shape[:-1], dtype=torch.float32, device=scores.device)
    _need_cuda(mass, "mass", torch.float32)
    if mass.numel() != rows or not mass.is_contiguous():
        raise FxError(FX_ERR_INVALID_ARG, "mass must be a contiguous tensor of one value per row")
    _check(lib.fx_focal_mass(_ptr(scores), rows, n, int(R), int(bool(accumulate)), _ptr(mass), int(flags),
                             _stream(stream)))
    return mass


def fx_choose_focal_layers(ratio, C: int):
    """The C layers with the largest image-attention ratio (ties: the lower layer), ascending."""
    lib = load_library()
    r = (ctypes.c_float * len(ratio))(*[float(x) for x in ratio])
    out = (ctypes.c_int32 * int(C))()
    _check(lib.fx_choose_focal_layers(r, len(ratio), int(C), out))
    return [int(x) for x in out]


def fx_topk_select(scores, k: int, *, prev=None, out=None, stream=None, flags: int = 0):
    """Top-k of each row of ``scores`` [..., n] (fp32, contiguous): int32 [..., k], ascending indices."""
    lib = load_library()
    _need_cuda(scores, "scores", torch.float32)
    if not scores.is_contiguous():
        raise FxError(FX_ERR_INVALID_ARG, "scores must be contiguous")
    n = scores.shape[-1]
    rows = scores.numel() // n if n else 0
    if out is None:
        out = torch.empty(scores.shape[:-1] + (k,), dtype=torch.int32, device=scores.device)
    if prev is not None:
        _need_cuda(prev, "prev", torch.int32)
        if prev.numel() != rows * k or not prev.is_contiguous():
            raise FxError(FX_ERR_INVALID_ARG, "prev must be a contiguous [rows, k] int32 tensor")
    _check(lib.fx_topk_select(_ptr(scores), rows, n, int(k), _ptr(prev), _ptr(out), int(flags), _stream(stream)))
    return out


def fx_csfr_schedule(n_layers: int, focal_layers, first_step: bool):
    """Per layer of one decode step: (kind, src) -- FX_CSFR_FOCAL (src = the layer), FX_CSFR_CURRENT /
    FX_CSFR_PREVIOUS (attend over this / the previous step's set of focal layer src) or FX_CSFR_DENSE
    (src = -1).  Host only."""
    lib = load_library()
    f = [int(x) for x in focal_layers]
    kind = (ctypes.c_int32 * n_layers)()
    src = (ctypes.c_int32 * n_layers)()
    _check(lib.fx_csfr_schedule(int(n_layers), (ctypes.c_int32 * len(f))(*f), len(f), 1 if first_step else 0,
                                kind, src))
    return list(kind), list(src)


def fx_sparse_gqa_decode(k, v, length, q, idx, tail_lo: int, *, scale=None, out=None, ws=None, stream=None,
                         flags: int = 0):
    """Decode attention of q [B, Hq, 1, 128] over idx [B, Hkv, kk] (or None) plus the tail [tail_lo, len)."""
    lib = load_library()
    desc = _kv_desc(k, v, length)
    _need_cuda(q, "q", torch.bfloat16)
    if not q.is_contiguous() or q.dim() != 4 or q.shape[2] != 1:
        raise FxError(FX_ERR_INVALID_ARG, "q must be a contiguous [B, Hq, 1, 128] tensor")
    B, Hkv, Tcap, d = k.shape
    Hq = q.shape[1]
    kk = 0
    if idx is not None:
        _need_cuda(idx, "idx", torch.int32)
        if not idx.is_contiguous() or idx.dim() != 3 or tuple(idx.shape[:2]) != (B, Hkv):
            raise FxError(FX_ERR_INVALID_ARG, "idx must be a contiguous [B, Hkv, k] int32 tensor")
        kk = idx.shape[2]
    if out is None:
        out = torch.empty((B, Hq, 1, d), dtype=torch.float32, device=k.device)
    nbytes = lib.fx_sparse_workspace_bytes(B, Hkv, Hq, kk, int(tail_lo), Tcap)
    buf = _workspace(ws, nbytes, k.device, stream)
    sc = _default_scale(d) if scale is None else float(scale)
    _check(lib.fx_sparse_gqa_decode(ctypes.byref(desc), _ptr(q), Hq, _ptr(idx) if kk else None, kk, int(tail_lo),
                                    sc, _ptr(out), _ptr(buf), buf.numel(), int(flags), _stream(stream)))
    return out


def fx_kv_compact(k, v, length, idx, tail_lo: int, dst_k, dst_v, dst_len, *, stream=None, flags: int = 0):
    """Compact the retained rows of one layer ([B, Hkv, T, 128]) or of L layers ([L, B, Hkv, T, 128]).

    idx: [B, Hkv, k] (one set for every layer) or, for L layers, [L, B, Hkv, k] (a set per layer)."""
    lib = load_library()
    if k.dim() == 5:
        n_layers = k.shape[0]
        if dst_k.dim() != 5 or dst_k.shape[0] != n_layers:
            raise FxError(FX_ERR_INVALID_ARG, "dst must have the same number of layers")
        s_layer, d_layer = k.stride(0), dst_k.stride(0)
        if v.stride(0) != s_layer or dst_v.stride(0) != d_layer:
            raise FxError(FX_ERR_INVALID_ARG, "k/v layer strides must match")
        src = _kv_desc(k[0], v[0], length)
        dst = _kv_desc(dst_k[0], dst_v[0], dst_len)
    else:
        n_layers, s_layer, d_layer = 1, 0, 0
        src = _kv_desc(k, v, length)
        dst = _kv_desc(dst_k, dst_v, dst_len)
    kk, i_layer = 0, 0
    if idx is not None:
        _need_cuda(idx, "idx", torch.int32)
        if not idx.is_contiguous():
            raise FxError(FX_ERR_INVALID_ARG, "idx must be contiguous [B, Hkv, k] or [L, B, Hkv, k]")
        kk = idx.shape[-1]
        if idx.dim() == 4:
            if k.dim() != 5 or idx.shape[0] != n_layers:
                raise FxError(FX_ERR_INVALID_ARG, "a per-layer idx [L, B, Hkv, k] needs L-layer caches")
            i_layer = idx.stride(0)
    dst_out = KVOutDesc(*[getattr(dst, f) for f, _ in KVDesc._fields_])
    _check(lib.fx_kv_compact(ctypes.byref(src), s_layer, _ptr(idx) if kk else None, i_layer, kk, int(tail_lo),
                             ctypes.byref(dst_out), d_layer, n_layers, int(flags), _stream(stream)))
    return dst_k, dst_v, dst_len


def fx_kv_append(k, v, k_new, v_new, pos, *, stream=None, flags: int = 0):
    """Write one new key/value row per (layer, sequence, KV head) into the caches: row pos[b] of
    k, v ([B, Hkv, T, 128], or [L, B, Hkv, T, 128] for L layers) takes k_new, v_new ([B, Hkv, 128] or
    [L, B, Hkv, 128], contiguous).  pos: int32 [B] on the device."""
    lib = load_library()
    if k.dim() == 5:
        n_layers, s_layer = k.shape[0], k.stride(0)
        if v.stride(0) != s_layer:
            raise FxError(FX_ERR_INVALID_ARG, "k/v layer strides must match")
        cache = _kv_desc(k[0], v[0], pos)
    else:
        n_layers, s_layer = 1, 0
        cache = _kv_desc(k, v, pos)
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        _need_cuda(t, name, torch.bfloat16)
        if not t.is_contiguous() or t.numel() != n_layers * cache.B * cache.Hkv * cache.d:
            raise FxError(FX_ERR_INVALID_ARG, f"{name} must be a contiguous [L, B, Hkv, 128] tensor")
    out = KVOutDesc(*[getattr(cache, f) for f, _ in KVDesc._fields_])
    _check(lib.fx_kv_append(ctypes.byref(out), s_layer, n_layers, _ptr(k_new), _ptr(v_new), _ptr(pos), int(flags),
                            _stream(stream)))
    return k, v


def fx_kv_retain_per_layer(k, v, length, q, keep_k: int, cand_hi: int, tail_lo: int, dst_k, dst_v, dst_len, *,
                           q_pos0: int = -1, scale=None, idx_out=None, ws=None, stream=None, flags: int = 0):
    """FastKV retention with a selection per layer: window scores of every layer, its top keep_k, and
    the compaction of every layer with its own set plus the tail [tail_lo, len).

    k, v [L, B, Hkv, T, 128]; q [L, B, Hq, Mq, 128] (each layer's window queries); dst_k, dst_v
    [L, B, Hkv, cap, 128]; dst_len int32 [B].  Returns idx [L, B, Hkv, keep_k] (ascending rows)."""
    lib = load_library()
    if k.dim() != 5 or dst_k.dim() != 5 or q.dim() != 5 or not (k.shape[0] == dst_k.shape[0] == q.shape[0]):
        raise FxError(FX_ERR_INVALID_ARG, "k, v, dst and q need a leading layer dimension of the same size")
    L, B, Hkv, T, d = k.shape
    _need_cuda(q, "q", torch.bfloat16)
    if not q.is_contiguous():
        raise FxError(FX_ERR_INVALID_ARG, "q must be a contiguous [L, B, Hq, Mq, 128] tensor")
    s_layer, d_layer = k.stride(0), dst_k.stride(0)
    if v.stride(0) != s_layer or dst_v.stride(0) != d_layer:
        raise FxError(FX_ERR_INVALID_ARG, "k/v layer strides must match")
    src = _kv_desc(k[0], v[0], length)
    dst = _kv_desc(dst_k[0], dst_v[0], dst_len)
    dst_out = KVOutDesc(*[getattr(dst, f) for f, _ in KVDesc._fields_])
    _, _, Hq, Mq, _ = q.shape
    if idx_out is None:
        idx_out = torch.empty((L, B, Hkv, int(keep_k)), dtype=torch.int32, device=k.device)
    _need_cuda(idx_out, "idx_out", torch.int32)
    if idx_out.numel() != L * B * Hkv * int(keep_k) or not idx_out.is_contiguous():
        raise FxError(FX_ERR_INVALID_ARG, "idx_out must be a contiguous [L, B, Hkv, keep_k] int32 tensor")
    nbytes = lib.fx_retain_workspace_bytes(B, Hkv, Hq, Mq, T, int(cand_hi))
    buf = _workspace(ws, nbytes, k.device, stream)
    sc = _default_scale(d) if scale is None else float(scale)
    _check(lib.fx_kv_retain_per_layer(ctypes.byref(src), s_layer, L, _ptr(q), Hq, Mq, int(q_pos0), sc, int(cand_hi),
                                      int(keep_k), int(tail_lo), _ptr(idx_out), ctypes.byref(dst_out), d_layer,
                                      _ptr(buf), buf.numel(), int(flags), _stream(stream)))
    return idx_out


def fx_shared_prefix_decode(pk, pv, sk, sv, off, dk, dv, q, *, max_suffix: int, prefix_idx=None, scale=None,
                            prefix_len=None, suf_len=None, out=None, ws=None, stream=None, flags: int = 0):
    """Draft verification of Br branches over one shared prefix.

    pk, pv [Hkv, P, 128]; sk, sv [Hkv, S, 128]; dk, dv [Br, Mq, Hkv, 128]; q [Br, Hq, Mq, 128];
    prefix_idx [Br, Hkv, kp] or None.  Branch b owns suffix rows off[b]..off[b+1]-1 (off int32 [Br+1]),
    or off[b]..off[b]+suf_len[b]-1 when suf_len [Br] is given; it sees the first prefix_len[b] prefix
    rows (its fork position; all P when prefix_len is None).
    """
    lib = load_library()
    for t, n in ((pk, "pk"), (pv, "pv"), (sk, "sk"), (sv, "sv"), (dk, "dk"), (dv, "dv"), (q, "q")):
        _need_cuda(t, n, torch.bfloat16)
    _need_cuda(off, "off", torch.int32)
    if pk.stride() != pv.stride() or sk.stride() != sv.stride() or dk.stride() != dv.stride():
        raise FxError(FX_ERR_INVALID_ARG, "paired K/V tensors must share strides")
    if not q.is_contiguous():
        raise FxError(FX_ERR_INVALID_ARG, "q must be contiguous")
    Hkv, P, d = pk.shape
    Br, Hq, Mq, _ = q.shape
    for t, n in ((prefix_len, "prefix_len"), (suf_len, "suf_len")):
        if t is not None:
            _need_cuda(t, n, torch.int32)
            if t.numel() != Br or not t.is_contiguous():
                raise FxError(FX_ERR_INVALID_ARG, f"{n} must be a contiguous [Br] int32 tensor")
    if off.numel() != (Br if suf_len is not None else Br + 1):
        raise FxError(FX_ERR_INVALID_ARG, "off must hold Br + 1 offsets (or Br starts with suf_len)")
    pre = PrefixDesc(pk.data_ptr(), pv.data_ptr(), pk.stride(0), pk.stride(1), P, Hkv, d,
                     prefix_len.data_ptr() if prefix_len is not None else None)
    brd = BranchDesc(sk.data_ptr(), sv.data_ptr(), sk.stride(0), sk.stride(1), off.data_ptr(), sk.shape[1],
                     int(max_suffix), dk.data_ptr(), dv.data_ptr(), dk.stride(0), dk.stride(1), dk.stride(2), Br, Mq,
                     suf_len.data_ptr() if suf_len is not None else None)
    kp = 0
    if prefix_idx is not None:
        _need_cuda(prefix_idx, "prefix_idx", torch.int32)
        if not prefix_idx.is_contiguous():
            raise FxError(FX_ERR_INVALID_ARG, "prefix_idx must be contiguous [Br, Hkv, kp]")
        kp = prefix_idx.shape[-1]
    if out is None:
        out = torch.empty((Br, Hq, Mq, d), dtype=torch.float32, device=q.device)
    np_ = kp if prefix_idx is not None else P
    nbytes = lib.fx_shared_prefix_workspace_bytes(Br, Hkv, Hq, Mq, np_, int(max_suffix))
    buf = _workspace(ws, nbytes, q.device, stream)
    sc = _default_scale(d) if scale is None else float(scale)
    _check(lib.fx_shared_prefix_decode(ctypes.byref(pre), ctypes.byref(brd), _ptr(q), Hq, _ptr(prefix_idx), kp, sc,
                                       _ptr(out), _ptr(buf), buf.numel(), int(flags), _stream(stream)))
    return out


def _strides(t):
    """The strides of a view, 0 for a dimension of one entry (whose stride addresses nothing)."""
    return tuple([s if n > 1 else 0 for s, n in zip(t.stride(), t.shape)])


class PagedKV:
    """One layer's paged KV cache (include/fx.h: paged KV cache), as the fx_paged_* calls take it.

    k, v       bf16 [n_pages, Hkv, page_rows, 128], or uint8 [n_pages, Hkv, page_rows, 64] (4-bit codes)
    k_scale, v_scale   uint8 or float8_e4m3fn [n_pages, Hkv, page_rows, 8] (4-bit only)
    table      int32 [B, max_pages]: the pages of each sequence in order
    length     int32 [B]: rows of each sequence, read on the device by every call
    k_exp, v_exp       4-bit: the values held are code * scale * 2^exp

    Views with any strides work (unit last stride, rows on 16-byte, scale rows on 8-byte boundaries; k and v,
    k_scale and v_scale with equal strides).  The object keeps its tensors; their contents may change between calls.
    """

    def __init__(self, k, v, table, length, *, k_scale=None, v_scale=None, k_exp: int = 0, v_exp: int = 0):
        packed = isinstance(k, torch.Tensor) and k.dtype == torch.uint8
        for t, name in ((k, "k"), (v, "v")):
            _need_cuda(t, name, torch.uint8 if packed else torch.bfloat16)
        width = 64 if packed else 128
        if k.dim() != 4 or k.shape != v.shape or _strides(k) != _strides(v) or k.shape[3] != width or k.stride(3) != 1:
            raise FxError(FX_ERR_INVALID_ARG, f"k and v must be [n_pages, Hkv, page_rows, {width}] views with equal "
                                              "strides, unit last stride")
        if (k_scale is None) == packed or (v_scale is None) == packed:
            raise FxError(FX_ERR_INVALID_ARG, "a 4-bit cache needs k_scale and v_scale, a bf16 cache has none")
        if packed:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _need_cuda(t, name, torch.float8_e4m3fn if getattr(t, "dtype", None) == torch.float8_e4m3fn
                           else torch.uint8)
            if k_scale.shape != k.shape[:3] + (8,) or k_scale.shape != v_scale.shape or k_scale.stride(3) != 1 or \
                    _strides(k_scale) != _strides(v_scale):
                raise FxError(FX_ERR_INVALID_ARG, "k_scale and v_scale must be [n_pages, Hkv, page_rows, 8] views with "
                                                  "equal strides, unit last stride")
        _need_cuda(table, "table", torch.int32)
        _need_cuda(length, "length", torch.int32)
        if table.dim() != 2 or table.stride(1) != 1 or length.dim() != 1 or length.shape[0] != table.shape[0] or \
                not length.is_contiguous():
            raise FxError(FX_ERR_INVALID_ARG, "table must be [B, max_pages] with unit last stride, length [B]")
        if any(t is not None and t.device != k.device for t in (v, table, length, k_scale, v_scale)):
            raise FxError(FX_ERR_INVALID_ARG, "the cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale, self.table, self.length = k, v, k_scale, v_scale, table, length
        self.device, self._index = k.device, k.get_device()
        self.n_pages, self.Hkv, self.page_rows, _ = k.shape
        self.B, self.max_pages = table.shape
        ks, ss = _strides(k), _strides(k_scale) if packed else (0, 0, 0, 0)
        self._desc = PagedDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if packed else None,
                               v_scale.data_ptr() if packed else None, table.data_ptr(), length.data_ptr(),
                               ks[0], ks[1], ks[2], ss[0], ss[1], ss[2],
                               table.stride(0) if self.B > 1 else self.max_pages,
                               FX_PAGED_E2M1 if packed else FX_PAGED_BF16, self.B, self.Hkv, 128, self.page_rows,
                               self.n_pages, self.max_pages, int(k_exp), int(v_exp))
        self._ref = ctypes.addressof(self._desc)
        self._rows = self.max_pages * self.page_rows


# These calls run once or more per layer and token: their checks are written for few interpreter steps.
# The current stream's handle without a Stream object around it (3 us against 0.1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device   # (CUDA is up: a cache exists)
_ROWS = struct.Struct("@PPqqPPqqqqPPPPiiiiixxxx")   # PagedRows
assert _ROWS.size == ctypes.sizeof(PagedRows)


def _paged_bad(cache, t, name, dtype, shape, contiguous):
    if not isinstance(t, torch.Tensor) or t.device != cache.device:
        raise FxError(FX_ERR_INVALID_ARG, f"{name} must be a tensor on {cache.device}")
    if t.dtype != dtype or t.shape != shape:
        raise FxError(FX_ERR_INVALID_ARG, f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if contiguous:
        raise FxError(FX_ERR_INVALID_ARG, f"{name} must be contiguous")


def _paged_tensor(cache, t, name, dtype, shape):
    """The address of a contiguous tensor of that type and shape on the cache's device; raises otherwise."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == cache._index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _paged_bad(cache, t, name, dtype, shape, True)


def _paged_view(cache, t, name, shape):
    """(address, strides) of a bf16 view with unit last stride."""
    try:
        if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == cache._index:
            st = t.stride()
            if st[-1] == 1:
                if (st[0] | st[1] | st[-2]) & 7:   # (views of 3 or 4 dimensions)
                    return t.data_ptr(), _strides(t)   # (the library refuses what then still is no multiple of 8)
                return t.data_ptr(), st
            raise FxError(FX_ERR_INVALID_ARG, f"{name} must have unit last stride")
    except AttributeError:
        pass
    _paged_bad(cache, t, name, torch.bfloat16, shape, False)
    raise FxError(FX_ERR_INVALID_ARG, f"{name} must be a bf16 view")


def _paged_launch(cache, stream):
    """(library, stream handle) of a call on the cache, which must live on the current device."""
    if type(cache) is not PagedKV and not isinstance(cache, PagedKV):
        raise FxError(FX_ERR_INVALID_ARG, "cache must be a PagedKV")
    if _current_device() != cache._index:
        raise FxError(FX_ERR_INVALID_ARG, f"the cache is on {cache.device}, the current device is another one")
    if stream is None:
        return _lib or load_library(), _raw_stream(cache._index)
    return _lib or load_library(), stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _paged_alloc(cache, stream, shape, dtype):
    with _on_stream(cache.device, stream):
        return torch.empty(shape, dtype=dtype, device=cache.device)


def fx_paged_append(cache, k_new, v_new, seq, pos, *, cos_sin=None, rope_pos=None, interleaved: bool = False, q=None,
                    q_out=None, stream=None, flags: int = 0):
    """Append the rows of n tokens to a paged cache, rotated by position on the way; returns the rotated queries.

    k_new, v_new [n, Hkv, 128] bf16 views with equal strides; seq, pos int32 [n]: the sequence (-1: padding, left
    out) and the row each token writes.  cos_sin fp32 [n_pos, rot] (rot/2 cosines, rot/2 sines a row) rotates the
    first rot dimensions of K and of q [n, Hq, 128] by rope_pos (int32 [n]; pos when None), in halves or, with
    interleaved, in neighbouring pairs.  q_out [n, Hq, 128] (allocated when None; may be q).
    """
    lib, st = _paged_launch(cache, stream)
    n = seq.shape[0] if isinstance(seq, torch.Tensor) and seq.dim() == 1 else -1
    seq_at = _paged_tensor(cache, seq, "seq", torch.int32, (n,))
    pos_at = _paged_tensor(cache, pos, "pos", torch.int32, (n,))
    k_at, ks = _paged_view(cache, k_new, "k_new", (n, cache.Hkv, 128))
    v_at, vs = _paged_view(cache, v_new, "v_new", (n, cache.Hkv, 128))
    if ks != vs:
        ks = _strides(k_new)
        if ks != _strides(v_new):
            raise FxError(FX_ERR_INVALID_ARG, "k_new and v_new must have equal strides")
    q_at = o_at = Hq = 0
    qs = os_ = (0, 0, 1)
    if q is not None:
        Hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
        q_at, qs = _paged_view(cache, q, "q", (n, Hq, 128))
        if q_out is None:
            q_out = _paged_alloc(cache, stream, (n, Hq, 128), torch.bfloat16)
        o_at, os_ = _paged_view(cache, q_out, "q_out", (n, Hq, 128))
    elif q_out is not None:
        raise FxError(FX_ERR_INVALID_ARG, "q_out needs q")
    if n == 0:
        return q_out
    rope_at = 0 if rope_pos is None else _paged_tensor(cache, rope_pos, "rope_pos", torch.int32, (n,))
    cs_at = rot = n_pos = 0
    if cos_sin is not None:
        n_pos, rot = cos_sin.shape if isinstance(cos_sin, torch.Tensor) and cos_sin.dim() == 2 else (-1, -1)
        cs_at = _paged_tensor(cache, cos_sin, "cos_sin", torch.float32, (n_pos, rot))
    rows = _ROWS.pack(k_at, v_at, ks[0], ks[1], q_at, o_at, qs[0], qs[1], os_[0], os_[1], seq_at, pos_at, rope_at, cs_at,
                      n, Hq, rot, n_pos, 1 if interleaved else 0)
    rc = lib.fx_paged_append(cache._ref, rows, flags, st)
    if rc:
        _check(rc)
    return q_out


def fx_paged_gather(cache, n: int, *, idx=None, lo=None, k_out=None, v_out=None, stream=None, flags: int = 0):
    """Rows of a paged cache as bf16 [B, Hkv, n, 128] K and V: rows idx [B, Hkv, n] (int32) of each (sequence, KV
    head), or rows lo[b] .. lo[b] + n - 1 (lo int32 [B], 0 when None).  Rows past the length are not written: give
    k_out and v_out where that can happen and their old contents count.
    """
    lib, st = _paged_launch(cache, stream)
    n = int(n)
    if n < 0:
        raise FxError(FX_ERR_INVALID_ARG, "n must be >= 0")
    shape = (cache.B, cache.Hkv, n, 128)
    idx_at = None if idx is None else _paged_tensor(cache, idx, "idx", torch.int32, shape[:3])
    lo_at = None if lo is None else _paged_tensor(cache, lo, "lo", torch.int32, (cache.B,))
    if k_out is None:
        k_out = _paged_alloc(cache, stream, shape, torch.bfloat16)
    if v_out is None:
        v_out = _paged_alloc(cache, stream, shape, torch.bfloat16)
    k_at = _paged_tensor(cache, k_out, "k_out", torch.bfloat16, shape)
    v_at = _paged_tensor(cache, v_out, "v_out", torch.bfloat16, shape)
    rc = lib.fx_paged_gather(cache._ref, idx_at, lo_at, n, k_at, v_at, flags, st) if n else 0
    if rc:
        _check(rc)
    return k_out, v_out


def fx_paged_decode_workspace_bytes(B, Hkv, Hq, Mq) -> int:
    return int(load_library().fx_paged_decode_workspace_bytes(B, Hkv, Hq, Mq))


_stream_ws = {}


def _paged_workspace(cache, nbytes, stream, handle):
    """The workspace of a call without one of its caller's: one for each device and stream (two streams never share
    one), kept for the next call.  A call on a stream that is being captured gets one of its own, from the graph's
    memory."""
    if handle == _PER_THREAD:
        raise FxError(FX_ERR_INVALID_ARG, _PER_THREAD_TEXT)
    with _on_stream(cache.device, stream):
        if torch.cuda.is_current_stream_capturing():
            ws = Workspace(cache.device)
        else:
            ws = _stream_ws.get((cache._index, handle))
            if ws is None:
                ws = _stream_ws[(cache._index, handle)] = Workspace(cache.device)
        return ws.ensure(nbytes, stream)


def _paged_queries(cache, q):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise FxError(FX_ERR_INVALID_ARG, f"q must be a bf16 [{cache.B}, Hq, Mq, 128] tensor on {cache.device}")
    _, Hq, Mq, _ = q.shape
    at, st = _paged_view(cache, q, "q", (cache.B, Hq, Mq, 128))
    return at, st, Hq, Mq


_SCALE = _default_scale(128)


def fx_paged_decode(cache, q, idx=None, tail_lo=None, *, scale=None, out=None, lse=None, want_lse=False, ws=None,
                    stream=None, flags: int = 0):
    """Attention of q [B, Hq, Mq, 128] (bf16, any strides) over a paged cache; query i sits at row len - Mq + i.

    Dense, or over the rows idx [B, Hkv, k] (int32) and the tail from row tail_lo[b] (int32 [B]) on.  Returns out
    [B, Hq, Mq, 128] fp32, or (out, lse [B, Hq, Mq]) when lse is given or wanted.

    Without ws the call takes the scratch memory that is kept for its stream, or, on a stream that is being captured, some
    of the graph's.  The per-thread default stream (handle 2) is refused without ws: its handle does not tell threads apart.
    A stream of one's own that is destroyed has finished its calls first: its handle may come back.
    """
    lib, st = _paged_launch(cache, stream)
    q_at, qs, Hq, Mq = _paged_queries(cache, q)
    B = cache.B
    kk, idx_at = 0, None
    if idx is not None:
        kk = idx.shape[-1] if isinstance(idx, torch.Tensor) and idx.dim() == 3 else -1
        idx_at = _paged_tensor(cache, idx, "idx", torch.int32, (B, cache.Hkv, kk)) or None
    lo_at = None if tail_lo is None else _paged_tensor(cache, tail_lo, "tail_lo", torch.int32, (B,))
    if out is None:
        out = _paged_alloc(cache, stream, (B, Hq, Mq, 128), torch.float32)
    out_at = _paged_tensor(cache, out, "out", torch.float32, (B, Hq, Mq, 128))
    if lse is None and want_lse:
        lse = _paged_alloc(cache, stream, (B, Hq, Mq), torch.float32)
    lse_at = None if lse is None else _paged_tensor(cache, lse, "lse", torch.float32, (B, Hq, Mq))
    nbytes = lib.fx_paged_decode_workspace_bytes(B, cache.Hkv, Hq, Mq)
    buf = _paged_workspace(cache, nbytes, stream, st) if ws is None else ws.ensure(nbytes, stream)
    if buf.get_device() != cache._index:
        raise FxError(FX_ERR_INVALID_ARG, f"ws must be a workspace on {cache.device}")
    rc = lib.fx_paged_decode(cache._ref, q_at, qs[0], qs[1], qs[2], Hq, Mq, idx_at, kk, lo_at,
                             _SCALE if scale is None else scale, out_at, lse_at, buf.data_ptr(), buf.numel(), flags, st)
    if rc:
        _check(rc)
    return out if lse is None else (out, lse)


def fx_paged_importance(cache, q, lse, *, scale=None, cand=None, scores=None, stream=None, flags: int = 0):
    """Importance of the rows cand = (lo, hi) of a paged cache (default: the whole capacity, or the width of scores
    when given): fp32 [B, Hkv, hi - lo], from the queries and the lse [B, Hq, Mq] of fx_paged_decode."""
    lib, st = _paged_launch(cache, stream)
    q_at, qs, Hq, Mq = _paged_queries(cache, q)
    lse_at = _paged_tensor(cache, lse, "lse", torch.float32, (cache.B, Hq, Mq))
    if cand is not None:
        lo, hi = int(cand[0]), int(cand[1])
    else:
        lo, hi = 0, cache._rows
        if isinstance(scores, torch.Tensor) and scores.dim() == 3:
            hi = scores.shape[2]
    if not 0 <= lo <= hi <= cache._rows:
        raise FxError(FX_ERR_INVALID_ARG, f"need 0 <= cand[0] <= cand[1] <= {cache._rows}")
    if scores is None:
        scores = _paged_alloc(cache, stream, (cache.B, cache.Hkv, hi - lo), torch.float32)
    s_at = _paged_tensor(cache, scores, "scores", torch.float32, (cache.B, cache.Hkv, hi - lo))
    rc = 0 if hi == lo else lib.fx_paged_importance(cache._ref, q_at, qs[0], qs[1], qs[2], Hq, Mq, lse_at,
                                                    _SCALE if scale is None else scale, lo, hi, s_at, flags, st)
    if rc:
        _check(rc)
    return scores


class BranchPool:
    """Host bookkeeping of content branches forked from one shared prefix (include/fx.h: branch pool).
    Thin wrapper: every method is one C call; errors raise FxError."""

    def __init__(self, prefix_cap: int, max_branches: int, slot_rows: int):
        lib = load_library()
        self._lib = lib
        self._h = lib.fx_branch_pool_create(int(prefix_cap), int(max_branches), int(slot_rows))
        if not self._h:
            _check(FX_ERR_INVALID_ARG)
        self.max_branches = int(max_branches)
        self.slot_rows = int(slot_rows)

    def _int(self, r):
        if r < 0:
            raise FxError(FX_ERR_INVALID_ARG, self._lib.fx_last_error().decode(errors="replace"))
        return int(r)

    def extend_prefix(self, n: int) -> int:
        return self._int(self._lib.fx_branch_pool_extend_prefix(self._h, int(n)))

    def fork(self) -> int:
        return self._int(self._lib.fx_branch_pool_fork(self._h))

    def append(self, branch: int, n: int) -> int:
        return self._int(self._lib.fx_branch_pool_append(self._h, int(branch), int(n)))

    def release(self, branch: int) -> int:
        return self._int(self._lib.fx_branch_pool_release(self._h, int(branch)))

    def release_parent(self) -> int:
        return self._int(self._lib.fx_branch_pool_release_parent(self._h))

    def prefix_refs(self) -> int:
        return self._int(self._lib.fx_branch_pool_prefix_refs(self._h))

    def prefix_len(self) -> int:
        return self._int(self._lib.fx_branch_pool_prefix_len(self._h))

    def batch(self):
        """(ids, suf_start, suf_len, prefix_len) of the live branches, as int32 CPU tensors."""
        m = self.max_branches
        arrs = [(ctypes.c_int32 * m)() for _ in range(4)]
        n = self._int(self._lib.fx_branch_pool_batch(self._h, *arrs))
        return tuple(torch.tensor(list(a)[:n], dtype=torch.int32) for a in arrs)

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h:
            self._lib.fx_branch_pool_destroy(h)


def fx_device_errors(stream=None) -> int:
    """Synchronise the stream and return (and clear) the FX_DEVERR_* bits of the current device."""
    bits = ctypes.c_uint(0)
    st = load_library().fx_device_errors(ctypes.byref(bits), _stream(stream))
    if st not in (FX_OK, FX_ERR_DEVICE):
        _check(st)
    return int(bits.value)
