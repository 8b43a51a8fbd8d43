"""Thin ctypes binding of libmapflow (include/mapflow.h).

Argument marshalling only: every step of the method runs in the CUDA
library.  PyTorch supplies device memory (its caching allocator is handed to
the library as the BSR allocator) and streams.  If the shared library is
missing, importing this module raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Dict, List, Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmapflow.so")

MF_OK, MF_ERR_ARG, MF_ERR_UNSUPPORTED, MF_ERR_CUDA, MF_ERR_OOM, MF_ERR_TIMEOUT, MF_ERR_STATE = range(7)
MF_DTYPE_F32, MF_DTYPE_BF16 = 0, 1

EXPORTED = ("mf_version", "mf_last_error", "mf_supported", "mf_bsr_create", "mf_bsr_destroy",
            "mf_compress", "mf_retrieve", "mf_bsr_info", "mf_bsr_export", "mf_bsr_copy",
            "mf_bsr_release_layer", "mf_bsr_offload", "mf_bsr_prefetch", "mf_calibrate_head_map",
            "mf_device_status", "mf_selftest_wait", "mf_profile",
            "mf_profile_read", "mf_profile_kinds", "mf_select_noalloc", "mf_bsr_set_exact",
            "mf_bsr_create_chunked", "mf_prefix_hashes", "mf_bm_create", "mf_bm_destroy",
            "mf_bm_insert", "mf_bm_match", "mf_bm_assemble", "mf_bm_stats",
            "mf_rope_frequencies", "mf_qk_norm_rope", "mf_attn_create_packed", "mf_attn_create_cache",
            "mf_attn_destroy", "mf_attn_workspace", "mf_attn_packed", "mf_attn_cached", "mf_attn_status",
            "mf_cache_append", "mf_cache_read", "mf_attn_paged_workspace", "mf_attn_paged",
            "mf_cache_append_args", "mf_cache_read_args", "mf_attn_paged_args")
KERNELS = ("stats", "select", "scan", "pack", "union", "retrieve")


class MapFlowError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"mapflow error {code}: {msg}")
        self.code = code


ALLOC_FN = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p)
FREE_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)

class CacheStruct(ctypes.Structure):
    """mf_cache_t of mapflow.h."""
    _fields_ = [("format", ctypes.c_int), ("page_size", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int),
                ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


# mf_cache_append_args_t, mf_cache_read_args_t and mf_attn_paged_args_t: an argument
# through ctypes costs 0.07 us, here 0.01
_append_args = struct.Struct("=13q2d6i").pack
_read_args = struct.Struct("=10q4i").pack
_paged_args = struct.Struct("=13q2d6i").pack


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmapflow.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i32, i64p = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)
    lib.mf_version.restype = i32
    lib.mf_last_error.restype = ctypes.c_char_p
    lib.mf_supported.argtypes = [i32, i32, i32]
    lib.mf_bsr_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, i32,
                                  ctypes.POINTER(ctypes.c_int32), i32, ALLOC_FN, FREE_FN, vp]
    lib.mf_bsr_destroy.argtypes = [vp]
    lib.mf_bsr_destroy.restype = None
    lib.mf_compress.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, ctypes.c_float,
                                i32, vp]
    lib.mf_retrieve.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32,
                                ctypes.POINTER(ctypes.c_int32), i32, vp]
    lib.mf_bsr_info.argtypes = [vp, i32, i64p, i64p, i64p]
    lib.mf_bsr_export.argtypes = [vp, i32] + [ctypes.POINTER(vp)] * 6
    lib.mf_bsr_copy.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.mf_bsr_release_layer.argtypes = [vp, i32]
    lib.mf_bsr_offload.argtypes = [vp, i32, vp]
    lib.mf_calibrate_head_map.argtypes = [vp, i32, vp, i32, ctypes.c_float, vp, vp]
    lib.mf_bsr_prefetch.argtypes = [vp, i32, vp]
    lib.mf_bsr_set_exact.argtypes = [vp, i32]
    lib.mf_device_status.argtypes = [vp, vp]
    lib.mf_selftest_wait.argtypes = [vp, i32, vp]
    lib.mf_select_noalloc.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), i32, i32, i32, i32,
                                      ctypes.c_float, vp, vp, ctypes.c_int64, vp, vp]
    lib.mf_profile.argtypes = [vp, i32]
    lib.mf_profile_kinds.argtypes = [vp, i32]
    lib.mf_profile_read.argtypes = [vp, i32, i64p, ctypes.POINTER(ctypes.c_double)]
    u64p = ctypes.POINTER(ctypes.c_uint64)
    lib.mf_prefix_hashes.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                     vp, i32, i32, ctypes.c_uint64, u64p, ctypes.c_int64, i64p]
    lib.mf_bsr_create_chunked.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, i32,
                                          ctypes.POINTER(ctypes.c_int32), vp, i32, ALLOC_FN,
                                          FREE_FN, vp]
    lib.mf_bm_create.argtypes = [ctypes.POINTER(vp), i32, i32, ctypes.c_int64, ALLOC_FN, FREE_FN,
                                 vp, vp]
    lib.mf_bm_destroy.argtypes = [vp]
    lib.mf_bm_insert.argtypes = [vp, i32, vp, i32, u64p, i64p, vp]
    lib.mf_bm_match.argtypes = [vp, i32, u64p, i32, ctypes.POINTER(i32)]
    lib.mf_bm_assemble.argtypes = [vp, i32, u64p, vp, i32, vp]
    lib.mf_bm_stats.argtypes = [vp, i64p]
    i64, f32, f64 = ctypes.c_int64, ctypes.c_float, ctypes.c_double
    lib.mf_rope_frequencies.argtypes = [i32, f64, i32, f64, i32, f64, f64, u64p, ctypes.POINTER(f32)]
    lib.mf_qk_norm_rope.argtypes = [vp, i64] * 4 + [vp, vp, i32, f32, vp, vp, i32, i32, f32, i32, i32, i32,
                                                    i32, i32, vp]
    lib.mf_attn_create_packed.argtypes = [ctypes.POINTER(vp), vp, vp, i32, i32, i32, i32, i32, i32, ALLOC_FN,
                                          FREE_FN, vp]
    lib.mf_attn_create_cache.argtypes = [ctypes.POINTER(vp)] + [i32] * 9 + [ALLOC_FN, FREE_FN, vp]
    lib.mf_attn_destroy.argtypes = [vp]
    lib.mf_attn_destroy.restype = None
    lib.mf_attn_workspace.argtypes = [vp, i32, i64p]
    lib.mf_attn_packed.argtypes = [vp] + [vp, i64] * 4 + [vp, i32, f32, vp, i64, vp]
    lib.mf_attn_cached.argtypes = [vp, i32] + [vp, i64] * 3 + [vp] + [vp, i64] * 3 + [vp, i32, f32, vp, i64, vp]
    lib.mf_attn_status.argtypes = [vp, vp]
    lib.mf_cache_append.argtypes = [vp] + [vp, i64] * 2 + [i32, vp, vp, vp, i64, i32, i32, vp, vp, i32, i32, f32, vp,
                                                           i32, f32, vp]
    lib.mf_cache_read.argtypes = [vp, i32, vp, vp, vp, i64, i32, i32, vp, i64, vp, i64, vp]
    lib.mf_attn_paged_workspace.argtypes = [i32, i32, i32, i32, i64p]
    lib.mf_attn_paged.argtypes = [vp, i32, i32, i32, vp, i64, vp, i64, i32, vp, vp, i64, vp, vp, f32, i32, i32, f32,
                                  vp, i64, vp]
    for name in ("mf_cache_append_args", "mf_cache_read_args", "mf_attn_paged_args"):
        getattr(lib, name).argtypes = [ctypes.c_char_p]
    for name in EXPORTED:
        getattr(lib, name)
    _lib = lib
    return lib


def _check(rc: int) -> None:
    if rc != MF_OK:
        raise MapFlowError(rc, load_library().mf_last_error().decode(errors="replace"))


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MF_DTYPE_BF16
    if t.dtype == torch.float32:
        return MF_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _on(t, stream):
    """(guard, raw stream) for a call on the GPU of tensor or device `t`:
    inside the guard, device and stream are the call's, so that memory made
    there belongs to the stream the call runs on."""
    import torch
    device = getattr(t, "device", t)
    if device.type != "cuda":
        raise MapFlowError(MF_ERR_ARG, f"a CUDA tensor is needed, not one on {device}")
    if stream is None:
        with torch.cuda.device(device):
            stream = torch.cuda.current_stream()
    elif stream.device != device:
        raise MapFlowError(MF_ERR_ARG, f"the stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream), stream.cuda_stream  # (the stream's device becomes current too)


def _raw_current(index: int):
    """The current stream of GPU `index` where that is the current device
    (no guard is needed then), else None.  A decode step makes several such
    calls a layer: this takes 0.3 us, a guard with its stream objects 7."""
    import torch
    c = torch._C
    if index >= 0 and c._cuda_getDevice() == index:
        return c._cuda_getCurrentRawStream(index)
    return None


_INT_MAX = 2 ** 31 - 1


def _int(name: str, x) -> int:
    """x as an int of the C ABI (ctypes would cut it to 32 bits)."""
    x = int(x)
    if not -_INT_MAX <= x <= _INT_MAX:
        raise MapFlowError(MF_ERR_ARG, f"{name} = {x} is out of range")
    return x


def _ints(name: str, xs) -> np.ndarray:
    """xs as an int32 array (a cast of a wider one would cut it to 32 bits)."""
    wide = np.asarray(xs, dtype=np.int64)
    cut = np.ascontiguousarray(wide.astype(np.int32))
    if (cut != wide).any():
        raise MapFlowError(MF_ERR_ARG, f"{name}: a value is out of range")
    return cut


def _span(name: str, x, least: int) -> int:
    """A number of keys, at least `least`; more than any sequence has is as many as the C ABI can say."""
    if x < least:
        raise MapFlowError(MF_ERR_ARG, f"{name} = {x} must be >= {least}" + (" (None: no window)" if least else ""))
    return min(int(x), _INT_MAX)


def _empty(t, shape):
    """A new contiguous tensor like t, of `shape` (t's, checked before)."""
    import torch
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(shape, dtype=t.dtype, device=t.device)


def _rows(name: str, t, shape, dtype, gpu: int) -> int:
    """Checks a tensor of `shape` [..., heads, d] on GPU `gpu` whose leading
    dimensions are equally spaced tokens; returns the values between two
    tokens."""
    heads, d = shape[-2:]
    if t.dtype is dtype and t.get_device() == gpu and t.shape == shape:
        if t.is_contiguous():
            return heads * d
        st = t.stride()
        if st[-1] == 1 and (st[-2] == d or heads == 1):
            if len(st) == 3:
                return st[0] if shape[0] != 1 else heads * d
            n, ld = 1, None
            for i in range(len(st) - 3, -1, -1):
                if shape[i] != 1:
                    if ld is None:
                        ld = st[i]
                    elif st[i] != n * ld:
                        raise MapFlowError(MF_ERR_ARG, f"{name}: its tokens are not equally spaced")
                n *= shape[i]
            return heads * d if ld is None else ld
        raise MapFlowError(MF_ERR_ARG, f"{name}: a token's heads must lie next to each other")
    raise MapFlowError(MF_ERR_ARG, f"{name} must be a {dtype} tensor {tuple(shape)} on cuda:{gpu}, is {t.dtype} "
                                   f"{tuple(t.shape)} on {t.device}")


def _vector(name: str, t, shape, dtype, gpu: int):
    if t.dtype is not dtype or t.get_device() != gpu or t.shape != shape or not t.is_contiguous():
        raise MapFlowError(MF_ERR_ARG, f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on cuda:{gpu}")


# ------------------------------------------------------ torch allocator ----
def _torch_allocator():
    import torch

    def _alloc(nbytes, ctx, stream):
        try:
            return torch.cuda.caching_allocator_alloc(int(nbytes), device=torch.cuda.current_device(),
                                                      stream=stream or 0)
        except Exception:  # noqa: BLE001 - signalled to the library as NULL
            return None

    def _free(ptr, ctx, stream):
        if ptr:
            torch.cuda.caching_allocator_delete(ptr)
    return ALLOC_FN(_alloc), FREE_FN(_free)


# ------------------------------------- memory that pending kernels read ----
_parked: List = []  # releases put off while a stream was captured


def _capturing(gpu: int) -> bool:
    """Whether a stream is known to be captured: this thread's current one, on
    its device or on `gpu`, or the one that torch.cuda.graph takes by itself."""
    import torch
    if not torch.cuda.is_initialized():
        return False
    if torch.cuda.is_current_stream_capturing():
        return True
    if gpu != torch.cuda.current_device():
        with torch.cuda.device(gpu):
            if torch.cuda.is_current_stream_capturing():
                return True
    s = getattr(torch.cuda.graph, "default_capture_stream", None)
    if s is not None:
        with torch.cuda.stream(s):
            return torch.cuda.is_current_stream_capturing()
    return False


def _release(gpu: int, wait_and_free) -> None:
    """Calls wait_and_free(), which waits for GPU `gpu` before it gives memory
    back.  A device cannot be waited for while one of its streams is captured
    (that ends the capture): then the release is put off to the next one."""
    _parked.append((gpu, wait_and_free))
    _release_parked()


def _release_parked() -> None:
    for _ in range(len(_parked)):
        try:
            gpu, wait_and_free = _parked.pop(0)
        except IndexError:  # another thread has taken it
            return
        try:
            if _capturing(gpu):
                _parked.append((gpu, wait_and_free))
            else:
                wait_and_free()
        except Exception:  # noqa: BLE001 - the wait failed: keep the memory, see to the others
            _parked.append((gpu, wait_and_free))


# --------------------------------------------- same names as the C ABI -----
def mf_version() -> int:
    return load_library().mf_version()


def mf_supported(dtype: int, d: int, B: int) -> bool:
    return bool(load_library().mf_supported(dtype, d, B))


def mf_bsr_create(n_layers: int, T: int, H_s: int, B: int, causal: bool,
                  cu_seqlens: Sequence[int], use_torch_allocator: bool = True,
                  q_begin: Optional[Sequence[int]] = None):
    """Returns (handle, keepalive); keepalive holds the allocator callbacks.
    With q_begin the handle covers query chunks (mf_bsr_create_chunked)."""
    lib = load_library()
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    h = ctypes.c_void_p()
    if use_torch_allocator:
        a, f = _torch_allocator()
    else:
        a, f = ALLOC_FN(), FREE_FN()
    i32p = ctypes.POINTER(ctypes.c_int32)
    if q_begin is None:
        rc = lib.mf_bsr_create(ctypes.byref(h), n_layers, T, H_s, B, int(causal),
                               cu.ctypes.data_as(i32p), len(cu) - 1, a, f, None)
    else:
        qb = np.ascontiguousarray(np.asarray(q_begin, dtype=np.int32))
        rc = lib.mf_bsr_create_chunked(ctypes.byref(h), n_layers, T, H_s, B, int(causal),
                                       cu.ctypes.data_as(i32p), qb.ctypes.data_as(ctypes.c_void_p),
                                       len(cu) - 1, a, f, None)
    _check(rc)
    return h, (a, f)


def mf_bsr_destroy(h) -> None:
    load_library().mf_bsr_destroy(h)


def mf_compress(h, layer: int, q, k, T: int, H_s: int, H_ks: int, d: int, B: int, p: float,
                causal: bool, stream=None) -> None:
    _check(load_library().mf_compress(h, layer, _ptr(q), _ptr(k), _dtype_code(q), T, H_s, H_ks,
                                      d, B, float(p), int(causal), _stream(stream)))


def mf_retrieve(h, W, v, o, H_r: int, H_kv: int, d: int, layer_map: Sequence[int],
                stream=None) -> None:
    lm = np.ascontiguousarray(np.asarray(layer_map, dtype=np.int32))
    _check(load_library().mf_retrieve(h, _ptr(W), _ptr(v), _ptr(o), _dtype_code(v), H_r, H_kv, d,
                                       lm.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(lm),
                                       _stream(stream)))


def mf_bsr_set_exact(h, exact: bool) -> None:
    _check(load_library().mf_bsr_set_exact(h, int(exact)))


def mf_bsr_info(h, layer: int):
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(load_library().mf_bsr_info(h, layer, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def mf_bsr_copy(h, layer: int, row_ptr=None, col_idx=None, values=None, mass=None,
                row_max=None, row_sum=None, stream=None) -> None:
    _check(load_library().mf_bsr_copy(h, layer, _ptr(row_ptr), _ptr(col_idx), _ptr(values),
                                      _ptr(mass), _ptr(row_max), _ptr(row_sum), _stream(stream)))


def mf_bsr_release_layer(h, layer: int) -> None:
    _check(load_library().mf_bsr_release_layer(h, layer))


def mf_bsr_offload(h, layer: int, stream=None) -> None:
    _check(load_library().mf_bsr_offload(h, layer, _stream(stream)))


def mf_bsr_prefetch(h, layer: int, stream=None) -> None:
    _check(load_library().mf_bsr_prefetch(h, layer, _stream(stream)))


def calibrate_head_map(sender: "BSR", sender_layer: int, receiver: "BSR", receiver_layer: int,
                       ridge: float = 0.0, stream=None) -> np.ndarray:
    """Least-squares head map W [H_r, H_s] from two compressed layers over the
    same sequences (see mf_calibrate_head_map)."""
    W = np.zeros((receiver.H_s, sender.H_s), np.float32)
    _check(load_library().mf_calibrate_head_map(
        sender.handle, sender_layer, receiver.handle, receiver_layer, float(ridge),
        W.ctypes.data_as(ctypes.c_void_p), _stream(stream)))
    return W


def mf_device_status(h, stream=None) -> None:
    _check(load_library().mf_device_status(h, _stream(stream)))


def mf_selftest_wait(h, limit_ms: int, stream=None) -> None:
    _check(load_library().mf_selftest_wait(h, int(limit_ms), _stream(stream)))


def mf_select_noalloc(mass, cu_seqlens: Sequence[int], H_s: int, B: int, causal: bool,
                      p: float, row_ptr, col_idx, nnz, stream=None) -> None:
    """Selection into caller buffers with no device allocation (see mapflow.h).

    The library sees only pointers, so the buffer sizes, dtypes and devices
    are checked here, before any kernel could read or write past them."""
    import torch
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    lens = np.diff(cu.astype(np.int64))
    if len(cu) < 2 or cu[0] != 0 or (lens < 0).any() or B <= 0 or H_s <= 0:
        raise MapFlowError(MF_ERR_ARG, "cu_seqlens must start at 0 and be non-decreasing; "
                                       "B and H_s positive")
    nb = (lens + B - 1) // B
    R = int(nb.sum())
    C = int((nb * (nb + 1) // 2).sum()) if causal else int((nb * nb).sum())
    need = (("mass", mass, torch.float32, H_s * C), ("row_ptr", row_ptr, torch.int32, H_s * R + 1),
            ("col_idx", col_idx, torch.int32, 0), ("nnz", nnz, torch.int64, 1))
    for name, t, dt, n in need:
        if t.device.type != "cuda" or t.dtype != dt or not t.is_contiguous():
            raise MapFlowError(MF_ERR_ARG, f"{name} must be a contiguous CUDA {dt} tensor")
        if t.numel() < n:
            raise MapFlowError(MF_ERR_ARG, f"{name} holds {t.numel()} elements, needs {n}")
    _check(load_library().mf_select_noalloc(
        _ptr(mass), cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(cu) - 1, H_s, B,
        int(causal), float(p), _ptr(row_ptr), _ptr(col_idx), int(col_idx.numel()), _ptr(nnz),
        _stream(stream)))


def mf_profile(h, enable: bool) -> None:
    _check(load_library().mf_profile(h, int(enable)))


def mf_profile_kinds(h, mask: int) -> None:
    _check(load_library().mf_profile_kinds(h, int(mask)))


def mf_profile_read(h, kernel: int):
    n, ms = ctypes.c_int64(), ctypes.c_double()
    _check(load_library().mf_profile_read(h, kernel, ctypes.byref(n), ctypes.byref(ms)))
    return n.value, ms.value


def mf_prefix_hashes(tokens, cu_seqlens: Sequence[int], B: int, seed: int = 0,
                     q_begin: Optional[Sequence[int]] = None) -> np.ndarray:
    """Chained prefix hashes of the B-token blocks of each packed sequence
    (uint64 [R], the block-row order of a BSR handle with these cu_seqlens and
    q_begin)."""
    lib = load_library()
    tok = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    if len(cu) < 2 or cu[-1] != len(tok):
        raise ValueError("cu_seqlens must end at len(tokens)")
    qb = None if q_begin is None else np.ascontiguousarray(np.asarray(q_begin, dtype=np.int32))
    qb_ptr = None if qb is None else qb.ctypes.data_as(ctypes.c_void_p)
    i32p = ctypes.POINTER(ctypes.c_int32)
    n = ctypes.c_int64()
    _check(lib.mf_prefix_hashes(tok.ctypes.data_as(i32p), cu.ctypes.data_as(i32p), qb_ptr, len(cu) - 1,
                                B, ctypes.c_uint64(seed), None, 0, ctypes.byref(n)))
    out = np.zeros(n.value, np.uint64)
    _check(lib.mf_prefix_hashes(tok.ctypes.data_as(i32p), cu.ctypes.data_as(i32p), qb_ptr, len(cu) - 1,
                                B, ctypes.c_uint64(seed),
                                out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), n.value,
                                ctypes.byref(n)))
    return out


def _u64(hashes) -> Tuple[np.ndarray, "ctypes._Pointer"]:
    a = np.ascontiguousarray(np.asarray(hashes, dtype=np.uint64))
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64))


class BlockManager:
    """Owner of one mf_bm_t: block-rows of compressed layers cached under
    prefix hashes in a device tile pool (see mf_bm_* in mapflow.h)."""

    def __init__(self, H_s: int, B: int, tile_capacity: int, use_torch_allocator: bool = True,
                 stream=None):
        lib = load_library()
        self.H_s, self.B, self.tile_capacity = H_s, B, int(tile_capacity)
        h = ctypes.c_void_p()
        if use_torch_allocator:
            a, f = _torch_allocator()
        else:
            a, f = ALLOC_FN(), FREE_FN()
        self._keep = (a, f)
        _check(lib.mf_bm_create(ctypes.byref(h), H_s, B, self.tile_capacity, a, f, None,
                                _stream(stream)))
        self.handle = h

    def insert(self, key_layer: int, bsr: "BSR", layer: int, hashes, stream=None) -> Tuple[int, int, int]:
        """Caches the layer's block-rows; returns (inserted, already cached, evicted)."""
        arr, ptr = _u64(hashes)
        counts = (ctypes.c_int64 * 3)()
        _check(load_library().mf_bm_insert(self.handle, key_layer, bsr.handle, layer, ptr, counts,
                                           _stream(stream)))
        return int(counts[0]), int(counts[1]), int(counts[2])

    def match(self, key_layer: int, hashes) -> int:
        arr, ptr = _u64(hashes)
        n = ctypes.c_int()
        _check(load_library().mf_bm_match(self.handle, key_layer, ptr, len(arr), ctypes.byref(n)))
        return int(n.value)

    def assemble(self, key_layer: int, hashes, bsr: "BSR", layer: int, stream=None) -> None:
        """Makes `layer` of `bsr` a view of the cached block-rows `hashes`."""
        arr, ptr = _u64(hashes)
        _check(load_library().mf_bm_assemble(self.handle, key_layer, ptr, bsr.handle, layer,
                                             _stream(stream)))

    def stats(self) -> Dict[str, int]:
        out = (ctypes.c_int64 * 7)()
        _check(load_library().mf_bm_stats(self.handle, out))
        keys = ("entries", "tiles_used", "tile_capacity", "hits", "misses", "evictions", "pinned")
        return {k: int(v) for k, v in zip(keys, out)}

    def close(self) -> None:
        if self.handle is not None:
            _check(load_library().mf_bm_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass


# ---------------------------------- rotary embedding and attention layers --
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_LAYOUTS = {"half": 0, "interleaved": 1}


def mf_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                        original_length: int = 0, beta_fast: float = 32.0,
                        beta_slow: float = 1.0) -> Tuple[np.ndarray, float]:
    """(turns uint64 [rot_dim/2], gain): the rotary table (see mapflow.h)."""
    if scaling not in _SCALINGS:
        raise MapFlowError(MF_ERR_ARG, f"unknown scaling {scaling!r} ({', '.join(_SCALINGS)})")
    rot_dim, original_length = _int("rot_dim", rot_dim), _int("original_length", original_length)
    turns = np.zeros(max(rot_dim // 2, 1), np.uint64)
    gain = ctypes.c_float()
    _check(load_library().mf_rope_frequencies(
        rot_dim, float(base), _SCALINGS[scaling], float(factor), original_length, float(beta_fast),
        float(beta_slow), turns.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), ctypes.byref(gain)))
    return turns, float(gain.value)


def _wait_for(gpu: int, table) -> None:
    """Waits for GPU `gpu` while `table` is held."""
    import torch
    torch.cuda.synchronize(gpu)


class RotaryPlan:
    """A rotary table on the device: per-head norm and rotary embedding of
    queries and keys in one pass (see mf_qk_norm_rope in mapflow.h).

    scaling: "none", "linear", "ntk" or "yarn"; layout: "half" (pairs i and
    i + rot_dim/2) or "interleaved" (pairs 2i and 2i + 1).  No gradient is
    recorded.

    The plan may be used on any stream and dropped right after a call: its
    table goes back to the stream that was current when it was made, so where
    a call ran on another one, dropping the plan waits for the device.  A
    captured call reads the table at every replay: keep the plan as long as
    the graph."""

    _abroad = False  # a call ran on another stream than the table's

    def __init__(self, rot_dim: int, base: float = 10000.0, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original_length: int = 0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, device=None):
        import torch
        if layout not in _LAYOUTS:
            raise MapFlowError(MF_ERR_ARG, f"unknown layout {layout!r} ({', '.join(_LAYOUTS)})")
        turns, self.gain = mf_rope_frequencies(rot_dim, base, scaling, factor, original_length, beta_fast,
                                               beta_slow)
        self.rot_dim, self.layout, self._layout = int(rot_dim), layout, _LAYOUTS[layout]
        self._call = load_library().mf_qk_norm_rope
        device = torch.device("cuda" if device is None else device)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self._turns, self._gpu = self.turns.data_ptr(), self.turns.get_device()
        self._home = torch._C._cuda_getCurrentRawStream(self._gpu) if self._gpu >= 0 else None

    def __del__(self):
        if self._abroad:
            try:
                _release(self._gpu, functools.partial(_wait_for, self._gpu, self.turns))
            except Exception:  # noqa: BLE001
                pass

    def apply(self, q, k, positions, q_weight=None, k_weight=None, eps: float = 1e-6, norm: Optional[bool] = None,
              q_out=None, k_out=None, stream=None):
        """q [T, H_q, d] and k [T, H_k, d] (or None) normed and rotated;
        returns (q_out, k_out), new tensors unless given (q_out=q: in place).
        The norm is taken when a weight is given or norm is True."""
        code = _dtype_code(q)
        gpu = q.get_device()
        raw = None if stream is not None else _raw_current(gpu)
        if raw is not None:
            return self._apply(raw, gpu, code, q, k, positions, q_weight, k_weight, eps, norm, q_out, k_out)
        guard, raw = _on(q, stream)
        with guard:
            return self._apply(raw, gpu, code, q, k, positions, q_weight, k_weight, eps, norm, q_out, k_out)

    def _apply(self, raw, gpu, code, q, k, positions, q_weight, k_weight, eps, norm, q_out, k_out):
        import torch
        dt = q.dtype
        if self._gpu != gpu:
            raise MapFlowError(MF_ERR_ARG, f"q is on cuda:{gpu}, the plan on {self.turns.device}")
        if q.dim() != 3 or (k is not None and k.dim() != 3):
            raise MapFlowError(MF_ERR_ARG, "q and k must be [T, heads, d]")
        shape_q = T, H_q, d = q.shape
        ld_q = _rows("q", q, shape_q, dt, gpu)
        if q_out is None:
            q_out, ld_qo = _empty(q, shape_q), H_q * d
        else:
            ld_qo = _rows("q_out", q_out, shape_q, dt, gpu)
        H_k = ld_k = ld_ko = 0
        pk = pko = pwq = pwk = None
        if k is not None:
            H_k = k.shape[1]
            shape_k = (T, H_k, d)
            ld_k = _rows("k", k, shape_k, dt, gpu)
            if k_out is None:
                k_out, ld_ko = _empty(k, shape_k), H_k * d
            else:
                ld_ko = _rows("k_out", k_out, shape_k, dt, gpu)
            pk, pko = k.data_ptr(), k_out.data_ptr()
        elif k_out is not None:
            raise MapFlowError(MF_ERR_ARG, "k_out without k")
        _vector("positions", positions, (T,), torch.int32, gpu)
        if q_weight is not None:
            _vector("q_weight", q_weight, (d,), dt, gpu)
            pwq = q_weight.data_ptr()
        if k_weight is not None:
            _vector("k_weight", k_weight, (d,), dt, gpu)
            pwk = k_weight.data_ptr()
        if norm is None:
            norm = pwq is not None or pwk is not None
        if raw != self._home:
            self._abroad = True
        rc = self._call(
            q.data_ptr(), ld_q, q_out.data_ptr(), ld_qo, pk, ld_k, pko, ld_ko, pwq, pwk, norm, eps,
            positions.data_ptr(), self._turns, self.rot_dim, self._layout, self.gain, code, T, H_q, H_k, d, raw)
        if rc:
            _check(rc)
        return q_out, k_out


def _destroy_plan(handle, keep) -> None:
    """Waits for the plan's GPU and frees it; `keep` holds its allocator."""
    load_library().mf_attn_destroy(handle)


class _AttentionPlan:
    """Owner of one mf_attn_t.  Dropping it waits for its GPU, or, during a
    stream capture, puts the release off to the next one.  A captured call
    reads the plan at every replay: keep it as long as the graph."""

    handle = None
    _gpu = None

    def _workspace_bytes(self, n: int) -> int:
        need = ctypes.c_int64()
        _check(load_library().mf_attn_workspace(self.handle, n, ctypes.byref(need)))
        return need.value

    def status(self, stream=None) -> None:
        """Waits for the stream; raises if a device-side wait of a call timed out."""
        guard, raw = _on(self.device, stream)
        with guard:
            _check(load_library().mf_attn_status(self.handle, raw))

    def close(self) -> None:
        if self.handle is not None:
            h, self.handle = self.handle, None
            _release(0 if self._gpu is None else self._gpu, functools.partial(_destroy_plan, h, self._keep))

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass


class WindowAttention(_AttentionPlan):
    """Attention over packed sequences with an optional sliding window and
    `sinks` first tokens that stay visible; with q_begin, over query chunks
    (see mf_attn_create_packed in mapflow.h).  bf16; no gradient is recorded."""

    def __init__(self, cu_seqlens: Sequence[int], H_q: int, H_kv: int, d: int, window: Optional[int] = None,
                 sinks: int = 0, q_begin: Optional[Sequence[int]] = None, use_torch_allocator: bool = True):
        lib = load_library()
        _release_parked()
        self._call = lib.mf_attn_packed
        window, sinks = 0 if window is None else _span("window", window, 1), _span("sinks", sinks, 0)
        cu = _ints("cu_seqlens", cu_seqlens)
        if cu.ndim != 1 or len(cu) < 2:
            raise MapFlowError(MF_ERR_ARG, "cu_seqlens must hold at least two offsets")
        qb = None if q_begin is None else _ints("q_begin", q_begin)
        if qb is not None and qb.shape != (len(cu) - 1,):
            raise MapFlowError(MF_ERR_ARG, f"q_begin must hold {len(cu) - 1} rows")
        self.H_q, self.H_kv, self.d, self.T = _int("H_q", H_q), _int("H_kv", H_kv), _int("d", d), int(cu[-1])
        a, f = _torch_allocator() if use_torch_allocator else (ALLOC_FN(), FREE_FN())
        self._keep = (a, f)
        h = ctypes.c_void_p()
        _check(lib.mf_attn_create_packed(
            ctypes.byref(h), cu.ctypes.data_as(ctypes.c_void_p),
            None if qb is None else qb.ctypes.data_as(ctypes.c_void_p), len(cu) - 1, self.H_q, self.H_kv, self.d,
            window, sinks, a, f, None))
        self.handle = h
        self._ws_bytes = self._workspace_bytes(1)
        import torch
        self._gpu = torch.cuda.current_device()
        self.device = torch.device("cuda", self._gpu)
        self._scale = self.d ** -0.5

    def attend(self, q, k, v, scale: Optional[float] = None, o=None, lse=None, stream=None):
        """q [T, H_q, d], k and v [T, H_kv, d] -> o [T, H_q, d] (rows before a
        q_begin are left as they are); lse: fp32 [T, H_q] to fill, or None."""
        raw = None if stream is not None else _raw_current(self._gpu)
        if raw is not None:
            return self._attend(raw, q, k, v, scale, o, lse)
        guard, raw = _on(self.device, stream)
        with guard:
            return self._attend(raw, q, k, v, scale, o, lse)

    def _attend(self, raw, q, k, v, scale, o, lse):
        import torch
        dt, gpu = torch.bfloat16, self._gpu
        shape_q, shape_k = (self.T, self.H_q, self.d), (self.T, self.H_kv, self.d)
        ld_q = _rows("q", q, shape_q, dt, gpu)
        ld_k = _rows("k", k, shape_k, dt, gpu)
        ld_v = _rows("v", v, shape_k, dt, gpu)
        if o is None:
            o, ld_o = _empty(q, shape_q), self.H_q * self.d
        else:
            ld_o = _rows("o", o, shape_q, dt, gpu)
        p_lse = p_ws = None
        if lse is not None:
            _vector("lse", lse, shape_q[:2], torch.float32, gpu)
            p_lse = lse.data_ptr()
        if self._ws_bytes:  # a workspace of its own for every call: calls may overlap
            ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=self.device)
            p_ws = ws.data_ptr()
        rc = self._call(
            self.handle, q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v, o.data_ptr(), ld_o, p_lse,
            MF_DTYPE_BF16, self._scale if scale is None else scale, p_ws, self._ws_bytes, raw)
        if rc:
            _check(rc)
        return o


class CacheAttention(_AttentionPlan):
    """Decoding attention of up to n requests with Lq new tokens each over
    their caches of `capacity` rows, with an optional window and sinks, or over
    a prefix of prefix_len tokens that all requests share (see
    mf_attn_create_cache in mapflow.h).  bf16; no gradient is recorded."""

    def __init__(self, n: int, Lq: int, capacity: int, H_q: int, H_kv: int, d: int,
                 window: Optional[int] = None, sinks: int = 0, prefix_len: int = 0,
                 use_torch_allocator: bool = True):
        lib = load_library()
        _release_parked()
        self._call = lib.mf_attn_cached
        window, sinks = 0 if window is None else _span("window", window, 1), _span("sinks", sinks, 0)
        self.n, self.Lq, self.capacity = _int("n", n), _int("Lq", Lq), _int("capacity", capacity)
        self.prefix_len = _int("prefix_len", prefix_len)
        self.H_q, self.H_kv, self.d = _int("H_q", H_q), _int("H_kv", H_kv), _int("d", d)
        a, f = _torch_allocator() if use_torch_allocator else (ALLOC_FN(), FREE_FN())
        self._keep = (a, f)
        h = ctypes.c_void_p()
        _check(lib.mf_attn_create_cache(
            ctypes.byref(h), self.n, self.Lq, self.capacity, self.prefix_len, self.H_q, self.H_kv, self.d,
            window, sinks, a, f, None))
        self.handle = h
        self._ws_of: Dict[int, int] = {}  # workspace bytes by the number of requests
        import torch
        self._gpu = torch.cuda.current_device()
        self.device = torch.device("cuda", self._gpu)
        self._scale = self.d ** -0.5

    def attend(self, q, k_cache, v_cache, lens, k_prefix=None, v_prefix=None, scale: Optional[float] = None,
               o=None, lse=None, stream=None):
        """q [m, Lq, H_q, d] of m <= n requests, k_cache and v_cache [m,
        capacity, H_kv, d], lens int32 [m] on the device (keys in each cache,
        the new tokens' among them), k_prefix and v_prefix [prefix_len, H_kv,
        d] -> o [m, Lq, H_q, d]; lse: fp32 [m, Lq, H_q] to fill, or None."""
        raw = None if stream is not None else _raw_current(self._gpu)
        if raw is not None:
            return self._attend(raw, q, k_cache, v_cache, lens, k_prefix, v_prefix, scale, o, lse)
        guard, raw = _on(self.device, stream)
        with guard:
            return self._attend(raw, q, k_cache, v_cache, lens, k_prefix, v_prefix, scale, o, lse)

    def _attend(self, raw, q, k_cache, v_cache, lens, k_prefix, v_prefix, scale, o, lse):
        import torch
        dt, gpu = torch.bfloat16, self._gpu
        m = q.shape[0]
        shape_q, shape_k = (m, self.Lq, self.H_q, self.d), (m, self.capacity, self.H_kv, self.d)
        ld_q = _rows("q", q, shape_q, dt, gpu)
        ld_k = _rows("k_cache", k_cache, shape_k, dt, gpu)
        ld_v = _rows("v_cache", v_cache, shape_k, dt, gpu)
        _vector("lens", lens, (m,), torch.int32, gpu)
        if o is None:
            o, ld_o = _empty(q, shape_q), self.H_q * self.d
        else:
            ld_o = _rows("o", o, shape_q, dt, gpu)
        p_lse = p_kp = p_vp = None
        if lse is not None:
            _vector("lse", lse, shape_q[:3], torch.float32, gpu)
            p_lse = lse.data_ptr()
        ld_kp = ld_vp = 0
        if self.prefix_len:
            if k_prefix is None or v_prefix is None:
                raise MapFlowError(MF_ERR_ARG, "the plan has a prefix: k_prefix and v_prefix are needed")
            shape_p = (self.prefix_len, self.H_kv, self.d)
            ld_kp = _rows("k_prefix", k_prefix, shape_p, dt, gpu)
            ld_vp = _rows("v_prefix", v_prefix, shape_p, dt, gpu)
            p_kp, p_vp = k_prefix.data_ptr(), v_prefix.data_ptr()
        elif k_prefix is not None or v_prefix is not None:
            raise MapFlowError(MF_ERR_ARG, "the plan has no prefix")
        need = self._ws_of.get(m)
        if need is None:
            need = self._ws_of[m] = self._workspace_bytes(m)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)  # its own for every call: calls may overlap
        rc = self._call(
            self.handle, m, q.data_ptr(), ld_q, k_cache.data_ptr(), ld_k, v_cache.data_ptr(), ld_v, lens.data_ptr(),
            p_kp, ld_kp, p_vp, ld_vp, o.data_ptr(), ld_o, p_lse, MF_DTYPE_BF16,
            self._scale if scale is None else scale, ws.data_ptr(), need, raw)
        if rc:
            _check(rc)
        return o


# ------------------------------------------------------------ paged cache --
MF_CACHE_BF16, MF_CACHE_FP4 = 0, 1


_default_ws: Dict[int, "object"] = {}  # PagedCache.attend's workspace of each GPU's default stream


class PagedCache:
    """A paged cache of one layer's keys and values over tensors of the caller
    (see mf_cache_t in mapflow.h): PagedCache.fp4 for pages of 4 bits,
    PagedCache.bf16 for bf16 rows.  Calls leave no state behind but what they
    write to these tensors (attend keeps the workspace of each GPU's default
    stream, up to 18 MB, for its next call); no gradient is recorded.

    Tokens are named by `seq` and `at`, int32 [T] on the device: a token's row of
    `table` (int32 [n_seqs, max_pages], page numbers) and its place in that
    sequence; tokens with seq = -1 are left out."""

    def __init__(self, fmt: int, page_size: int, H: int, d: int, n_pages: int, tensors, ld_k: int = 0, ld_v: int = 0):
        lib = load_library()
        self._append_call, self._read_call = lib.mf_cache_append_args, lib.mf_cache_read_args
        self._attend_call = lib.mf_attn_paged_args
        self.format, self.page_size, self.H, self.d, self.n_pages = fmt, page_size, H, d, n_pages
        self._tensors = tensors  # kept: the calls read their memory
        k, v, ks, vs = tensors
        self.device, self._gpu = k.device, k.get_device()
        self._struct = CacheStruct(fmt, _int("page_size", page_size), _int("H", H), _int("d", d), n_pages,
                                   k.data_ptr(), _ptr(v), ld_k, ld_v, _ptr(ks), _ptr(vs))
        self._c = ctypes.addressof(self._struct)
        self._scale, self._ld = d ** -0.5, H * d
        import torch
        self._bf16, self._i32, self._f32 = torch.bfloat16, torch.int32, torch.float32
        self._ws_of: Dict[Tuple[int, int], int] = {}  # workspace bytes by Lq and H_q

    @classmethod
    def fp4(cls, pages, page_size: int, d: int, k_scale=None, v_scale=None) -> "PagedCache":
        """pages: uint8 [n_pages, H, page_size / 16 * 18 * d] on a GPU, contiguous
        (any contents until a token is appended); k_scale and v_scale: fp32 [H],
        2^-64 to 2^64, a scale for each head's keys and values (under any other an
        append holds NaN), or None (1)."""
        import torch
        page_size, d = _int("page_size", page_size), _int("d", d)
        if d not in (64, 128) or page_size < 16 or page_size % 16:
            raise MapFlowError(MF_ERR_ARG, f"page_size = {page_size} must be a multiple of 16, d = {d} 64 or 128")
        if pages.dim() != 3:
            raise MapFlowError(MF_ERR_ARG, "pages must be [n_pages, H, page_size / 16 * 18 * d]")
        gpu = pages.get_device()
        if gpu < 0:
            raise MapFlowError(MF_ERR_ARG, f"a CUDA tensor is needed, not one on {pages.device}")
        n, H = pages.shape[:2]
        _vector("pages", pages, (n, H, page_size // 16 * 18 * d), torch.uint8, gpu)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                _vector(name, t, (H,), torch.float32, gpu)
        return cls(MF_CACHE_FP4, page_size, H, d, n, (pages, None, k_scale, v_scale))

    @classmethod
    def bf16(cls, k, v) -> "PagedCache":
        """k and v: bf16 [n_pages, page_size, H, d] on a GPU, tokens equally
        spaced.  With a page to a request these are CacheAttention's caches."""
        import torch
        if k.dim() != 4:
            raise MapFlowError(MF_ERR_ARG, "k and v must be [n_pages, page_size, H, d]")
        gpu = k.get_device()
        if gpu < 0:
            raise MapFlowError(MF_ERR_ARG, f"a CUDA tensor is needed, not one on {k.device}")
        n, page_size, H, d = shape = k.shape
        ld_k, ld_v = _rows("k", k, shape, torch.bfloat16, gpu), _rows("v", v, shape, torch.bfloat16, gpu)
        return cls(MF_CACHE_BF16, page_size, H, d, n, (k, v, None, None), ld_k, ld_v)

    def _table(self, table, rows=None) -> Tuple[int, int, int]:
        """Checks a table; returns the numbers between two of its rows, its rows and
        its columns."""
        if table.dtype is self._i32 and table.get_device() == self._gpu and table.dim() == 2:
            n, m = table.shape
            if rows is None or n == rows:
                if table.is_contiguous():
                    return m, n, m
                if m == 1 or table.stride(1) == 1:
                    return table.stride(0) if n > 1 else m, n, m
        raise MapFlowError(MF_ERR_ARG, f"table must be an int32 tensor [{'n_seqs' if rows is None else rows}, max_pages] "
                                       f"on cuda:{self._gpu} with a row's numbers next to each other")

    # (The calls below are made for every layer of a decoding step: a tensor is looked
    # at in place, by _vector and _rows only to say what is wrong or odd.)
    def append(self, k, v, seq, at, table, rope: Optional["RotaryPlan"] = None, positions=None, k_weight=None,
               eps: float = 1e-6, norm: Optional[bool] = None, stream=None) -> None:
        """Puts k and v (bf16 [T, H, d]) of T tokens in their places, the keys
        normed (when a weight is given or norm is True) and rotated by `rope` at
        `positions` (int32 [T]; None: `at`) on the way (see mf_cache_append)."""
        gpu = self._gpu
        raw = None if stream is not None else _raw_current(gpu)
        if raw is None:
            guard, _ = _on(self.device, stream)
            with guard:
                return self.append(k, v, seq, at, table, rope, positions, k_weight, eps, norm)
        dt, i32 = self._bf16, self._i32
        T = k.shape[0]
        shape, one = (T, self.H, self.d), (T,)
        ld_k = ld_v = self._ld
        if k.dtype is not dt or k.shape != shape or k.get_device() != gpu or not k.is_contiguous():
            ld_k = _rows("k", k, shape, dt, gpu)
        if v.dtype is not dt or v.shape != shape or v.get_device() != gpu or not v.is_contiguous():
            ld_v = _rows("v", v, shape, dt, gpu)
        if seq.dtype is not i32 or seq.shape != one or seq.get_device() != gpu or not seq.is_contiguous():
            _vector("seq", seq, one, i32, gpu)
        if at.dtype is not i32 or at.shape != one or at.get_device() != gpu or not at.is_contiguous():
            _vector("at", at, one, i32, gpu)
        ld_t, n_seqs, max_pages = self._table(table)
        p_pos = p_w = turns = rot = layout = 0
        gain = 1.0
        if positions is not None:
            if positions.dtype is not i32 or positions.shape != one or positions.get_device() != gpu or \
                    not positions.is_contiguous():
                _vector("positions", positions, one, i32, gpu)
            p_pos = positions.data_ptr()
        if rope is not None:
            if rope._gpu != gpu:
                raise MapFlowError(MF_ERR_ARG, f"the cache is on cuda:{gpu}, the rotary plan on {rope.turns.device}")
            if raw != rope._home:
                rope._abroad = True
            turns, rot, layout, gain = rope._turns, rope.rot_dim, rope._layout, rope.gain
        elif positions is not None:
            raise MapFlowError(MF_ERR_ARG, "positions without a rotary plan")
        if k_weight is not None:
            _vector("k_weight", k_weight, (self.d,), dt, gpu)
            p_w = k_weight.data_ptr()
        if norm is None:
            norm = p_w != 0
        rc = self._append_call(_append_args(
            self._c, k.data_ptr(), ld_k, v.data_ptr(), ld_v, seq.data_ptr(), at.data_ptr(), table.data_ptr(), ld_t,
            p_pos, turns, p_w, raw, gain, eps, T, n_seqs, max_pages, rot, layout, norm))
        if rc:
            _check(rc)

    def read(self, seq, at, table, k=None, v=None, stream=None):
        """(k, v): bf16 [T, H, d] of T tokens, new tensors unless given; rows of
        tokens that are left out keep what was there (see mf_cache_read)."""
        gpu = self._gpu
        raw = None if stream is not None else _raw_current(gpu)
        if raw is None:
            guard, _ = _on(self.device, stream)
            with guard:
                return self.read(seq, at, table, k, v)
        dt, i32 = self._bf16, self._i32
        T = seq.shape[0]
        shape, one = (T, self.H, self.d), (T,)
        if seq.dtype is not i32 or seq.shape != one or seq.get_device() != gpu or not seq.is_contiguous():
            _vector("seq", seq, one, i32, gpu)
        if at.dtype is not i32 or at.shape != one or at.get_device() != gpu or not at.is_contiguous():
            _vector("at", at, one, i32, gpu)
        ld_t, n_seqs, max_pages = self._table(table)
        ld_k = ld_v = self._ld
        if k is not None and (k.dtype is not dt or k.shape != shape or k.get_device() != gpu or not k.is_contiguous()):
            ld_k = _rows("k", k, shape, dt, gpu)
        if v is not None and (v.dtype is not dt or v.shape != shape or v.get_device() != gpu or not v.is_contiguous()):
            ld_v = _rows("v", v, shape, dt, gpu)
        if k is None or v is None:
            import torch
            new = torch.zeros((1 + (k is v), *shape), dtype=dt, device=self.device)
            k, v = new[0] if k is None else k, new[-1] if v is None else v
        rc = self._read_call(_read_args(self._c, seq.data_ptr(), at.data_ptr(), table.data_ptr(), ld_t, k.data_ptr(), ld_k,
                                        v.data_ptr(), ld_v, raw, T, n_seqs, max_pages, 0))
        if rc:
            _check(rc)
        return k, v

    def attend(self, q, table, lens, window: Optional[int] = None, sinks: int = 0, softcap: Optional[float] = None,
               slopes=None, scale: Optional[float] = None, o=None, lse=None, stream=None):
        """Decoding attention over a 4-bit cache: q [n, Lq, H_q, d] of n requests,
        table int32 [n, max_pages], lens int32 [n] on the device (keys of each
        request, the new tokens' among them) -> o [n, Lq, H_q, d].  softcap: scores
        are capped by a tanh; slopes: fp32 [H_q], a bias by distance; lse: fp32 [n,
        Lq, H_q] to fill, or None (see mf_attn_paged)."""
        gpu = self._gpu
        raw = None if stream is not None else _raw_current(gpu)
        if raw is None:
            guard, _ = _on(self.device, stream)
            with guard:
                return self.attend(q, table, lens, window, sinks, softcap, slopes, scale, o, lse)
        dt, i32, f32 = self._bf16, self._i32, self._f32
        if q.dim() != 4:
            raise MapFlowError(MF_ERR_ARG, "q must be [n, Lq, H_q, d]")
        n, Lq, H_q, d = shape = q.shape
        if d != self.d:
            raise MapFlowError(MF_ERR_ARG, f"q has heads of {d}, the cache of {self.d}")
        ld_q = ld_o = H_q * d
        if q.dtype is not dt or q.get_device() != gpu or not q.is_contiguous():
            ld_q = _rows("q", q, shape, dt, gpu)
        if lens.dtype is not i32 or lens.shape != (n,) or lens.get_device() != gpu or not lens.is_contiguous():
            _vector("lens", lens, (n,), i32, gpu)
        ld_t, _, max_pages = self._table(table, n)
        window, sinks = 0 if window is None else _span("window", window, 1), _span("sinks", sinks, 0)
        if softcap is None:
            softcap = 0.0
        elif not softcap > 0:
            raise MapFlowError(MF_ERR_ARG, f"softcap = {softcap} must be positive (None: none)")
        if o is None:
            o = _empty(q, shape)
        elif o.dtype is not dt or o.shape != shape or o.get_device() != gpu or not o.is_contiguous():
            ld_o = _rows("o", o, shape, dt, gpu)
        p_lse = p_slopes = 0
        if lse is not None:
            if lse.dtype is not f32 or lse.shape != shape[:3] or lse.get_device() != gpu or not lse.is_contiguous():
                _vector("lse", lse, shape[:3], f32, gpu)
            p_lse = lse.data_ptr()
        if slopes is not None:
            _vector("slopes", slopes, (H_q,), f32, gpu)
            p_slopes = slopes.data_ptr()
        need = self._ws_of.get((Lq, H_q))
        if need is None:
            bytes_ = ctypes.c_int64()
            _check(load_library().mf_attn_paged_workspace(Lq, H_q, self.H, self.d, ctypes.byref(bytes_)))
            need = self._ws_of[Lq, H_q] = bytes_.value
        # The default stream's calls follow each other and are never captured: they
        # share a workspace (beside launches an allocation takes 6 us).  Others may
        # overlap and have their own.
        ws = _default_ws.get(gpu) if raw == 0 else None
        if ws is None or ws.shape[0] < need:
            import torch
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            if raw == 0:
                _default_ws[gpu] = ws
        rc = self._attend_call(_paged_args(
            self._c, q.data_ptr(), ld_q, table.data_ptr(), ld_t, lens.data_ptr(), o.data_ptr(), ld_o, p_lse, p_slopes,
            ws.data_ptr(), need, raw, softcap, self._scale if scale is None else scale, n, Lq, H_q, max_pages, window,
            sinks))
        if rc:
            _check(rc)
        return o


# ------------------------------------------------------ convenience class --
def _destroy_bsr(handle, keep) -> None:
    """Waits for the state's GPU and frees it; `keep` holds its allocator."""
    mf_bsr_destroy(handle)


class BSR:
    """Owner of one mf_bsr_t (compressed sender state of several layers)."""

    handle = None

    def __init__(self, n_layers: int, T: int, H_s: int, B: int, cu_seqlens: Sequence[int],
                 causal: bool = True, use_torch_allocator: bool = True,
                 q_begin: Optional[Sequence[int]] = None):
        _release_parked()
        self.n_layers, self.T, self.H_s, self.B, self.causal = n_layers, T, H_s, B, causal
        self.cu_seqlens = [int(x) for x in cu_seqlens]
        self.q_begin = None if q_begin is None else [int(x) for x in q_begin]
        self.handle, self._keep = mf_bsr_create(n_layers, T, H_s, B, causal, self.cu_seqlens,
                                                use_torch_allocator, self.q_begin)
        import torch
        self._gpu = torch.cuda.current_device()
        self.d: Optional[int] = None

    def compress(self, layer: int, q, k, p: float, stream=None) -> None:
        T, H_s, d = q.shape
        self.d = d
        mf_compress(self.handle, layer, q, k, T, H_s, k.shape[1], d, self.B, p, self.causal,
                    stream)

    def retrieve(self, W, v, o, layer_map: Sequence[int], stream=None) -> None:
        n, T, H_kv, d = v.shape
        H_r = o.shape[2]
        mf_retrieve(self.handle, W, v, o, H_r, H_kv, d, layer_map, stream)

    def set_exact(self, exact: bool) -> None:
        mf_bsr_set_exact(self.handle, exact)

    def info(self, layer: int):
        return mf_bsr_info(self.handle, layer)

    def export(self, layer: int, stream=None) -> Dict[str, "object"]:
        """Copies of the layer's BSR arrays as torch tensors on the device."""
        import torch
        nnz, n_rows, n_cand = self.info(layer)
        dev = torch.device("cuda", torch.cuda.current_device())
        out = {
            "row_ptr": torch.empty(n_rows + 1, dtype=torch.int32, device=dev),
            "col_idx": torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)[:nnz],
            "values": torch.empty((max(nnz, 1), self.B, self.B), dtype=torch.bfloat16,
                                  device=dev)[:nnz],
            "mass": torch.empty(n_cand, dtype=torch.float32, device=dev),
            "row_max": torch.empty((self.H_s, self.T), dtype=torch.float32, device=dev),
            "row_sum": torch.empty((self.H_s, self.T), dtype=torch.float32, device=dev),
        }
        mf_bsr_copy(self.handle, layer, out["row_ptr"], out["col_idx"] if nnz else None,
                    out["values"] if nnz else None, out["mass"], out["row_max"],
                    out["row_sum"], stream)
        return out

    def structure(self, layer: int):
        """(row_ptr, col_idx) of a compressed layer as host numpy arrays."""
        import torch
        nnz, n_rows, _ = self.info(layer)
        dev = torch.device("cuda", torch.cuda.current_device())
        rp = torch.empty(n_rows + 1, dtype=torch.int32, device=dev)
        ci = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
        mf_bsr_copy(self.handle, layer, rp, ci if nnz else None, None, None, None, None, None)
        torch.cuda.synchronize()
        return rp.cpu().numpy(), ci[:nnz].cpu().numpy().astype(np.int64)

    def release_layer(self, layer: int) -> None:
        mf_bsr_release_layer(self.handle, layer)

    def offload(self, layer: int, stream=None) -> None:
        """Move the layer's BSR to pinned host memory (see mf_bsr_offload)."""
        mf_bsr_offload(self.handle, layer, stream)

    def prefetch(self, layer: int, stream=None) -> None:
        """Bring an offloaded layer back to the device on `stream`."""
        mf_bsr_prefetch(self.handle, layer, stream)

    def device_status(self, stream=None) -> None:
        mf_device_status(self.handle, stream)

    def profile(self, enable: bool) -> None:
        mf_profile(self.handle, enable)

    def profile_kinds(self, names) -> None:
        """Time only the named kernel kinds (e.g. ("stats", "pack"))."""
        mf_profile_kinds(self.handle, sum(1 << KERNELS.index(n) for n in names))

    def profile_read(self) -> Dict[str, tuple]:
        """{kernel: (launches, total device ms)} since profiling was enabled."""
        return {name: mf_profile_read(self.handle, i) for i, name in enumerate(KERNELS)}

    def close(self) -> None:
        """Waits for the GPU and frees the state; during a stream capture the
        release is put off to the next one."""
        if self.handle is not None:
            h, self.handle = self.handle, None
            _release(self._gpu, functools.partial(_destroy_bsr, h, self._keep))

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass
