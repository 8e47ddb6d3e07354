"""FP8 paged-KV decode attention for GB300 (sm_103a).

Thin Python binding over the C ABI in ``include/fkv.h`` (``libfkv.so``, built
in-tree by ``_build.py``).  Every function here only checks tensor metadata and
passes raw device pointers, sizes and the current CUDA stream to the library;
all computation runs in the library's CUDA kernels.  There is no CPU path: if
the library is missing or no GPU is present the calls raise.  The calls that a
decode step makes with a 4-bit cache, and ``paged_decode_attn``, are marshalled
by the ``_fkv_bind`` module (host C++, ``csrc/bind.cpp``, built for one torch
version): in Python their checks took 4 to 9 us a call, more than some of the
kernels.  Without it ``paged_decode_attn`` and the calls that do not use it
still run.

Entry points (same names as the C ABI):
  kv_append_fp8 / kv_append_bf16   write new tokens into the paged pools
  kv_calibrate_scales              per-KV-head FP8 scales of a prompt (bulk write)
  kv_page_tag_check                the separate per-page generation-tag check
  kv_append_fp8_tag_check          the step's FP8 append and the tag check in one launch
  kv_append_bf16_tag_check         the same for a BF16 cache
  kv_append_fp4                    the same into a 4-bit cache (also kv_append_fp4_tag_check)
  kv_gather                        cached tokens read back as bf16
  qk_norm_rope                     RMS norm of the q and k heads and the position rotation in one pass
  kv_step_tables                   page table, slots and positions of a step from request lengths
  kv_page_realloc                  bump tags (and optionally zero pages) of reallocated pages
  paged_decode_attn                decode attention over the paged cache
  paged_decode_attn_workspace_size bytes of scratch paged_decode_attn needs
  kv_append_rope                   qk_norm_rope and the append of a step's keys and values in one pass
  paged_tree_attn                  attention of every request's tree of drafted tokens over the paged cache
  paged_window_attn                decode attention over a sliding window and a few first tokens
  kv_tree_commit                   the accepted drafted tokens' rows moved into place, left-over pages given back
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "FkvError", "KV_FP8_E4M3", "KV_BF16", "KV_FP4", "FP4_ROW_BYTES", "library_path", "load_library", "kv_append_fp8", "kv_append_bf16",
    "kv_calibrate_scales", "kv_page_tag_check", "kv_append_fp8_tag_check", "kv_append_bf16_tag_check", "kv_page_realloc",
    "kv_append_fp4", "kv_append_fp4_tag_check", "kv_gather", "qk_norm_rope", "kv_step_tables",
    "kv_step_tables_workspace_size", "alloc_step_tables_workspace",
    "paged_decode_attn",
    "paged_decode_attn_workspace_size",
    "alloc_workspace",
    "paged_decode_attn_noalloc",
    "kv_append_rope", "paged_tree_attn", "paged_tree_attn_workspace_size", "alloc_tree_workspace", "paged_window_attn",
    "kv_tree_commit",
    "device_error", "kernels_per_call", "selftest_wait", "EXPORTED_SYMBOLS",
]

KV_FP8_E4M3 = 0
KV_BF16 = 1
KV_FP4 = 2
FP4_ROW_BYTES = 72
DEVERR_APPEND_SLOT = 0x1
DEVERR_ATTN_PAGE = 0x2
DEVERR_TIMEOUT = 0x4
DEVERR_REALLOC_PAGE = 0x8
DEVERR_GATHER_SLOT = 0x10
DEVERR_TABLES = 0x20
DEVERR_ROPE_AXIS = 0x40
DEVERR_TREE = 0x80
HEAD_DIM = 128

EXPORTED_SYMBOLS = (
    "fkv_status_string", "kv_append_fp8", "kv_append_bf16", "kv_calibrate_scales", "kv_page_tag_check",
    "kv_append_fp8_tag_check", "kv_append_bf16_tag_check", "kv_page_realloc",
    "paged_decode_attn_workspace_size", "paged_decode_attn", "paged_decode_attn_noalloc", "fkv_device_error",
    "fkv_kernels_per_call", "fkv_selftest_wait",
    "kv_append_fp4", "kv_append_fp4_tag_check", "kv_gather", "qk_norm_rope", "kv_step_tables",
    "kv_step_tables_workspace_size",
    "kv_append_rope", "paged_tree_attn_workspace_size", "paged_tree_attn", "paged_window_attn", "kv_tree_commit",
)
ERR_SCRATCH_LIMIT = 4
NOALLOC_SCRATCH_BYTES = 16 << 20

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None
_bind = None      # the compiled marshalling, once loaded
_BIND_CALLS = ("fkv_status_string", "kv_append_fp4", "kv_append_fp4_tag_check", "kv_gather", "qk_norm_rope", "kv_step_tables",
               "paged_decode_attn", "kv_append_rope", "paged_tree_attn", "paged_window_attn",
               "kv_tree_commit")         # the entry points that it calls, in the order its setup takes them


class FkvError(RuntimeError):
    pass


def library_path() -> str:
    """The in-tree libfkv.so (``FKV_LIBRARY_PATH`` points at another build,
    e.g. a variant compiled with different options)."""
    return os.environ.get("FKV_LIBRARY_PATH") or os.path.join(_HERE, "libfkv.so")


def load_library():
    """Load libfkv.so (raises if it has not been built)."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise FkvError("libfkv.so is not built; run fp8_paged_kv_decode_gb300._build.build()")
        lib = ctypes.CDLL(path)
        P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        lib.fkv_status_string.restype = ctypes.c_char_p
        lib.fkv_status_string.argtypes = [ctypes.c_int]
        lib.kv_append_fp8.restype = ctypes.c_int
        lib.kv_append_fp8.argtypes = [P, P, P, i32, P, P, P, P, i32, i32, i32, i32, P]
        lib.kv_append_bf16.restype = ctypes.c_int
        lib.kv_append_bf16.argtypes = [P, P, P, i32, P, P, i32, i32, i32, i32, P]
        lib.kv_page_tag_check.restype = ctypes.c_int
        lib.kv_page_tag_check.argtypes = [P, i32, P, P, P, i32, i64, P, P]
        lib.kv_append_fp8_tag_check.restype = ctypes.c_int
        lib.kv_append_fp8_tag_check.argtypes = [P, P, P, i32, P, P, P, P, i32, i32, i32, i32, P, P, P, P, i32, i64,
                                                P, P]
        lib.kv_append_bf16_tag_check.restype = ctypes.c_int
        lib.kv_append_bf16_tag_check.argtypes = [P, P, P, i32, P, P, i32, i32, i32, i32, P, P, P, P, i32, i64, P, P]
        lib.kv_append_fp4.restype = ctypes.c_int
        lib.kv_append_fp4.argtypes = lib.kv_append_fp8.argtypes
        lib.kv_append_fp4_tag_check.restype = ctypes.c_int
        lib.kv_append_fp4_tag_check.argtypes = lib.kv_append_fp8_tag_check.argtypes
        lib.kv_gather.restype = ctypes.c_int
        lib.kv_gather.argtypes = [P, P, i32, P, P, P, i32, P, P, i32, i32, i32, i32, P]
        lib.qk_norm_rope.restype = ctypes.c_int
        lib.qk_norm_rope.argtypes = [P, i64, i32, P, i64, i32, P, i64, P, i64, i32, P, P, f32, P, i32, P, P, i32, i32,
                                     f32, i32, P]
        lib.kv_step_tables_workspace_size.restype = ctypes.c_size_t
        lib.kv_step_tables_workspace_size.argtypes = [i32]
        lib.kv_step_tables.restype = ctypes.c_int
        lib.kv_step_tables.argtypes = [P, P, i32, P, P, i32, P, i32, P, P, i32, i32, P, P, P, P, P, P, i32, P, P, P,
                                       i32, P, P, ctypes.c_size_t, P]
        lib.kv_calibrate_scales.restype = ctypes.c_int
        lib.kv_calibrate_scales.argtypes = [P, P, i64, i32, i32, P, P, P]
        lib.kv_page_realloc.restype = ctypes.c_int
        lib.kv_page_realloc.argtypes = [P, i32, P, i32, P, P, P, i32, i32, i32, i32, P]
        lib.paged_decode_attn_workspace_size.restype = ctypes.c_size_t
        lib.paged_decode_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.paged_decode_attn.restype = ctypes.c_int
        lib.paged_decode_attn.argtypes = [P, i32, i32, P, P, i32, P, P, i32, i32, i32, i32, P, P, i64, P, P, f32,
                                          P, P, ctypes.c_size_t, P]
        lib.paged_decode_attn_noalloc.restype = ctypes.c_int
        lib.paged_decode_attn_noalloc.argtypes = [P, i32, i32, P, P, i32, P, P, i32, i32, i32, i32, P, P, i64, P, P,
                                                  f32, P, P]
        lib.kv_append_rope.restype = ctypes.c_int
        lib.kv_append_rope.argtypes = [P, i64, i32, P, i64, P, i64, i32, P, i64, i32, P, P, f32, P, i32, P, P, i32, i32, f32, P,
                                       i32, P, P, P, P, i32, i32, i32, P]
        lib.paged_tree_attn_workspace_size.restype = ctypes.c_size_t
        lib.paged_tree_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.paged_tree_attn.restype = ctypes.c_int
        lib.paged_tree_attn.argtypes = [P, i32, i32, P, P, i32, P, P, i32, i32, i32, i32, P, P, i64, P, i32, P, P, i32, i32, i32,
                                        P, f32, P, P, ctypes.c_size_t, P]
        lib.paged_window_attn.restype = ctypes.c_int
        lib.paged_window_attn.argtypes = [P, i32, i32, P, P, i32, P, P, i32, i32, i32, i32, P, P, i64, P, i32, i32, P, f32, P, P,
                                          ctypes.c_size_t, P]
        lib.kv_tree_commit.restype = ctypes.c_int
        lib.kv_tree_commit.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, i64, P, i32, P, i32, P, i32, P, P, P, P, i32, P, P, P,
                                       P]
        lib.fkv_device_error.restype = ctypes.c_int
        lib.fkv_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
        lib.fkv_kernels_per_call.restype = i32
        lib.fkv_kernels_per_call.argtypes = [ctypes.c_char_p]
        lib.fkv_selftest_wait.restype = ctypes.c_int
        lib.fkv_selftest_wait.argtypes = [ctypes.c_uint64, i32, P, P]
        _lib = lib
        return lib


def _load_bind(needed=True):
    """Load the marshalling module for this torch and give it the library's
    entry points.  Where it has not been built: an error, or None (not needed)."""
    global _bind
    lib = load_library()
    with _lock:
        if _bind is None:
            import importlib.machinery
            import importlib.util

            import torch  # noqa: F401  (its libraries, which the module links against)

            from . import _build
            path = _build.bind_path()
            if not os.path.exists(path):
                if not needed:
                    return None
                raise FkvError("%s is not built; run fp8_paged_kv_decode_gb300._build.build()" % os.path.basename(path))
            loader = importlib.machinery.ExtensionFileLoader("_fkv_bind", path)
            mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fkv_bind", loader))
            loader.exec_module(mod)
            mod.setup(FkvError, *(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in _BIND_CALLS))
            _bind = mod
        return _bind


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _ptr(t):
    # plain integers: the entry points' argtypes convert them to void *
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        # the raw handle of the current stream: torch.cuda.current_stream() builds a
        # Stream object for it, 5 us a call on the host of a GB300
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(cond, msg):
    if not cond:
        raise FkvError(msg)


def _dev(*ts):
    for t in ts:
        if t is not None:
            _need(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")


def _raise(status: int, name: str):
    if status != 0:
        msg = load_library().fkv_status_string(status).decode()
        raise FkvError("%s failed: %s (status %d)" % (name, msg, status))


def _is_byte_cache(t):
    import torch
    return t.dtype in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))


def _is_fp4_cache(t):
    import torch
    return t.dtype is torch.uint8 and t.shape[-1] == FP4_ROW_BYTES and t.dim() == 4


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def kv_append_fp8(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, stream=None):
    """Quantize bf16 ``k_new/v_new`` [N][Hkv][128] to e4m3 into ``k_cache/v_cache``
    [P][Hkv][S][128] (uint8) at ``slot_mapping`` [N] (int64, <0 = skip)."""
    import torch
    _dev(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache)
    _need(k_new.dtype == torch.bfloat16 and v_new.dtype == torch.bfloat16, "k_new/v_new must be bf16")
    _need(slot_mapping.dtype == torch.int64, "slot_mapping must be int64")
    _need(k_scale.dtype == torch.float32 and v_scale.dtype == torch.float32, "scales must be float32")
    _need(_is_byte_cache(k_cache) and _is_byte_cache(v_cache), "FP8 caches must be uint8/float8_e4m3fn")
    P, Hkv, S, D = k_cache.shape
    _need(tuple(v_cache.shape) == (P, Hkv, S, D), "k_cache/v_cache shapes differ")
    N = slot_mapping.numel()
    _need(tuple(k_new.shape) == (N, Hkv, D) and tuple(v_new.shape) == (N, Hkv, D), "k_new/v_new shape")
    _raise(load_library().kv_append_fp8(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), N, _ptr(k_scale),
                                        _ptr(v_scale), _ptr(k_cache), _ptr(v_cache), P, Hkv, S, D,
                                        _stream(stream)), "kv_append_fp8")


def kv_append_bf16(k_new, v_new, slot_mapping, k_cache, v_cache, stream=None):
    """BF16-cache counterpart of ``kv_append_fp8`` (values stored unchanged)."""
    import torch
    _dev(k_new, v_new, slot_mapping, k_cache, v_cache)
    _need(k_new.dtype == torch.bfloat16 and k_cache.dtype == torch.bfloat16, "bf16 tensors expected")
    P, Hkv, S, D = k_cache.shape
    N = slot_mapping.numel()
    _need(tuple(k_new.shape) == (N, Hkv, D) and tuple(v_new.shape) == (N, Hkv, D), "k_new/v_new shape")
    _raise(load_library().kv_append_bf16(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), N, _ptr(k_cache),
                                         _ptr(v_cache), P, Hkv, S, D, _stream(stream)), "kv_append_bf16")


def kv_page_tag_check(page_tags, page_indptr, page_indices, expected_tags, abort_mask, stream=None):
    """abort_mask[r] = 1 iff a page request r expects has a different live tag
    (or is outside the pool).  All tensors on the GPU; the mask stays there."""
    import torch
    _dev(page_tags, page_indptr, page_indices, expected_tags, abort_mask)
    _need(page_tags.dtype == torch.uint32 or page_tags.dtype == torch.int32, "page_tags must be 32-bit")
    _need(expected_tags.dtype == page_tags.dtype, "expected_tags dtype must match page_tags")
    _need(page_indptr.dtype == torch.int32 and page_indices.dtype == torch.int32, "CSR must be int32")
    _need(abort_mask.dtype == torch.uint8, "abort_mask must be uint8")
    B = page_indptr.numel() - 1
    _need(abort_mask.numel() == B and expected_tags.numel() == page_indices.numel(), "size mismatch")
    _raise(load_library().kv_page_tag_check(_ptr(page_tags), page_tags.numel(), _ptr(page_indptr),
                                            _ptr(page_indices), _ptr(expected_tags), B, page_indices.numel(),
                                            _ptr(abort_mask), _stream(stream)), "kv_page_tag_check")


def kv_append_fp8_tag_check(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache,
                            page_tags, page_indptr, page_indices, expected_tags, abort_mask, stream=None):
    """``kv_append_fp8`` then ``kv_page_tag_check`` (same arguments, same
    results) in one launch; ``page_tags`` has one entry per page of the pool."""
    import torch
    _dev(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, page_tags, page_indptr, page_indices,
         expected_tags, abort_mask)
    _need(k_new.dtype == torch.bfloat16 and v_new.dtype == torch.bfloat16, "k_new/v_new must be bf16")
    _need(slot_mapping.dtype == torch.int64, "slot_mapping must be int64")
    _need(k_scale.dtype == torch.float32 and v_scale.dtype == torch.float32, "scales must be float32")
    _need(_is_byte_cache(k_cache) and _is_byte_cache(v_cache), "FP8 caches must be uint8/float8_e4m3fn")
    P, Hkv, S, D = k_cache.shape
    _need(tuple(v_cache.shape) == (P, Hkv, S, D), "k_cache/v_cache shapes differ")
    N = slot_mapping.numel()
    _need(tuple(k_new.shape) == (N, Hkv, D) and tuple(v_new.shape) == (N, Hkv, D), "k_new/v_new shape")
    _need(page_tags.dtype in (torch.uint32, torch.int32) and expected_tags.dtype == page_tags.dtype,
          "tags must be 32-bit, both of one dtype")
    _need(page_tags.numel() == P, "page_tags must have one entry per page of the pool")
    _need(page_indptr.dtype == torch.int32 and page_indices.dtype == torch.int32, "CSR must be int32")
    _need(abort_mask.dtype == torch.uint8, "abort_mask must be uint8")
    B = page_indptr.numel() - 1
    _need(abort_mask.numel() == B and expected_tags.numel() == page_indices.numel(), "size mismatch")
    _raise(load_library().kv_append_fp8_tag_check(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), N, _ptr(k_scale), _ptr(v_scale), _ptr(k_cache),
        _ptr(v_cache), P, Hkv, S, D, _ptr(page_tags), _ptr(page_indptr), _ptr(page_indices), _ptr(expected_tags),
        B, page_indices.numel(), _ptr(abort_mask), _stream(stream)), "kv_append_fp8_tag_check")


def kv_append_bf16_tag_check(k_new, v_new, slot_mapping, k_cache, v_cache,
                             page_tags, page_indptr, page_indices, expected_tags, abort_mask, stream=None):
    """``kv_append_bf16`` then ``kv_page_tag_check`` (same arguments, same
    results) in one launch; ``page_tags`` has one entry per page of the pool."""
    import torch
    _dev(k_new, v_new, slot_mapping, k_cache, v_cache, page_tags, page_indptr, page_indices, expected_tags,
         abort_mask)
    _need(k_new.dtype == torch.bfloat16 and v_new.dtype == torch.bfloat16, "k_new/v_new must be bf16")
    _need(k_cache.dtype == torch.bfloat16 and v_cache.dtype == torch.bfloat16, "BF16 caches expected")
    _need(slot_mapping.dtype == torch.int64, "slot_mapping must be int64")
    P, Hkv, S, D = k_cache.shape
    _need(tuple(v_cache.shape) == (P, Hkv, S, D), "k_cache/v_cache shapes differ")
    N = slot_mapping.numel()
    _need(tuple(k_new.shape) == (N, Hkv, D) and tuple(v_new.shape) == (N, Hkv, D), "k_new/v_new shape")
    _need(page_tags.dtype in (torch.uint32, torch.int32) and expected_tags.dtype == page_tags.dtype,
          "tags must be 32-bit, both of one dtype")
    _need(page_tags.numel() == P, "page_tags must have one entry per page of the pool")
    _need(page_indptr.dtype == torch.int32 and page_indices.dtype == torch.int32, "CSR must be int32")
    _need(abort_mask.dtype == torch.uint8, "abort_mask must be uint8")
    B = page_indptr.numel() - 1
    _need(abort_mask.numel() == B and expected_tags.numel() == page_indices.numel(), "size mismatch")
    _raise(load_library().kv_append_bf16_tag_check(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), N, _ptr(k_cache), _ptr(v_cache), P, Hkv, S, D,
        _ptr(page_tags), _ptr(page_indptr), _ptr(page_indices), _ptr(expected_tags), B, page_indices.numel(),
        _ptr(abort_mask), _stream(stream)), "kv_append_bf16_tag_check")


def kv_calibrate_scales(k, v, k_scale, v_scale, stream=None):
    """Per-KV-head scales fl32(amax / 448) of a prompt's bf16 K/V [N][Hkv][128]
    (1 for an all-zero head), written into ``k_scale``/``v_scale`` (fp32 [Hkv])."""
    import torch
    _dev(k, v, k_scale, v_scale)
    _need(k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16, "k/v must be bf16")
    _need(k_scale.dtype == torch.float32 and v_scale.dtype == torch.float32, "scales must be float32")
    N, Hkv, D = k.shape
    _need(tuple(v.shape) == (N, Hkv, D) and k_scale.numel() == Hkv and v_scale.numel() == Hkv, "shape mismatch")
    _raise(load_library().kv_calibrate_scales(_ptr(k), _ptr(v), N, Hkv, D, _ptr(k_scale), _ptr(v_scale),
                                              _stream(stream)), "kv_calibrate_scales")


def kv_append_fp4(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, stream=None):
    """Quantize bf16 ``k_new/v_new`` [N][Hkv][128] to e2m1 codes with an e4m3
    scale per 16 dims into ``k_cache/v_cache`` [P][Hkv][S][72] (uint8) at
    ``slot_mapping`` [N] (int64, <0 = skip).  The per-head fp32 scales are the
    ones an FP8 cache would use (``kv_calibrate_scales``)."""
    (_bind or _load_bind()).kv_append_fp4(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, stream)


def kv_append_fp4_tag_check(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache,
                            page_tags, page_indptr, page_indices, expected_tags, abort_mask, stream=None):
    """``kv_append_fp4`` then ``kv_page_tag_check`` (same arguments, same
    results) in one launch; ``page_tags`` has one entry per page of the pool."""
    (_bind or _load_bind()).kv_append_fp4_tag_check(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache,
                                                    page_tags, page_indptr, page_indices, expected_tags, abort_mask,
                                                    stream)


def kv_gather(k_cache, v_cache, slots, k_out, v_out, k_scale=None, v_scale=None, stream=None):
    """Cached tokens at ``slots`` [N] (int64; <0 gives zeros) as bf16
    ``k_out/v_out`` [N][Hkv][128].  Caches: FP8 uint8 / float8_e4m3fn or bf16
    [P][Hkv][S][128], or FP4 uint8 [P][Hkv][S][72]; scales fp32 [Hkv] unless bf16."""
    (_bind or _load_bind()).kv_gather(k_cache, v_cache, slots, k_out, v_out, k_scale, v_scale, stream)


def qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, axis_map=None,
                 interleaved=False, rot_scale=1.0, stream=None):
    """RMS norm of every head of ``q`` [N][Hq][128] and ``k`` [N][Hkv][128]
    (bf16; heads contiguous, any token stride that is a multiple of 8) with
    bf16 weights [128] (None: no norm), then the rotation by ``positions``
    (int32 [N], or [axes][N] with ``axis_map`` uint8 [R/2]) at fp32
    ``inv_freq`` [R/2], R <= 128 a multiple of 16; pairs are (j, j + R/2), or
    (2j, 2j + 1) when ``interleaved``.  ``q_out``/``k_out`` may be q/k.
    ``k`` and ``k_out`` may be None."""
    (_bind or _load_bind()).qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_weight, k_weight, eps, axis_map,
                                         interleaved, rot_scale, stream)
    return q_out, k_out


def kv_step_tables_workspace_size(batch):
    n = load_library().kv_step_tables_workspace_size(batch)
    _need(n > 0, "batch must not be negative")
    return int(n)


def alloc_step_tables_workspace(batch, device="cuda"):
    import torch
    return torch.empty(kv_step_tables_workspace_size(batch), dtype=torch.uint8, device=device)


def kv_step_tables(cached_lens, new_lens, block_table, block_tags, free_pages, free_count, page_tags, page_size,
                   step_lens, cached_lens_out, refused, page_indptr, page_indices, expected_tags, token_indptr,
                   slot_mapping, positions, free_left, workspace, stream=None):
    """The tables of a step from the requests' lengths, pages taken from a free
    list where a request grows into them (``block_table``/``block_tags``
    [B][max_blocks] updated in place).  int32 throughout, but slot_mapping int64,
    refused uint8 and tags 32-bit; the capacities are the arrays' lengths.  For
    the next step pass ``cached_lens_out`` as ``cached_lens`` and ``free_left``
    as ``free_count`` (each may also be the same array in one call)."""
    (_bind or _load_bind()).kv_step_tables(
        cached_lens, new_lens, block_table, block_tags, free_pages, free_count, page_tags, page_size, step_lens,
        cached_lens_out, refused, page_indptr, page_indices, expected_tags, token_indptr, slot_mapping, positions,
        free_left, workspace, stream)


def kv_page_realloc(page_tags, pages, new_tags, k_cache=None, v_cache=None, stream=None):
    """Bump the live tag of each listed page (new owners record ``new_tags``)
    and, if the pools are given, zero those pages."""
    import torch
    _dev(page_tags, pages, new_tags, k_cache, v_cache)
    _need(page_tags.dtype in (torch.int32, torch.uint32) and new_tags.dtype == page_tags.dtype, "32-bit tags")
    _need(pages.dtype == torch.int32 and new_tags.numel() == pages.numel(), "pages int32, one new tag each")
    _need(k_cache is not None or v_cache is None, "both pools, or neither")
    if k_cache is not None:
        _need(v_cache is not None and tuple(k_cache.shape) == tuple(v_cache.shape), "both pools, same shape")
        _need(k_cache.dtype == v_cache.dtype or (_is_byte_cache(k_cache) and _is_byte_cache(v_cache)), "pools of one type")
        P, Hkv, S, D = k_cache.shape
        _need(P >= page_tags.numel(), "the pools must have every page that has a tag")
        if _is_fp4_cache(k_cache):
            D, kv = HEAD_DIM, KV_FP4
        else:
            _need(_is_byte_cache(k_cache) or k_cache.dtype == torch.bfloat16, "pools must be uint8 (e4m3, or FP4 rows of 72) or bf16")
            kv = KV_FP8_E4M3 if _is_byte_cache(k_cache) else KV_BF16
    else:
        Hkv = S = 0
        D, kv = HEAD_DIM, KV_FP8_E4M3
    _raise(load_library().kv_page_realloc(_ptr(page_tags), page_tags.numel(), _ptr(pages), pages.numel(),
                                          _ptr(new_tags), _ptr(k_cache), _ptr(v_cache), kv, Hkv, S, D,
                                          _stream(stream)), "kv_page_realloc")


def paged_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim=HEAD_DIM, kv_dtype=KV_FP8_E4M3):
    n = load_library().paged_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, kv_dtype)
    _need(n > 0 or batch == 0, "unsupported shape for paged_decode_attn")
    return int(n)


def alloc_workspace(batch, num_q_heads, num_kv_heads, kv_dtype=KV_FP8_E4M3, device="cuda"):
    import torch
    n = paged_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, HEAD_DIM, kv_dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def paged_decode_attn(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out, workspace,
                      k_scale=None, v_scale=None, abort_mask=None, stream=None):
    """out[r][i] = softmax(sm_scale q k^T) v over request r's paged tokens.

    q, out: bf16 [B][Hq][128]; caches [P][Hkv][S][128] uint8 (FP8 e4m3, with
    k_scale/v_scale fp32 [Hkv]) or bf16, or [P][Hkv][S][72] uint8 (FP4, with
    the same scales; workspace for KV_FP4); CSR page table int32; seq_lens int32
    [B]; abort_mask uint8 [B] or None (no tracker)."""
    bind = _bind or _load_bind(needed=False)
    if bind is not None:
        bind.paged_decode_attn(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out, workspace, k_scale,
                               v_scale, abort_mask, stream)
    else:               # not built for this torch: the library alone serves the call, at more host time
        _dev(workspace)
        _raise(load_library().paged_decode_attn(
            *_attn_args(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out, k_scale, v_scale, abort_mask),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)), "paged_decode_attn")
    return out


def _attn_args(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out, k_scale, v_scale, abort_mask):
    """The checked C arguments of decode attention, up to ``out``."""
    import torch
    _dev(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, out, k_scale, v_scale, abort_mask)
    _need(q.dim() == 3 and k_cache.dim() == 4 and k_cache.shape == v_cache.shape, "q [B][Hq][128], caches of one shape")
    B, Hq, D = q.shape
    P, Hkv, S, row = k_cache.shape
    if _is_fp4_cache(k_cache) and _is_fp4_cache(v_cache):
        kv, row = KV_FP4, HEAD_DIM
    elif k_cache.dtype == torch.bfloat16:
        _need(v_cache.dtype == torch.bfloat16, "k_cache and v_cache types differ")
        kv = KV_BF16
    else:
        _need(_is_byte_cache(k_cache) and _is_byte_cache(v_cache), "cache must be uint8 (e4m3, or FP4 rows of 72) or bf16")
        kv = KV_FP8_E4M3
    if kv == KV_BF16:
        k_scale = v_scale = None
    else:
        for s in (k_scale, v_scale):
            _need(s is not None and s.dtype == torch.float32 and s.numel() >= Hkv, "scales must be float32 [Hkv]")
    _need(q.dtype == torch.bfloat16 and out.dtype == torch.bfloat16, "q/out must be bf16")
    _need(page_indptr.dtype in (torch.int32, torch.uint32) and page_indices.dtype in (torch.int32, torch.uint32), "CSR must be int32")
    _need(seq_lens.dtype == torch.int32 and seq_lens.numel() >= B, "seq_lens must be int32 [B]")
    _need(abort_mask is None or (abort_mask.dtype == torch.uint8 and abort_mask.numel() >= B), "abort_mask must be uint8 [B]")
    _need(tuple(out.shape) == (B, Hq, D) and row == D and page_indptr.numel() == B + 1, "shape mismatch")
    return (_ptr(q), B, Hq, _ptr(k_cache), _ptr(v_cache), kv, _ptr(k_scale), _ptr(v_scale), P, Hkv, S, D, _ptr(page_indptr),
            _ptr(page_indices), page_indices.numel(), _ptr(seq_lens), _ptr(abort_mask), float(sm_scale), _ptr(out))


def paged_decode_attn_noalloc(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out,
                              k_scale=None, v_scale=None, abort_mask=None, stream=None):
    """``paged_decode_attn`` without a workspace argument, for callers that
    cannot allocate device memory: its scratch is a fixed array of
    ``NOALLOC_SCRATCH_BYTES`` inside the library (shared by all calls on a
    device, so calls must not overlap on the GPU).  Shapes needing more
    scratch raise FkvError (status ERR_SCRATCH_LIMIT)."""
    _raise(load_library().paged_decode_attn_noalloc(
        *_attn_args(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out, k_scale, v_scale, abort_mask),
        _stream(stream)), "paged_decode_attn_noalloc")
    return out


def kv_append_rope(q, k, v, positions, inv_freq, slot_mapping, q_out, k_cache, v_cache, k_scale=None, v_scale=None,
                   q_weight=None, k_weight=None, eps=1e-6, axis_map=None, interleaved=False, rot_scale=1.0, stream=None):
    """``qk_norm_rope`` of ``q`` [N][Hq][128] (into ``q_out``) and ``k``, with ``k``
    and ``v`` [N][Hkv][128] going into the cache at ``slot_mapping`` [N] (int64, <0 =
    skip) in the same pass; the keys are rounded once.  q, k and v are bf16, heads
    contiguous, any token stride that is a multiple of 8.  Caches: FP8 uint8 /
    float8_e4m3fn or bf16 [P][Hkv][S][128], or FP4 uint8 [P][Hkv][S][72]; scales fp32
    [Hkv] unless bf16.  ``q_out`` may be q; ``q`` and ``q_out`` may be None."""
    (_bind or _load_bind()).kv_append_rope(q, k, v, positions, inv_freq, slot_mapping, q_out, k_cache, v_cache, k_scale, v_scale,
                                           q_weight, k_weight, eps, axis_map, interleaved, rot_scale, stream)
    return q_out


def paged_tree_attn_workspace_size(n_tokens, batch, num_q_heads, num_kv_heads, head_dim=HEAD_DIM, kv_dtype=KV_FP8_E4M3):
    n = load_library().paged_tree_attn_workspace_size(n_tokens, batch, num_q_heads, num_kv_heads, head_dim, kv_dtype)
    _need(n > 0, "unsupported shape for paged_tree_attn")
    return int(n)


def alloc_tree_workspace(n_tokens, batch, num_q_heads, num_kv_heads, kv_dtype=KV_FP8_E4M3, device="cuda"):
    """Scratch for ``paged_tree_attn`` of n_tokens drafted tokens, or ``paged_window_attn`` (n_tokens = batch)."""
    import torch
    n = paged_tree_attn_workspace_size(n_tokens, batch, num_q_heads, num_kv_heads, HEAD_DIM, kv_dtype)
    return torch.empty(n, dtype=torch.uint8, device=device)


def paged_tree_attn(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, token_indptr, tree_mask, sm_scale, out, workspace,
                    k_scale=None, v_scale=None, abort_mask=None, window=0, sinks=0, stream=None):
    """Attention of drafted tokens: rows ``token_indptr[r]`` .. of ``q``/``out`` [N][Hq][128] are
    request r's, whose drafted tokens are the last of its ``seq_lens[r]`` cached ones.  A row sees the
    committed tokens before them (with ``window``: those less than that far behind its own depth, and
    the first ``sinks``) and drafted token j if bit j of its ``tree_mask`` (int64 or uint64 [N] or
    [N][words], up to 4 words) is set, whatever the window.  The other arguments are ``paged_decode_attn``'s;
    workspace from ``alloc_tree_workspace``."""
    (_bind or _load_bind()).paged_tree_attn(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, token_indptr, tree_mask,
                                            sm_scale, out, workspace, k_scale, v_scale, abort_mask, window, sinks, stream)
    return out


def paged_window_attn(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out, workspace, window, sinks=0,
                      k_scale=None, v_scale=None, abort_mask=None, stream=None):
    """``paged_decode_attn`` over each request's last ``window`` tokens and its first ``sinks``;
    workspace from ``alloc_tree_workspace(B, B, ...)``."""
    (_bind or _load_bind()).paged_window_attn(q, k_cache, v_cache, page_indptr, page_indices, seq_lens, sm_scale, out, workspace,
                                              k_scale, v_scale, abort_mask, window, sinks, stream)
    return out


def kv_tree_commit(k_cache, v_cache, page_indptr, page_indices, seq_lens, token_indptr, accepted, accepted_counts, lens_out,
                   abort_mask=None, free_pages=None, free_count=None, free_left=None, page_tags=None, stream=None):
    """Moves the cache rows of each request's accepted drafted tokens (``accepted`` int32 [B][max],
    strictly increasing indices, ``accepted_counts`` [B]) behind its committed ones and writes the kept
    lengths to ``lens_out``.  With ``free_pages``, ``free_count`` and ``free_left`` (which may be
    free_count) the pages past them go back onto ``kv_step_tables``' free list, their ``page_tags``
    bumped where given.  Requests that are aborted or not valid are left as they are."""
    (_bind or _load_bind()).kv_tree_commit(k_cache, v_cache, page_indptr, page_indices, seq_lens, token_indptr, accepted,
                                           accepted_counts, lens_out, abort_mask, free_pages, free_count, free_left, page_tags,
                                           stream)


def device_error(clear: bool = True) -> int:
    """Sticky device error word of the current device (synchronises)."""
    v = ctypes.c_uint32(0)
    _raise(load_library().fkv_device_error(ctypes.byref(v), 1 if clear else 0), "fkv_device_error")
    return int(v.value)


def kernels_per_call(entry_point: str) -> int:
    return int(load_library().fkv_kernels_per_call(entry_point.encode()))


def selftest_wait(limit_ns: int, complete: bool = False, result=None, stream=None):
    """Run the failure path of the kernels' bounded waits on the GPU: one
    block waits, with the library's three wait helpers, on an mbarrier that
    nothing completes (``complete=False``) and gives up after ``limit_ns``,
    setting DEVERR_TIMEOUT; with ``complete=True`` the waits return at once.
    ``result``: None or a CUDA uint32 tensor of 2 (1 = the wait saw the
    barrier complete, 0 = it gave up; [0] of the spinning helper and that of
    tree and window attention, 2 if they differ, [1] of the sleeping one)."""
    if result is not None:
        _dev(result)
        import torch
        _need(result.dtype in (torch.uint32, torch.int32) and result.numel() >= 2, "result: 2 x 32-bit")
    _raise(load_library().fkv_selftest_wait(int(limit_ns), 1 if complete else 0, _ptr(result), _stream(stream)),
           "fkv_selftest_wait")
