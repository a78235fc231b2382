"""Thin Python binding of libfp (FlashPrefill-style block-sparse causal prefill on sm_100a).

Argument marshalling only: every step of the path (pooling, search, attention) runs in the
CUDA kernels of libfp.so; PyTorch supplies device memory and the current stream. There is no
CPU or PyTorch fallback: importing this module without the built library raises.

Entry points mirror the C ABI in include/fp.h:
    problem(...)            -> Problem (fp_problem_init)
    index_buffer_elems(...) -> fp_index_buffer_elems (index buffer length from sequence lengths)
    check_device_status(..) -> fp_check_device_status (dev_status word -> FpError)
    block_pool(...)         -> fp_block_pool
    block_search(...)       -> fp_block_search
    block_search_topp(...)  -> fp_block_search_topp (the cumulative top-p comparison selector)
    block_pool_search(...)  -> fp_block_pool_search (steps 1 + 2 fused)
    block_sparse_attn(...)  -> fp_block_sparse_attn
    block_sparse_attn_fp8 / dense_attn_fp8 -> e4m3 Q / K attention, per-tensor scales (fp_*_fp8)
    block_sparse_attn_fp8_blockscaled / dense_attn_fp8_blockscaled -> per-block power-of-two scales
    dense_attn(...)         -> fp_dense_attn
    sparse_prefill(...)     -> fp_sparse_prefill (all three steps, caller workspace)
    validate_lists(...)     -> fp_validate_lists
    paged_cache(...)        -> PagedCache (fp_paged_cache_init: chunked prefill onto a paged K/V cache)
    paged_block_pool / paged_block_search / paged_block_sparse_attn / paged_dense_attn /
    paged_validate_lists    -> the fp_paged_* calls
    kv_cache(...)           -> KVCache (fp_kv_cache_init: serving from a paged K/V cache)
    cache_append / cache_attn / cache_select / cache_compact -> the fp_cache_* calls
and SparsePrefill bundles the three steps with caller-side buffers.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp.so")

FP_OK, FP_ERR_INVALID_ARG, FP_ERR_UNSUPPORTED, FP_ERR_CUDA, FP_ERR_TIMEOUT = 0, 1, 2, 3, 4
FP_DEV_TIMEOUT, FP_DEV_BAD_LIST, FP_DEV_BAD_PROBLEM = 1, 2, 4
FP_MAX_SEQS = 1024
FP_SCHED_WORDS = 2  # int32 words of the attention work counter (fp_problem.sched)
FP_NOALLOC_MAX_BYTES = 64 << 20
EXPORTED = ("fp_problem_init", "fp_block_pool", "fp_block_search", "fp_block_pool_search", "fp_block_sparse_attn",
            "fp_dense_attn", "fp_sparse_prefill_workspace", "fp_sparse_prefill", "fp_sparse_prefill_noalloc",
            "fp_validate_lists", "fp_selftest_exp2", "fp_last_error", "fp_version", "fp_paged_cache_init",
            "fp_paged_block_pool", "fp_paged_block_search", "fp_paged_block_sparse_attn", "fp_paged_dense_attn",
            "fp_paged_validate_lists", "fp_block_search_topp", "fp_block_sparse_attn_fp8", "fp_dense_attn_fp8",
            "fp_index_buffer_elems", "fp_check_device_status", "fp_key_split_bytes", "fp_block_sparse_attn_fp8_blockscaled",
            "fp_dense_attn_fp8_blockscaled", "fp_kv_cache_init", "fp_cache_append", "fp_cache_attn_workspace",
            "fp_cache_attn", "fp_cache_select", "fp_cache_compact")


class FpError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"fp status {status}: {msg}")
        self.status = status


class fp_problem(C.Structure):
    _fields_ = [("cu_seqlens", C.c_void_p), ("num_seqs", C.c_int32), ("total_tokens", C.c_int32),
                ("total_blocks", C.c_int32), ("max_seq_blocks", C.c_int32), ("index_elems", C.c_int64),
                ("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("block_size", C.c_int32), ("sched", C.c_void_p), ("key_split", C.c_void_p),
                ("key_split_bytes", C.c_int64)]


class fp_paged_cache(C.Structure):
    _fields_ = [("prefix_lens", C.c_void_p), ("block_table", C.c_void_p), ("max_pages", C.c_int32),
                ("page_size", C.c_int32), ("num_pages", C.c_int32), ("total_kv_blocks", C.c_int32),
                ("index_elems", C.c_int64)]


class fp_kv_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("weights", C.c_void_p), ("positions", C.c_void_p),
                ("lens", C.c_void_p), ("block_table", C.c_void_p), ("max_pages", C.c_int32),
                ("page_size", C.c_int32), ("num_pages", C.c_int32), ("max_len", C.c_int32), ("max_new", C.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libfp.so is not built ({LIB_PATH}); run python block_sparse_long_causal_b200/build.py")
    lib = C.CDLL(LIB_PATH)
    vp, i32, f32 = C.c_void_p, C.c_int32, C.c_float
    P = C.POINTER(fp_problem)
    PC = C.POINTER(fp_paged_cache)
    KV = C.POINTER(fp_kv_cache)
    i64 = C.c_int64
    sig = {
        "fp_paged_cache_init": [PC, P, vp, vp, vp, vp, i32, i32, i32],
        "fp_block_search_topp": [P, vp, vp, f32, vp, vp, vp, vp, vp],
        "fp_block_sparse_attn_fp8": [P, vp, vp, vp, f32, f32, vp, vp, f32, vp, vp, vp, vp],
        "fp_dense_attn_fp8": [P, vp, vp, vp, f32, f32, f32, vp, vp, vp, vp],
        "fp_block_sparse_attn_fp8_blockscaled": [P, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, vp],
        "fp_dense_attn_fp8_blockscaled": [P, vp, vp, vp, vp, vp, f32, vp, vp, vp, vp],
        "fp_paged_block_pool": [P, PC, vp, vp, vp, vp, vp],
        "fp_paged_block_search": [P, PC, vp, vp, f32, vp, vp, vp, vp],
        "fp_paged_block_sparse_attn": [P, PC, vp, vp, vp, vp, vp, f32, vp, vp, vp, vp],
        "fp_paged_dense_attn": [P, PC, vp, vp, vp, f32, vp, vp, vp, vp],
        "fp_paged_validate_lists": [P, PC, vp, vp, vp, vp],
        "fp_problem_init": [P, vp, i32, vp, i32, i32, i32, i32],
        "fp_block_pool": [P, vp, vp, vp, vp, vp],
        "fp_block_search": [P, vp, vp, f32, vp, vp, vp, vp],
        "fp_block_pool_search": [P, vp, vp, f32, vp, vp, vp, vp, vp, vp],
        "fp_block_sparse_attn": [P, vp, vp, vp, vp, vp, f32, vp, vp, vp, vp],
        "fp_dense_attn": [P, vp, vp, vp, f32, vp, vp, vp, vp],
        "fp_validate_lists": [P, vp, vp, vp, vp],
        "fp_selftest_exp2": [vp, vp, vp, C.c_int64, vp],
        "fp_sparse_prefill_workspace": [P, C.POINTER(C.c_int64)],
        "fp_sparse_prefill": [P, vp, vp, vp, f32, f32, vp, C.c_int64, vp, vp, vp, vp],
        "fp_sparse_prefill_noalloc": [P, vp, vp, vp, f32, f32, vp, vp, vp, vp],
        "fp_index_buffer_elems": [vp, i32, i32, i32, C.POINTER(C.c_int64)],
        "fp_check_device_status": [i32],
        "fp_key_split_bytes": [P, vp, C.POINTER(C.c_int64)],
        "fp_kv_cache_init": [KV, P, vp, vp, vp, vp, vp, i32, i32, i32, i32],
        "fp_cache_append": [P, KV, vp, i64, vp, i64, vp, vp, vp],
        "fp_cache_attn_workspace": [P, KV, C.POINTER(C.c_int64)],
        "fp_cache_attn": [P, KV, vp, i64, f32, vp, i64, vp, vp, f32, vp, vp],
        "fp_cache_select": [P, KV, i32, i32, i32, vp, vp, vp, vp, vp, vp],
        "fp_cache_compact": [P, KV, i32, vp, vp, vp, vp, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = C.c_int
    lib.fp_last_error.restype = C.c_char_p
    lib.fp_last_error.argtypes = []
    lib.fp_version.restype = C.c_int32
    lib.fp_version.argtypes = []
    return lib


_lib = _load()


def version() -> int:
    return int(_lib.fp_version())


def _check(st: int):
    if st != FP_OK:
        raise FpError(st, _lib.fp_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return C.c_void_p(t.data_ptr())
    return C.c_void_p(int(t))


def _stream(stream):
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


class Problem:
    """fp_problem plus the device tensors it points to (kept alive here): cu_seqlens and, with
    work_counter (the default on a CUDA device), the attention calls' work counter -- zeroed once,
    left at zero by every launch, so launches of this problem must be ordered (one stream, or
    events); give concurrent streams one Problem each. With key_split (the default on a CUDA device)
    the searches of the plain problem split the pooled keys once per call into a scratch buffer held
    here (fp_problem.key_split)."""

    def __init__(self, cu_seqlens_host, cu_seqlens_dev: torch.Tensor, num_q_heads: int, num_kv_heads: int,
                 head_dim: int, block_size: int, work_counter: bool = True, key_split: bool = True):
        host = np.ascontiguousarray(cu_seqlens_host, np.int32)
        if cu_seqlens_dev.dtype != torch.int32:
            raise ValueError("cu_seqlens must be int32")
        self.cu_host = host
        self.cu_dev = cu_seqlens_dev
        self.c = fp_problem()
        _check(_lib.fp_problem_init(C.byref(self.c), host.ctypes.data_as(C.c_void_p), len(host) - 1,
                                    _ptr(cu_seqlens_dev), num_q_heads, num_kv_heads, head_dim, block_size))
        self.sched = None
        if work_counter and cu_seqlens_dev.is_cuda:
            self.sched = torch.zeros(FP_SCHED_WORDS, dtype=torch.int32, device=cu_seqlens_dev.device)
            self.c.sched = self.sched.data_ptr()
        self.key_split = None
        if key_split and cu_seqlens_dev.is_cuda:
            nbytes = key_split_bytes(self)
            self.key_split = torch.empty(nbytes, dtype=torch.uint8, device=cu_seqlens_dev.device)
            self.c.key_split = self.key_split.data_ptr()
            self.c.key_split_bytes = nbytes

    def __getattr__(self, name):
        return getattr(self.__dict__["c"], name)

    @property
    def ref(self):
        return C.byref(self.c)


def problem(cu_seqlens_host, num_q_heads: int, num_kv_heads: int, head_dim: int = 128, block_size: int = 128,
            device="cuda", work_counter: bool = True, key_split: bool = True) -> Problem:
    host = np.ascontiguousarray(cu_seqlens_host, np.int32)
    dev = torch.from_numpy(host.copy()).to(device)
    return Problem(host, dev, num_q_heads, num_kv_heads, head_dim, block_size, work_counter, key_split)


def _cache_ref(cache):
    return cache.ref if isinstance(cache, PagedCache) else C.byref(cache)


def key_split_bytes(p, cache=None) -> int:
    """fp_key_split_bytes: bytes of the search's key split scratch for this problem (and paged cache)."""
    n = C.c_int64(0)
    ref = p.ref if isinstance(p, Problem) else C.byref(p)
    _check(_lib.fp_key_split_bytes(ref, None if cache is None else _cache_ref(cache), C.byref(n)))
    return int(n.value)


def index_buffer_elems(seqlens, block_size: int, num_q_heads: int) -> int:
    """fp_index_buffer_elems: int32 entries of the index buffer for these sequence lengths."""
    lens = np.ascontiguousarray(seqlens, np.int32)
    n = C.c_int64(0)
    _check(_lib.fp_index_buffer_elems(lens.ctypes.data_as(C.c_void_p), len(lens), int(block_size), int(num_q_heads),
                                      C.byref(n)))
    return int(n.value)


def check_device_status(bits: int) -> None:
    """fp_check_device_status: raise FpError (status FP_ERR_TIMEOUT / FP_ERR_INVALID_ARG) for a
    non-zero dev_status word read back after the stream completed."""
    _check(_lib.fp_check_device_status(int(bits)))


def block_pool(p: Problem, q, k, q_pool, k_pool, stream=None):
    _check(_lib.fp_block_pool(p.ref, _ptr(q), _ptr(k), _ptr(q_pool), _ptr(k_pool), _stream(stream)))


def block_search(p: Problem, q_pool, k_pool, tau: float, counts, indices, dev_status=None, stream=None):
    _check(_lib.fp_block_search(p.ref, _ptr(q_pool), _ptr(k_pool), float(tau), _ptr(counts), _ptr(indices),
                                _ptr(dev_status), _stream(stream)))


def block_search_topp(p: Problem, q_pool, k_pool, gamma: float, scores, counts, indices, dev_status=None,
                      stream=None):
    """Cumulative top-p block selection (the comparison selector); scores: float32 [index_elems] scratch."""
    _check(_lib.fp_block_search_topp(p.ref, _ptr(q_pool), _ptr(k_pool), float(gamma), _ptr(scores), _ptr(counts),
                                     _ptr(indices), _ptr(dev_status), _stream(stream)))


def block_pool_search(p: Problem, q, k, tau: float, q_pool, k_pool, counts, indices, dev_status=None, stream=None):
    _check(_lib.fp_block_pool_search(p.ref, _ptr(q), _ptr(k), float(tau), _ptr(q_pool), _ptr(k_pool), _ptr(counts),
                                     _ptr(indices), _ptr(dev_status), _stream(stream)))


def block_sparse_attn(p: Problem, q, k, v, counts, indices, softmax_scale: float, out, lse=None, dev_status=None,
                      stream=None):
    _check(_lib.fp_block_sparse_attn(p.ref, _ptr(q), _ptr(k), _ptr(v), _ptr(counts), _ptr(indices),
                                     float(softmax_scale), _ptr(out), _ptr(lse), _ptr(dev_status), _stream(stream)))


def block_sparse_attn_fp8(p: Problem, q_e4m3, k_e4m3, v, q_scale: float, k_scale: float, counts, indices,
                          softmax_scale: float, out, lse=None, dev_status=None, stream=None):
    """FP8 attention: e4m3 Q / K codes (uint8 tensors) with per-tensor scales, bf16 V."""
    _check(_lib.fp_block_sparse_attn_fp8(p.ref, _ptr(q_e4m3), _ptr(k_e4m3), _ptr(v), float(q_scale), float(k_scale),
                                         _ptr(counts), _ptr(indices), float(softmax_scale), _ptr(out), _ptr(lse),
                                         _ptr(dev_status), _stream(stream)))


def dense_attn_fp8(p: Problem, q_e4m3, k_e4m3, v, q_scale: float, k_scale: float, softmax_scale: float, out, lse=None,
                   dev_status=None, stream=None):
    _check(_lib.fp_dense_attn_fp8(p.ref, _ptr(q_e4m3), _ptr(k_e4m3), _ptr(v), float(q_scale), float(k_scale),
                                  float(softmax_scale), _ptr(out), _ptr(lse), _ptr(dev_status), _stream(stream)))


def block_sparse_attn_fp8_blockscaled(p: Problem, q_e4m3, k_e4m3, v, q_exp, k_exp, counts, indices,
                                      softmax_scale: float, out, lse=None, dev_status=None, stream=None):
    """FP8 attention with per-block power-of-two scales: q_exp int8 [total_blocks, Hq], k_exp int8
    [total_blocks, Hkv] (dequantised value = 2^exp * e4m3 code)."""
    _check(_lib.fp_block_sparse_attn_fp8_blockscaled(p.ref, _ptr(q_e4m3), _ptr(k_e4m3), _ptr(v), _ptr(q_exp),
                                                     _ptr(k_exp), _ptr(counts), _ptr(indices), float(softmax_scale),
                                                     _ptr(out), _ptr(lse), _ptr(dev_status), _stream(stream)))


def dense_attn_fp8_blockscaled(p: Problem, q_e4m3, k_e4m3, v, q_exp, k_exp, softmax_scale: float, out, lse=None,
                               dev_status=None, stream=None):
    _check(_lib.fp_dense_attn_fp8_blockscaled(p.ref, _ptr(q_e4m3), _ptr(k_e4m3), _ptr(v), _ptr(q_exp), _ptr(k_exp),
                                              float(softmax_scale), _ptr(out), _ptr(lse), _ptr(dev_status),
                                              _stream(stream)))


def dense_attn(p: Problem, q, k, v, softmax_scale: float, out, lse=None, dev_status=None, stream=None):
    _check(_lib.fp_dense_attn(p.ref, _ptr(q), _ptr(k), _ptr(v), float(softmax_scale), _ptr(out), _ptr(lse),
                              _ptr(dev_status), _stream(stream)))


def validate_lists(p: Problem, counts, indices, dev_status, stream=None):
    _check(_lib.fp_validate_lists(p.ref, _ptr(counts), _ptr(indices), _ptr(dev_status), _stream(stream)))


def sparse_prefill_workspace(p: Problem) -> int:
    n = C.c_int64(0)
    _check(_lib.fp_sparse_prefill_workspace(p.ref, C.byref(n)))
    return int(n.value)


def sparse_prefill(p: Problem, q, k, v, tau: float, softmax_scale: float, workspace, out, lse=None, dev_status=None,
                   stream=None):
    _check(_lib.fp_sparse_prefill(p.ref, _ptr(q), _ptr(k), _ptr(v), float(tau), float(softmax_scale),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
                                  _ptr(dev_status), _stream(stream)))


def sparse_prefill_noalloc(p: Problem, q, k, v, tau: float, softmax_scale: float, out, lse=None, dev_status=None,
                           stream=None):
    """fp_sparse_prefill for callers that cannot allocate: intermediates in the library's static array."""
    _check(_lib.fp_sparse_prefill_noalloc(p.ref, _ptr(q), _ptr(k), _ptr(v), float(tau), float(softmax_scale),
                                          _ptr(out), _ptr(lse), _ptr(dev_status), _stream(stream)))


def selftest_exp2(x, y_poly, y_mufu, stream=None):
    _check(_lib.fp_selftest_exp2(_ptr(x), _ptr(y_poly), _ptr(y_mufu), x.numel(), _stream(stream)))


class PagedCache:
    """fp_paged_cache plus the device prefix-length and block-table tensors it points to."""

    def __init__(self, p: Problem, prefix_lens_host, prefix_lens_dev: torch.Tensor, block_table_dev: torch.Tensor,
                 page_size: int, num_pages: int):
        pre = np.ascontiguousarray(prefix_lens_host, np.int32)
        if prefix_lens_dev.dtype != torch.int32 or block_table_dev.dtype != torch.int32:
            raise ValueError("prefix_lens and block_table must be int32")
        if block_table_dev.dim() != 2 or block_table_dev.shape[0] != p.num_seqs:
            raise ValueError("block_table must be [num_seqs, max_pages]")
        self.p = p
        self.prefix_host = pre
        self.prefix_dev = prefix_lens_dev
        self.table_dev = block_table_dev.contiguous()
        self.c = fp_paged_cache()
        _check(_lib.fp_paged_cache_init(C.byref(self.c), p.ref, p.cu_host.ctypes.data_as(C.c_void_p),
                                        pre.ctypes.data_as(C.c_void_p), _ptr(prefix_lens_dev), _ptr(self.table_dev),
                                        int(self.table_dev.shape[1]), int(page_size), int(num_pages)))
        # the paged search's key split covers the cached prefixes' key blocks too
        self.key_split = None
        if p.key_split is not None:
            nbytes = key_split_bytes(p, self)
            self.key_split = torch.empty(nbytes, dtype=torch.uint8, device=prefix_lens_dev.device)
            self.search_problem = fp_problem.from_buffer_copy(p.c)
            self.search_problem.key_split = self.key_split.data_ptr()
            self.search_problem.key_split_bytes = nbytes

    def __getattr__(self, name):
        return getattr(self.__dict__["c"], name)

    @property
    def ref(self):
        return C.byref(self.c)


def paged_cache(p: Problem, prefix_lens_host, block_table, page_size: int, num_pages: int, device="cuda") -> PagedCache:
    pre = np.ascontiguousarray(prefix_lens_host, np.int32)
    table = block_table if isinstance(block_table, torch.Tensor) else torch.from_numpy(
        np.ascontiguousarray(block_table, np.int32))
    return PagedCache(p, pre, torch.from_numpy(pre.copy()).to(device), table.to(device=device, dtype=torch.int32),
                      page_size, num_pages)


def paged_block_pool(p: Problem, c: PagedCache, q, k_cache, q_pool, k_pool, stream=None):
    _check(_lib.fp_paged_block_pool(p.ref, c.ref, _ptr(q), _ptr(k_cache), _ptr(q_pool), _ptr(k_pool), _stream(stream)))


def paged_block_search(p: Problem, c: PagedCache, q_pool, k_pool, tau: float, counts, indices, dev_status=None,
                       stream=None):
    ref = C.byref(c.search_problem) if c.key_split is not None and p is c.p else p.ref
    _check(_lib.fp_paged_block_search(ref, c.ref, _ptr(q_pool), _ptr(k_pool), float(tau), _ptr(counts),
                                      _ptr(indices), _ptr(dev_status), _stream(stream)))


def paged_block_sparse_attn(p: Problem, c: PagedCache, q, k_cache, v_cache, counts, indices, softmax_scale: float, out,
                            lse=None, dev_status=None, stream=None):
    _check(_lib.fp_paged_block_sparse_attn(p.ref, c.ref, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(counts),
                                           _ptr(indices), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(dev_status),
                                           _stream(stream)))


def paged_dense_attn(p: Problem, c: PagedCache, q, k_cache, v_cache, softmax_scale: float, out, lse=None,
                     dev_status=None, stream=None):
    _check(_lib.fp_paged_dense_attn(p.ref, c.ref, _ptr(q), _ptr(k_cache), _ptr(v_cache), float(softmax_scale),
                                    _ptr(out), _ptr(lse), _ptr(dev_status), _stream(stream)))


def paged_validate_lists(p: Problem, c: PagedCache, counts, indices, dev_status, stream=None):
    _check(_lib.fp_paged_validate_lists(p.ref, c.ref, _ptr(counts), _ptr(indices), _ptr(dev_status),
                                        _stream(stream)))


# The cache calls are made once per token and layer: their checks are plain attribute reads, and names that are
# looked up at every call are bound here.
_Tensor, _BF16, _I32 = torch.Tensor, torch.bfloat16, torch.int32


def _rows_of(t, name: str, tokens: int, heads: int, d: int, device):
    """Pointer and token-row stride of a bf16 [tokens, heads, head_dim] tensor whose rows may lie apart (a
    slice of a fused projection)."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.device != device:
        _want(t, name, _BF16, device)  # says what is wrong
    if t.shape != (tokens, heads, d):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {d}], got {list(t.shape)}")
    if tokens == 0:
        return None, 0
    row, head, col = t.stride()
    if col != 1 or (head != d and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if tokens == 1:
        return t.data_ptr(), 0
    if row < heads * d:  # an expanded tensor has stride 0, which the C call takes for packed rows
        raise ValueError(f"{name}: the rows of its tokens overlap (stride {row}, at least {heads * d})")
    return t.data_ptr(), row


def _want(t, name: str, dtype, device, numel=None) -> int:
    """Check a tensor argument; its address."""
    if not isinstance(t, _Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if numel is not None and (t.numel() != numel or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous with {numel} elements")
    return t.data_ptr()


class KVCache:
    """fp_kv_cache for the new tokens of problem p, plus the device tensors that it points to: k_cache
    and v_cache bf16 [num_pages * page_size, Hkv, d] (or [num_pages, page_size, Hkv, d]), lens int32
    [num_seqs], block_table int32 [num_seqs, max_pages], optional weights float32 and positions int32
    [num_pages, Hkv, page_size]. The tensors are used in place: a serving loop keeps one KVCache per
    problem shape over the same tensors."""

    def __init__(self, p: Problem, k_cache, v_cache, lens, block_table, page_size: int, weights=None, positions=None,
                 max_len: int = 0):
        page_size, hkv, d = int(page_size), int(p.num_kv_heads), int(p.head_dim)
        dev = k_cache.device
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            _want(t, name, torch.bfloat16, dev, k_cache.numel())
            if t.dim() not in (3, 4) or tuple(t.shape[-2:]) != (hkv, d):
                raise ValueError(f"{name} must be [num_pages * page_size, {hkv}, {d}]")
        if page_size < 1 or k_cache.numel() == 0 or k_cache.numel() % (page_size * hkv * d):
            raise ValueError(f"k_cache must hold whole pages of {page_size} slots")
        num_pages = k_cache.numel() // (page_size * hkv * d)
        _want(lens, "lens", torch.int32, dev, p.num_seqs)
        _want(block_table, "block_table", torch.int32, dev)
        if block_table.dim() != 2 or block_table.shape[0] != p.num_seqs or not block_table.is_contiguous():
            raise ValueError("block_table must be contiguous [num_seqs, max_pages]")
        if p.cu_dev.device != dev:
            raise ValueError(f"the problem is on {p.cu_dev.device}, the cache on {dev}")
        for name, t, dt in (("weights", weights, torch.float32), ("positions", positions, torch.int32)):
            if t is not None:
                _want(t, name, dt, dev, num_pages * hkv * page_size)
        self.p, self.device = p, dev
        self.k, self.v, self.lens, self.table = k_cache, v_cache, lens, block_table
        self.weights, self.positions = weights, positions
        self.c = fp_kv_cache()
        _check(_lib.fp_kv_cache_init(C.byref(self.c), p.ref, p.cu_host.ctypes.data_as(C.c_void_p), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(lens), _ptr(block_table), int(block_table.shape[1]),
                                     page_size, num_pages, int(max_len)))
        if weights is not None:
            self.c.weights = weights.data_ptr()
        if positions is not None:
            self.c.positions = positions.data_ptr()
        # what every call looks up, as plain attributes
        self.ref, self.p_ref = C.byref(self.c), p.ref
        self.tokens, self.seqs = int(p.total_tokens), int(p.num_seqs)
        self.hq, self.hkv, self.d = int(p.num_q_heads), hkv, d
        self.index = dev.index if dev.type == "cuda" else -1

    def __getattr__(self, name):
        return getattr(self.__dict__["c"], name)


def kv_cache(p: Problem, k_cache, v_cache, lens, block_table, page_size: int, weights=None, positions=None,
             max_len: int = 0) -> KVCache:
    return KVCache(p, k_cache, v_cache, lens, block_table, page_size, weights, positions, max_len)


def _cache_args(p: Problem, c: KVCache, next_pos, dev_status):
    """Addresses of next_pos and dev_status (None: NULL)."""
    if p is not c.p:
        raise ValueError("the cache was described for another problem (kv_cache(p, ...))")
    return (None if next_pos is None else _want(next_pos, "next_pos", _I32, c.device, c.seqs),
            None if dev_status is None else _want(dev_status, "dev_status", _I32, c.device, 1))


def _call(c: KVCache, stream, fn, *args):
    """fn on the cache's device, on `stream` or that device's current one."""
    index = c.index
    if index < 0:
        raise ValueError(f"the cache is on {c.device}: the kernels run on a CUDA device only")
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(c, stream, fn, *args)
    st = fn(c.p_ref, c.ref, *args, torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream))
    if st != FP_OK:
        _check(st)


def cache_append(p: Problem, c: KVCache, k, v, next_pos=None, dev_status=None, stream=None):
    """fp_cache_append: the new tokens' K and V rows into their slots."""
    pos, status = _cache_args(p, c, next_pos, dev_status)
    kp, ks = _rows_of(k, "k", c.tokens, c.hkv, c.d, c.device)
    vp, vs = _rows_of(v, "v", c.tokens, c.hkv, c.d, c.device)
    _call(c, stream, _lib.fp_cache_append, kp, ks, vp, vs, pos, status)


def cache_attn_workspace(p: Problem, c: KVCache) -> int:
    n = C.c_int64(0)
    with torch.cuda.device(c.device):
        _check(_lib.fp_cache_attn_workspace(p.ref, c.ref, C.byref(n)))
    return int(n.value)


def cache_attn(p: Problem, c: KVCache, q, softmax_scale: float, workspace, out, lse=None, decay=None, dev_status=None,
               stream=None):
    """fp_cache_attn; decay None leaves the cache's weights alone."""
    _, status = _cache_args(p, c, None, dev_status)
    qp, qs = _rows_of(q, "q", c.tokens, c.hq, c.d, c.device)
    rows = c.tokens * c.hq
    op = _want(out, "out", _BF16, c.device, rows * c.d)
    lp = None if lse is None else _want(lse, "lse", torch.float32, c.device, rows)
    if not isinstance(workspace, torch.Tensor) or workspace.device != c.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {c.device}")
    if decay is None:
        decay = -1.0
    elif not 0.0 <= decay <= 1.0:
        raise ValueError("decay must be in [0, 1]")
    _call(c, stream, _lib.fp_cache_attn, qp, qs, softmax_scale, workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), op, lp, decay, status)


def _move_args(c: KVCache, budget: int, moves, move_counts, new_lens):
    n = c.seqs * c.hkv
    return (_want(moves, "moves", _I32, c.device, 2 * n * budget),
            _want(move_counts, "move_counts", _I32, c.device, n),
            _want(new_lens, "new_lens", _I32, c.device, c.seqs))


def cache_select(p: Problem, c: KVCache, budget: int, sinks: int, recent: int, next_pos, moves, move_counts, new_lens,
                 dev_status=None, stream=None):
    """fp_cache_select: the slots that stay, as moves int32 [num_seqs, Hkv, budget, 2]."""
    pos, status = _cache_args(p, c, next_pos, dev_status)
    out = _move_args(c, budget, moves, move_counts, new_lens)
    _call(c, stream, _lib.fp_cache_select, budget, sinks, recent, pos, *out, status)


def cache_compact(p: Problem, c: KVCache, budget: int, moves, move_counts, new_lens, dev_status=None, stream=None):
    """fp_cache_compact: apply the moves of cache_select and set lens."""
    _, status = _cache_args(p, c, None, dev_status)
    out = _move_args(c, budget, moves, move_counts, new_lens)
    _call(c, stream, _lib.fp_cache_compact, budget, *out, status)


class SparsePrefill:
    """Caller-side buffers for one problem shape, and the three-step sparse prefill.

    Buffers are allocated once (through PyTorch) and reused by every call; the library itself
    never allocates.
    """

    def __init__(self, p: Problem, device="cuda", with_lse: bool = False):
        self.p = p
        nb, hq, hkv, d = p.total_blocks, p.num_q_heads, p.num_kv_heads, p.head_dim
        self.q_pool = torch.empty((max(nb, 1), hq, d), dtype=torch.float32, device=device)
        self.k_pool = torch.empty((max(nb, 1), hkv, d), dtype=torch.float32, device=device)
        self.counts = torch.zeros((hq, max(nb, 1)), dtype=torch.int32, device=device)
        self.indices = torch.zeros(max(p.index_elems, 1), dtype=torch.int32, device=device)
        self.out = torch.empty((max(p.total_tokens, 1), hq, d), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((hq, max(p.total_tokens, 1)), dtype=torch.float32, device=device) if with_lse else None
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=device)

    def search(self, q, k, tau: float, stream=None, fused: bool = True):
        if fused:
            block_pool_search(self.p, q, k, tau, self.q_pool, self.k_pool, self.counts, self.indices,
                              self.dev_status, stream)
        else:
            block_pool(self.p, q, k, self.q_pool, self.k_pool, stream)
            block_search(self.p, self.q_pool, self.k_pool, tau, self.counts, self.indices, self.dev_status, stream)

    def attend(self, q, k, v, softmax_scale: float = 0.0, stream=None):
        block_sparse_attn(self.p, q, k, v, self.counts, self.indices, softmax_scale, self.out, self.lse,
                          self.dev_status, stream)
        return self.out

    def __call__(self, q, k, v, tau: float, softmax_scale: float = 0.0, stream=None):
        self.search(q, k, tau, stream)
        return self.attend(q, k, v, softmax_scale, stream)

    def dense(self, q, k, v, softmax_scale: float = 0.0, stream=None):
        dense_attn(self.p, q, k, v, softmax_scale, self.out, self.lse, self.dev_status, stream)
        return self.out
