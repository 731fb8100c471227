"""Python binding of libdsv4attn.so (ctypes).

Argument marshalling only: every step of the attention computation runs in
the library's CUDA kernels.  PyTorch supplies device memory (outputs and the
workspace are allocated here when the caller passes none) and the current
stream.  With stream= the kernels are queued on that stream instead, which
waits for nothing queued on the current one: ordering the two, and keeping
what is passed in alive until that stream has used it, is the caller's part.
Loading fails loudly when the library has not been built; there is
no fallback path.

The entry points mirror include/dsv4attn.h:
  dsv4_attn_swa, dsv4_attn_c4_sparse, dsv4_attn_c128_dense, dsv4_attn_verify,
  dsv4_attn_plan, dsv4_attn_workspace_size, dsv4_attn_get_device_error,
  dsv4_attn_strerror;
include/dsv4kvstore.h (the cache write before the step):
  dsv4_kv_store;
include/dsv4topk.h (the top-k selection that makes the C4 index lists):
  dsv4_topk, dsv4_topk_max_length;
and include/dsv4gqa.h (the cache of a grouped-query model, such as a separate
one that drafts the tokens dsv4_attn_verify checks: its write, its one-token
attention and the eviction of its rows):
  make_gqa_cache, dsv4_gqa_store, dsv4_gqa_decode, dsv4_gqa_evict,
  dsv4_gqa_decode_workspace_size, dsv4_gqa_evict_workspace_size.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsv4attn.so")

DSV4_KV_BF16 = 0
DSV4_KV_FP8_PACKED = 1
DSV4_GQA_BF16 = 0
DSV4_GQA_F16 = 1
DSV4_GQA_E4M3 = 2
DEV_ERR = {
    "SWA_PAGE": 0x01, "EXTRA_PAGE": 0x02, "INDEX_RANGE": 0x04, "POSITION": 0x08,
    "PLAN": 0x10, "TIMEOUT": 0x20, "REQ_ROW": 0x40, "STORE_ROW": 0x80, "TOPK_LENGTH": 0x100,
    "GQA_PAGE": 0x200, "GQA_LENGTH": 0x400,
}
EXPORTED = [
    "dsv4_attn_swa", "dsv4_attn_c4_sparse", "dsv4_attn_c128_dense", "dsv4_attn_verify",
    "dsv4_attn_plan", "dsv4_attn_workspace_size", "dsv4_attn_get_device_error",
    "dsv4_attn_strerror", "dsv4_attn_c4_sparse_noalloc", "dsv4_kv_store",
    "dsv4_topk", "dsv4_topk_max_length",
    "dsv4_gqa_store", "dsv4_gqa_decode", "dsv4_gqa_decode_workspace_size", "dsv4_gqa_evict",
    "dsv4_gqa_evict_workspace_size",
]
NOALLOC_SCRATCH_BYTES = 16 << 20


class KvPool(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64),
        ("row_bytes", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("page_table", ctypes.c_void_p),
        ("page_table_rows", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
    ]


class GqaCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64),
        ("page_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("page_table", ctypes.c_void_p),
        ("page_table_rows", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("page_table_width", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


class Dsv4Error(RuntimeError):
    pass


def load_library(path=LIB_PATH):
    if not os.path.exists(path):
        raise Dsv4Error(f"{path} is missing: build it with hybrid_sparse_mqa_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    PP = ctypes.POINTER(KvPool)
    lib.dsv4_attn_swa.argtypes = [P, I32, I32, P, P, PP, I32, P, F32, P, P, I32, P, SZ, P, P]
    lib.dsv4_attn_c4_sparse.argtypes = [P, I32, I32, P, P, PP, I32, PP, P, I32, P, F32, P, P, I32, P, SZ, P, P]
    lib.dsv4_attn_c128_dense.argtypes = [P, I32, I32, P, P, PP, I32, PP, I32, P, F32, P, P, I32, P, SZ, P, P]
    lib.dsv4_attn_verify.argtypes = [P, I32, I32, I32, P, P, P, PP, I32, I32, PP, P, I32, I32, P, F32,
                                     P, P, I32, P, SZ, P, P]
    lib.dsv4_attn_c4_sparse_noalloc.argtypes = [P, I32, I32, P, P, PP, I32, PP, P, I32, P, F32, P, P, I32, P, P]
    for name in ("dsv4_attn_swa", "dsv4_attn_c4_sparse", "dsv4_attn_c128_dense", "dsv4_attn_verify",
                 "dsv4_attn_c4_sparse_noalloc"):
        getattr(lib, name).restype = ctypes.c_int
    lib.dsv4_attn_plan.argtypes = [I32, I32, I32, I32, I32, I32, I32,
                                   ctypes.POINTER(I32), ctypes.POINTER(I32)]
    lib.dsv4_attn_plan.restype = ctypes.c_int
    lib.dsv4_attn_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32, I32]
    lib.dsv4_attn_workspace_size.restype = SZ
    lib.dsv4_attn_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), P]
    lib.dsv4_attn_get_device_error.restype = ctypes.c_int
    lib.dsv4_attn_strerror.argtypes = [ctypes.c_int]
    lib.dsv4_attn_strerror.restype = ctypes.c_char_p
    lib.dsv4_kv_store.argtypes = [P, I32, P, P, PP, P]
    lib.dsv4_kv_store.restype = ctypes.c_int
    lib.dsv4_topk.argtypes = [P, I32, ctypes.c_int64, P, I32, I32, P, P]
    lib.dsv4_topk.restype = ctypes.c_int
    lib.dsv4_topk_max_length.argtypes = [I32]
    lib.dsv4_topk_max_length.restype = I32
    I64, PG = ctypes.c_int64, ctypes.c_void_p
    lib.dsv4_gqa_store.argtypes = [P, I64, I64, P, I64, I64, I32, I32, P, P, PG, P, P, I64, P, P]
    lib.dsv4_gqa_decode.argtypes = [P, I64, I32, I32, I32, P, P, PG, I32, I32, P, F32, P, P, I64, F32,
                                    P, P, P, SZ, P]
    lib.dsv4_gqa_evict.argtypes = [I32, P, P, P, PG, I32, I32, I32, I32, P, P, P, P, I64, P, P, SZ, P]
    for name in ("dsv4_gqa_store", "dsv4_gqa_decode", "dsv4_gqa_evict"):
        getattr(lib, name).restype = ctypes.c_int
    lib.dsv4_gqa_decode_workspace_size.argtypes = [PG, I32, I32, I32, I32]
    lib.dsv4_gqa_decode_workspace_size.restype = SZ
    lib.dsv4_gqa_evict_workspace_size.argtypes = [PG, I32, I32, I32]
    lib.dsv4_gqa_evict_workspace_size.restype = SZ
    return lib


_lib = None


def lib():
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


# ---------------------------------------------------------------- helpers
def _ptr(x):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _new(shape, dtype, device, stream):
    """A tensor that kernels on `stream` (None: the current one) write.  It comes from that stream's own memory: a
    block of the current stream's may still be in use by kernels queued there, which `stream` does not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _new_output(shape, dtype, device, stream):
    """As _new, for a tensor that the caller gets and reads on the current stream."""
    x = _new(shape, dtype, device, stream)
    if stream is not None:
        x.record_stream(torch.cuda.current_stream())
    return x


def make_pool(rows, page_table, kv_format=None):
    """dsv4_kv_pool for a device pool tensor ([rows, 512] bf16 or [rows, 608]
    uint8) and its int32 page table [request rows, logical pages]."""
    if kv_format is None:
        kv_format = DSV4_KV_BF16 if rows.dtype == torch.bfloat16 else DSV4_KV_FP8_PACKED
    row_bytes = rows.shape[1] * rows.element_size()
    pool = KvPool()
    pool.rows = rows.data_ptr()
    pool.num_pages = rows.shape[0] // 256
    pool.row_bytes = row_bytes
    pool.format = kv_format
    pool.page_table = page_table.data_ptr()
    pool.page_table_rows = page_table.shape[0]
    pool.page_table_stride = page_table.stride(0)
    pool.page_size = 256
    pool._keep = (rows, page_table)
    return pool


def _check(rc):
    if rc != 0:
        raise Dsv4Error(f"dsv4attn: {lib().dsv4_attn_strerror(rc).decode()} ({rc})")


def _outputs(q, out, lse, stream):
    T, H = q.shape[0], q.shape[1]
    if out is None:
        out = _new_output(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _new_output((T, H), torch.float32, q.device, stream)
    return out, lse


def _workspace(workspace, T, H, ratio, window, topk, max_seq_len, num_splits, device, stream):
    need = lib().dsv4_attn_workspace_size(T, H, ratio, window, topk, max_seq_len, num_splits)
    if workspace is None and need > 0:
        workspace = _new(need, torch.uint8, device, stream)
    return workspace, (0 if workspace is None else workspace.numel() * workspace.element_size())


def debug_stride(ratio, window, topk=0, max_seq_len=0):
    return window + (topk if ratio == 4 else (max_seq_len // 128 if ratio == 128 else 0))


# ---------------------------------------------------------------- entry points
def dsv4_attn_swa(q, seq_lens, swa_pool, sink, *, scale=1.0 / math.sqrt(512), window=128,
                  req_pool_indices=None, out=None, lse=None, num_splits=0, workspace=None,
                  debug_rows=None, stream=None):
    T, H = q.shape[0], q.shape[1]
    out, lse = _outputs(q, out, lse, stream)
    workspace, wsb = _workspace(workspace, T, H, 0, window, 0, 0, num_splits, q.device, stream)
    _check(lib().dsv4_attn_swa(_ptr(q), T, H, _ptr(seq_lens), _ptr(req_pool_indices),
                               ctypes.byref(swa_pool), window, _ptr(sink), scale, _ptr(out), _ptr(lse),
                               num_splits, _ptr(workspace), wsb, _ptr(debug_rows), _stream(stream)))
    return out, lse


def dsv4_attn_c4_sparse(q, seq_lens, swa_pool, extra_pool, topk_idx, sink, *,
                        scale=1.0 / math.sqrt(512), window=128, req_pool_indices=None, out=None,
                        lse=None, num_splits=0, workspace=None, debug_rows=None, stream=None):
    T, H = q.shape[0], q.shape[1]
    topk = topk_idx.shape[1]
    out, lse = _outputs(q, out, lse, stream)
    workspace, wsb = _workspace(workspace, T, H, 4, window, topk, 0, num_splits, q.device, stream)
    _check(lib().dsv4_attn_c4_sparse(_ptr(q), T, H, _ptr(seq_lens), _ptr(req_pool_indices),
                                     ctypes.byref(swa_pool), window, ctypes.byref(extra_pool),
                                     _ptr(topk_idx), topk, _ptr(sink), scale, _ptr(out), _ptr(lse),
                                     num_splits, _ptr(workspace), wsb, _ptr(debug_rows), _stream(stream)))
    return out, lse


def dsv4_attn_c4_sparse_noalloc(q, seq_lens, swa_pool, extra_pool, topk_idx, sink, *,
                                scale=1.0 / math.sqrt(512), window=128, req_pool_indices=None,
                                out=None, lse=None, num_splits=0, debug_rows=None, stream=None):
    """dsv4_attn_c4_sparse without a workspace argument: for callers that
    cannot allocate device memory, the split merge uses the library's own
    static scratch buffer (see include/dsv4attn.h for its limits)."""
    T, H = q.shape[0], q.shape[1]
    topk = topk_idx.shape[1]
    if out is None or lse is None:
        out, lse = _outputs(q, out, lse, stream)
    _check(lib().dsv4_attn_c4_sparse_noalloc(_ptr(q), T, H, _ptr(seq_lens), _ptr(req_pool_indices),
                                             ctypes.byref(swa_pool), window, ctypes.byref(extra_pool),
                                             _ptr(topk_idx), topk, _ptr(sink), scale, _ptr(out), _ptr(lse),
                                             num_splits, _ptr(debug_rows), _stream(stream)))
    return out, lse


def dsv4_attn_c128_dense(q, seq_lens, swa_pool, extra_pool, sink, *, max_seq_len,
                         scale=1.0 / math.sqrt(512), window=128, req_pool_indices=None, out=None,
                         lse=None, num_splits=0, workspace=None, debug_rows=None, stream=None):
    T, H = q.shape[0], q.shape[1]
    out, lse = _outputs(q, out, lse, stream)
    workspace, wsb = _workspace(workspace, T, H, 128, window, 0, max_seq_len, num_splits, q.device, stream)
    _check(lib().dsv4_attn_c128_dense(_ptr(q), T, H, _ptr(seq_lens), _ptr(req_pool_indices),
                                      ctypes.byref(swa_pool), window, ctypes.byref(extra_pool),
                                      max_seq_len, _ptr(sink), scale, _ptr(out), _ptr(lse), num_splits,
                                      _ptr(workspace), wsb, _ptr(debug_rows), _stream(stream)))
    return out, lse


def dsv4_attn_verify(q, seq_lens, cu_seqlens_q, swa_pool, sink, *, compress_ratio, batch,
                     extra_pool=None, topk_idx=None, max_seq_len=0, scale=1.0 / math.sqrt(512),
                     window=128, req_pool_indices=None, out=None, lse=None, num_splits=0,
                     workspace=None, debug_rows=None, stream=None):
    T, H = q.shape[0], q.shape[1]
    topk = 0 if topk_idx is None else topk_idx.shape[1]
    out, lse = _outputs(q, out, lse, stream)
    workspace, wsb = _workspace(workspace, T, H, compress_ratio, window, topk, max_seq_len,
                                num_splits, q.device, stream)
    _check(lib().dsv4_attn_verify(_ptr(q), T, batch, H, _ptr(seq_lens), _ptr(cu_seqlens_q),
                                  _ptr(req_pool_indices), ctypes.byref(swa_pool), window,
                                  compress_ratio,
                                  None if extra_pool is None else ctypes.byref(extra_pool),
                                  _ptr(topk_idx), topk, max_seq_len, _ptr(sink), scale, _ptr(out),
                                  _ptr(lse), num_splits, _ptr(workspace), wsb, _ptr(debug_rows),
                                  _stream(stream)))
    return out, lse


def dsv4_attn_plan(num_tokens, num_heads, compress_ratio, window=128, topk=0, max_seq_len=0,
                   num_splits=0):
    sc, sg = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().dsv4_attn_plan(num_tokens, num_heads, compress_ratio, window, topk, max_seq_len,
                                num_splits, ctypes.byref(sc), ctypes.byref(sg)))
    return sc.value, sg.value


def dsv4_attn_workspace_size(num_tokens, num_heads, compress_ratio, window=128, topk=0,
                             max_seq_len=0, num_splits=0):
    return lib().dsv4_attn_workspace_size(num_tokens, num_heads, compress_ratio, window, topk,
                                          max_seq_len, num_splits)


def dsv4_attn_get_device_error(stream=None):
    v = ctypes.c_uint32()
    _check(lib().dsv4_attn_get_device_error(ctypes.byref(v), _stream(stream)))
    return v.value


def dsv4_attn_strerror(status):
    return lib().dsv4_attn_strerror(status).decode()


# ---------------------------------------------------------------- one call per workload
def dsv4_kv_store(k, req_rows, positions, pool, *, stream=None):
    """Store new key rows k (bf16 [n, 512]) into `pool` (a make_pool()
    descriptor) at logical row positions[i] of page-table row req_rows[i]
    (int32 [n] each), packing them to FP8 for a packed pool."""
    if k.dtype != torch.bfloat16 or k.dim() != 2 or k.shape[1] != 512 or not k.is_contiguous():
        raise Dsv4Error("k must be a contiguous bf16 [n, 512] tensor")
    n = k.shape[0]
    for name, x in (("req_rows", req_rows), ("positions", positions)):
        if x.dtype != torch.int32 or x.numel() != n or not x.is_contiguous():
            raise Dsv4Error(f"{name} must be a contiguous int32 tensor of {n} entries")
    _check(lib().dsv4_kv_store(_ptr(k), n, _ptr(req_rows), _ptr(positions), ctypes.byref(pool),
                               _stream(stream)))


def dsv4_topk_max_length(k):
    return lib().dsv4_topk_max_length(k)


def dsv4_topk(scores, lengths, k, *, max_length=None, out=None, stream=None):
    """Indices of the k best scores of every row (ascending, -1 padded):
    scores fp32 [rows, stride] (stride a multiple of 4), lengths int32 [rows]."""
    if scores.dtype != torch.float32 or scores.dim() != 2 or scores.stride(1) != 1:
        raise Dsv4Error("scores must be a row-major fp32 [rows, stride] tensor")
    rows = scores.shape[0]
    if lengths.dtype != torch.int32 or lengths.numel() != rows or not lengths.is_contiguous():
        raise Dsv4Error(f"lengths must be a contiguous int32 tensor of {rows} entries")
    if max_length is None:
        max_length = scores.shape[1]
    if out is None:
        out = _new_output((rows, k), torch.int32, scores.device, stream)
    _check(lib().dsv4_topk(_ptr(scores), rows, scores.stride(0), _ptr(lengths), max_length, k, _ptr(out),
                           _stream(stream)))
    return out


# ---------------------------------------------------------------- the grouped-query cache
_GQA_TYPES = {torch.bfloat16: DSV4_GQA_BF16, torch.float16: DSV4_GQA_F16, torch.float8_e4m3fn: DSV4_GQA_E4M3}


def make_gqa_cache(k_pages, v_pages, page_table, *, k_scale=None, v_scale=None):
    """dsv4_gqa_cache for K and V pools [pages, KV heads, page_size, head_dim]
    (bf16, f16 or float8_e4m3fn; any strides whose rows are contiguous, so
    token-major pages are passed as pages.transpose(1, 2)) and their int32
    page table [request rows, logical pages].  k_scale, v_scale: fp32
    [KV heads] of an e4m3 cache.  Keep the descriptor as long as the pools:
    building it costs more than passing it."""
    if k_pages.dim() != 4 or k_pages.dtype not in _GQA_TYPES:
        raise Dsv4Error("k_pages must be a [pages, KV heads, page_size, head_dim] tensor of bf16, f16 or float8_e4m3fn")
    if v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or v_pages.stride() != k_pages.stride():
        raise Dsv4Error("v_pages must have the shape, type and strides of k_pages")
    if k_pages.stride(3) != 1:
        raise Dsv4Error("the head_dim values of a cache row must be contiguous")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise Dsv4Error("page_table must be an int32 [request rows, logical pages] tensor with contiguous rows")
    pages, heads, page_size, dim = k_pages.shape
    for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
        if x is None:
            continue
        if k_pages.dtype != torch.float8_e4m3fn:
            raise Dsv4Error(f"{name} goes with a float8_e4m3fn cache")
        if x.dtype != torch.float32 or x.shape != (heads,) or not x.is_contiguous():
            raise Dsv4Error(f"{name} must be a contiguous fp32 tensor of {heads} entries")
    keep = (k_pages, v_pages, page_table, k_scale, v_scale)
    if any(x is not None and x.device != k_pages.device for x in keep):
        raise Dsv4Error("the tensors of a cache must be on one device")
    es = k_pages.element_size()
    c = GqaCache()
    c.k, c.v = k_pages.data_ptr(), v_pages.data_ptr()
    c.num_pages = pages
    # (a dimension of one entry may have any stride)
    c.page_stride, c.head_stride, c.row_stride = (k_pages.stride(i) * es if k_pages.shape[i] > 1 else 0
                                                  for i in range(3))
    c.page_table = page_table.data_ptr()
    c.page_table_rows, c.page_table_width = page_table.shape
    c.page_table_stride = page_table.stride(0) if page_table.shape[0] > 1 else page_table.shape[1]
    c.num_kv_heads, c.head_dim, c.page_size = heads, dim, page_size
    c.format = _GQA_TYPES[k_pages.dtype]
    c.k_scale = None if k_scale is None else k_scale.data_ptr()
    c.v_scale = None if v_scale is None else v_scale.data_ptr()
    c._keep = keep
    c._ref = ctypes.addressof(c)
    lib()                       # (a descriptor is only good for the library's calls)
    c._index = k_pages.get_device()
    c._rows = torch.Size((heads, dim))
    c._slots = min(page_table.shape[1] * page_size, 1 << 30)     # (a call's bound on lengths)
    c._scale = 1.0 / math.sqrt(dim)
    return c


# The checks below are one expression per call where nothing is wrong; which
# of them failed is worked out only then (a decode step's calls are bound by
# the host).
def _is(x, dtype, n, index):
    return x.dtype is dtype and x.numel() == n and x.is_contiguous() and x.get_device() == index


def _need(x, name, dtype, n, index):
    """x is a contiguous `dtype` tensor of n entries on the cache's device."""
    if not _is(x, dtype, n, index):
        raise Dsv4Error(f"{name} must be a contiguous {dtype} tensor of {n} entries on the cache's device")


def _width(name, x, dtype, cache):
    """The width of a [request rows, KV heads, width] contiguous tensor."""
    if x.dim() == 3:
        rows, heads, width = x.shape
        if x.dtype is dtype and rows == cache.page_table_rows and heads == cache.num_kv_heads and x.is_contiguous() \
                and x.get_device() == cache._index:
            return width
    raise Dsv4Error(f"{name} must be a contiguous {dtype} [{cache.page_table_rows}, {cache.num_kv_heads}, width] tensor "
                    "on the cache's device")


def _raw_stream(stream, index):
    """The stream's handle; the cache's device has to be the current one, as for every launch."""
    if index < 0 or index != torch._C._cuda_getDevice():
        raise Dsv4Error("the cache must be on the current CUDA device")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _scratch(workspace, need, cache, stream):
    if workspace is None:
        workspace = _new(need, torch.uint8, cache._keep[0].device, stream)
    elif not workspace.is_contiguous() or workspace.get_device() != cache._index:
        raise Dsv4Error("workspace must be a contiguous tensor on the cache's device")
    return workspace, workspace.numel() * workspace.element_size()


def _gqa_type(x, cache):
    """The type code of q, k or v for this cache."""
    t = _GQA_TYPES.get(x.dtype, DSV4_GQA_E4M3)
    if t == DSV4_GQA_E4M3 or (cache.format != t and cache.format != DSV4_GQA_E4M3):
        raise Dsv4Error("rows must be bf16 or f16, and have the cache's type unless that is float8_e4m3fn")
    return t


def dsv4_gqa_store(k, v, req_rows, slots, cache, *, weights=None, positions=None, token_positions=None, stream=None):
    """Write new rows k, v ([n, KV heads, head_dim], bf16 or f16, rows
    contiguous) to slot slots[i] of page-table row req_rows[i] (int32 [n]
    each), packed for an e4m3 cache.  weights (fp32 [request rows, KV heads,
    width]) starts at 0 there, positions (int32, same shape) at
    token_positions[i]."""
    index = cache._index
    if k.dim() != 3 or v.dim() != 3:
        raise Dsv4Error("k and v must be [n, KV heads, head_dim] tensors")
    shape = k.shape
    n = shape[0]
    kt, kh, k1 = k.stride()
    vt, vh, v1 = v.stride()
    type_ = _gqa_type(k, cache)
    if shape[1:] != cache._rows or v.shape != shape or v.dtype is not k.dtype or k1 != 1 or v1 != 1 \
            or k.get_device() != index or v.get_device() != index:
        raise Dsv4Error(f"k and v must be {[n, cache.num_kv_heads, cache.head_dim]} tensors of one type with contiguous "
                        "rows on the cache's device")
    if n <= 1 or cache.num_kv_heads == 1:         # a dimension of one entry may have any stride
        kt, vt = (0, 0) if n <= 1 else (kt, vt)
        kh, vh = (0, 0) if cache.num_kv_heads == 1 else (kh, vh)
    _need(req_rows, "req_rows", torch.int32, n, index)
    _need(slots, "slots", torch.int32, n, index)
    wp = pp = tp = None
    width = 0
    if weights is not None:
        width = _width("weights", weights, torch.float32, cache)
        wp = weights.data_ptr()
    if positions is not None and token_positions is not None:
        w2 = _width("positions", positions, torch.int32, cache)
        if wp is not None and w2 != width:
            raise Dsv4Error("weights and positions must have one width")
        width = w2
        _need(token_positions, "token_positions", torch.int32, n, index)
        pp, tp = positions.data_ptr(), token_positions.data_ptr()
    elif positions is not None or token_positions is not None:
        raise Dsv4Error("positions and token_positions go together")
    rc = _lib.dsv4_gqa_store(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, type_, n, req_rows.data_ptr(),
                             slots.data_ptr(), cache._ref, wp, pp, width, tp, _raw_stream(stream, index))
    if rc:
        _check(rc)


def dsv4_gqa_decode_workspace_size(cache, batch, num_heads, max_len=None, weights=False):
    return lib().dsv4_gqa_decode_workspace_size(cache._ref, batch, num_heads,
                                                cache._slots if max_len is None else max_len, int(weights))


def dsv4_gqa_decode(q, lens, cache, *, sink=None, scale=None, window=0, max_len=None, req_pool_indices=None,
                    weights=None, weights_out=None, decay=1.0, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per request over its cached rows: q
    [batch, heads, head_dim] (bf16 or f16; a slice of a wider projection is
    fine), lens int32 [batch].  Returns (out, lse).  With weights (fp32
    [request rows, KV heads, width]) every cached row's weight is accumulated
    into weights_out, by default in place.  max_len: a bound on lens, by default
    every slot of the page table; the smaller, the fewer launches and (with
    weights) the smaller the workspace."""
    index = cache._index
    type_ = _gqa_type(q, cache)
    if q.dim() != 3 or q.get_device() != index:
        raise Dsv4Error("q must be a [batch, heads, head_dim] tensor on the cache's device")
    batch, heads, dim = q.shape
    qs, q2, q1 = q.stride()
    if dim != cache.head_dim or q1 != 1 or (q2 != dim and heads > 1):
        raise Dsv4Error(f"q's rows must be heads of {cache.head_dim} contiguous values, one behind the other")
    _need(lens, "lens", torch.int32, batch, index)
    rp = None
    if req_pool_indices is not None:
        _need(req_pool_indices, "req_pool_indices", torch.int32, batch, index)
        rp = req_pool_indices.data_ptr()
    elif batch > cache.page_table_rows:
        raise Dsv4Error("without req_pool_indices the page table needs a row for every request")
    sp = None
    if sink is not None:
        _need(sink, "sink", torch.float32, heads, index)
        sp = sink.data_ptr()
    if max_len is None:
        max_len = cache._slots
    wp = op = None
    width = 0
    if weights is not None:
        width = _width("weights", weights, torch.float32, cache)
        wp = op = weights.data_ptr()
        if weights_out is not None:
            if _width("weights_out", weights_out, torch.float32, cache) != width:
                raise Dsv4Error("weights and weights_out must have one width")
            op = weights_out.data_ptr()
        if max_len > width:
            raise Dsv4Error("weights must be at least max_len wide")
    elif weights_out is not None:
        raise Dsv4Error("weights_out goes with weights")
    if out is None:
        out = _new_output((batch, heads, dim), q.dtype, q.device, stream)
    elif out.shape != q.shape or not _is(out, q.dtype, batch * heads * dim, index):
        raise Dsv4Error("out must be a contiguous tensor like q")
    if lse is None:
        lse = _new_output((batch, heads), torch.float32, q.device, stream)
    else:
        _need(lse, "lse", torch.float32, batch * heads, index)
    if batch == 0:
        return out, lse
    need = 0 if workspace is not None else dsv4_gqa_decode_workspace_size(cache, batch, heads, max_len, wp is not None)
    workspace, have = _scratch(workspace, need, cache, stream)
    rc = _lib.dsv4_gqa_decode(q.data_ptr(), qs if batch > 1 else heads * dim, type_, batch, heads, lens.data_ptr(), rp,
                              cache._ref, window, max_len, sp, cache._scale if scale is None else scale, wp, op, width,
                              decay, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), have,
                              _raw_stream(stream, index))
    if rc:
        _check(rc)
    return out, lse


def dsv4_gqa_evict_workspace_size(cache, batch, max_len, keep):
    return lib().dsv4_gqa_evict_workspace_size(cache._ref, batch, cache._slots if max_len is None else max_len, keep)


def dsv4_gqa_evict(lens, cache, weights, keep, *, seq_lens=None, positions=None, first=0, recent=0,
                   req_pool_indices=None, max_len=None, weights_out=None, positions_out=None, lens_out=None,
                   workspace=None, stream=None):
    """Cut every request with more than `keep` cached rows (lens int32
    [batch]) to the `keep` that matter per KV head: positions below `first`,
    the `recent` newest of seq_lens tokens, then the largest weights.  Rows
    that stay but stand behind the bound move into the freed slots, with their
    weights and positions (in place unless weights_out / positions_out are
    given).  Returns lens_out (a new tensor unless given; may be lens
    or seq_lens).  max_len: a bound on lens, by default every slot there is; one
    launch does it all where max_len - keep <= 4 and lens_out is a tensor of its
    own."""
    index = cache._index
    batch = lens.numel()
    _need(lens, "lens", torch.int32, batch, index)
    np_ = rp = None
    if seq_lens is not None:
        _need(seq_lens, "seq_lens", torch.int32, batch, index)
        np_ = seq_lens.data_ptr()
    if req_pool_indices is not None:
        _need(req_pool_indices, "req_pool_indices", torch.int32, batch, index)
        rp = req_pool_indices.data_ptr()
    elif batch > cache.page_table_rows:
        raise Dsv4Error("without req_pool_indices the page table needs a row for every request")
    width = _width("weights", weights, torch.float32, cache)
    wp = op = weights.data_ptr()
    same = True
    if weights_out is not None:
        same = _width("weights_out", weights_out, torch.float32, cache) == width
        op = weights_out.data_ptr()
    pp = qp = None
    if positions is not None:
        same = same and _width("positions", positions, torch.int32, cache) == width
        pp = qp = positions.data_ptr()
        if positions_out is not None:
            same = same and _width("positions_out", positions_out, torch.int32, cache) == width
            qp = positions_out.data_ptr()
    elif positions_out is not None:
        raise Dsv4Error("positions_out goes with positions")
    if not same:
        raise Dsv4Error("weights and positions must have one width")
    if max_len is None:
        max_len = min(cache._slots, width)
    if max_len > width:
        raise Dsv4Error("weights must be at least max_len wide")
    if lens_out is None:
        lens_out = _new_output(lens.shape, torch.int32, lens.device, stream)
    else:
        _need(lens_out, "lens_out", torch.int32, batch, index)
    if batch == 0:
        return lens_out
    need = 0 if workspace is not None else dsv4_gqa_evict_workspace_size(cache, batch, max_len, keep)
    workspace, have = _scratch(workspace, need, cache, stream)
    rc = _lib.dsv4_gqa_evict(batch, lens.data_ptr(), np_, rp, cache._ref, max_len, keep, first, recent, wp, op, pp, qp,
                             width, lens_out.data_ptr(), workspace.data_ptr(), have, _raw_stream(stream, index))
    if rc:
        _check(rc)
    return lens_out


def run_inputs(inp, *, num_splits=0, debug_rows=None, out=None, lse=None, workspace=None, stream=None):
    """Dispatch a synth.Inputs batch (already on the GPU) to the matching entry point."""
    w = inp.work
    swa = make_pool(inp.swa_pool, inp.swa_page_table)
    kw = dict(scale=inp.scale, window=w.window, req_pool_indices=inp.req_pool_indices, out=out,
              lse=lse, num_splits=num_splits, workspace=workspace, debug_rows=debug_rows, stream=stream)
    extra = None if inp.extra_pool is None else make_pool(inp.extra_pool, inp.extra_page_table)
    if inp.cu_seqlens_q is not None:
        return dsv4_attn_verify(inp.q, inp.seq_lens, inp.cu_seqlens_q, swa, inp.sink,
                                compress_ratio=w.ratio, batch=w.batch, extra_pool=extra,
                                topk_idx=inp.topk_idx, max_seq_len=inp.max_seq_len, **kw)
    if w.ratio == 0:
        return dsv4_attn_swa(inp.q, inp.seq_lens, swa, inp.sink, **kw)
    if w.ratio == 4:
        return dsv4_attn_c4_sparse(inp.q, inp.seq_lens, swa, extra, inp.topk_idx, inp.sink, **kw)
    return dsv4_attn_c128_dense(inp.q, inp.seq_lens, swa, extra, inp.sink,
                                max_seq_len=inp.max_seq_len, **kw)


def debug_stride_for(inp):
    w = inp.work
    return debug_stride(w.ratio, w.window, w.topk if w.ratio == 4 else 0, inp.max_seq_len)
