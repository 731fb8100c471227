// dsv4_gqa.cuh - what the grouped-query cache kernels share: the cache's
// layout as the kernels see it, the reading of a request's length and row,
// and the host-side checks (include/dsv4gqa.h states the rules).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "dsv4gqa.h"
#include "dsv4_device.cuh"
#include "dsv4_internal.h"

namespace dsv4 {
namespace gqa {

struct Cache {
    uint8_t* k;
    uint8_t* v;
    long long num_pages, page_stride, head_stride, row_stride;
    const int* table;
    int table_rows, table_stride;
    int kv_heads, page_shift;
    const float* k_scale;
    const float* v_scale;
};

// Request b as the kernels read it: its row of the tables and the number of
// its cached rows (0 for a row outside the table).
struct Request {
    int row, n;
};

// `err` collects DSV4_DEV_ERR_* bits.  A request without rows is not asked
// for its request row, so padded entries may hold anything there.
__device__ __forceinline__ Request read_request(const int* lens, const int* req, int table_rows, int max_len, int b,
                                                unsigned& err) {
    Request r;
    r.n = __ldg(lens + b);
    r.row = req ? __ldg(req + b) : b;
    if (r.n < 0 || r.n > max_len) {
        err |= DSV4_DEV_ERR_GQA_LENGTH;
        r.n = r.n < 0 ? 0 : max_len;
    }
    if (r.row < 0 || r.row >= table_rows) {
        if (r.n > 0) err |= DSV4_DEV_ERR_REQ_ROW;
        r.row = 0;
        r.n = 0;
    }
    return r;
}

inline Cache device_cache(const dsv4_gqa_cache* c) {
    Cache d;
    d.k = static_cast<uint8_t*>(c->k);
    d.v = static_cast<uint8_t*>(c->v);
    d.num_pages = c->num_pages;
    d.page_stride = c->page_stride;
    d.head_stride = c->head_stride;
    d.row_stride = c->row_stride;
    d.table = c->page_table;
    d.table_rows = c->page_table_rows;
    d.table_stride = c->page_table_stride;
    d.kv_heads = c->num_kv_heads;
    d.page_shift = 0;
    while ((1 << d.page_shift) < c->page_size) ++d.page_shift;
    d.k_scale = c->format == DSV4_GQA_E4M3 ? c->k_scale : nullptr;
    d.v_scale = c->format == DSV4_GQA_E4M3 ? c->v_scale : nullptr;
    return d;
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// [a, a + na) and [b, b + nb) bytes have none in common (null: nothing there).
inline bool apart(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return !a || !b || x + na <= y || y + nb <= x;
}

// An array and what replaces it: one and the same, or apart.
inline bool same_or_apart(const void* a, const void* b, size_t n) { return a == b || apart(a, n, b, n); }

// Bytes of a [request rows, KV heads, width] array of 4-byte entries.
inline size_t row_array_bytes(const dsv4_gqa_cache* c, int64_t width) {
    return size_t(c->page_table_rows) * c->num_kv_heads * width * 4;
}

// DSV4_OK, DSV4_ERR_INVALID or DSV4_ERR_UNSUPPORTED.
inline int check_cache(const dsv4_gqa_cache* c) {
    if (!c || !c->k || !c->v || !c->page_table || !aligned16(c->k) || !aligned16(c->v)) return DSV4_ERR_INVALID;
    if (c->num_pages < 1 || c->page_table_rows < 1 || c->page_table_width < 1 ||
        c->page_table_stride < c->page_table_width || c->num_kv_heads < 1)
        return DSV4_ERR_INVALID;
    if (c->page_stride % 16 || c->head_stride % 16 || c->row_stride % 16 || c->page_stride < 0 || c->head_stride < 0 ||
        c->row_stride < 0)
        return DSV4_ERR_INVALID;
    if (c->format != DSV4_GQA_BF16 && c->format != DSV4_GQA_F16 && c->format != DSV4_GQA_E4M3)
        return DSV4_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return DSV4_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) || c->num_kv_heads > 256)
        return DSV4_ERR_UNSUPPORTED;
    return DSV4_OK;
}

// Bound on lengths and on the tokens of a store: slots and tokens are ints, and
// a tile or a run of them may end up to 2^25 behind the last.
constexpr int kMostSlots = 1 << 30;

// 0 < max_len <= the slots that a request's table row addresses, and the bound.
inline bool max_len_fits(const dsv4_gqa_cache* c, int max_len) {
    return max_len >= 1 && max_len <= kMostSlots && max_len <= static_cast<long long>(c->page_table_width) * c->page_size;
}

// Launch on `stream` with programmatic stream serialisation (every kernel
// here waits for its predecessor before it touches memory) and an optional
// cluster along x.
template <typename... KA, typename... A>
inline int launch(void (*kernel)(KA...), dim3 grid, int threads, size_t smem, void* stream, int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return DSV4_ERR_CUDA;
    }
    return DSV4_OK;
}

// Loads kernels on the current device.  CUDA does so at a kernel's first launch
// otherwise, which a stream that is being captured does not take.
template <class... K>
inline bool load_kernels(K... kernels) {
    cudaFuncAttributes a;
    return ((cudaFuncGetAttributes(&a, kernels) == cudaSuccess) && ...);
}

// prepare() where the current device's bit of `ready` is not set yet (two
// threads at once may both do it).
template <class F>
inline int once_per_device(unsigned long long& ready, F&& prepare) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSV4_ERR_CUDA;
    if (__atomic_load_n(&ready, __ATOMIC_ACQUIRE) >> dev & 1) return DSV4_OK;
    if (!prepare()) {
        cudaGetLastError();
        return DSV4_ERR_CUDA;
    }
    __atomic_fetch_or(&ready, 1ull << dev, __ATOMIC_RELEASE);
    return DSV4_OK;
}

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace gqa
}  // namespace dsv4
