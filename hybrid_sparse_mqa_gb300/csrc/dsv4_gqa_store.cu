// dsv4_gqa_store.cu - the write of new K and V rows into a grouped-query
// cache (include/dsv4gqa.h states what is computed).
//
// How: the work is n x KV heads x 2 (K and V) rows of head_dim values.  A
// thread moves 16 values (two 16-byte loads; 32 bytes stored, or 16 e4m3
// codes), consecutive threads on consecutive pieces of a row, then heads,
// then tokens, so loads and stores are full lines.  Bound by HBM: 2 bytes
// read and 2 (or 1) written per value; the indices and the page-table entry
// are read through L1 by the threads of a token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsv4_gqa.cuh"

namespace dsv4 {
namespace gqa {
namespace {

constexpr int kStoreThreads = 256;

struct StoreParams {
    Cache c;
    const uint8_t* src[2];                      // K, V
    long long token_stride[2], head_stride[2];  // bytes
    int n;
    const int* req_rows;
    const int* slots;
    int table_width;
    float* weights;
    int* positions;
    long long width;
    const int* token_positions;
    unsigned int* err;
};

template <int TYPE>
__device__ __forceinline__ float2 widen(uint32_t w) {
    if constexpr (TYPE == DSV4_GQA_BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// e4m3 codes of two values: the fp32 quotient, nearest code, ties to even,
// saturating (one rounding to fp32, one to e4m3, as the header states).
template <int TYPE>
__device__ __forceinline__ uint32_t codes2(uint32_t w, float scale) {
    const float2 x = widen<TYPE>(w);
    return __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale)), __NV_SATFINITE,
                                    __NV_E4M3);
}

// One (tensor, token, head, 16-value piece) per thread.
template <int TYPE, bool PACK, int PIECES>
__global__ void __launch_bounds__(kStoreThreads) dsv4_gqa_store_kernel(const __grid_constant__ StoreParams p) {
    grid_dependency_wait();
    grid_dependents_go();
    const long long id = (long long)blockIdx.x * kStoreThreads + threadIdx.x;
    const int piece = static_cast<int>(id % PIECES);
    const long long rest = id / PIECES;
    const int h = static_cast<int>(rest % p.c.kv_heads);
    const long long both = rest / p.c.kv_heads;
    const int which = static_cast<int>(both & 1);
    const long long i = both >> 1;
    if (i >= p.n) return;
    const uint4* src = reinterpret_cast<const uint4*>(p.src[which] + i * p.token_stride[which] +
                                                      h * p.head_stride[which]) + 2 * piece;
    const uint4 a = __ldcs(src), b = __ldcs(src + 1);
    const int r = __ldg(p.req_rows + i), s = __ldg(p.slots + i);
    const int lp = s >> p.c.page_shift;
    int page = -1;
    if (r >= 0 && r < p.c.table_rows && s >= 0 && lp < p.table_width && s < p.width)
        page = __ldg(p.c.table + (long long)r * p.c.table_stride + lp);
    if (page < 0 || page >= p.c.num_pages) {
        if (piece == 0) atomicOr(p.err, DSV4_DEV_ERR_STORE_ROW);
        return;
    }
    const long long at = page * p.c.page_stride + h * p.c.head_stride +
                         (s & ((1 << p.c.page_shift) - 1)) * p.c.row_stride;
    uint4* dst = reinterpret_cast<uint4*>((which ? p.c.v : p.c.k) + at);
    if constexpr (PACK) {
        const float* scales = which ? p.c.v_scale : p.c.k_scale;
        const float scale = scales ? __ldg(scales + h) : 1.f;
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = codes2<TYPE>(w[2 * j], scale) | (codes2<TYPE>(w[2 * j + 1], scale) << 16);
        dst[piece] = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
        dst[2 * piece] = a;
        dst[2 * piece + 1] = b;
    }
    if (piece == 0 && which == 0) {
        const long long t = ((long long)r * p.c.kv_heads + h) * p.width + s;
        if (p.weights) p.weights[t] = 0.f;
        if (p.positions) p.positions[t] = __ldg(p.token_positions + i);
    }
}

template <int TYPE, bool PACK>
int launch_store(const StoreParams& p, int head_dim, void* stream) {
    const long long threads = (long long)p.n * 2 * p.c.kv_heads * (head_dim / 16);
    const long long blocks = (threads + kStoreThreads - 1) / kStoreThreads;
    if (blocks > 0x7fffffffLL) return DSV4_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (head_dim == 64) return launch(dsv4_gqa_store_kernel<TYPE, PACK, 4>, grid, kStoreThreads, 0, stream, 1, p);
    if (head_dim == 128) return launch(dsv4_gqa_store_kernel<TYPE, PACK, 8>, grid, kStoreThreads, 0, stream, 1, p);
    return launch(dsv4_gqa_store_kernel<TYPE, PACK, 16>, grid, kStoreThreads, 0, stream, 1, p);
}

}  // namespace
}  // namespace gqa
}  // namespace dsv4

extern "C" int dsv4_gqa_store(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                              int64_t v_token_stride, int64_t v_head_stride, int32_t type, int32_t n,
                              const int32_t* req_rows, const int32_t* slots, const dsv4_gqa_cache* cache,
                              float* weights, int32_t* positions, int64_t width, const int32_t* token_positions,
                              void* stream) {
    using namespace dsv4;
    using namespace dsv4::gqa;
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (n < 0) return DSV4_ERR_INVALID;
    if (type != DSV4_GQA_BF16 && type != DSV4_GQA_F16) return DSV4_ERR_UNSUPPORTED;
    if (cache->format != DSV4_GQA_E4M3 && cache->format != type) return DSV4_ERR_UNSUPPORTED;
    if (n == 0) return DSV4_OK;
    if (!k || !v || !req_rows || !slots || !aligned16(k) || !aligned16(v)) return DSV4_ERR_INVALID;
    if (k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8) return DSV4_ERR_INVALID;
    if ((positions && !token_positions) || ((weights || positions) && width < 1)) return DSV4_ERR_INVALID;
    unsigned int* err = device_error_word();
    if (!err) return DSV4_ERR_CUDA;
    StoreParams p;
    p.c = device_cache(cache);
    p.src[0] = static_cast<const uint8_t*>(k);
    p.src[1] = static_cast<const uint8_t*>(v);
    p.token_stride[0] = 2 * k_token_stride;
    p.token_stride[1] = 2 * v_token_stride;
    p.head_stride[0] = 2 * k_head_stride;
    p.head_stride[1] = 2 * v_head_stride;
    p.n = n;
    p.req_rows = req_rows;
    p.slots = slots;
    p.table_width = cache->page_table_width;
    p.weights = weights;
    p.positions = positions;
    p.width = weights || positions ? width : INT64_MAX;
    p.token_positions = token_positions;
    p.err = err;
    const int d = cache->head_dim;
    if (cache->format != DSV4_GQA_E4M3) return launch_store<DSV4_GQA_BF16, false>(p, d, stream);
    return type == DSV4_GQA_BF16 ? launch_store<DSV4_GQA_BF16, true>(p, d, stream)
                                 : launch_store<DSV4_GQA_F16, true>(p, d, stream);
}
