// dsv4_gqa_load.cu - rows of a grouped-query cache back as 16-bit rows
// (include/dsv4gqa.h states what is computed).
//
// How: the store's layout the other way round.  A block reads one head of K or
// of V for a run of tokens, so that consecutive slots are one contiguous
// stretch of a page; a thread takes 16 values of each of kItems tokens (32, 16
// or 8 bytes of codes, and a block scale), all page-table loads and then all
// rows before the first store.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dsv4_gqa.cuh"

namespace dsv4 {
namespace gqa {
namespace {

constexpr int kLoadThreads = 128;
constexpr int kItems = 2;                  // tokens per thread

struct LoadParams {
    Cache c;
    uint8_t* dst[2];                            // K, V
    long long token_stride[2], head_stride[2];  // bytes
    int n;
    const int* req_rows;
    const int* slots;
    int table_width;
    unsigned int* err;
};

// Two values in the output's type.
template <int TYPE>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    if constexpr (TYPE == DSV4_GQA_BF16) {
        return pack_bf16x2(lo, hi);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// Four pairs of f16 values, exactly, of eight e2m1 codes.
__device__ __forceinline__ void widen8(uint32_t codes, __half2 (&r)[4]) {
    uint32_t x[4];
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = *reinterpret_cast<const __half2*>(&x[i]);
}

// FORMAT: of the cache; TYPE: of the rows (BF16 for a plain copy of either).
template <int TYPE, int FORMAT, int PIECES>
__global__ void __launch_bounds__(kLoadThreads) dsv4_gqa_load_kernel(const __grid_constant__ LoadParams p) {
    constexpr int kTokens = kLoadThreads / PIECES;           // of one item
    grid_dependency_wait();
    grid_dependents_go();
    const int heads2 = 2 * p.c.kv_heads;
    const int hw = blockIdx.x % heads2, which = hw & 1, h = hw >> 1;
    const int piece = threadIdx.x % PIECES;
    const int i0 = blockIdx.x / heads2 * (kTokens * kItems) + threadIdx.x / PIECES;
    int s[kItems], page[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = i0 + k * kTokens;
        page[k] = -1;
        s[k] = 0;
        if (i >= p.n) continue;
        const int r = __ldg(p.req_rows + i);
        s[k] = __ldg(p.slots + i);
        const int lp = s[k] >> p.c.page_shift;
        if (r >= 0 && r < p.c.table_rows && s[k] >= 0 && lp < p.table_width)
            page[k] = __ldg(p.c.table + (long long)r * p.c.table_stride + lp);
    }
    float scale = 1.f;
    if constexpr (FORMAT != TYPE) {
        const float* scales = which ? p.c.v_scale : p.c.k_scale;
        if (scales) scale = __ldg(scales + h);
    }
    const uint8_t* pool = (which ? p.c.v : p.c.k) + h * p.c.head_stride;
    const uint8_t* blocks = (which ? p.c.vb : p.c.kb) + h * p.c.b_head_stride;
    uint4 a[kItems], b[kItems];
    uint32_t block[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
        block[k] = 0;
        if (page[k] < 0 || page[k] >= p.c.num_pages) {
            if (piece == 0 && i0 + k * kTokens < p.n) atomicOr(p.err, DSV4_DEV_ERR_LOAD_ROW);
            continue;
        }
        const int in_page = s[k] & ((1 << p.c.page_shift) - 1);
        const uint4* src = reinterpret_cast<const uint4*>(pool + page[k] * p.c.page_stride + in_page * p.c.row_stride);
        if constexpr (FORMAT == DSV4_GQA_E2M1) {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(src) + piece);
            a[k].x = x.x;
            a[k].y = x.y;
            block[k] = __ldg(blocks + page[k] * p.c.b_page_stride + in_page * p.c.b_row_stride + piece);
        } else if constexpr (FORMAT == DSV4_GQA_E4M3) {
            a[k] = __ldg(src + piece);
        } else {
            a[k] = __ldg(src + 2 * piece);
            b[k] = __ldg(src + 2 * piece + 1);
        }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = i0 + k * kTokens;
        if (i >= p.n) break;
        uint32_t w[8] = {a[k].x, a[k].y, a[k].z, a[k].w, b[k].x, b[k].y, b[k].z, b[k].w};
        if constexpr (FORMAT == DSV4_GQA_E2M1) {
            // code times block scale is exact in fp32, so is their product's way there; one rounding by the head's scale
            float f[4];
            e4m3x4_to_f32(block[k], f);
            const float step = f[0];
            __half2 x[8];
            widen8(a[k].x, *reinterpret_cast<__half2(*)[4]>(&x[0]));
            widen8(a[k].y, *reinterpret_cast<__half2(*)[4]>(&x[4]));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = __half22float2(x[j]);
                w[j] = narrow<TYPE>(v.x * step * scale, v.y * step * scale);
            }
        } else if constexpr (FORMAT == DSV4_GQA_E4M3) {
            const uint32_t c[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[4];
                e4m3x4_to_f32(c[j], f);
                w[2 * j] = narrow<TYPE>(f[0] * scale, f[1] * scale);
                w[2 * j + 1] = narrow<TYPE>(f[2] * scale, f[3] * scale);
            }
        }
        uint4* dst = reinterpret_cast<uint4*>(p.dst[which] + i * p.token_stride[which] + h * p.head_stride[which]) + 2 * piece;
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <int TYPE, int FORMAT>
int launch_load(const LoadParams& p, int head_dim, void* stream) {
    const int tokens = kLoadThreads / (head_dim / 16) * kItems;
    const long long blocks = ((long long)p.n + tokens - 1) / tokens * 2 * p.c.kv_heads;
    if (blocks > 0x7fffffffLL) return DSV4_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (head_dim == 64) return launch(dsv4_gqa_load_kernel<TYPE, FORMAT, 4>, grid, kLoadThreads, 0, stream, 1, p);
    if (head_dim == 128) return launch(dsv4_gqa_load_kernel<TYPE, FORMAT, 8>, grid, kLoadThreads, 0, stream, 1, p);
    return launch(dsv4_gqa_load_kernel<TYPE, FORMAT, 16>, grid, kLoadThreads, 0, stream, 1, p);
}

template <int TYPE, int FORMAT>
bool load_load() {
    return load_kernels(dsv4_gqa_load_kernel<TYPE, FORMAT, 4>, dsv4_gqa_load_kernel<TYPE, FORMAT, 8>,
                        dsv4_gqa_load_kernel<TYPE, FORMAT, 16>);
}
int load_all() {
    static unsigned long long ready = 0;
    return once_per_device(ready, [] {
        return load_load<DSV4_GQA_BF16, DSV4_GQA_BF16>() && load_load<DSV4_GQA_BF16, DSV4_GQA_E4M3>() &&
               load_load<DSV4_GQA_F16, DSV4_GQA_E4M3>() && load_load<DSV4_GQA_BF16, DSV4_GQA_E2M1>() &&
               load_load<DSV4_GQA_F16, DSV4_GQA_E2M1>();
    });
}

// Whether no two rows of `dim` values share memory: `count` entries each of
// dimensions that lie `stride` elements apart (multiples of 8, as dim is).
struct Dimension {
    long long count, stride;
};
bool rows_apart(Dimension a, Dimension b, Dimension c, long long dim) {
    Dimension d[3] = {a, b, c};
    std::sort(d, d + 3, [](const Dimension& x, const Dimension& y) { return x.stride < y.stride; });
    long long extent = dim;
    for (const Dimension& x : d) {
        if (x.count < 2) continue;
        if (x.stride < extent) return false;
        extent += (x.count - 1) * x.stride;
    }
    return true;
}

}  // namespace
}  // namespace gqa
}  // namespace dsv4

extern "C" int dsv4_gqa_load(const int32_t* req_rows, const int32_t* slots, int32_t n, const dsv4_gqa_cache* cache,
                             void* k, int64_t k_token_stride, int64_t k_head_stride, void* v, int64_t v_token_stride,
                             int64_t v_head_stride, int32_t type, void* stream) {
    using namespace dsv4;
    using namespace dsv4::gqa;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (n < 0 || n > kMostSlots) return DSV4_ERR_INVALID;
    if (!type_fits(cache, type)) return DSV4_ERR_UNSUPPORTED;
    if (n == 0) return DSV4_OK;
    if (!k || !v || !req_rows || !slots || !aligned16(k) || !aligned16(v)) return DSV4_ERR_INVALID;
    if (k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8) return DSV4_ERR_INVALID;
    // outputs whose rows overlap would be written in no order
    const long long heads = cache->num_kv_heads, dim = cache->head_dim;
    auto span = [&](__int128 token, __int128 head) { return 2 * ((n - 1) * token + (heads - 1) * head + dim); };
    if (span(k_token_stride, k_head_stride) >> 62 || span(v_token_stride, v_head_stride) >> 62) return DSV4_ERR_INVALID;
    if (!rows_apart({n, k_token_stride}, {heads, k_head_stride}, {1, 0}, dim) ||
        !rows_apart({n, v_token_stride}, {heads, v_head_stride}, {1, 0}, dim))
        return DSV4_ERR_INVALID;
    if (!apart(k, static_cast<size_t>(span(k_token_stride, k_head_stride)), v,
               static_cast<size_t>(span(v_token_stride, v_head_stride)))) {
        // interleaved: parts of one tensor, K and V a third dimension of it
        const long long off = static_cast<uint16_t*>(v) - static_cast<uint16_t*>(k);
        if ((n > 1 && k_token_stride != v_token_stride) || (heads > 1 && k_head_stride != v_head_stride) ||
            !rows_apart({n, k_token_stride}, {heads, k_head_stride}, {2, off < 0 ? -off : off}, dim))
            return DSV4_ERR_INVALID;
    }
    unsigned int* err = device_error_word();
    if (!err) return DSV4_ERR_CUDA;
    LoadParams p;
    p.c = device_cache(cache);
    p.dst[0] = static_cast<uint8_t*>(k);
    p.dst[1] = static_cast<uint8_t*>(v);
    p.token_stride[0] = 2 * k_token_stride;
    p.token_stride[1] = 2 * v_token_stride;
    p.head_stride[0] = 2 * k_head_stride;
    p.head_stride[1] = 2 * v_head_stride;
    p.n = n;
    p.req_rows = req_rows;
    p.slots = slots;
    p.table_width = cache->page_table_width;
    p.err = err;
    rc = load_all();
    if (rc) return rc;
    const int d = cache->head_dim;
    if (cache->format == type) return launch_load<DSV4_GQA_BF16, DSV4_GQA_BF16>(p, d, stream);
    if (cache->format == DSV4_GQA_E4M3)
        return type == DSV4_GQA_BF16 ? launch_load<DSV4_GQA_BF16, DSV4_GQA_E4M3>(p, d, stream)
                                     : launch_load<DSV4_GQA_F16, DSV4_GQA_E4M3>(p, d, stream);
    return type == DSV4_GQA_BF16 ? launch_load<DSV4_GQA_BF16, DSV4_GQA_E2M1>(p, d, stream)
                                 : launch_load<DSV4_GQA_F16, DSV4_GQA_E2M1>(p, d, stream);
}
