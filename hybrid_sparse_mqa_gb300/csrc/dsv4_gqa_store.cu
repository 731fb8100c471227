// dsv4_gqa_store.cu - the write of new K and V rows into a grouped-query
// cache (include/dsv4gqa.h states what is computed).
//
// How: a block stores one head of K or of V for a run of tokens, so that rows
// of consecutive slots are written as one contiguous stretch; blocks that run
// together cover all heads of the same tokens, whose rows lie side by side in
// the input.  A thread moves 16 values of each of kItems tokens (two 16-byte
// loads; 32 bytes stored, or 16 e4m3 codes), all loads and then all page-table
// loads before the first store: three round trips per thread, over kItems
// times the bytes.  Bound by HBM: 2 bytes read and 2 (or 1) written per value.
// 65536 tokens of 8 heads of 128: 83 us as bf16 (537 MB, 6.5 TB/s), 79 us as
// e4m3 (402 MB, 5.1 TB/s: the conversions keep the issue slots 60 % busy).
// kItems and kStoreThreads are the best of 1 to 4 and 128, 256 (80 to 93 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsv4_gqa.cuh"

namespace dsv4 {
namespace gqa {
namespace {

constexpr int kStoreThreads = 128;
constexpr int kItems = 2;                  // tokens per thread
// Blocks of 16 values of a token that a thread takes: two of a 4-bit cache, whose codes cost the issue slots so much that
// the token's addresses should not be worked out for every block: 64 x 1024 tokens
// written and read back 120 us, 130 with one block, 118 with four blocks of one token, which leaves lanes of 64-wide rows far
// apart.
template <int FORMAT>
constexpr int kBlocks = FORMAT == DSV4_GQA_E2M1 ? 2 : 1;

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
template <int TYPE>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    if constexpr (TYPE == DSV4_GQA_BF16) {
        return pack_bf16x2(lo, hi);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// Two fp32 values in one 64-bit register (each lane of a packed operation
// rounds as the scalar one does).
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint32_t e4m3x2(float2 q) {
    return __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
}

// The pair w clamped to +-lim (lim: the type's bits, twice), NaN kept.
template <int TYPE>
__device__ __forceinline__ uint32_t clamp2(uint32_t w, uint32_t lim) {
    const uint32_t neg = lim ^ 0x80008000u;
    if constexpr (TYPE == DSV4_GQA_BF16) {
        __nv_bfloat162 x = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&lim));
        x = __hmax2_nan(x, *reinterpret_cast<const __nv_bfloat162*>(&neg));
        return *reinterpret_cast<uint32_t*>(&x);
    } else {
        __half2 x = __hmin2_nan(*reinterpret_cast<__half2*>(&w), *reinterpret_cast<const __half2*>(&lim));
        x = __hmax2_nan(x, *reinterpret_cast<const __half2*>(&neg));
        return *reinterpret_cast<uint32_t*>(&x);
    }
}

// What the codes of one head need: its scale, and whether the quotients can
// be had without dividing.
template <int TYPE>
struct Packer {
    float scale;
    bool fast;
    uint32_t lim;                          // 512 scale, as a pair of the input's type
    uint64_t ny2, s2;                      // -RN(1 / scale) and scale, twice

    __device__ __forceinline__ explicit Packer(float s) : scale(s) {
        fast = TYPE == DSV4_GQA_BF16 ? s >= 0x1p-60f && s <= 0x1p60f : s >= 0x1p-23f && s <= 127.f;
        const float y = -__frcp_rn(s), l = 512.f * s;
        lim = narrow<TYPE>(l, l);
        ny2 = f32x2(y, y);
        s2 = f32x2(s, s);
    }

    // The e4m3 codes of 16 values: of the correctly rounded fp32 quotients
    // x / scale, nearest code, ties to even, saturating.  Fast path: values
    // are first clamped to 512 scale (beyond 448 scale every code saturates),
    // so nothing overflows, then one Markstein correction of q0 = x y with
    // y = RN(1 / scale) gives the correctly rounded quotient (residuals are
    // exact where a code depends on them: quotients below 2^-11 have code 0
    // either way).  Worked on n = -x: q0 = n (-y), r = q0 scale + n,
    // q = r (-y) + q0, whose zeros have the sign of x.  Dividing instead took
    // 19 instructions a value and 114 us for 64 x 1024 tokens of 8 heads; this
    // takes about 5, and the kernel is bound by memory.
    __device__ __forceinline__ uint4 codes16(uint4 a, uint4 b) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t c[8];
        if (fast) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 n = widen<TYPE>(clamp2<TYPE>(w[j], lim) ^ 0x80008000u);
                const uint64_t n2 = f32x2(n.x, n.y);
                const uint64_t q0 = mul_f32x2(n2, ny2);
                const uint64_t q = fma_f32x2(fma_f32x2(q0, s2, n2), ny2, q0);
                float2 v;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(q));
                c[j] = e4m3x2(v);
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                const float2 x = widen<TYPE>(w[j]);
                c[j] = e4m3x2(make_float2(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale)));
            }
        }
        return make_uint4(c[0] | c[1] << 16, c[2] | c[3] << 16, c[4] | c[5] << 16, c[6] | c[7] << 16);
    }
};

// max(|x|, |y|) of two pairs, NaN kept; the sign is any.
template <int TYPE>
__device__ __forceinline__ uint32_t abs_max2(uint32_t x, uint32_t y) {
    uint32_t r;
    if constexpr (TYPE == DSV4_GQA_BF16)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
// An e4m3 code -> float, exactly.
__device__ __forceinline__ float e4m3_f32(uint32_t code) {
    uint32_t h;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(code));
    return __low2float(*reinterpret_cast<const __half2*>(&h));
}
// Eight values -> eight e2m1 codes (to nearest, ties to even, saturating), the first in the lowest half byte.
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&v)[4]) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
    return r;
}

// The same for 4-bit codes: a thread's 16 values are one block.  The block's
// scale by one division; the codes of the correctly rounded quotients by one
// Markstein correction of x y, y = RN(1 / step), as above.  There the bounds on
// the head's scale keep the step (2^-9 to 448 times it) where nothing over- or
// underflows that a code depends on: a block's values are at most 9 steps, or
// where the largest step is too small for them clamped to 8 first (6.x and more
// saturate); quotients below 1/4 have code 0 either way.
template <int TYPE>
struct BlockPacker {
    float scale;
    bool fast;

    __device__ __forceinline__ explicit BlockPacker(float s) : scale(s) {
        fast = TYPE == DSV4_GQA_BF16 ? s >= 0x1p-60f && s <= 0x1p60f : s >= 0x1p-14f && s <= 16.f;
    }
    // codes of the block's 16 values; returns the e4m3 code of its scale
    __device__ __forceinline__ uint32_t codes16(uint4 a, uint4 b, uint2& codes) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = abs_max2<TYPE>(w[0], w[1]);
#pragma unroll
        for (int j = 2; j < 8; ++j) m = abs_max2<TYPE>(m, w[j]);
        const float top = fabsf(widen<TYPE>(abs_max2<TYPE>(m, m >> 16)).x);
        const uint32_t code = e4m3x2(make_float2(__fdiv_rn(top, 6.f * scale), 0.f)) & 0xffu;
        const float step = e4m3_f32(code) * scale;
        uint32_t c[2];
        if (fast) {
            const float y = __frcp_rn(step);
            uint32_t x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = w[j];
            if (code == 0x7eu) {                   // (else no value has more than 9 steps)
                const uint32_t lim = narrow<TYPE>(8.f * step, 8.f * step);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = clamp2<TYPE>(w[j], lim);
            }
            const uint64_t ny2 = f32x2(-y, -y), s2 = f32x2(step, step);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float2 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 n = widen<TYPE>(x[4 * i + j] ^ 0x80008000u);
                    const uint64_t n2 = f32x2(n.x, n.y);
                    const uint64_t q0 = mul_f32x2(n2, ny2);
                    const uint64_t q = fma_f32x2(fma_f32x2(q0, s2, n2), ny2, q0);
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(v[j].x), "=f"(v[j].y) : "l"(q));
                }
                c[i] = e2m1x8(v);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                float2 v[4];
                for (int j = 0; j < 4; ++j) {
                    const float2 x = widen<TYPE>(w[4 * i + j]);
                    v[j] = make_float2(__fdiv_rn(x.x, step), __fdiv_rn(x.y, step));
                }
                c[i] = e2m1x8(v);
            }
        }
        const bool any = step > 0.f;              // (no scale, or a NaN)
        codes = make_uint2(any ? c[0] : 0u, any ? c[1] : 0u);
        return code;
    }
};

// FORMAT: of the cache; TYPE: of the rows (BF16 for a plain copy of either).
template <int TYPE, int FORMAT, int PIECES>
__global__ void __launch_bounds__(kStoreThreads) dsv4_gqa_store_kernel(const __grid_constant__ StoreParams p) {
    constexpr int kB = kBlocks<FORMAT>, kLanes = PIECES / kB, kTokens = kStoreThreads / kLanes;        // of one item
    grid_dependency_wait();
    grid_dependents_go();
    const int heads2 = 2 * p.c.kv_heads;
    const int hw = blockIdx.x % heads2, which = hw & 1, h = hw >> 1;
    const int piece = threadIdx.x % kLanes;      // and those kLanes further on
    const int i0 = blockIdx.x / heads2 * (kTokens * kItems) + threadIdx.x / kLanes;
    uint4 a[kItems][kB], b[kItems][kB];
    int r[kItems], s[kItems], page[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = i0 + k * kTokens;
        r[k] = s[k] = -1;
        if (i < p.n) {
            const uint4* src = reinterpret_cast<const uint4*>(p.src[which] + i * p.token_stride[which] +
                                                              h * p.head_stride[which]) + 2 * piece;
            r[k] = __ldg(p.req_rows + i);
            s[k] = __ldg(p.slots + i);
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                a[k][u] = __ldcs(src + 2 * kLanes * u);
                b[k][u] = __ldcs(src + 2 * kLanes * u + 1);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        page[k] = -1;
        const int lp = s[k] >> p.c.page_shift;
        if (r[k] >= 0 && r[k] < p.c.table_rows && s[k] >= 0 && lp < p.table_width && s[k] < p.width)
            page[k] = __ldg(p.c.table + (long long)r[k] * p.c.table_stride + lp);
    }
    float scale = 1.f;
    if constexpr (FORMAT != TYPE) {
        const float* scales = which ? p.c.v_scale : p.c.k_scale;
        if (scales) scale = __ldg(scales + h);
    }
    const Packer<TYPE> pack(scale);
    const BlockPacker<TYPE> pack_block(scale);
    uint8_t* pool = (which ? p.c.v : p.c.k) + h * p.c.head_stride;
    uint8_t* blocks = (which ? p.c.vb : p.c.kb) + h * p.c.b_head_stride;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = i0 + k * kTokens;
        if (i >= p.n) break;
        if (page[k] < 0 || page[k] >= p.c.num_pages) {
            if (piece == 0) atomicOr(p.err, DSV4_DEV_ERR_STORE_ROW);
            continue;
        }
        const int in_page = s[k] & ((1 << p.c.page_shift) - 1);
        uint4* dst = reinterpret_cast<uint4*>(pool + page[k] * p.c.page_stride + in_page * p.c.row_stride);
        if constexpr (FORMAT == DSV4_GQA_E2M1) {
            uint8_t* scales = blocks + page[k] * p.c.b_page_stride + in_page * p.c.b_row_stride + piece;
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                uint2 codes;
                scales[kLanes * u] = static_cast<uint8_t>(pack_block.codes16(a[k][u], b[k][u], codes));
                reinterpret_cast<uint2*>(dst)[piece + kLanes * u] = codes;
            }
        } else if constexpr (FORMAT == DSV4_GQA_E4M3) {
            dst[piece] = pack.codes16(a[k][0], b[k][0]);
        } else {
            dst[2 * piece] = a[k][0];
            dst[2 * piece + 1] = b[k][0];
        }
        if (piece == 0 && which == 0) {
            const long long t = ((long long)r[k] * p.c.kv_heads + h) * p.width + s[k];
            if (p.weights) p.weights[t] = 0.f;
            if (p.positions) p.positions[t] = __ldg(p.token_positions + i);
        }
    }
}

template <int TYPE, int FORMAT>
int launch_store(const StoreParams& p, int head_dim, void* stream) {
    const int tokens = kStoreThreads / (head_dim / 16) * kBlocks<FORMAT> * kItems;
    const long long blocks = ((long long)p.n + tokens - 1) / tokens * 2 * p.c.kv_heads;
    if (blocks > 0x7fffffffLL) return DSV4_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (head_dim == 64) return launch(dsv4_gqa_store_kernel<TYPE, FORMAT, 4>, grid, kStoreThreads, 0, stream, 1, p);
    if (head_dim == 128) return launch(dsv4_gqa_store_kernel<TYPE, FORMAT, 8>, grid, kStoreThreads, 0, stream, 1, p);
    return launch(dsv4_gqa_store_kernel<TYPE, FORMAT, 16>, grid, kStoreThreads, 0, stream, 1, p);
}

template <int TYPE, int FORMAT>
bool load_store() {
    return load_kernels(dsv4_gqa_store_kernel<TYPE, FORMAT, 4>, dsv4_gqa_store_kernel<TYPE, FORMAT, 8>,
                        dsv4_gqa_store_kernel<TYPE, FORMAT, 16>);
}
int load_all() {
    static unsigned long long ready = 0;
    return once_per_device(ready, [] {
        return load_store<DSV4_GQA_BF16, DSV4_GQA_BF16>() && load_store<DSV4_GQA_BF16, DSV4_GQA_E4M3>() &&
               load_store<DSV4_GQA_F16, DSV4_GQA_E4M3>() && load_store<DSV4_GQA_BF16, DSV4_GQA_E2M1>() &&
               load_store<DSV4_GQA_F16, DSV4_GQA_E2M1>();
    });
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
    int rc = check_cache(cache);
    if (rc) return rc;
    if (n < 0 || n > kMostSlots) return DSV4_ERR_INVALID;
    if (!type_fits(cache, type)) return DSV4_ERR_UNSUPPORTED;
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
    rc = load_all();
    if (rc) return rc;
    const int d = cache->head_dim;
    if (cache->format == type) return launch_store<DSV4_GQA_BF16, DSV4_GQA_BF16>(p, d, stream);
    if (cache->format == DSV4_GQA_E4M3)
        return type == DSV4_GQA_BF16 ? launch_store<DSV4_GQA_BF16, DSV4_GQA_E4M3>(p, d, stream)
                                     : launch_store<DSV4_GQA_F16, DSV4_GQA_E4M3>(p, d, stream);
    return type == DSV4_GQA_BF16 ? launch_store<DSV4_GQA_BF16, DSV4_GQA_E2M1>(p, d, stream)
                                 : launch_store<DSV4_GQA_F16, DSV4_GQA_E2M1>(p, d, stream);
}
