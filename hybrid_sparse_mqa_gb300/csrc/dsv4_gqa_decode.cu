// dsv4_gqa_decode.cu - host side of the one-token attention over a paged
// grouped-query cache, and the two kernels behind the attention kernel
// (dsv4_gqa_decode.cuh): the join of split requests and the accumulation of
// weights.
#include "dsv4_gqa_decode.cuh"

namespace dsv4 {
namespace gqa {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kWeightThreads = 256;
constexpr int kWeightSlots = 4;            // slots per thread

// Joins the pieces of split segments: block (segment, n-tile of 8 heads).
// With M = max_i m_i, out = sum_i 2^(m_i - M) o_i / (sum_i 2^(m_i - M) l_i +
// sink term).  Every block finds its segment's tiles from the lengths, as the
// attention kernel did.  Requests without rows get their output here.
template <int D, int TT, int HEADS>
__global__ void __launch_bounds__(kJoinThreads) dsv4_gqa_join_kernel(const __grid_constant__ DecodeParams p) {
    __shared__ unsigned s_sum[2][kJoinThreads / 32];
    __shared__ int s_near[2][kJoinThreads / 32];
    __shared__ float s_w[kMaxCtas][8];
    __shared__ float2 s_ml[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hcs = p.c.kv_heads * p.chunks;
    const int b = blockIdx.x / hcs, hc = blockIdx.x % hcs;
    grid_dependency_wait();
    grid_dependents_go();

    unsigned err = 0, before = 0, total = 0;
    int next = 0x7fffffff, earlier = 0;
    const Request rq = read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err);
    const Range rg = key_range<TT>(p, rq.n);
    const bool link = p.info && hc == 0 && blockIdx.y == 0;
    for (int e = tid; e < p.batch; e += kJoinThreads) {
        const Request x = read_request(p.lens, p.req, p.c.table_rows, p.max_len, e, err);
        const unsigned cnt = key_range<TT>(p, x.n).tiles * hcs;
        total += cnt;
        if (e < b) before += cnt;
        if (link && x.n > 0 && x.row == rq.row) {
            if (e < b) earlier = 1;
            if (e > b) next = min(next, e);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
        next = min(next, __shfl_xor_sync(0xffffffffu, next, o));
        earlier |= __shfl_xor_sync(0xffffffffu, earlier, o);
    }
    if (lane == 0) {
        s_sum[0][warp] = before;
        s_sum[1][warp] = total;
        s_near[0][warp] = next;
        s_near[1][warp] = earlier;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        before += s_sum[0][w];
        total += s_sum[1][w];
        next = min(next, s_near[0][w]);
        earlier |= s_near[1][w];
    }
    if (link && tid == 0)
        p.info[b] = make_int4(static_cast<int>(before), next == 0x7fffffff ? -1 : next, !earlier, rq.n);

    const int h = hc / p.chunks, chunk = hc % p.chunks;
    const int first = chunk * HEADS + blockIdx.y * 8;          // in the KV head's group
    const int nheads = min(8, p.group - first);
    if (nheads <= 0) return;
    const int head0 = h * p.group + first;
    uint16_t* out = static_cast<uint16_t*>(p.out) + ((size_t)b * p.heads + head0) * D;
    if (rg.tiles == 0) {
        for (int e = tid; e < nheads * D / 4; e += kJoinThreads) reinterpret_cast<uint2*>(out)[e] = make_uint2(0u, 0u);
        if (tid < nheads) {
            const float l2 = p.sink ? __ldg(p.sink + head0 + tid) * kLog2e : -INFINITY;
            if (p.lse) p.lse[(size_t)b * p.heads + head0 + tid] = l2 * kLn2;
            if (p.lse2) p.lse2[(size_t)b * p.heads + head0 + tid] = l2;
        }
        return;
    }
    const int ctas = share_count(p, total);
    const unsigned seg = before + hc * rg.tiles;
    const int c0 = share_of(total, ctas, seg), c1 = share_of(total, ctas, seg + rg.tiles - 1);
    if (c0 == c1) return;
    const int pieces = c1 - c0 + 1;
    // warp w: head w
    if (warp < nheads) {
        const float2* ml = p.part_ml + blockIdx.y * 8 + warp;
        float mx = kNoMax, l = 0.f;
        for (int i = lane; i < pieces; i += 32) mx = fmaxf(mx, ml[(size_t)(2 * (c0 + i) + (i == 0)) * HEADS].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        for (int i = lane; i < pieces; i += 32) {
            const float2 x = ml[(size_t)(2 * (c0 + i) + (i == 0)) * HEADS];
            const float f = fast_exp2(x.x - mx);
            s_w[i][warp] = f;
            l += f * x.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            const float sk = p.sink ? __ldg(p.sink + head0 + warp) * kLog2e : -INFINITY;
            const float top = fmaxf(mx, sk);
            const float f = fast_exp2(mx - top);
            l = l * f + fast_exp2(sk - top);
            const float vmul = p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f;
            const bool any = l > 0.f || l != l;
            s_ml[warp] = make_float2(any ? vmul * f / l : 0.f, 0.f);
            const float l2 = any ? top + log2f(l) : -INFINITY;
            if (p.lse) p.lse[(size_t)b * p.heads + head0 + warp] = l2 * kLn2;
            if (p.lse2) p.lse2[(size_t)b * p.heads + head0 + warp] = l2;
        }
    }
    __syncthreads();
    for (int e = tid; e < nheads * D / 4; e += kJoinThreads) {
        const int c = e / (D / 4);
        const float* at = p.part_o + (size_t)(2 * c0) * HEADS * D + (size_t)blockIdx.y * 8 * D + e * 4;
        constexpr size_t kStep = 2 * (size_t)HEADS * D;
        const float4 x0 = *reinterpret_cast<const float4*>(at + kStep / 2);
        const float f0 = s_w[0][c];
        float4 a = make_float4(x0.x * f0, x0.y * f0, x0.z * f0, x0.w * f0);
#pragma unroll 8
        for (int i = 1; i < pieces; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(at + i * kStep);
            const float f = s_w[i][c];
            a.x += x.x * f; a.y += x.y * f; a.z += x.z * f; a.w += x.w * f;
        }
        const float inv = s_ml[c].x;
        reinterpret_cast<uint2*>(out)[e] =
            p.q_bf16 ? make_uint2(pack2<true>(a.x * inv, a.y * inv), pack2<true>(a.z * inv, a.w * inv))
                     : make_uint2(pack2<false>(a.x * inv, a.y * inv), pack2<false>(a.z * inv, a.w * inv));
    }
}

// weights_out[r][h][j] = decay weights[r][h][j] + sum over requests of row r
// and heads i of h of 2^(score_ij - lse_i), in the order of requests, chunks
// and heads: block (slots, request, KV head), one thread per slot, no
// atomics.  Bound by memory: HEADS x 4 bytes of scores and 8 of weights per
// slot.
template <int TT, int HEADS>
__global__ void __launch_bounds__(kWeightThreads) dsv4_gqa_weight_kernel(const __grid_constant__ DecodeParams p) {
    __shared__ float s_lse[64 + 16];
    const int tid = threadIdx.x;
    const int b = blockIdx.y / p.c.kv_heads, h = blockIdx.y % p.c.kv_heads;
    const int slot0 = blockIdx.x * kWeightThreads * kWeightSlots + tid;
    grid_dependency_wait();
    grid_dependents_go();
    int4 info = p.info[b];
    if (!info.z || info.w == 0) return;
    unsigned err = 0;
    const int row = read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err).row;
    float acc[kWeightSlots] = {};
    int most = 0;
    for (int e = b;;) {
        const Range rg = key_range<TT>(p, info.w);
        most = max(most, rg.n);
        if (blockIdx.x * kWeightThreads * kWeightSlots < rg.n) {
            __syncthreads();
            if (tid < p.chunks * HEADS) {
                // +inf makes a head contribute nothing: padding, and heads none of whose rows could be read
                const float l = tid < p.group ? p.lse2[(size_t)e * p.heads + h * p.group + tid] : INFINITY;
                s_lse[tid] = l == -INFINITY ? INFINITY : l;
            }
            __syncthreads();
            for (int ch = 0; ch < p.chunks; ++ch) {
                const unsigned seg = static_cast<unsigned>(info.x) + (h * p.chunks + ch) * rg.tiles;
                const float* base = p.logits + ((size_t)seg * TT - rg.lo / TT * TT) * HEADS;
#pragma unroll
                for (int k = 0; k < kWeightSlots; ++k) {
                    const int slot = slot0 + k * kWeightThreads;
                    if (slot < rg.lo || slot >= rg.n) continue;
                    const float4* x = reinterpret_cast<const float4*>(base + (size_t)slot * HEADS);
                    float4 y[HEADS / 4];
#pragma unroll
                    for (int i = 0; i < HEADS / 4; ++i) y[i] = __ldcs(x + i);
#pragma unroll
                    for (int i = 0; i < HEADS / 4; ++i) {
                        const float* l = s_lse + ch * HEADS + 4 * i;
                        acc[k] += fast_exp2(y[i].x - l[0]);
                        acc[k] += fast_exp2(y[i].y - l[1]);
                        acc[k] += fast_exp2(y[i].z - l[2]);
                        acc[k] += fast_exp2(y[i].w - l[3]);
                    }
                }
            }
        }
        if (info.y < 0) break;
        e = info.y;
        info = p.info[e];
    }
    const size_t at = ((size_t)row * p.c.kv_heads + h) * p.width;
#pragma unroll
    for (int k = 0; k < kWeightSlots; ++k) {
        const int slot = slot0 + k * kWeightThreads;
        if (slot < most) p.w_out[at + slot] = p.decay * p.w_in[at + slot] + acc[k];
    }
}

int tile_slots(int format, int head_dim) {
    const int rows = 4096 / (head_dim * (format == DSV4_GQA_E4M3 ? 1 : 2));
    return rows < 16 ? 16 : rows;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

struct Plan {
    int group, nt, chunks, tt;
    long long tiles;                       // bound on the tile list
    size_t part_o, part_ml, lse2, info, logits, bytes;      // offsets, size
};

// DSV4_OK and the plan, or why there is none.
int make_plan(const dsv4_gqa_cache* c, int batch, int heads, int max_len, bool weights, Plan& pl) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (batch < 1 || heads < 1 || heads % c->num_kv_heads || !max_len_fits(c, max_len)) return DSV4_ERR_INVALID;
    pl.group = heads / c->num_kv_heads;
    if (pl.group > 64) return DSV4_ERR_UNSUPPORTED;
    pl.nt = pl.group > 8 ? 2 : 1;
    pl.chunks = (pl.group + 8 * pl.nt - 1) / (8 * pl.nt);
    pl.tt = tile_slots(c->format, c->head_dim);
    const long long segments = (long long)batch * c->num_kv_heads * pl.chunks;
    pl.tiles = segments * ((max_len + pl.tt - 1) / pl.tt);
    if (pl.tiles >= 1LL << 31 || segments >= 1LL << 31) return DSV4_ERR_UNSUPPORTED;
    pl.part_o = 0;
    pl.part_ml = pl.part_o + up256(size_t(2) * kMaxCtas * 8 * pl.nt * c->head_dim * sizeof(float));
    pl.lse2 = pl.part_ml + up256(size_t(2) * kMaxCtas * 8 * pl.nt * sizeof(float2));
    pl.info = pl.lse2 + (weights ? up256(size_t(batch) * heads * sizeof(float)) : 0);
    pl.logits = pl.info + (weights ? up256(size_t(batch) * sizeof(int4)) : 0);
    pl.bytes = pl.logits + (weights ? size_t(pl.tiles) * pl.tt * 8 * pl.nt * sizeof(float) : 0);
    return DSV4_OK;
}

int sm_count() {
    static int counts[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = __atomic_load_n(&counts[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        __atomic_store_n(&counts[dev], n, __ATOMIC_RELAXED);
    }
    return n;
}

template <int D, int TT>
int launch_join(const DecodeParams& p, int nt, void* stream) {
    const unsigned segments = p.batch * p.c.kv_heads * p.chunks;
    return nt == 1 ? launch(dsv4_gqa_join_kernel<D, TT, 8>, dim3(segments, 1), kJoinThreads, 0, stream, 1, p)
                   : launch(dsv4_gqa_join_kernel<D, TT, 16>, dim3(segments, 2), kJoinThreads, 0, stream, 1, p);
}

template <int TT>
int launch_weights(const DecodeParams& p, int nt, void* stream) {
    constexpr int kSlots = kWeightThreads * kWeightSlots;
    const dim3 grid((p.max_len + kSlots - 1) / kSlots, p.batch * p.c.kv_heads);
    return nt == 1 ? launch(dsv4_gqa_weight_kernel<TT, 8>, grid, kWeightThreads, 0, stream, 1, p)
                   : launch(dsv4_gqa_weight_kernel<TT, 16>, grid, kWeightThreads, 0, stream, 1, p);
}

}  // namespace
}  // namespace gqa
}  // namespace dsv4

extern "C" {

size_t dsv4_gqa_decode_workspace_size(const dsv4_gqa_cache* cache, int32_t batch, int32_t num_heads, int32_t max_len,
                                      int32_t with_weights) {
    dsv4::gqa::Plan pl;
    return dsv4::gqa::make_plan(cache, batch, num_heads, max_len, with_weights != 0, pl) ? 0 : pl.bytes;
}

int dsv4_gqa_decode(const void* q, int64_t q_stride, int32_t type, int32_t batch, int32_t num_heads,
                    const int32_t* lens, const int32_t* req_pool_indices, const dsv4_gqa_cache* cache,
                    int32_t window, int32_t max_len, const float* sink, float scale, const float* weights,
                    float* weights_out, int64_t width, float decay, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
    using namespace dsv4;
    using namespace dsv4::gqa;
    Plan pl;
    int rc = make_plan(cache, batch, num_heads, max_len, weights_out != nullptr, pl);
    if (rc) return rc;
    if (type != DSV4_GQA_BF16 && type != DSV4_GQA_F16) return DSV4_ERR_UNSUPPORTED;
    if (cache->format != DSV4_GQA_E4M3 && cache->format != type) return DSV4_ERR_UNSUPPORTED;
    if (!q || !out || !lens || !aligned16(q) || !aligned16(out) || q_stride % 8 || window < 0) return DSV4_ERR_INVALID;
    if (!weights != !weights_out || (weights && width < max_len)) return DSV4_ERR_INVALID;
    // the weight kernel's grid holds (request, KV head) in its y dimension
    if (weights && (long long)batch * cache->num_kv_heads > 65535) return DSV4_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < pl.bytes) return DSV4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DSV4_ERR_INVALID;
    unsigned int* err = device_error_word();
    const int sms = sm_count();
    if (!err || !sms) return DSV4_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    DecodeParams p;
    p.c = device_cache(cache);
    p.q = q;
    p.q_stride = q_stride;
    p.q_bf16 = type == DSV4_GQA_BF16;
    p.batch = batch;
    p.heads = num_heads;
    p.group = pl.group;
    p.chunks = pl.chunks;
    p.lens = lens;
    p.req = req_pool_indices;
    p.window = window;
    p.max_len = max_len;
    p.sink = sink;
    p.scale_log2 = scale * kLog2e;
    p.out = out;
    p.lse = lse;
    p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
    p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
    p.lse2 = weights ? reinterpret_cast<float*>(ws + pl.lse2) : nullptr;
    p.info = weights ? reinterpret_cast<int4*>(ws + pl.info) : nullptr;
    p.logits = weights ? reinterpret_cast<float*>(ws + pl.logits) : nullptr;
    p.w_in = weights;
    p.w_out = weights_out;
    p.width = width;
    p.decay = decay;
    p.min_tiles = 4;
    const long long most = pl.tiles / p.min_tiles;
    const int grid = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    p.ctas = most < 1 ? 1 : (most < grid ? static_cast<int>(most) : grid);
    p.err = err;

    const int d = cache->head_dim;
    rc = cache->format == DSV4_GQA_BF16  ? launch_decode_bf16(p, d, pl.nt, stream)
         : cache->format == DSV4_GQA_F16 ? launch_decode_f16(p, d, pl.nt, stream)
                                         : launch_decode_e4m3(p, d, pl.nt, stream);
    if (rc) return rc;
    if (d == 64)
        rc = pl.tt == 32 ? launch_join<64, 32>(p, pl.nt, stream) : launch_join<64, 64>(p, pl.nt, stream);
    else if (d == 128)
        rc = pl.tt == 16 ? launch_join<128, 16>(p, pl.nt, stream) : launch_join<128, 32>(p, pl.nt, stream);
    else
        rc = launch_join<256, 16>(p, pl.nt, stream);
    if (rc || !weights) return rc;
    return pl.tt == 16   ? launch_weights<16>(p, pl.nt, stream)
           : pl.tt == 32 ? launch_weights<32>(p, pl.nt, stream)
                         : launch_weights<64>(p, pl.nt, stream);
}

}  // extern "C"
