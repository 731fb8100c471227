// dsv4_gqa_decode.cu - host side of the one-token attention over a paged
// grouped-query cache, and the two kernels behind the attention kernel
// (dsv4_gqa_decode.cuh): the join of split requests and the accumulation of
// weights.
#include <algorithm>
#include <atomic>

#include "dsv4_gqa_decode.cuh"

namespace dsv4 {
namespace gqa {
namespace {

constexpr int kWeightThreads = 256;
constexpr int kWeightSlots = 4;            // slots per thread
// Tiles per share at least: 1 where no segment has more than kFewTiles, else 2.
// Lists as short as that are shared out only for calls with weights that name
// request rows or have more than 16 heads per KV head (all others take a
// cluster per segment).  us with 1 and with 2, weights and rows named: 1 x 8 KV
// heads of 100 rows 8.1 and 9.6, of 333 8.9 and 9.8, of 512 9.25 and 9.4; 8 x
// 512 12.3 and 12.0; 64 x 512 34.9 and 34.8; one KV head of 64 heads, 333 rows,
// 11.1 and 12.9.
constexpr int kFewTiles = 32;

// Joins the pieces of cut segments.  With M = max_i m_i,
//   out = sum_i 2^(m_i - M) o_i / (sum_i 2^(m_i - M) l_i + sink term).
// Block (segment, 8 / PW heads or one, slice of D / SLICES dims): PW warps per
// head share its pieces, so that a long segment's many pieces are read at once,
// and short segments do not cost a block per head (PW = 1).  Every block finds
// its segment's tiles from the lengths, as the attention kernel did; that part
// runs before the wait for it (the attention kernel itself starts behind the
// call's inputs, and only then lets this one go).  Requests without rows get
// their output here.  Bound by latency: a round trip for the lengths, one per
// batch of pieces.
template <int D, int TT, int HEADS, int PW, int SLICES>
__global__ void __launch_bounds__(PW > 8 ? PW * 32 : 256) dsv4_gqa_join_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int kHeads = PW < 8 ? 8 / PW : 1;              // per block
    constexpr int kThreads = PW * kHeads * 32;
    constexpr int DS = D / SLICES, V = DS / 32;              // dims of the block, values per lane
    __shared__ unsigned s_sum[2][kThreads / 32];
    __shared__ int s_near[2][kThreads / 32];
    __shared__ float2 s_ml[PW * kHeads];
    __shared__ float s_o[PW > 1 ? PW : 1][PW > 1 ? DS : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hcs = p.c.kv_heads * p.chunks;
    const int b = blockIdx.x / hcs, hc = blockIdx.x % hcs;

    unsigned err = 0, before = 0, total = 0;
    int next = 0x7fffffff, earlier = 0;
    const Request rq = read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err);
    const Range rg = key_range<TT>(p, rq.n);
    const bool link = p.info && hc == 0 && blockIdx.y == 0 && blockIdx.z == 0;
    for (int e = tid; e < p.batch; e += kThreads) {
        const Request x = read_request(p.lens, p.req, p.c.table_rows, p.max_len, e, err);
        const unsigned cnt = key_range<TT>(p, x.n).tiles * hcs;
        total += cnt;
        if (e < b) before += cnt;
        if (link && x.n > 0 && x.row == rq.row) {
            if (e < b) earlier = 1;
            if (e > b) next = min(next, e);
        }
    }
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    if (link) {
        next = __reduce_min_sync(0xffffffffu, next);
        earlier = __reduce_or_sync(0xffffffffu, earlier);
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
    for (int w = 0; w < kThreads / 32; ++w) {
        before += s_sum[0][w];
        total += s_sum[1][w];
        next = min(next, s_near[0][w]);
        earlier |= s_near[1][w];
    }
    int c0 = 0, c1 = 0;
    if (rg.tiles > 0) {
        const Shares shares = make_shares(p, total);
        const unsigned seg = before + hc * rg.tiles;
        c0 = share_of(shares, seg);
        c1 = share_of(shares, seg + rg.tiles - 1);
    }
    grid_dependency_wait();
    grid_dependents_go();
    if (link && tid == 0)
        p.info[b] = make_int4(static_cast<int>(before), next == 0x7fffffff ? -1 : next, !earlier, rq.n);

    const int h = hc / p.chunks, chunk = hc % p.chunks;
    const int head = blockIdx.y * kHeads + warp / PW;          // in the segment
    const bool mine = chunk * HEADS + head < p.group;
    const size_t at = (size_t)b * p.heads + h * p.group + chunk * HEADS + head;
    const int d0 = SLICES > 1 ? blockIdx.z * DS : 0;
    uint16_t* out = static_cast<uint16_t*>(p.out) + at * D + d0 + lane * V;
    const float sk = p.sink && mine ? __ldg(p.sink + h * p.group + chunk * HEADS + head) * kLog2e : -INFINITY;
    if (rg.tiles == 0) {
        if (mine && warp % PW == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = 0;
            if (lane == 0 && d0 == 0) {
                if (p.lse) p.lse[at] = sk * kLn2;
                if (p.lse2) p.lse2[at] = sk;
            }
        }
        return;
    }
    if (c0 == c1) return;
    const int pieces = c1 - c0 + 1;
    float a[V] = {}, mx = kNoMax, l = 0.f;
    if (mine) {
        // this warp's pieces, kBatch at a time; the reference moves between batches
        constexpr int kBatch = V > 4 ? 4 : V > 1 ? 8 : 16;
        for (int i0 = warp % PW; i0 < pieces; i0 += PW * kBatch) {
            float2 ml[kBatch];
            float x[kBatch][V];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * PW;
                ml[k] = make_float2(kNoMax, 0.f);
                if (i < pieces) {
                    const size_t e = (size_t)piece_entry(c0 + i, i == 0) * HEADS + head;
                    ml[k] = p.part_ml[e];
                    const float* from = p.part_o + e * D + d0 + lane * V;
                    if constexpr (V == 1) {
                        x[k][0] = *from;
                    } else if constexpr (V == 2) {
                        const float2 y = *reinterpret_cast<const float2*>(from);
                        x[k][0] = y.x; x[k][1] = y.y;
                    } else {
#pragma unroll
                        for (int q = 0; q < V; q += 4) {
                            const float4 y = *reinterpret_cast<const float4*>(from + q);
                            x[k][q] = y.x; x[k][q + 1] = y.y; x[k][q + 2] = y.z; x[k][q + 3] = y.w;
                        }
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < V; ++q) x[k][q] = 0.f;
                }
            }
            float top = mx;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
            const float f = fast_exp2(mx - top);
            mx = top;
            l *= f;
#pragma unroll
            for (int q = 0; q < V; ++q) a[q] *= f;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float w = fast_exp2(ml[k].x - top);
                l += w * ml[k].y;
#pragma unroll
                for (int q = 0; q < V; ++q) a[q] += w * x[k][q];
            }
        }
    }
    if constexpr (PW > 1) {
        // dims over the block's first D threads, each adding up its dim of all warps
        if (lane == 0) s_ml[warp] = make_float2(mx, l);
#pragma unroll
        for (int q = 0; q < V; ++q) s_o[warp][lane * V + q] = a[q];
        __syncthreads();
        if (tid >= DS || !mine) return;
        mx = kNoMax;
#pragma unroll
        for (int w = 0; w < PW; ++w) mx = fmaxf(mx, s_ml[w].x);
        l = 0.f;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < PW; ++w) {
            const float f = fast_exp2(s_ml[w].x - mx);
            l += f * s_ml[w].y;
            x += f * s_o[w][tid];
        }
        const float top = fminf(fmaxf(mx, sk), 3e38f);
        const float f = fast_exp2(mx - top);
        l = l * f + fast_exp2(sk - top);
        const bool any = l > 0.f || l != l;
        x *= any ? (p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f) * f / l : 0.f;
        const uint32_t w2 = p.q_bf16 ? pack2<true>(x, 0.f) : pack2<false>(x, 0.f);
        static_cast<uint16_t*>(p.out)[at * D + d0 + tid] = static_cast<uint16_t>(w2);
        if (tid == 0 && d0 == 0) {
            const float l2 = any ? top + log2f(l) : -INFINITY;
            if (p.lse) p.lse[at] = l2 * kLn2;
            if (p.lse2) p.lse2[at] = l2;
        }
        return;
    }
    if (!mine) return;
    const float top = fminf(fmaxf(mx, sk), 3e38f);
    const float f = fast_exp2(mx - top);
    l = l * f + fast_exp2(sk - top);
    const bool any = l > 0.f || l != l;
    const float inv = any ? (p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f) * f / l : 0.f;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float x = a[2 * i] * inv, y = a[2 * i + 1] * inv;
        reinterpret_cast<uint32_t*>(out)[i] = p.q_bf16 ? pack2<true>(x, y) : pack2<false>(x, y);
    }
    if (lane == 0) {
        const float l2 = any ? top + log2f(l) : -INFINITY;
        if (p.lse) p.lse[at] = l2 * kLn2;
        if (p.lse2) p.lse2[at] = l2;
    }
}

// weights_out[r][h][j] = decay weights[r][h][j] + sum over requests of row r
// and heads i of h of 2^(score_ij - lse_i), in the order of requests, chunks
// and heads: block (slots, request, KV head), one thread per slot, no
// atomics.  Bound by memory: HEADS x 4 bytes of scores and 8 of weights per
// slot.
template <int TT, int HEADS>
__global__ void __launch_bounds__(kWeightThreads) dsv4_gqa_weight_kernel(const __grid_constant__ DecodeParams p) {
    __shared__ __align__(16) float s_lse[64 + 16];
    const int tid = threadIdx.x;
    const int b = blockIdx.y / p.c.kv_heads, h = blockIdx.y % p.c.kv_heads;
    const int slot0 = blockIdx.x * kWeightThreads * kWeightSlots + tid;
    grid_dependency_wait();
    grid_dependents_go();
    int4 info = p.info[b];
    if (!info.z || info.w == 0) return;
    unsigned err = 0;
    const int row = read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err).row;
    const size_t at = ((size_t)row * p.c.kv_heads + h) * p.width;
    // each request's first slots of every chunk are on their way while the lse of its heads is fetched
    float prior[kWeightSlots], acc[kWeightSlots] = {};
#pragma unroll
    for (int k = 0; k < kWeightSlots; ++k) {
        const int slot = slot0 + k * kWeightThreads;
        prior[k] = slot < p.max_len ? __ldcs(p.w_in + at + slot) : 0.f;
    }
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
            for (int ch = 0; ch < p.chunks; ++ch) {
                const unsigned seg = static_cast<unsigned>(info.x) + (h * p.chunks + ch) * rg.tiles;
                const float* base = p.logits + ((size_t)seg * TT - rg.lo / TT * TT) * HEADS;
                float4 y[kWeightSlots][HEADS / 4];
#pragma unroll
                for (int k = 0; k < kWeightSlots; ++k) {
                    const int slot = slot0 + k * kWeightThreads;
                    const bool in = slot >= rg.lo && slot < rg.n;
                    const float4* x = reinterpret_cast<const float4*>(base + (size_t)slot * HEADS);
#pragma unroll
                    for (int i = 0; i < HEADS / 4; ++i)
                        y[k][i] = in ? __ldcs(x + i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                }
                if (ch == 0) __syncthreads();
#pragma unroll
                for (int i = 0; i < HEADS / 4; ++i) {
                    const float4 l = *reinterpret_cast<const float4*>(s_lse + ch * HEADS + 4 * i);
#pragma unroll
                    for (int k = 0; k < kWeightSlots; ++k)
                        acc[k] += (fast_exp2(y[k][i].x - l.x) + fast_exp2(y[k][i].y - l.y)) +
                                  (fast_exp2(y[k][i].z - l.z) + fast_exp2(y[k][i].w - l.w));
                }
            }
        }
        if (info.y < 0) break;
        e = info.y;
        info = p.info[e];
    }
#pragma unroll
    for (int k = 0; k < kWeightSlots; ++k) {
        const int slot = slot0 + k * kWeightThreads;
        if (slot < most) p.w_out[at + slot] = p.decay * prior[k] + acc[k];
    }
}

int tile_slots(int format, int head_dim) {
    const int rows = 4096 / (head_dim * (format == DSV4_GQA_E4M3 ? 1 : 2));
    return rows < 16 ? 16 : rows;
}

std::atomic<int> g_claim_ahead{kClaimAhead}, g_claim_polls{kWaitLimit};

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

struct Plan {
    int group, nt, chunks, tt, min_tiles;
    long long tiles;                       // bound on the tile list
    int places;                            // CTAs that run at once
    int ctas, claims;                      // resident CTAs of the attention kernel, and claimable ones
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
    if (pl.tiles >= 1LL << 31 || segments > kMostSlots) return DSV4_ERR_UNSUPPORTED;
    // (512-byte rows: one CTA's ring fills an SM's shared memory)
    const int most = c->head_dim * (c->format == DSV4_GQA_E4M3 ? 1 : 2) > 256 ? kMaxCtas / 2 : kMaxCtas;
    pl.places = most;
    pl.min_tiles = (max_len + pl.tt - 1) / pl.tt <= kFewTiles ? 1 : 2;
    const long long want = pl.tiles / pl.min_tiles;
    pl.ctas = want < 1 ? 1 : (want < most ? static_cast<int>(want) : most);
    pl.claims = pl.ctas == most && pl.tiles >= (long long)most * kWarps * kClaimTiles ? most : 0;
    const size_t entries = size_t(2) * (pl.ctas + pl.claims) * kWarps * 8 * pl.nt;
    pl.part_o = 0;
    pl.part_ml = pl.part_o + up256(entries * c->head_dim * sizeof(float));
    pl.lse2 = pl.part_ml + up256(entries * sizeof(float2));
    pl.info = pl.lse2 + (weights ? up256(size_t(batch) * heads * sizeof(float)) : 0);
    pl.logits = pl.info + (weights ? up256(size_t(batch) * sizeof(int4)) : 0);
    pl.bytes = pl.logits + (weights ? size_t(pl.tiles) * pl.tt * 8 * pl.nt * sizeof(float) : 0);
    return DSV4_OK;
}

// CTAs per segment where every segment is done by a cluster of its own, or 0
// where the list is shared out.  Clusters are as large as run at once, and
// taken where they leave their warps few tiles of the longest segment: 8 where
// they do not fill the GPU or a second wave would be mostly empty, 16 where
// they run at once (a ragged batch then ends with its longest request), 32
// where the hardware hands them out in several waves.  In us, cluster and list:
//   1 request x 8 KV heads: 333 rows 5.0 and 6.7, 4000 rows 8.9 and 11.2, 10000
//   rows (not taken) 15.8 and 15.2; 1 KV head x 5000 rows (not taken) 9.9 and 8.0
//   8 x 1000..2000 rows 11.8 and 15.7; 64 x 4 KV heads of 100..4000 e4m3 rows,
//   31 tiles per warp (not taken), 37.3 and 33.2
//   40 x 1000 rows, 320 CTAs for 304 places (not taken), 36.5 and 32.1
//   64 x 1..2048 rows 48.8 and 51.9; 64 x 2000..2048 rows 79.2 and 88.8; 128 x
//   1..2048 rows 85.5 and 96.6; 48 x 16 heads of 64, up to 1024 rows 31.5 and 34.2
//   with weights, 1 x 333 rows 6.2 and 8.8, 8 x 500..1000 rows 9.3 and 14.6
int segment_cluster(const DecodeParams& p, const Plan& pl) {
    const long long segments = (long long)p.batch * p.c.kv_heads * p.chunks;
    const int span = p.window > 0 ? std::min<long long>(p.max_len, (long long)p.window + pl.tt) : p.max_len;
    const int tiles = (span + pl.tt - 1) / pl.tt;
    int c = 8;
    while (c > 1 && segments * c > pl.places) c /= 2;
    const long long ctas = segments * c;
    const int most = ctas < pl.places / 2 ? 8 : ctas <= pl.places ? 16 : ctas < pl.places * 14 / 10 ? 8 : 32;
    return tiles <= c * kWarps * most && ctas <= 0x7fffffffLL ? c : 0;
}

template <int D, int TT, int HEADS>
int launch_join_heads(const DecodeParams& p, void* stream) {
    const unsigned segments = p.batch * p.c.kv_heads * p.chunks;
    // pieces of a segment, if all are about as long, and blocks of one head each.  (us of a whole decode call with the
    // choice made and with the other: 1 segment x 131072 rows, 1216 pieces of 8 heads: slices 26.6, no slices 35.9;
    // 16 segments, 85 pieces: PW = 16 165, slices 171, PW = 1 180; 8 segments, 10 pieces: PW = 8 7.7, PW = 1 8.1;
    // 256 segments, 5 pieces: PW = 1 98, PW = 8 105)
    const unsigned pieces = p.pieces / segments + 1;
    const unsigned long long heads = (unsigned long long)segments * HEADS;
    if (pieces > 96 && heads <= 64)
        return launch(dsv4_gqa_join_kernel<D, TT, HEADS, 16, D / 32>, dim3(segments, HEADS, D / 32), 512, 0, stream, 1, p);
    if (pieces > 96)
        return launch(dsv4_gqa_join_kernel<D, TT, HEADS, 16, 1>, dim3(segments, HEADS), 512, 0, stream, 1, p);
    if (pieces > 8 && heads <= 1024)
        return launch(dsv4_gqa_join_kernel<D, TT, HEADS, 8, 1>, dim3(segments, HEADS), 256, 0, stream, 1, p);
    return launch(dsv4_gqa_join_kernel<D, TT, HEADS, 1, 1>, dim3(segments, HEADS / 8), 256, 0, stream, 1, p);
}

template <int D, int TT>
int launch_join(const DecodeParams& p, int nt, void* stream) {
    return nt == 1 ? launch_join_heads<D, TT, 8>(p, stream) : launch_join_heads<D, TT, 16>(p, stream);
}

template <int TT>
int launch_weights(const DecodeParams& p, int nt, void* stream) {
    constexpr int kSlots = kWeightThreads * kWeightSlots;
    const dim3 grid((p.max_len + kSlots - 1) / kSlots, p.batch * p.c.kv_heads);
    return nt == 1 ? launch(dsv4_gqa_weight_kernel<TT, 8>, grid, kWeightThreads, 0, stream, 1, p)
                   : launch(dsv4_gqa_weight_kernel<TT, 16>, grid, kWeightThreads, 0, stream, 1, p);
}

template <int D, int TT, int HEADS>
bool load_join_heads() {
    return load_kernels(dsv4_gqa_join_kernel<D, TT, HEADS, 16, D / 32>, dsv4_gqa_join_kernel<D, TT, HEADS, 16, 1>,
                        dsv4_gqa_join_kernel<D, TT, HEADS, 8, 1>, dsv4_gqa_join_kernel<D, TT, HEADS, 1, 1>,
                        dsv4_gqa_weight_kernel<TT, HEADS>);
}

// Every kernel behind the attention kernel for rows of this size, at the first call with such rows (one that takes a
// cluster per segment too).
template <int D, int TT>
int load_join() {
    static unsigned long long ready = 0;
    return once_per_device(ready, [] { return load_join_heads<D, TT, 8>() && load_join_heads<D, TT, 16>(); });
}
int load_joins(int d, int tt) {
    if (d == 64) return tt == 32 ? load_join<64, 32>() : load_join<64, 64>();
    if (d == 128) return tt == 16 ? load_join<128, 16>() : load_join<128, 32>();
    return load_join<256, 16>();
}

}  // namespace
}  // namespace gqa
}  // namespace dsv4

extern "C" {

void dsv4_gqa_test_claim_limits(int32_t ahead, int32_t polls) {
    dsv4::gqa::g_claim_ahead = ahead < 0 ? dsv4::gqa::kClaimAhead : ahead;
    dsv4::gqa::g_claim_polls = polls < 0 ? dsv4::gqa::kWaitLimit : polls;
}

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
    if (weights && !same_or_apart(weights, weights_out, row_array_bytes(cache, width))) return DSV4_ERR_INVALID;
    // the weight kernel's grid holds (request, KV head) in its y dimension
    if (weights && (long long)batch * cache->num_kv_heads > 65535) return DSV4_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < pl.bytes) return DSV4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DSV4_ERR_INVALID;
    unsigned int* err = device_error_word();
    if (!err) return DSV4_ERR_CUDA;
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
    p.min_tiles = pl.min_tiles;
    p.warps = pl.ctas * kWarps;
    p.claims = pl.claims;
    p.claim_ahead = g_claim_ahead.load(std::memory_order_relaxed);
    p.claim_polls = g_claim_polls.load(std::memory_order_relaxed);
    p.pieces = static_cast<int>(std::min<long long>(p.warps + p.claims * kWarps, pl.tiles / pl.min_tiles));
    // (with weights, requests may add to one row only through the list's kernels, and so may several chunks of heads)
    p.cluster = weights && (req_pool_indices || pl.chunks > 1) ? 0 : segment_cluster(p, pl);
    p.err = err;

    const int d = cache->head_dim;
    rc = load_joins(d, pl.tt);
    if (rc) return rc;
    rc = cache->format == DSV4_GQA_BF16  ? launch_decode_bf16(p, d, pl.nt, stream)
         : cache->format == DSV4_GQA_F16 ? launch_decode_f16(p, d, pl.nt, stream)
         : p.q_bf16                      ? launch_decode_e4m3(p, d, pl.nt, stream)
                                         : launch_decode_e4m3_f16(p, d, pl.nt, stream);
    if (rc || p.cluster) return rc;
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
