// dsv4_gqa_evict.cu - eviction from a grouped-query cache by accumulated
// weight (include/dsv4gqa.h states what is computed).
//
// Two kernels.  The select kernel gives every (request, KV head) to one
// cluster of 1 to 8 CTAs: weights become order-preserving 32-bit keys (held
// in shared memory where they fit), a radix select of 11 + 11 + 10 bits finds
// the key of the last row kept and how many rows of that very key stay, and
// one ordered pass lists the freed slots below `keep` and the kept rows
// behind it.  Histograms and counts are combined over the cluster through
// distributed shared memory; every count is exact and every order is that of
// the slots, so the result does not depend on timing.  The move kernel copies
// the listed rows: only rows that change their slot are read and written,
// each once.  It is bound by HBM (4 head_dim bytes x element size per moved
// row and direction); the select kernel by its passes over shared memory.
#include "dsv4_gqa.cuh"

namespace dsv4 {
namespace gqa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;              // rows per block of the move kernel
constexpr int kMaxCluster = 8;
constexpr int kKeysPerCta = 48 * 1024;     // keys that a CTA holds in shared memory, at most

struct EvictParams {
    Cache c;
    int batch;
    const int* lens;
    const int* seen;
    const int* req;
    int max_len, keep, first, recent;
    const float* w_in;
    float* w_out;
    const int* p_in;
    int* p_out;
    long long width;
    int* lens_out;
    int* counts;                           // [batch][KV heads] rows to move
    int* holes;                            // [batch][KV heads][most] their new slots
    int* movers;                           // [batch][KV heads][most] their slots
    int most;
    int cached;                            // keys per CTA that shared memory holds
    int row_pieces;                        // 16-byte pieces of a row
    unsigned int* err;
};

// Larger key = kept first.  Weights in numeric order (-0 = +0), NaN with
// -inf; guarded rows above everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

struct SelectShared {
    uint32_t hist[2][kBins];               // a CTA's histogram; the second for the next digit
    uint32_t warp_sum[kSelWarps];
    uint32_t count[2][4];                  // this CTA's ties / holes / movers, for the cluster
    uint32_t pick[2];                      // chosen bin, rows wanted in it
    int skip;
};

template <int CLUSTER>
__device__ __forceinline__ void lane_sync() {
    if constexpr (CLUSTER > 1)
        cluster_sync();
    else
        __syncthreads();
}

// Exclusive prefix of v over the block's threads, and the block's total.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sum, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        if (w < warp) base += warp_sum[w];
        total += warp_sum[w];
    }
    return base + incl - v;
}

template <int CLUSTER>
__global__ void __launch_bounds__(kSelThreads) dsv4_gqa_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelectShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int id = blockIdx.x / CLUSTER, rank = blockIdx.x % CLUSTER;
    const int b = id / p.c.kv_heads, h = id % p.c.kv_heads;
    grid_dependency_wait();
    grid_dependents_go();

    unsigned err = 0;
    const Request rq = read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err);
    const int seen = p.seen ? __ldg(p.seen + b) : rq.n;
    if (tid == 0) sh.skip = 0;
    __syncthreads();
    if (p.req && rq.n > 0) {                 // a row that an earlier request of the call names too
        for (int e = tid; e < b; e += kSelThreads) {
            unsigned ignored = 0;
            const Request x = read_request(p.lens, p.req, p.c.table_rows, p.max_len, e, ignored);
            if (x.n > 0 && x.row == rq.row) sh.skip = 1;
        }
        __syncthreads();
        if (sh.skip) err |= DSV4_DEV_ERR_REQ_ROW;
    }
    if (err && h == 0 && rank == 0 && tid == 0) atomicOr(p.err, err);

    const size_t at = ((size_t)rq.row * p.c.kv_heads + h) * p.width;
    const float* w_in = p.w_in + at;
    float* w_out = p.w_out + at;
    const int* p_in = p.p_in ? p.p_in + at : nullptr;
    int* p_out = p.p_out ? p.p_out + at : nullptr;
    const bool copy_w = w_in != w_out, copy_p = p_in != p_out;
    if (rq.n <= p.keep || sh.skip) {         // (uniform over the cluster)
        if (rank == 0 && tid == 0) p.counts[id] = 0;
        if ((copy_w || copy_p) && !sh.skip)
            for (int s = rank * kSelThreads + tid; s < rq.n; s += CLUSTER * kSelThreads) {
                if (copy_w) w_out[s] = w_in[s];
                if (copy_p) p_out[s] = p_in[s];
            }
        return;
    }

    // this CTA's slots, a multiple of 32 each
    const int n = rq.n;
    const int per = ((n + CLUSTER - 1) / CLUSTER + 31) & ~31;
    const int s0 = min(n, rank * per), s1 = min(n, s0 + per);
    const bool cached = s1 - s0 <= p.cached;
    auto make_key = [&](int s) -> uint32_t {
        const int pos = p_in ? __ldg(p_in + s) : s;
        if (pos < p.first || pos >= seen - p.recent) return 0xffffffffu;
        return weight_key(__ldg(w_in + s));
    };
    auto key = [&](int s) -> uint32_t { return cached ? keys[s - s0] : make_key(s); };
    for (int i = tid; i < 2 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    if (cached)
        for (int s = s0 + tid; s < s1; s += kSelThreads) keys[s - s0] = make_key(s);
    __syncthreads();

    // ---- the key of the last row kept: `want` rows of key `prefix` stay ----
    uint32_t prefix = 0, want = p.keep, equal = 0;
#pragma unroll
    for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
        const int bits = digit == 2 ? 10 : 11;
        uint32_t* hist = sh.hist[digit & 1];
        for (int s = s0 + tid; s < s1; s += kSelThreads) {
            const uint32_t k = key(s);
            if (digit == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits)))
                atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
        }
        lane_sync<CLUSTER>();
        // thread t: bins from the top, kBins / kSelThreads of them
        constexpr int kPer = kBins / kSelThreads;
        uint32_t mine[kPer], sum = 0;
        const int top = (1 << bits) - 1 - tid * kPer;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            mine[i] = 0;
            if (top - i >= 0) {
                const uint32_t a = smem_u32(&hist[top - i]);
                if constexpr (CLUSTER == 1) {
                    mine[i] = hist[top - i];
                } else {
#pragma unroll
                    for (int r = 0; r < CLUSTER; ++r) mine[i] += ld_cluster_u32(mapa(a, r));
                }
            }
            sum += mine[i];
        }
        uint32_t total;
        uint32_t above = block_exclusive(sum, sh.warp_sum, total);
        if (above < want && above + sum >= want) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (above < want && above + mine[i] >= want) {
                    sh.pick[0] = static_cast<uint32_t>(top - i);
                    sh.pick[1] = want - above;
                    sh.count[0][3] = mine[i];
                }
                above += mine[i];
            }
        }
        __syncthreads();
        prefix |= sh.pick[0] << shift;
        want = sh.pick[1];
        equal = sh.count[0][3];
        // the other histogram is ready for the next digit; this one is cleared once every
        // CTA of the cluster has read it (the next digit's barrier)
        if (digit == 1) {
            uint32_t* old = sh.hist[0];
            for (int i = tid; i < kBins; i += kSelThreads) old[i] = 0;
        }
        __syncthreads();
    }

    // ---- warp w of a CTA: a contiguous run of its slots, 32 at a time ----
    const int run = (((s1 - s0) + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int r0 = min(s1, s0 + warp * run), r1 = min(s1, r0 + run);
    const uint32_t below = (1u << lane) - 1u;
    // ranks of this warp's first element among the lane's ties
    uint32_t tie = 0;
    const bool every = equal == want;        // all rows of the last key stay
    if (!every) {
        uint32_t c = 0;
        for (int s = r0 + lane; s - lane < r1; s += 32)
            c += __popc(__ballot_sync(0xffffffffu, s < r1 && key(s) == prefix));
        uint32_t total;
        const uint32_t ex = block_exclusive(lane == 0 ? c : 0, sh.warp_sum, total);
        tie = __shfl_sync(0xffffffffu, ex, 0);
        if (tid == 0) sh.count[0][0] = total;
        lane_sync<CLUSTER>();
        if constexpr (CLUSTER > 1) {
            const uint32_t a = smem_u32(&sh.count[0][0]);
            for (int r = 0; r < rank; ++r) tie += ld_cluster_u32(mapa(a, r));
        }
    }
    auto walk = [&](auto&& visit) {          // visit(slot, kept, inside) for the warp's slots, ties resolved
        uint32_t t = tie;
        for (int s = r0 + lane; s - lane < r1; s += 32) {
            const bool in = s < r1;
            const uint32_t k = in ? key(s) : 0u;
            const bool same = in && k == prefix;
            bool kept = in && k > prefix;
            if (every) {
                kept |= same;
            } else {
                const unsigned m = __ballot_sync(0xffffffffu, same);
                kept |= same && t + __popc(m & below) < want;
                t += __popc(m);
            }
            visit(s, kept, in);
        }
    };
    uint32_t nh = 0, nm = 0;
    walk([&](int s, bool kept, bool in) {
        nh += __popc(__ballot_sync(0xffffffffu, in && !kept && s < p.keep));
        nm += __popc(__ballot_sync(0xffffffffu, kept && s >= p.keep));
    });
    uint32_t hole_total, move_total;
    uint32_t hole = block_exclusive(lane == 0 ? nh : 0, sh.warp_sum, hole_total);
    uint32_t move = block_exclusive(lane == 0 ? nm : 0, sh.warp_sum, move_total);
    hole = __shfl_sync(0xffffffffu, hole, 0);
    move = __shfl_sync(0xffffffffu, move, 0);
    if (tid == 0) {
        sh.count[1][0] = hole_total;
        sh.count[1][1] = move_total;
    }
    lane_sync<CLUSTER>();
    if constexpr (CLUSTER > 1) {
        const uint32_t a = smem_u32(&sh.count[1][0]);
        for (int r = 0; r < rank; ++r) {
            hole += ld_cluster_u32(mapa(a, r));
            move += ld_cluster_u32(mapa(a + 4, r));
        }
    }
    if (rank == CLUSTER - 1 && tid == 0) p.counts[id] = move + move_total;   // (warp 0's prefix is the ranks before)
    int* holes = p.holes + (size_t)id * p.most;
    int* movers = p.movers + (size_t)id * p.most;
    walk([&](int s, bool kept, bool in) {
        const bool is_hole = in && !kept && s < p.keep, is_move = kept && s >= p.keep;
        const unsigned mh = __ballot_sync(0xffffffffu, is_hole), mm = __ballot_sync(0xffffffffu, is_move);
        if (is_hole) holes[hole + __popc(mh & below)] = s;
        if (is_move) movers[move + __popc(mm & below)] = s;
        hole += __popc(mh);
        move += __popc(mm);
        if (kept && s < p.keep) {
            if (copy_w) w_out[s] = w_in[s];
            if (copy_p) p_out[s] = p_in[s];
        }
    });
    // no CTA of the cluster may end while another still reads its counts
    if constexpr (CLUSTER > 1) cluster_sync();
}

// Rows holes[j] <- movers[j]: block (32 rows, request and KV head).  A warp
// takes whole rows; K and V pieces of a row go to its lanes.
__global__ void __launch_bounds__(kMoveThreads) dsv4_gqa_move_kernel(const __grid_constant__ EvictParams p) {
    const int tid = threadIdx.x;
    const int id = blockIdx.y, b = id / p.c.kv_heads, h = id % p.c.kv_heads;
    grid_dependency_wait();
    grid_dependents_go();
    if (blockIdx.x == 0 && h == 0 && tid == 0) {
        int n = __ldg(p.lens + b);
        n = n < 0 ? 0 : n > p.max_len ? p.max_len : n;
        const int row = p.req ? __ldg(p.req + b) : b;
        if (row < 0 || row >= p.c.table_rows) n = 0;
        p.lens_out[b] = n < p.keep ? n : p.keep;
    }
    const int count = p.counts[id];
    const int j0 = blockIdx.x * kMoveRows, j1 = min(count, j0 + kMoveRows);
    if (j0 >= j1) return;
    const int row = p.req ? __ldg(p.req + b) : b;
    const int* table = p.c.table + (long long)row * p.c.table_stride;
    const int mask = (1 << p.c.page_shift) - 1;
    const int* holes = p.holes + (size_t)id * p.most;
    const int* movers = p.movers + (size_t)id * p.most;
    const size_t at = ((size_t)row * p.c.kv_heads + h) * p.width;
    const int pieces = 2 * p.row_pieces;                 // K, then V
    for (int e = tid; e < (j1 - j0) * pieces; e += kMoveThreads) {
        const int j = j0 + e / pieces, piece = e % pieces;
        const int dst = holes[j], src = movers[j];
        const int to = __ldg(table + (dst >> p.c.page_shift)), of = __ldg(table + (src >> p.c.page_shift));
        if (piece == 0) {
            if (p.w_out) p.w_out[at + dst] = p.w_in[at + src];
            if (p.p_out) p.p_out[at + dst] = p.p_in[at + src];
        }
        if (to < 0 || to >= p.c.num_pages || of < 0 || of >= p.c.num_pages) {
            if (piece == 0) atomicOr(p.err, DSV4_DEV_ERR_GQA_PAGE);
            continue;
        }
        uint8_t* pool = piece < p.row_pieces ? p.c.k : p.c.v;
        const int x = piece < p.row_pieces ? piece : piece - p.row_pieces;
        const long long head = h * p.c.head_stride + x * 16;
        *reinterpret_cast<uint4*>(pool + to * p.c.page_stride + (dst & mask) * p.c.row_stride + head) =
            __ldcs(reinterpret_cast<const uint4*>(pool + of * p.c.page_stride + (src & mask) * p.c.row_stride + head));
    }
}

// The rows that can move for one (request, KV head): at most those kept and
// at most those behind `keep`.
int most_moved(int max_len, int keep) {
    const int behind = max_len - keep;
    return behind < 1 ? 1 : (behind < keep ? behind : keep);
}

struct Layout {
    size_t counts, holes, movers, bytes;
};
int layout(const dsv4_gqa_cache* c, int batch, int max_len, int keep, Layout& l) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (batch < 1 || keep < 1 || !max_len_fits(c, max_len)) return DSV4_ERR_INVALID;
    const size_t ids = (size_t)batch * c->num_kv_heads;
    if (ids > 65535) return DSV4_ERR_UNSUPPORTED;
    const size_t list = (ids * most_moved(max_len, keep) * sizeof(int) + 255) & ~size_t(255);
    l.counts = 0;
    l.holes = (ids * sizeof(int) + 255) & ~size_t(255);
    l.movers = l.holes + list;
    l.bytes = l.movers + list;
    return DSV4_OK;
}

template <int CLUSTER>
int launch_select(const EvictParams& p, size_t smem, void* stream) {
    static unsigned long long ready = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSV4_ERR_CUDA;
    if (!(__atomic_load_n(&ready, __ATOMIC_ACQUIRE) >> dev & 1)) {
        if (cudaFuncSetAttribute(dsv4_gqa_select_kernel<CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kKeysPerCta * 4) != cudaSuccess) {
            cudaGetLastError();
            return DSV4_ERR_CUDA;
        }
        __atomic_fetch_or(&ready, 1ull << dev, __ATOMIC_RELEASE);
    }
    return launch(dsv4_gqa_select_kernel<CLUSTER>, dim3(p.batch * p.c.kv_heads * CLUSTER), kSelThreads, smem, stream,
                  CLUSTER, p);
}

}  // namespace
}  // namespace gqa
}  // namespace dsv4

extern "C" {

size_t dsv4_gqa_evict_workspace_size(const dsv4_gqa_cache* cache, int32_t batch, int32_t max_len, int32_t keep) {
    dsv4::gqa::Layout l;
    return dsv4::gqa::layout(cache, batch, max_len, keep, l) ? 0 : l.bytes;
}

int dsv4_gqa_evict(int32_t batch, const int32_t* lens, const int32_t* seq_lens, const int32_t* req_pool_indices,
                   const dsv4_gqa_cache* cache, int32_t max_len, int32_t keep, int32_t first, int32_t recent,
                   const float* weights, float* weights_out, const int32_t* positions, int32_t* positions_out,
                   int64_t width, int32_t* lens_out, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace dsv4;
    using namespace dsv4::gqa;
    Layout l;
    const int rc = layout(cache, batch, max_len, keep, l);
    if (rc) return rc;
    if (!lens || !lens_out || !weights || !weights_out || !positions != !positions_out) return DSV4_ERR_INVALID;
    if (first < 0 || recent < 0 || first > keep || recent > keep - first || width < max_len) return DSV4_ERR_INVALID;
    if (!workspace || workspace_bytes < l.bytes) return DSV4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DSV4_ERR_INVALID;
    unsigned int* err = device_error_word();
    if (!err) return DSV4_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    EvictParams p;
    p.c = device_cache(cache);
    p.batch = batch;
    p.lens = lens;
    p.seen = seq_lens;
    p.req = req_pool_indices;
    p.max_len = max_len;
    p.keep = keep;
    p.first = first;
    p.recent = recent;
    p.w_in = weights;
    p.w_out = weights_out;
    p.p_in = positions;
    p.p_out = positions_out;
    p.width = width;
    p.lens_out = lens_out;
    p.counts = reinterpret_cast<int*>(ws + l.counts);
    p.holes = reinterpret_cast<int*>(ws + l.holes);
    p.movers = reinterpret_cast<int*>(ws + l.movers);
    p.most = most_moved(max_len, keep);
    p.row_pieces = cache->head_dim * (cache->format == DSV4_GQA_E4M3 ? 1 : 2) / 16;
    p.err = err;

    // a cluster per (request, KV head): more CTAs where there are few and long ones
    const int ids = batch * cache->num_kv_heads;
    int cluster = 1;
    while (cluster < kMaxCluster && (max_len > cluster * kKeysPerCta || (ids * cluster < 152 && max_len > 4096 * cluster)))
        cluster *= 2;
    const int per = ((max_len + cluster - 1) / cluster + 31) & ~31;
    p.cached = per <= kKeysPerCta ? per : 0;
    const size_t smem = (size_t)p.cached * 4;
    int r = cluster == 1   ? launch_select<1>(p, smem, stream)
            : cluster == 2 ? launch_select<2>(p, smem, stream)
            : cluster == 4 ? launch_select<4>(p, smem, stream)
                           : launch_select<8>(p, smem, stream);
    if (r) return r;
    return launch(dsv4_gqa_move_kernel, dim3((p.most + kMoveRows - 1) / kMoveRows, ids), kMoveThreads, 0, stream, 1, p);
}

}  // extern "C"
