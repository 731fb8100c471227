// dsv4_gqa_evict.cu - eviction from a grouped-query cache by accumulated
// weight (include/dsv4gqa.h states what is computed).
//
// Two kernels.  The select kernel gives every (request, KV head) to one
// cluster of 1 to 8 CTAs.  Weights become order-preserving 32-bit keys, which
// stay in registers: a warp holds a run of consecutive slots, lane l of its
// i-th register slot 32 i + l of the run.  A radix select of four 8-bit digits
// finds the key of the last row kept and how many rows of that very key stay;
// its histograms have eight copies, so that the few hot bins of a digit
// (weights lie in a few binades) cost few conflicts.  Then lane i holds the
// kept rows of chunk i as a bit mask, so counting and ranking the freed slots
// below `keep` and the kept rows behind it is one scan over lanes, and only
// chunks that have any are visited again.  Histograms and
// counts are combined over the cluster through distributed shared memory;
// every count is exact and every order is that of the slots, so the result
// does not depend on timing.  Bound by the chain of round trips and barriers:
// 13 us for 256 heads of 4200 to 5120 rows (load 4, then 1.3 per digit), 18 us
// for 64 of 20000 to 32768 with clusters of four.  The move kernel copies the
// listed rows: only rows that change their slot are read and written, each
// once.  It is bound by HBM: 38 us for 188 MB of 256-byte rows from anywhere
// in 32768 slots (4.9 TB/s).  One kernel for both took longer (61 us and not 58
// for those), except where each head moves a few rows at most.
#include "dsv4_gqa.cuh"

namespace dsv4 {
namespace gqa {
namespace {

constexpr int kBins = 256;
constexpr int kCopies = 8;
constexpr int kMoveThreads = 128;
// rows that a warp of the move kernel copies, by the 16-byte pieces of a K and a V row
__host__ __device__ constexpr int warp_rows(int pieces) { return pieces >= 32 ? 16 : 32; }
constexpr int kMaxCluster = 8;
constexpr int kFew = 4;                    // rows over the bound that are looked for one by one
constexpr int kHeldKeys = 32 * 1024;       // keys that the largest CTA holds in registers

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
    int row_pieces;                        // 16-byte pieces of a row
    int alone;                             // no request can be more than kFew rows over the bound: the select kernel
                                           // moves them itself and writes the new lengths
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

__device__ __forceinline__ uint4 ld_cluster_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int WARPS>
struct SelectShared {
    uint4 hist[kBins][kCopies / 4];        // lane l counts in copy l mod kCopies
    uint4 bins[2][kBins / 4];              // this CTA's sums, for the cluster (by digit parity)
    uint32_t warp_sum[2][WARPS];
    uint32_t count[2][2];                  // this CTA's ties; holes and movers, for the cluster
    int few[2][4], few_count;              // slots freed and refilled, where they are few
    uint32_t pick[3];                      // chosen bin, rows wanted in it, rows in it
    int skip;
};

template <int CLUSTER>
__device__ __forceinline__ void lane_sync() {
    if constexpr (CLUSTER > 1)
        cluster_sync();
    else
        __syncthreads();
}

// Exclusive prefixes of v and w (uniform in a warp) over the block's warps, and
// the block's totals.
template <int WARPS>
__device__ __forceinline__ void warps_exclusive(uint32_t& v, uint32_t& w, uint32_t (*sums)[WARPS], uint32_t& total_v,
                                                uint32_t& total_w) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) {
        sums[0][warp] = v;
        sums[1][warp] = w;
    }
    __syncthreads();
    const uint32_t a = lane < WARPS ? sums[0][lane] : 0u, c = lane < WARPS ? sums[1][lane] : 0u;
    total_v = __reduce_add_sync(0xffffffffu, a);
    total_w = __reduce_add_sync(0xffffffffu, c);
    v = __reduce_add_sync(0xffffffffu, lane < warp ? a : 0u);
    w = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0u);
}

// THREADS x KEYS slots per CTA; KEYS = 0: any number, keys made anew in every
// pass (rows beyond 8 x 32768 slots).
template <int THREADS, int KEYS, int CLUSTER>
__global__ void __launch_bounds__(THREADS, KEYS > 16 ? 1 : 1024 / THREADS) dsv4_gqa_select_kernel(const __grid_constant__ EvictParams p) {
    constexpr int WARPS = THREADS / 32;
    __shared__ SelectShared<WARPS> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int id = blockIdx.x / CLUSTER, rank = blockIdx.x % CLUSTER;
    const int b = id / p.c.kv_heads, h = id % p.c.kv_heads;
    for (int i = tid; i < kBins * kCopies / 4; i += THREADS) (&sh.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sh.skip = 0;
    grid_dependency_wait();
    grid_dependents_go();

    unsigned err = 0;
    const Request rq = read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err);
    const int seen = p.seen ? __ldg(p.seen + b) : rq.n;
    if (p.req && rq.n > 0) {                 // a row that an earlier request of the call names too
        __syncthreads();
        for (int e = tid; e < b; e += THREADS) {
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
    const bool skip = err & DSV4_DEV_ERR_REQ_ROW;
    if (p.alone && h == 0 && rank == 0 && tid == 0) p.lens_out[b] = min(rq.n, p.keep);
    if (rq.n <= p.keep || skip) {            // (uniform over the cluster)
        if (rank == 0 && tid == 0) p.counts[id] = 0;
        if ((copy_w || copy_p) && !skip)
            for (int s = rank * THREADS + tid; s < rq.n; s += CLUSTER * THREADS) {
                if (copy_w) w_out[s] = w_in[s];
                if (copy_p) p_out[s] = p_in[s];
            }
        return;
    }

    // this warp's run of slots: equal shares of the CTAs, then of their warps, in chunks of 32
    const int n = rq.n;
    const int per = ((n + CLUSTER * WARPS - 1) / (CLUSTER * WARPS) + 31) & ~31;
    const int r0 = min(n, (rank * WARPS + warp) * per), r1 = min(n, r0 + per);
    const int chunks = (r1 - r0 + 31) >> 5;
    auto make_key = [&](float w, int pos) -> uint32_t {
        return pos < p.first || pos >= seen - p.recent ? 0xffffffffu : weight_key(w);
    };
    uint32_t held[KEYS ? KEYS : 1];
    if constexpr (KEYS > 0) {
        // a batch's loads before their uses: 4 KB (with positions) per warp in flight
        constexpr int kBatch = 16;
#pragma unroll
        for (int i0 = 0; i0 < KEYS; i0 += kBatch) {
            float w[kBatch];
            int pos[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int s = r0 + 32 * (i0 + i) + lane;
                w[i] = 0.f;
                pos[i] = s;
                if (s < r1) {
                    w[i] = __ldg(w_in + s);
                    if (p_in) pos[i] = __ldg(p_in + s);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int s = r0 + 32 * (i0 + i) + lane;
                held[i0 + i] = make_key(w[i], pos[i]);
                // slots below `keep` in case their rows stay; the move kernel writes the others' again
                if (s < r1 && s < p.keep) {
                    if (copy_w) w_out[s] = w[i];
                    if (copy_p) p_out[s] = pos[i];
                }
            }
        }
    } else if (copy_w || copy_p) {
        for (int s = r0 + lane; s < min(r1, p.keep); s += 32) {
            if (copy_w) w_out[s] = __ldg(w_in + s);
            if (copy_p) p_out[s] = __ldg(p_in + s);
        }
    }
    // visit(chunk, key, inside) for chunks from .. from + COUNT - 1 of the warp, in order
    auto each = [&](int from, int count, auto&& visit) {
        if constexpr (KEYS > 0) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i)
                if (i >= from && i < from + count && i < chunks) visit(i, held[i], r0 + 32 * i + lane < r1);
        } else {
            for (int i = from; i < min(from + count, chunks); ++i) {
                const int s = r0 + 32 * i + lane;
                const bool in = s < r1;
                visit(i, in ? make_key(__ldg(w_in + s), p_in ? __ldg(p_in + s) : s) : 0u, in);
            }
        }
    };
    __syncthreads();

    int* holes = p.holes + (size_t)id * p.most;
    int* movers = p.movers + (size_t)id * p.most;
    if constexpr (CLUSTER == 1 && KEYS > 0) {
        // A cache just over its bound, as after every step of a decode loop: the few rows to go are looked for one by
        // one, smallest key first, of equal ones the highest slot.  (One of 2049 rows for each of 512 heads, with the
        // move: 17 us by the radix select, 8.2 so, 6.5 where no other kernel has to move rows; four of 2052: 15.8,
        // 12.7 and 11.4.)
        if (n - p.keep <= kFew) {
            int gone[kFew];
            for (int e = 0; e < n - p.keep; ++e) {
                uint32_t low = 0xffffffffu;
                int at = -1;
                each(0, chunks, [&](int i, uint32_t k, bool in) {
                    const int s = r0 + 32 * i + lane;
                    bool was = false;
#pragma unroll
                    for (int x = 0; x < kFew; ++x) was |= x < e && gone[x] == s;
                    if (in && !was && k <= low) {
                        low = k;
                        at = s;
                    }
                });
                const uint32_t wlow = __reduce_min_sync(0xffffffffu, low);
                const int wat = __reduce_max_sync(0xffffffffu, low == wlow ? at : -1);
                if (lane == 0) {
                    sh.warp_sum[0][warp] = wlow;
                    sh.warp_sum[1][warp] = static_cast<uint32_t>(wat);
                }
                __syncthreads();
                const uint32_t x = lane < WARPS ? sh.warp_sum[0][lane] : 0xffffffffu;
                const int y = lane < WARPS ? static_cast<int>(sh.warp_sum[1][lane]) : -1;
                const uint32_t least = __reduce_min_sync(0xffffffffu, x);
                const int slot = __reduce_max_sync(0xffffffffu, x == least ? y : -1);
#pragma unroll
                for (int q = 0; q < kFew; ++q)
                    if (q == e) gone[q] = slot;
                __syncthreads();
            }
            if (tid == 0) {
                // freed slots below `keep` in ascending order, and the rows behind it that stay
                int count = 0, last = -1;
                for (;;) {
                    int next = p.keep;
#pragma unroll
                    for (int q = 0; q < kFew; ++q)
                        if (q < n - p.keep && gone[q] > last) next = min(next, gone[q]);
                    if (next >= p.keep) break;
                    sh.few[0][count++] = last = next;
                }
                sh.few_count = count;
                int to = 0;
                for (int s = p.keep; s < n; ++s) {
                    bool stays = true;
#pragma unroll
                    for (int q = 0; q < kFew; ++q) stays &= !(q < n - p.keep && gone[q] == s);
                    if (stays) sh.few[1][to++] = s;
                }
            }
            __syncthreads();
            const int count = sh.few_count;
            if (!p.alone) {
                if (tid == 0) p.counts[id] = count;
                if (tid < count) {
                    holes[tid] = sh.few[0][tid];
                    movers[tid] = sh.few[1][tid];
                }
                return;
            }
            // a 16-byte piece of a K or V row per thread
            const int* table = p.c.table + (long long)rq.row * p.c.table_stride;
            const int in_page = (1 << p.c.page_shift) - 1, pieces = 2 * p.row_pieces;
            for (int e = tid; e < count * pieces; e += THREADS) {
                const int j = e / pieces, piece = e % pieces, dst = sh.few[0][j], src = sh.few[1][j];
                const int tp = __ldg(table + (dst >> p.c.page_shift)), fp = __ldg(table + (src >> p.c.page_shift));
                if (piece == 0) {
                    w_out[dst] = w_in[src];
                    if (p_out) p_out[dst] = p_in[src];
                }
                if (tp < 0 || tp >= p.c.num_pages || fp < 0 || fp >= p.c.num_pages) {
                    if (piece == 0) atomicOr(p.err, DSV4_DEV_ERR_GQA_PAGE);
                    continue;
                }
                uint8_t* pool = (piece < p.row_pieces ? p.c.k : p.c.v) + h * p.c.head_stride +
                                (piece < p.row_pieces ? piece : piece - p.row_pieces) * 16;
                *reinterpret_cast<uint4*>(pool + tp * p.c.page_stride + (dst & in_page) * p.c.row_stride) =
                    *reinterpret_cast<const uint4*>(pool + fp * p.c.page_stride + (src & in_page) * p.c.row_stride);
            }
            return;
        }
    }

    // ---- the key of the last row kept: `want` of the `equal` rows of key `prefix` stay ----
    uint32_t prefix = 0, mask = 0, want = p.keep, equal = 0;
    for (int digit = 0; digit < 4; ++digit) {
        const int shift = 24 - 8 * digit;
        each(0, chunks, [&](int, uint32_t k, bool in) {
            if (in && (k & mask) == prefix) atomicAdd(reinterpret_cast<uint32_t*>(sh.hist[(k >> shift) & 255u]) + lane % kCopies, 1u);
        });
        __syncthreads();
        // bin sums (a bin's copies are two neighbouring uint4); the copies are cleared for the next digit
        uint4* bins = sh.bins[digit & 1];
        for (int i = tid; i < kBins * kCopies / 4; i += THREADS) {
            uint4* c = &sh.hist[0][0] + i;
            const uint4 x = *c;
            *c = make_uint4(0, 0, 0, 0);
            uint32_t v = x.x + x.y + x.z + x.w;
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            if ((i & 1) == 0) reinterpret_cast<uint32_t*>(bins)[i >> 1] = v;
        }
        lane_sync<CLUSTER>();
        // one warp looks for the bin: lane l holds bins 255 - 8 l .. 248 - 8 l
        if (warp == 0) {
            uint32_t mine[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) mine[i] = 0;
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4* at = &bins[63 - 2 * lane - i];
                    uint4 x;
                    if constexpr (CLUSTER == 1)
                        x = *at;
                    else
                        x = ld_cluster_u4(mapa(smem_u32(at), r));
                    mine[4 * i] += x.w;
                    mine[4 * i + 1] += x.z;
                    mine[4 * i + 2] += x.y;
                    mine[4 * i + 3] += x.x;
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += mine[i];
            uint32_t above = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += x;
            }
            above -= sum;
            if (above < want && above + sum >= want) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (above < want && above + mine[i] >= want) {
                        sh.pick[0] = 255 - 8 * lane - i;
                        sh.pick[1] = want - above;
                        sh.pick[2] = mine[i];
                    }
                    above += mine[i];
                }
            }
        }
        __syncthreads();
        prefix |= sh.pick[0] << shift;
        mask |= 255u << shift;
        want = sh.pick[1];
        equal = sh.pick[2];
        if (equal == want) break;            // all rows of this prefix stay (uniform over the cluster)
    }
    // kept: keys above the prefix, and of those at it all (equal == want) or the first `want`
    const bool every = equal == want;

    uint32_t tie = 0;                        // rows at the prefix before this warp's
    if (!every) {
        uint32_t c = 0;
        each(0, chunks, [&](int, uint32_t k, bool in) { c += __popc(__ballot_sync(0xffffffffu, in && k == prefix)); });
        uint32_t none = 0, total, zero;
        warps_exclusive<WARPS>(c, none, sh.warp_sum, total, zero);
        tie = c;
        if (tid == 0) sh.count[0][0] = total;
        lane_sync<CLUSTER>();
        if constexpr (CLUSTER > 1) {
            const uint32_t a = smem_u32(&sh.count[0][0]);
            for (int r = 0; r < rank; ++r) tie += ld_cluster_u32(mapa(a, r));
        }
    }
    const uint32_t below = (1u << lane) - 1u;
    // bits 0 .. count - 1
    auto low_bits = [](int count) { return count >= 32 ? ~0u : count <= 0 ? 0u : (1u << count) - 1u; };
    // lane i: the kept rows of chunk from + i; t: rows at the prefix so far
    auto kept_rows = [&](int from, uint32_t& t) {
        uint32_t own = 0;
        each(from, 32, [&](int i, uint32_t k, bool in) {
            const uint32_t top = k & mask;
            bool kept = in && (top > prefix || (every && top == prefix));
            if (!every) {
                const bool same = in && k == prefix;
                const unsigned m = __ballot_sync(0xffffffffu, same);
                kept |= same && t + __popc(m & below) < want;
                t += __popc(m);
            }
            const unsigned m = __ballot_sync(0xffffffffu, kept);
            if (lane == i - from) own = m;
        });
        return own;
    };
    // lane i's chunk: evicted slots below `keep`, kept ones behind it
    auto hole_bits = [&](int from, uint32_t own) {
        const int s = r0 + 32 * (from + lane);
        return ~own & low_bits(r1 - s) & low_bits(p.keep - s);
    };
    auto move_bits = [&](int from, uint32_t own) { return own & ~low_bits(p.keep - (r0 + 32 * (from + lane))); };

    constexpr int kGroups = KEYS ? (KEYS + 31) / 32 : 1;     // groups of 32 chunks whose masks stay in registers
    uint32_t own[kGroups], nh = 0, nm = 0;
    {
        uint32_t t = tie;
        if constexpr (KEYS > 0) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                own[i] = kept_rows(32 * i, t);
                nh += __popc(hole_bits(32 * i, own[i]));
                nm += __popc(move_bits(32 * i, own[i]));
            }
        } else {
            for (int from = 0; from < chunks; from += 32) {
                own[0] = kept_rows(from, t);
                nh += __popc(hole_bits(from, own[0]));
                nm += __popc(move_bits(from, own[0]));
            }
        }
    }
    nh = __reduce_add_sync(0xffffffffu, nh);
    nm = __reduce_add_sync(0xffffffffu, nm);
    uint32_t hole = nh, move = nm, hole_total, move_total;
    warps_exclusive<WARPS>(hole, move, sh.warp_sum, hole_total, move_total);
    if constexpr (CLUSTER > 1) {
        if (tid == 0) {
            sh.count[1][0] = hole_total;
            sh.count[1][1] = move_total;
        }
        cluster_sync();
        const uint32_t a = smem_u32(&sh.count[1][0]);
        for (int r = 0; r < rank; ++r) {
            hole += ld_cluster_u32(mapa(a, r));
            move += ld_cluster_u32(mapa(a + 4, r));
        }
    }
    if (rank == CLUSTER - 1 && tid == 0) p.counts[id] = move + move_total;   // (warp 0's prefix: the CTAs before)
    auto list = [&](int from, uint32_t kept) {
        const uint32_t hb = hole_bits(from, kept), mb = move_bits(from, kept);
        // both counts of a chunk in one word: at most 1024 of each in 32 chunks
        const uint32_t both = __popc(hb) | __popc(mb) << 16;
        uint32_t incl = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const uint32_t ex = incl - both, sum = __shfl_sync(0xffffffffu, incl, 31);
        for (unsigned todo = __ballot_sync(0xffffffffu, both != 0); todo; todo &= todo - 1) {
            const int i = __ffs(todo) - 1;
            const uint32_t hm = __shfl_sync(0xffffffffu, hb, i), mm = __shfl_sync(0xffffffffu, mb, i);
            const uint32_t at = __shfl_sync(0xffffffffu, ex, i);
            const int s = r0 + 32 * (from + i) + lane;
            if (hm >> lane & 1) holes[hole + (at & 0xffffu) + __popc(hm & below)] = s;
            if (mm >> lane & 1) movers[move + (at >> 16) + __popc(mm & below)] = s;
        }
        hole += sum & 0xffffu;
        move += sum >> 16;
    };
    if constexpr (KEYS > 0) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) list(32 * i, own[i]);
    } else {
        uint32_t t = tie;
        for (int from = 0; from < chunks; from += 32) list(from, kept_rows(from, t));
    }
    // no CTA of the cluster may end while another still reads its counts
    if constexpr (CLUSTER > 1) cluster_sync();
}

// Rows holes[j] <- movers[j]: a warp copies 16 or 32 of them.  Lane j first
// finds the places of row j (slot lists and page table, one round trip each
// for all rows), then the warp copies row after row, PIECES = 16-byte pieces
// of the K and V rows together, all loads of eight warp-wide copies before
// their stores.
template <int PIECES>
__global__ void __launch_bounds__(kMoveThreads, 8) dsv4_gqa_move_kernel(const __grid_constant__ EvictParams p) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int id = blockIdx.y, b = id / p.c.kv_heads, h = id % p.c.kv_heads;
    grid_dependency_wait();
    grid_dependents_go();
    const int row = p.req ? __ldg(p.req + b) : b;
    const bool placed = row >= 0 && row < p.c.table_rows;
    if (blockIdx.x == 0 && h == 0 && tid == 0) {
        int n = __ldg(p.lens + b);
        n = n < 0 || !placed ? 0 : n > p.max_len ? p.max_len : n;
        p.lens_out[b] = n < p.keep ? n : p.keep;
    }
    const int count = p.counts[id];
    constexpr int kWarpRows = warp_rows(PIECES);
    const int j0 = (blockIdx.x * (kMoveThreads / 32) + warp) * kWarpRows;
    if (j0 >= count) return;
    const int rows = min(kWarpRows, count - j0);
    const int mask = (1 << p.c.page_shift) - 1;
    long long to = -1, of = -1;              // byte offsets of row j0 + lane
    if (lane < rows) {
        const int dst = p.holes[(size_t)id * p.most + j0 + lane], src = p.movers[(size_t)id * p.most + j0 + lane];
        const int* table = p.c.table + (long long)row * p.c.table_stride;
        const int tp = __ldg(table + (dst >> p.c.page_shift)), fp = __ldg(table + (src >> p.c.page_shift));
        const size_t at = ((size_t)row * p.c.kv_heads + h) * p.width;
        p.w_out[at + dst] = p.w_in[at + src];
        if (p.p_out) p.p_out[at + dst] = p.p_in[at + src];
        if (tp < 0 || tp >= p.c.num_pages || fp < 0 || fp >= p.c.num_pages) {
            atomicOr(p.err, DSV4_DEV_ERR_GQA_PAGE);
        } else {
            to = tp * p.c.page_stride + (dst & mask) * p.c.row_stride + h * p.c.head_stride;
            of = fp * p.c.page_stride + (src & mask) * p.c.row_stride + h * p.c.head_stride;
        }
    }
    // a warp-wide copy moves 32 / PIECES rows, or a part of one
    constexpr int kRows = PIECES < 32 ? 32 / PIECES : 1, kParts = PIECES < 32 ? 1 : PIECES / 32;
    constexpr int kBatch = 8 / kParts;
    const int piece = lane % PIECES, sub = lane / PIECES;
#pragma unroll 1
    for (int r = 0; r < rows; r += kRows * kBatch) {
        uint4 x[kBatch][kParts];
        auto pool_of = [&](int q) {
            const int at = piece + 32 * q;
            return at >= PIECES / 2 ? p.c.v + (at - PIECES / 2) * 16 : p.c.k + at * 16;
        };
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = r + i * kRows + sub;
            const long long f = __shfl_sync(0xffffffffu, of, j & 31);
            if (j < rows && f >= 0)
#pragma unroll
                for (int q = 0; q < kParts; ++q) x[i][q] = __ldcs(reinterpret_cast<const uint4*>(pool_of(q) + f));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = r + i * kRows + sub;
            const long long t = __shfl_sync(0xffffffffu, to, j & 31);
            if (j < rows && t >= 0)
#pragma unroll
                for (int q = 0; q < kParts; ++q) *reinterpret_cast<uint4*>(pool_of(q) + t) = x[i][q];
        }
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

template <int THREADS, int KEYS, int CLUSTER>
int launch_select_one(const EvictParams& p, void* stream) {
    return launch(dsv4_gqa_select_kernel<THREADS, KEYS, CLUSTER>, dim3(p.batch * p.c.kv_heads * CLUSTER), THREADS, 0,
                  stream, CLUSTER, p);
}

template <int PIECES>
int launch_move(const EvictParams& p, void* stream) {
    constexpr int kRows = kMoveThreads / 32 * warp_rows(PIECES);
    return launch(dsv4_gqa_move_kernel<PIECES>, dim3((p.most + kRows - 1) / kRows, p.batch * p.c.kv_heads),
                  kMoveThreads, 0, stream, 1, p);
}

template <int CLUSTER>
int launch_select_cluster(const EvictParams& p, int per, void* stream) {
    return per <= 8192    ? launch_select_one<512, 16, CLUSTER>(p, stream)
           : per <= 16384 ? launch_select_one<512, 32, CLUSTER>(p, stream)
                          : launch_select_one<512, 64, CLUSTER>(p, stream);
}

// The smallest CTA that holds a row's keys, or a cluster of them: where there
// are few rows, several CTAs share one, as long as each has 2048 slots or more.
// (64 rows of 32768: one CTA each 77.8 us with the move, clusters of four 57.8,
// of eight 73.1, which no longer run all at once; 8 rows of 100000: clusters
// of four, the fewest that hold the keys, 44 us, of eight 28.7.)
int launch_select(const EvictParams& p, void* stream) {
    const int ids = p.batch * p.c.kv_heads;
    int cluster = 1;
    while (!p.alone && cluster < kMaxCluster &&
           (p.max_len > cluster * kHeldKeys || (ids * cluster < 152 && p.max_len > 4096 * cluster)))
        cluster *= 2;
    const int per = (p.max_len + cluster - 1) / cluster;
    if (per > kHeldKeys) return launch_select_one<512, 0, 8>(p, stream);
    switch (cluster) {
        case 1: return per <= 4096 ? launch_select_one<256, 16, 1>(p, stream) : launch_select_cluster<1>(p, per, stream);
        case 2: return launch_select_cluster<2>(p, per, stream);
        case 4: return launch_select_cluster<4>(p, per, stream);
        default: return launch_select_cluster<8>(p, per, stream);
    }
}

template <int CLUSTER>
bool load_select_cluster() {
    return load_kernels(dsv4_gqa_select_kernel<512, 16, CLUSTER>, dsv4_gqa_select_kernel<512, 32, CLUSTER>,
                        dsv4_gqa_select_kernel<512, 64, CLUSTER>);
}
int load_all() {
    static unsigned long long ready = 0;
    return once_per_device(ready, [] {
        return load_select_cluster<1>() && load_select_cluster<2>() && load_select_cluster<4>() && load_select_cluster<8>() &&
               load_kernels(dsv4_gqa_select_kernel<256, 16, 1>, dsv4_gqa_select_kernel<512, 0, 8>, dsv4_gqa_move_kernel<8>,
                            dsv4_gqa_move_kernel<16>, dsv4_gqa_move_kernel<32>, dsv4_gqa_move_kernel<64>);
    });
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
    const size_t list = size_t(batch) * sizeof(int), entries = row_array_bytes(cache, width);
    if (!same_or_apart(weights, weights_out, entries) || !same_or_apart(positions, positions_out, entries) ||
        !same_or_apart(lens, lens_out, list) || !same_or_apart(seq_lens, lens_out, list) ||
        !apart(req_pool_indices, list, lens_out, list))
        return DSV4_ERR_INVALID;
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

    // (new lengths that replace the old ones, or the tokens seen, have to wait for every head's CTA to have read those:
    // the move kernel does)
    p.alone = max_len - keep <= kFew && max_len <= kHeldKeys && lens != lens_out && seq_lens != lens_out;
    int r = load_all();
    if (r) return r;
    r = launch_select(p, stream);
    if (r || p.alone) return r;
    switch (p.row_pieces) {
        case 4: return launch_move<8>(p, stream);
        case 8: return launch_move<16>(p, stream);
        case 16: return launch_move<32>(p, stream);
        default: return launch_move<64>(p, stream);
    }
}

}  // extern "C"
