// dsv4_gqa_decode4.cuh - the attention over long lists of 4-bit rows
// (DSV4_GQA_E2M1; include/dsv4gqa.h states what is computed), on the
// block-scaled 4-bit tensor cores.  It shares the list of tiles, its division
// into shares, the pieces of cut segments and the kernels behind it with
// dsv4_gqa_decode.cuh, whose own kernel takes the short lists; a share here
// belongs to a CTA and a tile has 128 slots.
//
// The instructions that turn codes into 16-bit operands bound a kernel on
// mma.sync (two conversions and two products for every 4 codes of K and of V
// and 16 slots; 4.5 bits a value come in faster than that: 48 % of the memory's
// rate).  Here no thread touches a code:
//   S   K is the A operand of a 4-bit MMA as it lies in the cache, block scales
//       and all.  q becomes a B operand of 4 bits without losing any: eight
//       digits of base 8,
//         q = 2^(E - 1) sum_k 8^-k d_k,   d_k = -4 .. 4,
//       each an e2m1 code (E: exponent of the head's largest value; what is left
//       out lies 2^-24 below that value).  Digits are columns, of which CH in a row are
//       summed by the accumulator, their weights being B's block scales (1, 2^-3,
//       2^-6, 2^-9); the softmax adds up the others.
//   V   its blocks run along the dims, not along the slots that O sums over, so
//       an MMA with the identity as A and V as B writes V^T, block scales
//       included, to TMEM as fp32 (every value exact), where it lies as the A
//       operand of
//   O^T += V^T P^T, a tf32 MMA.  Values have 6 bits; P is rounded to tf32's 11,
//       or is two of them where the output is f16.
// A NaN among the block scales of V would reach all dims of its row through the
// identity's zeros, and the MMA takes scales without a sign.  So the issuing
// warps look through the scales of each tile; a NaN block is noted and its scale
// zeroed, a negative scale's sign moves into its codes.
//
// Roles of the 8 warps: 0 .. 3 softmax and output (a thread is a slot of S and
// a dim of O), 4 and 5 copy (cp.async into a ring whose entries are K and V of a
// tile in turn), 6 issues S, 7 V^T and O.  Two CTAs an SM.
//
// An MMA here costs 9 (tf32, N = 16), 17 (N = 32), 48 (4 bits, N = 64) and
// 64 clk (identity, N = 128) when its issuer is one thread that elect.sync picked
// in a converged warp, and 88 clk of issue for each where the thread is picked by
// its index.  A tile of 8 heads of 128 takes the tensor pipe 370 clk, and its 18
// KB take an SM 780 clk at the memory's rate.
#pragma once
#include <cstddef>

#include "dsv4_gqa_decode.cuh"

namespace dsv4 {
namespace gqa {

constexpr int kTile4 = 128;                // slots
constexpr int kThreads4 = 256;
constexpr int kRing4 = 16;                 // tiles whose notes are kept: more than the copies are ahead
// Sums stay in the accumulator for so many tiles: it truncates, 16 times a tile, and what that loses is below 2^-16 of
// the sum this way, however long the list.
constexpr int kFlushTiles = 8;
constexpr uint64_t kWaitNs4 = 2000000000ull;

template <int QKIND, int D_>
struct Shape4 {
    static constexpr int D = D_, HEADS = 8;
    static constexpr bool QBF16 = QKIND == DSV4_GQA_BF16, TWO = !QBF16;
    static constexpr int KS = D / 64;                        // K steps of S, and of V^T
    static constexpr int DIGITS = 8, NS = DIGITS * HEADS;    // columns of S
    static constexpr int USED = HEADS * (TWO ? 2 : 1);       // columns of O: heads, once for each piece of P
    static constexpr int NP = 16;                            // and of its MMA, which takes 16 at least
    // TMEM columns; block scales of K, V and (all 1) of the digits and the identity
    static constexpr int T_V = 0, T_S = 128, T_O = T_S + NS, T_K = T_O + NP, T_VS = T_K + 4 * KS, T_ONE = T_VS + 4 * KS;
    static constexpr int COLS = 256, CTAS = 2;
    static_assert(T_ONE + 4 <= COLS, "TMEM");
    // shared memory
    static constexpr int ROWB = D / 2;                       // bytes of a row's codes
    static constexpr int SFB = kTile4 * D / 16;              // of a tile's block scales
    static constexpr int ENTRY = kTile4 * ROWB + SFB;
    static constexpr int I_BYTES = 128 * ROWB, Q_BYTES = NS * ROWB, P_BYTES = kTile4 * NP * 4;
    static constexpr int NOTES = 1280;                       // barriers and notes
    static constexpr int FIT = (113 * 1024 - I_BYTES - Q_BYTES - P_BYTES - NOTES) / ENTRY / 2 * 2;
    static constexpr int ENTRIES = FIT < 16 ? FIT : 16;
    static_assert(ENTRIES >= 4 && ENTRIES / 2 + 2 < kRing4, "the ring");
    static constexpr int O_I = 0, O_Q = O_I + I_BYTES, O_P = O_Q + Q_BYTES, O_RING = O_P + P_BYTES,
                         O_NOTES = O_RING + ENTRIES * ENTRY, SMEM = O_NOTES + NOTES;
    static_assert(O_P % 1024 == 0 && O_RING % 1024 == 0 && (kTile4 * ROWB) % 1024 == 0 && ENTRY % 512 == 0, "swizzle atoms");
};

// Shared memory matrix descriptor of a K-major operand with rows of `rowb` = 32, 64 or 128 bytes, swizzled over as many.
__device__ __forceinline__ uint64_t desc_rows(uint32_t start, int rowb) {
    return (uint64_t)((start & 0x3FFFFu) >> 4) | 1ull << 16 | (uint64_t)(rowb * 8 >> 4) << 32 | 1ull << 46 |
           (uint64_t)(rowb == 32 ? 6 : rowb == 64 ? 4 : 2) << 61;
}
// Of 128 rows' scales: 32 lines of 16 bytes, 4 bytes of rows i, i + 32, i + 64, i + 96 each.
__device__ __forceinline__ uint64_t desc_scales(uint32_t start) {
    return (uint64_t)((start & 0x3FFFFu) >> 4) | 1ull << 16 | 8ull << 32 | 1ull << 46;
}
// Byte `at` of row `row` in such an operand.
template <int ROWB>
__device__ __forceinline__ uint32_t row_offset(int row, int at) {
    constexpr int kShift = ROWB == 128 ? 0 : ROWB == 64 ? 1 : 2, kMask = ROWB / 16 - 1;
    return row * ROWB + ((((at >> 4) ^ (row >> kShift)) & kMask) << 4) + (at & 15);
}
// 4-bit operands, K = 64, a ue4m3 scale for 16 of them
__host__ __device__ constexpr uint32_t idesc_e2m1(uint32_t m, uint32_t n) {
    return 1u << 7 | 1u << 10 | (n >> 3) << 17 | (m >> 4) << 24;
}
__host__ __device__ constexpr uint32_t idesc_tf32(uint32_t m, uint32_t n) {
    return 1u << 4 | 2u << 7 | 2u << 10 | (n >> 3) << 17 | (m >> 4) << 24;
}
__device__ __forceinline__ void mma_e2m1(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t a_scales,
                                         uint32_t b_scales, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_tf32_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_copy_scales(uint32_t to, uint64_t from) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(from) : "memory");
}
// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(is));
    return is != 0;
}
// N columns of this thread's lane, waited.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[N]) {
    static_assert(N == 8 || N == 16 || N == 32, "columns");
    if constexpr (N == 32) {
        tmem_ld32(t, v);
    } else if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
            "tcgen05.wait::ld.sync.aligned;\n"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
              "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
            : "r"(t)
            : "memory");
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
            "tcgen05.wait::ld.sync.aligned;\n"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
            : "r"(t)
            : "memory");
    }
}
__device__ __forceinline__ void tmem_st1(uint32_t t, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\ntcgen05.wait::st.sync.aligned;\n" ::"r"(t), "r"(v)
                 : "memory");
}
// Whether any of the 128 softmax threads' `x` holds, on named barrier 1.
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { named_barrier_sync(1, 128); }

__device__ __forceinline__ uint32_t to_tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint64_t f32_pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// An integer of -4 .. 4 as an e2m1 code.
__device__ __forceinline__ uint32_t digit_e2m1(int d) {
    const int a = abs(d);
    return static_cast<uint32_t>(min(2 * a, a + 2)) | (static_cast<uint32_t>(d) >> 28 & 8u);
}
// 4-byte global -> shared copy; src_bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// What a CTA's warps tell each other.
template <class S>
struct Notes {
    uint64_t full[S::ENTRIES], empty[S::ENTRIES];            // ring entries: rows have landed; MMAs have read them
    uint64_t s_go, s_full;                                   // S may be written (q is there, the last S is read); is
    uint64_t p_full, v_full, o_full;                         // P is written; V^T is; O's MMAs of the tile are done
    uint64_t drained;
    uint32_t tmem;
    int abort, fresh;                                        // P's tile begins a new sum in O
    uint8_t ok[kRing4][2];                                   // of tiles: valid 16-slot groups, four bits for each copying warp
    uint16_t nan[kRing4];                                    // and blocks of V that hold a NaN
    alignas(16) float mul[2][S::HEADS];                      // score factors, by parity of the piece (read as float4)
    float odd[2][S::HEADS];                                  // NaN for a head whose query is not finite, else 0
    float sum[4][S::HEADS], top[4][S::HEADS];
};

template <class S>
__global__ void __launch_bounds__(kThreads4, S::CTAS) dsv4_gqa_decode4_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int D = S::D, HEADS = S::HEADS, NP = S::NP, KS = S::KS, ROWB = S::ROWB, NE = S::ENTRIES;
    extern __shared__ __align__(1024) uint8_t smem4[];
    uint8_t* smem = smem4;
    using N = Notes<S>;
    static_assert(sizeof(N) <= S::NOTES && offsetof(N, mul) % 16 == 0 && S::O_NOTES % 16 == 0,
                  "notes");
    N& notes = *reinterpret_cast<N*>(smem + S::O_NOTES);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t base = smem_u32(smem);
    const uint32_t s_i = base + S::O_I, s_q = base + S::O_Q, s_p = base + S::O_P, ring = base + S::O_RING;
    auto bar = [&](uint64_t& b) { return smem_u32(&b); };

    // ---- what does not depend on the call's data ----
    if (warp == 7) tmem_alloc(smem_u32(&notes.tmem), S::COLS);
    if (tid == 0) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            mbar_init(bar(notes.full[e]), 64 + 2);
            mbar_init(bar(notes.empty[e]), 1);
        }
        mbar_init(bar(notes.s_go), 128);
        mbar_init(bar(notes.s_full), 1);
        mbar_init(bar(notes.p_full), 128);
        mbar_init(bar(notes.v_full), 1);
        mbar_init(bar(notes.o_full), 1);
        mbar_init(bar(notes.drained), 2);
        notes.abort = 0;
        fence_mbar_init_cluster();
    }
    for (int i = tid; i < 128 * ROWB / 16; i += kThreads4) {
        const int r = i / (ROWB / 16), at = i % (ROWB / 16) * 16;         // row r: code 2 (1.0) at dim r
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = (at + 4 * k) * 2 == (r & ~7) ? 2u << 4 * (r & 7) : 0u;
        st_shared_v4(s_i + row_offset<ROWB>(r, at), w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = notes.tmem;
    if (warp < 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_st1(tmem + (warp * 32u << 16) + S::T_ONE + i, 0x38383838u);       // (e4m3: 1)
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();
    grid_dependents_go();

    // ---- this CTA's share ----
    const int hcs = p.c.kv_heads;              // (one group of query heads each)
    unsigned err = 0;
    auto request_of = [&](int b) {
        Request r{0, 0};
        return b < p.batch ? read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err) : r;
    };
    const Request early = request_of(lane);
    unsigned total = key_range<kTile4>(p, early.n).tiles;
    for (int b = lane + 32; b < p.batch; b += 32) total += key_range<kTile4>(p, request_of(b).n).tiles;
    total = __reduce_add_sync(0xffffffffu, total) * hcs;
    if (err && blockIdx.x == 0 && warp == 0) atomicOr(p.err, err);
    Shares shares{};
    if (total) shares = make_shares(p, total);
    const int share = blockIdx.x;
    const bool any = share < shares.count;
    const unsigned t0 = any ? share_begin(shares, share) : 0u, t1 = any ? share_begin(shares, share + 1) : 0u;
    const int tiles = static_cast<int>(t1 - t0);

    // a wait that is given up (after two seconds: a bug) ends all others, and the call's outputs are undefined
    auto wait = [&](uint64_t& b, uint32_t parity) {
        const uint32_t at = smem_u32(&b);
        uint64_t since = 0;
        for (uint32_t n = 1; !mbar_try(at, parity); ++n) {
            if (n & 63u) continue;                 // (the clock's reading is slow)
            const uint64_t now = globaltimer_ns();
            if (!since) since = now;
            if (*(volatile int*)&notes.abort) return;
            if (now - since > kWaitNs4) {
                atomicOr(p.err, DSV4_DEV_ERR_TIMEOUT);
                *(volatile int*)&notes.abort = 1;
                return;
            }
        }
    };
    // (a warp's lanes may leave it one by one)
    auto warp_wait = [&](uint64_t& b, uint32_t parity) {
        wait(b, parity);
        __syncwarp();
    };

    if (warp == 4 || warp == 5) {
        // ============================================================ copies
        // A warp copies 64 slots of every tile: four groups of 16, each on one page.
        if (tiles > 0) {
            const int w = warp - 4;
            constexpr int PPR = ROWB / 16, RPI = 32 / PPR;             // pieces of a row, rows per warp-wide copy
            const int lane_row = lane / PPR, lane_piece = lane % PPR;
            const int page_mask = (1 << p.c.page_shift) - 1;
            const long long lane_off = lane_row * p.c.row_stride + lane_piece * 16, step = RPI * p.c.row_stride;
            const long long lane_block = (lane & 15) * p.c.b_row_stride;
            const uint32_t dst0 = 64 * w * ROWB + row_offset<ROWB>(lane_row, lane_piece * 16);
            const uint32_t dst1 = kTile4 * ROWB + lane * 16 + w * 8;
            Cursor<kTile4> at;
            at.at = t0;
            at.locate(p, hcs, lane, early, request_of);
            at.bound(t1);
            // lanes 0 .. 3: the page of a group of the tile, and whether it holds slots to attend
            int page = -1;
            bool wanted = false;
            auto slot_of = [&]() { return (at.rg.lo / kTile4 + static_cast<int>(at.at - at.seg)) * kTile4 + 64 * w; };
            auto look = [&]() {
                const int slot = slot_of() + lane * 16;
                page = -1;
                wanted = lane < 4 && slot < at.rg.n && slot + 16 > at.rg.lo;
                if (wanted) page = __ldg(p.c.table + (long long)at.rq.row * p.c.table_stride + (slot >> p.c.page_shift));
            };
            look();
            int e = 0;
            uint32_t turn = 1;                     // parity that an entry's last reading has; 1: nothing was there
            for (int i = 0; i < tiles; ++i) {
                const int slot0 = slot_of(), lo = at.rg.lo, n = at.rg.n;
                const bool valid = page >= 0 && page < p.c.num_pages;
                if (wanted && !valid) atomicOr(p.err, DSV4_DEV_ERR_GQA_PAGE);
                const unsigned okm = __ballot_sync(0xffffffffu, wanted && valid);
                const int in_page = slot0 + lane * 16 & page_mask;
                const long long off = valid ? page * p.c.page_stride + at.hc * p.c.head_stride + in_page * p.c.row_stride : 0;
                const long long block_off =
                    valid ? page * p.c.b_page_stride + at.hc * p.c.b_head_stride + in_page * p.c.b_row_stride : 0;
                long long go[4], bo[2];
#pragma unroll
                for (int g = 0; g < 4; ++g) go[g] = __shfl_sync(0xffffffffu, off, g) + lane_off;
#pragma unroll
                for (int u = 0; u < 2; ++u) bo[u] = __shfl_sync(0xffffffffu, block_off, 2 * u + (lane >> 4)) + lane_block;
                const bool whole = okm == 15u && slot0 >= lo && slot0 + 64 <= n;
                // the next tile's pages are on their way while this one's entries are waited for
                ++at.at;
                if (at.at < at.end || at.next_segment(p, hcs, t1)) look();
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    warp_wait(notes.empty[e], turn);
                    fence_proxy_async();
                    if (kv == 0 && lane == 0) *(volatile uint8_t*)&notes.ok[i % kRing4][w] = okm;
                    const uint32_t dst = ring + e * S::ENTRY;
                    const uint8_t *pool = kv ? p.c.v : p.c.k, *blocks = kv ? p.c.vb : p.c.kb;
                    // lane's rows lane and 32 + lane: block scales, 4 of them to a line of each K step
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int s = slot0 + 32 * u + lane;
                        const bool in = whole || ((okm >> (2 * u + (lane >> 4)) & 1) && s >= lo && s < n);
                        const uint8_t* src = blocks + (in ? bo[u] : 0);
#pragma unroll
                        for (int k = 0; k < KS; ++k)
                            cp_async_4(dst + dst1 + 512 * k + 4 * u, src + (in ? 4 * k : 0), in ? 4u : 0u);
                    }
                    if (whole) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint8_t* src = pool + go[g];
#pragma unroll
                            for (int j = 0; j < 16 / RPI; ++j) {
                                cp_async_16(dst + dst0 + (16 * g + j * RPI) * ROWB, src, 16u);
                                src += step;
                            }
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < 4; ++g)
#pragma unroll
                            for (int j = 0; j < 16 / RPI; ++j) {
                                const int s = slot0 + 16 * g + j * RPI + lane_row;
                                const bool in = (okm >> g & 1) && s >= lo && s < n;
                                cp_async_16(dst + dst0 + (16 * g + j * RPI) * ROWB, pool + (in ? go[g] + j * step : 0), in ? 16u : 0u);
                            }
                    }
                    cp_async_arrive_noinc(bar(notes.full[e]));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(notes.full[e]));
                    if (++e == NE) {
                        e = 0;
                        turn ^= 1;
                    }
                }
            }
            cp_async_wait_all();
        }
    } else if (warp == 6) {
        // ============================================================ S
        constexpr uint32_t idesc = idesc_e2m1(128, S::NS);
        for (int i = 0; i < tiles; ++i) {
            const int e = 2 * i % NE, use = 2 * i / NE;
            const uint32_t entry = ring + e * S::ENTRY, scales = entry + kTile4 * ROWB;
            warp_wait(notes.full[e], use & 1);
            bool odd = false;
            for (int at = lane * 16; at < S::SFB; at += 512) {
                const uint4 x = ld_shared_u4(scales + at);
                odd |= ((x.x | x.y | x.z | x.w) & 0x80808080u) != 0;
            }
            if (__any_sync(0xffffffffu, odd)) {
                // the signs of scales go to their codes
                for (int at = lane; at < S::SFB; at += 32) {
                    const int r = (at >> 4 & 31) + 32 * (at >> 2 & 3), block = 4 * (at >> 9) + (at & 3);
                    uint8_t* sf = smem + (scales - base) + at;
                    if (*sf & 0x80) {
                        uint2* codes = reinterpret_cast<uint2*>(smem + (entry - base) + row_offset<ROWB>(r, 8 * block));
                        *codes = make_uint2(codes->x ^ 0x88888888u, codes->y ^ 0x88888888u);
                        *sf &= 0x7f;
                    }
                }
                __syncwarp();
            }
            warp_wait(notes.s_go, i & 1);
            fence_proxy_async();
            tc_fence_after();
            __syncwarp();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < KS; ++k) tmem_copy_scales(tmem + S::T_K + 4 * k, desc_scales(scales + 512 * k));
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    mma_e2m1(tmem + S::T_S, desc_rows(entry + 32 * k, ROWB), desc_rows(s_q + 32 * k, ROWB), idesc,
                             tmem + S::T_K + 4 * k, tmem + S::T_ONE, k);
                mma_commit(bar(notes.s_full));
                mma_commit(bar(notes.empty[e]));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(notes.drained));
        __syncwarp();
    } else if (warp == 7) {
        // ============================================================ V^T and O
        constexpr uint32_t idesc_v = idesc_e2m1(128, kTile4), idesc_o = idesc_tf32(128, NP);
        for (int i = 0; i < tiles; ++i) {
            const int e = (2 * i + 1) % NE, use = (2 * i + 1) / NE;
            const uint32_t entry = ring + e * S::ENTRY, scales = entry + kTile4 * ROWB;
            warp_wait(notes.full[e], use & 1);
            bool odd = false;
            for (int at = lane * 16; at < S::SFB; at += 512) {
                const uint4 x = ld_shared_u4(scales + at);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) odd |= ((((w[k] & 0x7f7f7f7fu) + 0x01010101u) | w[k]) & 0x80808080u) != 0;
            }
            uint32_t nan = 0;
            if (__any_sync(0xffffffffu, odd)) {
                for (int at = lane; at < S::SFB; at += 32) {
                    const int r = (at >> 4 & 31) + 32 * (at >> 2 & 3), block = 4 * (at >> 9) + (at & 3);
                    uint8_t* sf = smem + (scales - base) + at;
                    if ((*sf & 0x7f) == 0x7f) {
                        nan |= 1u << block;
                        *sf = 0;
                    } else if (*sf & 0x80) {
                        uint2* codes = reinterpret_cast<uint2*>(smem + (entry - base) + row_offset<ROWB>(r, 8 * block));
                        *codes = make_uint2(codes->x ^ 0x88888888u, codes->y ^ 0x88888888u);
                        *sf &= 0x7f;
                    }
                }
                nan = __reduce_or_sync(0xffffffffu, nan);
            }
            if (lane == 0) *(volatile uint16_t*)&notes.nan[i % kRing4] = nan;
            if (i > 0) warp_wait(notes.o_full, (i - 1) & 1);           // (V^T has been read)
            fence_proxy_async();
            tc_fence_after();
            __syncwarp();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < KS; ++k) tmem_copy_scales(tmem + S::T_VS + 4 * k, desc_scales(scales + 512 * k));
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    mma_e2m1(tmem + S::T_V, desc_rows(s_i + 32 * k, ROWB), desc_rows(entry + 32 * k, ROWB), idesc_v,
                             tmem + S::T_ONE, tmem + S::T_VS + 4 * k, k);
                mma_commit(bar(notes.v_full));
                mma_commit(bar(notes.empty[e]));
            }
            __syncwarp();
            warp_wait(notes.p_full, i & 1);
            warp_wait(notes.v_full, i & 1);
            const uint32_t sum = *(volatile int*)&notes.fresh ? 0u : 1u;
            fence_proxy_async();
            tc_fence_after();
            __syncwarp();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTile4 / 8; ++k)
                    mma_tf32_ts(tmem + S::T_O, tmem + S::T_V + 8 * k,
                                desc_rows(s_p + (k >> 2) * NP * 128 + (k & 3) * 32, 128), idesc_o, k ? 1u : sum);
                mma_commit(bar(notes.o_full));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(notes.drained));
        __syncwarp();
    } else if (tiles > 0) {
        // ============================================================ softmax and output
        const uint32_t lane_t = tmem + (warp * 32u << 16), p_to = s_p + warp * NP * 128 + (lane & 3) * 4;
        Cursor<kTile4> at;
        at.at = t0;
        at.locate(p, hcs, lane, early, request_of);
        at.bound(t1);

        // q: a head to 128 / HEADS threads, of which each takes DP dims
        constexpr int TPH = 128 / HEADS, DP = D / TPH, NW = DP / 2;
        uint32_t qw[NW];
        const int q_head = tid / TPH, q_dim = tid % TPH * DP;
        float kscale = 1.f;
        auto load_q = [&](const Cursor<kTile4>& of) {
            const int h = of.hc;
            const bool have = q_head < p.group;
            const uint16_t* from = static_cast<const uint16_t*>(p.q) + of.b * p.q_stride +
                                   (long long)(h * p.group + q_head) * D + q_dim;
            if constexpr (NW == 2) {
                const uint2 x = have ? __ldg(reinterpret_cast<const uint2*>(from)) : make_uint2(0, 0);
                qw[0] = x.x; qw[1] = x.y;
            } else {
#pragma unroll
                for (int k = 0; k < NW; k += 4) {
                    const uint4 x = have ? __ldg(reinterpret_cast<const uint4*>(from) + k / 4) : make_uint4(0, 0, 0, 0);
                    qw[k] = x.x; qw[k + 1] = x.y; qw[k + 2] = x.z; qw[k + 3] = x.w;
                }
            }
            kscale = p.c.k_scale ? __ldg(p.c.k_scale + h) : 1.f;
        };
        auto write_q = [&](int parity) {
            float amax = 0.f;
            bool bad = false;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float2 f = unpack2<S::QBF16>(qw[k]);
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                bad |= !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
            }
#pragma unroll
            for (int k = 1; k < TPH; k <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
            bad = (__ballot_sync(0xffffffffu, bad) >> (lane & ~(TPH - 1)) & ((1u << TPH) - 1u)) != 0;
            int e = static_cast<int>(__float_as_uint(amax) >> 23 & 255u) - 127;
            e = e < -100 ? -100 : e;
            const float up = __uint_as_float(static_cast<uint32_t>(128 - (bad ? 0 : e)) << 23);      // 2^(1 - e)
#pragma unroll
            for (int k0 = 0; k0 < NW; k0 += 4) {
                float y[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = k0 + k < NW && !bad ? unpack2<S::QBF16>(qw[k0 + k < NW ? k0 + k : 0]) : make_float2(0.f, 0.f);
                    y[2 * k] = f.x * up;
                    y[2 * k + 1] = f.y * up;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t codes = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int d = __float2int_rn(y[j]);
                        y[j] = (y[j] - static_cast<float>(d)) * 8.f;
                        codes |= digit_e2m1(d) << 4 * j;
                    }
                    uint8_t* to = smem + S::O_Q + row_offset<ROWB>(k * HEADS + q_head, (q_dim + 2 * k0) / 2);
                    if constexpr (NW == 2) *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(codes);
                    else *reinterpret_cast<uint32_t*>(to) = codes;
                }
            }
            // (a head with a value that is not finite has no finite score: its sums become NaN)
            if (tid % TPH == 0) {
                notes.mul[parity][q_head] =
                    bad ? 0.f : p.scale_log2 * kscale * __uint_as_float(static_cast<uint32_t>(126 + e) << 23);
                notes.odd[parity][q_head] = bad ? NAN : 0.f;
            }
            fence_proxy_async();
        };

        load_q(at);
        write_q(0);
        mbar_arrive(bar(notes.s_go));
        softmax_sync();                            // (factors)

        float o[HEADS], lsum[HEADS];               // sums taken out of the accumulator; of this thread's weights
        float ref[HEADS];                          // the softmax's references, the same in all threads
        uint32_t nan = 0;
        int parity = 0, kept = 0;                  // kept: tiles in the accumulator
        bool starts = true;
        // O of the tiles up to i comes out of the accumulator
        auto take_o = [&](int i) {
            wait(notes.o_full, i & 1);
            __syncwarp();
            tc_fence_after();
            float x[S::USED];
            tmem_ld<S::USED>(lane_t + S::T_O, x);
#pragma unroll
            for (int c = 0; c < HEADS; ++c) {
                o[c] += x[c];
                if constexpr (S::TWO) o[c] += x[HEADS + c];
            }
            tc_fence_before();
        };
        for (int i = 0; i < tiles; ++i) {
            if (starts) {
#pragma unroll
                for (int c = 0; c < HEADS; ++c) {
                    o[c] = lsum[c] = 0.f;
                    ref[c] = kNoMax;
                }
                nan = 0;
                kept = 0;
            }
            const unsigned tile = at.at;
            const bool ends = tile + 1 == at.end;
            const int slot = (at.rg.lo / kTile4 + static_cast<int>(tile - at.seg)) * kTile4 + tid, lo = at.rg.lo, n = at.rg.n;
            Cursor<kTile4> next;                   // (read where the piece ends)
            bool more = false;
            if (ends) {
                next = at;
                more = next.next_segment(p, hcs, t1);
                if (more) load_q(next);
            }

            // S: the digits' columns, the smallest weight first, heads in pairs
            warp_wait(notes.s_full, i & 1);
            tc_fence_after();
            uint64_t s2[HEADS / 2];
            const uint64_t eighth = f32_pair(0.125f, 0.125f);
#pragma unroll
            for (int part = S::NS / 32 - 1; part >= 0; --part) {
                float x[32];
                tmem_ld<32>(lane_t + S::T_S + 32 * part, x);
#pragma unroll
                for (int g = 32 / HEADS - 1; g >= 0; --g)
#pragma unroll
                    for (int c = 0; c < HEADS; c += 2) {
                        const uint64_t y = f32_pair(x[g * HEADS + c], x[g * HEADS + c + 1]);
                        s2[c / 2] = part == S::NS / 32 - 1 && g == 32 / HEADS - 1 ? y : fma_pair(s2[c / 2], eighth, y);
                    }
            }
            tc_fence_before();
            if (more) write_q(parity ^ 1);
            mbar_arrive(bar(notes.s_go));
            // log2-unit scores below their reference
            const bool in = slot >= lo && slot < n &&
                            (*(volatile uint8_t*)&notes.ok[i % kRing4][warp >> 1] >> ((warp & 1) * 2 + (lane >> 4)) & 1);
            float s[HEADS], x[HEADS], mul[HEADS];
            bool above = false;
#pragma unroll
            for (int c = 0; c < HEADS; c += 4) {
                const float4 m = *reinterpret_cast<const float4*>(&notes.mul[parity][c]);
                mul[c] = m.x; mul[c + 1] = m.y; mul[c + 2] = m.z; mul[c + 3] = m.w;
            }
#pragma unroll
            for (int c = 0; c < HEADS; ++c) {
                asm("{\n .reg .b32 h;\n mov.b64 {%0, h}, %1;\n}\n" : "=f"(s[c]) : "l"(c & 1 ? s2[c / 2] >> 32 : s2[c / 2]));
                x[c] = in ? fmaf(s[c], mul[c], -ref[c]) : -INFINITY;
                above |= x[c] > 8.f;
            }
            if (p.logits) {
                float4* to = reinterpret_cast<float4*>(p.logits + ((size_t)tile * kTile4 + tid) * HEADS);
#pragma unroll
                for (int c = 0; c < HEADS; c += 4) {
                    float y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k] = in ? s[c + k] * mul[c + k] : -INFINITY;
                    to[c / 4] = make_float4(y[0], y[1], y[2], y[3]);
                }
            }
            const bool moves = softmax_any(above);
            if (i > 0 && !starts) {
                if (moves || kept == kFlushTiles) {
                    take_o(i - 1);
                    kept = 0;
                } else {
                    warp_wait(notes.o_full, (i - 1) & 1);              // (P has been read)
                }
                nan |= *(volatile uint16_t*)&notes.nan[(i - 1) % kRing4];
            }
            if (moves) {
#pragma unroll
                for (int c = 0; c < HEADS; ++c) {
                    // the warp's largest score, as an integer of the same order (a NaN counts as -inf)
                    const int y = __float_as_int(in ? fmaxf(s[c] * mul[c], -INFINITY) : -INFINITY);
                    const int m = __reduce_max_sync(0xffffffffu, y ^ (y >> 31 & 0x7fffffff));
                    if (lane == 0) notes.top[warp][c] = __int_as_float(m ^ (m >> 31 & 0x7fffffff));
                }
                softmax_sync();
#pragma unroll
                for (int c = 0; c < HEADS; ++c) {
                    const float top = fmaxf(fmaxf(notes.top[0][c], notes.top[1][c]), fmaxf(notes.top[2][c], notes.top[3][c]));
                    const float r = fmaxf(ref[c], top), f = fast_exp2(ref[c] - r);
                    ref[c] = r;
                    lsum[c] *= f;
                    o[c] *= f;
                    x[c] = in ? fmaf(s[c], mul[c], -r) : -INFINITY;
                }
                // (the next tile's vote lies between this reading and the next writing)
            }
            // P, head by head a line of 32 slots
#pragma unroll
            for (int c = 0; c < HEADS; ++c) {
                const uint32_t to = p_to + c * 128 + (((lane >> 2) ^ c) << 4);
                const float y = fast_exp2(x[c]);
                lsum[c] += y;
                const uint32_t hi = to_tf32(y);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(hi) : "memory");
                if constexpr (S::TWO)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + HEADS * 128), "r"(__float_as_uint(y - __uint_as_float(hi)))
                                 : "memory");
            }
            if (tid == 0) *(volatile int*)&notes.fresh = kept == 0;
            ++kept;
            fence_proxy_async();
            mbar_arrive(bar(notes.p_full));
            starts = ends;
            if (!ends) {
                ++at.at;
                continue;
            }

            // ---- the piece's sums, and its output ----
            const bool cut = at.end != at.seg + at.rg.tiles || at.seg < t0;
            const bool begins = at.seg >= t0;
            const int h = at.hc, head0 = h * p.group, nheads = p.group;
#pragma unroll
            for (int c = 0; c < HEADS; ++c) {
                float x = lsum[c];
#pragma unroll
                for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
                if (lane == 0) notes.sum[warp][c] = x;
            }
            softmax_sync();
            take_o(i);
            nan |= *(volatile uint16_t*)&notes.nan[i % kRing4];
            const float vmul = p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f;
            const size_t row = (size_t)at.b * p.heads + head0;
            const int entry = piece_entry(share, begins);
#pragma unroll
            for (int c = 0; c < HEADS; ++c) {
                if (c >= nheads) break;
                float l = (notes.sum[0][c] + notes.sum[1][c]) + (notes.sum[2][c] + notes.sum[3][c]);
                if (l > 0.f) l += notes.odd[parity][c];
                float inv = 1.f;
                if (!cut) {
                    const float sk = p.sink ? __ldg(p.sink + head0 + c) * kLog2e : -INFINITY;
                    const float top = fminf(fmaxf(ref[c], sk), 3e38f);         // (a sink of +inf: out = 0)
                    const float f = fast_exp2(ref[c] - top);
                    const float all = l * f + fast_exp2(sk - top);
                    const bool some = all > 0.f || all != all;
                    inv = some ? vmul * f / all : 0.f;
                    if (tid == 0) {
                        const float l2 = some ? top + log2f(all) : -INFINITY;
                        if (p.lse) p.lse[row + c] = l2 * kLn2;
                        if (p.lse2) p.lse2[row + c] = l2;
                    }
                } else if (tid == 0) {
                    p.part_ml[(size_t)entry * HEADS + c] = make_float2(ref[c], l);
                }
                if (tid >= D) continue;
                const float x = nan >> (tid >> 4) & 1 || l != l ? NAN : o[c] * inv;
                if (cut)
                    p.part_o[((size_t)entry * HEADS + c) * D + tid] = x;
                else
                    static_cast<uint16_t*>(p.out)[(row + c) * D + tid] = static_cast<uint16_t>(pack2<S::QBF16>(x, 0.f));
            }
            at = next;
            parity ^= 1;
            softmax_sync();                        // (sums and references have been read)
        }
    } else {
        // (no tiles: nothing is waited for)
    }

    // every MMA and copy has ended before shared memory and TMEM go
    if (warp == 7) {
        const uint64_t since = globaltimer_ns();
        while (!mbar_try(bar(notes.drained), 0))
            if (globaltimer_ns() - since > kWaitNs4) break;
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 7) tmem_dealloc(tmem, S::COLS);
}

template <class S>
inline bool prepare_decode4_shape() {
    return cudaFuncSetAttribute(dsv4_gqa_decode4_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) ==
               cudaSuccess &&
           load_kernels(dsv4_gqa_decode4_kernel<S>);
}

// Rows of 64 and 128 dims: a cluster per segment, or the list on this file's kernel for up to 8 heads and on the other's
// for more.  The first call loads all.
template <int QKIND, int D>
inline int launch_decode4_dim(const DecodeParams& p, int nt, void* stream) {
    static unsigned long long ready = 0;
    using S = Shape4<QKIND, D>;
    using One = Shape<DSV4_GQA_E2M1, QKIND, D, 1>;
    using Two = Shape<DSV4_GQA_E2M1, QKIND, D, 2>;
    const int rc = once_per_device(ready, [] {
        return prepare_decode_shape<One>() && prepare_decode_shape<Two>() && prepare_decode4_shape<S>();
    });
    if (rc) return rc;
    if (nt == 2) return launch_decode_shape<Two>(p, stream);
    if (p.cluster) return launch_decode_shape<One>(p, stream);
    return launch(dsv4_gqa_decode4_kernel<S>, dim3(p.warps), kThreads4, S::SMEM, stream, 1, p);
}

template <int QKIND>
inline int launch_decode4(const DecodeParams& p, int head_dim, int nt, void* stream) {
    if (head_dim == 64) return launch_decode4_dim<QKIND, 64>(p, nt, stream);
    if (head_dim == 128) return launch_decode4_dim<QKIND, 128>(p, nt, stream);
    return launch_decode_dim<DSV4_GQA_E2M1, QKIND, 256>(p, nt, stream);
}

}  // namespace gqa
}  // namespace dsv4
