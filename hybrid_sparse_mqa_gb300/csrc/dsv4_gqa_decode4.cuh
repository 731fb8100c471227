// dsv4_gqa_decode4.cuh - the attention over long lists of 4-bit rows
// (DSV4_GQA_E2M1; include/dsv4gqa.h states what is computed), on the
// block-scaled 4-bit tensor cores.  It shares the list of tiles, its division
// into shares, the pieces of cut segments and the kernels behind it with
// dsv4_gqa_decode.cuh, whose own kernel takes the short lists; a share here
// belongs to a CTA and a tile has 128 slots.
//
// The instructions that turn codes into 16-bit operands bound a kernel on
// mma.sync (two conversions and two products for every 4 codes of K and of V
// and 16 slots; 4.5 bits a value come in faster than that: 32 x 2048..32768 rows,
// 32 / 8 heads of 128, 187 us for 659 MB, 2 x 131072 rows 89 us for 302 MB; this
// kernel, with the join: 124 and 60 us of device time, 5.3 and 5.0 TB/s).  Here no thread touches a code:
//   S   K is the A operand of a 4-bit MMA as it lies in the cache, block scales
//       and all.  q becomes a B operand of 4 bits, in eight digits of base 8,
//         q = 2^(E - 1) sum_k 8^-k d_k,   d_k = -4 .. 4,
//       each an e2m1 code (E: exponent of the head's largest value, of which what
//       is left out is 2^-23 at most).  Digits are columns; the accumulator sums
//       pairs of them, B's block scales being their weights (1, 2^-3), and the
//       softmax adds up the four sums.
//   V   its blocks run along the dims, not along the slots that O sums over, so
//       an MMA with the identity as A and V as B writes V^T, block scales
//       included, to TMEM as fp32 (every value exact), where it lies as the A
//       operand of
//   O^T += V^T P^T, a tf32 MMA.  Values have 6 bits; P is rounded to tf32's 11,
//       or is two of them where the output is f16.  (bf16 outputs of those two
//       calls with one piece are off by 1.67e-3 and 1.66e-3, relative rms, of
//       which their own rounding is 1.66e-3 and 1.65e-3; two pieces take 134 and
//       65 us.)
// A NaN among the block scales of V would reach all dims of its row through the
// identity's zeros, and the MMA takes scales without a sign.  So the issuing
// warps look through the scales of each tile; a NaN block is noted and its scale
// zeroed, a negative scale's sign moves into its codes.
//
// Roles of the 14 warps: 0 .. 3 and 4 .. 7 softmax of the even and of the odd
// tiles (a thread is a slot of S and a dim of O), each with references, sums and
// an O of its own, which meet at the end of a segment's part; 8 .. 11 copy
// (cp.async into a ring whose entries are K and V of a tile in turn); 12 looks
// through the scales and issues S, 13 V^T and O.  Two CTAs an SM.  (One softmax
// group: a tile's chain of waits and steps took 2300 clk of it.)
//
// An MMA here costs 9 (tf32, N = 16), 40 (4 bits, N = 32) and 64 clk (identity, N
// = 128) when its issuer is one thread that elect.sync picked in a converged
// warp, and 88 clk of issue for each where the thread is picked by its index.  A
// tile of 8 heads of 128 takes the tensor pipe 440 clk, and its 18 KB take an SM
// 780 clk at the memory's rate.  Bound by the instructions of the copying
// warps (without the copies of codes the same call takes 51 us for 57, without a
// part of the MMAs, the votes or the look through the scales no less), beside a
// start and a join of 12 us together.
#pragma once
#include <cstddef>

#include "dsv4_gqa_decode.cuh"

namespace dsv4 {
namespace gqa {

constexpr int kTile4 = 128;                // slots
constexpr int kThreads4 = 448;
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
    static constexpr int NS = 32;                            // columns of S: four pairs of digits of the heads
    static constexpr int USED = HEADS * (TWO ? 2 : 1);       // columns of O: heads, once for each piece of P
    static constexpr int NO = 16;                            // and of its MMA, which takes 16 at least
    // TMEM columns: V^T; S and O of each group; block scales of K (of each group) and V, of the digits and the identity
    static constexpr int T_V = 0, T_S = 128, T_O = T_S + 2 * NS, T_K = T_O + 2 * NO, T_VS = T_K + 8 * KS,
                         T_ONE = T_VS + 4 * KS, T_EIGHTH = T_ONE + 4;
    static constexpr int COLS = 256, CTAS = 2;
    static_assert(T_EIGHTH + 4 <= COLS, "TMEM");
    // shared memory
    static constexpr int ROWB = D / 2;                       // bytes of a row's codes
    static constexpr int SFB = kTile4 * D / 16;              // of a tile's block scales
    static constexpr int ENTRY = kTile4 * ROWB + SFB;
    static constexpr int I_BYTES = 128 * ROWB, Q_SET = NS * ROWB, Q_BYTES = 2 * Q_SET, P_BYTES = kTile4 * NO * 4;
    static constexpr int NOTES = 2048;                       // barriers and notes
    static constexpr int FIT = (113 * 1024 - I_BYTES - 2 * Q_BYTES - 2 * P_BYTES - NOTES) / ENTRY / 2 * 2;
    // (f16, 128 dims: 6 and not 8, which leaves the L1 cache more.  Device time of 32 x 2048..32768 rows, 32 / 8 heads of 128:
    // f16 133 us with 6 and 131 with 8, with weights kept 180 and 188; bf16 127 and 124, with weights 174 and 180.  The same
    // rows of 64 / 16 heads of 64, as many bytes: bf16 206 with 6 and 191 with 16, f16 211 and 197)
    static constexpr int ENTRIES = TWO && D == 128 ? 6 : FIT < 16 ? FIT : 16;
    static_assert(ENTRIES >= 4 && ENTRIES / 2 + 4 < kRing4, "the ring");
    static constexpr int O_I = 0, O_Q = O_I + I_BYTES, O_P = O_Q + 2 * Q_BYTES, O_RING = O_P + 2 * P_BYTES,
                         O_NOTES = O_RING + ENTRIES * ENTRY, SMEM = O_NOTES + NOTES;
    static_assert(O_P % 1024 == 0 && O_RING % 1024 == 0 && P_BYTES % 1024 == 0 && Q_SET % 1024 == 0 && ENTRY % 512 == 0,
                  "swizzle atoms");
};

// Shared memory matrix descriptor of a K-major operand with rows of `rowb` = 32, 64 or 128 bytes, swizzled over as many,
// groups of 8 rows `stride` bytes apart.
__device__ __forceinline__ uint64_t desc_rows(uint32_t start, int rowb, int stride) {
    return (uint64_t)((start & 0x3FFFFu) >> 4) | 1ull << 16 | (uint64_t)(stride >> 4) << 32 | 1ull << 46 |
           (uint64_t)(rowb == 32 ? 6 : rowb == 64 ? 4 : 2) << 61;
}
// The same operand `bytes` (a constant) further on.
__device__ __forceinline__ uint64_t desc_plus(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
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
// Whether any `x` of a softmax group's 128 threads holds, on its named barrier (1 or 2).
__device__ __forceinline__ bool softmax_any(bool x, int group) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x)), "r"(group + 1)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync(int group) { named_barrier_sync(group + 1, 128); }

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
__device__ __forceinline__ float2 f32_of(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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
// Global -> shared copy of N = 4 or 8 bytes; src_bytes = 0 writes zeros and reads nothing.
template <int N>
__device__ __forceinline__ void cp_async_few(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(src_bytes) : "memory");
}

// What a CTA's warps tell each other.
template <class S>
struct Notes {
    uint64_t full[S::ENTRIES], empty[S::ENTRIES];            // ring entries: rows have landed; MMAs have read them
    uint64_t v_fit[S::ENTRIES / 2];                          // V's scales have been looked through
    uint64_t q_full[2];                                      // digits of a piece are there (by its parity)
    uint64_t s_full[2], s_free[2], p_full[2], o_full[2];     // by group: S is written; read; P is written; O's MMAs are done
    uint64_t v_full;                                         // V^T is written
    uint64_t drained;
    uint32_t tmem;
    int abort, fresh[2];                                     // P's tile begins a new sum in the group's O
    // of tiles: valid 16-slot groups, two bits for each copying warp; bit 4: begins a piece
    uint8_t ok[kRing4][4];
    uint16_t nan[kRing4];                                    // and blocks of V that hold a NaN
    uint32_t nans[2];                                        // the same of a group's tiles of a piece
    alignas(16) float mul[2][S::HEADS];                      // score factors, by parity of the piece (read as float4)
    float odd[2][S::HEADS];                                  // NaN for a head whose query is not finite, else 0
    float top[2][4][S::HEADS], sum[2][4][S::HEADS], ref[2][S::HEADS];
};

template <class S>
__global__ void __launch_bounds__(kThreads4, S::CTAS) dsv4_gqa_decode4_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int D = S::D, HEADS = S::HEADS, KS = S::KS, ROWB = S::ROWB, NE = S::ENTRIES;
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

    // ---- what does not depend on the call's data (TMEM before the next kernel may start, which could take it first) ----
    if (warp == 13) tmem_alloc(smem_u32(&notes.tmem), S::COLS);
    if (tid == 0) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            mbar_init(bar(notes.full[e]), 128 + 4);
            mbar_init(bar(notes.empty[e]), 1);
            if (e & 1) mbar_init(bar(notes.v_fit[e / 2]), 1);
        }
        mbar_init(bar(notes.v_full), 1);
        mbar_init(bar(notes.drained), 2);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            mbar_init(bar(notes.q_full[g]), 128);
            mbar_init(bar(notes.s_full[g]), 1);
            mbar_init(bar(notes.s_free[g]), 128);
            mbar_init(bar(notes.p_full[g]), 128);
            mbar_init(bar(notes.o_full[g]), 1);
        }
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
        for (int i = 0; i < 4; ++i) {
            tmem_st1(tmem + (warp * 32u << 16) + S::T_ONE + i, 0x38383838u);             // e4m3: 1
            tmem_st1(tmem + (warp * 32u << 16) + S::T_EIGHTH + i, 0x20202020u);          // 2^-3
        }
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

    if (warp >= 8 && warp < 12) {
        // ============================================================ copies
        // A warp copies 32 slots of every tile: two groups of 16, each on one page.
        if (tiles > 0) {
            const int w = warp - 8;
            constexpr int PPR = ROWB / 16, RPI = 32 / PPR;             // pieces of a row, rows per warp-wide copy
            const int lane_row = lane / PPR, lane_piece = lane % PPR;
            const int page_mask = (1 << p.c.page_shift) - 1;
            const long long lane_off = lane_row * p.c.row_stride + lane_piece * 16, step = RPI * p.c.row_stride;
            const long long lane_block = (lane & 15) * p.c.b_row_stride;
            const uint32_t dst0 = 32 * w * ROWB + row_offset<ROWB>(lane_row, lane_piece * 16);
            const uint32_t dst1 = kTile4 * ROWB + (KS == 1 ? lane * 16 + w * 4 : (32 * w + lane) * 8);
            Cursor<kTile4> at;
            at.at = t0;
            at.locate(p, hcs, lane, early, request_of);
            at.bound(t1);
            // lanes 0 and 1: the page of a group of the tile, and whether it holds slots to attend
            int page = -1;
            bool wanted = false;
            int slot = 0;                          // the first of the warp's slots of the tile
            const int* table = nullptr;
            auto look = [&]() {
                const int s = slot + lane * 16;
                page = -1;
                wanted = lane < 2 && s < at.rg.n && s + 16 > at.rg.lo;
                if (wanted) page = __ldg(table + (s >> p.c.page_shift));
            };
            long long head = 0, block_head = 0;    // this lane's place in the KV head
            auto come_to = [&]() {
                head = at.hc * p.c.head_stride + lane_off;
                block_head = at.hc * p.c.b_head_stride + lane_block;
                slot = (at.rg.lo / kTile4 + static_cast<int>(at.at - at.seg)) * kTile4 + 32 * w;
                table = p.c.table + (long long)at.rq.row * p.c.table_stride;
            };
            come_to();
            look();
            int e = 0;
            uint32_t turn = 1;                     // parity that an entry's last reading has; 1: nothing was there
            for (int i = 0; i < tiles; ++i) {
                const int slot0 = slot, lo = at.rg.lo, n = at.rg.n;
                const bool begins = i == 0 || at.at == at.seg;
                const bool valid = page >= 0 && page < p.c.num_pages;
                if (wanted && !valid) atomicOr(p.err, DSV4_DEV_ERR_GQA_PAGE);
                const unsigned okm = __ballot_sync(0xffffffffu, wanted && valid);
                const int in_page = slot0 + lane * 16 & page_mask;
                const long long off = page * p.c.page_stride + in_page * p.c.row_stride;       // (used where valid)
                const long long block_off = page * p.c.b_page_stride + in_page * p.c.b_row_stride;
                long long go[2];
#pragma unroll
                for (int g = 0; g < 2; ++g) go[g] = __shfl_sync(0xffffffffu, off, g) + head;
                const long long bo = __shfl_sync(0xffffffffu, block_off, lane >> 4) + block_head;
                const bool whole = okm == 3u && slot0 >= lo && slot0 + 32 <= n;
                // the next tile's pages are on their way while this one's entries are waited for
                ++at.at;
                if (at.at < at.end) {
                    slot += kTile4;
                    look();
                } else if (at.next_segment(p, hcs, t1)) {
                    come_to();
                    look();
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    warp_wait(notes.empty[e], turn);
                    if (kv == 0 && lane == 0) *(volatile uint8_t*)&notes.ok[i % kRing4][w] = okm | (begins ? 16 : 0);
                    const uint32_t dst = ring + e * S::ENTRY;
                    const uint8_t *pool = kv ? p.c.v : p.c.k, *blocks = kv ? p.c.vb : p.c.kb;
                    {
                        // a lane's row: its block scales (128 dims: as they lie; warp 12 puts them where the MMA wants them)
                        const int s = slot0 + lane;
                        const bool in = whole || ((okm >> (lane >> 4) & 1) && s >= lo && s < n);
                        cp_async_few<4 * KS>(dst + dst1, blocks + (in ? bo : 0), in ? 4u * KS : 0u);
                    }
                    if (whole) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const uint8_t* src = pool + go[g];
#pragma unroll
                            for (int j = 0; j < 16 / RPI; ++j) {
                                cp_async_16(dst + dst0 + (16 * g + j * RPI) * ROWB, src, 16u);
                                src += step;
                            }
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < 2; ++g)
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
    } else if (warp == 12) {
        // ============================================================ scales, and S
        // An entry's block scales to the order of desc_scales, 512 bytes for each K step; bit 7 where a lane's have a NaN or a
        // sign.
        auto odd_scales = [&](uint32_t entry) {
            const uint32_t at = entry + kTile4 * ROWB;
            uint4 x, y = make_uint4(0, 0, 0, 0);
            if constexpr (KS == 1) {
                x = ld_shared_u4(at + lane * 16);
            } else {
                const uint2 a = ld_shared_u2(at + lane * 8), b = ld_shared_u2(at + 256 + lane * 8);
                const uint2 c = ld_shared_u2(at + 512 + lane * 8), d = ld_shared_u2(at + 768 + lane * 8);
                x = make_uint4(a.x, b.x, c.x, d.x);
                y = make_uint4(a.y, b.y, c.y, d.y);
                __syncwarp();
                st_shared_v4(at + lane * 16, x.x, x.y, x.z, x.w);
                st_shared_v4(at + 512 + lane * 16, y.x, y.y, y.z, y.w);
            }
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            uint32_t odd = 0;
#pragma unroll
            for (int k = 0; k < 4 * KS; ++k) odd |= ((w[k] & 0x7f7f7f7fu) + 0x01010101u) | w[k];
            return odd & 0x80808080u;
        };
        // Signs go to the codes; of V, NaN scales become 0 and their blocks are returned (a bit each).
        auto mend_scales = [&](uint32_t entry, bool is_v) {
            uint32_t nan = 0;
            __syncwarp();                          // (the lanes' lines are there)
#pragma unroll 1
            for (int at = lane; at < S::SFB; at += 32) {
                const int r = (at >> 4 & 31) + 32 * (at >> 2 & 3), block = 4 * (at >> 9) + (at & 3);
                uint8_t* sf = smem + (entry - base) + kTile4 * ROWB + at;
                if (is_v && (*sf & 0x7f) == 0x7f) {
                    nan |= 1u << block;
                    *sf = 0;
                } else if (*sf & 0x80) {
                    uint2* codes = reinterpret_cast<uint2*>(smem + (entry - base) + row_offset<ROWB>(r, 8 * block));
                    *codes = make_uint2(codes->x ^ 0x88888888u, codes->y ^ 0x88888888u);
                    *sf &= 0x7f;
                }
            }
            return __reduce_or_sync(0xffffffffu, nan);
        };
        constexpr uint32_t idesc = idesc_e2m1(128, S::NS);
        int e = 0, piece = -1;
        uint32_t turn = 0;
        for (int i = 0; i < tiles; ++i) {
            const int g = i & 1;
            const uint32_t entry = ring + e * S::ENTRY, scales = entry + kTile4 * ROWB;
            warp_wait(notes.full[e], turn);
            warp_wait(notes.full[e + 1], turn);
            uint32_t nan = 0;
            const uint32_t odd = odd_scales(entry) | odd_scales(entry + S::ENTRY);
            if (__any_sync(0xffffffffu, odd != 0)) {
                mend_scales(entry, false);
                nan = mend_scales(entry + S::ENTRY, true);
            }
            if (lane == 0) *(volatile uint16_t*)&notes.nan[i % kRing4] = nan;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(notes.v_fit[e / 2]));
            if (*(volatile uint8_t*)&notes.ok[i % kRing4][0] & 16) {
                ++piece;
                warp_wait(notes.q_full[piece & 1], piece >> 1 & 1);
            }
            warp_wait(notes.s_free[g], i >> 1 & 1 ^ 1);
            tc_fence_after();
            __syncwarp();
            if (elect_one()) {
                const uint32_t t_k = tmem + S::T_K + g * 4 * KS, t_s = tmem + S::T_S + g * S::NS;
                const uint64_t rows = desc_rows(entry, ROWB, 8 * ROWB), sf = desc_scales(scales);
                const uint64_t digits = desc_rows(s_q + (piece & 1) * S::Q_BYTES, ROWB, 8 * ROWB);
#pragma unroll
                for (int k = 0; k < KS; ++k) tmem_copy_scales(t_k + 4 * k, desc_plus(sf, 512 * k));
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        mma_e2m1(t_s, desc_plus(rows, 32 * k), desc_plus(digits, c * S::Q_SET + 32 * k), idesc, t_k + 4 * k,
                                 tmem + (c ? S::T_EIGHTH : S::T_ONE), k || c);
                mma_commit(bar(notes.s_full[g]));
                mma_commit(bar(notes.empty[e]));
            }
            __syncwarp();
            e += 2;
            if (e == NE) {
                e = 0;
                turn ^= 1;
            }
        }
        if (elect_one()) mma_commit(bar(notes.drained));
        __syncwarp();
    } else if (warp == 13) {
        // ============================================================ V^T and O
        const uint64_t identity = desc_rows(s_i, ROWB, 8 * ROWB);
        constexpr uint32_t idesc_v = idesc_e2m1(128, kTile4), idesc_o = idesc_tf32(128, S::NO);
        int e = 0;
        uint32_t turn = 0;
        for (int i = 0; i < tiles; ++i) {
            const int g = i & 1;
            const uint32_t entry = ring + (e + 1) * S::ENTRY, scales = entry + kTile4 * ROWB;
            warp_wait(notes.v_fit[e / 2], turn);
            if (i > 0) warp_wait(notes.o_full[g ^ 1], (i - 1) >> 1 & 1);         // (V^T has been read)
            tc_fence_after();
            __syncwarp();
            if (elect_one()) {
                const uint64_t rows = desc_rows(entry, ROWB, 8 * ROWB), sf = desc_scales(scales);
#pragma unroll
                for (int k = 0; k < KS; ++k) tmem_copy_scales(tmem + S::T_VS + 4 * k, desc_plus(sf, 512 * k));
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    mma_e2m1(tmem + S::T_V, desc_plus(identity, 32 * k), desc_plus(rows, 32 * k), idesc_v, tmem + S::T_ONE,
                             tmem + S::T_VS + 4 * k, k);
                mma_commit(bar(notes.v_full));
                mma_commit(bar(notes.empty[e + 1]));
            }
            __syncwarp();
            warp_wait(notes.p_full[g], i >> 1 & 1);
            const uint32_t sum = *(volatile int*)&notes.fresh[g] ? 0u : 1u;
            warp_wait(notes.v_full, i & 1);
            tc_fence_after();
            __syncwarp();
            if (elect_one()) {
                const uint64_t weights = desc_rows(s_p + g * S::P_BYTES, 128, 1024);
                const uint32_t t_o = tmem + S::T_O + g * S::NO;
                // (bf16 outputs: rows 8 .. 15 hold anything, and nobody reads their columns of O)
                mma_tf32_ts(t_o, tmem + S::T_V, weights, idesc_o, sum);
#pragma unroll
                for (int k = 1; k < kTile4 / 8; ++k)
                    mma_tf32_ts(t_o, tmem + S::T_V + 8 * k, desc_plus(weights, (k >> 2) * S::NO * 128 + (k & 3) * 32), idesc_o, 1u);
                mma_commit(bar(notes.o_full[g]));
            }
            __syncwarp();
            e += 2;
            if (e == NE) {
                e = 0;
                turn ^= 1;
            }
        }
        if (elect_one()) mma_commit(bar(notes.drained));
        __syncwarp();
    } else if (tiles > 0) {
        // ============================================================ softmax and output
        const int g = warp >> 2, quad = warp & 3, gt = tid & 127;
        const uint32_t lane_t = tmem + (quad * 32u << 16);
        // this slot's place in a line of P, of which piece c of 16 bytes lies at c ^ head
        const uint32_t p_to = s_p + g * S::P_BYTES + quad * S::NO * 128 + lane * 4;
        Cursor<kTile4> at;
        at.at = t0;
        at.locate(p, hcs, lane, early, request_of);
        at.bound(t1);

        // q: a head to 128 / HEADS threads, of which each takes DP dims
        constexpr int TPH = 128 / HEADS, DP = D / TPH, NW = DP / 2;
        uint32_t qw[NW];
        const int q_head = gt / TPH, q_dim = gt % TPH * DP;
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
        // the digits of a piece and its factors
        auto write_q = [&](int piece) {
            const int parity = piece & 1;
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
            // (held where 2^(1 - e) and the score's factor are normal; a smaller head loses nothing by it: bf16's values are
            // multiples of 2^-133, and the last digit counts 2^-147)
            e = e < -125 ? -125 : e;
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
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    uint32_t codes = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int d = __float2int_rn(y[j]);
                        y[j] = (y[j] - static_cast<float>(d)) * 8.f;
                        codes |= digit_e2m1(d) << 4 * j;
                    }
                    uint8_t* to = smem + S::O_Q + parity * S::Q_BYTES + (k & 1) * S::Q_SET +
                                  row_offset<ROWB>((k >> 1) * HEADS + q_head, (q_dim + 2 * k0) / 2);
                    if constexpr (NW == 2) *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(codes);
                    else *reinterpret_cast<uint32_t*>(to) = codes;
                }
            }
            // (a head with a value that is not finite has no finite score: its sums become NaN)
            if (gt % TPH == 0) {
                notes.mul[parity][q_head] =
                    bad ? 0.f : p.scale_log2 * kscale * __uint_as_float(static_cast<uint32_t>(126 + e) << 23);
                notes.odd[parity][q_head] = bad ? NAN : 0.f;
            }
            fence_proxy_async();
            mbar_arrive(bar(notes.q_full[parity]));
        };

        if (g == 0) {
            load_q(at);
            write_q(0);
        }
        // Pairs of heads: sums taken out of the accumulator; of this thread's weights; and, the same in all threads of the
        // group, the softmax's references, negated
        uint64_t o[HEADS / 2], lsum[HEADS / 2], ref[HEADS / 2];
        uint32_t nan = 0;
        int kept = 0;                              // tiles in the accumulator
        // the sums over the group's tiles up to i come out of the accumulator
        auto take_o = [&](int i) {
            warp_wait(notes.o_full[g], i >> 1 & 1);
            tc_fence_after();
            float x[S::USED];
            tmem_ld<S::USED>(lane_t + S::T_O + g * S::NO, x);
#pragma unroll
            for (int c = 0; c < HEADS; c += 2) {
                o[c / 2] = add_pair(o[c / 2], f32_pair(x[c], x[c + 1]));
                if constexpr (S::TWO) o[c / 2] = add_pair(o[c / 2], f32_pair(x[HEADS + c], x[HEADS + c + 1]));
            }
            tc_fence_before();
        };
        for (int i0 = 0, piece = 0; i0 < tiles; ++piece) {
            const int count = static_cast<int>(at.end - at.at);        // tiles of the piece
            Cursor<kTile4> next = at;
            bool ask = next.next_segment(p, hcs, t1) && g == 0;        // the next piece's digits are still to be written
            if (ask) load_q(next);
#pragma unroll
            for (int c = 0; c < HEADS / 2; ++c) {
                o[c] = lsum[c] = 0;
                ref[c] = f32_pair(-kNoMax, -kNoMax);
            }
            nan = 0;
            kept = 0;
            const int slot_0 = (at.rg.lo / kTile4 + static_cast<int>(at.at - at.seg)) * kTile4 + gt;
            int i = i0 + ((i0 ^ g) & 1);           // the group's first tile
            for (; i < i0 + count; i += 2) {
                const int k = i >> 1, slot = slot_0 + (i - i0) * kTile4;
                // S: the columns of digits, the smallest weight first, heads in pairs
                warp_wait(notes.s_full[g], k & 1);
                tc_fence_after();
                uint64_t s2[HEADS / 2];
                {
                    float x[32];
                    tmem_ld<32>(lane_t + S::T_S + g * S::NS, x);
                    const uint64_t step = f32_pair(0x1p-6f, 0x1p-6f);
#pragma unroll
                    for (int j = 32 / HEADS - 1; j >= 0; --j)
#pragma unroll
                        for (int c = 0; c < HEADS; c += 2) {
                            const uint64_t y = f32_pair(x[j * HEADS + c], x[j * HEADS + c + 1]);
                            s2[c / 2] = j == 32 / HEADS - 1 ? y : fma_pair(s2[c / 2], step, y);
                        }
                }
                tc_fence_before();
                mbar_arrive(bar(notes.s_free[g]));
                // log2-unit scores below their reference
                const bool in = slot >= at.rg.lo && slot < at.rg.n &&
                                (*(volatile uint8_t*)&notes.ok[i % kRing4][quad] >> (lane >> 4) & 1);
                uint64_t x[HEADS / 2];
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < HEADS / 2; c += 2) {
                    const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(&notes.mul[piece & 1][2 * c]);
                    x[c] = fma_pair(s2[c], m.x, ref[c]);
                    x[c + 1] = fma_pair(s2[c + 1], m.y, ref[c + 1]);
                }
                const bool all_in = __all_sync(0xffffffffu, in);
                if (!all_in) {
#pragma unroll
                    for (int c = 0; c < HEADS / 2; ++c) x[c] = in ? x[c] : f32_pair(-INFINITY, -INFINITY);
                }
#pragma unroll
                for (int c = 0; c < HEADS / 2; ++c) {
                    const float2 y = f32_of(x[c]);
                    top = fmaxf(top, fmaxf(y.x, y.y));
                }
                const bool above = top > 8.f;
                if (p.logits) {
                    float4* to = reinterpret_cast<float4*>(p.logits + ((size_t)(at.at + (i - i0)) * kTile4 + gt) * HEADS);
#pragma unroll
                    for (int c = 0; c < HEADS; c += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(&notes.mul[piece & 1][c]);
                        const float2 y = f32_of(s2[c / 2]), z = f32_of(s2[c / 2 + 1]);
                        to[c / 4] = in ? make_float4(y.x * m.x, y.y * m.y, z.x * m.z, z.y * m.w)
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    }
                }
                const bool moves = softmax_any(above, g);
                if (kept > 0) {
                    // (P of the group's last tile has been read)
                    if (moves || kept == kFlushTiles) {
                        take_o(i - 2);
                        kept = 0;
                    } else {
                        warp_wait(notes.o_full[g], (i - 2) >> 1 & 1);
                    }
                    nan |= *(volatile uint16_t*)&notes.nan[(i - 2) % kRing4];
                }
                if (moves) {
                    const float* mul = notes.mul[piece & 1];
#pragma unroll
                    for (int c = 0; c < HEADS; ++c) {
                        // the warp's largest score, as an integer of the same order (a NaN counts as -inf)
                        const float2 y2 = f32_of(s2[c / 2]);
                        const float z = (c & 1 ? y2.y : y2.x) * mul[c];
                        const int y = __float_as_int(in ? fmaxf(z, -INFINITY) : -INFINITY);
                        const int m = __reduce_max_sync(0xffffffffu, y ^ (y >> 31 & 0x7fffffff));
                        if (lane == 0) notes.top[g][quad][c] = __int_as_float(m ^ (m >> 31 & 0x7fffffff));
                    }
                    softmax_sync(g);
#pragma unroll
                    for (int c = 0; c < HEADS; c += 2) {
                        const float2 was = f32_of(ref[c / 2]), y = f32_of(s2[c / 2]), ls = f32_of(lsum[c / 2]), os = f32_of(o[c / 2]);
                        auto largest = [&](int k) {
                            return fmaxf(fmaxf(notes.top[g][0][k], notes.top[g][1][k]), fmaxf(notes.top[g][2][k], notes.top[g][3][k]));
                        };
                        const float r0 = fmaxf(-was.x, largest(c)), r1 = fmaxf(-was.y, largest(c + 1));
                        const float f0 = fast_exp2(-was.x - r0), f1 = fast_exp2(-was.y - r1);
                        ref[c / 2] = f32_pair(-r0, -r1);
                        lsum[c / 2] = f32_pair(ls.x * f0, ls.y * f1);
                        o[c / 2] = f32_pair(os.x * f0, os.y * f1);
                        x[c / 2] = in ? f32_pair(fmaf(y.x, mul[c], -r0), fmaf(y.y, mul[c + 1], -r1)) : f32_pair(-INFINITY, -INFINITY);
                    }
                    // (the next tile's vote lies between this reading and the next writing)
                }
                // P, head by head a line of 32 slots
                auto put = [&](int c, float y) {
                    const uint32_t to = (p_to ^ (c << 4)) + c * 128, hi = to_tf32(y);
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(hi) : "memory");
                    if constexpr (S::TWO)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + HEADS * 128), "r"(__float_as_uint(y - __uint_as_float(hi)))
                                     : "memory");
                };
#pragma unroll
                for (int c = 0; c < HEADS; c += 2) {
                    const float2 z = f32_of(x[c / 2]);
                    const float y0 = fast_exp2(z.x), y1 = fast_exp2(z.y);
                    lsum[c / 2] = add_pair(lsum[c / 2], f32_pair(y0, y1));
                    put(c, y0);
                    put(c + 1, y1);
                }
                if (gt == 0) *(volatile int*)&notes.fresh[g] = kept == 0;
                ++kept;
                fence_proxy_async();
                mbar_arrive(bar(notes.p_full[g]));
                if (ask) {
                    write_q(piece + 1);
                    ask = false;
                }
            }
            if (ask) write_q(piece + 1);

            // ---- the piece's sums meet in shared memory; its output, heads in turn to the groups ----
            // (loops and not straight code: what runs once a piece comes from far away)
            {
                // a head's sum over the warp to lanes 4 head .. 4 head + 3
                const bool up = lane & 16, mid = lane & 8, low = lane & 4;
                auto across = [&](uint64_t x, int k) {
                    const float2 y = f32_of(x);
                    return f32_pair(__shfl_xor_sync(0xffffffffu, y.x, k), __shfl_xor_sync(0xffffffffu, y.y, k));
                };
                const uint64_t a0 = add_pair(up ? lsum[2] : lsum[0], across(up ? lsum[0] : lsum[2], 16));
                const uint64_t a1 = add_pair(up ? lsum[3] : lsum[1], across(up ? lsum[1] : lsum[3], 16));
                const float2 b = f32_of(add_pair(mid ? a1 : a0, across(mid ? a0 : a1, 8)));
                float l = (low ? b.y : b.x) + __shfl_xor_sync(0xffffffffu, low ? b.x : b.y, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                if (!(lane & 3)) notes.sum[g][quad][lane >> 2] = l;
            }
            if (kept > 0) {
                take_o(i - 2);
                nan |= *(volatile uint16_t*)&notes.nan[(i - 2) % kRing4];
            }
            float* const sums = reinterpret_cast<float*>(smem + S::O_P);         // (P of both has been read)
#pragma unroll
            for (int c = 0; c < HEADS; c += 2) {
                const float2 os = f32_of(o[c / 2]), r = f32_of(ref[c / 2]);
                float* to = sums + (g * S::P_BYTES + c * 512) / 4 + gt;
                to[0] = os.x;
                to[128] = os.y;
                if (gt == 0) {
                    notes.ref[g][c] = -r.x;
                    notes.ref[g][c + 1] = -r.y;
                }
            }
            if (gt == 0) notes.nans[g] = nan;
            named_barrier_sync(3, 256);
            {
                nan |= notes.nans[g ^ 1];
                const bool begins = at.seg >= t0, cut = !begins || at.end != at.seg + at.rg.tiles;
                const int h = at.hc, head0 = h * p.group;
                const float vmul = p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f;
                const size_t row = (size_t)at.b * p.heads + head0;
                const int entry = piece_entry(share, begins);
#pragma unroll 1
                for (int c = g; c < p.group; c += 2) {
                    const float r0 = notes.ref[0][c], r1 = notes.ref[1][c], r = fmaxf(r0, r1);
                    const float f0 = fast_exp2(r0 - r), f1 = fast_exp2(r1 - r);
                    float l = ((notes.sum[0][0][c] + notes.sum[0][1][c]) + (notes.sum[0][2][c] + notes.sum[0][3][c])) * f0 +
                              ((notes.sum[1][0][c] + notes.sum[1][1][c]) + (notes.sum[1][2][c] + notes.sum[1][3][c])) * f1;
                    if (l > 0.f) l += notes.odd[piece & 1][c];
                    float inv = 1.f;
                    if (!cut) {
                        const float sk = p.sink ? __ldg(p.sink + head0 + c) * kLog2e : -INFINITY;
                        const float top = fminf(fmaxf(r, sk), 3e38f);          // (a sink of +inf: out = 0)
                        const float f = fast_exp2(r - top);
                        const float all = l * f + fast_exp2(sk - top);
                        const bool some = all > 0.f || all != all;
                        inv = some ? vmul * f / all : 0.f;
                        if (gt == 0) {
                            const float l2 = some ? top + log2f(all) : -INFINITY;
                            if (p.lse) p.lse[row + c] = l2 * kLn2;
                            if (p.lse2) p.lse2[row + c] = l2;
                        }
                    } else if (gt == 0) {
                        p.part_ml[(size_t)entry * HEADS + c] = make_float2(r, l);
                    }
                    if (gt >= D) continue;
                    const float* from = sums + c * 128 + gt;
                    const float x = nan >> (gt >> 4) & 1 || l != l ? NAN : (from[0] * f0 + from[S::P_BYTES / 4] * f1) * inv;
                    if (cut)
                        p.part_o[((size_t)entry * HEADS + c) * D + gt] = x;
                    else
                        static_cast<uint16_t*>(p.out)[(row + c) * D + gt] = static_cast<uint16_t>(pack2<S::QBF16>(x, 0.f));
                }
            }
            named_barrier_sync(3, 256);            // (all of it has been read)
            at = next;
            i0 += count;
        }
    }

    // every MMA and copy has ended before shared memory and TMEM go
    if (warp == 13) {
        const uint64_t since = globaltimer_ns();
        while (!mbar_try(bar(notes.drained), 0))
            if (globaltimer_ns() - since > kWaitNs4) break;
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13) tmem_dealloc(tmem, S::COLS);
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
    using Many = Shape<DSV4_GQA_E2M1, QKIND, D, 1, true>;
    const int rc = once_per_device(ready, [] {
        return prepare_decode_shape<One>() && prepare_decode_shape<Many>() && prepare_decode_shape<Two>() &&
               prepare_decode4_shape<S>();
    });
    if (rc) return rc;
    if (nt == 2) return launch_decode_shape<Two>(p, stream);
    if (p.cluster)
        return (long long)p.batch * p.c.kv_heads > kMaxCtas ? launch_decode_shape<Many>(p, stream)
                                                            : launch_decode_shape<One>(p, stream);
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
