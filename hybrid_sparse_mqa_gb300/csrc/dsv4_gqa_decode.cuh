// dsv4_gqa_decode.cuh - one-token attention over a paged grouped-query cache
// (include/dsv4gqa.h states what is computed).  The kernel is a template over
// the cache's element type, compiled once per type in
// dsv4_gqa_decode_{bf16,f16,e4m3,e4m3_f16,e2m1,e2m1_f16}.cu; dsv4_gqa_decode.cu holds the host side
// and the kernels that join split requests and accumulate weights.
//
// Work: a segment is one (request, KV head, group of up to 8 NT query heads);
// its key range is cut into tiles of TT slots.  All tiles of the batch form
// one list, of which every warp of the grid takes a contiguous share, so a
// ragged batch is as balanced as a uniform one and a long request is split
// over as many warps as it needs.  A segment that lies in one share is finished
// there; of a cut one every share leaves (unnormalised output, reference, sum)
// in fp32 in the workspace, at most two pieces each, which the join kernel
// merges.  (A CTA per share with a merge of its warps in shared memory took
// 56 us where a share per warp takes 35: 48 requests of up to 2000 rows, 16
// heads of 64.)
//
// SMs do not get equal bandwidth (equal shares ended between 117 and 165 us
// for 2 x 131072 rows), so of a long list the last 3/32 of every warp's part
// are given out to whoever is free.  A share for each warp of a CTA makes up one
// more CTA of the grid, which a resident CTA that runs out of tiles takes over
// before it is launched (clusterlaunchcontrol.try_cancel): the hardware's own
// queue, with no counter in memory.  What a share holds does not depend on who
// takes it, so results do not either.
//
// Short lists (SEG) are done in one launch: a cluster of 1 to 8 CTAs takes a
// segment, its warps equal parts of the tiles, and they merge through
// distributed shared memory; with weights, every warp then adds those of its
// own tiles.  That spares the other launches (2.4 us of host time each) and the
// pieces' way through L2.
//
// A warp streams its tiles through its own ring of cp.async stages, which runs
// ahead over segment and share boundaries, and the queries of the next segment
// with them.  Scores are computed transposed, S^T = K Q^T, so the 16 rows of an
// m16n8k16 MMA are slots and its 8 columns query heads: a group of 8 heads
// wastes nothing.  The exponentials become the B operand of
// O^T = V^T P^T by one 8x8 transposition in registers (movmatrix).  The
// softmax is online with a lazy reference: a tile's scores are compared with
// the running reference by one vote, and the reference moves (and O and the
// sums are rescaled) only when some score exceeds it by more than 2^8 (f16
// operands: 2^15, see Shape).
//
// Bound by HBM for lists of 100 tiles per warp and more: 334 us for 2.34 GB (32 x
// 2048..32768 rows, 8 KV heads of 128, bf16: 7.0 TB/s), 165 us for 1.07 GB (2 x
// 131072).  Shorter lists lose to the uneven end (98 us for 566 MB, 64 x
// 1024..16384 e4m3 rows), the start (3 us: length, page, rows) and the join (4 us).
//
// Precision: scores, references, sums, O and the merge are fp32.  For 16-bit
// caches P enters the MMA as the sum of two 16-bit values (the rounded value
// and the rounded rest), so its rounding stays below 2^-16 of it and the
// output's own rounding is what remains; the second MMA costs nothing
// measurable in a kernel bound by memory.  For e4m3 caches codes are exact in
// f16, and P is two f16 values where the output is f16, one where it is bf16
// (Shape::TWO).  Pieces of f16 end at 2^-24, which adds 2^-36 of the largest P
// at most (Shape::DROP).  q beside e4m3 rows is scaled by a power of two per
// head so that its largest value lies in [2^14, 2^15): a bf16 value keeps all
// its bits down to 2^-31 of the largest, and below that is off by at most
// 2^-39 of it.
#pragma once

#include "dsv4_gqa.cuh"

namespace dsv4 {
namespace gqa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3e38f;           // reference of a head that has seen no score: below every finite one
constexpr int kWarps = 4;                  // warps per CTA
constexpr int kMaxCtas = 304;              // resident at once: two on each of 152 SMs
// What is kept back of a warp's part of a long list, in 32nds.  Taking another
// share costs a piece to write and join and some stalled loads: 32 x
// 2048..32768 rows (230 tiles per warp) go from 345 to 328 us, 2 x 131072 rows
// (108) from 170 to 163, while 64 x 1024..16384 e4m3 rows (57) would go from 98
// to 99 and 48 x up to 2000 rows of 64 (15) from 34 to 36.  Two or three rounds
// of smaller shares gained no more.
constexpr int kTail = 3;
constexpr int kClaimTiles = 64;            // a list is long from so many tiles per resident warp
constexpr int kClaimAhead = 4;             // tiles before the end of a share at which the next is asked for
constexpr int kClaimRing = 16;             // claims that a warp may be behind another of its CTA
constexpr int kWaitLimit = 1 << 20;        // polls (some ten ns each) before a claim is given up

struct DecodeParams {
    Cache c;
    const void* q;
    long long q_stride;                    // elements
    int q_bf16;                            // q and out: bf16 (else f16)
    int batch, heads, group, chunks;       // group: query heads per KV head; chunks of 8 NT heads each
    const int* lens;
    const int* req;
    int window, max_len;
    const float* sink;
    float scale_log2;                      // scale * log2 e
    void* out;
    float* lse;
    // workspace
    float* part_o;                         // [2 shares][8 NT][D]
    float2* part_ml;                       // [2 shares][8 NT]
    float* lse2;                           // [batch][heads], log2 units (with weights)
    int4* info;                            // [batch] (with weights): first tile, next request of the same row or
                                           // -1, whether it is the row's first, rows
    float* logits;                         // [tiles][TT][8 NT], log2 units (with weights), or null
    // weights
    const float* w_in;
    float* w_out;
    long long width;
    float decay;
    int min_tiles;                         // a share has at least this many tiles (where there are as many)
    int warps;                             // of the resident CTAs
    int claims;                            // CTAs of the grid behind those, to be claimed (0: none)
    int claim_ahead, claim_polls;          // kClaimAhead, kWaitLimit (a test sets others)
    int pieces;                            // bound on the shares (for the host)
    int cluster;                           // CTAs per segment, where segments are not cut (0: by shares)
    unsigned int* err;
};

// The slots lo .. n-1 that a request attends and the tiles of TT slots that
// they touch.
struct Range {
    int lo, n, tiles;
};
template <int TT>
__device__ __forceinline__ Range key_range(const DecodeParams& p, int n) {
    Range r;
    r.n = n;
    r.lo = p.window > 0 && n > p.window ? n - p.window : 0;
    r.tiles = n > 0 ? (n - 1) / TT - r.lo / TT + 1 : 0;
    return r;
}

// How the list's `total` tiles are shared out: n parts of q tiles each (the
// first r one more), each a share; or, where tail > 0, each part two shares, of
// which the second holds `tail` tiles.  Shares are numbered in the order of the
// list.
struct Shares {
    int count, n;
    unsigned q, r, tail;
};
__device__ __forceinline__ Shares make_shares(const DecodeParams& p, unsigned total) {
    Shares s;
    const bool cut = p.claims && total >= (unsigned)p.warps * kClaimTiles;
    const unsigned most = total / p.min_tiles;
    s.n = cut ? p.warps : most < 1u ? 1 : (most > (unsigned)p.warps ? p.warps : (int)most);
    s.q = total / s.n;
    s.r = total - s.q * s.n;
    s.tail = cut ? s.q * kTail / 32 : 0u;
    s.count = cut ? 2 * s.n : s.n;
    return s;
}
// The list index that share i begins at.
__device__ __forceinline__ unsigned share_begin(const Shares& s, int i) {
    const unsigned part = s.tail ? (i + 1) >> 1 : i;       // it begins, or the one before it ends
    const unsigned at = part * s.q + min(part, s.r);
    return s.tail && i & 1 ? at - s.tail : at;
}
// The share that tile t lies in.
__device__ __forceinline__ int share_of(const Shares& s, unsigned t) {
    const unsigned longer = s.r * (s.q + 1);
    const unsigned part = t < longer ? t / (s.q + 1) : s.r + (t - longer) / s.q;
    if (!s.tail) return static_cast<int>(part);
    const unsigned left = (part + 1) * s.q + min(part + 1, s.r) - t;         // tiles to the end of the part
    return static_cast<int>(2 * part) + (left <= s.tail ? 1 : 0);
}
// The workspace entry of share i's piece of a cut segment: one that begins
// with its segment can only be the share's last, any other its first.
__device__ __forceinline__ int piece_entry(int share, bool begins) { return 2 * share + (begins ? 1 : 0); }

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes (low 16 bits) -> two f16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(codes));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(r) : "r"(codes));
    return r;
}
// Eight e2m1 codes -> four pairs of f16 values (byte i holds pair i, the low half first), exactly.
__device__ __forceinline__ void e2m1x8_f16x2(uint32_t codes, uint32_t (&r)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(codes));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (x & mask) | (y & ~mask)
__device__ __forceinline__ uint32_t pick_bits(uint32_t x, uint32_t y, uint32_t mask) {
    return (x & mask) | (y & ~mask);
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_shared_u2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        return pack_bf16x2(lo, hi);
    } else {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&v);
    }
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// How the copies below use L2: lines that are the first to go where a cache row
// is read once per call (what is written for the kernels behind stays: with
// weights 37 MB of scores), ordinary ones where every 16 query heads read it
// again (64 heads per KV head: 635 us and not 665).  16-byte global -> shared
// copy; src_bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ uint64_t read_policy(bool once) {
    uint64_t p;
    if (once)
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    else
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void cp_async_16_hint(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async_16_whole(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
// The same for N = 4, 8 or 16 bytes (block scales of a row).
template <int N>
__device__ __forceinline__ void cp_async_hint(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %2, %3, %4;" ::"r"(dst), "l"(src), "n"(N),
                 "r"(src_bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Asks for a CTA of the grid that has not been launched; the answer's 16 bytes
// land at `result` and complete on `bar`.
__device__ __forceinline__ void claim_submit(uint32_t result, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     result),
                 "r"(bar)
                 : "memory");
}
// The index of the CTA that was taken over, or -1 if none was left.
__device__ __forceinline__ int claim_result(uint32_t result) {
    uint32_t ok, x;
    asm volatile(
        "{\n .reg .pred p;\n .reg .b128 r;\n"
        " ld.shared.b128 r, [%2];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
        " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
        : "=r"(ok), "=r"(x)
        : "r"(result)
        : "memory");
    return ok ? static_cast<int>(x) : -1;
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// ---------------------------------------------------------------- shape
// KIND: DSV4_GQA_BF16 / F16 / E4M3 / E2M1; QKIND: of the queries and the output,
// BF16 or F16.  A warp's stage is TT rows of K and of V, and of their block scales
// behind both (E2M1).
template <int KIND_, int QKIND, int D_, int NT_, bool MANY = false>
struct Shape {
    static constexpr int KIND = KIND_, D = D_, NT = NT_;
    static constexpr bool FP8 = KIND == DSV4_GQA_E4M3, FP4 = KIND == DSV4_GQA_E2M1, CODES = FP8 || FP4;
    static constexpr bool BF16 = KIND == DSV4_GQA_BF16;      // operand type of the MMAs (codes: f16)
    static constexpr bool QBF16 = QKIND == DSV4_GQA_BF16;
    static_assert(CODES || QKIND == KIND, "only rows of codes are read by queries of another type");
    // P in two pieces.  One f16 is off by up to 2^-11 of it, a quarter of a bf16 output's rounding but as much as an f16
    // output's: 8 x 1024..16384 e4m3 rows of 128, 32 / 4 heads, f16 out: an error of 5.7e-6 (rms) with one piece and of
    // 4.3e-6, the output's own rounding, with two
    static constexpr bool TWO = !CODES || !QBF16;
    static constexpr bool LIST = !(FP4 && D <= 128 && NT == 1);      // else dsv4_gqa_decode4.cuh takes the lists
    // Queries as B operands in shared memory and not in registers: 16 heads of 256 beside 4-bit rows would want 64 of them
    // beside the output's 128 (64 x 1024..16384 rows, 32 / 2 heads: 141 us with
    // them in registers, some spilled, and 125 without).
    static constexpr bool QSMEM = FP4 && D == 256 && NT == 2;
    static constexpr int ROWB = FP4 ? D / 2 : D * (FP8 ? 1 : 2);       // bytes of a row
    static constexpr int BLKB = FP4 ? D / 16 : 0;            // bytes of its block scales
    static constexpr int TT = FP4 ? 2048 / ROWB : 4096 / ROWB < 16 ? 16 : 4096 / ROWB;
    static constexpr int MT = TT / 16;                       // 16-slot MMA tiles
    static constexpr int DT = D / 16;                        // 16-dim tiles
    static constexpr int HEADS = 8 * NT;                     // query heads of a segment (padded)
    // The reference of a softmax lies DROP below the largest score when it moves, and moves when a score exceeds that
    // score by more than SLACK (log2 units).  P as f16 ends at 2^-24, so it is kept as large as f16 allows: its largest
    // values lie in [2^11, 2^15], and rounding to zero or to subnormals is off by at most 2^-25 2^-DROP = 2^-36 of the
    // largest.  (bf16 has the exponents of fp32 and does without.)  Both are added with the rounding that keeps P in that
    // range where scores are so large that fp32 holds them 2 units apart or more.
    static constexpr float DROP = BF16 ? 0.f : 11.f, SLACK = BF16 ? 8.f : 4.f;
    static constexpr int W = kWarps;
    static constexpr int TILE_BYTES = TT * ROWB;             // K or V of a stage
    static constexpr int BLOCK_BYTES = TT * BLKB;            // their block scales
    // MANY (rows of 4 bits, a CTA per segment, more of them than run at once): shallower rings, so that more CTAs do.
    // 128 x 1..1000 rows, 8 KV heads of 128: 39.4 us without and 34.0 with, 48 x 1..1000, 16 of 64: 23.6 and 21.5; where all
    // run at once anyway, 32 x 500..1000 rows: 15.0 and 17.7
    static constexpr int STAGES = QSMEM ? 4 : FP4 && !MANY ? 5 : 3;
    static constexpr int STAGE_BYTES = 2 * (TILE_BYTES + BLOCK_BYTES);
    static constexpr int CTAS = TILE_BYTES > 4096 ? 1 : !MANY ? 2 : D == 64 ? 4 : 3;     // per SM (what shared memory holds)
    static constexpr int WARP_RING = STAGES * STAGE_BYTES;
    static constexpr int RING_BYTES = W * WARP_RING;
    // queries of a segment, a row per head (16 bytes of padding spread the rows over the banks where there is room)
    static constexpr int QROW = D * 2 + (NT == 1 ? 16 : 0);
    // (16 heads of 256 beside e4m3 rows: two CTAs fit an SM only without the buffers; 64 x 1024..16384 rows, 64 / 4
    // heads: 354 us with them and 246 without)
    static constexpr int Q_BYTES = CODES && D == 256 && NT == 2 ? 0 : HEADS * QROW;
    static constexpr int OPERAND_BYTES = QSMEM ? D / 16 * NT * 256 : 0;
    static constexpr int SMEM = RING_BYTES + W * (Q_BYTES + OPERAND_BYTES);
    static constexpr int PPR = ROWB / 16;                    // 16-byte pieces per row
    static constexpr int RPI = 32 / PPR;                     // rows per warp-wide copy
};

// Byte offset of 16-byte piece `piece` of row `row` in a K (V) tile.  The
// swizzles spread what one phase of the readers' loads touches over all
// banks: ldmatrix reads 8 rows of one piece; the e4m3 readers read rows
// (g, g + 1) x pieces 4j .. 4j + 3 of K and rows 2t (t = 0..3) x two
// neighbouring pieces of V; the e2m1 readers 128 bytes of neighbouring rows of
// K (rows of 32 and 64 bytes lie as they are) and rows 2t x 32 bytes of V.
template <class S>
__device__ __forceinline__ uint32_t k_offset(int row, int piece) {
    if constexpr (!S::CODES) return row * S::ROWB + ((piece ^ (row & 7)) << 4);
    if constexpr (S::ROWB <= 64) return row * S::ROWB + (piece << 4);
    return row * S::ROWB + ((piece ^ ((row & 1) << 2)) << 4);
}
template <class S>
__device__ __forceinline__ uint32_t v_offset(int row, int piece) {
    if constexpr (!S::CODES) return row * S::ROWB + ((piece ^ (row & 7)) << 4);
    if constexpr (S::ROWB == 32) return (row >> 2) * 128 + (((((row & 3) << 1) | piece) ^ ((row >> 1) & 2)) << 4);
    const int f = ((row >> 1) & 3) << 1;
    if constexpr (S::ROWB == 64) return (row >> 1) * 128 + (((((row & 1) << 2) | piece) ^ f) << 4);
    return row * S::ROWB + ((piece ^ f) << 4);
}

// ---------------------------------------------------------------- the walk over tiles
// A position in a warp's share of the tile list.  Every warp has two: one that
// runs ahead issuing copies and one that follows computing.
template <int TT>
struct Cursor {
    int b, hc;                 // request; KV head * chunks + chunk
    Request rq;
    Range rg;
    unsigned seg;              // list index of the segment's first tile
    unsigned end;              // end of the share's part of it
    unsigned at;               // current tile

    __device__ __forceinline__ void load(const DecodeParams& p) {
        unsigned ignored = 0;
        rq = read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, ignored);
        rg = key_range<TT>(p, rq.n);
    }
    __device__ __forceinline__ void bound(unsigned t1) {
        end = seg + rg.tiles < t1 ? seg + rg.tiles : t1;
    }
    // finds the segment of list index `at`; the whole warp (lane's requests: early, later(32 + lane), ...)
    template <class F>
    __device__ __forceinline__ void locate(const DecodeParams& p, int hcs, int lane, const Request& early, F&& later) {
        unsigned run = 0;
        for (int from = 0;; from += 32) {
            const Request mine = from ? later(from + lane) : early;
            const unsigned cnt = key_range<TT>(p, mine.n).tiles * hcs;
            unsigned incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned here = __ballot_sync(0xffffffffu, at < run + incl);
            if (here || from + 32 >= p.batch) {
                const int i = here ? __ffs(here) - 1 : 0;
                b = from + i;
                seg = run + __shfl_sync(0xffffffffu, incl - cnt, i);
                rq.row = __shfl_sync(0xffffffffu, mine.row, i);
                rq.n = __shfl_sync(0xffffffffu, mine.n, i);
                break;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        rg = key_range<TT>(p, rq.n);
        hc = rg.tiles > 0 ? static_cast<int>((at - seg) / rg.tiles) : 0;
        seg += hc * rg.tiles;
    }
    // to the next segment that has tiles; false at the end of the share
    __device__ __forceinline__ bool next_segment(const DecodeParams& p, int hcs, unsigned t1) {
        if (end >= t1) return false;
        seg = at = end;
        if (++hc == hcs) {
            hc = 0;
            do {
                if (++b >= p.batch) return false;
                load(p);
            } while (rg.tiles == 0);
        }
        bound(t1);
        return true;
    }
};

// The infinities among the values of slots s0 .. s1 - 1 of a request row, 16-bit caches: two bits for each of the D / 32
// dims from lane D / 32 on, 1 for +inf and 2 for -inf (both: a NaN too).  The whole warp calls.  A piece's V rows are read
// once more, eight at a time: 1270 us and not 330 for 32 x 2048..32768 rows where every piece holds an infinity.
template <class S>
__device__ __noinline__ uint32_t infinite_values(const DecodeParams& p, int row, int h, int s0, int s1) {
    constexpr int V = S::D / 32;
    constexpr uint32_t kInf = S::BF16 ? 0x7f80u : 0x7c00u;
    const int* table = p.c.table + (long long)row * p.c.table_stride;
    const uint8_t* base = p.c.v + h * p.c.head_stride + (threadIdx.x & 31) * (V * 2);
    constexpr int kAtOnce = 8;                     // rows whose loads go out together (the last one again behind the end)
    uint32_t found = 0;
    for (int s = s0; s < s1; s += kAtOnce) {
        uint32_t x[kAtOnce][V / 2];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int t = min(s + k, s1 - 1), page = __ldg(table + (t >> p.c.page_shift));
            const bool ok = page >= 0 && page < p.c.num_pages;
            const uint32_t* from = reinterpret_cast<const uint32_t*>(
                base + (ok ? page * p.c.page_stride + (t & ((1 << p.c.page_shift) - 1)) * p.c.row_stride : 0));
#pragma unroll
            for (int i = 0; i < V / 2; ++i) x[k][i] = ok ? __ldg(from + i) : 0u;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t y = x[k][i / 2] >> (16 * (i & 1)), size = y & 0x7fffu;
                if (size >= kInf) found |= (size > kInf ? 3u : y & 0x8000u ? 2u : 1u) << (2 * i);
            }
    }
    return found;
}

// SEG: a cluster per segment; else a share of the list per warp.
template <class S, bool SEG>
__global__ void __launch_bounds__(S::W * 32, S::CTAS) dsv4_gqa_decode_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int D = S::D, NT = S::NT, W = S::W, TT = S::TT, MT = S::MT, DT = S::DT, HEADS = S::HEADS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_ok[W][S::STAGES];            // a bit per 16-slot group: its page is in the pool
    // CTAs whose shares this one has taken, in order (-1: there are no more), how many entries are there, and which
    // each warp computes; one request is on its way at a time, its sender holds the lock
    __shared__ int s_cta[kClaimRing], s_known, s_done[W], s_lock, s_phase;
    __shared__ __align__(16) uint8_t s_answer[16];
    __shared__ __align__(8) uint64_t s_bar;
    __shared__ float2 s_ml[SEG ? W : 1][SEG ? HEADS : 1];     // references and sums of the warps
    __shared__ __align__(16) float s_lse[SEG ? HEADS : 4];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    const int hcs = p.c.kv_heads * p.chunks;
    const uint32_t bar = smem_u32(&s_bar);
    if (!SEG && tid == 0) {
        s_cta[0] = blockIdx.x;
        s_known = 1;
        s_lock = s_phase = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) s_done[w] = 0;
        mbar_init(bar, 1);
        fence_mbar_init_cluster();
    }
    if constexpr (!SEG) __syncthreads();
    grid_dependency_wait();
    grid_dependents_go();

    unsigned err = 0;
    auto request_of = [&](int b) {
        Request r{0, 0};
        return b < p.batch ? read_request(p.lens, p.req, p.c.table_rows, p.max_len, b, err) : r;
    };
    Request early{0, 0};                          // one request per lane: the first 32 stay in registers
    Shares shares{};
    Cursor<TT> cons;
    unsigned c1 = 0;                              // end of cons's share
    if constexpr (SEG) {
        const int seg = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
        cons.b = seg / hcs;
        cons.hc = seg % hcs;
        cons.rq = read_request(p.lens, p.req, p.c.table_rows, p.max_len, cons.b, err);
        if (err && cons.hc == 0 && rank == 0 && tid == 0) atomicOr(p.err, err);
        cons.rg = key_range<TT>(p, cons.rq.n);
        cons.seg = seg * ((p.max_len + TT - 1) / TT);          // (numbers the tiles' scores)
        const int i = warp * p.cluster + rank, n = W * p.cluster;        // this warp's part
        cons.at = cons.seg + cons.rg.tiles * i / n;
        c1 = cons.end = cons.seg + cons.rg.tiles * (i + 1) / n;
    } else {
        early = request_of(lane);
        unsigned total = key_range<TT>(p, early.n).tiles;
        for (int b = lane + 32; b < p.batch; b += 32) total += key_range<TT>(p, request_of(b).n).tiles;
        total = __reduce_add_sync(0xffffffffu, total) * hcs;
        if (err && blockIdx.x == 0 && warp == 0) atomicOr(p.err, err);
        if (total == 0) return;
        shares = make_shares(p, total);
    }
    const unsigned tail = SEG ? 0u : shares.tail;
    // warps of one resident CTA take shares far apart, so that few shares spread over all SMs
    const int ctas = p.warps / W;
    auto share_id = [&](int cta) {
        if (cta < ctas) return (warp * ctas + cta) * (tail ? 2 : 1);
        const int j = (cta - ctas) * W + warp;
        return tail ? 2 * j + 1 : shares.count;       // (short list: nothing)
    };
    const int first = SEG ? 0 : share_id(blockIdx.x);
    if (!SEG && first >= shares.count) {
        if (lane == 0) *(volatile int*)&s_done[warp] = 0x3fffffff;
        return;
    }

    // Entry k of s_cta for this warp, -2 while it is not known.  The first warp to ask for it sends the request; no
    // call waits.  (The whole warp calls.)
    bool sent = false;                            // by this warp's lane 0, answer outstanding
    auto taken = [&](int k) {
        int got = -2;
        if (lane == 0) {
            volatile int *known = &s_known, *phase = &s_phase, *done = s_done;
            if (!sent && *known <= k && atomicCAS(&s_lock, 0, 1) == 0) {
                __threadfence_block();
                bool room = *known == k;          // (not answered meanwhile, and no warp a ring behind)
#pragma unroll
                for (int w = 0; w < W; ++w) room &= done[w] + kClaimRing > k;
                if (room) {
                    fence_proxy_async();
                    mbar_arrive_expect_tx(bar, 16);
                    claim_submit(smem_u32(s_answer), bar);
                    sent = true;
                } else {
                    atomicExch(&s_lock, 0);
                }
            }
            if (sent && mbar_test(bar, *phase)) {
                *(volatile int*)&s_cta[k % kClaimRing] = claim_result(smem_u32(s_answer));
                *phase ^= 1;
                __threadfence_block();
                *known = k + 1;
                __threadfence_block();
                atomicExch(&s_lock, 0);
                sent = false;
            }
            if (*known > k) {
                __threadfence_block();
                got = *(volatile int*)&s_cta[k % kClaimRing];
            }
        }
        return __shfl_sync(0xffffffffu, got, 0);
    };

    if constexpr (!SEG) {
        c1 = share_begin(shares, first + 1);
        cons.at = share_begin(shares, first);
        cons.locate(p, hcs, lane, early, request_of);
        cons.bound(c1);
    }

    // ---- the copying side ----
    const uint32_t ring = smem_u32(smem) + warp * S::WARP_RING;
    const int lane_row = lane / S::PPR, lane_piece = lane % S::PPR;
    const long long lane_off = lane_row * p.c.row_stride + lane_piece * 16;
    const int page_mask = (1 << p.c.page_shift) - 1;
    const uint64_t policy = read_policy(p.chunks == 1);
    // the K scale of cons's KV head, loaded as soon as cons comes to it: ahead of the copies
    auto load_kscale = [&]() { return S::CODES && p.c.k_scale ? __ldg(p.c.k_scale + cons.hc / p.chunks) : 1.f; };
    float kscale = load_kscale();
    Cursor<TT> prod = cons;
    unsigned p1 = c1;
    int entry_p = 0, next_p = -2;                  // prod's entry of s_cta; the one behind it, once it is known
    bool asking = false;
    bool more = !SEG || cons.at < cons.end;
    int page = -1;                                 // lane m < MT: page of 16-slot group m of the next tile
    bool wanted = false;                           // that group holds slots to attend
    const uint32_t qbuf = smem_u32(smem) + S::RING_BYTES + warp * S::Q_BYTES;
    int pslot = 0;                                 // first slot of prod's tile
    long long phead = 0;                           // byte offset of its KV head, and of this lane's first piece
    // block scales: lanes 0 .. 15 copy those of 16 rows of K, the others of V
    const uint8_t* bhead = nullptr;
    auto come_to = [&]() {
        pslot = (prod.rg.lo / TT + static_cast<int>(prod.at - prod.seg)) * TT;
        phead = (prod.hc / p.chunks) * p.c.head_stride + lane_off;
        if constexpr (S::FP4)
            bhead = (lane < 16 ? p.c.kb : p.c.vb) + (prod.hc / p.chunks) * p.c.b_head_stride + (lane & 15) * p.c.b_row_stride;
    };
    come_to();
    int pieces = 0, piece = 0;                     // pieces (a share's part of a segment) that prod has come to; cons's
    int q_piece = -1;                              // piece whose queries the buffer holds or is getting
    bool q_free = S::Q_BYTES > 0, fresh = true;              // they have been read; prod has just come to its piece

    // prod to the tile that is copied next; its page ids are loaded one tile ahead of their use
    auto settle = [&]() {
        if (tail && more) {
            // the next share is asked for a little before this one ends
            asking |= prod.at + p.claim_ahead >= p1;
            if (asking && next_p == -2) next_p = taken(entry_p + 1);
        }
        if (more && prod.at >= prod.end) {
            fresh = true;
            ++pieces;
            if (SEG) {
                more = false;
            } else if (!prod.next_segment(p, hcs, p1)) {
                for (int tries = 0; tail && next_p == -2; ++tries) {
                    if (tries >= p.claim_polls) {
                        // given up: nobody may compute this warp's part of what the CTA takes over.  But an answer on its
                        // way to this warp has to land before the CTA may end
                        if (tries == p.claim_polls && lane == 0) atomicOr(p.err, DSV4_DEV_ERR_TIMEOUT);
                        if (tries - p.claim_polls >= kWaitLimit || !__shfl_sync(0xffffffffu, sent, 0)) {
                            next_p = -1;
                            break;
                        }
                    }
                    next_p = taken(entry_p + 1);
                }
                more = next_p >= 0;
                if (more) {
                    ++entry_p;
                    const int id = share_id(next_p);
                    next_p = -2;
                    asking = false;
                    p1 = share_begin(shares, id + 1);
                    prod.at = share_begin(shares, id);
                    prod.locate(p, hcs, lane, early, request_of);
                    prod.bound(p1);
                }
            }
            come_to();
        }
        page = -1;
        wanted = false;
        if (more && lane < MT) {
            const int slot = pslot + lane * 16;
            wanted = slot < prod.rg.n && slot + 16 > prod.rg.lo;
            if (wanted) page = __ldg(p.c.table + (long long)prod.rq.row * p.c.table_stride + (slot >> p.c.page_shift));
        }
    };
    auto issue = [&](int stage) {
        if (more && fresh && q_free) {
            // the piece's queries, with its first tile
            const int chunk = prod.hc % p.chunks, head0 = prod.hc / p.chunks * p.group + chunk * HEADS;
            const int nheads = min(HEADS, p.group - chunk * HEADS);
            const uint8_t* from = static_cast<const uint8_t*>(p.q) + (prod.b * p.q_stride + (long long)head0 * D) * 2;
            for (int i = lane; i < HEADS * D / 8; i += 32) {
                const int c = i / (D / 8), piece = i % (D / 8);
                const bool have = c < nheads;
                cp_async_16(qbuf + c * S::QROW + piece * 16, from + (have ? i * 16 : 0), have ? 16u : 0u);
            }
            q_piece = pieces;
            q_free = false;
        }
        fresh = false;
        if (more) {
            const bool ok = page >= 0 && page < p.c.num_pages;
            if (wanted && !ok) atomicOr(p.err, DSV4_DEV_ERR_GQA_PAGE);
            const unsigned okm = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) s_ok[warp][stage] = okm;
            const uint32_t kd = ring + stage * S::STAGE_BYTES, vd = kd + S::TILE_BYTES;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int pg = __shfl_sync(0xffffffffu, page, m);
                const bool have = (okm >> m) & 1;
                const int s = pslot + m * 16;
                if constexpr (S::FP4) {
                    const int r = s + (lane & 15);
                    const bool in = have && r < prod.rg.n && r >= prod.rg.lo;
                    const uint32_t bd = vd + S::TILE_BYTES + (lane >> 4) * S::BLOCK_BYTES + (m * 16 + (lane & 15)) * S::BLKB;
                    cp_async_hint<S::BLKB>(
                        bd, in ? bhead + pg * p.c.b_page_stride + (s & page_mask) * p.c.b_row_stride : p.c.kb,
                        in ? S::BLKB : 0u, policy);
                }
                const long long base = have ? pg * p.c.page_stride + (s & page_mask) * p.c.row_stride + phead : 0;
                const uint8_t *ks = p.c.k + base, *vs = p.c.v + base;
                if (have && s >= prod.rg.lo && s + 16 <= prod.rg.n) {
#pragma unroll
                    for (int i = 0; i < 16 / S::RPI; ++i) {
                        const int r = m * 16 + i * S::RPI + lane_row;
                        cp_async_16_whole(kd + k_offset<S>(r, lane_piece), ks, policy);
                        cp_async_16_whole(vd + v_offset<S>(r, lane_piece), vs, policy);
                        ks += S::RPI * p.c.row_stride;
                        vs += S::RPI * p.c.row_stride;
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < 16 / S::RPI; ++i) {
                        const int r = i * S::RPI + lane_row;        // row in the group
                        const bool in = have && s + r < prod.rg.n && s + r >= prod.rg.lo;
                        const long long off = in ? i * S::RPI * p.c.row_stride : 0;
                        cp_async_16_hint(kd + k_offset<S>(m * 16 + r, lane_piece), in ? ks + off : p.c.k, in ? 16u : 0u, policy);
                        cp_async_16_hint(vd + v_offset<S>(m * 16 + r, lane_piece), in ? vs + off : p.c.v, in ? 16u : 0u, policy);
                    }
                }
            }
            pslot += TT;
            ++prod.at;
            settle();
        }
        cp_async_commit();
    };

    settle();
#pragma unroll
    for (int s = 0; s < S::STAGES; ++s) issue(s);

    // ---- the computing side ----
    int stage = 0;
    int share = first, entry_c = 0;                // cons's share and entry of s_cta
    for (bool on = true; on;) {
        const bool begins = cons.at == cons.seg;
        const int h = cons.hc / p.chunks, chunk = cons.hc % p.chunks;
        const int head0 = h * p.group + chunk * HEADS;
        const int nheads = min(HEADS, p.group - chunk * HEADS);
        // q as the B operand; head g of n-tile nt.  From the buffer, if the copying side found it free when it came
        // to this piece (very short pieces: from global memory).
        cp_async_wait_group<S::STAGES - 1>();
        __syncwarp();
        const bool in_buffer = q_piece == piece;
        const uint8_t* qbase = in_buffer ? smem + S::RING_BYTES + warp * S::Q_BYTES
                                         : static_cast<const uint8_t*>(p.q) +
                                               (cons.b * p.q_stride + (long long)head0 * D) * 2;
        const int qrow = in_buffer ? S::QROW : D * 2;
        uint32_t qf[S::QSMEM ? 1 : DT][NT][2];
        const uint32_t q_operands = smem_u32(smem) + S::RING_BYTES + W * S::Q_BYTES + warp * S::OPERAND_BYTES + lane * 16;
        float smul[NT][2];                         // score factor of the two heads whose columns this thread holds
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const bool have = nt * 8 + g < nheads;
            const uint32_t* qr = reinterpret_cast<const uint32_t*>(qbase + (nt * 8 + g) * qrow);
            if constexpr (!S::CODES) {
#pragma unroll
                for (int kk = 0; kk < DT; ++kk) {
                    qf[kk][nt][0] = have ? qr[kk * 8 + t4] : 0u;
                    qf[kk][nt][1] = have ? qr[kk * 8 + t4 + 4] : 0u;
                }
                smul[nt][0] = smul[nt][1] = p.scale_log2;
            } else {
                // MMA kk = 4 j + i takes dims 16 (t + 4 j) + 4 i .. + 3 from the thread with that t (e2m1 rows of 128
                // and 256: kk = 8 j + i dims 32 (t + 4 j) + 4 i .. + 3)
                constexpr int PER = S::FP4 && D > 64 ? 8 : 4;
                float amax = 0.f;
                auto word = [&](int kk, int u) {
                    const int d2 = (4 * PER * (t4 + 4 * (kk / PER)) + 4 * (kk % PER)) / 2;
                    return have ? qr[d2 + u] : 0u;
                };
#pragma unroll
                for (int kk = 0; kk < DT; ++kk)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t w = word(kk, u);
                        if constexpr (!S::QSMEM) qf[kk][nt][u] = w;
                        const float2 f = unpack2<S::QBF16>(w);
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^e with amax 2^e in [2^14, 2^15); exponents kept where 2^-e and 2^e are normal
                int e = 14 - (static_cast<int>((__float_as_uint(amax) >> 23) & 255u) - 127);
                e = amax == 0.f || !(amax < INFINITY) ? 0 : (e > 120 ? 120 : (e < -120 ? -120 : e));
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int kk = 0; kk < DT; ++kk) {
                    uint32_t w[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t raw;
                        if constexpr (S::QSMEM) raw = word(kk, u);
                        else raw = qf[kk][nt][u];
                        const float2 f = unpack2<S::QBF16>(raw);
                        w[u] = pack2<false>(f.x * up, f.y * up);
                        if constexpr (!S::QSMEM) qf[kk][nt][u] = w[u];
                    }
                    // (read by the lane that writes it)
                    if constexpr (S::QSMEM)
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_operands + kk * 512 + nt * 8), "r"(w[0]), "r"(w[1])
                                     : "memory");
                }
                const float mul = p.scale_log2 * kscale * down;
                smul[nt][0] = __shfl_sync(0xffffffffu, mul, 8 * t4);
                smul[nt][1] = __shfl_sync(0xffffffffu, mul, 8 * t4 + 4);
            }
        }
        if (in_buffer) {
            __syncwarp();
            q_free = true;
        }
        ++piece;
        float o[DT][NT][4], mref[NT][2], lsum[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mref[nt][0] = mref[nt][1] = kNoMax;
            lsum[nt][0] = lsum[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < DT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[j][nt][c] = 0.f;
        }

        for (unsigned tile = cons.at; tile < cons.end; ++tile) {
            cp_async_wait_group<S::STAGES - 1>();
            __syncwarp();
            const uint32_t ks = ring + stage * S::STAGE_BYTES, vs = ks + S::TILE_BYTES;
            const unsigned okm = s_ok[warp][stage];
            const int slot0 = (cons.rg.lo / TT + static_cast<int>(tile - cons.seg)) * TT;

            // S^T = K Q^T (a lone accumulator as two chains of MMAs)
            constexpr int kChains = MT * NT == 1 ? 2 : 1;
            float s2[1][1][4] = {};
            float s[MT][NT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[m][nt][c] = 0.f;
            if constexpr (!S::CODES) {
                const int mrow = lane & 15, mpiece = lane >> 4;
#pragma unroll
                for (int kk = 0; kk < DT; ++kk)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        uint32_t a[4];
                        ldsm4(a, ks + k_offset<S>(m * 16 + mrow, 2 * kk + mpiece));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<S::BF16>(kChains > 1 && kk & 1 ? s2[0][0] : s[m][nt], a, qf[kk][nt][0], qf[kk][nt][1]);
                    }
                if constexpr (kChains > 1)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[0][0][c] += s2[0][0][c];
            } else if constexpr (S::FP4) {
                // A thread's 16 bytes of rows g and g + 8 are two blocks (64 dims: 8 bytes, one).  Code times block scale
                // is exact in f16: 2 + 4 significant bits, 2^-10 .. 2688
                constexpr int WORDS = D == 64 ? 2 : 4;
                const uint32_t kb = vs + S::TILE_BYTES;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < (D == 256 ? 2 : 1); ++j) {
                        uint32_t w[2][WORDS], sc[2][2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int row = m * 16 + g + 8 * u;
                            if constexpr (D == 64) {
                                const uint2 x = ld_shared_u2(ks + row * S::ROWB + t4 * 8);
                                w[u][0] = x.x; w[u][1] = x.y;
                                const uint32_t b = e4m3x2_f16x2(ld_shared_u8(kb + row * S::BLKB + t4));
                                sc[u][0] = sc[u][1] = __byte_perm(b, b, 0x1010);
                            } else {
                                const uint4 x = ld_shared_u4(ks + k_offset<S>(row, t4 + 4 * j));
                                w[u][0] = x.x; w[u][1] = x.y; w[u][2] = x.z; w[u][3] = x.w;
                                const uint32_t b = e4m3x2_f16x2(ld_shared_u16(kb + row * S::BLKB + 8 * j + 2 * t4));
                                sc[u][0] = __byte_perm(b, b, 0x1010);
                                sc[u][1] = __byte_perm(b, b, 0x3232);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < WORDS; ++i) {
                            uint32_t x[4], y[4];
                            e2m1x8_f16x2(w[0][i], x);
                            e2m1x8_f16x2(w[1][i], y);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                x[k] = mul_f16x2(x[k], sc[0][i >> 1]);
                                y[k] = mul_f16x2(y[k], sc[1][i >> 1]);
                            }
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t a[4] = {x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1]};
                                const int kk = 8 * j + 2 * i + k;
                                if constexpr (S::QSMEM) {
                                    const uint4 q = ld_shared_u4(q_operands + kk * 512);
                                    mma16816<false>(s[m][0], a, q.x, q.y);
                                    mma16816<false>(s[m][1], a, q.z, q.w);
                                } else {
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        mma16816<false>(kChains > 1 && k ? s2[0][0] : s[m][nt], a, qf[kk][nt][0], qf[kk][nt][1]);
                                }
                            }
                        }
                    }
                if constexpr (kChains > 1)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[0][0][c] += s2[0][0][c];
            } else {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        const uint4 x = ld_shared_u4(ks + k_offset<S>(m * 16 + g, t4 + 4 * j));
                        const uint4 y = ld_shared_u4(ks + k_offset<S>(m * 16 + g + 8, t4 + 4 * j));
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a[4] = {e4m3x2_f16x2(xs[i]), e4m3x2_f16x2(ys[i]), e4m3x2_hi_f16x2(xs[i]),
                                                   e4m3x2_hi_f16x2(ys[i])};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(s[m][nt], a, qf[4 * j + i][nt][0], qf[4 * j + i][nt][1]);
                        }
                    }
            }

            // log2-unit scores, masked; the vote on the reference
            const bool whole = slot0 >= cons.rg.lo && slot0 + TT <= cons.rg.n && okm == (1u << MT) - 1u;
            bool above = false;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float x = s[m][nt][c] * smul[nt][c & 1];
                        if (!whole) {
                            const int slot = slot0 + m * 16 + g + (c >> 1) * 8;
                            if (slot < cons.rg.lo || slot >= cons.rg.n || !((okm >> m) & 1)) x = -INFINITY;
                        }
                        s[m][nt][c] = x;
                        above |= x > __fadd_rd(mref[nt][c & 1], S::DROP + S::SLACK);
                    }
            if (p.logits) {
                float* to = p.logits + (size_t)tile * TT * HEADS;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            *reinterpret_cast<float2*>(to + (m * 16 + g + 8 * u) * HEADS + nt * 8 + 2 * t4) =
                                make_float2(s[m][nt][2 * u], s[m][nt][2 * u + 1]);
            }
            if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int m = 0; m < MT; ++m) mx = fmaxf(mx, fmaxf(s[m][nt][u], s[m][nt][u + 2]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        mx = fmaxf(mref[nt][u], __fsub_ru(mx, S::DROP));
                        const float f = fast_exp2(mref[nt][u] - mx);
                        mref[nt][u] = mx;
                        lsum[nt][u] *= f;
#pragma unroll
                        for (int j = 0; j < DT; ++j) {
                            o[j][nt][u] *= f;
                            o[j][nt][u + 2] *= f;
                        }
                    }
            }

            // P^T and O^T += V^T P^T
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float x = fast_exp2(s[m][nt][2 * u] - mref[nt][0]);
                        const float y = fast_exp2(s[m][nt][2 * u + 1] - mref[nt][1]);
                        lsum[nt][0] += x;
                        lsum[nt][1] += y;
                        const uint32_t w = pack2<S::BF16>(x, y);
                        hi[nt][u] = transpose8x8(w);
                        if constexpr (S::TWO) {
                            const float2 r = unpack2<S::BF16>(w);
                            lo[nt][u] = transpose8x8(pack2<S::BF16>(x - r.x, y - r.y));
                        }
                    }
                if constexpr (!S::CODES) {
                    const int mrow = (lane & 7) + ((lane >> 4) << 3), mpiece = (lane >> 3) & 1;
#pragma unroll
                    for (int j = 0; j < DT; ++j) {
                        uint32_t a[4];
                        ldsm4_trans(a, vs + v_offset<S>(m * 16 + mrow, 2 * j + mpiece));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<S::BF16>(o[j][nt], a, hi[nt][0], hi[nt][1]);
                            mma16816<S::BF16>(o[j][nt], a, lo[nt][0], lo[nt][1]);
                        }
                    }
                } else if constexpr (S::FP4) {
                    // slots 2t, 2t + 1, 2t + 8, 2t + 9; the codes of a pair of slots become bytes of one dim each, whose
                    // two halves convert to an A operand.  Dims as for e4m3 rows; a thread's 16 dims are one block (8 of
                    // 64 dims: half of one)
                    constexpr int WORDS = D == 64 ? 1 : 2;       // 32-bit words per thread, slot and half
                    const uint32_t vb = vs + S::TILE_BYTES + S::BLOCK_BYTES;
#pragma unroll
                    for (int hh = 0; hh < (D == 256 ? 2 : 1); ++hh) {
                        uint32_t v[4][WORDS], b[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int row = m * 16 + 2 * t4 + (u & 1) + (u >> 1) * 8;
                            if constexpr (D == 64) {
                                v[u][0] = ld_shared_u32(vs + v_offset<S>(row, g >> 2) + (g & 3) * 4);
                                b[u] = ld_shared_u8(vb + row * S::BLKB + (g >> 1));
                            } else {
                                const uint2 x = ld_shared_u2(vs + v_offset<S>(row, (g >> 1) + 4 * hh) + (g & 1) * 8);
                                v[u][0] = x.x; v[u][1] = x.y;
                                b[u] = ld_shared_u8(vb + row * S::BLKB + g + 8 * hh);
                            }
                        }
                        const uint32_t s01 = e4m3x2_f16x2(b[0] | b[1] << 8), s23 = e4m3x2_f16x2(b[2] | b[3] << 8);
#pragma unroll
                        for (int w = 0; w < WORDS; ++w) {
                            uint32_t a[4][4];
                            e2m1x8_f16x2(pick_bits(v[0][w], v[1][w] << 4, 0x0f0f0f0fu), a[0]);
                            e2m1x8_f16x2(pick_bits(v[0][w] >> 4, v[1][w], 0x0f0f0f0fu), a[1]);
                            e2m1x8_f16x2(pick_bits(v[2][w], v[3][w] << 4, 0x0f0f0f0fu), a[2]);
                            e2m1x8_f16x2(pick_bits(v[2][w] >> 4, v[3][w], 0x0f0f0f0fu), a[3]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t x[4] = {mul_f16x2(a[0][i], s01), mul_f16x2(a[1][i], s01),
                                                       mul_f16x2(a[2][i], s23), mul_f16x2(a[3][i], s23)};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma16816<false>(o[hh * 8 + w * 4 + i][nt], x, hi[nt][0], hi[nt][1]);
                                    if constexpr (S::TWO) mma16816<false>(o[hh * 8 + w * 4 + i][nt], x, lo[nt][0], lo[nt][1]);
                                }
                            }
                        }
                    }
                } else {
                    // slots 2t, 2t + 1, 2t + 8, 2t + 9; tile j's rows g and g + 8 are the two
                    // neighbouring dims dim_of(j, g): words of four dims, slot pairs byte-interleaved
                    constexpr int WORDS = D == 64 ? 2 : 4;       // 32-bit words per thread, slot and half
#pragma unroll
                    for (int hh = 0; hh < (D == 256 ? 2 : 1); ++hh) {
                        uint32_t v[4][WORDS];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int row = m * 16 + 2 * t4 + (u & 1) + (u >> 1) * 8;
                            if constexpr (D == 64) {
                                const uint32_t at = vs + v_offset<S>(row, g >> 1) + (g & 1) * 8;
                                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                             : "=r"(v[u][0]), "=r"(v[u][1])
                                             : "r"(at)
                                             : "memory");
                            } else {
                                const uint4 x = ld_shared_u4(vs + v_offset<S>(row, g + 8 * hh));
                                v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
                            }
                        }
#pragma unroll
                        for (int jj = 0; jj < 2 * WORDS; ++jj) {
                            const uint32_t sel = jj & 1 ? 0x7362u : 0x5140u;
                            const uint32_t x = __byte_perm(v[0][jj >> 1], v[1][jj >> 1], sel);
                            const uint32_t y = __byte_perm(v[2][jj >> 1], v[3][jj >> 1], sel);
                            const uint32_t a[4] = {e4m3x2_f16x2(x), e4m3x2_hi_f16x2(x), e4m3x2_f16x2(y),
                                                   e4m3x2_hi_f16x2(y)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<false>(o[hh * 8 + jj][nt], a, hi[nt][0], hi[nt][1]);
                                if constexpr (S::TWO) mma16816<false>(o[hh * 8 + jj][nt], a, lo[nt][0], lo[nt][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            issue(stage);
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
        }

        // ---- the piece's sums, and its output ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                lsum[nt][u] += __shfl_xor_sync(0xffffffffu, lsum[nt][u], 4);
                lsum[nt][u] += __shfl_xor_sync(0xffffffffu, lsum[nt][u], 8);
                lsum[nt][u] += __shfl_xor_sync(0xffffffffu, lsum[nt][u], 16);
            }
        if constexpr (!S::CODES) {
            // P's two parts times an infinite value can be inf - inf or 0 inf, which is NaN where the sum is infinite:
            // where a NaN comes of finite scores, the infinities are looked up
            bool odd = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    bool any = false;
#pragma unroll
                    for (int j = 0; j < DT; ++j) any |= isnan(o[j][nt][u]) || isnan(o[j][nt][u + 2]);
                    odd |= any && !isnan(lsum[nt][u]);
                }
            if (__any_sync(0xffffffffu, odd)) {
                const int t0 = cons.rg.lo / TT - static_cast<int>(cons.seg);
                const uint32_t found = infinite_values<S>(p, cons.rq.row, h,
                                                          max(cons.rg.lo, (t0 + static_cast<int>(cons.at)) * TT),
                                                          min(cons.rg.n, (t0 + static_cast<int>(cons.end)) * TT));
#pragma unroll
                for (int j = 0; j < DT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        const int d = 16 * j + 4 * c + g;
                        const uint32_t f = __shfl_sync(0xffffffffu, found, d / (D / 32)) >> (2 * (d % (D / 32))) & 3u;
                        if (f == 1u || f == 2u)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    if (isnan(o[j][nt][c + u]) && !isnan(lsum[nt][u]))
                                        o[j][nt][c + u] = f == 1u ? INFINITY : -INFINITY;
                    }
            }
        }
        // the next piece, if there is one
        const bool cut = !begins || cons.end != cons.seg + cons.rg.tiles;
        const int here_b = cons.b, here = share;
        if constexpr (SEG) {
            // the warps' rings become their outputs, [HEADS][D] fp32 (padded rows), and the cluster adds them up
            constexpr int kRow = D + 4;
            static_assert(HEADS * kRow * 4 <= S::WARP_RING, "a warp's output fits its ring");
            cp_async_wait_group<0>();
            __syncwarp();
            float* mine = reinterpret_cast<float*>(smem + warp * S::WARP_RING);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = nt * 8 + 2 * t4 + u;
                    if (g == 0) s_ml[warp][c] = make_float2(mref[nt][u], lsum[nt][u]);
#pragma unroll
                    for (int j = 0; j < DT; ++j) {
                        if constexpr (!S::CODES) {
                            mine[c * kRow + 16 * j + g] = o[j][nt][u];
                            mine[c * kRow + 16 * j + 8 + g] = o[j][nt][u + 2];
                        } else {
                            const int d = D == 64 ? 8 * g + 2 * j : 16 * (g + 8 * (j >> 3)) + 2 * (j & 7);
                            *reinterpret_cast<float2*>(mine + c * kRow + d) = make_float2(o[j][nt][u], o[j][nt][u + 2]);
                        }
                    }
                }
            cluster_sync();
            const int rank = blockIdx.x % p.cluster;
            const float vmul = S::CODES && p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f;
            const uint32_t ml0 = smem_u32(&s_ml[0][0]), o0 = smem_u32(smem);
            for (int e = rank * W * 32 + tid; e < nheads * D / 2; e += p.cluster * W * 32) {
                const int c = e / (D / 2), d = e % (D / 2) * 2;
                // one CTA's warps after another; the reference moves between CTAs
                float mx = kNoMax, l = 0.f, x = 0.f, y = 0.f;
                for (int r = 0; r < p.cluster; ++r) {
                    float2 ml[W], v[W];
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        ml[w] = ld_cluster_f2(mapa(ml0 + (w * HEADS + c) * 8, r));
                        v[w] = ld_cluster_f2(mapa(o0 + w * S::WARP_RING + (c * kRow + d) * 4, r));
                    }
                    float top = mx;
#pragma unroll
                    for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w].x);
                    const float f = fast_exp2(mx - top);
                    mx = top;
                    l *= f;
                    x *= f;
                    y *= f;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float k = fast_exp2(ml[w].x - top);
                        l += k * ml[w].y;
                        x += k * v[w].x;
                        y += k * v[w].y;
                    }
                }
                const float sk = p.sink ? __ldg(p.sink + head0 + c) * kLog2e : -INFINITY;
                const float top = fminf(fmaxf(mx, sk), 3e38f);
                const float f = fast_exp2(mx - top);
                l = l * f + fast_exp2(sk - top);
                const bool any = l > 0.f || l != l;
                const float inv = any ? vmul * f / l : 0.f;
                const size_t at = (size_t)here_b * p.heads + head0 + c;
                *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at * D + d) =
                    pack2<S::QBF16>(x * inv, y * inv);
                if (d == 0 && p.lse) p.lse[at] = any ? (top + log2f(l)) * kLn2 : -INFINITY;
            }
            if (p.w_out) {
                // lse of every head, by a warp each; then the weights of this warp's own tiles, whose scores it wrote
                for (int c = warp; c < HEADS; c += W) {
                    const bool in = lane < W * p.cluster && c < nheads;
                    const float2 ml = in ? ld_cluster_f2(mapa(ml0 + (lane % W * HEADS + c) * 8, lane / W))
                                         : make_float2(kNoMax, 0.f);
                    float mx = ml.x;
#pragma unroll
                    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                    const float sk = p.sink && c < nheads ? __ldg(p.sink + head0 + c) * kLog2e : -INFINITY;
                    const float top = fminf(fmaxf(mx, sk), 3e38f);
                    float l = ml.y * fast_exp2(ml.x - top);
#pragma unroll
                    for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
                    l += fast_exp2(sk - top);
                    // +inf makes a head contribute nothing: padding, and heads none of whose rows could be read
                    if (lane == 0) s_lse[c] = c < nheads && (l > 0.f || l != l) ? top + log2f(l) : INFINITY;
                }
                __syncthreads();
                const size_t to = ((size_t)cons.rq.row * p.c.kv_heads + h) * p.width;
                const int t0 = cons.rg.lo / TT - static_cast<int>(cons.seg);
                const int s0 = (t0 + static_cast<int>(cons.at)) * TT, s1 = (t0 + static_cast<int>(cons.end)) * TT;
                const int first_s = max(s0, cons.rg.lo), end_s = min(s1, cons.rg.n);
                constexpr int kAtOnce = HEADS > 8 ? 2 : 4;        // slots per lane whose loads go out together
                for (int s = first_s + lane; s < end_s; s += 32 * kAtOnce) {
                    float prior[kAtOnce];
                    float4 x[kAtOnce][HEADS / 4];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const int at = min(s + 32 * i, end_s - 1);
                        prior[i] = p.w_in[to + at];
                        const float4* from =
                            reinterpret_cast<const float4*>(p.logits + ((size_t)cons.at * TT + (at - s0)) * HEADS);
#pragma unroll
                        for (int k = 0; k < HEADS / 4; ++k) x[i][k] = __ldcg(from + k);
                    }
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        float add = 0.f;
#pragma unroll
                        for (int k = 0; k < HEADS / 4; ++k) {
                            const float4 l = *reinterpret_cast<const float4*>(s_lse + 4 * k);
                            add += (fast_exp2(x[i][k].x - l.x) + fast_exp2(x[i][k].y - l.y)) +
                                   (fast_exp2(x[i][k].z - l.z) + fast_exp2(x[i][k].w - l.w));
                        }
                        if (s + 32 * i < end_s) p.w_out[to + s + 32 * i] = p.decay * prior[i] + add;
                    }
                }
                for (int s = rank * W * 32 + tid; s < cons.rg.lo; s += p.cluster * W * 32)
                    p.w_out[to + s] = p.decay * p.w_in[to + s];
            }
            cluster_sync();                       // (no CTA may end while another reads its shared memory)
            return;
        }
        on = cons.next_segment(p, hcs, c1);
        if (!on && entry_c < entry_p) {
            ++entry_c;
            // (the entry is overwritten only once every warp's s_done is past it, which takes this warp's next time here)
            share = share_id(*(volatile int*)&s_cta[entry_c % kClaimRing]);
            if (lane == 0) *(volatile int*)&s_done[warp] = entry_c;
            c1 = share_begin(shares, share + 1);
            cons.at = share_begin(shares, share);
            cons.locate(p, hcs, lane, early, request_of);
            cons.bound(c1);
            on = true;
        }
        if (on) kscale = load_kscale();
        if (cut) {
            const int entry = piece_entry(here, begins);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = nt * 8 + 2 * t4 + u;
                    if (c >= nheads) continue;
                    float* to = p.part_o + ((size_t)entry * HEADS + c) * D;
                    if constexpr (!S::CODES) {
#pragma unroll
                        for (int j = 0; j < DT; ++j) {
                            to[16 * j + g] = o[j][nt][u];
                            to[16 * j + 8 + g] = o[j][nt][u + 2];
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < DT; j += 2) {
                            const int d = D == 64 ? 8 * g + 2 * j : 16 * (g + 8 * (j >> 3)) + 2 * (j & 7);
                            *reinterpret_cast<float4*>(to + d) =
                                make_float4(o[j][nt][u], o[j][nt][u + 2], o[j + 1][nt][u], o[j + 1][nt][u + 2]);
                        }
                    }
                    if (g == 0) p.part_ml[entry * HEADS + c] = make_float2(mref[nt][u], lsum[nt][u]);
                }
            continue;
        }
        const float vmul = S::CODES && p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f;
        const size_t row = (size_t)here_b * p.heads + head0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float inv[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = nt * 8 + 2 * t4 + u;
                const float sk = p.sink && c < nheads ? __ldg(p.sink + head0 + c) * kLog2e : -INFINITY;
                const float top = fminf(fmaxf(mref[nt][u], sk), 3e38f);     // (a sink of +inf: out = 0)
                const float f = fast_exp2(mref[nt][u] - top);
                const float l = lsum[nt][u] * f + fast_exp2(sk - top);
                const bool any = l > 0.f || l != l;
                inv[u] = any ? vmul * f / l : 0.f;
                if (g == 0 && c < nheads) {
                    const float l2 = any ? top + log2f(l) : -INFINITY;
                    if (p.lse) p.lse[row + c] = l2 * kLn2;
                    if (p.lse2) p.lse2[row + c] = l2;
                }
            }
            uint16_t* out = static_cast<uint16_t*>(p.out);
            if constexpr (!S::CODES) {
                // pairs of heads to pairs of dims: this thread then holds head g, dims 2t and 2t + 1 of an 8-dim block
#pragma unroll
                for (int j = 0; j < DT; ++j)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t w = transpose8x8(
                            pack2<S::BF16>(o[j][nt][2 * u] * inv[0], o[j][nt][2 * u + 1] * inv[1]));
                        if (nt * 8 + g < nheads)
                            *reinterpret_cast<uint32_t*>(out + (row + nt * 8 + g) * D + 16 * j + 8 * u + 2 * t4) = w;
                    }
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = nt * 8 + 2 * t4 + u;
                    if (c >= nheads) continue;
#pragma unroll
                    for (int j = 0; j < DT; j += 4) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x = o[j + i][nt][u] * inv[u], y = o[j + i][nt][u + 2] * inv[u];
                            w[i] = pack2<S::QBF16>(x, y);
                        }
                        const int d = D == 64 ? 8 * g : 16 * (g + 8 * (j >> 3)) + 2 * (j & 7);
                        *reinterpret_cast<uint4*>(out + (row + c) * D + d) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    }
}

// The host side of one cache type (and type of queries, where they differ).
int launch_decode_bf16(const DecodeParams& p, int head_dim, int nt, void* stream);
int launch_decode_f16(const DecodeParams& p, int head_dim, int nt, void* stream);
int launch_decode_e4m3(const DecodeParams& p, int head_dim, int nt, void* stream);
int launch_decode_e4m3_f16(const DecodeParams& p, int head_dim, int nt, void* stream);
int launch_decode_e2m1(const DecodeParams& p, int head_dim, int nt, void* stream);
int launch_decode_e2m1_f16(const DecodeParams& p, int head_dim, int nt, void* stream);

template <class S>
inline int launch_decode_shape(const DecodeParams& p, void* stream) {
    if (p.cluster)
        return launch(dsv4_gqa_decode_kernel<S, true>, dim3(p.batch * p.c.kv_heads * p.chunks * p.cluster), S::W * 32,
                      S::SMEM, stream, p.cluster, p);
    if constexpr (!S::LIST)
        return DSV4_ERR_INVALID;
    else
        return launch(dsv4_gqa_decode_kernel<S, false>, dim3(p.warps / S::W + p.claims), S::W * 32, S::SMEM, stream, 1, p);
}

// shared memory beyond 48 KB is asked for once (which loads the kernel)
template <class S>
inline bool prepare_decode_shape() {
    if constexpr (S::LIST)
        if (cudaFuncSetAttribute(dsv4_gqa_decode_kernel<S, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) !=
                cudaSuccess ||
            !load_kernels(dsv4_gqa_decode_kernel<S, false>))
            return false;
    return cudaFuncSetAttribute(dsv4_gqa_decode_kernel<S, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) ==
               cudaSuccess &&
           load_kernels(dsv4_gqa_decode_kernel<S, true>);
}

template <int KIND, int QKIND, int D>
inline int launch_decode_dim(const DecodeParams& p, int nt, void* stream) {
    static unsigned long long ready = 0;
    const int rc = once_per_device(ready, [] {
        return prepare_decode_shape<Shape<KIND, QKIND, D, 1>>() && prepare_decode_shape<Shape<KIND, QKIND, D, 2>>();
    });
    if (rc) return rc;
    return nt == 1 ? launch_decode_shape<Shape<KIND, QKIND, D, 1>>(p, stream)
                   : launch_decode_shape<Shape<KIND, QKIND, D, 2>>(p, stream);
}

template <int KIND, int QKIND>
inline int launch_decode_kind(const DecodeParams& p, int head_dim, int nt, void* stream) {
    if (head_dim == 64) return launch_decode_dim<KIND, QKIND, 64>(p, nt, stream);
    if (head_dim == 128) return launch_decode_dim<KIND, QKIND, 128>(p, nt, stream);
    return launch_decode_dim<KIND, QKIND, 256>(p, nt, stream);
}

}  // namespace gqa
}  // namespace dsv4
