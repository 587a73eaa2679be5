// Attention of few query rows per sequence (decoded tokens, small draft trees) over the paged cache,
// with a sliding window or behind shared prefixes: bf16 queries, head dim 64 or 128, K/V bf16 or
// e4m3.
//
// A unit is 8 or 16 rows (tokens x query heads) of one sequence and kv head.  It is bound by the
// reading of K and V, not by arithmetic: 4 D operations per row and token against 4 D bytes (bf16) per
// token.  In chunk_tc.cuh the chain S -> softmax -> P V over tensor memory takes 0.8 (bf16) to 1.3 us
// (e4m3) per KV tile and SM however few the rows are.  Here warps of their own run over the tiles, and
// no step waits for another warp's.  A warp holds 8 NR rows of Q and O in registers (NR = 1 or 2), and
// a step is 32 tokens in 16 x 8 x 16 matrix instructions with the rows across: S^T = K Q^T (16 tokens x
// 8 rows) and O^T += V^T P^T (16 head elements x 8 rows), so eight rows waste nothing; with the rows
// along the other side of 16, window decode (below) took 3% longer.  A lane reads 16 bytes of K at
// a time, which permutes the head elements (Q's alike); V^T is transposed on the way from shared memory
// (ldmatrix), P^T by movmatrix.
//
// A CTA is four such warps, two that fill the K and V rings by TMA and one that walks along the CTA's
// range and hands its segments on, ahead of the others (without it window decode took 6% longer); two CTAs to an SM,
// so that one computes while the other joins.  The warps take the steps of the range in turn.  Units,
// pieces and segments are those of chunk_units.cuh, one range per CTA laid out by chunk_plan.cu; at the
// end of a unit (or piece) the warps' states are joined through shared memory, and the pieces of a cut
// unit by the last CTA to finish.
//
// Measured (calls replayed from a graph, 32 / 8 heads of 128): 64 tokens over bf16 windows of up to 4100
// (window decode) 171 us, 6.0 TB/s, 0.88 of the copy rate; 32 tokens of 64 / 8 heads over e4m3 windows of
// up to 2063 45 us, 2.8 TB/s: 8 of it the plan, and then about 900 clocks of S and softmax and 1200 of P V
// for a warp's step, mostly the widening of codes, and 9000 for a unit's end.
//
// e4m3: K's codes are widened to f16 (exact), and Q, scaled by a power of two per row, with them: f16
// holds Q's 8 bits from the row's largest element down to 2^-28 of it, and what is smaller is off by
// 2^-39 of that element.  V's codes are widened to bf16 (exact), as P times V's scale is bf16, whose
// range it needs.
//
// P (over e4m3 times V's scale) is rounded to bf16 for the product with V, by at most 2^-8 of each weight;
// the sum that divides it, O and the running maxima stay in 32 bits.  With both the weights and the result rounded, a
// bf16 result is off by 0.0023 of its norm, by 0.0017 with the result alone; P in two halves would double P V.
//
// A value that a row may not see must not reach it, and P V multiplies it by zero.  V of tokens that no
// row of the unit sees is overwritten with zeros before use; a step that only some rows see whole is
// then looked through for values that are not finite, and where there is one its P V is done token by
// token without the hidden ones.
//
// Every wait is bounded, as in chunk_tc.cuh.
#pragma once

#include <type_traits>

#include "chunk_units.cuh"

namespace treespec {

namespace {

constexpr int kWarps = 4;                // warps that compute
constexpr int kFewThreads = 256;         // and a warpgroup of which two warps produce
constexpr int kStep = 32;                // tokens a warp takes at a time
// registers of the computing warps and of the others: 128 (168 + 88) = 256 x the 128 of the launch
constexpr uint32_t kRegsCompute = 168, kRegsProduce = 88;
constexpr int kWarpProduce = kWarps, kWarpWalk = kWarps + 2;   // the first of two that produce; the one that walks
constexpr int kSegRing = 4;              // segments that the walking warp is ahead, at most
constexpr int kNoPlan = -2;              // in place of a range's begin: the plan did not come

template <int D, bool E4M3, int NR>
struct CfgFew {
    static constexpr int kNP = E4M3 ? 1 : D / 64;         // panels of a stage
    static constexpr int kRowBytes = E4M3 ? D : 128;      // of a token in a panel
    static constexpr int kPanel = kStep * kRowBytes;
    static constexpr int kStage = kNP * kPanel;           // a step of K or V: one warp's
    static constexpr int kPitch = D + 4;                  // floats of a row of a warp's part
    static constexpr int kPartBytes = kWarps * 8 * NR * (kPitch * 4 + 8);
    // Stages of the K ring, and of the V ring: one or two for each warp, as two CTAs to an SM leave room.
    // Stage s is always warp s % 4's: a parity tells a warp that waits for a use of a stage from the use
    // before it only, so no use may be another warp's (its data may land later than that of a step behind it)
    static constexpr int kRoom = (113 * 1024 - 2560 - kPartBytes) / (2 * (kStage + (E4M3 ? kStep * 4 : 0)));
    static constexpr int kNS = kRoom >= 2 * kWarps ? 2 * kWarps : kWarps;
    static constexpr bool kPairs = kNS == 2 * kWarps;     // the tile that a producing warp takes is a quarter of the ring
    struct Bars {
        uint64_t k_full[kNS], k_empty[kNS], v_full[kNS], v_empty[kNS], part_full, part_empty, seg_full[kSegRing],
            seg_empty[kSegRing];
    };
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kNS * kStage;
    static constexpr int kOffScale = kOffV + kNS * kStage;                     // [K, V][kNS][kStep]
    static constexpr int kOffPart = kOffScale + (E4M3 ? 2 * kNS * kStep * 4 : 0);   // [kWarps][8 NR] rows
    static constexpr int kOffMl = kOffPart + kWarps * 8 * NR * kPitch * 4;     // [kWarps][8 NR] (m, l)
    static constexpr int kOffBar = kOffMl + kWarps * 8 * NR * 8;
    static constexpr int kOffMisc = kOffBar + int(sizeof(Bars));
    static constexpr int kOffEnds = (kOffMisc + 16 + 15) / 16 * 16;            // the CTA's plan
    static constexpr int kOffSeg = kOffEnds + int(sizeof(CtaPlan));            // [kSegRing] segments
    static constexpr int kSmemBytes = kOffSeg + kSegRing * 128;
    static_assert(kOffV % 1024 == 0 && kOffScale % 64 == 0 && kOffPart % 16 == 0 && kOffBar % 8 == 0 && kOffSeg % 8 == 0 &&
                      kRoom >= kWarps, "alignment");
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs to an SM");
};

// D[16 x 8] += A[16 x 16] B[16 x 8].  Lane 4 g + q: A rows g and g + 8 (a0, a2 and a1, a3), inner
// elements 2 q, 2 q + 1 (a0, a1; b0) and 8 more (a2, a3; b1); B column g; D rows g (d0, d1), g + 8,
// columns 2 q, 2 q + 1.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four 8 x 8 matrices of 16-bit elements, transposed: lane l gives the address of row l % 8 of matrix
// l / 8 and gets elements (column g; rows 2 q, 2 q + 1) of each.
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// (row g; columns 2 q, 2 q + 1) of an 8 x 8 matrix -> (column g; rows 2 q, 2 q + 1)
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
    uint32_t r;
    asm("{\n\t.reg .f16 lo, hi;\n\t.reg .f32 a, b;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 a, lo;\n\tcvt.f32.f16 b, hi;\n\t"
        "cvt.rn.bf16x2.f32 %0, b, a;\n\t}"
        : "=r"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void copy_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// An arrival once all the thread's copies so far are there.
__device__ __forceinline__ void arrive_behind_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Row r = it * G + g of a unit: its place in the batch.
template <ChunkMode M>
__device__ __forceinline__ Row few_row(const ChunkParams& p, const Seg<M>& s, int r, int D) {
    Row o;
    const int it = (r * p.inv_g) >> 16, g = r - it * p.G;   // r / G: exact for r < 128, G <= 128
    o.ok = it < s.tokens;
    o.i = s.i0 + (o.ok ? it : 0);
    o.hq = s.h * p.G + (o.ok ? g : 0);
    o.at = (size_t(s.row0 + (o.ok ? it : 0)) * p.Hq + o.hq) * D;
    return o;
}

template <int DS>
__device__ __forceinline__ void store_slice(float* dst, const float (&x)[DS]) {
    if constexpr (DS == 4) __stcg(reinterpret_cast<float4*>(dst), make_float4(x[0], x[1], x[2], x[3]));
    else __stcg(reinterpret_cast<float2*>(dst), make_float2(x[0], x[1]));
}

// Row r of a finished unit or part: where its float32 state or its result goes, a lane the elements
// lane * D / 32 on.
template <int D, ChunkMode M>
__device__ __forceinline__ void store_row(const ChunkParams& p, const Row& ro, int side, float m, float l, float (&acc)[D / 32]) {
    constexpr int DS = D / 32;
    const int lane = threadIdx.x & 31;
    if (M == kChunkShared && side >= 0) {
        float* dst = p.rows_acc + side_offset(p, side) * D + ro.at + lane * DS;
        store_slice<DS>(dst, acc);
        if (lane == 0) reinterpret_cast<float2*>(p.rows_ml)[side_offset(p, side) + ro.at / D] = make_float2(m, l);
        return;
    }
    const float f = 1.f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + ro.at) + lane * (DS / 2);
    if constexpr (DS == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f));
    else
        *dst = pack_bf16x2(acc[0] * f, acc[1] * f);
}

// What a state (m, l) weighs beside others of maximum `top`: -1, left out, where it saw no token of a
// weight above 0; 1 where its scores were NaN.
__device__ __forceinline__ float state_weight(float m, float l, float top) {
    return m == -INFINITY ? (l == 0.f ? -1.f : 1.f) : ex2(m - top);
}

// Rows r, r + 4, .. of a cut unit, by one warp: piece k of a row is in slot 2 c0 + 1 (k = 0)
// or 2 (c0 + k).  Four rows are on their way at a time, their (m, l) with a piece per lane.
template <int D, ChunkMode M>
__device__ __noinline__ void join_rows(const ChunkParams& p, const Seg<M>& s, int c0, int pieces, int r, int used) {
    constexpr int DS = D / 32, kR = 4, by = kWarps;
    const int lane = threadIdx.x & 31;
    auto slot = [&](int k) { return size_t(k == 0 ? 2 * c0 + 1 : 2 * (c0 + k)) * 16; };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    for (; r < used; r += kR * by) {
        int row[kR];                                       // behind the last: the last again, not stored
        float top[kR], l[kR], w[kR], acc[kR][DS];
        float2 x[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            row[i] = r + i * by < used ? r + i * by : r;
            top[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < DS; ++e) acc[i][e] = 0.f;
        }
        auto fetch = [&](int k) {
#pragma unroll
            for (int i = 0; i < kR; ++i) x[i] = k < pieces ? __ldcg(ml + slot(k) + row[i]) : make_float2(-INFINITY, 0.f);
        };
        for (int k0 = 0; k0 < pieces; k0 += 32) {
            fetch(k0 + lane);
#pragma unroll
            for (int i = 0; i < kR; ++i) top[i] = fmaxf(top[i], warp_max(x[i].x));
        }
        for (int k0 = 0; k0 < pieces; k0 += 32) {
            if (pieces > 32) fetch(k0 + lane);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                w[i] = state_weight(x[i].x, x[i].y, top[i]);
                l[i] += warp_sum(w[i] < 0.f ? 0.f : x[i].y * w[i]);
            }
            const int kn = min(32, pieces - k0);
#pragma unroll 4
            for (int k = 0; k < kn; ++k) {
                const float* src = p.part_acc + slot(k0 + k) * D + lane * DS;
                float y[kR][DS];
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    if constexpr (DS == 4) {
                        const float4 z = __ldcg(reinterpret_cast<const float4*>(src + row[i] * D));
                        y[i][0] = z.x; y[i][1] = z.y; y[i][2] = z.z; y[i][3] = z.w;
                    } else {
                        const float2 z = __ldcg(reinterpret_cast<const float2*>(src + row[i] * D));
                        y[i][0] = z.x; y[i][1] = z.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, w[i], k);
#pragma unroll
                    for (int e = 0; e < DS; ++e) acc[i][e] = wi < 0.f ? acc[i][e] : fmaf(y[i][e], wi, acc[i][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kR; ++i)
            if (r + i * by < used) store_row<D, M>(p, few_row<M>(p, s, row[i], D), s.part(), top[i], l[i], acc[i]);
    }
}

// Whether a row of the unit sees a token of the page at `pos` (of its sequence, in the segment).
template <ChunkMode M>
__device__ __forceinline__ bool needed_page(const ChunkParams& p, const Seg<M>& s, int pos) {
    if constexpr (M == kChunkWindow) return pos < s.t1 && (pos + 16 > s.low || pos < p.sinks);
    return pos < s.t1;
}
// Page ids of the segment's KV tiles 8 i .. 8 i + 7, four lanes each, by one warp-wide load.
template <ChunkMode M>
__device__ __forceinline__ int tile_pages(const ChunkParams& p, const Seg<M>& s, int i) {
    const int lane = threadIdx.x & 31, tile = 8 * i + (lane >> 2), pos = s.place(tile) + (lane & 3) * 16;
    if (tile >= s.ntiles || !needed_page<M>(p, s, pos)) return -1;
    return __ldg(p.page_table + size_t(s.sequence()) * p.max_pages + (pos >> 4));
}

// One of the two producing warps fills the rings with a segment's K, V and scales.  An iteration is a
// chain of a wait, two votes, an arrival and the issue of the copies, 0.5 us or more however little it
// copies.  With two stages to a computing warp (kPairs) it therefore takes the whole KV tile, K and V of
// two steps, and the producers take every second tile of the CTA; as one warp for K and one for V, a step at a
// time, the computing warps waited for them (window decode e4m3 took a fifth longer).  With one
// stage to a warp, V of a step would hold up K of the next, so there they are one for K and one
// for V (in tiles, window decode took 28% longer).
//
// Lanes 4 i .. 4 i + 3 own page i of the iteration, the first of them its TMA copy and each a quarter of
// its scales, which come by plain asynchronous copies: a bulk copy of 64 bytes takes as long to issue as
// a page's.  A page that some row of the unit sees a token of arrives whole, whatever its other tokens
// hold; one whose id is bad (flagged) is written by the warp as zeros; others are left as they are.
// `cur`: the ids of tile_pages(0).  `ring` counts steps over the CTA's life.  False after a timeout or an
// abort.
template <int D, bool E4M3, int NR, ChunkMode M>
__device__ __forceinline__ bool produce(const ChunkParams& p, const CUtensorMap* tmk, const CUtensorMap* tmv, unsigned char* sm,
                                        typename CfgFew<D, E4M3, NR>::Bars* bars, const Seg<M>& s, int cur, int ring, int who,
                                        int& armed, volatile uint32_t* abort_flag) {
    using C = CfgFew<D, E4M3, NR>;
    constexpr int kNS = C::kNS, kPageBytes = 16 * D * (E4M3 ? 1 : 2), kSteps = C::kPairs ? 2 : 1;
    constexpr int kPages = C::kPairs ? 8 : 2, kBars = C::kPairs ? 4 : 1;   // of an iteration: (K, V), step, page; (K, V), step
    const int lane = threadIdx.x & 31, h = s.h;
    // the lane's page
    const int pi = lane >> 2, half = C::kPairs ? (pi >> 1) & 1 : 0, sub = pi & 1;
    const bool page_is_v = C::kPairs ? pi >= 4 : who == 1;
    unsigned char* const pages = sm + (page_is_v ? C::kOffV : C::kOffK) + sub * 16 * C::kRowBytes;
    float* const lines = reinterpret_cast<float*>(sm + C::kOffScale) + (page_is_v ? kNS * kStep : 0) + sub * 16 + (lane & 3) * 4;
    const CUtensorMap* map = page_is_v ? tmv : tmk;
    const float* scales = (page_is_v ? p.v_scales : p.k_scales) + (lane & 3) * 4;
    uint64_t* const page_full = page_is_v ? bars->v_full : bars->k_full;
    // the barrier of lanes 0 .. kBars - 1, and its pages among the lanes that issue copies
    const int bar_half = C::kPairs ? lane & 1 : 0;
    const bool bar_is_v = C::kPairs ? (lane & 2) != 0 : who == 1;
    uint64_t* const bar_full = bar_is_v ? bars->v_full : bars->k_full;
    uint64_t* const bar_empty = bar_is_v ? bars->v_empty : bars->k_empty;
    const unsigned bar_pages = 0x11u << (C::kPairs ? 8 * (lane & 3) : 0);
    static_assert(!C::kPairs || (kBars == 4 && kPages == 8), "lanes 2 v + half of the barriers, 4 v + 2 half + sub of the pages");
    int nxt = tile_pages<M>(p, s, 1);
    for (int i = 0; i < 2 * s.ntiles; i += kSteps) {
        const int j = i >> 1, g = ring + i;
        if (i > 0 && (i & 15) == 0) {
            cur = nxt;
            nxt = tile_pages<M>(p, s, j / 8 + 1);
        }
        if (C::kPairs && ((g >> 1) & 1) != who) continue;
        const int in_tile = 2 * ((i & 1) + half) + sub;
        const int page = __shfl_sync(0xffffffffu, cur, (j & 7) * 4 + in_tile);
        const bool mine = pi < kPages && needed_page<M>(p, s, s.place(j) + in_tile * 16);
        const bool ok = mine && page >= 0 && page < p.num_pool_pages;
        const int bar_step = g + bar_half, bar_stage = bar_step % kNS;
        const bool room = lane >= kBars || bar_step < kNS ||
                          mbar_wait_bounded(&bar_empty[bar_stage], (bar_step / kNS - 1) & 1, p.wait_ns);
        if (!__all_sync(0xffffffffu, room && *abort_flag == 0)) {
            if (!room) {
                *abort_flag = 1;
                atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
            }
            return false;
        }
        const unsigned by_tma = __ballot_sync(0xffffffffu, ok);
        const int st = (g + half) % kNS;
        if (__any_sync(0xffffffffu, mine && !ok)) {
            if (mine && !ok) {                             // a lane a quarter of the page's rows
                atomicOr(p.status, TREESPEC_STATUS_BAD_PAGE);
                unsigned char* dst = pages + st * C::kStage + (lane & 3) * 4 * C::kRowBytes;
                for (int pn = 0; pn < C::kNP; ++pn)
                    for (int e = 0; e < 4 * C::kRowBytes / 16; ++e)
                        *reinterpret_cast<uint4*>(dst + pn * C::kPanel + e * 16) = make_uint4(0, 0, 0, 0);
                if (E4M3) *reinterpret_cast<float4*>(lines + st * kStep) = make_float4(0.f, 0.f, 0.f, 0.f);
                fence_proxy_async_smem();                  // the next use of the stage may be by TMA
            }
            __syncwarp();
        }
        if (lane < kBars) mbar_arrive_expect_tx(&bar_full[bar_stage], uint32_t(__popc(by_tma & bar_pages)) * kPageBytes);
        armed = g + kSteps;
        __syncwarp();
        if (ok && (lane & 3) == 0) {
            unsigned char* dst = pages + st * C::kStage;
#pragma unroll
            for (int pn = 0; pn < C::kNP; ++pn) tma_load_3d(dst + pn * C::kPanel, map, 64 * pn, h, page * 16, &page_full[st]);
        }
        if (E4M3 && pi < kPages) {                         // each of the lanes arrives once its copy, if any, is there
            if (ok) copy_16(lines + st * kStep, scales + (size_t(page) * p.Hkv + h) * kPage);
            arrive_behind_copies(&page_full[st]);
        }
        __syncwarp();
    }
    return true;
}

// Whether the plan is there, waited for as all waits are.  By the time that this launch may start it has long been.
__device__ __forceinline__ bool plan_published(const ChunkParams& p) {
    if (load_acquire(p.published) == p.epoch) return true;
    const uint64_t t0 = global_ns();
    do {
        if (load_acquire(p.published) == p.epoch) return true;
    } while (global_ns() - t0 < p.wait_ns);
    return false;
}

template <int D, bool E4M3, int NR, ChunkMode M>
__global__ void __launch_bounds__(kFewThreads, 2)
    chunk_few_kernel(const ChunkParams p, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = CfgFew<D, E4M3, NR>;
    using Bars = typename C::Bars;
    constexpr int kNS = C::kNS;
    constexpr int NM = D / 16;                             // tiles of 16 head elements
    constexpr int kRows = 8 * NR;                          // of a warp
    constexpr int DS = D / 32;
    static_assert(128 * (kRegsCompute + kRegsProduce) <= kFewThreads * 128, "register split exceeds the launch allocation");
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars* bars = reinterpret_cast<Bars*>(sm + C::kOffBar);
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
    const CtaPlan& plan = *reinterpret_cast<const CtaPlan*>(sm + C::kOffEnds);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(sm) & 1023u) {                            // never expected; refuse rather than misread tiles
        grid_dep_wait();
        if (tid == 0) atomicOr(p.status, TREESPEC_STATUS_INTERNAL);
        return;
    }
    if (tid == 0) {
        constexpr int kFullCount = E4M3 ? 9 : 1;           // and the lanes that copy the scales of two pages
        for (int s = 0; s < kNS; ++s) {
            mbar_init(&bars->k_full[s], kFullCount);
            mbar_init(&bars->k_empty[s], 1);               // a step is one warp's
            mbar_init(&bars->v_full[s], kFullCount);
            mbar_init(&bars->v_empty[s], 1);
        }
        for (int s = 0; s < kSegRing; ++s) {
            mbar_init(&bars->seg_full[s], 1);
            mbar_init(&bars->seg_empty[s], kWarps + 2);    // its readers
        }
        mbar_init(&bars->part_full, 32 * kWarps);
        mbar_init(&bars->part_empty, 32 * kWarps);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpProduce && lane == 0) {
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    // Behind the groups' launch, which lets this one start once the plan is there, the wait for that launch comes
    // last: for what follows, the end of this launch stands for the end of that one.  A start that early carries no
    // promise on what the plan and all that came before it have written, so this launch gets it from the plan itself:
    // the plan's first block, which writes or has waited for everything that is read here, stores the call's epoch with
    // release when it is done, the first warp reads it with acquire, and the barrier below hands that on to the others.
    // (The call's last kernel takes the epoch away again, so a replayed graph does not find its own old one.)
    const bool behind_groups = M == kChunkShared && p.published;
    if (!behind_groups) grid_dep_wait();                   // the plan
    grid_dep_release();
    const int me = blockIdx.x;
    if (warp == 0) {
        static_assert(sizeof(CtaPlan) / 4 <= 32, "a word of the plan per lane");
        const bool there = !behind_groups || __all_sync(0xffffffffu, plan_published(p));
        if (!there && lane == 0) atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
        if (lane < int(sizeof(CtaPlan) / 4))
            reinterpret_cast<uint32_t*>(sm + C::kOffEnds)[lane] =
                there ? reinterpret_cast<const uint32_t*>(p.plan + me)[lane] : uint32_t(kNoPlan);
    }
    __syncthreads();
    const bool idle = plan.begin.x < 0;                    // nothing to compute
    // a wait of the whole warp: false for all of its lanes after a timeout of one, or when the CTA has been told to stop
    auto ready = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.wait_ns) && *abort_flag == 0);
    };
    auto give_up = [&]() {
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
    };
    struct Slot {                                          // segment i of the CTA's range, or the end of it
        Seg<M> seg;
        int more;
    };
    static_assert(sizeof(Slot) <= 128, "a slot of the ring of segments");
    auto slot = [&](int i) -> Slot& { return *reinterpret_cast<Slot*>(sm + C::kOffSeg + (i & (kSegRing - 1)) * 128); };
    auto seg_ready = [&](int i) { return ready(&bars->seg_full[i & (kSegRing - 1)], (i / kSegRing) & 1); };
    auto seg_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_empty[i & (kSegRing - 1)]);
    };
    if (warp >= kWarps) {
        regs_lower<kRegsProduce>();
        if (warp > kWarpWalk) {
            if (plan.begin.x != kNoPlan) zero_rows<M, D>(p, lane, 32);
            if (behind_groups) grid_dep_wait();
            return;
        }
        if (idle) return;
        if (behind_groups) fence_proxy_async_global();     // K and V come by TMA: what was acquired, for its proxy too
        if (warp == kWarpWalk) {
            // ------------------------------------------------------------ segments
            Walk<M> walk;
            walk.start(p, plan);
            bool more = true;
            for (int i = 0; more; ++i) {
                Seg<M> s;
                more = walk.next(s);
                if (i >= kSegRing && !ready(&bars->seg_empty[i & (kSegRing - 1)], (i / kSegRing - 1) & 1)) {
                    give_up();
                    break;
                }
                if (lane == 0) {
                    if (more) slot(i).seg = s;
                    slot(i).more = more;
                    mbar_arrive(&bars->seg_full[i & (kSegRing - 1)]);
                }
            }
            return;
        }
        // ---------------------------------------------------------------- TMA producers
        const int who = warp - kWarpProduce;
        int ring = 0, armed = 0, ids = 0;                  // steps before the segment; behind the last tile armed here
        Seg<M> s{}, nxt{};
        auto take = [&](int i, Seg<M>& to, int& pages) -> bool {   // segment i and its first page ids
            if (!seg_ready(i)) {
                give_up();
                return false;
            }
            const bool more = slot(i).more != 0;
            if (more) {
                to = slot(i).seg;
                pages = tile_pages<M>(p, to, 0);
            }
            seg_done(i);
            return more;
        };
        bool more = take(0, s, ids);
        for (int i = 1; more; ++i) {
            int next_ids = 0;
            const bool next_more = take(i, nxt, next_ids);   // its page ids are on their way while this one is copied
            if (!produce<D, E4M3, NR, M>(p, &tmk, &tmv, sm, bars, s, ids, ring, who, armed, abort_flag)) break;
            ring += 2 * s.ntiles;
            s = nxt;
            ids = next_ids;
            more = next_more;
        }
        // the copies on their way land before the CTA may end: the last use of each stage that this
        // warp fills, a lane for each stage of each ring
        const int stage = lane % kNS, last = armed - 1 - ((armed - 1 - stage) & (kNS - 1));
        const bool own = C::kPairs ? ((stage >> 1) & 1) == who : lane / kNS == who;
        if (lane < 2 * kNS && own && last >= 0)
            mbar_wait_bounded(&(lane < kNS ? bars->k_full : bars->v_full)[stage], (last / kNS) & 1, kDefaultWaitNs);
        return;
    }

    // -------------------------------------------------------------------- warps that compute
    regs_raise<kRegsCompute>();
    if (idle) return;
    const int g = lane >> 2, q = lane & 3;
    float* part = reinterpret_cast<float*>(sm + C::kOffPart) + warp * kRows * C::kPitch;
    float2* part_ml = reinterpret_cast<float2*>(sm + C::kOffMl) + warp * kRows;
    // bytes of the lane's chunk c of row g of K in a tile's panel
    int koff[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) koff[c] = E4M3 ? g * D + q * (D / 4) + c * 16 : int(sw128_offset(g, 2 * q + c));
    constexpr int kRowBytes = C::kRowBytes;
    int ring = 0;                                          // steps over the CTA's life
    int segs = 0;
    // Q of a segment, row g + 8 h; matrix instruction kk has the elements of `inner`
    uint32_t qb[NR][NM][2];
    auto load_q = [&](const Seg<M>& s) {
#pragma unroll
        for (int h = 0; h < NR; ++h) {
            const Row r = few_row<M>(p, s, 8 * h + g, D);
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + r.at;
#pragma unroll
            for (int kk = 0; kk < NM; ++kk) {
                const int inner = E4M3 ? q * (D / 4) + kk * 4 : (kk >> 2) * 64 + q * 16 + (kk & 3) * 4;
                const uint2 x = r.ok ? *reinterpret_cast<const uint2*>(src + inner) : make_uint2(0, 0);
                qb[h][kk][0] = x.x;
                qb[h][kk][1] = x.y;
            }
        }
    };
    bool alive = seg_ready(0), more = alive && slot(0).more;
    if (more) load_q(slot(0).seg);
    while (alive && more) {
        const Seg<M>& s = slot(segs).seg;
        float sc[NR][2];                                   // of a score of rows 2 q, 2 q + 1, to base 2
#pragma unroll
        for (int h = 0; h < NR; ++h) {
            float f = p.scale_log2;
            if constexpr (E4M3) {                          // to f16, the largest element to 2^14 .. 2^15
                uint32_t top = 0;                          // its bits; a row with a NaN or an infinity is spoiled anyway
#pragma unroll
                for (int kk = 0; kk < NM; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = qb[h][kk][i] & 0x7fff7fffu;
                        top = max(top, max(x & 0xffffu, x >> 16));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(max(int(top >> 7) - 127, -110), 127);   // exponent of the largest element
                const float up = __int_as_float((14 - e + 127) << 23);    // 2^(14 - e): within 2^-113 .. 2^124
                f *= __int_as_float((e - 14 + 127) << 23);
#pragma unroll
                for (int kk = 0; kk < NM; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qb[h][kk][i] = pack_f16x2(bf16_lo(qb[h][kk][i]) * up, bf16_hi(qb[h][kk][i]) * up);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) sc[h][b] = __shfl_sync(0xffffffffu, f, (2 * q + b) * 4);
        }
        const int used = s.tokens * p.G;                   // rows of the unit
        // what every row of the unit sees: of prefix and new tokens those below all_end, of the window those from
        // all_low on
        const int t1 = s.t1, ntiles = s.ntiles, all_end = min(t1, p.offsets ? s.S + s.i0 + 1 : s.S);
        int low = 0, all_low = 0;
        if constexpr (M == kChunkWindow) {
            low = s.low;
            all_low = p.offsets ? low + s.tokens - 1 : min(s.S, low + p.N - 1);
        }
        float o[NM][NR][4], m[NR][2], l[NR][2];            // O: head elements g, g + 8 of a tile, rows 2 q, 2 q + 1
#pragma unroll
        for (int h = 0; h < NR; ++h) {
            m[h][0] = m[h][1] = -INFINITY;
            l[h][0] = l[h][1] = 0.f;
#pragma unroll
            for (int t = 0; t < NM; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][h][i] = 0.f;
        }

        // the warp's steps of the segment, each a half of a KV tile: of all steps of the CTA, warp, warp + 4, ..
        for (int step = (warp - ring) & (kWarps - 1); step < 2 * ntiles; step += kWarps) {
            const int st = (ring + step) % kNS;
            const uint32_t ph = ((ring + step) / kNS) & 1;
            const int pos0 = s.place(step >> 1) + (step & 1) * kStep;
            const unsigned char* kt = sm + C::kOffK + st * C::kStage;
            const unsigned char* vt = sm + C::kOffV + st * C::kStage;
            bool any = pos0 < t1;                          // some row sees a token
            if constexpr (M == kChunkWindow) any = any && (pos0 + kStep > low || pos0 < p.sinks);
            if (!ready(&bars->k_full[st], ph)) { alive = false; break; }
            if (!any) {
                if (!ready(&bars->v_full[st], ph)) { alive = false; break; }
                if (lane == 0) {
                    mbar_arrive(&bars->k_empty[st]);
                    mbar_arrive(&bars->v_empty[st]);
                }
                continue;
            }
            // ---- S^T: tokens 16 u + g and 8 more, rows 2 q, 2 q + 1 of row tile h
            float x[2][NR][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < NR; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[u][h][i] = 0.f;
            if constexpr (E4M3) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint4 w[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint4*>(kt + koff[c] + 8 * t * kRowBytes);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t a = word_of(w[2 * u], i), b = word_of(w[2 * u + 1], i);
                            const uint32_t a0 = e4m3x2_to_f16x2(uint16_t(a)), a2 = e4m3x2_to_f16x2(uint16_t(a >> 16));
                            const uint32_t a1 = e4m3x2_to_f16x2(uint16_t(b)), a3 = e4m3x2_to_f16x2(uint16_t(b >> 16));
#pragma unroll
                            for (int h = 0; h < NR; ++h) mma_f16(x[u][h], a0, a1, a2, a3, qb[h][4 * c + i][0], qb[h][4 * c + i][1]);
                        }
                }
            } else {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {         // panel c / 2, chunk 2 q + c % 2 of its row
                    uint4 w[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        w[t] = *reinterpret_cast<const uint4*>(kt + (c >> 1) * C::kPanel + koff[c & 1] + 8 * t * kRowBytes);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < NR; ++h)
                            mma_bf16(x[u][h], w[2 * u].x, w[2 * u + 1].x, w[2 * u].y, w[2 * u + 1].y, qb[h][2 * c][0], qb[h][2 * c][1]);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < NR; ++h)
                            mma_bf16(x[u][h], w[2 * u].z, w[2 * u + 1].z, w[2 * u].w, w[2 * u + 1].w, qb[h][2 * c + 1][0],
                                     qb[h][2 * c + 1][1]);
                }
            }
            if constexpr (E4M3) {
                const float* scl = reinterpret_cast<const float*>(sm + C::kOffScale) + st * kStep + g;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float ks = scl[16 * u + 8 * i];
#pragma unroll
                        for (int h = 0; h < NR; ++h)
#pragma unroll
                            for (int b = 0; b < 2; ++b) {  // in this order: ks sc may pass the range where the score does not
                                float& y = x[u][h][2 * i + b];
                                y = y * sc[h][b] * ks;
                            }
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->k_empty[st]);
            // ---- which of the lane's scores count: bit 4 (NR u + h) + i
            uint32_t seen = 0xffffu;
            const bool all = pos0 + kStep <= all_end && (M != kChunkWindow || pos0 >= all_low || pos0 + kStep <= p.sinks);
            if (!all) {
                seen = 0;
#pragma unroll
                for (int h = 0; h < NR; ++h)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const Row r = few_row<M>(p, s, 8 * h + 2 * q + b, D);
                        const Sight<M> si = sight_of<M>(p, s, r);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int pos = pos0 + 16 * u + 8 * i + g;
                                if (r.ok && pos < t1 && sees<M>(p, s, si, pos)) seen |= 1u << (4 * (NR * u + h) + 2 * i + b);
                                else x[u][h][2 * i + b] = -INFINITY;
                            }
                    }
            }
            // ---- the running maxima move only where a score exceeds one by more than 8: P stays below 2^8
            float mx[NR][2];
            bool up = false;
#pragma unroll
            for (int h = 0; h < NR; ++h)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    mx[h][b] = fmaxf(fmax3(x[0][h][b], x[0][h][2 + b], x[1][h][b]), x[1][h][2 + b]) * (E4M3 ? 1.f : sc[h][b]);
                    up |= mx[h][b] > m[h][b] + 8.f;
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int h = 0; h < NR; ++h)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float y = mx[h][b];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                        float al = 1.f;
                        if (y > m[h][b] + 8.f) {
                            al = ex2(m[h][b] - y);
                            m[h][b] = y;
                        }
                        l[h][b] *= al;
#pragma unroll
                        for (int t = 0; t < NM; ++t) {
                            o[t][h][b] *= al;
                            o[t][h][2 + b] *= al;
                        }
                    }
            }
            uint32_t pb[2][NR][2];                         // P^T as the second operand
#pragma unroll
            for (int h = 0; h < NR; ++h)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    // while no score above -inf has come, 0 is subtracted: such a score weighs 0, not NaN
                    const float sub = m[h][b] == -INFINITY ? 0.f : -m[h][b];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float& y = x[u][h][2 * i + b];
                            y = ex2(fmaf(y, E4M3 ? 1.f : sc[h][b], sub));
                            // also where a row's maximum is +inf
                            if (!all && !((seen >> (4 * (NR * u + h) + 2 * i + b)) & 1u)) y = 0.f;
                        }
                    l[h][b] += (x[0][h][b] + x[0][h][2 + b]) + (x[1][h][b] + x[1][h][2 + b]);
                }
            if (!ready(&bars->v_full[st], ph)) { alive = false; break; }
            if constexpr (E4M3) {                          // P times V's scale: one rounding, to bf16
                const float* scl = reinterpret_cast<const float*>(sm + C::kOffScale) + (kNS + st) * kStep + g;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float vs = scl[16 * u + 8 * i];
#pragma unroll
                        for (int h = 0; h < NR; ++h)
#pragma unroll
                            for (int b = 0; b < 2; ++b) {  // a scale that the row does not see may hold anything
                                const float y = x[u][h][2 * i + b] * vs;
                                x[u][h][2 * i + b] = all || ((seen >> (4 * (NR * u + h) + 2 * i + b)) & 1u) ? y : 0.f;
                            }
                    }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < NR; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) pb[u][h][i] = transpose(pack_bf16x2(x[u][h][2 * i], x[u][h][2 * i + 1]));
            bool odd = false;                              // a value that is not finite, in a step that some row sees in part
            if (!all) {
                // V of tokens that no row of the unit sees: zeros, whatever was in their slots
                const int pos = pos0 + lane;
                bool dead = pos >= t1;
                if constexpr (M == kChunkWindow) dead = dead || (pos < low && pos >= p.sinks);
                if (dead) {
#pragma unroll
                    for (int e = 0; e < C::kNP * kRowBytes / 16; ++e)
                        *reinterpret_cast<uint4*>(const_cast<unsigned char*>(vt) + (e >> 3) * C::kPanel + lane * kRowBytes +
                                                  (e & 7) * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();              // the stage's next use is by TMA
                }
                __syncwarp();
                uint32_t found = 0;                        // a carry out of a value's exponent (and mantissa, e4m3)
#pragma unroll 4
                for (int e = lane; e < C::kStage / 16; e += 32) {
                    const uint4 v = *reinterpret_cast<const uint4*>(vt + e * 16);
                    constexpr uint32_t kMost = E4M3 ? 0x7f7f7f7fu : 0x7f807f80u, kOne = E4M3 ? 0x01010101u : 0x00800080u;
                    found |= ((v.x & kMost) + kOne) | ((v.y & kMost) + kOne) | ((v.z & kMost) + kOne) | ((v.w & kMost) + kOne);
                }
                odd = __any_sync(0xffffffffu, (found & (E4M3 ? 0x80808080u : 0x80008000u)) != 0);
            }
            if (!odd) {
                // ---- O^T += V^T P^T, 16 tokens at a time
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if constexpr (E4M3) {
                        // the lane has D / 8 head elements from g D / 8 on of tokens 2 q, 2 q + 1 and 8 more:
                        // elements 2 t and 2 t + 1 are rows g and g + 8 of tile t
                        uint32_t w[4][D / 32];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const unsigned char* src = vt + (16 * u + 2 * q + (i & 1) + 8 * (i >> 1)) * D + g * (D / 8);
                            if constexpr (D == 128) {
                                const uint4 y = *reinterpret_cast<const uint4*>(src);
                                w[i][0] = y.x; w[i][1] = y.y; w[i][2] = y.z; w[i][3] = y.w;
                            } else {
                                const uint2 y = *reinterpret_cast<const uint2*>(src);
                                w[i][0] = y.x; w[i][1] = y.y;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) { // words of 4 elements: tiles 2 k, 2 k + 1
                            const uint32_t lo0 = __byte_perm(w[0][k], w[1][k], 0x5140), hi0 = __byte_perm(w[0][k], w[1][k], 0x7362);
                            const uint32_t lo1 = __byte_perm(w[2][k], w[3][k], 0x5140), hi1 = __byte_perm(w[2][k], w[3][k], 0x7362);
                            auto wide = [](uint32_t two) { return f16x2_to_bf16x2(e4m3x2_to_f16x2(uint16_t(two))); };
                            const uint32_t a0 = wide(lo0), a1 = wide(lo0 >> 16), a2 = wide(lo1), a3 = wide(lo1 >> 16);
                            const uint32_t b0 = wide(hi0), b1 = wide(hi0 >> 16), b2 = wide(hi1), b3 = wide(hi1 >> 16);
#pragma unroll
                            for (int h = 0; h < NR; ++h) {
                                mma_bf16(o[2 * k][h], a0, a1, a2, a3, pb[u][h][0], pb[u][h][1]);
                                mma_bf16(o[2 * k + 1][h], b0, b1, b2, b3, pb[u][h][0], pb[u][h][1]);
                            }
                        }
                    } else {
                        // matrices: tokens 0 .. 7 of chunks 2 t and 2 t + 1, then tokens 8 .. 15 of both
                        const int row = 16 * u + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
                        for (int t = 0; t < NM; ++t) {
                            uint32_t a[4];
                            ldmatrix_trans(a, smem_u32(vt + (t >> 2) * C::kPanel +
                                                       sw128_offset(row, 2 * (t & 3) + ((lane >> 3) & 1))));
#pragma unroll
                            for (int h = 0; h < NR; ++h) mma_bf16(o[t][h], a[0], a[1], a[2], a[3], pb[u][h][0], pb[u][h][1]);
                        }
                    }
                }
            } else {
                // token by token, of what each row sees
#pragma unroll 1
                for (int tok = 0; tok < kStep; ++tok) {
                    const int from = (tok & 7) * 4 + q;
                    const uint32_t sb = __shfl_sync(0xffffffffu, seen, from);
#pragma unroll
                    for (int h = 0; h < NR; ++h)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float lo = tok & 8 ? x[0][h][2 + b] : x[0][h][b], hi = tok & 8 ? x[1][h][2 + b] : x[1][h][b];
                            const float y = __shfl_sync(0xffffffffu, tok & 16 ? hi : lo, from);
                            if (!((sb >> (4 * (NR * (tok >> 4) + h) + 2 * ((tok >> 3) & 1) + b)) & 1u)) continue;
#pragma unroll
                            for (int t = 0; t < NM; ++t)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float v;
                                    if constexpr (E4M3) {
                                        const unsigned char c = vt[tok * D + g * (D / 8) + 2 * t + i];
                                        v = __uint_as_float(f16x2_to_bf16x2(e4m3x2_to_f16x2(c)) << 16);
                                    } else {
                                        v = bf16_to_f32(*reinterpret_cast<const uint16_t*>(
                                            vt + (t >> 2) * C::kPanel + sw128_offset(tok, 2 * (t & 3) + i) + 2 * g));
                                    }
                                    o[t][h][2 * i + b] = fmaf(y, v, o[t][h][2 * i + b]);
                                }
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->v_empty[st]);
        }
        if (!alive) break;
        ring += 2 * ntiles;

        // ---- the warps' states of the unit's rows, joined through shared memory
        if (segs > 0 && !ready(&bars->part_empty, (segs - 1) & 1)) { alive = false; break; }
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[h][b] += __shfl_xor_sync(0xffffffffu, l[h][b], d);
                const int r = 8 * h + 2 * q + b;
                if (r >= used) continue;
                if (g == 0) part_ml[r] = make_float2(m[h][b], l[h][b]);
                float* dst = part + r * C::kPitch;
#pragma unroll
                for (int t = 0; t < NM; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) dst[E4M3 ? g * (D / 8) + 2 * t + i : 16 * t + 8 * i + g] = o[t][h][2 * i + b];
            }
        mbar_arrive(&bars->part_full);
        // the next segment's Q is on its way while this one's rows are joined
        if (!seg_ready(segs + 1)) { alive = false; break; }
        more = slot(segs + 1).more;
        if (more) load_q(slot(segs + 1).seg);
        if (!ready(&bars->part_full, segs & 1)) { alive = false; break; }
        const bool whole = s.whole(), head = s.j0 == 0;
#pragma unroll 4
        for (int r = warp; r < used; r += kWarps) {
            float2 x[kWarps];
            float top = -INFINITY, sum = 0.f, acc[DS];
#pragma unroll
            for (int e = 0; e < DS; ++e) acc[e] = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                x[k] = reinterpret_cast<const float2*>(sm + C::kOffMl)[k * kRows + r];
                top = fmaxf(top, x[k].x);
            }
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float w = state_weight(x[k].x, x[k].y, top);
                if (w < 0.f) continue;
                sum = fmaf(x[k].y, w, sum);
                const float* src = reinterpret_cast<const float*>(sm + C::kOffPart) + (k * kRows + r) * C::kPitch + lane * DS;
                float y[DS];
                if constexpr (DS == 4) {
                    const float4 z = *reinterpret_cast<const float4*>(src);
                    y[0] = z.x; y[1] = z.y; y[2] = z.z; y[3] = z.w;
                } else {
                    const float2 z = *reinterpret_cast<const float2*>(src);
                    y[0] = z.x; y[1] = z.y;
                }
#pragma unroll
                for (int e = 0; e < DS; ++e) acc[e] = fmaf(y[e], w, acc[e]);
            }
            if (whole) {
                store_row<D, M>(p, few_row<M>(p, s, r, D), s.part(), top, sum, acc);
            } else {
                const size_t slot = size_t(2 * me + (head ? 1 : 0)) * 16 + r;
                store_slice<DS>(p.part_acc + slot * D + lane * DS, acc);
                if (lane == 0) __stcg(reinterpret_cast<float2*>(p.part_ml) + slot, make_float2(top, sum));
            }
        }
        mbar_arrive(&bars->part_empty);
        if (!whole) {
            // the last of the warps that hold these rows of a cut unit joins its pieces
            const int c0 = head ? me : plan.first_cta, pieces = head ? plan.last_pieces : plan.first_pieces;
            __threadfence();
            __syncwarp();
            int n = 0;
            if (lane == 0) n = atomicAdd(p.counters + c0 * 8 + warp, 1);
            n = __shfl_sync(0xffffffffu, n, 0);
            if (n == pieces - 1) {
                __threadfence();
                join_rows<D, M>(p, s, c0, pieces, warp, used);
            }
        }
        seg_done(segs);
        ++segs;
    }
    if (!alive) give_up();
}

template <int D, bool E4M3, int NR, ChunkMode M>
cudaError_t launch_few(const ChunkParams& p, cudaStream_t s) {
    using C = CfgFew<D, E4M3, NR>;
    if (p.ctas < 1 || p.ctas > kChunkMaxCtas || p.tpu < 1 || p.tpu * p.G > 8 * NR)
        return cudaErrorInvalidValue;
    CUtensorMap mk = {}, mv = {};
    const long long pool_tokens = (long long)p.num_pool_pages * kPage;
    auto make = E4M3 ? make_code_map : make_pool_map;
    if (!make(&mk, p.k, p.Hkv, pool_tokens, D) || !make(&mv, p.v, p.Hkv, pool_tokens, D)) return cudaErrorInvalidValue;
    auto kern = chunk_few_kernel<D, E4M3, NR, M>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(kern, C::kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.ctas));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;                                      // start while the plan is made
    e = cudaLaunchKernelEx(&cfg, kern, p, mk, mv);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

template <ChunkMode M>
cudaError_t launch_chunk_few(const ChunkParams& p, int kv_dtype, cudaStream_t s) {
    auto launch = [&](auto dim, auto codes) {
        constexpr int D = decltype(dim)::value;
        constexpr bool kCodes = decltype(codes)::value;
        return p.few_rows == 8 ? launch_few<D, kCodes, 1, M>(p, s) : launch_few<D, kCodes, 2, M>(p, s);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (kv_dtype == TREESPEC_DTYPE_E4M3) return p.D == 64 ? launch(D64{}, std::true_type{}) : launch(D128{}, std::true_type{});
    return p.D == 64 ? launch(D64{}, std::false_type{}) : launch(D128{}, std::false_type{});
}

}  // namespace treespec
