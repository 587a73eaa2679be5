// Attention of few query rows per sequence (decoded tokens, small draft trees) over the paged cache,
// with a sliding window or behind shared prefixes: bf16 queries, head dim 64 or 128, K/V bf16 or
// e4m3.
//
// Such a unit, floor(16 R / G) tokens of one sequence and one kv head in R = 1, 2 or 4 row tiles of 16,
// does 4 rows of arithmetic where the 256-row units of chunk_tc.cuh do 256: it is bound by the
// reading of K and V.  There, the chain S -> softmax -> P V over tensor memory takes 0.8 (bf16) to
// 1.3 us (e4m3) per KV tile and SM however few the rows are.  Here warps of their own run over the
// pages of a tile: a warp holds 16 rows of Q and O in registers, a page of 16 tokens is one step of
// 16 x 8 x 16 matrix instructions (S = Q K^T, then P as it lies in registers times V), and no step waits for another
// warp's.  The fragments' inner order is free, so a lane reads 16 bytes of K or V at a time: of K
// the head elements, of V the elements of a token are permuted alike in Q and in O.
//
// A CTA is four such warps and two that fill the K and V rings by TMA, two CTAs to an SM.  With R row tiles, warp w holds
// tile w % R and takes every (4 / R)-th page of a KV tile.  Units, the cut into one range per CTA, pieces
// and the join by the last to finish are those of chunk_units.cuh; at the end of a unit (or piece) the
// warps' states are joined through shared memory.
//
// e4m3: K's codes are widened to f16 (exact), and Q, scaled by a power of two per row, with them: f16
// holds Q's 8 bits from the row's largest element down to 2^-28 of it, and what is smaller is off by
// 2^-39 of that element.  V's codes are widened to bf16 (exact), as P times V's scale is bf16, whose range it needs.
//
// A value that a row may not see must not reach it, and P V multiplies it by zero.  Tokens that no row
// of the unit sees are zeros where the page holds none that is seen; a page that only some rows see whole is looked
// through for values that are not finite, and where there is one its step of P V is done row by row without the hidden
// tokens.
//
// Every wait is bounded, as in chunk_tc.cuh.
#pragma once

#include "chunk_units.cuh"

namespace treespec {

namespace {

constexpr int kWarps = 4;                // warps that compute
constexpr int kFewThreads = 32 * (kWarps + 2);
constexpr int kWarpFewK = kWarps, kWarpFewV = kWarps + 1;

struct TuneFew {
    static constexpr int kKappa = 3;
    static constexpr int kMinTiles = 2, kMinTilesManyRows = 2;
    static constexpr int kWholeTiles = 2;
};

template <int D, bool E4M3>
struct CfgFew {
    static constexpr int kNP = D / 64;
    static constexpr int kPanel = kBN * 128;
    static constexpr int kTile = E4M3 ? kBN * D : kNP * kPanel;
    static constexpr int kNS = 32 * 1024 / kTile > 6 ? 6 : 32 * 1024 / kTile;   // stages of the K ring, and of the V ring
    struct Bars {
        uint64_t k_full[kNS], k_empty[kNS], v_full[kNS], v_empty[kNS], part_full, part_empty;
    };
    static constexpr int kPitch = D + 4;                  // floats of a row of a warp's part
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kNS * kTile;
    static constexpr int kOffScale = kOffV + kNS * kTile;                      // [K, V][kNS][64]
    static constexpr int kOffPart = kOffScale + (E4M3 ? 2 * kNS * kBN * 4 : 0);
    static constexpr int kOffMl = kOffPart + kWarps * 16 * kPitch * 4;         // [kWarps][16] (m, l)
    static constexpr int kOffBar = kOffMl + kWarps * 16 * 8;
    static constexpr int kOffMisc = kOffBar + int(sizeof(Bars));
    static constexpr int kOffEnds = kOffMisc + 16;
    static constexpr int kOffWarp = kOffEnds + 3 * 16;    // scratch of the scan
    static constexpr int kOffTiles = kOffWarp + 8 * 24;   // [entries + 1] tiles before an entry, then units
    static constexpr int smem_bytes(int entries) { return kOffTiles + (entries + 1) * 12; }
    static_assert(kOffBar % 8 == 0 && kOffTiles % 8 == 0 && kOffMl % 8 == 0, "alignment");
    static_assert(2 * (kOffTiles + (kChunkMaxBatch + 1) * 12 + 1024) <= 228 * 1024, "two CTAs to an SM");
};

// D[16 x 8] += A[16 x 16] B[16 x 8].  Lane 4 g + q: A rows g and g + 8 (a0, a2 and a1, a3), inner
// elements 2 q, 2 q + 1 (a0, a1; b0) and 8 more (a2, a3; b1); B column g; D rows g (d0, d1), g + 8,
// columns 2 q, 2 q + 1.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Row r of a finished unit or part: where its float32 state or its result goes, a lane the elements
// lane * D / 32 on.
template <int D, ChunkMode M>
__device__ __forceinline__ void store_row(const ChunkParams& p, const Row& ro, int side, float m, float l, float (&acc)[D / 32]) {
    constexpr int DS = D / 32;
    const int lane = threadIdx.x & 31;
    if (M == kChunkShared && side >= 0) {
        float* dst = p.rows_acc + side_offset(p, side) * D + ro.at + lane * DS;
#pragma unroll
        for (int e = 0; e < DS; ++e) dst[e] = acc[e];
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

// A row's pieces of a cut unit, by one warp: piece k is in slot 2 c0 + 1 (k = 0) or 2 (c0 + k).
template <int D, ChunkMode M>
__device__ __noinline__ void join_row(const ChunkParams& p, int c0, int pieces, int r, const Row& ro, int side) {
    constexpr int DS = D / 32;
    const int lane = threadIdx.x & 31;
    auto slot = [&](int k) { return size_t(k == 0 ? 2 * c0 + 1 : 2 * (c0 + k)) * 64 + r; };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    float top = -INFINITY, l = 0.f, acc[DS];
    float2 x;
    auto fetch = [&](int k) { x = k < pieces ? __ldcg(ml + slot(k)) : make_float2(-INFINITY, 0.f); };
#pragma unroll
    for (int e = 0; e < DS; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < pieces; k0 += 32) {
        fetch(k0 + lane);
        top = fmaxf(top, warp_max(x.x));
    }
    for (int k0 = 0; k0 < pieces; k0 += 32) {
        if (pieces > 32) fetch(k0 + lane);
        const float w = state_weight(x.x, x.y, top);
        l += warp_sum(w < 0.f ? 0.f : x.y * w);
        const int kn = min(32, pieces - k0);
        for (int k = 0; k < kn; k += 8) {                  // eight rows on their way at a time
            float y[8][DS];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float* src = p.part_acc + slot(k0 + min(k + i, kn - 1)) * D + lane * DS;
                if constexpr (DS == 4) {
                    const float4 z = __ldcg(reinterpret_cast<const float4*>(src));
                    y[i][0] = z.x; y[i][1] = z.y; y[i][2] = z.z; y[i][3] = z.w;
                } else {
                    const float2 z = __ldcg(reinterpret_cast<const float2*>(src));
                    y[i][0] = z.x; y[i][1] = z.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, (k + i) & 31);
                if (k + i < kn && wi >= 0.f) {
#pragma unroll
                    for (int e = 0; e < DS; ++e) acc[e] = fmaf(y[i][e], wi, acc[e]);
                }
            }
        }
    }
    store_row<D, M>(p, ro, side, top, l, acc);
}

template <int D, bool E4M3, ChunkMode M>
__global__ void __launch_bounds__(kFewThreads, 2)
    chunk_few_kernel(const ChunkParams p, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = CfgFew<D, E4M3>;
    using Bars = typename C::Bars;
    constexpr int kNS = C::kNS;
    constexpr int NT = D / 8;                              // tiles of 8 head elements of O
    constexpr int DS = D / 32;
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars* bars = reinterpret_cast<Bars*>(sm + C::kOffBar);
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
    int* longest = reinterpret_cast<int*>(sm + C::kOffMisc + 4);
    End* ends = reinterpret_cast<End*>(sm + C::kOffEnds);
    SeqRows* first_rows = reinterpret_cast<SeqRows*>(ends + 2);
    const int entries = chunk_entries<M>(p);
    long long* tiles_s = reinterpret_cast<long long*>(sm + C::kOffTiles);
    int* units_s = reinterpret_cast<int*>(tiles_s + entries + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(sm) & 1023u) {                            // never expected; refuse rather than misread tiles
        grid_dep_wait();
        if (tid == 0) atomicOr(p.status, TREESPEC_STATUS_INTERNAL);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < kNS; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], kWarps);
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], kWarps);
        }
        mbar_init(&bars->part_full, 32 * kWarps);
        mbar_init(&bars->part_empty, 32 * kWarps);
        *abort_flag = 0;
        *longest = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_dep_wait();                                       // the prologues' results
    scan_units<M, kFewThreads>(p, tiles_s, units_s, reinterpret_cast<long long*>(sm + C::kOffWarp), longest);
    const Cut cut = cut_of<M, TuneFew>(p, tiles_s, units_s, *longest);
    zero_rows<M, D, kFewThreads>(p);
    const int me = blockIdx.x;
    if (cut.total == 0 || me >= cut.parts) return;         // nothing to compute
    if (warp < 2) {                                        // warp 0 the begin, warp 1 the end of the range
        const int c = me + warp;
        End e;
        if (cut.m) {
            e = unit_at(p, cut, me / cut.m);
            const SeqRows r = entry_rows<M>(p, e.b);
            const SeqUnits<M> u = seq_units<M>(p, e.b, r);
            const int n = u.tiles(e.pr);
            const int pieces = unit_pieces<TuneFew>(n, 1, cut.m), k = me % cut.m + warp;
            e.j = k > pieces ? n : int((long long)n * k / pieces);   // beyond the last piece: nothing
        } else if (c >= cut.parts) {
            e = End{cut.B, 0, 0, 0};
        } else {
            e = locate<M>(p, cut, cut.bound(c));
            const int n = seq_units<M>(p, e.b).tiles(e.pr);
            if (n <= TuneFew::kWholeTiles) e.j = 2 * e.j < n ? 0 : n;   // short units stay whole
        }
        if (lane == 0) {
            ends[warp] = e;
            if (warp == 0) *first_rows = entry_rows<M>(p, e.b);
        }
    }
    __syncthreads();
    Walk<M> walk;
    walk.start(p, ends[0], ends[1], *first_rows);
    Seg<M> s;

    if (warp >= kWarps) {
        // ---------------------------------------------------------------- TMA producers
        const bool is_v = warp == kWarpFewV;
        uint64_t* full = is_v ? bars->v_full : bars->k_full;
        uint64_t* empty = is_v ? bars->v_empty : bars->k_empty;
        tcparts::ProducerArgs a{};
        a.map = is_v ? &tmv : &tmk;
        a.ring = sm + (is_v ? C::kOffV : C::kOffK);
        a.full = full;
        a.empty = empty;
        a.nst = kNS;
        int armed = 0;
        if constexpr (E4M3) {
            while (walk.next(s))
                if (!produce_codes<D, M, kNS>(p, a.map, static_cast<const unsigned char*>(is_v ? p.v : p.k),
                                              is_v ? p.v_scales : p.k_scales, a.ring,
                                              reinterpret_cast<float*>(sm + C::kOffScale) + (is_v ? kNS * kBN : 0), full, empty,
                                              s, armed, abort_flag))
                    break;
        } else {
            a.src = static_cast<const uint16_t*>(is_v ? p.v : p.k);
            a.stage_bytes = C::kTile;
            a.panel_bytes = C::kPanel;
            a.npg = kBN / 16;
            a.ndp = C::kNP;
            while (walk.next(s)) {
                bool ok = true;
                if constexpr (M == kChunkWindow) {         // the sinks' tiles, then the window's
                    a.low = s.low;
                    a.sinks = p.sinks;
                    const int nh = s.head_tiles();
                    if (nh > 0)
                        ok = tcparts::produce_pages<kBN, D, true>(p, a, s.sequence(), s.h, s.t0, s.t1, s.L, nh, armed, abort_flag);
                    if (ok && nh < s.ntiles)
                        ok = tcparts::produce_pages<kBN, D, true>(p, a, s.sequence(), s.h, s.place(nh), s.t1, s.L, s.ntiles - nh,
                                                                  armed, abort_flag);
                } else {
                    ok = tcparts::produce_pages<kBN, D>(p, a, s.sequence(), s.h, s.t0, s.t1, s.L, s.ntiles, armed, abort_flag);
                }
                if (!ok) break;
            }
        }
        tcparts::drain_copies(a, armed);
        return;
    }

    // -------------------------------------------------------------------- warps that compute
    const int g = lane >> 2, q = lane & 3;
    const int R = p.row_tiles, WT = kWarps / R, rt = warp % R, wt = warp / R;
    float* part = reinterpret_cast<float*>(sm + C::kOffPart) + warp * 16 * C::kPitch;
    float2* part_ml = reinterpret_cast<float2*>(sm + C::kOffMl) + warp * 16;
    // a wait of the whole warp: false for all of its lanes after a timeout of one, or when the CTA has been told to stop
    auto ready = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.wait_ns) && *abort_flag == 0);
    };
    bool alive = true;
    int ring = 0;                                          // tiles over the CTA's life
    int segs = 0;
    while (alive && walk.next(s)) {
        // ---- Q: rows g and g + 8 of the row tile; matrix instruction kk has the elements of `inner`
        Row ro[2];
        Sight<M> si[2];
        uint32_t qa[D / 16][4];
        float sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ro[h] = few_row<M>(p, s, rt * 16 + g + 8 * h, D);
            si[h] = sight_of<M>(p, s, ro[h]);
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + ro[h].at;
            const uint2 none = make_uint2(0, 0);
            sc[h] = p.scale_log2;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int inner = E4M3 ? q * (D / 4) + kk * 4 : (kk >> 2) * 64 + q * 16 + (kk & 3) * 4;
                const uint2 x = ro[h].ok ? *reinterpret_cast<const uint2*>(src + inner) : none;
                qa[kk][h] = x.x;
                qa[kk][2 + h] = x.y;
            }
            if constexpr (E4M3) {                          // to f16, the largest element to 2^14 .. 2^15
                uint32_t top = 0;                          // its bits; a row with a NaN or an infinity is spoiled anyway
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const uint32_t x = qa[kk][h + i] & 0x7fff7fffu;
                        top = max(top, max(x & 0xffffu, x >> 16));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(max(int(top >> 7) - 127, -110), 127);   // exponent of the largest element
                const float up = __int_as_float((14 - e + 127) << 23);    // 2^(14 - e): within 2^-113 .. 2^124
                sc[h] = p.scale_log2 * __int_as_float((e - 14 + 127) << 23);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
                        qa[kk][h + i] = pack_f16x2(bf16_lo(qa[kk][h + i]) * up, bf16_hi(qa[kk][h + i]) * up);
            }
        }
        const bool rows = __any_sync(0xffffffffu, ro[0].ok || ro[1].ok);
        // what every row of the unit sees: of prefix and new tokens those below `all_end`, of the window those from all_low on
        const int all_end = p.offsets ? s.S + s.i0 + 1 : s.S;
        int all_low = 0;
        if constexpr (M == kChunkWindow) all_low = p.offsets ? s.low + s.tokens - 1 : min(s.S, s.low + p.N - 1);
        float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] = 0.f;

        for (int j = 0; j < s.ntiles; ++j, ++ring) {
            const int st = ring % kNS;
            const uint32_t ph = (ring / kNS) & 1;
            const int base = s.place(j);
            const unsigned char* kt = sm + C::kOffK + st * C::kTile;
            const unsigned char* vt = sm + C::kOffV + st * C::kTile;
            // S of this warp's pages waits for K alone, P V then for V
            if (!ready(&bars->k_full[st], ph)) { alive = false; break; }
            bool have_v = false;
            for (int pg = wt; pg < 4; pg += WT) {
                const int pos0 = base + 16 * pg;
                bool any = rows && pos0 < s.t1;
                if constexpr (M == kChunkWindow) any = any && (pos0 + 16 > s.low || pos0 < p.sinks);
                if (!any) continue;                        // no row sees a token of the page
                // ---- S: tokens 8 t + g of the page in column g of tile t
                float x[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[t][i] = 0.f;
                    const int row = 16 * pg + 8 * t + g;
                    if constexpr (E4M3) {
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            const uint4 w = *reinterpret_cast<const uint4*>(kt + row * D + q * (D / 4) + c * 16);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t y = word_of(w, i);
                                mma_f16(x[t], qa[4 * c + i], e4m3x2_to_f16x2(uint16_t(y)), e4m3x2_to_f16x2(uint16_t(y >> 16)));
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) { // panel c / 2, chunk 2 q + c % 2 of its row
                            const uint4 w = *reinterpret_cast<const uint4*>(kt + (c >> 1) * C::kPanel +
                                                                            sw128_offset(row, 2 * q + (c & 1)));
                            mma_bf16(x[t], qa[2 * c], w.x, w.y);
                            mma_bf16(x[t], qa[2 * c + 1], w.z, w.w);
                        }
                    }
                }
                float2 vs[2];
                if constexpr (E4M3) {
                    const float* scl = reinterpret_cast<const float*>(sm + C::kOffScale) + st * kBN + 16 * pg + 2 * q;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float2 ks = *reinterpret_cast<const float2*>(scl + 8 * t);
                        x[t][0] *= ks.x * sc[0];
                        x[t][1] *= ks.y * sc[0];
                        x[t][2] *= ks.x * sc[1];
                        x[t][3] *= ks.y * sc[1];
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[t][i] *= sc[0];
                }
                // ---- which of the lane's 8 scores count: bit 4 t + i
                uint32_t seen = 0xffu;
                const bool all = pos0 + 16 <= all_end && (M != kChunkWindow || pos0 >= all_low || pos0 + 16 <= p.sinks);
                if (!all) {
                    seen = 0;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int pos = pos0 + 8 * t + 2 * q + (i & 1), h = i >> 1;
                            if (ro[h].ok && pos < s.t1 && sees<M>(p, s, si[h], pos)) seen |= 1u << (4 * t + i);
                        }
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!((seen >> (4 * t + i)) & 1u)) x[t][i] = -INFINITY;
                }
                // ---- the running maxima and sums
                float mn[2], al[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float y = fmaxf(fmaxf(x[0][2 * h], x[0][2 * h + 1]), fmaxf(x[1][2 * h], x[1][2 * h + 1]));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
                    mn[h] = fmaxf(m[h], y);
                }
                if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        al[h] = mn[h] > m[h] ? ex2(m[h] - mn[h]) : 1.f;
                        l[h] *= al[h];
                        m[h] = mn[h];
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        o[t][0] *= al[0];
                        o[t][1] *= al[0];
                        o[t][2] *= al[1];
                        o[t][3] *= al[1];
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int h = i >> 1;
                        // while no score above -inf has come, 0 is subtracted: such a score weighs 0, not NaN
                        x[t][i] = ex2(x[t][i] - (m[h] == -INFINITY ? 0.f : m[h]));
                        if (!all && !((seen >> (4 * t + i)) & 1u)) x[t][i] = 0.f;
                        l[h] += x[t][i];
                    }
                if (!have_v) {
                    if (!ready(&bars->v_full[st], ph)) { alive = false; break; }
                    have_v = true;
                }
                if constexpr (E4M3) {                      // P times V's scale: one rounding, to bf16
                    const float* scl = reinterpret_cast<const float*>(sm + C::kOffScale) + kNS * kBN + st * kBN + 16 * pg + 2 * q;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        vs[t] = *reinterpret_cast<const float2*>(scl + 8 * t);
#pragma unroll
                        for (int i = 0; i < 4; ++i)        // a scale that the row does not see may hold anything
                            x[t][i] = (seen >> (4 * t + i)) & 1u ? x[t][i] * (i & 1 ? vs[t].y : vs[t].x) : 0.f;
                    }
                }
                // ---- O += P V; the lane has the head elements of column g, tokens 2 q, 2 q + 1 and 8 more
                const uint32_t pa[4] = {pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3]),
                                        pack_bf16x2(x[1][0], x[1][1]), pack_bf16x2(x[1][2], x[1][3])};
                auto token = [&](int i) { return 16 * pg + 2 * q + (i & 1) + 8 * (i >> 1); };
                uint32_t w[C::kNP][4][4];                  // e4m3, D 64: two words a token
                bool odd = false;                          // a value that is not finite
#pragma unroll
                for (int pn = 0; pn < (E4M3 ? 1 : C::kNP); ++pn)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint4 y;
                        if constexpr (!E4M3) {
                            y = *reinterpret_cast<const uint4*>(vt + pn * C::kPanel + sw128_offset(token(i), g));
                        } else if constexpr (D == 128) {
                            y = *reinterpret_cast<const uint4*>(vt + token(i) * D + g * 16);
                        } else {
                            const uint2 z = *reinterpret_cast<const uint2*>(vt + token(i) * D + g * 8);
                            y = make_uint4(z.x, z.y, 0, 0);
                        }
                        w[pn][i][0] = y.x; w[pn][i][1] = y.y; w[pn][i][2] = y.z; w[pn][i][3] = y.w;
                    }
                if (!all) {
#pragma unroll
                    for (int pn = 0; pn < (E4M3 ? 1 : C::kNP); ++pn)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t y = w[pn][i][k];
                                if constexpr (E4M3) odd |= (((y & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                                else odd |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
                            }
                    odd = __any_sync(0xffffffffu, odd);
                }
                if (!odd) {
                    if constexpr (E4M3) {
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) { // words of 4 elements: tiles 4 k .. 4 k + 3
                            const uint32_t lo0 = __byte_perm(w[0][0][k], w[0][1][k], 0x5140), hi0 = __byte_perm(w[0][0][k], w[0][1][k], 0x7362);
                            const uint32_t lo1 = __byte_perm(w[0][2][k], w[0][3][k], 0x5140), hi1 = __byte_perm(w[0][2][k], w[0][3][k], 0x7362);
                            auto wide = [](uint32_t two) { return f16x2_to_bf16x2(e4m3x2_to_f16x2(uint16_t(two))); };
                            mma_bf16(o[4 * k], pa, wide(lo0), wide(lo1));
                            mma_bf16(o[4 * k + 1], pa, wide(lo0 >> 16), wide(lo1 >> 16));
                            mma_bf16(o[4 * k + 2], pa, wide(hi0), wide(hi1));
                            mma_bf16(o[4 * k + 3], pa, wide(hi0 >> 16), wide(hi1 >> 16));
                        }
                    } else {
#pragma unroll
                        for (int pn = 0; pn < C::kNP; ++pn)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t(&v)[4][4] = w[pn];
                                mma_bf16(o[8 * pn + 2 * k], pa, __byte_perm(v[0][k], v[1][k], 0x5410),
                                         __byte_perm(v[2][k], v[3][k], 0x5410));
                                mma_bf16(o[8 * pn + 2 * k + 1], pa, __byte_perm(v[0][k], v[1][k], 0x7632),
                                         __byte_perm(v[2][k], v[3][k], 0x7632));
                            }
                    }
                } else {
                    // row by row and token by token, of what each row sees: element (t, i) of column b is that of
                    // D's column 2 q + b
                    for (int tok = 0; tok < 16; ++tok) {
                        const int from = (lane & ~3) | ((tok & 7) >> 1), bit = 4 * (tok >> 3) + (tok & 1);
                        const uint32_t sb = __shfl_sync(0xffffffffu, seen, from);
                        float pt[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float y = tok >= 8 ? ((tok & 1) ? x[1][2 * h + 1] : x[1][2 * h]) : ((tok & 1) ? x[0][2 * h + 1] : x[0][2 * h]);
                            pt[h] = __shfl_sync(0xffffffffu, y, from);
                        }
                        const int row = 16 * pg + tok;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                float v;
                                if constexpr (E4M3) {
                                    const unsigned char c = vt[row * D + (2 * q + b) * (D / 8) + t];
                                    v = __uint_as_float(f16x2_to_bf16x2(e4m3x2_to_f16x2(c)) << 16);
                                } else {
                                    v = bf16_to_f32(*reinterpret_cast<const uint16_t*>(
                                        vt + (t >> 3) * C::kPanel + sw128_offset(row, 2 * q + b) + 2 * (t & 7)));
                                }
                                if ((sb >> bit) & 1u) o[t][b] = fmaf(pt[0], v, o[t][b]);
                                if ((sb >> (bit + 2)) & 1u) o[t][2 + b] = fmaf(pt[1], v, o[t][2 + b]);
                            }
                    }
                }
            }
            if (!alive) break;
            if (!have_v && !ready(&bars->v_full[st], ph)) { alive = false; break; }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars->k_empty[st]);
                mbar_arrive(&bars->v_empty[st]);
            }
        }
        if (!alive) break;

        // ---- the warps' states of the unit's rows, joined through shared memory
        if (segs > 0 && !ready(&bars->part_empty, (segs - 1) & 1)) { alive = false; break; }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (!ro[h].ok) continue;
            float* dst = part + (g + 8 * h) * C::kPitch;
            if (q == 0) part_ml[g + 8 * h] = make_float2(m[h], l[h]);
            // tiles t of a panel (all, over codes) are consecutive elements, D / 8 (8 over bf16) per column
            constexpr int kRun = E4M3 ? D / 8 : 8;
#pragma unroll
            for (int t0 = 0; t0 < NT; t0 += kRun)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int t = 0; t < kRun; t += 4)
                        *reinterpret_cast<float4*>(dst + t0 * 8 + (2 * q + b) * kRun + t) =
                            make_float4(o[t0 + t][2 * h + b], o[t0 + t + 1][2 * h + b], o[t0 + t + 2][2 * h + b],
                                        o[t0 + t + 3][2 * h + b]);
        }
        mbar_arrive(&bars->part_full);
        if (!ready(&bars->part_full, segs & 1)) { alive = false; break; }
        ++segs;
        const bool whole = s.whole(), head = s.j0 == 0;
        const int used = min(16, s.tokens * p.G - rt * 16);    // rows of the tile
        for (int r = wt; r < used; r += WT) {
            float2 x[kWarps];
            float top = -INFINITY, sum = 0.f, acc[DS];
#pragma unroll
            for (int e = 0; e < DS; ++e) acc[e] = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k)
                if (k < WT) {
                    x[k] = reinterpret_cast<const float2*>(sm + C::kOffMl)[(k * R + rt) * 16 + r];
                    top = fmaxf(top, x[k].x);
                }
#pragma unroll
            for (int k = 0; k < kWarps; ++k)
                if (k < WT) {
                    const float w = state_weight(x[k].x, x[k].y, top);
                    if (w < 0.f) continue;
                    sum = fmaf(x[k].y, w, sum);
                    const float* src = reinterpret_cast<const float*>(sm + C::kOffPart) + ((k * R + rt) * 16 + r) * C::kPitch + lane * DS;
#pragma unroll
                    for (int e = 0; e < DS; ++e) acc[e] = fmaf(src[e], w, acc[e]);
                }
            if (whole) {
                store_row<D, M>(p, few_row<M>(p, s, rt * 16 + r, D), s.part(), top, sum, acc);
            } else {
                const size_t slot = size_t(2 * me + (head ? 1 : 0)) * 64 + rt * 16 + r;
#pragma unroll
                for (int e = 0; e < DS; ++e) __stcg(p.part_acc + slot * D + lane * DS + e, acc[e]);
                if (lane == 0) __stcg(reinterpret_cast<float2*>(p.part_ml) + slot, make_float2(top, sum));
            }
        }
        mbar_arrive(&bars->part_empty);
        if (!whole && used > 0) {
            // the last of the warps that hold these rows of a cut unit joins its pieces
            int c0, pieces;
            if (cut.m) {
                c0 = me / cut.m * cut.m;
                pieces = unit_pieces<TuneFew>(s.n, 1, cut.m);
            } else {
                const SeqUnits<M> u = seq_units<M>(p, s.b);
                const long long ub = cut.before(s.b) + s.h * div_pos(cut.before(s.b + 1) - cut.before(s.b), cut.Hkv) +
                                     u.tiles_before(s.pr) + (long long)cut.k * s.pr + cut.k;
                c0 = cut.owner(ub);
                pieces = cut.owner(ub + s.n - 1) - c0 + 1;
            }
            __threadfence();
            __syncwarp();
            int n = 0;
            if (lane == 0) n = atomicAdd(p.counters + c0 * 8 + warp, 1);
            n = __shfl_sync(0xffffffffu, n, 0);
            if (n == pieces - 1) {
                __threadfence();
                for (int r = wt; r < used; r += WT)
                    join_row<D, M>(p, c0, pieces, rt * 16 + r, few_row<M>(p, s, rt * 16 + r, D), s.part());
            }
        }
    }
    if (!alive) {
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
    }
}

template <int D, bool E4M3, ChunkMode M>
cudaError_t launch_few(const ChunkParams& p, cudaStream_t s) {
    using C = CfgFew<D, E4M3>;
    const int entries = M == kChunkShared ? p.entries : p.B;
    if (entries > kChunkMaxBatch || p.ctas < 1 || p.ctas > kChunkMaxCtas || p.tpu < 1 || p.tpu * p.G > 16 * p.row_tiles)
        return cudaErrorInvalidValue;
    if (p.row_tiles != 1 && p.row_tiles != 2 && p.row_tiles != 4) return cudaErrorInvalidValue;
    CUtensorMap mk = {}, mv = {};
    const long long pool_tokens = (long long)p.num_pool_pages * kPage;
    auto make = E4M3 ? make_code_map : make_pool_map;
    if (!make(&mk, p.k, p.Hkv, pool_tokens, D) || !make(&mv, p.v, p.Hkv, pool_tokens, D)) return cudaErrorInvalidValue;
    auto kern = chunk_few_kernel<D, E4M3, M>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(kern, C::smem_bytes(kChunkMaxBatch), smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.ctas));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = C::smem_bytes(entries);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.offsets && M != kChunkShared ? 0 : 1;   // trees and groups: start while the prologue runs
    e = cudaLaunchKernelEx(&cfg, kern, p, mk, mv);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

template <ChunkMode M>
cudaError_t launch_chunk_few(const ChunkParams& p, int kv_dtype, cudaStream_t s) {
    if (kv_dtype == TREESPEC_DTYPE_E4M3) return p.D == 64 ? launch_few<64, true, M>(p, s) : launch_few<128, true, M>(p, s);
    return p.D == 64 ? launch_few<64, false, M>(p, s) : launch_few<128, false, M>(p, s);
}

}  // namespace treespec
