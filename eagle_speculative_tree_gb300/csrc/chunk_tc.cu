// Attention of packed chunks (tree_chunk_attn), and of trees over 8-bit pools, on the
// 5th-generation tensor cores: bf16 queries, head dim 64 or 128, K/V bf16 or e4m3.
//
// A unit is 2 floor(128 / G) consecutive new tokens of one sequence and one kv head: their
// rows (token x query head of the group) fill two 128-row query tiles, the second of which
// is idle where the unit's tokens fit the first.  A unit runs over the sequence's logical
// tokens, from 0 to the last that one of its rows may see, in KV tiles of 64.
//
// One CTA per SM.  The units, ordered (sequence, kv head, rows), and within them their KV
// tiles are cut into equal contiguous ranges, one per CTA, so single decoded tokens over a
// long cache, prompts and any mixture load every SM alike, whatever the lengths; they are
// on the device and the host does not know them.  A unit costs kKappa tiles beyond its own
// (its epilogue and the restart of the pipeline).  A unit cut between CTAs leaves a partial
// (m, l, O) of each piece in the CTAs' slots; of the warps that hold the same 32 rows the
// one that finishes last joins them, in the order of the pieces, so the result does not
// depend on which one that is and nobody waits for another CTA.
//
// Within a CTA, as in the two-tile tree kernel: S_t(j) = Q_t K(j)^T in 64 tensor-memory
// columns, double-buffered, P_t(j) written over it as bf16, O_t += P_t(j) V(j); one warp
// issues the MMAs of each query tile, one warpgroup runs each tile's softmax with a row per
// thread, and O is rescaled only when a row's running maximum grows by more than 2^8.
//   bf16 K/V: warps 8 and 9 fill the K and V rings by TMA, a page of 16 tokens at a time.
//   e4m3 K/V: warps 8 and 9 fill rings of codes and scales in the same way, and four more
//   warps widen the codes exactly to bf16 operands.  K's scale multiplies a column of S
//   inside the exponent's fused multiply-add, V's multiplies P before it is rounded.
//
// Rows are spread over the four warps of a tile (row r in lane r / 4 of warp r % 4), so that
// the few rows of a decoded token share the epilogue's work.
//
// A value that a row may not see must not reach it.  S is masked by selection, but P V
// multiplies a masked token's V by zero, and 0 x NaN is NaN.  A row whose O comes out
// non-finite, and does not see what makes it so, is therefore recomputed from the visible tokens
// alone, on CUDA cores: rare and slow, and no cost to the others but a test in the epilogue.  It is done behind the CTA's last
// segment, where no hand-off of the pipeline, whose waits are bounded, depends on its time.
//
// Every mbarrier wait is bounded; on expiry the CTA records TREESPEC_STATUS_TIMEOUT, drains
// its own copies and MMAs, frees its tensor memory and exits.
#include <type_traits>

#include "attn_tc_parts.cuh"

namespace treespec {

namespace {

using namespace sm100;

constexpr int kM = 128;              // rows of a query tile = TMEM lanes
constexpr int kNQ = 2;               // query tiles
constexpr int kBN = 64;              // tokens per KV tile
constexpr int kKappa = 7;            // a unit's fixed cost, in tiles
constexpr int kRaw = 5;              // e4m3: stages of the rings of codes
// No piece of a unit with CTAs of its own is shorter than this.  Joining costs by the row, so
// units of many rows are cut into longer pieces (8 nodes x 4 heads over 2048 e4m3 tokens: 28.7
// us in pieces of 4 tiles, 30.9 of 9; 3 prompts of up to 816 tokens, 4 heads: 33 and 25).
constexpr int kMinTiles = 4, kMinTilesManyRows = 9;
constexpr int kWholeTiles = 4;       // units up to this long are not cut
constexpr int kScaleRing = 4;        // e4m3: tiles of scales
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;        // S buffer b of tile t: [128 t + 64 b, 128 t + 64 b + 64)
constexpr uint32_t kColO = 256;      // O_t: [256 + 128 t, 256 + 128 t + D)
constexpr int kWarpK = 8, kWarpV = 9, kWarpMma = 10, kWarpConv = 12;

template <int D, bool E4M3>
struct Cfg {
    static constexpr int kNP = D / 64;                    // 64-element panels of a row
    static constexpr int kNS = E4M3 ? 2 : D == 128 ? 4 : 6;   // stages of the K ring, and of the V ring
    static constexpr int kThreads = E4M3 ? 512 : 384;
    static constexpr int kQPanel = kM * 128;
    static constexpr int kQTile = kNP * kQPanel;
    static constexpr int kPanel = kBN * 128;
    static constexpr int kTile = kNP * kPanel;
    static constexpr int kRawTile = E4M3 ? kBN * D : 0;   // codes of one operand's tile
    // registers: two softmax warpgroups, the producer / issuer one, the converting one; the
    // sum is what the launch allocates (384 x 168 or 512 x 128)
    static constexpr uint32_t kRegsSoftmax = 200;
    static constexpr uint32_t kRegsOther = E4M3 ? 40 : 56;
    static constexpr uint32_t kRegsConv = 72;
    static_assert(E4M3 ? 128 * (2 * kRegsSoftmax + kRegsOther + kRegsConv) <= 512 * 128
                       : 128 * (2 * kRegsSoftmax + kRegsOther) <= 384 * 168,
                  "register split exceeds the launch allocation");
    struct Bars {
        uint64_t k_full[kNS], k_empty[kNS], v_full[kNS], v_empty[kNS];
        uint64_t q_full[kNQ], s_full[kNQ][2], p_full[kNQ][2], pv_done[kNQ][2], o_full[kNQ], o_free[kNQ], drain[kNQ];
        // e4m3: a tile's codes have landed / been read; its scales stand where the softmax reads them
        uint64_t rk_full[kRaw], rk_empty[kRaw], rv_full[kRaw], rv_empty[kRaw], sck_full[kScaleRing],
            scv_full[kScaleRing];
    };
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kNQ * kQTile;
    static constexpr int kOffV = kOffK + kNS * kTile;
    static constexpr int kOffRaw = kOffV + kNS * kTile;
    static constexpr int kOffRawScale = kOffRaw + 2 * kRaw * kRawTile;              // [K, V][kRaw][64]
    static constexpr int kOffScale = kOffRawScale + (E4M3 ? 2 * kRaw * kBN * 4 : 0);   // [kScaleRing][K, V][64]
    static constexpr int kOffBar = kOffScale + (E4M3 ? kScaleRing * 2 * kBN * 4 : 0);
    static constexpr int kOffMisc = kOffBar + int(sizeof(Bars));
    static constexpr int kOffEnds = kOffMisc + 16;        // the two ends of the CTA's range
    static constexpr int kOffWarp = kOffEnds + 3 * 16;    // scratch of the scan
    static constexpr int kOffTiles = kOffWarp + 16 * 24;  // [kChunkMaxBatch + 1] tiles before a sequence, one kv head
    static constexpr int kOffUnits = kOffTiles + (kChunkMaxBatch + 1) * 8;   // and units
    static constexpr int kSmemBytes = kOffUnits + (kChunkMaxBatch + 1) * 4;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
    static_assert(kOffBar % 8 == 0 && kOffTiles % 8 == 0, "alignment");
};

// ------------------------------------------------------------------ units and the cut

// a / b of non-negative numbers; a 64-bit division costs several times a 32-bit one, and
// nearly every batch's positions fit 32 bits
__device__ __forceinline__ long long div_pos(long long a, long long b) {
    if (((a | b) >> 32) == 0) return uint32_t(a) / uint32_t(b);
    return a / b;
}

// sum over i = 0 .. n - 1 of floor((a i + b) / m), by the Euclidean reduction of (a, m) that counts the
// lattice points under a line; all terms and the sum within 32 bits / 64 bits
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    long long ans = 0;
    while (n) {
        if (a >= m) {
            ans += (long long)(n) * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            ans += (long long)n * (b / m);
            b %= m;
        }
        const uint32_t y = a * n + b;                      // < 64 (n + 1): n is below 2^24
        if (y < m) break;
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return ans;
}

// The units of one sequence and one kv head.
struct SeqUnits {
    int S, live, np;                  // prefix, rows' tokens, units
    int tpu;                          // tokens per unit
    bool tree;
    // KV tiles of unit pr
    __device__ __forceinline__ int tiles(int pr) const {
        return (S + (tree ? live : min(live, (pr + 1) * tpu)) + kBN - 1) / kBN;
    }
    // KV tiles of units 0 .. pr - 1
    __device__ __forceinline__ long long tiles_before(int pr) const {
        if (pr <= 0) return 0;
        if (tree) return (long long)pr * tiles(0);
        const int full = min(pr, live / tpu);              // units whose tokens are all there
        const int A = S + kBN - 1 + tpu;                   // sum of floor((A + k tpu) / 64), k = 0 .. full - 1
        const int a1 = tpu / kBN, r = tpu % kBN;
        long long s = (long long)full * (A / kBN) + (long long)full * (full - 1) / 2 * a1;
        if (r) s += floor_sum(uint32_t(full), kBN, uint32_t(r), uint32_t(A % kBN));
        return pr > full ? s + tiles(pr - 1) : s;
    }
};
__device__ __forceinline__ SeqUnits seq_units(const ChunkParams& p, const SeqRows& r) {
    SeqUnits u;
    u.tree = !p.offsets;
    u.tpu = 2 * p.tpq;
    u.S = r.S;
    u.live = r.S < 0 ? 0 : r.live;
    u.np = (u.live + u.tpu - 1) / u.tpu;
    return u;
}

// Positions of the cut: unit (b, h, pr) begins at Hkv (tiles[b] + k units[b]) + h (tiles and
// k units of the sequence) + (tiles and k units before pr), and its tile j lies k + j after
// that.
struct Cut {
    const long long* tiles;           // [B + 1], shared memory
    const int* units;
    long long total;
    int B, Hkv, k, parts;
    int m;                            // 0: even cut; else parts m u .. m u + m - 1 share unit u
    __device__ __forceinline__ long long before(int b) const { return Hkv * (tiles[b] + (long long)k * units[b]); }
    __device__ __forceinline__ long long bound(int c) const { return div_pos(total * c, parts); }    // total x CTAs < 2^63
    // the part that holds position x: the last c with bound(c) <= x
    __device__ __forceinline__ int owner(long long x) const { return int(div_pos((x + 1) * parts - 1, total)); }
};
struct End {                          // tile j of unit (b, h, pr)
    int b, h, pr, j;
};
// Pieces of a unit of n tiles and that many rows that m CTAs share.
__device__ __forceinline__ int unit_pieces(int n, int rows, int m) {
    return min(m, max(1, n / (rows > 64 ? kMinTilesManyRows : kMinTiles)));
}

// The cut of a batch: the prefix sums and the KV tiles of its longest unit.
__device__ __forceinline__ Cut cut_of(const ChunkParams& p, const long long* tiles, const int* units, int longest) {
    // A range that holds pieces of two units pays the fixed cost twice, so where there is less
    // than about that cost for each CTA, every unit gets CTAs of its own instead (119 new
    // tokens, 32 q / 8 kv heads: 35 us cut evenly, 21 this way; 8 nodes over 2048 e4m3 tokens:
    // 42 and 29), unless one long unit among short ones would then run far longer than its
    // share of all tiles
    Cut cut;
    const long long n = (long long)p.Hkv * units[p.B];
    cut.tiles = tiles;
    cut.units = units;
    cut.B = p.B;
    cut.Hkv = p.Hkv;
    cut.k = kKappa;
    cut.total = p.Hkv * tiles[p.B] + kKappa * n;
    cut.m = 0;
    if (cut.total < (long long)(kKappa + 2) * gridDim.x && n <= gridDim.x && n > 0) {
        const int m = int(gridDim.x) / int(n);
        if (longest / unit_pieces(longest, 1, m) <= int(cut.total) / int(gridDim.x) + 2 * kKappa) cut.m = m;
    }
    cut.parts = cut.m ? cut.m * int(n) : int(min((long long)gridDim.x, max(1ll, cut.total / (kKappa + 1))));
    return cut;
}

// Unit u of the batch, in the order of the cut.
__device__ __forceinline__ End unit_at(const ChunkParams& p, const Cut& q, int u) {
    int lo = 0, hi = q.B;                                  // the last b whose units begin at or before u
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.Hkv * q.units[mid] <= u) lo = mid;
        else hi = mid;
    }
    const int np = q.units[lo + 1] - q.units[lo], off = u - q.Hkv * q.units[lo];
    return End{lo, off / np, off % np, 0};
}

// The tile at or after position x of the cut, by one warp.  x < total.
__device__ __forceinline__ End locate(const ChunkParams& p, const Cut& q, long long x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = q.B;                                  // the last b with before(b) <= x
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.before(mid) <= x) lo = mid;
        else hi = mid;
    }
    End e;
    e.b = lo;
    const SeqUnits u = seq_units(p, seq_rows(p, lo));
    const long long head = div_pos(q.before(lo + 1) - q.before(lo), q.Hkv);
    long long y = x - q.before(lo);
    e.h = int(div_pos(y, head));
    y -= e.h * head;
    int at = 0, n = u.np;                                  // the last unit that begins at or before y, 32 ways
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool le = i < n && u.tiles_before(at + i) + (long long)q.k * (at + i) <= y;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int last = 31 - __clz(m);                    // lane 0 always holds
        at += last * step;
        n = min(step, n - last * step);
    }
    e.pr = at;
    y -= u.tiles_before(at) + (long long)q.k * at;
    e.j = int(max(0ll, y - q.k));
    return e;
}

// One contiguous range of KV tiles of one unit.
struct Seg {
    int b, h, pr;
    int S, live, L;        // prefix, rows' tokens and logical tokens of the sequence
    int row0;              // q row of the unit's first token
    int i0, tokens;        // the unit's tokens: i0 .. i0 + tokens - 1 of the sequence's new ones
    int j0, ntiles, n;     // tiles j0 .. j0 + ntiles - 1 of n
    int t0, t1;            // their logical tokens
    int nq;                // query tiles in use
    __device__ __forceinline__ bool whole() const { return ntiles == n; }
};

// The segments of a CTA's range, in order.  Every role walks them by itself.
struct Walk {
    const ChunkParams* p;
    End e, end;            // next segment's first tile; the first tile behind the range
    SeqUnits u;
    SeqRows rows;
    __device__ __forceinline__ void load() {
        rows = seq_rows(*p, e.b);
        u = seq_units(*p, rows);
    }
    __device__ __forceinline__ void start(const ChunkParams& pp, const End& a, const End& z, const SeqRows& r) {
        p = &pp;
        e = a;
        end = z;
        rows = r;                                          // of sequence a.b
        u = seq_units(pp, r);
        if (e.b < pp.B && e.j >= u.tiles(e.pr)) advance();
    }
    __device__ __forceinline__ bool next(Seg& s) {
        // behind the range: also where both its ends were moved to the same unit's end
        if (e.b > end.b || (e.b == end.b && (e.h > end.h || (e.h == end.h && e.pr > end.pr)))) return false;
        const bool last = e.b == end.b && e.h == end.h && e.pr == end.pr;
        if (last && e.j >= end.j) return false;
        s.b = e.b;
        s.h = e.h;
        s.pr = e.pr;
        s.S = u.S;
        s.live = u.live;
        s.L = u.S + u.live;
        s.i0 = e.pr * u.tpu;
        s.tokens = min(u.tpu, u.live - s.i0);
        s.row0 = rows.row0 + s.i0;
        s.nq = s.tokens > u.tpu / 2 ? 2 : 1;
        s.n = u.tiles(e.pr);
        s.j0 = e.j;
        s.ntiles = (last ? min(end.j, s.n) : s.n) - e.j;
        const int vis = u.S + (u.tree ? u.live : s.i0 + s.tokens);
        s.t0 = s.j0 * kBN;
        s.t1 = min(vis, (s.j0 + s.ntiles) * kBN);
        if (last) e.b = end.b + 1;                         // done
        else advance();
        return true;
    }
    // to the first tile of the next unit
    __device__ __forceinline__ void advance() {
        e.j = 0;
        if (++e.pr >= u.np) {
            e.pr = 0;
            if (++e.h >= p->Hkv) {
                e.h = 0;
                do {
                    ++e.b;
                    if (e.b >= p->B || e.b > end.b) { e.b = end.b + 1; break; }
                    load();
                } while (u.np == 0);
            }
        }
    }
};

// ------------------------------------------------------------------ rows

// A thread's query row of a segment.
struct Row {
    int i, hq;             // token of the sequence's new ones, query head
    size_t at;             // element offset of the row in q and out
    bool ok;
};
__device__ __forceinline__ Row row_of(const ChunkParams& p, const Seg& s, int t, int r, int D) {
    const int tpq = p.tpq;
    Row o;
    const int it = (r * p.inv_g) >> 16, g = r - it * p.G;   // r / G: exact for r < 128, G <= 128
    o.ok = it < tpq && t * tpq + it < s.tokens;
    const int i = o.ok ? t * tpq + it : 0;
    o.i = s.i0 + i;
    o.hq = s.h * p.G + (o.ok ? g : 0);
    o.at = (size_t(s.row0 + i) * p.Hq + o.hq) * D;
    return o;
}
// What a row may see: the prefix and, of the new tokens, 0 .. i (a chunk) or its ancestors.
struct Sight {
    int end;               // chunks: first logical token it may not see
    uint64_t a0, a1;       // trees
};
__device__ __forceinline__ Sight sight_of(const ChunkParams& p, const Seg& s, const Row& r) {
    Sight v{0, 0, 0};
    if (!r.ok) return v;
    if (p.offsets) {
        v.end = s.S + r.i + 1;
    } else {
        const uint64_t* a = p.anc + (size_t(s.b) * p.N + r.i) * kAncWords;
        v.a0 = a[0];
        v.a1 = a[1];
    }
    return v;
}

// Whether the row sees the token at `pos`, below the segment's t1.
__device__ __forceinline__ bool sees(const ChunkParams& p, const Seg& s, const Sight& v, int pos) {
    const int j = pos - s.S;
    return j < 0 || (p.offsets ? pos < v.end : ((j < 64 ? v.a0 >> j : v.a1 >> (j - 64)) & 1ull) != 0);
}

// A row's exact attention over the segment's visible tokens, by one warp on CUDA cores:
// (m, l) and O in lane-wise slices of D / 32 elements.  Nothing of a token that the row does
// not see is read.
template <int D, bool E4M3>
__device__ __noinline__ void slow_row(const ChunkParams& p, const Seg& s, const Row& r, const Sight& v, float (&o)[4],
                                      float& m_out, float& l_out) {
    constexpr int DS = D / 32;
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < DS; ++e) o[e] = 0.f;
    const int* ptab = p.page_table + size_t(s.b) * p.max_pages;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + r.at;
    for (int base = s.t0; base < s.t1; base += 32) {
        const int pos = base + lane;
        const bool ok = pos < s.t1 && sees(p, s, v, pos);
        long long slot = -1;                               // a page outside the pool holds zeros
        if (ok) {
            const int page = ptab[pos >> 4];
            if (page >= 0 && page < p.num_pool_pages) slot = (long long)page * kPage + (pos & 15);
        }
        float x = 0.f, vs = 1.f;
        if (slot >= 0) {
            if constexpr (E4M3) {
                const unsigned char* k = static_cast<const unsigned char*>(p.k) + (slot * p.Hkv + s.h) * D;
                for (int d = 0; d < D; d += 2) {
                    const uint32_t h2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(k + d));
                    const uint32_t q2 = *reinterpret_cast<const uint32_t*>(q + d);
                    float a, b;
                    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
                        : "=f"(a), "=f"(b) : "r"(h2));
                    x = fmaf(bf16_lo(q2), a, x);
                    x = fmaf(bf16_hi(q2), b, x);
                }
                const size_t sc = ((slot >> 4) * p.Hkv + s.h) * kPage + (slot & 15);
                x *= p.k_scales[sc];
                vs = p.v_scales[sc];
            } else {
                const uint16_t* k = static_cast<const uint16_t*>(p.k) + (slot * p.Hkv + s.h) * D;
                for (int d = 0; d < D; d += 2) {
                    const uint32_t k2 = *reinterpret_cast<const uint32_t*>(k + d);
                    const uint32_t q2 = *reinterpret_cast<const uint32_t*>(q + d);
                    x = fmaf(bf16_lo(q2), bf16_lo(k2), x);
                    x = fmaf(bf16_hi(q2), bf16_hi(k2), x);
                }
            }
        }
        x *= p.scale_log2;
        const float mt = warp_max(ok ? x : -INFINITY);
        const float mn = fmaxf(m, mt);
        const float alpha = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float pr = ok ? exp2f(x - (mn == -INFINITY ? 0.f : mn)) : 0.f;   // a score of -inf weighs 0
        l = l * alpha + warp_sum(pr);
        m = mn;
#pragma unroll
        for (int e = 0; e < DS; ++e) o[e] *= alpha;
        const unsigned who = __ballot_sync(0xffffffffu, slot >= 0);
        for (unsigned w = who; w; w &= w - 1) {
            const int t = __ffs(w) - 1;
            const long long st = __shfl_sync(0xffffffffu, slot, t);
            const float pt = __shfl_sync(0xffffffffu, pr, t), vt = __shfl_sync(0xffffffffu, vs, t);
            const size_t at = (st * p.Hkv + s.h) * D + lane * DS;
#pragma unroll
            for (int e = 0; e < DS; ++e) {
                float y;
                if constexpr (E4M3) {
                    const uint32_t h2 = e4m3x2_to_f16x2(static_cast<const unsigned char*>(p.v)[at + e]);
                    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(y) : "r"(h2));
                    y *= vt;
                } else {
                    y = bf16_to_f32(static_cast<const uint16_t*>(p.v)[at + e]);
                }
                o[e] = fmaf(pt, y, o[e]);
            }
        }
    }
    m_out = m;
    l_out = l;
}

// One warp's 32 rows of a cut unit: partial k of the unit is in slot 2 c0 + 1 (k = 0) or
// 2 (c0 + k).  M = max m_k, out = sum O_k 2^(m_k - M) / sum l_k 2^(m_k - M), the pieces in
// their order; a piece that gives the row no weight (no visible token, or only scores of -inf) has
// l = 0 and is left out, one whose weight rounds to 0 is not: a NaN that the row sees stays a NaN.
// `valid`: the lanes that hold rows.  O is read with the columns across the lanes.  Few pieces (a unit of many rows cut once or twice): a lane works out its own row's
// weights, then eight rows at a time (54 nodes x 4 heads over 736 tokens, three pieces: 32 us a call, 39 by the
// other way).  More: four rows at a time, their (m, l) with a piece per lane.
template <int D>
__device__ __noinline__ void join_pieces(const ChunkParams& p, int c0, int pieces, int t, int quarter, size_t my_at,
                                         unsigned valid) {
    constexpr int DS = D / 32, kR = 4;
    const int lane = threadIdx.x & 31;
    auto slot = [&](int k) { return (size_t(k == 0 ? 2 * c0 + 1 : 2 * (c0 + k)) * kNQ + t) * kM + quarter * 32; };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    auto store = [&](size_t at, const float (&x)[DS]) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at) + lane * (DS / 2);
        if constexpr (DS == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        else *dst = pack_bf16x2(x[0], x[1]);
    };
    if (pieces <= 4 && __popc(valid) > kR) {
        constexpr int kF = 8;
        float2 x[4];
        float M = -INFINITY, l = 0.f, w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = k < pieces && ((valid >> lane) & 1u) ? __ldcg(ml + slot(k) + lane) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) M = fmaxf(M, x[k].x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = x[k].x == -INFINITY ? (x[k].y == 0.f ? -1.f : 1.f) : ex2(x[k].x - M);
            if (w[k] >= 0.f) l += x[k].y * w[k];
        }
        const float inv = 1.f / l;
        for (unsigned left = valid; left;) {
            int row[kF];
            bool on[kF];
            float acc[kF][DS];
#pragma unroll
            for (int i = 0; i < kF; ++i) {
                on[i] = left != 0;
                row[i] = on[i] ? __ffs(left) - 1 : 0;
                left &= left - 1;
#pragma unroll
                for (int e = 0; e < DS; ++e) acc[i][e] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= pieces) break;
                const float* src = p.part_acc + slot(k) * D + lane * DS;
                float y[kF][DS];
#pragma unroll
                for (int i = 0; i < kF; ++i) {
                    if constexpr (DS == 4) {
                        const float4 z = on[i] ? __ldcg(reinterpret_cast<const float4*>(src + row[i] * D))
                                               : make_float4(0, 0, 0, 0);
                        y[i][0] = z.x; y[i][1] = z.y; y[i][2] = z.z; y[i][3] = z.w;
                    } else {
                        const float2 z = on[i] ? __ldcg(reinterpret_cast<const float2*>(src + row[i] * D)) : make_float2(0, 0);
                        y[i][0] = z.x; y[i][1] = z.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < kF; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, w[k], row[i]);
#pragma unroll
                    for (int e = 0; e < DS; ++e) acc[i][e] = wi < 0.f ? acc[i][e] : fmaf(y[i][e], wi, acc[i][e]);
                }
            }
#pragma unroll
            for (int i = 0; i < kF; ++i) {
                const float f = __shfl_sync(0xffffffffu, inv, row[i]);
                const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)my_at, row[i]);
#pragma unroll
                for (int e = 0; e < DS; ++e) acc[i][e] *= f;
                if (on[i]) store(at, acc[i]);
            }
        }
        return;
    }
    for (unsigned left = valid; left;) {
        int row[kR];
        bool on[kR];
        float acc[kR][DS], M[kR], l[kR], w[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            on[i] = left != 0;
            row[i] = on[i] ? __ffs(left) - 1 : 0;
            left &= left - 1;
            M[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < DS; ++e) acc[i][e] = 0.f;
        }
        float2 x[kR];
        auto fetch = [&](int k0) {                         // pieces k0 .. k0 + 31
            const int k = k0 + lane;
            const size_t s0 = slot(k < pieces ? k : 0);
#pragma unroll
            for (int i = 0; i < kR; ++i)
                x[i] = on[i] && k < pieces ? __ldcg(ml + s0 + row[i]) : make_float2(-INFINITY, 0.f);
        };
        for (int k0 = 0; k0 < pieces; k0 += 32) {
            fetch(k0);
#pragma unroll
            for (int i = 0; i < kR; ++i) M[i] = fmaxf(M[i], warp_max(x[i].x));
        }
        for (int k0 = 0; k0 < pieces; k0 += 32) {
            if (pieces > 32) fetch(k0);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                w[i] = x[i].x == -INFINITY ? (x[i].y == 0.f ? -1.f : 1.f) : ex2(x[i].x - M[i]);
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
                        const float4 z = on[i] ? __ldcg(reinterpret_cast<const float4*>(src + row[i] * D))
                                               : make_float4(0, 0, 0, 0);
                        y[i][0] = z.x; y[i][1] = z.y; y[i][2] = z.z; y[i][3] = z.w;
                    } else {
                        const float2 z = on[i] ? __ldcg(reinterpret_cast<const float2*>(src + row[i] * D)) : make_float2(0, 0);
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
        for (int i = 0; i < kR; ++i) {
            const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)my_at, row[i]);
            const float f = 1.f / l[i];
#pragma unroll
            for (int e = 0; e < DS; ++e) acc[i][e] *= f;
            if (on[i]) store(at, acc[i]);
        }
    }
}

// What a run of tokens holds that is not finite, in the lane's D / 32 columns (a bit each).
struct Spoil {
    uint32_t nan, inf;     // of V, in tokens that the row sees
    uint32_t hidden;       // of V as the MMA reads it, in tokens that it does not see
    bool key;              // a NaN in K of a token that it sees
};
// Adds tokens from .. to - 1 of the segment's sequence, by one warp; pages outside the pool hold zeros.
template <int D, bool E4M3>
__device__ __forceinline__ void look(const ChunkParams& p, const Seg& s, const Sight& v, int from, int to, Spoil& f) {
    constexpr int DS = D / 32;
    using Code = std::conditional_t<E4M3, unsigned char, uint16_t>;
    using Word = std::conditional_t<DS * sizeof(Code) == 8, unsigned long long,
                                    std::conditional_t<DS * sizeof(Code) == 4, uint32_t, uint16_t>>;
    const int lane = threadIdx.x & 31;
    const int* ptab = p.page_table + size_t(s.b) * p.max_pages;
    for (int q0 = from & ~(kPage - 1); q0 < to; q0 += kPage) {
        const int page = __ldg(ptab + q0 / kPage);
        if (page < 0 || page >= p.num_pool_pages) continue;
#pragma unroll 8
        for (int i = 0; i < kPage; ++i) {
            const int pos = q0 + i;
            const size_t at = ((size_t(page) * kPage + i) * p.Hkv + s.h) * D + lane * DS;
            uint32_t nan[2] = {0, 0}, inf[2] = {0, 0};     // K, V
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const Word word = __ldg(reinterpret_cast<const Word*>(static_cast<const Code*>(kv ? p.v : p.k) + at));
#pragma unroll
                for (int e = 0; e < DS; ++e) {
                    const uint32_t x = uint32_t(word >> (8 * int(sizeof(Code)) * e)) & (E4M3 ? 0x7fu : 0x7fffu);
                    nan[kv] |= uint32_t(E4M3 ? x == 0x7fu : x > 0x7f80u) << e;
                    inf[kv] |= uint32_t(!E4M3 && x == 0x7f80u) << e;
                }
            }
            const bool in = pos >= from && pos < to, seen = in && sees(p, s, v, pos);
            if (in && !seen) f.hidden |= nan[1] | inf[1];
            if constexpr (E4M3) {                          // the scale of a token that a row does not see never counts
                const size_t sc = (size_t(page) * p.Hkv + s.h) * kPage + i;
                const float ks = __ldg(p.k_scales + sc), vs = __ldg(p.v_scales + sc);
                if (ks != ks) nan[0] = 1;
                if (vs != vs) nan[1] = ~0u;
                else if (isinf(vs)) inf[1] = ~0u;
            }
            if (seen) {
                f.nan |= nan[1];
                f.inf |= inf[1];
                f.key |= nan[0] != 0;
            }
        }
    }
}

// The last of the warps that hold these rows of a cut unit joins its pieces.
template <int D>
__device__ __forceinline__ void join_unit(const ChunkParams& p, const Cut& cut, const Seg& s, int me, int t, int quarter,
                                          const Row& ro) {
    int c0, pieces;
    if (cut.m) {
        c0 = me / cut.m * cut.m;
        pieces = unit_pieces(s.n, s.tokens * p.G, cut.m);
    } else {
        const SeqUnits u = seq_units(p, seq_rows(p, s.b));
        const long long ub = cut.before(s.b) + s.h * div_pos(cut.before(s.b + 1) - cut.before(s.b), cut.Hkv) +
                             u.tiles_before(s.pr) + (long long)cut.k * s.pr + cut.k;
        c0 = cut.owner(ub);
        pieces = cut.owner(ub + s.n - 1) - c0 + 1;
    }
    __threadfence();
    __syncwarp();
    int n = 0;
    if ((threadIdx.x & 31) == 0) n = atomicAdd(p.counters + c0 * 8 + t * 4 + quarter, 1);
    n = __shfl_sync(0xffffffffu, n, 0);
    if (n == pieces - 1) {
        __threadfence();
        join_pieces<D>(p, c0, pieces, t, quarter, ro.at, __ballot_sync(0xffffffffu, ro.ok));
    }
}

// One warp's rows that came out non-finite, segment by segment of the CTA's range, recomputed and
// stored behind what the epilogue stored; then the joins that waited for them: those of the
// range's last (pending & 2) and first (pending & 1) piece.  `sm`: the CTA's shared memory.
//
// A row stands as it is where it sees what spoils it: a NaN in K spoils the whole row; a NaN in
// a column of V, or an infinity there and nothing hidden in that column, spoils that column and
// no other.  (An infinity at a weight below 2^-126 gives NaN.)  So what a row may not see counts
// only among the unit's own tokens and those that share a page with its last one, and one NaN in a
// prompt does not have all rows behind it recomputed (64 heads, 512 new tokens over 3000, a NaN in
// token 19: 84 ms if every row is recomputed, 1.8 ms this way, 0.16 ms without the NaN; 32 heads, a
// prompt of 32768 tokens, a NaN in token 5: 87 ms, 6.0 without).
template <int D, bool E4M3>
__device__ __noinline__ void redo_rows(const ChunkParams& p, const unsigned char* sm, uint32_t pending) {
    using C = Cfg<D, E4M3>;
    constexpr int DS = D / 32;
    const int lane = threadIdx.x & 31, t = threadIdx.x >> 7, quarter = (threadIdx.x >> 5) & 3, me = blockIdx.x;
    const Cut cut = cut_of(p, reinterpret_cast<const long long*>(sm + C::kOffTiles),
                           reinterpret_cast<const int*>(sm + C::kOffUnits),
                           *reinterpret_cast<const int*>(sm + C::kOffMisc + 8));
    const End* ends = reinterpret_cast<const End*>(sm + C::kOffEnds);
    __syncwarp();                                          // the lanes' stores come before what is read and stored here
    Walk walk;
    walk.start(p, ends[0], ends[1], *reinterpret_cast<const SeqRows*>(ends + 2));
    Seg s;
    Spoil before{};                                        // tokens `from` .. `upto` - 1 of kv head h of sequence b, which
    int b = -1, h = -1, from = 0, upto = 0;                // every row of the units at hand sees
    while (walk.next(s)) {
        if (t >= s.nq) continue;
        const Row ro = row_of(p, s, t, lane * 4 + quarter, D);
        const unsigned valid = __ballot_sync(0xffffffffu, ro.ok);
        if (!valid) continue;
        const bool whole = s.whole(), head = s.j0 == 0;
        const size_t prow = (size_t(2 * me + (head ? 1 : 0)) * kNQ + t) * kM + quarter * 32;
        for (unsigned w = valid; w; w &= w - 1) {
            const int x = __ffs(w) - 1;
            const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)ro.at, x);
            float o[4];
#pragma unroll
            for (int e = 0; e < DS; ++e) {
                const int d = lane * DS + e;
                o[e] = whole ? bf16_to_f32(__ldcg(static_cast<const uint16_t*>(p.out) + at + d))
                             : __ldcg(p.part_acc + (prow + x) * D + d);
            }
            uint32_t odd = 0;
#pragma unroll
            for (int e = 0; e < DS; ++e) odd |= uint32_t(!(o[e] * 0.f == 0.f)) << e;
            if (!__any_sync(0xffffffffu, odd != 0)) continue;
            const Row rx = row_of(p, s, t, x * 4 + quarter, D);
            const Sight v = sight_of(p, s, rx);
            const int own = min(s.t1, s.S + (p.offsets ? s.i0 : 0));      // the first token that a row may not see
            if (s.b != b || s.h != h || s.t0 != from) {
                before = Spoil{};
                b = s.b;
                h = s.h;
                from = upto = s.t0;
            }
            look<D, E4M3>(p, s, v, upto, own, before);
            upto = max(upto, own);
            Spoil f = before;
            look<D, E4M3>(p, s, v, max(s.t0, own), min(s.L, (s.t1 + kPage - 1) & ~(kPage - 1)), f);
            if (__any_sync(0xffffffffu, f.key) || !__any_sync(0xffffffffu, (odd & ~(f.nan | (f.inf & ~f.hidden))) != 0)) continue;
            float m, l;
            slow_row<D, E4M3>(p, s, rx, v, o, m, l);
#pragma unroll
            for (int e = 0; e < DS; ++e) {
                const int d = lane * DS + e;
                if (whole) static_cast<uint16_t*>(p.out)[at + d] = f32_to_bf16_rne(o[e] / l);
                else __stcg(p.part_acc + (prow + x) * D + d, o[e]);
            }
            if (!whole && lane == 0) __stcg(reinterpret_cast<float2*>(p.part_ml) + prow + x, make_float2(m, l));
        }
        if (!whole && (pending & (head ? 2u : 1u))) join_unit<D>(p, cut, s, me, t, quarter, ro);
    }
}

// (d0, d1) = (a0 b0 + c, a1 b1 + c) and (d0, d1) *= (b0, b1), one packed instruction each
__device__ __forceinline__ void fma_pairs(float& d0, float& d1, float a0, float a1, float b0, float b1, float c) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %6};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c));
}
__device__ __forceinline__ void mul_pairs(float& d0, float& d1, float b0, float b1) {
    asm("{\n\t.reg .b64 rb, rd;\n\tmov.b64 rd, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
        "mul.rn.f32x2 rd, rd, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "+f"(d0), "+f"(d1) : "f"(b0), "f"(b1));
}

// ------------------------------------------------------------------ e4m3 -> operands

// Two e4m3 codes -> packed bf16, exact: every e4m3 value, NaN among them, is a bf16 value.
// (Moving the bits with prmt, shifts, masks and a multiplication by 2^120 measured slower,
// 599 us against 585 at 32 x 64 rows x 8 heads over 8256 tokens, before its NaN codes.)
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t c) {
    const uint32_t h = e4m3x2_to_f16x2(uint16_t(c));
    uint32_t r;
    asm("{\n\t.reg .f16 lo, hi;\n\t.reg .f32 a, b;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 a, lo;\n\tcvt.f32.f16 b, hi;\n\t"
        "cvt.rn.bf16x2.f32 %0, b, a;\n\t}"
        : "=r"(r) : "r"(h));
    return r;
}
// 16 codes -> 16 bf16
__device__ __forceinline__ void codes_to_bf16(const uint4& in, uint4& a, uint4& b) {
    a = make_uint4(e4m3x2_to_bf16x2(in.x), e4m3x2_to_bf16x2(in.x >> 16), e4m3x2_to_bf16x2(in.y),
                   e4m3x2_to_bf16x2(in.y >> 16));
    b = make_uint4(e4m3x2_to_bf16x2(in.z), e4m3x2_to_bf16x2(in.z >> 16), e4m3x2_to_bf16x2(in.w),
                   e4m3x2_to_bf16x2(in.w >> 16));
}

// 64 contiguous bytes (a page's scales of one head) into shared memory
__device__ __forceinline__ void bulk_load_64(void* dst, const void* src, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 64, [%2];" ::"r"(
                     smem_u32(dst)), "l"(src), "r"(smem_u32(bar))
                 : "memory");
}

// One warp streams the codes and scales of K (or V) of a segment into rings of kRaw stages,
// a tile of 64 rows of D bytes and 64 floats per stage.  Lanes 0 .. 3 own a page each: a
// page that lies wholly in the sequence arrives by TMA, the partly filled last one is written
// by the warp, zeros behind the last token, and so is a bad page id (flagged) or a page
// behind the segment.  `g` counts tiles over the CTA's life.  False after a timeout or an
// abort.
template <int D>
__device__ __forceinline__ bool produce_codes(const ChunkParams& p, const CUtensorMap* map, const unsigned char* src,
                                              const float* scales, unsigned char* ring, float* sring, uint64_t* full,
                                              uint64_t* empty, const Seg& s, int& g, volatile uint32_t* abort_flag) {
    const int lane = threadIdx.x & 31;
    const int* ptab = p.page_table + size_t(s.b) * p.max_pages;
    auto fetch = [&](int bi) -> int {                      // page ids of 8 tiles, one warp-wide load
        const int pos = s.t0 + (8 * bi + lane / 4) * kBN + (lane % 4) * 16;
        return pos < s.t1 ? __ldg(ptab + (pos >> 4)) : -1;
    };
    int cur = fetch(0), nxt = fetch(1);
    for (int j = 0; j < s.ntiles; ++j, ++g) {
        const int st = g % kRaw;
        if (j > 0 && (j & 7) == 0) {
            cur = nxt;
            nxt = fetch(j / 8 + 1);
        }
        int page = __shfl_sync(0xffffffffu, cur, (j & 7) * 4 + (lane & 3));
        const int base = s.t0 + j * kBN, pos0 = base + (lane & 3) * 16;
        int kind = 0;                                      // 1: by TMA, 2: written here
        if (lane < 4) {
            kind = 2;
            if (pos0 < s.t1) {
                const bool ok = page >= 0 && page < p.num_pool_pages;
                if (!ok) atomicOr(p.status, TREESPEC_STATUS_BAD_PAGE);
                if (ok && pos0 + 16 <= s.L) kind = 1;
                if (!ok) page = -1;
            } else {
                page = -1;
            }
        }
        if (g >= kRaw && !mbar_wait_bounded(&empty[st], ((g / kRaw) - 1) & 1, p.wait_ns)) {
            *abort_flag = 1;
            atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
        }
        if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
        unsigned char* dst = ring + st * (kBN * D);
        float* sdst = sring + st * kBN;
        const unsigned manual = __ballot_sync(0xffffffffu, kind == 2);
        for (unsigned w = manual; w; w &= w - 1) {
            const int pg = __ffs(w) - 1;
            const int id = __shfl_sync(0xffffffffu, page, pg);
            const int q0 = base + pg * 16;
            for (int c = lane; c < D; c += 32) {
                const int rr = c / (D / 16), cc = c % (D / 16);
                uint4 val = make_uint4(0, 0, 0, 0);
                if (id >= 0 && q0 + rr < s.t1)
                    val = __ldg(reinterpret_cast<const uint4*>(src + ((size_t(id) * kPage + rr) * p.Hkv + s.h) * D) + cc);
                *reinterpret_cast<uint4*>(dst + (pg * 16 + rr) * D + cc * 16) = val;
            }
            if (lane < 16)
                sdst[pg * 16 + lane] =
                    id >= 0 && q0 + lane < s.t1 ? __ldg(scales + (size_t(id) * p.Hkv + s.h) * kPage + lane) : 0.f;
        }
        // the writes above reach the converting warps through the arrival below; the next use of
        // the stage by TMA comes after their own arrivals and needs the proxy fence
        if (manual) fence_proxy_async_smem();
        __syncwarp();
        const unsigned viatma = __ballot_sync(0xffffffffu, kind == 1);
        if (lane == 0) mbar_arrive_expect_tx(&full[st], uint32_t(__popc(viatma)) * (16u * D + 64u));
        __syncwarp();
        if (kind == 1) {
            tma_load_3d(dst + lane * 16 * D, map, 0, s.h, page * 16, &full[st]);
            bulk_load_64(sdst + lane * 16, scales + (size_t(page) * p.Hkv + s.h) * kPage, &full[st]);
        }
        __syncwarp();
    }
    return true;
}

// Wait for the phase with `parity` by polling, for the hand-offs inside the pipeline.  False
// after limit_ns, or when the CTA has been told to stop.  Reading the clock at every poll
// paces the polls: with one reading in 64 they take issue slots from the softmax (472 us
// against 463 for 2048 rows x 64 heads over 6000 .. 12000 tokens).
__device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* abort_flag) {
    if (mbar_test_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (mbar_test_wait(bar, parity)) return true;
        if (*abort_flag || global_ns() - t0 >= limit_ns) return false;
    }
}

// ------------------------------------------------------------------ the kernel

template <int D, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, E4M3>::kThreads, 1)
    chunk_tc_kernel(const ChunkParams p, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = Cfg<D, E4M3>;
    using Bars = typename C::Bars;
    constexpr int kNS = C::kNS;
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars* bars = reinterpret_cast<Bars*>(sm + C::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
    volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(sm + C::kOffMisc + 4);
    int* longest = reinterpret_cast<int*>(sm + C::kOffMisc + 8);       // KV tiles of the longest unit
    uint32_t* redo = reinterpret_cast<uint32_t*>(sm + C::kOffMisc + 12);   // 4 bits for each softmax warp: some row came
                                                           // out non-finite in the range's first (1) or last (2) piece, or
                                                           // in a whole unit (4)
    End* ends = reinterpret_cast<End*>(sm + C::kOffEnds);
    SeqRows* first_rows = reinterpret_cast<SeqRows*>(ends + 2);
    long long* tiles_s = reinterpret_cast<long long*>(sm + C::kOffTiles);
    int* units_s = reinterpret_cast<int*>(sm + C::kOffUnits);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(sm) & 1023u) {                            // never expected; refuse rather than misread tiles
        grid_dep_wait();
        if (tid == 0) atomicOr(p.status, TREESPEC_STATUS_INTERNAL);
        return;
    }
    // barriers and tensor memory, while other warps look at the lengths
    if (warp == kWarpMma) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    if (warp == kWarpMma + 1 && lane == 0) {
        for (int s = 0; s < kNS; ++s) {
            mbar_init(&bars->k_full[s], E4M3 ? 64 : 1);
            mbar_init(&bars->k_empty[s], kNQ);
            mbar_init(&bars->v_full[s], E4M3 ? 64 : 1);
            mbar_init(&bars->v_empty[s], kNQ);
        }
        for (int t = 0; t < kNQ; ++t) {
            mbar_init(&bars->q_full[t], kM);
            for (int bf = 0; bf < 2; ++bf) {
                mbar_init(&bars->s_full[t][bf], 1);
                mbar_init(&bars->p_full[t][bf], kM);
                mbar_init(&bars->pv_done[t][bf], 1);
            }
            mbar_init(&bars->o_full[t], 1);
            mbar_init(&bars->o_free[t], kM);
            mbar_init(&bars->drain[t], 1);
        }
        if (E4M3) {
            for (int s = 0; s < kRaw; ++s) {
                mbar_init(&bars->rk_full[s], 1);
                mbar_init(&bars->rk_empty[s], 64);
                mbar_init(&bars->rv_full[s], 1);
                mbar_init(&bars->rv_empty[s], 64);
            }
            for (int s = 0; s < kScaleRing; ++s) {
                mbar_init(&bars->sck_full[s], kBN);
                mbar_init(&bars->scv_full[s], kBN);
            }
        }
        *abort_flag = 0;
        *longest = 0;
        *redo = 0;
        fence_mbar_init();
    }
    grid_dep_wait();                                       // trees: the prologue's results

    // ---- the sequences' tiles and units, and this CTA's range
    {
        long long* wt = reinterpret_cast<long long*>(sm + C::kOffWarp);   // [16 warps] {tiles, units, rows}
        const int per = (p.B + C::kThreads - 1) / C::kThreads;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        long long nt = 0;
        int nu = 0, top = 0, rows_lo = 0, rows_hi = 0;     // rows in 16-bit halves: sums of 96 sequences fit
        bool bad = false;
        for (int b = b0; b < b1; ++b) {
            const SeqRows r = seq_rows(p, b);
            const SeqUnits u = seq_units(p, r);
            bad |= !seq_ok(p, b);
            rows_lo += r.n & 0xffff;
            rows_hi += r.n >> 16;
            tiles_s[b] = nt;                               // relative to the thread's first
            units_s[b] = nu;
            nt += u.np == 1 ? u.tiles(0) : u.tiles_before(u.np);
            nu += u.np;
            if (u.np) top = max(top, u.tiles(u.np - 1));
        }
        if (bad && blockIdx.x == 0) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
        long long it = nt;
        int iu = nu;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, it, o);
            const int y = __shfl_up_sync(0xffffffffu, iu, o);
            if (lane >= o) {
                it += x;
                iu += y;
            }
        }
        if (lane == 31) {
            wt[3 * warp] = it;
            wt[3 * warp + 1] = iu;
        }
        const long long warp_rows = (long long)__reduce_add_sync(0xffffffffu, rows_hi) * 65536 +
                                    __reduce_add_sync(0xffffffffu, rows_lo);
        if (lane == 0) wt[3 * warp + 2] = warp_rows;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) atomicMax(longest, top);
        long long bt = it - nt, bu = iu - nu, rows = warp_rows;   // a warp's units fit 31 bits
        for (int w = 0; w < warp; ++w) {
            bt += wt[3 * w];
            bu += wt[3 * w + 1];
            rows += wt[3 * w + 2];
        }
        for (int b = b0; b < b1; ++b) {
            tiles_s[b] += bt;
            units_s[b] += int(bu);
        }
        if (tid == C::kThreads - 1) {
            // Sequences that share rows (offsets out of order) may have more units than 32 bits count:
            // no row is computed then
            tiles_s[p.B] = rows > p.T ? 0 : bt + nt;
            units_s[p.B] = rows > p.T ? 0 : int(bu + nu);
        }
        __syncthreads();
    }
    const Cut cut = cut_of(p, tiles_s, units_s, *longest);
    // rows without a token (a padded tree's, and those of an invalid sequence) are zeros
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const SeqRows r = seq_rows(p, b);
        const int from = r.S < 0 ? 0 : r.live;
        const size_t words = size_t(r.n - from) * p.Hq * (D / 8);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + size_t(r.row0 + from) * p.Hq * D);
        for (size_t e = tid; e < words; e += C::kThreads) dst[e] = make_uint4(0, 0, 0, 0);
    }
    const int me = blockIdx.x;
    if (cut.total == 0 || me >= cut.parts) {               // nothing to compute
        __syncthreads();
        if (warp == kWarpMma) tmem_dealloc(*tmem_slot, kTmemCols);
        return;
    }
    if (warp < 2) {                                        // warp 0 the begin, warp 1 the end of the range
        const int c = me + warp;
        End e;
        if (cut.m) {
            e = unit_at(p, cut, me / cut.m);
            const SeqUnits u = seq_units(p, seq_rows(p, e.b));
            const int n = u.tiles(e.pr);
            const int pieces = unit_pieces(n, min(u.tpu, u.live - e.pr * u.tpu) * p.G, cut.m), k = me % cut.m + warp;
            e.j = k > pieces ? n : int((long long)n * k / pieces);   // beyond the last piece: nothing
        } else if (c >= cut.parts) {
            e = End{p.B, 0, 0, 0};
        } else {
            e = locate(p, cut, cut.bound(c));
            const int n = seq_units(p, seq_rows(p, e.b)).tiles(e.pr);
            // Short units stay whole: the cut moves to the nearer end of one, and both neighbours
            // see it there (160 units of 1 or 2 tiles: 43 us cut, 27 whole; with units of up to 10
            // tiles kept whole the ranges of ragged prompts get uneven, 388 us against 380)
            if (n <= kWholeTiles) e.j = 2 * e.j < n ? 0 : n;
        }
        if (lane == 0) {
            ends[warp] = e;
            if (warp == 0) *first_rows = seq_rows(p, e.b);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const uint32_t sbase = smem_u32(sm);
    Walk walk;
    walk.start(p, ends[0], ends[1], *first_rows);
    Seg sg;

    if (E4M3 && warp >= kWarpConv) {
        // ------------------------------------------------------------ e4m3 -> bf16 operands
        // Two warps convert K, two V.  Thread i of the 64 converts 16-byte word i % (D / 16) of rows
        // i / (D / 16) + (1024 / D) k, so that the lanes that read together cover whole rows.
        regs_lower<C::kRegsConv>();
        constexpr int WPR = D / 16;                        // words of a row
        constexpr int RPI = 64 / WPR;                      // rows at a time
        const bool is_v = warp >= kWarpConv + 2;
        const int i = tid & 63, word = i % WPR, row0 = (i / WPR) ^ (word >> 2);
        // element 16 word: panel word / 4, 16-byte chunks 2 (word % 4) and the next of its row.  The
        // lanes of the second panel work on the neighbouring row, whose swizzle sends them to the
        // banks that the first panel's lanes leave free
        const int ch = (word & 3) * 2;
        const unsigned char* raw = sm + C::kOffRaw + (is_v ? kRaw * C::kRawTile : 0) + row0 * D + word * 16;
        const float* rsc = reinterpret_cast<const float*>(sm + C::kOffRawScale) + (is_v ? kRaw * kBN : 0) + i;
        float* scales = reinterpret_cast<float*>(sm + C::kOffScale) + (is_v ? kBN : 0) + i;
        unsigned char* ring = sm + (is_v ? C::kOffV : C::kOffK) + (word >> 2) * C::kPanel;
        uint64_t* raw_full = is_v ? bars->rv_full : bars->rk_full;
        uint64_t* raw_empty = is_v ? bars->rv_empty : bars->rk_empty;
        uint64_t* full = is_v ? bars->v_full : bars->k_full;
        uint64_t* empty = is_v ? bars->v_empty : bars->k_empty;
        uint64_t* sc_full = is_v ? bars->scv_full : bars->sck_full;
        const float sc_mul = is_v ? 1.f : p.scale_log2;
        bool ok = true;
        int g = 0;
        while (ok && walk.next(sg)) {
            for (int j = 0; j < sg.ntiles; ++j, ++g) {
                const int st = g % kNS, rs = g % kRaw;
                ok = poll(&raw_full[rs], (g / kRaw) & 1, p.wait_ns, abort_flag) &&
                     (g < kNS || poll(&empty[st], ((g / kNS) - 1) & 1, p.wait_ns, abort_flag)) && !*abort_flag;
                if (!ok) break;
                // The scale slot's last readers worked four tiles ago: K's stage was handed back by
                // S of tile g - 2, which waited for P V of tile g - 4 (V's by P V of tile g - 2)
                scales[(g % kScaleRing) * 2 * kBN] = rsc[rs * kBN] * sc_mul;
                mbar_arrive(&sc_full[g % kScaleRing]);
                const unsigned char* src = raw + rs * C::kRawTile;
                unsigned char* dst = ring + st * C::kTile;
#pragma unroll 2
                for (int k = 0; k < kBN / RPI; ++k) {
                    const uint4 in = *reinterpret_cast<const uint4*>(src + RPI * k * D);
                    uint4 a, b;
                    codes_to_bf16(in, a, b);
                    const int r = row0 + RPI * k;
                    *reinterpret_cast<uint4*>(dst + sw128_offset(r, ch)) = a;
                    *reinterpret_cast<uint4*>(dst + sw128_offset(r, ch + 1)) = b;
                }
                mbar_arrive(&raw_empty[rs]);
                fence_proxy_async_smem();
                mbar_arrive(&full[st]);
            }
        }
        if (!ok) {
            *abort_flag = 1;
            atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
        }
    } else if (warp >= kWarpK) {
        regs_lower<C::kRegsOther>();
        if (warp == kWarpK || warp == kWarpV) {
            if constexpr (!E4M3) {
                // -------------------------------------------------------- TMA producers
                const bool is_v = warp == kWarpV;
                tcparts::ProducerArgs a;
                a.map = is_v ? &tmv : &tmk;
                a.src = static_cast<const uint16_t*>(is_v ? p.v : p.k);
                a.ring = sm + (is_v ? C::kOffV : C::kOffK);
                a.full = is_v ? bars->v_full : bars->k_full;
                a.empty = is_v ? bars->v_empty : bars->k_empty;
                a.nst = kNS;
                a.stage_bytes = C::kTile;
                a.panel_bytes = C::kPanel;
                a.pg0 = 0;
                a.npg = kBN / 16;
                a.dp0 = 0;
                a.ndp = C::kNP;
                int armed = 0;
                while (walk.next(sg))
                    if (!tcparts::produce_pages<kBN, D>(p, a, sg.b, sg.h, sg.t0, sg.t1, sg.L, sg.ntiles, armed, abort_flag))
                        break;
                tcparts::drain_copies(a, armed);
            } else {
                const bool is_v = warp == kWarpV;
                uint64_t* full = is_v ? bars->rv_full : bars->rk_full;
                int armed = 0;
                while (walk.next(sg))
                    if (!produce_codes<D>(p, is_v ? &tmv : &tmk, static_cast<const unsigned char*>(is_v ? p.v : p.k),
                                          is_v ? p.v_scales : p.k_scales, sm + C::kOffRaw + (is_v ? kRaw * C::kRawTile : 0),
                                          reinterpret_cast<float*>(sm + C::kOffRawScale) + (is_v ? kRaw * kBN : 0), full,
                                          is_v ? bars->rv_empty : bars->rk_empty, sg, armed, abort_flag))
                        break;
                tcparts::ProducerArgs a{};                 // only what the drain looks at
                a.full = full;
                a.nst = kRaw;
                tcparts::drain_copies(a, armed);
            }
        } else {
            // ------------------------------------------------------------ MMA issuers
            // Warp 10 + t issues every MMA of tile t; the whole warp runs the loop and one elected lane
            // issues (a loop run by one lane alone measured 590 us for 460).  g counts the KV tiles over the CTA's life (ring stages), a those that this
            // query tile takes part in (S buffers), k its segments (Q, O).  A tile that sits a
            // segment out only hands the stages back.
            const int t = warp - kWarpMma;
            auto ready = [&](uint64_t* x, uint32_t px) -> bool {   // poll() of the whole warp
                const uint64_t t0 = global_ns();
                for (;;) {
                    if (__all_sync(0xffffffffu, mbar_test_wait(x, px))) return true;
                    if (__any_sync(0xffffffffu, *abort_flag || global_ns() - t0 >= p.wait_ns)) return false;
                }
            };
            constexpr uint32_t kIdS = idesc_bf16_f32(128, kBN, false);
            constexpr uint32_t kIdO = idesc_bf16_f32(128, D, true);
            const uint32_t dS = tbase + kColS + uint32_t(t) * 128u;
            const uint32_t dO = tbase + kColO + uint32_t(t) * 128u;
            const uint64_t dq = smem_desc(sbase + C::kOffQ + t * C::kQTile, 16, 1024);
            const uint64_t dk = smem_desc(sbase + C::kOffK, 16, 1024);
            const uint64_t dv = smem_desc(sbase + C::kOffV, C::kPanel, 1024);
            bool ok = true;
            int g = 0, a = 0, k = 0;
            while (ok && walk.next(sg)) {
                const int ntiles = sg.ntiles;
                if (t >= sg.nq) {
                    for (int j = 0; ok && j < ntiles; ++j) {
                        const int st = (g + j) % kNS;
                        const uint32_t ph = ((g + j) / kNS) & 1;
                        ok = ready(&bars->k_full[st], ph);
                        if (ok && lane == 0) mbar_arrive(&bars->k_empty[st]);
                        ok = ok && ready(&bars->v_full[st], ph);
                        if (ok && lane == 0) mbar_arrive(&bars->v_empty[st]);
                    }
                    g += ntiles;
                    continue;
                }
                ok = ready(&bars->q_full[t], k & 1);
                for (int j = 0; ok && j <= ntiles; ++j) {
                    if (j < ntiles) {
                        // S_t = Q_t K^T, once K has landed and the P V that read this buffer is done
                        const int st = (g + j) % kNS, aj = a + j, bf = aj & 1;
                        ok = ready(&bars->k_full[st], ((g + j) / kNS) & 1) &&
                             (aj < 2 || ready(&bars->pv_done[t][bf], ((aj >> 1) - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t kb = dk + uint64_t((st * C::kTile) >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t qoff = uint64_t(((kk >> 2) * C::kQPanel + (kk & 3) * 32) >> 4);
                                const uint64_t koff = uint64_t(((kk >> 2) * C::kPanel + (kk & 3) * 32) >> 4);
                                mma_bf16_ss(dS + bf * 64u, dq + qoff, kb + koff, kIdS, kk > 0);
                            }
                            mma_commit(&bars->s_full[t][bf]);
                            mma_commit(&bars->k_empty[st]);
                        }
                        __syncwarp();
                    }
                    if (j > 0) {
                        // O_t += P_t V; a segment's first one overwrites O, once the last segment's O is read
                        const int jp = j - 1, ap = a + jp, st = (g + jp) % kNS, bf = ap & 1;
                        ok = ready(&bars->p_full[t][bf], (ap >> 1) & 1) && ready(&bars->v_full[st], ((g + jp) / kNS) & 1) &&
                             (jp > 0 || k == 0 || ready(&bars->o_free[t], (k - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vb = dv + uint64_t((st * C::kTile) >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < kBN / 16; ++kk)
                                mma_bf16_ts(dO, dS + bf * 64u + kk * 8, vb + uint64_t((kk * 2048) >> 4), kIdO,
                                            (jp > 0 || kk > 0));
                            mma_commit(&bars->pv_done[t][bf]);
                            mma_commit(&bars->v_empty[st]);
                            if (jp == ntiles - 1) mma_commit(&bars->o_full[t]);
                        }
                        __syncwarp();
                    }
                }
                g += ntiles;
                a += ntiles;
                ++k;
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
            }
            if (elect_one()) mma_commit(&bars->drain[t]);  // the pipe completes MMAs in issue order
            __syncwarp();
            mbar_wait_bounded(&bars->drain[t], 0, kDefaultWaitNs);
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------- softmax warps
        regs_raise<C::kRegsSoftmax>();
        const int t = warp >> 2, quarter = warp & 3;
        const int tlane = quarter * 32 + lane;             // TMEM lane, and row of Q's image
        const int r = lane * 4 + quarter;                  // row of the tile
        const uint32_t tl = tbase + (uint32_t(quarter * 32) << 16);
        const uint32_t scol0 = tl + kColS + uint32_t(t) * 128u;
        const uint32_t ocol = tl + kColO + uint32_t(t) * 128u;
        const float sc = p.scale_log2;
        bool alive = true;
        uint32_t v[kBN];
        // the next segment this tile takes part in; *skipped counts the KV tiles passed over
        auto next_seg = [&](Seg& s, int& skipped) -> bool {
            skipped = 0;
            while (walk.next(s)) {
                if (t < s.nq) return true;
                skipped += s.ntiles;
            }
            return false;
        };
        auto issue_q = [&](const Seg& s) {
            const Row ro = row_of(p, s, t, r, D);
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + ro.at);
            unsigned char* qt = sm + C::kOffQ + t * C::kQTile;
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch)
                cp_async_16_zfill(qt + (ch >> 3) * C::kQPanel + sw128_offset(tlane, ch & 7), ro.ok ? src + ch : p.q,
                                  ro.ok ? 16 : 0);
        };
        auto finish_q = [&]() {
            cp_async_wait_all_groups();
            fence_proxy_async_smem();
            mbar_arrive(&bars->q_full[t]);
        };
        Seg s, nxt;
        int skip, g = 0, a = 0, k = 0;                     // as the MMA issuer counts them
        bool have = next_seg(s, skip);
        g += skip;
        if (have) {
            issue_q(s);
            finish_q();
        }
        while (have) {
            const Row ro = row_of(p, s, t, r, D);
            const Sight si = sight_of(p, s, ro);
            const bool warp_rows = __any_sync(0xffffffffu, ro.ok);
            float m_used = -INFINITY, l = 0.f;
            bool more = false;
            int skip2 = 0;
            for (int j = 0; j < s.ntiles; ++j) {
                const int aj = a + j, bf = aj & 1;
                const uint32_t scol = scol0 + bf * 64u;
                const int base = s.t0 + j * kBN;
                uint32_t mw[2];
                if (p.offsets) {
                    const int nv = min(min(si.end, s.t1) - base, kBN);    // visible columns: the first nv
                    mw[0] = nv >= 32 ? 0xffffffffu : nv <= 0 ? 0u : (1u << nv) - 1u;
                    mw[1] = nv >= 64 ? 0xffffffffu : nv <= 32 ? 0u : (1u << (nv - 32)) - 1u;
                } else {
                    tcparts::tile_mask<kBN>(mw, base, s.S, s.t1, si.a0, si.a1, ro.ok);
                }
                const bool full = __all_sync(0xffffffffu, (mw[0] & mw[1]) == 0xffffffffu || !ro.ok);
                if (!poll(&bars->s_full[t][bf], (aj >> 1) & 1, p.wait_ns, abort_flag)) { alive = false; break; }
                tc_fence_after();
                if constexpr (E4M3) {
                    // Only behind S: a parity tells a slot's use from the one before it, not from
                    // older ones, and a tile that sat a segment out has passed over many.  S of tile
                    // g comes after K of g and V of g - 2 were converted, so the slot's use before
                    // this one, tile g - 4, is complete by now
                    const int ss = (g + j) % kScaleRing;
                    const uint32_t ph = ((g + j) / kScaleRing) & 1;
                    if (!poll(&bars->sck_full[ss], ph, p.wait_ns, abort_flag) ||
                        !poll(&bars->scv_full[ss], ph, p.wait_ns, abort_flag)) {
                        alive = false;
                        break;
                    }
                }
                if (j == s.ntiles - 1) {                   // Q is read no more: the next segment's may come
                    more = next_seg(nxt, skip2);
                    if (more) issue_q(nxt);
                }
                bool resc = false;
                float alpha = 1.f, ts;
                if (warp_rows) {
                    auto load_s = [&]() {
#pragma unroll
                        for (int c = 0; c < kBN / 32; ++c) tmem_ld32(scol + c * 32, v + c * 32);
                        tmem_wait_ld();
                    };
                    load_s();
                    if constexpr (!E4M3) {
                        if (__all_sync(0xffffffffu, tcparts::softmax_tile_fast<kBN>(v, mw, full, sc, m_used, ts))) {
                            l += ts;
                        } else {
                            load_s();
                            tcparts::softmax_tile<kBN>(v, mw, full, sc, m_used, l, resc, alpha);
                        }
                    } else {
                        const float* scl = reinterpret_cast<const float*>(sm + C::kOffScale) +
                                           ((g + j) % kScaleRing) * 2 * kBN;
                        // P = 2^(s ks - m), P vs leaves as bf16 (its one rounding); the sum is over P.
                        // Masked columns are replaced after the products: a scale that the row does not
                        // see may hold anything.
                        auto columns = [&](auto masked, float m, float& sum) {
                            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
                            for (int b = 0; b < kBN; b += 16) {    // 16 columns step by step: their chains overlap
                                float x[16], y[16];
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const float4 ks = reinterpret_cast<const float4*>(scl + b)[c];
                                    y[4 * c] = ks.x; y[4 * c + 1] = ks.y; y[4 * c + 2] = ks.z; y[4 * c + 3] = ks.w;
                                }
#pragma unroll
                                for (int c = 0; c < 16; c += 2)
                                    fma_pairs(x[c], x[c + 1], __uint_as_float(v[b + c]), __uint_as_float(v[b + c + 1]), y[c],
                                              y[c + 1], -m);
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const float4 vs = reinterpret_cast<const float4*>(scl + kBN + b)[c];
                                    y[4 * c] = vs.x; y[4 * c + 1] = vs.y; y[4 * c + 2] = vs.z; y[4 * c + 3] = vs.w;
                                }
                                if constexpr (decltype(masked)::value) {
#pragma unroll
                                    for (int c = 0; c < 16; ++c) {
                                        const bool seen = (mw[b >> 5] >> ((b + c) & 31)) & 1u;
                                        x[c] = seen ? x[c] : -INFINITY;
                                        y[c] = seen ? y[c] : 0.f;
                                    }
                                }
#pragma unroll
                                for (int c = 0; c < 16; ++c) x[c] = ex2(x[c]);
#pragma unroll
                                for (int c = 0; c < 16; c += 4) {
                                    add_f32x2(a0, a1, x[c], x[c + 1]);
                                    add_f32x2(a2, a3, x[c + 2], x[c + 3]);
                                }
#pragma unroll
                                for (int c = 0; c < 16; c += 2) {
                                    mul_pairs(x[c], x[c + 1], y[c], y[c + 1]);
                                    v[(b + c) / 2] = pack_bf16x2(x[c], x[c + 1]);
                                }
                            }
                            sum = (a0 + a1) + (a2 + a3);
                        };
                        auto pass = [&](float m, float& sum) {
                            if (full) columns(std::false_type{}, m, sum);
                            else columns(std::true_type{}, m, sum);
                        };
                        bool fine;
                        if (m_used == -INFINITY) {
                            fine = (mw[0] | mw[1]) == 0u;
                            ts = 0.f;
                            if (fine) {
#pragma unroll
                                for (int c = 0; c < kBN / 2; ++c) v[c] = 0u;
                            }
                        } else {
                            pass(m_used, ts);
                            fine = ts <= 256.f;
                        }
                        if (__all_sync(0xffffffffu, fine)) {
                            l += ts;
                        } else {
                            load_s();
                            float mt = -INFINITY;
#pragma unroll
                            for (int c = 0; c < kBN; ++c)
                                if ((mw[c >> 5] >> (c & 31)) & 1u) mt = fmaxf(mt, __uint_as_float(v[c]) * scl[c]);
                            if (mt > m_used + 8.f) {
                                alpha = ex2(m_used - mt);
                                resc = m_used != -INFINITY;
                                l *= alpha;
                                m_used = mt;
                            }
                            pass(m_used == -INFINITY ? 0.f : m_used, ts);
                            l += ts;
                        }
                    }
                    tmem_st32(scol, v);                    // P over the first 32 columns of the buffer
                    tmem_wait_st();
                }
                if (__any_sync(0xffffffffu, resc)) {
                    // O may be rescaled once P V of the tile before is in it; never at a segment's first tile
                    if (!mbar_wait_bounded(&bars->pv_done[t][bf ^ 1], ((aj - 1) >> 1) & 1, p.wait_ns)) { alive = false; break; }
                    tc_fence_after();
                    const float f = resc ? alpha : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(ocol + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(ocol + c * 32, o);
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                mbar_arrive(&bars->p_full[t][bf]);
            }
            if (!alive) break;
            if (more) finish_q();
            if (!mbar_wait_bounded(&bars->o_full[t], k & 1, p.wait_ns)) { alive = false; break; }
            tc_fence_after();
            // ---- epilogue: the rows, or this piece of them
            const bool whole = s.whole();
            const bool head = s.j0 == 0;
            const size_t slot = size_t(2 * me + (head ? 1 : 0)) * kNQ + t;
            const size_t prow = slot * kM + tlane;
            float odd = 0.f;                               // stays 0 unless some element is not finite
            if (warp_rows && whole) {
                const float inv = 1.f / l;
                uint32_t w2[D / 2];                        // the row in bf16: O is free before it is stored
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(ocol + c * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float x = __uint_as_float(o[2 * e]), y = __uint_as_float(o[2 * e + 1]);
                        odd = fmaf(x, 0.f, odd);
                        odd = fmaf(y, 0.f, odd);
                        w2[c * 16 + e] = pack_bf16x2(x * inv, y * inv);
                    }
                }
                tc_fence_before();
                mbar_arrive(&bars->o_free[t]);
                if (ro.ok) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + ro.at);
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(w2[4 * e], w2[4 * e + 1], w2[4 * e + 2], w2[4 * e + 3]);
                }
            } else {
                if (warp_rows) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(ocol + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) odd = fmaf(__uint_as_float(o[e]), 0.f, odd);
                        if (ro.ok) {
                            float4* dst = reinterpret_cast<float4*>(p.part_acc + prow * D + c * 32);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                __stcg(dst + e, make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3])));
                        }
                    }
                    if (ro.ok) __stcg(reinterpret_cast<float2*>(p.part_ml) + prow, make_float2(m_used, l));
                }
                tc_fence_before();
                mbar_arrive(&bars->o_free[t]);
            }
            if (warp_rows) {
                if (__any_sync(0xffffffffu, ro.ok && !(odd == 0.f))) {
                    if (lane == 0) atomicOr(redo, (whole ? 4u : head ? 2u : 1u) << (4 * warp));
                } else if (!whole) {
                    join_unit<D>(p, cut, s, me, t, quarter, ro);
                }
            }
            g += s.ntiles + skip2;
            a += s.ntiles;
            ++k;
            have = more;
            s = nxt;
        }
        if (!alive) {
            cp_async_wait_all_groups();                    // the next segment's Q may be on its way
            *abort_flag = 1;
            atomicOr(p.status, TREESPEC_STATUS_TIMEOUT);
        } else {
            __syncwarp();
            const uint32_t mine = (*redo >> (4 * warp)) & 15u;
            if (mine) redo_rows<D, E4M3>(p, sm, mine);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tbase, kTmemCols);
}

template <int D, bool E4M3>
cudaError_t launch_typed(const ChunkParams& p, cudaStream_t s) {
    using C = Cfg<D, E4M3>;
    if (p.B > kChunkMaxBatch || p.ctas < 1 || p.ctas > kChunkMaxCtas || p.G > kM) return cudaErrorInvalidValue;
    CUtensorMap mk = {}, mv = {};
    const long long pool_tokens = (long long)p.num_pool_pages * kPage;
    auto make = E4M3 ? make_code_map : make_pool_map;
    if (!make(&mk, p.k, p.Hkv, pool_tokens, D) || !make(&mv, p.v, p.Hkv, pool_tokens, D)) return cudaErrorInvalidValue;
    auto kern = chunk_tc_kernel<D, E4M3>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(kern, C::kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.ctas));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.offsets ? 0 : 1;                      // trees: start while the prologue runs
    e = cudaLaunchKernelEx(&cfg, kern, p, mk, mv);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool chunk_tc_supported(int dtype, int batch, long long pool_tokens) {
    return dtype == TREESPEC_DTYPE_BF16 && batch <= kChunkMaxBatch && pool_tokens < (1ll << 31);
}

cudaError_t launch_chunk_tc(const ChunkParams& p, int kv_dtype, cudaStream_t s) {
    if (kv_dtype == TREESPEC_DTYPE_E4M3) return p.D == 64 ? launch_typed<64, true>(p, s) : launch_typed<128, true>(p, s);
    return p.D == 64 ? launch_typed<64, false>(p, s) : launch_typed<128, false>(p, s);
}

}  // namespace treespec
