// What the persistent chunk kernels share (chunk_tc.cuh, chunk_few.cuh): the units of a batch, the cut
// of their KV tiles into one range per CTA, the walk along a range, what a row sees, and the
// producer of an 8-bit cache's codes.
#pragma once

#include "attn_tc_parts.cuh"

namespace treespec {

namespace {

using namespace sm100;

constexpr int kBN = 64;              // tokens per KV tile

// Of the cut: kKappa, a unit's fixed cost in tiles.  No piece of a unit with CTAs of its own is shorter
// than kMinTiles (kMinTilesManyRows of more than 64 rows), and units up to kWholeTiles long are not cut.
struct TuneUnits {                   // units of 256 rows (chunk_tc.cuh)
    static constexpr int kKappa = 7;
    // Joining costs by the row, so units of many rows are cut into longer pieces (8 nodes x 4 heads over
    // 2048 e4m3 tokens: 28.7 us in pieces of 4 tiles, 30.9 of 9; 3 prompts of up to 816 tokens, 4
    // heads: 33 and 25).
    static constexpr int kMinTiles = 4, kMinTilesManyRows = 9;
    // where the ranges are planned ahead (chunk_plan.cu), a CTA starts sooner and shorter pieces pay (8 nodes
    // x 4 heads over 2048 e4m3 tokens, 512 of them in the window: 29.1 us in pieces of 2 tiles, 31.1 of 4)
    static constexpr int kPlanMinTiles = 2;
    // There, too, the fixed cost counts in each type's tiles, 0.8 us of bf16 and 1.3 of e4m3 (4 prompts
    // through a window and 32 trees behind a shared prefix, bf16: 208 and 168 us, and 212 and 174 with 7;
    // 4 prompts and 47 short chunks behind 3 prefixes, e4m3: 376 and 104 us, and 393 and 106 with 7); but
    // the groups of decoded tokens are cut into pieces whose stores count for more (64 sequences, bf16 and
    // e4m3: 59 and 62 us, and 65 and 66 with 7).
    static constexpr int kPlanKappa = 10, kPlanKappaCodes = 5;
    static constexpr int kWholeTiles = 4;
};
struct TuneFew {                     // units of 8 or 16 rows (chunk_few.cuh)
    static constexpr int kKappa = 3;
    static constexpr int kMinTiles = 2;
    static constexpr int kWholeTiles = 2;
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

// The units of one entry (a sequence, or a group of them) and one kv head.  What a form of the call
// adds stands in a base of its own, so that the plain form's registers hold no more.
template <ChunkMode M>
struct UnitsOf {};
template <>
struct UnitsOf<kChunkWindow> {
    int full;                         // units whose tokens are all there
    int low, sink_tiles;              // first token of the window of row 0; tiles of the sinks
};
template <>
struct UnitsOf<kChunkShared> {
    int full;
    int base;                         // the first tile
};
template <ChunkMode M>
struct SeqUnits : UnitsOf<M> {
    int S, live, np;                  // prefix, rows' tokens, units
    int tpu;                          // tokens per unit
    bool tree;                        // all rows reach as far
    // tiles from the sequence's begin to the last that unit pr runs over
    __device__ __forceinline__ int end(int pr) const {
        return (S + (tree ? live : min(live, (pr + 1) * tpu)) + kBN - 1) / kBN;
    }
    // window: tiles between the sinks and unit pr's window
    __device__ __forceinline__ int gap(int pr) const {
        if constexpr (M == kChunkWindow) return max(0, ((this->low + (tree ? 0 : pr * tpu)) >> 6) - this->sink_tiles);
        return 0;
    }
    // KV tiles of unit pr
    __device__ __forceinline__ int tiles(int pr) const {
        if constexpr (M == kChunkWindow) return end(pr) - gap(pr);
        if constexpr (M == kChunkShared) return end(pr) - this->base;
        return end(pr);
    }
    // sum of floor((a + k tpu) / 64), k = 0 .. n - 1
    __device__ __forceinline__ long long sum_tiles(int n, int a) const {
        const int a1 = tpu / kBN, r = tpu % kBN;
        long long s = (long long)n * (a / kBN) + (long long)n * (n - 1) / 2 * a1;
        if (r) s += floor_sum(uint32_t(n), kBN, uint32_t(r), uint32_t(a % kBN));
        return s;
    }
    // KV tiles of units 0 .. pr - 1
    __device__ __forceinline__ long long tiles_before(int pr) const {
        if (pr <= 0) return 0;
        if (tree) return (long long)pr * tiles(0);
        int full;                                          // units whose tokens are all there
        if constexpr (M == kChunkPlain) full = min(pr, live / tpu);
        else full = min(pr, this->full);
        long long s = sum_tiles(full, S + kBN - 1 + tpu);
        if (pr > full) s += end(pr - 1);
        if constexpr (M == kChunkShared) s -= (long long)pr * this->base;
        if constexpr (M == kChunkWindow) {                 // the gaps, from the first unit that has one on
            const long long to_gap = (long long)kBN * (this->sink_tiles + 1) - this->low;
            const int k = to_gap <= 0 ? 0 : int(min(uint32_t(pr), (uint32_t(to_gap) + tpu - 1) / uint32_t(tpu)));   // < 2^32
            if (k < pr) s -= sum_tiles(pr - k, this->low + k * tpu) - (long long)(pr - k) * this->sink_tiles;
        }
        return s;
    }
};
// `base`: with shared prefixes, the first tile of a sequence's own units.
template <ChunkMode M>
__device__ __forceinline__ SeqUnits<M> seq_units(const ChunkParams& p, int v, const SeqRows& r, int base) {
    SeqUnits<M> u;
    u.tree = !p.offsets;
    u.tpu = p.tpu;
    u.S = r.S;
    u.live = r.S < 0 ? 0 : r.live;
    if constexpr (M == kChunkPlain) {
        u.np = (u.live + u.tpu - 1) / u.tpu;
    } else {
        u.full = u.live / u.tpu;
        u.np = u.full + (u.live > u.full * u.tpu);
    }
    if constexpr (M == kChunkWindow) {
        u.low = r.S - p.window + 1;
        u.sink_tiles = (p.sinks + kBN - 1) / kBN;
    }
    if constexpr (M == kChunkShared) {
        u.base = base;
        if (is_group<M>(p, v)) {                           // every unit over the shared tokens alone
            u.tree = true;
            u.live = 0;
        }
    }
    return u;
}
template <ChunkMode M>
__device__ __forceinline__ SeqUnits<M> seq_units(const ChunkParams& p, int v, const SeqRows& r) {
    int base = 0;
    if (M == kChunkShared && !is_group<M>(p, v)) base = p.skip[sequence_of<M>(p, v)].x / kBN;
    return seq_units<M>(p, v, r, base);
}
template <ChunkMode M>
__device__ __forceinline__ SeqUnits<M> seq_units(const ChunkParams& p, int v) {
    return seq_units<M>(p, v, entry_rows<M>(p, v));
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
    return min(m, max(1, n / (rows > 64 ? TuneUnits::kMinTilesManyRows : TuneUnits::kMinTiles)));
}

// The cut of a batch: the prefix sums and the KV tiles of its longest unit.
__device__ __forceinline__ Cut cut_of(const ChunkParams& p, const long long* tiles, const int* units, int longest, int ctas) {
    Cut cut;
    const long long n = (long long)p.Hkv * units[p.B];
    cut.tiles = tiles;
    cut.units = units;
    cut.B = p.B;
    cut.Hkv = p.Hkv;
    cut.k = TuneUnits::kKappa;
    cut.total = p.Hkv * tiles[p.B] + TuneUnits::kKappa * n;
    // A range that holds pieces of two units pays the fixed cost twice, so where there is less
    // than about that cost for each CTA, every unit gets CTAs of its own instead (119 new
    // tokens, 32 q / 8 kv heads: 35 us cut evenly, 21 this way; 8 nodes over 2048 e4m3 tokens:
    // 42 and 29), unless one long unit among short ones would then run far longer than its
    // share of all tiles
    cut.m = 0;
    if (cut.total < (long long)(TuneUnits::kKappa + 2) * ctas && n <= ctas && n > 0) {
        const int m = ctas / int(n);
        if (longest / unit_pieces(longest, 1, m) <= int(cut.total) / ctas + 2 * TuneUnits::kKappa) cut.m = m;
    }
    cut.parts = cut.m ? cut.m * int(n) : int(min((long long)ctas, max(1ll, cut.total / (TuneUnits::kKappa + 1))));
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
    const SeqUnits<kChunkPlain> u = seq_units<kChunkPlain>(p, lo);
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

// The prefix sums of the sequences' tiles and units, and *longest, the tiles of the longest unit, by all
// threads of the CTA; flags bad lengths.  wt: [warps] {tiles, units, rows}.
template <int kThreads>
__device__ __forceinline__ void scan_units(const ChunkParams& p, long long* tiles_s, int* units_s, long long* wt,
                                           int* longest) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long nt = 0;
    int nu = 0, top = 0, rows_lo = 0, rows_hi = 0;     // rows in 16-bit halves: sums of 96 sequences fit
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const SeqRows r = seq_rows(p, b);
        const SeqUnits<kChunkPlain> u = seq_units<kChunkPlain>(p, b, r);
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
    if (tid == kThreads - 1) {
        // Sequences that share rows (offsets out of order) may have more units than 32 bits count:
        // no row is computed then
        tiles_s[p.B] = rows > p.T ? 0 : bt + nt;
        units_s[p.B] = rows > p.T ? 0 : int(bu + nu);
    }
    __syncthreads();
}

// Rows without a token (a padded tree's, and those of an invalid sequence) are zeros; `threads` threads of the
// CTA, this one number `tid` of them.
template <ChunkMode M, int D>
__device__ __forceinline__ void zero_rows(const ChunkParams& p, int tid, int threads) {
    if (M == kChunkShared && p.entry0 + p.entries <= p.groups) return;   // a launch over the groups alone
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const SeqRows r = seq_rows(p, b);
        const int from = r.S < 0 ? 0 : r.live;
        const size_t words = size_t(r.n - from) * p.Hq * (D / 8);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + size_t(r.row0 + from) * p.Hq * D);
        for (size_t e = tid; e < words; e += threads) dst[e] = make_uint4(0, 0, 0, 0);
    }
}

// One contiguous range of KV tiles of one unit.
template <ChunkMode M>
struct SegOf {};
template <>
struct SegOf<kChunkWindow> {
    int cut_lo, cut_hi;    // the gap's tokens (none: both 0)
    int low;               // first token of the first row's window
};
template <>
struct SegOf<kChunkShared> {
    int seq;               // sequence whose pages are read
    int side;              // -1: the rows are whole; 0 / 1: the group's / their own part of them
};
template <ChunkMode M>
struct Seg : SegOf<M> {
    int b, h, pr;          // entry, kv head, unit
    int S, live, L;        // prefix, rows' tokens and logical tokens of the sequence
    int row0;              // q row of the unit's first token
    int i0, tokens;        // the unit's tokens: i0 .. i0 + tokens - 1 of the sequence's new ones
    int j0, ntiles, n;     // tiles j0 .. j0 + ntiles - 1 of n
    int t0, t1;            // their logical tokens
    int nq;                // query tiles in use
    __device__ __forceinline__ bool whole() const { return ntiles == n; }
    // first token of tile j of the segment
    __device__ __forceinline__ int place(int j) const {
        if constexpr (M == kChunkWindow) {
            const int t = (j0 + j) * kBN;
            return t < this->cut_lo || this->cut_hi == 0 ? t : t + (this->cut_hi - this->cut_lo);
        }
        return t0 + j * kBN;
    }
    // window: tiles of the segment before the gap
    __device__ __forceinline__ int head_tiles() const {
        if constexpr (M == kChunkWindow) return this->cut_hi == 0 ? ntiles : max(0, min(ntiles, this->cut_lo / kBN - j0));
        return ntiles;
    }
    // the token behind the gap where `pos` (on the border of a tile where one begins) lies in it
    __device__ __forceinline__ int over_gap(int pos) const {
        if constexpr (M == kChunkWindow) return pos >= this->cut_lo && pos < this->cut_hi ? this->cut_hi : pos;
        return pos;
    }
    __device__ __forceinline__ int sequence() const {
        if constexpr (M == kChunkShared) return this->seq;
        return b;
    }
    // the rows' result is one of two parts: 0 the group's, 1 their own; -1: it is whole
    __device__ __forceinline__ int part() const {
        if constexpr (M == kChunkShared) return this->side;
        return -1;
    }
};

// The segments of a CTA's range, in order.  Every role walks them by itself.
template <ChunkMode M>
struct Walk {
    const ChunkParams* p;
    End e, end;            // next segment's first tile; the first tile behind the range
    SeqUnits<M> u;
    SeqRows rows;
    __device__ __forceinline__ void load() {
        rows = entry_rows<M>(*p, e.b);
        u = seq_units<M>(*p, e.b, rows);
    }
    __device__ __forceinline__ void start(const ChunkParams& pp, const End& a, const End& z, const SeqRows& r) {
        start(pp, a, z, r, seq_units<M>(pp, a.b < chunk_entries<M>(pp) ? a.b : 0, r));
    }
    __device__ __forceinline__ void start(const ChunkParams& pp, const CtaPlan& plan) {
        const SeqRows r{plan.rows.x, plan.rows.y, plan.rows.z, plan.rows.w};
        start(pp, End{plan.begin.x, plan.begin.y, plan.begin.z, plan.begin.w},
              End{plan.end.x, plan.end.y, plan.end.z, plan.end.w}, r, seq_units<M>(pp, plan.begin.x, r, plan.base));
    }
    // rows and units: of entry a.b
    __device__ __forceinline__ void start(const ChunkParams& pp, const End& a, const End& z, const SeqRows& r,
                                          const SeqUnits<M>& su) {
        p = &pp;
        e = a;
        end = z;
        rows = r;
        u = su;
        if (e.b < chunk_entries<M>(pp) && e.j >= u.tiles(e.pr)) advance();
    }
    __device__ __forceinline__ bool next(Seg<M>& s) {
        // behind the range: also where both its ends were moved to the same unit's end
        if (e.b > end.b || (e.b == end.b && (e.h > end.h || (e.h == end.h && e.pr > end.pr)))) return false;
        const bool last = e.b == end.b && e.h == end.h && e.pr == end.pr;
        if (last && e.j >= end.j) return false;
        s.b = e.b;
        s.h = e.h;
        s.pr = e.pr;
        const bool group = is_group<M>(*p, e.b);
        s.S = u.S;
        s.live = u.live;
        s.L = u.S + u.live;                                // a group: the shared tokens
        s.i0 = e.pr * u.tpu;
        s.tokens = min(u.tpu, (group ? rows.n : u.live) - s.i0);
        s.row0 = rows.row0 + s.i0;
        s.nq = s.tokens > u.tpu / 2 ? 2 : 1;
        s.n = u.tiles(e.pr);
        s.j0 = e.j;
        s.ntiles = (last ? min(end.j, s.n) : s.n) - e.j;
        const int vis = u.S + (u.tree ? u.live : s.i0 + s.tokens);
        if constexpr (M == kChunkWindow) {
            const int gap = u.gap(e.pr);
            s.cut_lo = gap ? u.sink_tiles * kBN : 0;
            s.cut_hi = gap ? (u.sink_tiles + gap) * kBN : 0;
            s.low = u.low + (u.tree ? 0 : s.i0);
            s.t0 = s.place(0);
            s.t1 = min(vis, s.place(s.ntiles - 1) + kBN);
        } else if constexpr (M == kChunkShared) {
            s.seq = group ? p->gtab[e.b + p->entry0].w : sequence_of<M>(*p, e.b);
            s.side = group ? 0 : u.base ? 1 : -1;
            s.t0 = (u.base + s.j0) * kBN;
            s.t1 = min(vis, (u.base + s.j0 + s.ntiles) * kBN);
        } else {
            s.t0 = s.j0 * kBN;
            s.t1 = min(vis, (s.j0 + s.ntiles) * kBN);
        }
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
                    if (e.b >= chunk_entries<M>(*p) || e.b > end.b) { e.b = end.b + 1; break; }
                    load();
                } while (u.np == 0);
            }
        }
    }
};

// ------------------------------------------------------------------ rows

// A query row of a segment.
struct Row {
    int i, hq;             // token of the sequence's new ones, query head
    size_t at;             // element offset of the row in q and out
    bool ok;
};
// What a row may see: the prefix and, of the new tokens, 0 .. i (a chunk) or its ancestors.
template <ChunkMode M>
struct SightOf {};
template <>
struct SightOf<kChunkWindow> {
    int low = 0;           // first token of the window (trees: of the prefix; the sets say the rest)
};
template <ChunkMode M>
struct Sight : SightOf<M> {
    int end = 0;           // chunks: first logical token it may not see
    uint64_t a0 = 0, a1 = 0;   // trees
};
template <ChunkMode M>
__device__ __forceinline__ Sight<M> sight_of(const ChunkParams& p, const Seg<M>& s, const Row& r) {
    Sight<M> v;
    if (!r.ok) return v;
    if (p.offsets) {
        v.end = s.S + r.i + 1;
        if constexpr (M == kChunkWindow) v.low = s.S + r.i - p.window + 1;
    } else if (s.part() != 0) {                            // all of a group's tokens are prefix
        const uint64_t* a = p.anc + (size_t(s.sequence()) * p.N + r.i) * kAncWords;
        v.a0 = a[0];
        v.a1 = a[1];
        if constexpr (M == kChunkWindow) v.low = s.S + min(0, p.depth[size_t(s.b) * p.N + r.i] - p.window + 1);
    }
    return v;
}
// bits below column n of a tile's word w
__device__ __forceinline__ uint32_t columns_below(int n, int w) {
    n -= 32 * w;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Whether the row sees the token at `pos`, below the segment's t1.
template <ChunkMode M>
__device__ __forceinline__ bool sees(const ChunkParams& p, const Seg<M>& s, const Sight<M>& v, int pos) {
    const int j = pos - s.S;
    if constexpr (M == kChunkWindow)
        if (pos < v.low && pos >= p.sinks) return false;
    return j < 0 || (p.offsets ? pos < v.end : ((j < 64 ? v.a0 >> j : v.a1 >> (j - 64)) & 1ull) != 0);
}

// Rows of the parts that the merge joins: [group, own][T][Hq].
__device__ __forceinline__ size_t side_offset(const ChunkParams& p, int side) { return size_t(side) * p.T * p.Hq; }

// ------------------------------------------------------------------ codes of an 8-bit cache

// 64 contiguous bytes (a page's scales of one head) into shared memory
__device__ __forceinline__ void bulk_load_64(void* dst, const void* src, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 64, [%2];" ::"r"(
                     smem_u32(dst)), "l"(src), "r"(smem_u32(bar))
                 : "memory");
}

// One warp streams the codes and scales of K (or V) of a segment into rings of kStages stages,
// a tile of 64 rows of D bytes and 64 floats per stage.  Lanes 0 .. 3 own a page each: a
// page that lies wholly in the sequence arrives by TMA, the partly filled last one is written
// by the warp, zeros behind the last token, and so is a bad page id (flagged) or a page
// behind the segment.  `g` counts tiles over the CTA's life.  False after a timeout or an
// abort.
template <int D, ChunkMode M, int kStages>
__device__ __forceinline__ bool produce_codes(const ChunkParams& p, const CUtensorMap* map, const unsigned char* src,
                                              const float* scales, unsigned char* ring, float* sring, uint64_t* full,
                                              uint64_t* empty, const Seg<M>& s, int& g, volatile uint32_t* abort_flag) {
    const int lane = threadIdx.x & 31;
    const int* ptab = p.page_table + size_t(s.sequence()) * p.max_pages;
    auto fetch = [&](int bi) -> int {                      // page ids of 8 tiles, one warp-wide load
        const int jt = 8 * bi + lane / 4;
        const int pos = s.place(jt) + (lane % 4) * 16;
        return (M != kChunkWindow || jt < s.ntiles) && pos < s.t1 ? __ldg(ptab + (pos >> 4)) : -1;
    };
    auto needed = [&](int pos0) -> bool {                  // window: whether a row of the unit sees a token of the page
        if constexpr (M == kChunkWindow) return pos0 + 16 > s.low || pos0 < p.sinks;
        return true;
    };
    int cur = fetch(0), nxt = fetch(1);
    for (int j = 0; j < s.ntiles; ++j, ++g) {
        const int st = g % kStages;
        if (j > 0 && (j & 7) == 0) {
            cur = nxt;
            nxt = fetch(j / 8 + 1);
        }
        int page = __shfl_sync(0xffffffffu, cur, (j & 7) * 4 + (lane & 3));
        const int base = s.place(j), pos0 = base + (lane & 3) * 16;
        int kind = 0;                                      // 1: by TMA, 2: written here
        if (lane < 4) {
            kind = 2;
            if (pos0 < s.t1 && needed(pos0)) {
                const bool ok = page >= 0 && page < p.num_pool_pages;
                if (!ok) atomicOr(p.status, TREESPEC_STATUS_BAD_PAGE);
                if (ok && pos0 + 16 <= s.L) kind = 1;
                if (!ok) page = -1;
            } else {
                page = -1;
            }
        }
        if (g >= kStages && !mbar_wait_bounded(&empty[st], ((g / kStages) - 1) & 1, p.wait_ns)) {
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

}  // namespace

}  // namespace treespec
