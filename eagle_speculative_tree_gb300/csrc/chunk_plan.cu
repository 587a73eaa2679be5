// What the kernels over windows and shared prefixes find laid out: groups of sequences that share a
// prefix, checked, and the range of KV tiles of every CTA of the launches that follow.
//
// Group g is the sequences group_offsets[g] .. group_offsets[g + 1] - 1; their first
// shared_lens[g] logical tokens are the same.  Of these, whole KV tiles are computed for all
// rows of the group at once; what is left behind the last whole tile, fewer than 64 tokens,
// stays with each sequence.  A group shares nothing where it has fewer than two sequences with
// new tokens, where one of them has a shorter prefix (BAD_LENGTH) and, as the rows of a
// group have to be packed, anywhere in a batch whose offsets are out of order.
//
// The lengths are on the device.  One CTA per launch scans them and finds where all ranges begin, a thread
// per range; the launches' own CTAs then start with one load (when each scanned the batch by itself, the
// start of a small call took 3 to 4 us longer).  It reads and writes a few KB.  What bounds it is the
// fetching of its own instructions, which other kernels have displaced since its last run (5 us of a
// call; the same code took 11 us the first time and 5 right behind that): so it is short, with loops and
// calls where they save code.
#include "chunk_units.cuh"

namespace treespec {

namespace {

constexpr int kThreads = 1024;
constexpr int kUnitThreads = kThreads / 2;                 // where units are listed, half of the threads for them
static_assert(kChunkMaxBatch <= kThreads && kChunkMaxCtas <= kThreads, "a thread per entry and per range");

struct GroupSmem {
    int first[kMaxGroups], count[kMaxGroups], least[kMaxGroups];   // of the group's sequences with rows
    int off[kMaxGroups + 1], share[kMaxGroups];
    int4 table[kMaxGroups];
    int bad_groups, bad_chunks;
};
struct CutSmem {
    long long start[kChunkMaxBatch + 1];                   // position of each entry in the cut
    int units[kChunkMaxBatch + 1];                         // units before it, one kv head
    long long head[kChunkMaxBatch];                        // positions of one kv head of it
    int base[kChunkMaxBatch];                              // its first tile
    SeqRows rows[kChunkMaxBatch];
    int4 ends[kChunkMaxCtas];
    int pieces[kChunkMaxCtas];
    // of each warp's entries.  (Sums and maxima pass through here, not through 64-bit atomics on shared memory,
    // which took 64 sequences 3 to 4 us.)
    long long warp_size[32], warp_units[32], warp_rows[32];
    int warp_top[32];
    float warp_load[2][32];                                // tiles of the sequences' units and of the groups'
};
struct PlanSmem {
    GroupSmem groups;
    CutSmem cut;
};

// Checks the groups and writes their table and every sequence's share, by all threads.  `mine`: rows of
// sequence tid where there is one.
__device__ __forceinline__ void lay_out_groups(const ChunkParams& p, const GroupParams& g, GroupSmem& sm,
                                               const SeqRows& mine, bool flags) {
    const int tid = threadIdx.x, NG = p.groups;
    int4* gtab = const_cast<int4*>(p.gtab);
    int2* skip = const_cast<int2*>(p.skip);
    if (tid == 0) sm.bad_groups = sm.bad_chunks = 0;
    const int want0 = tid < NG ? g.shared_lens[tid] : 0;
    for (int k = tid; k <= NG; k += kThreads) sm.off[k] = g.group_offsets[k];
    for (int k = tid; k < NG; k += kThreads) {
        sm.first[k] = sm.least[k] = INT32_MAX;
        sm.count[k] = 0;
    }
    __syncthreads();
    for (int k = tid; k < NG; k += kThreads)
        if (sm.off[k] < 0 || sm.off[k + 1] < sm.off[k] || sm.off[k + 1] > p.B) sm.bad_groups = 1;
    if (p.offsets)
        for (int b = tid; b < p.B; b += kThreads)
            if (p.offsets[b] < 0 || p.offsets[b + 1] < p.offsets[b] || p.offsets[b + 1] > p.T) sm.bad_chunks = 1;
    __syncthreads();
    const bool fine = !sm.bad_groups && !sm.bad_chunks;
    auto group_of = [&](int b) -> int {                    // the last group that begins at or before b, or -1
        if (!fine || b < sm.off[0] || b >= sm.off[NG]) return -1;
        int lo = 0, hi = NG;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.off[mid] <= b) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    const int mine_of = tid < p.B ? group_of(tid) : -1;
    for (int b = tid; b < p.B; b += kThreads) {
        const int k = b == tid ? mine_of : group_of(b);
        if (k < 0) continue;
        const SeqRows r = b == tid ? mine : seq_rows(p, b);
        if (r.n == 0) continue;
        atomicMin(&sm.first[k], b);
        atomicMin(&sm.least[k], r.S);
        atomicAdd(&sm.count[k], 1);
    }
    __syncthreads();
    static_assert(kMaxGroups <= kThreads, "a thread per group");
    if (tid < NG) {
        const int k = tid, want = want0;
        const bool ok = fine && want >= 0 && (sm.count[k] == 0 || want <= sm.least[k]);
        if (!ok && !sm.bad_chunks && flags) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
        int4 e = make_int4(0, 0, 0, 0);
        if (fine) e.x = p.offsets ? p.offsets[sm.off[k]] : sm.off[k] * p.N;
        sm.share[k] = 0;
        if (ok && sm.count[k] >= 2 && want >= kSharedTile) {
            e.y = (p.offsets ? p.offsets[sm.off[k + 1]] : sm.off[k + 1] * p.N) - e.x;
            e.z = sm.share[k] = want / kSharedTile * kSharedTile;
            e.w = sm.first[k];
        }
        sm.table[k] = gtab[k] = e;
    }
    __syncthreads();
    for (int b = tid; b < p.B; b += kThreads) {
        const int k = b == tid ? mine_of : group_of(b);
        skip[b] = k < 0 ? make_int2(0, 0) : make_int2(sm.share[k], k);
    }
    __syncthreads();                                       // the cut reads other threads' sequences
}

struct Tuning {
    int kappa, min_tiles, min_tiles_many_rows, whole_tiles;
    int ctas;                                              // that get ranges
};

// Position of unit pr in its kv head: tiles and fixed costs of the units before it.  One copy of the code.
template <ChunkMode M>
__device__ __noinline__ long long unit_start(const SeqUnits<M>* u, int kappa, int pr) {
    return u->tiles_before(pr) + (long long)kappa * pr;
}

// Scans a launch's entries and lays out its ranges.  Positions, pieces and whole units are as in Cut
// (chunk_units.cuh), but ranges are even to one position: CTA c of `parts` begins at c size + min(c, rest).
template <ChunkMode M>
__device__ __forceinline__ void lay_out(const ChunkParams& p, PlanSmem& all, const SeqRows& mine, const Tuning tune,
                                        bool flags) {
    CutSmem& sm = all.cut;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int entries = chunk_entries<M>(p), Hkv = p.Hkv;
    // ---- prefix sums of the entries' positions and units
    long long size = 0;
    int nu = 0, top = 0, nr = 0;
    SeqUnits<M> u;
    if (tid < entries) {
        SeqRows r = mine;
        int base = 0;
        if (M == kChunkShared) {
            if (is_group<M>(p, tid)) {
                const int4 g = all.groups.table[tid + p.entry0];
                r = SeqRows{g.x, g.y, g.y, g.z};
            } else {
                const int b = sequence_of<M>(p, tid);
                if (b != tid) r = seq_rows(p, b);
                base = p.skip[b].x / kBN;                  // written by this block
            }
        }
        u = seq_units<M>(p, tid, r, base);
        nu = u.np;
        if (nu) {
            size = nu == 1 ? u.tiles(0) + tune.kappa : unit_start<M>(&u, tune.kappa, nu);
            top = u.tiles(nu - 1);
        }
        sm.rows[tid] = r;
        sm.base[tid] = base;
        sm.head[tid] = size;
        if (!is_group<M>(p, tid)) {
            nr = r.n;
            if (flags && !seq_ok(p, sequence_of<M>(p, tid))) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
        }
    }
    long long it = size;
    int iu = nu;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, it, o);
        const int c = __shfl_up_sync(0xffffffffu, iu, o);
        if (lane >= o) {
            it += a;
            iu += c;
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const long long rows = (long long)__reduce_add_sync(0xffffffffu, nr >> 16) * 65536 + __reduce_add_sync(0xffffffffu, nr & 0xffff);
    if (lane == 31) {
        sm.warp_size[warp] = it;
        sm.warp_units[warp] = iu;
        sm.warp_rows[warp] = rows;
        sm.warp_top[warp] = top;
    }
    __syncthreads();
    long long bt = 0, all_t = 0, bu = 0, all_u = 0, all_rows = 0;
    int longest = 0;
    const int used = (entries + 31) / 32;
#pragma unroll 1
    for (int w = 0; w < used; ++w) {
        if (w == warp) bt = all_t, bu = all_u;
        all_t += sm.warp_size[w];
        all_u += sm.warp_units[w];
        all_rows += sm.warp_rows[w];
        longest = max(longest, sm.warp_top[w]);
    }
    if (tid < entries) {
        sm.start[tid] = Hkv * (bt + it - size);
        sm.units[tid] = int(bu) + iu - nu;
        if (is_group<M>(p, tid)) const_cast<int32_t*>(p.group_units)[tid + p.entry0] = sm.units[tid];
    }
    if (tid == 0) {
        sm.start[entries] = Hkv * all_t;
        sm.units[entries] = int(all_u);
    }
    __syncthreads();

    // ---- the cut, as cut_of() makes it.  Sequences that share rows (offsets out of order) may have more units than
    // 32 bits count: no row is computed then
    const long long total = all_rows > p.T ? 0 : Hkv * all_t, n = Hkv * all_u;
    const int ctas = tune.ctas;
    auto pieces_of = [&](int tiles, int rows, int m) {
        return min(m, max(1, tiles / (rows > 64 ? tune.min_tiles_many_rows : tune.min_tiles)));
    };
    int m = 0;                                             // CTAs of each unit, 0: even ranges
    if (total < (long long)(tune.kappa + 2) * ctas && n <= ctas && total > 0) {
        m = ctas / int(n);
        if (longest / pieces_of(longest, 1, m) > int(total) / ctas + 2 * tune.kappa) m = 0;
    }
    const int parts = total == 0 ? 0 : m ? m * int(n) : int(min((long long)ctas, max(1ll, total / (tune.kappa + 1))));
    long long size_of = 1, rest = 0;                       // of a range
    if (parts && !m) {
        size_of = div_pos(total, parts);
        rest = total - size_of * parts;
    }
    const long long wide = rest * (size_of + 1);
    // The CTA that holds the first piece of a unit of `tiles` tiles at position `at` (number `index` of the batch),
    // and its pieces
    auto share_of = [&](long long at, int tiles, int rows, int index) -> int2 {
        if (m) return make_int2(index * m, pieces_of(tiles, rows, m));
        int c[2];
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            const long long x = at + (i ? tiles - 1 : 0);
            c[i] = int(x < wide ? div_pos(x, size_of + 1) : rest + div_pos(x - wide, size_of));
        }
        return make_int2(c[0], tiles <= tune.whole_tiles ? 1 : c[1] - c[0] + 1);
    };

    // ---- the ranges, and at the same time the groups' units of 256 rows for the merge: a thread per range or unit
    const bool table = M == kChunkShared && !p.few_rows && is_group<M>(p, 0);
    const int nunits = table && total > 0 ? Hkv * sm.units[min(entries, p.groups)] : 0;
    const bool unit_job = table && tid >= kUnitThreads;        // units; the other threads: ranges
    int job = unit_job ? tid - kUnitThreads : tid;
#pragma unroll 1
    for (int round = 0; round == 0 || round * kUnitThreads < nunits; ++round, job += kUnitThreads) {
        const bool by_unit = unit_job || m, on = unit_job ? job < nunits : round == 0 && job < parts;
        End e{0, 0, 0, 0};
        int2 share = make_int2(0, 0);
        int tiles = 0;
        if (on) {
            const int index = unit_job ? job : m ? job / m : 0;
            const long long x = by_unit ? index : job * size_of + min((long long)job, rest);
            int lo = 0, hi = entries;                  // the last entry that begins at or before x
#pragma unroll 1
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if ((by_unit ? (long long)Hkv * sm.units[mid] : sm.start[mid]) <= x) lo = mid;
                else hi = mid;
            }
            u = seq_units<M>(p, lo, sm.rows[lo], sm.base[lo]);
            long long y = x - (by_unit ? (long long)Hkv * sm.units[lo] : sm.start[lo]);
            const long long head = by_unit ? u.np : sm.head[lo];
            e.b = lo;
            e.h = int(div_pos(y, head));
            y -= e.h * head;
            long long at = 0;                          // of the unit, in its kv head
            if (by_unit) {
                e.pr = int(y);
                if (!m && u.np > 1) at = unit_start<M>(&u, tune.kappa, e.pr);
            } else if (u.np > 1) {
                int end = u.np;                        // the last unit that begins at or before y
#pragma unroll 1
                while (end - e.pr > 1) {
                    const int mid = (e.pr + end) >> 1;
                    const long long z = unit_start<M>(&u, tune.kappa, mid);
                    if (z <= y) {
                        e.pr = mid;
                        at = z;
                    } else {
                        end = mid;
                    }
                }
            }
            tiles = u.tiles(e.pr);
            const int rows = min(u.tpu, (is_group<M>(p, lo) ? sm.rows[lo].n : u.live) - e.pr * u.tpu) * p.G;
            share = share_of(sm.start[lo] + e.h * sm.head[lo] + at + tune.kappa, tiles, rows, index);
            if (!by_unit) {
                e.j = int(max(0ll, y - at - tune.kappa));
                // Short units stay whole: the cut moves to the nearer end of one, and both neighbours see it there
                if (tiles <= tune.whole_tiles) e.j = 2 * e.j < tiles ? 0 : tiles;
            }
        }
        if (unit_job && on) const_cast<int2*>(p.units)[job] = share;
        if (round > 0) continue;
        // one range ends where the next begins; of m CTAs for each unit, those beyond its pieces have nothing
        auto cut_at = [&](int k) {
            return k > share.y ? tiles : int(uint32_t(tiles) * uint32_t(k) / uint32_t(share.y));
        };
        int4 begin = make_int4(entries, 0, 0, 0);
        if (on) begin = make_int4(e.b, e.h, e.pr, m ? cut_at(job % m) : e.j);
        const bool range = !unit_job && job < p.ctas;
        if (range) {
            sm.ends[job] = begin;
            sm.pieces[job] = share.y;
        }
        __syncthreads();
        if (range) {
            CtaPlan out{};
            out.begin = begin;
            if (!on) {
                out.begin.x = -1;
            } else {
                const bool last = job + 1 >= parts;
                out.end = m ? make_int4(e.b, e.h, e.pr, cut_at(job % m + 1))
                            : last ? make_int4(entries, 0, 0, 0) : sm.ends[job + 1];
                out.last_pieces = m ? share.y : last ? 0 : sm.pieces[job + 1];
                out.first_cta = share.x;
                out.first_pieces = share.y;
                const SeqRows& r = sm.rows[e.b];
                out.rows = make_int4(r.row0, r.n, r.live, r.S);
                out.base = sm.base[e.b];
            }
            const_cast<CtaPlan*>(p.plan)[job] = out;
        }
    }
}

template <ChunkMode M>
__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanParams a) {
    extern __shared__ __align__(16) unsigned char smem[];
    PlanSmem& sm = *reinterpret_cast<PlanSmem*>(smem);
    grid_dep_release();                                    // the attention kernel may launch; it waits for this grid
    grid_dep_wait();                                       // trees: the prologue's results
    const bool first = blockIdx.x == 0;                    // the block that flags, and clears before that
    if (first) {
        for (int i = threadIdx.x; i < a.clear; i += kThreads) a.cleared[i] = 0;
        __syncthreads();
    }
    const ChunkParams& p = a.launch[blockIdx.x];
    if (first && a.flags)
        for (int b = threadIdx.x; b < p.B; b += kThreads)
            if (const uint32_t st = a.flags[b]) atomicOr(p.status, st);
    SeqRows mine{0, 0, 0, -1};
    if (int(threadIdx.x) < p.B) mine = seq_rows(p, threadIdx.x);
    if (M == kChunkShared) lay_out_groups(p, a.groups, sm.groups, mine, first);
    if (a.launches == 0) return;
    const int kappa = p.k_scales && a.launches == 1 ? TuneUnits::kPlanKappaCodes : TuneUnits::kPlanKappa;
    Tuning tune{kappa, TuneUnits::kPlanMinTiles, TuneUnits::kMinTilesManyRows, TuneUnits::kWholeTiles, p.ctas};
    if (p.few_rows) tune = Tuning{TuneFew::kKappa, TuneFew::kMinTiles, TuneFew::kMinTiles, TuneFew::kWholeTiles, p.ctas};
    if (M == kChunkShared && a.launches == 2) {
        // Two launches, the groups' on units of 256 rows with an SM for each CTA and the sequences' with
        // two CTAs to an SM, run at the same time: each gets SMs by its tiles, a tile of 256 rows
        // counted 2.3 times (64 sequences of one token, 20 .. 600 tokens of their own behind 8192
        // shared ones: 59 us, e4m3 62; 63 and 69 counted 1.4 times, 61 and 58 counted 3.4; one launch
        // after the other took an eighth longer).
        const int g0 = a.launch[1].groups, tpu = a.launch[1].tpu, few_tpu = a.launch[0].tpu;
        float load[2] = {0.f, 0.f};
        if (int(threadIdx.x) < p.B && mine.S >= 0) {
            const int base = p.skip[threadIdx.x].x / kBN;
            load[0] = float((mine.live + few_tpu - 1) / few_tpu) *
                      float((mine.S + mine.live + kBN - 1) / kBN - base + TuneFew::kKappa);
        }
        if (int(threadIdx.x) < g0) {
            const int4 e = sm.groups.table[threadIdx.x];
            if (e.y) load[1] = float((e.y + tpu - 1) / tpu) * float(e.z / kBN + kappa);
        }
#pragma unroll 1
        for (int o = 16; o; o >>= 1) {
            load[0] += __shfl_xor_sync(0xffffffffu, load[0], o);
            load[1] += __shfl_xor_sync(0xffffffffu, load[1], o);
        }
        if ((threadIdx.x & 31) == 0) {
            sm.cut.warp_load[0][threadIdx.x >> 5] = load[0];
            sm.cut.warp_load[1][threadIdx.x >> 5] = load[1];
        }
        __syncthreads();
        float own = 0.f, shared = 0.f;                     // added up in one order, whatever the run
#pragma unroll 1
        for (int w = 0; w < (max(p.B, g0) + 31) / 32; ++w) {
            own += sm.cut.warp_load[0][w];
            shared += 2.3f * sm.cut.warp_load[1][w];
        }
        const int sms = a.launch[1].ctas;
        int for_groups = shared == 0.f ? 0 : min(sms, max(1, int(float(sms) * shared / (shared + own) + 0.5f)));
        if (own > 0.f) for_groups = min(for_groups, max(1, sms - 1));
        tune.ctas = p.few_rows ? max(1, p.ctas - int((long long)p.ctas * for_groups / sms)) : max(1, for_groups);
    }
    lay_out<M>(p, sm, mine, tune, first);
    // The second of two launches does not wait for this grid but for this store (chunk_few.cuh)
    if (M == kChunkShared && first && p.published) {
        __syncthreads();
        if (threadIdx.x == 0) store_release(p.published, p.epoch);
    }
}

}  // namespace

cudaError_t launch_chunk_plan(const PlanParams& p, ChunkMode mode, cudaStream_t s) {
    for (int i = 0; i < p.launches; ++i) {
        const ChunkParams& q = p.launch[i];
        if ((mode == kChunkShared ? q.entries : q.B) > kChunkMaxBatch || q.ctas < 1 ||
            q.ctas > (mode == kChunkShared && !q.few_rows ? kUnitThreads : kChunkMaxCtas))
            return cudaErrorInvalidValue;
    }
    if (mode == kChunkShared && p.launch[0].groups > kMaxGroups) return cudaErrorInvalidValue;
    auto kern = mode == kChunkShared ? plan_kernel<kChunkShared> : plan_kernel<kChunkWindow>;
    static std::atomic<uint64_t> smem_set[2];
    cudaError_t e = allow_smem(kern, sizeof(PlanSmem), smem_set[mode == kChunkShared]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.launches > 1 ? p.launches : 1));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(PlanSmem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.launch[0].offsets ? 0 : 1;            // trees: start while the prologue runs
    e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace treespec
