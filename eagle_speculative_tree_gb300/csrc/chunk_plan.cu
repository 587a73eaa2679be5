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
// The lengths are on the device.  One CTA per launch scans them and finds both ends of all ranges, a thread
// per range; the launches' own CTAs then start with one load.  Scan and search in every one of these CTAs instead took
// about 5 us of each, as the plain persistent kernel's do.
#include "chunk_units.cuh"

namespace treespec {

namespace {

constexpr int kThreads = 1024;
static_assert(kChunkMaxBatch <= kThreads && kChunkMaxCtas <= kThreads, "a thread per entry and per range");

struct GroupSmem {
    int first[kMaxGroups], count[kMaxGroups], least[kMaxGroups];   // of the group's sequences with rows
    int off[kMaxGroups + 1], share[kMaxGroups];
    int bad_groups, bad_chunks;
};
struct CutSmem {
    long long tiles[kChunkMaxBatch + 1];
    long long warp_tiles[32], warp_rows[32];
    int units[kChunkMaxBatch + 1];
    int warp_units[32];
    int longest;
    SeqRows rows[kChunkMaxBatch];
    int4 ends[kChunkMaxCtas];
    int pieces[kChunkMaxCtas];
};

union PlanSmem {
    GroupSmem groups;
    CutSmem cut;
};

__device__ void lay_out_groups(const ChunkParams& p, const GroupParams& g, GroupSmem& sm, bool flags) {
    const int tid = threadIdx.x, NG = p.groups;
    int4* gtab = const_cast<int4*>(p.gtab);
    int2* skip = const_cast<int2*>(p.skip);
    if (tid == 0) sm.bad_groups = sm.bad_chunks = 0;
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
    for (int b = tid; b < p.B; b += kThreads) {
        const int k = group_of(b);
        if (k < 0) continue;
        const SeqRows r = seq_rows(p, b);
        if (r.n == 0) continue;
        atomicMin(&sm.first[k], b);
        atomicMin(&sm.least[k], r.S);
        atomicAdd(&sm.count[k], 1);
    }
    __syncthreads();
    for (int k = tid; k < NG; k += kThreads) {
        const int want = g.shared_lens[k];
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
        gtab[k] = e;
    }
    __syncthreads();
    for (int b = tid; b < p.B; b += kThreads) {
        const int k = group_of(b);
        skip[b] = k < 0 ? make_int2(0, 0) : make_int2(sm.share[k], k);
    }
    __syncthreads();
}

// The tile at or after position x of the cut, by one thread.  x < total.
template <ChunkMode M>
__device__ End find(const ChunkParams& p, const Cut& q, const SeqRows* rows, long long x) {
    int lo = 0, hi = q.B;                                  // the last b with before(b) <= x
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.before(mid) <= x) lo = mid;
        else hi = mid;
    }
    End e;
    e.b = lo;
    const SeqUnits<M> u = seq_units<M>(p, lo, rows[lo]);
    const long long head = div_pos(q.before(lo + 1) - q.before(lo), q.Hkv);
    long long y = x - q.before(lo);
    e.h = int(div_pos(y, head));
    y -= e.h * head;
    int at = 0, n = u.np;                                  // the last unit that begins at or before y
    while (n - at > 1) {
        const int mid = (at + n) >> 1;
        if (u.tiles_before(mid) + (long long)q.k * mid <= y) at = mid;
        else n = mid;
    }
    e.pr = at;
    e.j = int(max(0ll, y - u.tiles_before(at) - (long long)q.k * at - q.k));
    return e;
}

template <ChunkMode M, class Tune>
__device__ void lay_out_ranges(const ChunkParams& p, CutSmem& sm, bool flags) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int entries = chunk_entries<M>(p);
    if (tid == 0) sm.longest = 0;
    // ---- prefix sums of the entries' tiles and units
    SeqRows r{0, 0, 0, -1};
    long long nt = 0, nr = 0;
    int nu = 0, top = 0;
    if (tid < entries) {
        r = entry_rows<M>(p, tid);
        sm.rows[tid] = r;
        const SeqUnits<M> u = seq_units<M>(p, tid, r);
        nu = u.np;
        if (nu) {
            nt = nu == 1 ? u.tiles(0) : u.tiles_before(nu);
            top = u.tiles(nu - 1);
        }
        if (!is_group<M>(p, tid)) {
            nr = r.n;
            if (flags && !seq_ok(p, sequence_of<M>(p, tid))) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
        }
    }
    long long it = nt, ir = nr;
    int iu = nu;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ir, o);
        const int c = __shfl_up_sync(0xffffffffu, iu, o);
        if (lane >= o) {
            it += a;
            ir += b;
            iu += c;
        }
    }
    if (lane == 31) {
        sm.warp_tiles[warp] = it;
        sm.warp_rows[warp] = ir;
        sm.warp_units[warp] = iu;
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if (lane == 0 && top) atomicMax(&sm.longest, top);
    long long bt = 0, all_t = 0, all_r = 0, bu = 0, all_u = 0;
    const int used = (entries + 31) / 32;
    for (int w = 0; w < used; ++w) {
        if (w == warp) bt = all_t, bu = all_u;
        all_t += sm.warp_tiles[w];
        all_r += sm.warp_rows[w];
        all_u += sm.warp_units[w];
    }
    // Sequences that share rows (offsets out of order) may have more units than 32 bits count: no row is
    // computed then
    const bool none = all_r > p.T;
    if (tid < entries) {
        sm.tiles[tid] = bt + it - nt;
        sm.units[tid] = int(bu) + iu - nu;
        if (is_group<M>(p, tid)) const_cast<int32_t*>(p.group_units)[tid + p.entry0] = sm.units[tid];
    }
    if (tid == 0) {
        sm.tiles[entries] = none ? 0 : all_t;
        sm.units[entries] = none ? 0 : int(all_u);
    }
    __syncthreads();

    // ---- the ranges
    const Cut cut = cut_of<M, Tune>(p, sm.tiles, sm.units, sm.longest, p.ctas);
    // rows of unit pr of entry b
    auto rows_of = [&](int b, int pr, const SeqUnits<M>& u) {
        return min(u.tpu, (is_group<M>(p, b) ? sm.rows[b].n : u.live) - pr * u.tpu) * p.G;
    };
    // of unit e of n tiles: the CTA that holds its first piece, and its pieces
    auto share_of = [&](const End& e, const SeqUnits<M>& u, int n, int index) -> int2 {
        if (cut.m) return make_int2(index * cut.m, unit_pieces<Tune>(n, rows_of(e.b, e.pr, u), cut.m));
        const long long ub = cut.before(e.b) + e.h * div_pos(cut.before(e.b + 1) - cut.before(e.b), cut.Hkv) +
                             u.tiles_before(e.pr) + (long long)cut.k * e.pr + cut.k;
        const int c0 = cut.owner(ub);
        return make_int2(c0, n <= Tune::kWholeTiles ? 1 : cut.owner(ub + n - 1) - c0 + 1);
    };
    const int c = tid;
    CtaPlan out{};
    out.begin.x = -1;
    if (cut.total > 0 && cut.m) {                          // m CTAs for each unit
        if (c < cut.parts) {
            End a = unit_at(p, cut, c / cut.m);
            const SeqUnits<M> u = seq_units<M>(p, a.b, sm.rows[a.b]);
            const int n = u.tiles(a.pr), k = c % cut.m;
            const int2 share = share_of(a, u, n, c / cut.m);
            auto at = [&](int k) { return k > share.y ? n : int((long long)n * k / share.y); };   // beyond the last: nothing
            out.begin = make_int4(a.b, a.h, a.pr, at(k));
            out.end = make_int4(a.b, a.h, a.pr, at(k + 1));
            out.first_cta = share.x;
            out.first_pieces = out.last_pieces = share.y;
        }
    } else if (cut.total > 0) {                            // even ranges: one ends where the next begins
        int2 share = make_int2(0, 0);
        if (c < cut.parts) {
            End e = find<M>(p, cut, sm.rows, cut.bound(c));
            const SeqUnits<M> u = seq_units<M>(p, e.b, sm.rows[e.b]);
            const int n = u.tiles(e.pr);
            // Short units stay whole: the cut moves to the nearer end of one, and both neighbours see it there
            if (n <= Tune::kWholeTiles) e.j = 2 * e.j < n ? 0 : n;
            share = share_of(e, u, n, 0);
            out.begin = make_int4(e.b, e.h, e.pr, e.j);
        }
        sm.ends[c] = c < cut.parts ? out.begin : make_int4(cut.B, 0, 0, 0);
        sm.pieces[c] = share.y;
        __syncthreads();
        if (c < cut.parts) {
            const bool last = c + 1 >= cut.parts;
            out.end = last ? make_int4(cut.B, 0, 0, 0) : sm.ends[c + 1];
            out.first_cta = share.x;
            out.first_pieces = share.y;
            out.last_pieces = last ? 0 : sm.pieces[c + 1];
        }
    }
    if (c < p.ctas) {
        if (out.begin.x >= 0) {
            const SeqRows& r = sm.rows[out.begin.x];
            out.rows = make_int4(r.row0, r.n, r.live, r.S);
        }
        const_cast<CtaPlan*>(p.plan)[c] = out;
    }
    // ---- the groups' units of 256 rows, for the merge
    if (M == kChunkShared && !p.row_tiles && is_group<M>(p, 0)) {
        const long long n = cut.total > 0 ? (long long)cut.Hkv * cut.units[cut.B] : 0;
        for (int i = tid; i < n; i += kThreads) {
            const End e = unit_at(p, cut, i);
            if (!is_group<M>(p, e.b)) break;               // the sequences' come behind them
            const SeqUnits<M> u = seq_units<M>(p, e.b, sm.rows[e.b]);
            const_cast<int2*>(p.units)[i] = share_of(e, u, u.tiles(e.pr), i);
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
    if (M == kChunkShared) lay_out_groups(p, a.groups, sm.groups, first);
    if (a.launches == 0) return;
    if (p.row_tiles) lay_out_ranges<M, TuneFew>(p, sm.cut, first);
    else lay_out_ranges<M, TuneUnits>(p, sm.cut, first);
}

}  // namespace

cudaError_t launch_chunk_plan(const PlanParams& p, ChunkMode mode, cudaStream_t s) {
    for (int i = 0; i < p.launches; ++i) {
        const ChunkParams& q = p.launch[i];
        if ((mode == kChunkShared ? q.entries : q.B) > kChunkMaxBatch || q.ctas < 1 || q.ctas > kChunkMaxCtas)
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
