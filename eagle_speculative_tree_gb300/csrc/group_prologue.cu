// Groups of sequences that share a prefix: checks the caller's groups and lays out what the
// attention kernels run over.
//
// Group g is the sequences group_offsets[g] .. group_offsets[g + 1] - 1; their first
// shared_lens[g] logical tokens are the same.  Of these, whole KV tiles are computed for all
// rows of the group at once; what is left behind the last whole tile, fewer than 64 tokens,
// stays with each sequence.  A group shares nothing where it has fewer than two sequences with
// new tokens, where one of them has a shorter prefix (BAD_LENGTH) and, as the rows of a
// group have to be packed, anywhere in a batch whose offsets are out of order.
#include "common.cuh"

namespace treespec {

namespace {

constexpr int kThreads = 1024;

__global__ void __launch_bounds__(kThreads) group_prologue_kernel(const ChunkParams p, const GroupParams g) {
    __shared__ int first[kMaxGroups], count[kMaxGroups], least[kMaxGroups];   // of the group's sequences with rows
    __shared__ int off[kMaxGroups + 1], share[kMaxGroups];
    __shared__ int bad_groups, bad_chunks;
    grid_dep_release();                                    // the attention kernel may launch; it waits for this grid
    const int tid = threadIdx.x, NG = p.groups;
    if (tid == 0) bad_groups = bad_chunks = 0;
    for (int k = tid; k <= NG; k += kThreads) off[k] = g.group_offsets[k];
    for (int k = tid; k < NG; k += kThreads) {
        first[k] = least[k] = INT32_MAX;
        count[k] = 0;
    }
    __syncthreads();
    for (int k = tid; k < NG; k += kThreads)
        if (off[k] < 0 || off[k + 1] < off[k] || off[k + 1] > p.B) bad_groups = 1;
    if (p.offsets)
        for (int b = tid; b < p.B; b += kThreads)
            if (p.offsets[b] < 0 || p.offsets[b + 1] < p.offsets[b] || p.offsets[b + 1] > p.T) bad_chunks = 1;
    __syncthreads();
    const bool fine = !bad_groups && !bad_chunks;
    auto group_of = [&](int b) -> int {                    // the last group that begins at or before b, or -1
        if (!fine || b < off[0] || b >= off[NG]) return -1;
        int lo = 0, hi = NG;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (off[mid] <= b) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    for (int b = tid; b < p.B; b += kThreads) {
        const int k = group_of(b);
        if (k < 0) continue;
        const SeqRows r = seq_rows(p, b);
        if (r.n == 0) continue;
        atomicMin(&first[k], b);
        atomicMin(&least[k], r.S);
        atomicAdd(&count[k], 1);
    }
    __syncthreads();
    for (int k = tid; k < NG; k += kThreads) {
        const int want = g.shared_lens[k];
        const bool ok = fine && want >= 0 && (count[k] == 0 || want <= least[k]);
        if (!ok && !bad_chunks) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
        int4 e = make_int4(0, 0, 0, 0);
        if (fine) e.x = p.offsets ? p.offsets[off[k]] : off[k] * p.N;
        share[k] = 0;
        if (ok && count[k] >= 2 && want >= kSharedTile) {
            e.y = (p.offsets ? p.offsets[off[k + 1]] : off[k + 1] * p.N) - e.x;
            e.z = share[k] = want / kSharedTile * kSharedTile;
            e.w = first[k];
        }
        g.gtab[k] = e;
    }
    __syncthreads();
    for (int b = tid; b < p.B; b += kThreads) {
        const int k = group_of(b);
        g.skip[b] = k < 0 ? 0 : share[k];
    }
}

}  // namespace

cudaError_t launch_group_prologue(const ChunkParams& p, const GroupParams& g, cudaStream_t s) {
    group_prologue_kernel<<<1, kThreads, 0, s>>>(p, g);
    return cudaGetLastError();
}

}  // namespace treespec
