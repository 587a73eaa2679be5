// Attention of packed chunks on CUDA cores without a window or shared prefixes, and the merge of
// partial states.
#include "chunk_simt.cuh"

namespace treespec {

namespace {

// Partial states of the splits -> out: M = max m, out = sum acc 2^(m - M) / sum l 2^(m - M).
// One warp per (token, query head); rows that belong to no sequence are left alone.  Shared prefixes:
// the splits of the group's part lie before those of the row's own, and rows of sequences that share
// nothing have only the latter (in one split: they are in `out` already).
template <typename T, int D, ChunkMode M>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p) {
    constexpr int DS = D / 32;
    const long long gw = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (gw >= (long long)p.T * p.Hq) return;
    const int t = int(gw / p.Hq);
    int b;
    if (p.offsets) {
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.offsets[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = lo;
    } else {
        b = t / p.N;
    }
    const SeqRows sq = seq_rows(p, b);
    const int i = t - sq.row0;
    if (i < 0 || i >= sq.n) return;
    int from = 0, to = p.num_splits;
    if constexpr (M == kChunkShared) {
        to = 2 * p.num_splits;
        if (p.skip[b] == 0) from = p.num_splits;
        if (to - from == 1) return;
    }
    float acc[DS];
#pragma unroll
    for (int e = 0; e < DS; ++e) acc[e] = 0.f;
    float inv = 0.f;
    if (sq.S >= 0 && i < sq.live) {
        float mm = -INFINITY, lsum = 0.f;
        for (int s = from; s < to; ++s) mm = fmaxf(mm, p.part_ml[((size_t(s) * p.T) * p.Hq + gw) * 2]);
        for (int s = from; s < to; ++s) {
            const size_t pr = size_t(s) * p.T * p.Hq + gw;
            const float ms = p.part_ml[pr * 2], ls = p.part_ml[pr * 2 + 1];
            if (ms == -INFINITY && ls == 0.f) continue;
            const float f = ms == -INFINITY ? 1.f : exp2f(ms - mm);
            lsum = fmaf(ls, f, lsum);
            const float* src = p.part_acc + pr * D + lane * DS;
#pragma unroll
            for (int e = 0; e < DS; ++e) acc[e] = fmaf(src[e], f, acc[e]);
        }
        inv = 1.f / lsum;
    }
#pragma unroll
    for (int e = 0; e < DS; ++e) store_out<T>(p.out, size_t(gw) * D + lane * DS + e, acc[e] * inv);
}

template <typename T, int D>
cudaError_t launch_merge(const ChunkParams& p, ChunkMode mode, cudaStream_t s) {
    const unsigned blocks = unsigned(((long long)p.T * p.Hq + 7) / 8);
    if (mode == kChunkShared) chunk_merge_kernel<T, D, kChunkShared><<<blocks, 256, 0, s>>>(p);
    else chunk_merge_kernel<T, D, kChunkPlain><<<blocks, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int chunk_simt_min_rows(int D, int elem) {
    const int ts = 160 * 1024 / (4 * 32 * (D * elem + 16));
    return 64 / (ts >= 4 ? 4 : ts >= 2 ? 2 : 1);
}

template cudaError_t launch_chunk_simt<kChunkPlain>(const ChunkParams& p, int dtype, int kv_dtype, cudaStream_t s);

cudaError_t launch_chunk_merge(const ChunkParams& p, ChunkMode mode, int dtype, cudaStream_t s) {
    if (dtype == TREESPEC_DTYPE_F32) return p.D == 64 ? launch_merge<float, 64>(p, mode, s) : launch_merge<float, 128>(p, mode, s);
    return p.D == 64 ? launch_merge<uint16_t, 64>(p, mode, s) : launch_merge<uint16_t, 128>(p, mode, s);
}

}  // namespace treespec
