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
    if constexpr (M == kChunkShared) grid_dep_wait();      // the attention kernel
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
        if (p.skip[b].x == 0) from = p.num_splits;
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

// The same behind the tensor-core kernels: a row's own part is in rows_*[1], the group's in rows_*[0] or,
// where its unit was cut, in the slots of its pieces: piece k in slot 2 c0 + 1 (k = 0) or 2 (c0 + k), rows
// as in chunk_tc.cuh (token it of a query tile and head g of the group: row r = it G + g in place
// 32 (r % 4) + r / 4).  Bound by latency: a warp's row has one chain of loads to its states (a lane for
// each), and then the states' rows, eight of them on their way at a time; some 4 us behind the
// attention kernels for 2048 rows of 9 states.
template <int D>
__global__ void __launch_bounds__(256) group_merge_kernel(const ChunkParams p) {
    constexpr int DS = D / 32, kAhead = 8;
    const long long gw = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    grid_dep_wait();                                       // the attention kernels
    if (p.published && gw == 0 && lane == 0) *p.published = 0;   // read by them alone
    if (gw >= (long long)p.T * p.Hq) return;
    const int t = int(gw / p.Hq), hq = int(gw % p.Hq);
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
    const int2 skip = p.skip[b];
    if (skip.x == 0) return;                               // a row of no group: in `out` already
    const SeqRows sq = seq_rows(p, b);
    const int i = t - sq.row0;
    if (i < 0 || i >= sq.n) return;
    float acc[DS], lsum = 0.f;
#pragma unroll
    for (int e = 0; e < DS; ++e) acc[e] = 0.f;
    if (sq.S >= 0 && i < sq.live) {
        const size_t rows = size_t(p.T) * p.Hq;
        const float2* rows_ml = reinterpret_cast<const float2*>(p.rows_ml);
        const float2* part_ml = reinterpret_cast<const float2*>(p.part_ml);
        int2 unit = make_int2(0, 1);
        int place = 0;
        if (p.units) {
            const int4 g = p.gtab[skip.y];
            const int tok = t - g.x, pr = tok / p.tpu, it = tok - pr * p.tpu, np = (g.y + p.tpu - 1) / p.tpu;
            unit = p.units[p.Hkv * p.group_units[skip.y] + (hq / p.G) * np + pr];
            const int tile = it / p.tpq, r = (it - tile * p.tpq) * p.G + hq % p.G;
            place = tile * 128 + (r & 3) * 32 + (r >> 2);
        }
        // state k of the row: 0 its own, then the group's
        const int n = 1 + unit.y;
        auto ml_of = [&](int k) -> float2 {
            if (k == 0) return rows_ml[rows + gw];
            if (unit.y == 1) return rows_ml[gw];
            return part_ml[size_t(k == 1 ? 2 * unit.x + 1 : 2 * (unit.x + k - 1)) * 256 + place];
        };
        auto acc_of = [&](int k) -> const float* {
            if (k == 0) return p.rows_acc + (rows + gw) * D;
            if (unit.y == 1) return p.rows_acc + gw * D;
            return p.part_acc + (size_t(k == 1 ? 2 * unit.x + 1 : 2 * (unit.x + k - 1)) * 256 + place) * D;
        };
        float top = -INFINITY;
        for (int k0 = 0; k0 < n; k0 += 32) top = fmaxf(top, warp_max(k0 + lane < n ? ml_of(k0 + lane).x : -INFINITY));
        for (int k0 = 0; k0 < n; k0 += 32) {
            const float2 x = k0 + lane < n ? ml_of(k0 + lane) : make_float2(-INFINITY, 0.f);
            // left out: a state without a weight above 0, not one whose weight rounds to 0 (a NaN stays one)
            const float w = x.x == -INFINITY ? (x.y == 0.f ? -1.f : 1.f) : exp2f(x.x - top);
            lsum += warp_sum(w < 0.f ? 0.f : x.y * w);
            const int kn = min(32, n - k0);
            for (int k = 0; k < kn; k += kAhead) {
                float y[kAhead][DS];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const float* src = acc_of(k0 + min(k + a, kn - 1)) + lane * DS;
                    if constexpr (DS == 4) {
                        const float4 z = *reinterpret_cast<const float4*>(src);
                        y[a][0] = z.x; y[a][1] = z.y; y[a][2] = z.z; y[a][3] = z.w;
                    } else {
                        const float2 z = *reinterpret_cast<const float2*>(src);
                        y[a][0] = z.x; y[a][1] = z.y;
                    }
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const float wa = __shfl_sync(0xffffffffu, w, (k + a) & 31);
                    if (k + a < kn && wa >= 0.f) {
#pragma unroll
                        for (int e = 0; e < DS; ++e) acc[e] = fmaf(y[a][e], wa, acc[e]);
                    }
                }
            }
        }
        lsum = 1.f / lsum;
    }
#pragma unroll
    for (int e = 0; e < DS; ++e) store_out<uint16_t>(p.out, size_t(gw) * D + lane * DS + e, acc[e] * lsum);
}

template <class Kernel>
cudaError_t launch_rows(Kernel kern, const ChunkParams& p, bool dependent, cudaStream_t s) {   // a warp per row
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(((long long)p.T * p.Hq + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_merge(const ChunkParams& p, ChunkMode mode, cudaStream_t s) {
    if (mode == kChunkShared) return launch_rows(chunk_merge_kernel<T, D, kChunkShared>, p, true, s);
    return launch_rows(chunk_merge_kernel<T, D, kChunkPlain>, p, false, s);
}

}  // namespace

int chunk_simt_min_rows(int D, int elem) {
    const int ts = 160 * 1024 / (4 * 32 * (D * elem + 16));
    return 64 / (ts >= 4 ? 4 : ts >= 2 ? 2 : 1);
}

template cudaError_t launch_chunk_simt<kChunkPlain>(const ChunkParams& p, int dtype, int kv_dtype, cudaStream_t s);

cudaError_t launch_group_merge(const ChunkParams& p, cudaStream_t s) {
    return launch_rows(p.D == 64 ? group_merge_kernel<64> : group_merge_kernel<128>, p, true, s);
}

cudaError_t launch_chunk_merge(const ChunkParams& p, ChunkMode mode, int dtype, cudaStream_t s) {
    if (dtype == TREESPEC_DTYPE_F32) return p.D == 64 ? launch_merge<float, 64>(p, mode, s) : launch_merge<float, 128>(p, mode, s);
    return p.D == 64 ? launch_merge<uint16_t, 64>(p, mode, s) : launch_merge<uint16_t, 128>(p, mode, s);
}

}  // namespace treespec
