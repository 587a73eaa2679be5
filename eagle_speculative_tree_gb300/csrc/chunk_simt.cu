// Attention of packed chunks (tree_chunk_attn), and of trees over 8-bit pools, on CUDA
// cores: any dtype, head dim 64 or 128, any group size.
//
// A CTA holds up to RB = 16, 32 or 64 query rows of one kv head (the host takes the
// size that the batch's mean rows per sequence fill; row r = token i * G + g of a
// sequence's new tokens) and one split of the sequence's logical tokens, and keeps the usual partial
// state per row: m = max s, l = sum 2^(s - m), acc = sum 2^(s - m) V, with s = q . K
// log2(e) / sqrt(D), in float32.  Row i sees the prefix and, of the new tokens, j <= i
// (a chunk) or those in its ancestor set (a tree).  Which row block of which sequence a
// CTA takes follows from the packed offsets alone: sequence b owns the blocks from
// floor(offsets[b] G / RB) + b on, which leaves room for ceil(n_b G / RB) of them.
//
// Layout of a CTA: RW row-warps (8 rows each) x TS token slices (32 tokens each); QK^T has
// lane = token, PV lane = a slice of the head; K/V arrive by cp.async in two stages.  8-bit
// K/V stay codes in shared memory: the K scale multiplies the finished dot product, the V
// scale the probability.
#include "common.cuh"

namespace treespec {

namespace {

constexpr int kRows = 64;                // query rows per CTA, at most
constexpr int kMaxSmem = 224 * 1024;     // dynamic shared memory a CTA may ask for, beside its static 1 KB

enum KvKind { kKvF32, kKvBf16, kKvE4m3 };

template <KvKind KV, int D>
struct Cfg {
    static constexpr int EB = KV == kKvF32 ? 4 : KV == kKvBf16 ? 2 : 1;
    static constexpr int EPV = 16 / EB;          // elements per 16-byte vector
    static constexpr int VPR = D * EB / 16;      // vectors per K/V row
    static constexpr int ROWB = D * EB + 16;     // padded shared-memory row
    static constexpr int DS = D / 32;            // head elements per lane in PV
    // token slices: two stages of K and V within 160 KB, at most 4
    static constexpr int TSMAX = (160 * 1024) / (4 * 32 * ROWB) >= 4 ? 4 : (160 * 1024) / (4 * 32 * ROWB);
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(uint32_t(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes));
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(uint32_t(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes));
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float& a, float& b) {
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(h));
}

template <KvKind KV>
__device__ __forceinline__ void vec_to_f32(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (KV == kKvF32) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (KV == kKvBf16) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        } else {
            f16x2_to_f32(e4m3x2_to_f16x2(uint16_t(w[i])), f[4 * i], f[4 * i + 1]);
            f16x2_to_f32(e4m3x2_to_f16x2(uint16_t(w[i] >> 16)), f[4 * i + 2], f[4 * i + 3]);
        }
    }
}

// DS consecutive elements of a V row
template <KvKind KV, int DS>
__device__ __forceinline__ void load_slice(const unsigned char* src, float* f) {
    if constexpr (KV == kKvF32) {
        if constexpr (DS == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            f[0] = v.x; f[1] = v.y;
        }
    } else if constexpr (KV == kKvBf16) {
#pragma unroll
        for (int e = 0; e < DS; e += 2) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(src + 2 * e);
            f[e] = bf16_lo(v);
            f[e + 1] = bf16_hi(v);
        }
    } else {
#pragma unroll
        for (int e = 0; e < DS; e += 2)
            f16x2_to_f32(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(src + e)), f[e], f[e + 1]);
    }
}

template <typename T>
__device__ __forceinline__ float load_q(const void* q, size_t idx) {
    if constexpr (sizeof(T) == 4) return static_cast<const float*>(q)[idx];
    else return bf16_to_f32(static_cast<const uint16_t*>(q)[idx]);
}
template <typename T>
__device__ __forceinline__ void store_out(void* out, size_t idx, float v) {
    if constexpr (sizeof(T) == 4) static_cast<float*>(out)[idx] = v;
    else static_cast<uint16_t*>(out)[idx] = f32_to_bf16_rne(v);
}

struct Shape {
    int RW, TS, nwarps, TT;
    size_t q_bytes, kv_bytes, pt_bytes, sc_bytes, smem;
};
template <KvKind KV, int D>
__host__ __device__ inline Shape shape_of(int rows) {
    using C = Cfg<KV, D>;
    Shape s;
    s.RW = rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
    int ts = 8 / s.RW;
    s.TS = ts > C::TSMAX ? C::TSMAX : ts;
    s.nwarps = s.RW * s.TS;
    s.TT = 32 * s.TS;
    s.q_bytes = size_t(s.RW) * 8 * D * 4;
    const size_t stages = size_t(4) * s.TT * C::ROWB, merge = size_t(s.nwarps) * 8 * (D + 2) * 4;
    s.kv_bytes = stages > merge ? stages : merge;
    s.pt_bytes = size_t(s.nwarps) * 32 * 8 * 4;
    s.sc_bytes = KV == kKvE4m3 ? size_t(4) * s.TT * 4 : 0;
    s.smem = s.q_bytes + s.kv_bytes + s.pt_bytes + s.sc_bytes;
    return s;
}

// The block's first row on the list of row blocks: where sequence b's blocks begin.
__device__ __forceinline__ long long block_base(const ChunkParams& p, int b) {
    const int RB = p.rows_block;
    return p.offsets ? (long long)max(0, p.offsets[b]) * p.G / RB + b : (long long)b * ((p.N * p.G + RB - 1) / RB);
}

// float32 K/V take 139 KB of shared memory, so one CTA fits an SM: told so, the compiler uses the
// registers there are (5 short chunks of 64-element heads: 26.7 us, 29 with 128 registers and spills)
template <typename T, KvKind KV, int D>
__global__ void __launch_bounds__(256, KV == kKvF32 ? 1 : 0) chunk_simt_kernel(const ChunkParams p) {
    using C = Cfg<KV, D>;
    constexpr int DS = C::DS;
    extern __shared__ __align__(16) unsigned char smem[];
    const Shape sh = shape_of<KV, D>(p.rows_block);
    const int RW = sh.RW, TS = sh.TS, TT = sh.TT, nthr = sh.nwarps * 32;
    float* Qs = reinterpret_cast<float*>(smem);
    unsigned char* kv = smem + sh.q_bytes;
    float* Pt = reinterpret_cast<float*>(kv + sh.kv_bytes);
    float* Sc = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(Pt) + sh.pt_bytes);   // [stage][K, V][TT]
    __shared__ uint64_t anc_s[kRows][kAncWords];
    __shared__ unsigned long long at_s[kRows];           // element of q and out where a row begins
    __shared__ float fin_s[4][kRows];                    // weights of the token slices of a row in the result
    __shared__ int seq_s;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rw = warp % RW, ts = warp / RW;
    const int h = blockIdx.y, split = blockIdx.z;
    const long long unit = blockIdx.x;
    if (unit == 0 && h == 0 && split == 0) {             // the lengths, checked once
        bool bad = false;
        for (int b = tid; b < p.B; b += nthr) bad |= !seq_ok(p, b);
        if (bad) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
    }
    if (tid == 0) {                                      // the last b whose blocks begin at or before unit
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (block_base(p, mid) <= unit) lo = mid;
            else hi = mid;
        }
        seq_s = lo;
    }
    __syncthreads();
    const int b = seq_s;
    const SeqRows sq = seq_rows(p, b);
    const long long rb = unit - block_base(p, b);
    if (rb < 0 || rb * p.rows_block >= (long long)sq.n * p.G) return;
    const int r0 = int(rb) * p.rows_block;               // first row of the block in the sequence
    const int rows = min(p.rows_block, sq.n * p.G - r0);
    const int S = sq.S;
    // out / q element (local row lr, d)
    auto elem = [&](int lr) -> size_t {
        const int row = r0 + lr;
        return (size_t(sq.row0 + row / p.G) * p.Hq + h * p.G + row % p.G) * D;
    };
    auto part = [&](int lr) -> size_t {                  // partial of the row: [split][T][Hq]
        const int row = r0 + lr;
        return (size_t(split) * p.T + sq.row0 + row / p.G) * p.Hq + h * p.G + row % p.G;
    };
    for (int lr = tid; lr < rows; lr += nthr) at_s[lr] = elem(lr);
    __syncthreads();
    // last logical token any of the rows may see, and this split's share
    const int last_i = min((r0 + rows - 1) / p.G, sq.live - 1);
    const int L = S < 0 ? 0 : p.offsets ? S + last_i + 1 : S + sq.live;
    const int t0 = int(min((long long)L, (long long)split * p.split_tokens));
    const int t1 = p.num_splits == 1 ? L : int(min((long long)L, (long long)t0 + p.split_tokens));
    if (t0 >= t1) {                                      // nothing here: zeros, or an empty partial
        if (p.num_splits == 1) {
            for (int e = tid; e < rows * D; e += nthr) store_out<T>(p.out, at_s[e / D] + e % D, 0.f);
        } else {
            for (int lr = tid; lr < rows; lr += nthr) {
                p.part_ml[part(lr) * 2] = -INFINITY;
                p.part_ml[part(lr) * 2 + 1] = 0.f;
            }
        }
        return;
    }

    const int live_rows = min(rows, sq.live * p.G - r0);  // rows of a padded tree's other slots lie behind them
#pragma unroll 4
    for (int e = tid; e < RW * 8 * D; e += nthr) {
        const int lr = e / D;
        Qs[e] = lr < live_rows ? load_q<T>(p.q, at_s[lr] + e % D) * p.scale_log2 : 0.f;
    }
    if (!p.offsets) {
        for (int e = tid; e < rows * kAncWords; e += nthr)
            anc_s[e / kAncWords][e % kAncWords] =
                p.anc[(size_t(b) * p.N + (r0 + e / kAncWords) / p.G) * kAncWords + e % kAncWords];
    }

    const int* ptab = p.page_table + size_t(b) * p.max_pages;
    auto issue = [&](int tile, int stage) {
        const int base = t0 + tile * TT;
        unsigned char* Kd = kv + size_t(stage) * 2 * TT * C::ROWB;
        unsigned char* Vd = Kd + size_t(TT) * C::ROWB;
        // the tile's page ids, one load per warp: lane l has that of tokens base + 16 l
        const int at = base + kPage * lane;
        const int pages = lane < TT / kPage && at < t1 ? __ldg(ptab + at / kPage) : -1;
#pragma unroll 2
        for (int e = tid; e < TT * C::VPR; e += nthr) {  // a warp takes part in a round as a whole
            const int tt = e / C::VPR, vi = e % C::VPR;
            const int pos = base + tt;
            const int page = __shfl_sync(0xffffffffu, pages, tt / kPage);
            const unsigned char* ks = static_cast<const unsigned char*>(p.k);
            const unsigned char* vs = static_cast<const unsigned char*>(p.v);
            int bytes = 0;
            if (pos < t1) {
                if (page >= 0 && page < p.num_pool_pages) {
                    const size_t off = ((size_t(page) * kPage + pos % kPage) * p.Hkv + h) * (size_t(D) * C::EB) +
                                       size_t(vi) * 16;
                    ks += off;
                    vs += off;
                    bytes = 16;
                } else if (vi == 0) {
                    atomicOr(p.status, TREESPEC_STATUS_BAD_PAGE);
                }
            }
            cp_async16(Kd + tt * C::ROWB + vi * 16, ks, bytes);
            cp_async16(Vd + tt * C::ROWB + vi * 16, vs, bytes);
        }
        if constexpr (KV == kKvE4m3) {
            for (int tt = tid; tt < TT; tt += nthr) {
                const int pos = base + tt;
                size_t off = 0;
                int bytes = 0;
                if (pos < t1) {
                    const int page = ptab[pos / kPage];
                    if (page >= 0 && page < p.num_pool_pages) {
                        off = (size_t(page) * p.Hkv + h) * kPage + pos % kPage;
                        bytes = 4;
                    }
                }
                cp_async4(Sc + (stage * 2) * TT + tt, p.k_scales + off, bytes);
                cp_async4(Sc + (stage * 2 + 1) * TT + tt, p.v_scales + off, bytes);
            }
        }
        asm volatile("cp.async.commit_group;\n" ::);
    };

    float m[8], l[8], acc[8][DS];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < DS; ++e) acc[r][e] = 0.f;
    }
    const bool has_rows = rw * 8 < rows;
    const int ntiles = (t1 - t0 + TT - 1) / TT;
    float* pt_w = Pt + warp * 256;

    issue(0, 0);
    for (int tile = 0; tile < ntiles; ++tile) {
        if (tile + 1 < ntiles) issue(tile + 1, (tile + 1) & 1);
        else asm volatile("cp.async.commit_group;\n" ::);
        asm volatile("cp.async.wait_group 1;\n" ::);
        __syncthreads();
        if (has_rows) {
            const int stage = tile & 1;
            const unsigned char* Kd = kv + size_t(stage) * 2 * TT * C::ROWB;
            const unsigned char* Vd = Kd + size_t(TT) * C::ROWB;
            const int tt = ts * 32 + lane;
            const int pos = t0 + tile * TT + tt;
            float s[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) s[r] = 0.f;
            const unsigned char* krow = Kd + tt * C::ROWB;
            const float* qbase = Qs + rw * 8 * D;
#pragma unroll 4
            for (int d = 0; d < D; d += C::EPV) {
                float kf[C::EPV];
                vec_to_f32<KV>(*reinterpret_cast<const uint4*>(krow + d * C::EB), kf);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
#pragma unroll
                    for (int e = 0; e < C::EPV; e += 4) {
                        const float4 qv = *reinterpret_cast<const float4*>(qbase + r * D + d + e);
                        s[r] = fmaf(qv.x, kf[e], s[r]);
                        s[r] = fmaf(qv.y, kf[e + 1], s[r]);
                        s[r] = fmaf(qv.z, kf[e + 2], s[r]);
                        s[r] = fmaf(qv.w, kf[e + 3], s[r]);
                    }
                }
            }
            float vscale = 1.f;
            if constexpr (KV == kKvE4m3) {
                const float kscale = Sc[(stage * 2) * TT + tt];
                vscale = Sc[(stage * 2 + 1) * TT + tt];
#pragma unroll
                for (int r = 0; r < 8; ++r) s[r] *= kscale;
            }
            const int j = pos - S;                       // new token when >= 0
            unsigned seen_by = 0;                        // rows (of the warp's 8) that see this lane's token
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int lr = rw * 8 + r, i = (r0 + lr) / p.G;
                bool ok = pos < t1 && lr < rows && i < sq.live;
                if (ok && j >= 0) ok = p.offsets ? j <= i : (anc_s[lr][j >> 6] >> (j & 63)) & 1ull;
                if (ok) seen_by |= 1u << r;
                const float sv = ok ? s[r] : -INFINITY;
                const float mnew = fmaxf(m[r], warp_max(sv));
                const float alpha = (mnew == -INFINITY) ? 1.f : exp2f(m[r] - mnew);
                // while no score above -inf has come, 0 is subtracted: a score of -inf weighs 0, not NaN
                const float pv = ok ? exp2f(sv - (mnew == -INFINITY ? 0.f : mnew)) : 0.f;
                l[r] = fmaf(l[r], alpha, pv);
                m[r] = mnew;
#pragma unroll
                for (int e = 0; e < DS; ++e) acc[r][e] *= alpha;
                pt_w[lane * 8 + r] = KV == kKvE4m3 ? (ok ? pv * vscale : 0.f) : pv;
            }
            __syncwarp();
            const unsigned char* vrow = Vd + size_t(ts * 32) * C::ROWB + lane * DS * C::EB;
            // tokens that every row of the warp sees need no test: a value a row does not see
            // must not reach it even as 0 x NaN
            const bool all_seen = __all_sync(0xffffffffu, seen_by == 0xffu);
#pragma unroll 4
            for (int t = 0; t < 32; ++t) {
                float vf[DS];
                load_slice<KV, DS>(vrow + t * C::ROWB, vf);
                const float4 pa = *reinterpret_cast<const float4*>(pt_w + t * 8);
                const float4 pb = *reinterpret_cast<const float4*>(pt_w + t * 8 + 4);
                const float pr[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
                if (all_seen) {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
#pragma unroll
                        for (int e = 0; e < DS; ++e) acc[r][e] = fmaf(pr[r], vf[e], acc[r][e]);
                } else {
                    const unsigned who = __shfl_sync(0xffffffffu, seen_by, t);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        if (!((who >> r) & 1u)) continue;
#pragma unroll
                        for (int e = 0; e < DS; ++e) acc[r][e] = fmaf(pr[r], vf[e], acc[r][e]);
                    }
                }
            }
            __syncwarp();
        }
        __syncthreads();
    }
    asm volatile("cp.async.wait_group 0;\n" ::);

#pragma unroll
    for (int r = 0; r < 8; ++r) l[r] = warp_sum(l[r]);
    __syncthreads();
    float* scr = reinterpret_cast<float*>(kv);           // [nwarps][8][D + 2]
    if (has_rows) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float* dst = scr + size_t(warp * 8 + r) * (D + 2);
#pragma unroll
            for (int e = 0; e < DS; ++e) dst[lane * DS + e] = acc[r][e];
            if (lane == 0) {
                dst[D] = m[r];
                dst[D + 1] = l[r];
            }
        }
    }
    __syncthreads();
    // a row's state over the token slices, and what each slice's accumulators weigh in it
    for (int lr = tid; lr < rows; lr += nthr) {
        const int rwi = lr / 8, r = lr % 8;
        float mm = -INFINITY, lsum = 0.f;
        for (int t = 0; t < TS; ++t) mm = fmaxf(mm, scr[size_t((t * RW + rwi) * 8 + r) * (D + 2) + D]);
        for (int t = 0; t < TS; ++t) {
            const float* src = scr + size_t((t * RW + rwi) * 8 + r) * (D + 2);
            // a slice whose scores are all NaN has m = -inf and l = NaN: kept, not skipped
            const bool none = src[D] == -INFINITY && src[D + 1] == 0.f;
            // one without weight is left out (-1), not one whose weight rounds to 0: a NaN stays one
            const float f = none ? -1.f : src[D] == -INFINITY ? 1.f : exp2f(src[D] - mm);
            if (!none) lsum = fmaf(src[D + 1], f, lsum);
            fin_s[t][lr] = f;
        }
        if (p.num_splits == 1) {
            const float inv = 1.f / lsum;
            if (lsum == 0.f) fin_s[0][lr] = NAN;           // no token of a weight above 0: undefined
            else
                for (int t = 0; t < TS; ++t) fin_s[t][lr] *= inv;
        } else {
            p.part_ml[part(lr) * 2] = mm;
            p.part_ml[part(lr) * 2 + 1] = lsum;
        }
        at_s[lr] = p.num_splits == 1 ? at_s[lr] : part(lr) * D;
    }
    __syncthreads();
#pragma unroll 4
    for (int e = tid; e < rows * D; e += nthr) {
        const int lr = e / D, d = e % D;
        const float* src = scr + size_t(lr) * (D + 2) + d;   // slice t of the row: RW * 8 rows further each
        float a = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (t < TS && !(fin_s[t][lr] < 0.f)) a = fmaf(src[size_t(t) * RW * 8 * (D + 2)], fin_s[t][lr], a);
        if (p.num_splits == 1) store_out<T>(p.out, at_s[lr] + d, lr < live_rows ? a : 0.f);
        else p.part_acc[at_s[lr] + d] = a;
    }
}

// Partial states of the splits -> out: M = max m, out = sum acc 2^(m - M) / sum l 2^(m - M).
// One warp per (token, query head); rows that belong to no sequence are left alone.
template <typename T, int D>
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
    float acc[DS];
#pragma unroll
    for (int e = 0; e < DS; ++e) acc[e] = 0.f;
    float inv = 0.f;
    if (sq.S >= 0 && i < sq.live) {
        float mm = -INFINITY, lsum = 0.f;
        for (int s = 0; s < p.num_splits; ++s) mm = fmaxf(mm, p.part_ml[((size_t(s) * p.T) * p.Hq + gw) * 2]);
        for (int s = 0; s < p.num_splits; ++s) {
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

template <typename T, KvKind KV, int D>
cudaError_t launch_typed(const ChunkParams& p, cudaStream_t s) {
    const long long total_rows = (long long)p.T * p.G;
    const int RB = p.rows_block;
    if (RB != 16 && RB != 32 && RB != kRows) return cudaErrorInvalidValue;
    const long long units = p.offsets ? total_rows / RB + p.B : (long long)p.B * ((p.N * p.G + RB - 1) / RB);
    const Shape sh = shape_of<KV, D>(RB);
    if (sh.smem > size_t(kMaxSmem)) return cudaErrorInvalidValue;
    auto kern = chunk_simt_kernel<T, KV, D>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(kern, kMaxSmem, smem_set);
    if (e != cudaSuccess) return e;
    kern<<<dim3(unsigned(units), unsigned(p.Hkv), unsigned(p.num_splits)), sh.nwarps * 32, sh.smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int chunk_simt_min_rows(int D, int elem) {
    const int ts = 160 * 1024 / (4 * 32 * (D * elem + 16));
    return 64 / (ts >= 4 ? 4 : ts >= 2 ? 2 : 1);
}

cudaError_t launch_chunk_simt(const ChunkParams& p, int dtype, int kv_dtype, cudaStream_t s) {
    const bool d64 = p.D == 64;
    if (dtype == TREESPEC_DTYPE_F32) {
        if (kv_dtype == TREESPEC_DTYPE_E4M3)
            return d64 ? launch_typed<float, kKvE4m3, 64>(p, s) : launch_typed<float, kKvE4m3, 128>(p, s);
        return d64 ? launch_typed<float, kKvF32, 64>(p, s) : launch_typed<float, kKvF32, 128>(p, s);
    }
    if (kv_dtype == TREESPEC_DTYPE_E4M3)
        return d64 ? launch_typed<uint16_t, kKvE4m3, 64>(p, s) : launch_typed<uint16_t, kKvE4m3, 128>(p, s);
    return d64 ? launch_typed<uint16_t, kKvBf16, 64>(p, s) : launch_typed<uint16_t, kKvBf16, 128>(p, s);
}

cudaError_t launch_chunk_merge(const ChunkParams& p, int dtype, cudaStream_t s) {
    const long long blocks = ((long long)p.T * p.Hq + 7) / 8;
    if (dtype == TREESPEC_DTYPE_F32) {
        if (p.D == 64) chunk_merge_kernel<float, 64><<<unsigned(blocks), 256, 0, s>>>(p);
        else chunk_merge_kernel<float, 128><<<unsigned(blocks), 256, 0, s>>>(p);
    } else {
        if (p.D == 64) chunk_merge_kernel<uint16_t, 64><<<unsigned(blocks), 256, 0, s>>>(p);
        else chunk_merge_kernel<uint16_t, 128><<<unsigned(blocks), 256, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace treespec
