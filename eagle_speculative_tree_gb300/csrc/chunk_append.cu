// tree_chunk_append: norm, rotary positions and the write into the page pools, one pass.
//
// Every head of every new token is read once and written once; nothing else moves, so
// memory bounds it (and the latency of one dependent chain when the tokens are few).  A
// CTA takes TPB tokens and some or all of their Hq + 2 Hkv heads; D / 8 lanes hold a head,
// 8 elements each (16 bytes of bf16), so the sum of squares, the largest magnitude and the
// partner of a rotated pair are a few shuffles inside those lanes.
//   1. the first heads' loads are issued, then, while they are in flight:
//   2. one warp per token finds its sequence (32-way search of chunk_offsets), position
//      and page;
//   3. the threads turn position x frequency into TPB x rot / 2 cosines and sines in
//      shared memory, shared by all heads of a token;
//   4. norm, rotation, rounding, store.
// The angle: inv_freq / (2 pi) is held as a 64-bit fraction of a turn, position times it
// modulo 2^64 is the exact fraction of the turn (the product of two integers), and its
// top 32 bits go to sincospi.  A float32 product would be off by 2^-24 of the whole angle:
// 0.004 rad at position 65536.
#include "common.cuh"

namespace treespec {

namespace {

constexpr int kThreads = 256;
constexpr float kScaleMin = 7.8886090522101181e-31f;   // 2^-100, the scale of an all-zero head

// inv_freq in turns per position, as a fraction of 2^64 (modulo whole turns).  f = m 2^(e - 150)
// with a 24-bit m, and 2 / pi = C 2^-64, so f / (2 pi) 2^64 = m C 2^(e - 152).
__device__ __forceinline__ uint64_t turns_fixed(float f) {
    const uint32_t u = __float_as_uint(f);
    const int ex = int((u >> 23) & 255u);
    const uint64_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const uint64_t C = 0xA2F9836E4E441529ull;            // floor(2^65 / pi)
    const uint64_t lo = m * C, hi = __umul64hi(m, C);
    const int s = 152 - (ex ? ex : 1);                   // right shift of the 88-bit product
    uint64_t t;
    if (s >= 128) t = 0;
    else if (s >= 64) t = hi >> (s - 64);
    else if (s > 0) t = (lo >> s) | (hi << (64 - s));
    else if (s > -64) t = lo << (-s);
    else t = 0;
    return (u >> 31) ? 0ull - t : t;
}

template <typename T>
struct Vec8;                                             // 8 elements of a head as loaded
template <>
struct Vec8<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
        x[4] = bf16_lo(a.z); x[5] = bf16_hi(a.z); x[6] = bf16_lo(a.w); x[7] = bf16_hi(a.w);
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// The sequence of row t: the last b with offsets[b] <= t, by a 32-way search of one warp.
// Whatever the offsets hold, 0 <= b < B; where t is not in that sequence (it belongs to
// none, or the offsets are out of order) the first sequence that has it, if there is one.
__device__ __forceinline__ int find_seq(const int32_t* off, int B, int T, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;                                   // candidates lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane * step < n && off[at] <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        n = min(step, n - last * step);
    }
    auto has = [&](int b) { return off[b] >= 0 && off[b] <= t && t < off[b + 1] && off[b + 1] <= T; };
    if (has(lo)) return lo;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        const unsigned m = __ballot_sync(0xffffffffu, b < B && has(b));
        if (m) return b0 + __ffs(m) - 1;
    }
    return lo;
}

struct RowInfo {
    long long slot;      // token slot in the pools, -1: the row is left out
    int pos;             // rotary position
};

// U: heads in flight per thread.
template <typename T, bool E4M3, int D, int TPB, int U>
__global__ void __launch_bounds__(kThreads) chunk_append_kernel(const AppendParams p, int heads_per_cta) {
    constexpr int LPH = D / 8;                           // lanes per head
    constexpr int GRP = kThreads / LPH;                  // heads at a time
    __shared__ RowInfo info[TPB];
    __shared__ float2 cs[TPB][D / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int l = tid % LPH, grp = tid / LPH;
    const long long t0 = (long long)blockIdx.x * TPB;
    const int H = p.Hq + 2 * p.Hkv;
    const int h_lo = blockIdx.y * heads_per_cta, h_hi = min(H, h_lo + heads_per_cta);
    const int nh = h_hi - h_lo;
    const int ntok = int(min((long long)TPB, p.T - t0));

    auto src = [&](int tk, int h) -> const T* {
        const long long t = t0 + tk;
        if (h < p.Hq) return static_cast<const T*>(p.q) + t * p.q_stride + h * D + l * 8;
        if (h < p.Hq + p.Hkv) return static_cast<const T*>(p.k) + t * p.k_stride + (h - p.Hq) * D + l * 8;
        return static_cast<const T*>(p.v) + t * p.v_stride + (h - p.Hq - p.Hkv) * D + l * 8;
    };
    // work item e of this thread group: token e / nhg, head h_lo + (e % nhg) * GRP + grp
    const int nhg = (nh + GRP - 1) / GRP;
    const int items = ntok * nhg;
    Vec8<T> in[U];
    auto fetch = [&](int e0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u;
            const int h = h_lo + (e % nhg) * GRP + grp;
            if (e < items && h < h_hi) in[u].load(src(e / nhg, h));
        }
    };
    fetch(0);

    if (blockIdx.x == 0 && blockIdx.y == 0) {            // the lengths, checked once
        bool bad = false;
        for (int b = tid; b < p.B; b += kThreads) {
            const int o0 = p.offsets[b], o1 = p.offsets[b + 1];
            bad |= o0 < 0 || o1 < o0 || o1 > p.T || p.prefix_lens[b] < 0;
        }
        if (bad) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
    }
    for (int tk = warp; tk < ntok; tk += kThreads / 32) {
        const int t = int(t0) + tk;
        const int b = find_seq(p.offsets, p.B, p.T, t);
        if (lane == 0) {
            RowInfo r{-1, 0};
            const int o0 = p.offsets[b], o1 = p.offsets[b + 1], S = p.prefix_lens[b];
            if (o0 >= 0 && o0 <= t && t < o1 && o1 <= p.T) {
                const long long at = (long long)S + (t - o0);
                const int pos = p.positions ? p.positions[t] : int(at);
                if (pos >= 0) {
                    if (S < 0 || at >= (long long)p.max_pages * kPage) {
                        if (blockIdx.y == 0) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
                    } else {
                        const int page = p.page_table[size_t(b) * p.max_pages + (at >> 4)];
                        if (page < 0 || page >= p.num_pool_pages) {
                            if (blockIdx.y == 0) atomicOr(p.status, TREESPEC_STATUS_BAD_PAGE);
                        } else {
                            r.slot = (long long)page * kPage + (at & 15);
                            r.pos = pos;
                        }
                    }
                }
            }
            info[tk] = r;
        }
    }
    __syncthreads();
    const int r2 = p.rot >> 1;
    // a lane reads 8 (half layout) or 4 consecutive frequencies: kept so that the lanes of a
    // head read neighbouring words
    const bool half = p.layout == TREESPEC_ROPE_HALF;
    auto place = [&](int j) { return half ? (j & 7) * (D / 16) + (j >> 3) : (j & 3) * (D / 8) + (j >> 2); };
    for (int e = tid; e < ntok * r2; e += kThreads) {
        const int tk = e / r2, j = e - tk * r2;
        const float f = p.inv_freq[j];
        const uint64_t a = turns_fixed(f) * uint64_t(uint32_t(info[tk].pos));
        const float half_turns = float(int32_t(a >> 32)) * 4.656612873077393e-10f;   // 2^-31
        float s, c;
        sincospif(half_turns, &s, &c);
        if (!isfinite(f)) s = c = __int_as_float(0x7fc00000);
        cs[tk][place(j)] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    __syncthreads();

    // this lane's pairs: half layout, elements 8 l .. 8 l + 7 turn with the lane r2 / 8 away
    const int l2 = r2 >> 3;
    const bool turns = l < 2 * l2;
    const bool second = l >= l2;                         // the b of its pairs (half layout)
    const int jbase = half ? 8 * (second ? l - l2 : l) : 4 * l;
    const int partner = (lane & ~(LPH - 1)) + (!half || !turns ? l : second ? l - l2 : l + l2);

    for (int e0 = 0; e0 < items; e0 += U) {
        if (e0) fetch(e0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u;
            if (e >= items) break;                       // the same for the whole CTA
            const int tk = e / nhg, h = h_lo + (e % nhg) * GRP + grp;
            const RowInfo r = info[tk];
            if (r.slot < 0) continue;                    // the same for the whole CTA
            const bool have = h < h_hi;
            float x[8];
            if (have) in[u].get(x);
            else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
            }
            const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
            const float* w = is_v ? nullptr : is_q ? p.q_norm : p.k_norm;
            if (p.q_norm || p.k_norm) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (w) {
                    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                    const float4 w0 = *reinterpret_cast<const float4*>(w + 8 * l);
                    const float4 w1 = *reinterpret_cast<const float4*>(w + 8 * l + 4);
                    const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * ww[i];
                }
            }
            if (r2) {
                if (half) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
                    if (turns && !is_v) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 c = cs[tk][place(jbase + i)];
                            x[i] = fmaf(x[i], c.x, second ? y[i] * c.y : -(y[i] * c.y));
                        }
                    }
                } else if (turns && !is_v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 c = cs[tk][place(jbase + i)];
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = fmaf(a, c.x, -(b * c.y));
                        x[2 * i + 1] = fmaf(b, c.x, a * c.y);
                    }
                }
            }
            if constexpr (E4M3) {
                float mx = 0.f;                          // largest magnitude, NaN kept: compared as bits
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mx = __uint_as_float(max(__float_as_uint(mx), __float_as_uint(x[i]) & 0x7fffffffu));
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1)
                    mx = __uint_as_float(max(__float_as_uint(mx), __shfl_xor_sync(0xffffffffu, __float_as_uint(mx), o)));
                if (!have) continue;
                if (!is_q) {
                    const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
                    float sc = mx / 448.f;
                    if (sc < kScaleMin) sc = kScaleMin;
                    uint32_t c[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        c[i] = uint32_t(f32x2_to_e4m3x2(x[4 * i] / sc, x[4 * i + 1] / sc)) |
                               uint32_t(f32x2_to_e4m3x2(x[4 * i + 2] / sc, x[4 * i + 3] / sc)) << 16;
                    unsigned char* dst = static_cast<unsigned char*>(is_v ? p.v_pages : p.k_pages);
                    *reinterpret_cast<uint2*>(dst + (r.slot * p.Hkv + hk) * D + l * 8) = make_uint2(c[0], c[1]);
                    if (l == 0)
                        (is_v ? p.v_scales : p.k_scales)[((r.slot >> 4) * p.Hkv + hk) * kPage + (r.slot & 15)] = sc;
                    continue;
                }
            } else if (!have) {
                continue;
            }
            if (is_q) {
                store8(static_cast<T*>(p.q_out) + ((t0 + tk) * p.Hq + h) * D + l * 8, x);
            } else {
                const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
                store8(static_cast<T*>(is_v ? p.v_pages : p.k_pages) + (r.slot * p.Hkv + hk) * D + l * 8, x);
            }
        }
    }
}

template <typename T, bool E4M3, int D>
cudaError_t launch_typed(const AppendParams& p, cudaStream_t s) {
    constexpr int GRP = kThreads / (D / 8);
    const int H = p.Hq + 2 * p.Hkv;
    const long long rounds = (H + GRP - 1) / GRP;        // of GRP heads
    if (p.T * rounds <= 2ll * p.sms) {                   // few tokens: GRP heads of one token per CTA
        chunk_append_kernel<T, E4M3, D, 1, 1><<<dim3(unsigned(p.T), unsigned(rounds)), kThreads, 0, s>>>(p, GRP);
    } else {
        constexpr int TPB = 2;
        const unsigned blocks = unsigned((p.T + (long long)TPB - 1) / TPB);
        chunk_append_kernel<T, E4M3, D, TPB, 4><<<dim3(blocks), kThreads, 0, s>>>(p, H);
    }
    return cudaGetLastError();
}

template <typename T, bool E4M3>
cudaError_t launch_dim(const AppendParams& p, cudaStream_t s) {
    return p.D == 64 ? launch_typed<T, E4M3, 64>(p, s) : launch_typed<T, E4M3, 128>(p, s);
}

}  // namespace

cudaError_t launch_chunk_append(const AppendParams& p, int dtype, int kv_dtype, cudaStream_t s) {
    const bool q8 = kv_dtype == TREESPEC_DTYPE_E4M3;
    if (dtype == TREESPEC_DTYPE_F32) return q8 ? launch_dim<float, true>(p, s) : launch_dim<float, false>(p, s);
    return q8 ? launch_dim<uint16_t, true>(p, s) : launch_dim<uint16_t, false>(p, s);
}

}  // namespace treespec
