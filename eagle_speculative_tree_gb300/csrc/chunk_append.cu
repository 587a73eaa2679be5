// tree_chunk_append: norm, rotary positions and the write into the page pools, one pass.
//
// Every head of every new token is read once and written once; nothing else moves, so
// memory bounds it (and the latency of one dependent chain when the tokens are few), as
// long as the instructions per element are few too.  A CTA takes TPB tokens and some or all
// of their Hq + 2 Hkv heads; D / 8 lanes hold a head, two chunks of 4 elements each.  In the
// half layout a lane's chunks are rot / 2 elements apart, so that both elements of its four
// pairs are its own and the rotation needs no exchange; the sum of squares and the largest
// magnitude are a few shuffles.  Pairs of elements go through packed float32 instructions.
//   1. the first heads' loads are issued, then, while they are in flight:
//   2. one warp per token finds its sequence (32-way search of chunk_offsets), position
//      and page;
//   3. the threads turn position x frequency into TPB x rot / 2 cosines and sines in
//      shared memory, shared by all heads of a token;
//   4. norm, rotation, rounding, store, a lane's four cosines and sines in registers for
//      all heads of the token.
// The angle: inv_freq / (2 pi) is held as a 64-bit fraction of a turn, position times it
// modulo 2^64 is the exact fraction of the turn (the product of two integers), and its
// top 32 bits go to sincospi.  A float32 product would be off by 2^-24 of the whole angle:
// 0.004 rad at position 65536.
#include "common.cuh"

namespace treespec {

namespace {

constexpr float kScaleMin = 7.8886090522101181e-31f;   // 2^-100, the scale of an all-zero head

// inv_freq in turns per position, as a fraction of 2^64 (modulo whole turns).  f = m 2^(e - 150)
// with a 24-bit m, and 2 / pi = C 2^-96, so f / (2 pi) 2^64 = m C 2^(e - 184).  96 bits of 2 / pi
// leave f below 2^24 an error under 2^-73 of a turn per position.
__device__ __forceinline__ uint64_t turns_fixed(float f) {
    const uint32_t u = __float_as_uint(f);
    const int ex = int((u >> 23) & 255u);
    const uint64_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
    // C = floor(2^97 / pi) in words of 32 bits; m C in 120 bits, hi and lo
    const uint64_t p0 = m * 0xFC2757D1u;
    const uint64_t p1 = m * 0x4E441529u + (p0 >> 32);
    const uint64_t hi = m * 0xA2F9836Eu + (p1 >> 32);
    const uint64_t lo = (p1 << 32) | uint32_t(p0);
    const int s = 184 - (ex ? ex : 1);                   // right shift of the product
    uint64_t t;
    if (s >= 128) t = 0;
    else if (s >= 64) t = hi >> (s - 64);
    else if (s > 0) t = (lo >> s) | (hi << (64 - s));
    else if (s > -64) t = lo << (-s);
    else t = 0;
    return (u >> 31) ? 0ull - t : t;
}

// Two chunks of 4 elements as loaded.
template <typename T>
struct Chunks;
template <>
struct Chunks<uint16_t> {
    uint2 a, b;
    __device__ __forceinline__ void load(const uint16_t* p, int ca, int cb) {
        a = *reinterpret_cast<const uint2*>(p + ca);
        b = *reinterpret_cast<const uint2*>(p + cb);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
        x[4] = bf16_lo(b.x); x[5] = bf16_hi(b.x); x[6] = bf16_lo(b.y); x[7] = bf16_hi(b.y);
    }
};
template <>
struct Chunks<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, int ca, int cb) {
        a = *reinterpret_cast<const float4*>(p + ca);
        b = *reinterpret_cast<const float4*>(p + cb);
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
__device__ __forceinline__ void store_chunks(uint16_t* p, int ca, int cb, const float (&x)[8]) {
    *reinterpret_cast<uint2*>(p + ca) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
    *reinterpret_cast<uint2*>(p + cb) = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void store_chunks(float* p, int ca, int cb, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p + ca) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + cb) = make_float4(x[4], x[5], x[6], x[7]);
}

// Packed float32 pairs: one instruction for two elements.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// largest magnitude, NaN if either is one
__device__ __forceinline__ float max_abs(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
    return d;
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

// TPB tokens, U heads per thread at a time (those of the next token are loaded while the
// current one's are worked on).
template <typename T, bool E4M3, int D, int TPB, int U, int kThreads>
__global__ void __launch_bounds__(kThreads) chunk_append_kernel(const AppendParams p, int heads_per_cta) {
    constexpr int LPH = D / 8;                           // lanes per head
    constexpr int GRP = kThreads / LPH;                  // heads at a time
    __shared__ RowInfo info[TPB];
    __shared__ __align__(16) float cs[TPB][2][D / 2];    // cosines, sines
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int l = tid % LPH, grp = tid / LPH;
    const int r2 = p.rot >> 1;
    const bool half = p.layout == TREESPEC_ROPE_HALF;
    // the lane's chunks: in the half layout 4 l and 4 l + rot / 2 where those turn, and the
    // elements behind the rotated ones in order; else neighbours
    const bool turns = half ? 4 * l < r2 : 8 * l < p.rot;
    const int ca = half && turns ? 4 * l : 8 * l, cb = half && turns ? 4 * l + r2 : 8 * l + 4;
    const long long t0 = (long long)blockIdx.x * TPB;
    const int H = p.Hq + 2 * p.Hkv;
    const int h_lo = blockIdx.y * heads_per_cta, h_hi = min(H, h_lo + heads_per_cta);
    const int ntok = int(min((long long)TPB, p.T - t0));

    // heads h0 + u GRP + grp, u < U, of token tk
    Chunks<T> in[U];
    auto fetch = [&](int tk, int h0) {
        const long long t = t0 + tk;
        const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
        const T* k = static_cast<const T*>(p.k) + t * p.k_stride - p.Hq * D;
        const T* v = static_cast<const T*>(p.v) + t * p.v_stride - (p.Hq + p.Hkv) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * GRP + grp;
            if (h < h_hi) in[u].load((h < p.Hq ? q : h < p.Hq + p.Hkv ? k : v) + h * D, ca, cb);
        }
    };
    fetch(0, h_lo);

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
                const int pos = p.positions ? p.positions[t] : 0;
                if (pos >= 0) {
                    if (S < 0 || at >= (long long)p.max_pages * kPage) {
                        if (blockIdx.y == 0) atomicOr(p.status, TREESPEC_STATUS_BAD_LENGTH);
                    } else {
                        const int page = p.page_table[size_t(b) * p.max_pages + (at >> 4)];
                        if (page < 0 || page >= p.num_pool_pages) {
                            if (blockIdx.y == 0) atomicOr(p.status, TREESPEC_STATUS_BAD_PAGE);
                        } else {
                            r.slot = (long long)page * kPage + (at & 15);
                            r.pos = p.positions ? pos : int(at);   // at lies in the page table: below 2^30
                        }
                    }
                }
            }
            info[tk] = r;
        }
    }
    __syncthreads();
    if (r2) {
        for (int e = tid; e < ntok * (D / 2); e += kThreads) {
            const int tk = e / (D / 2), j = e % (D / 2);
            if (j >= r2) continue;
            const float f = p.inv_freq[j];
            const uint64_t a = turns_fixed(f) * uint64_t(uint32_t(info[tk].pos));
            const float half_turns = float(int32_t(a >> 32)) * 4.656612873077393e-10f;   // 2^-31
            float s, c;
            sincospif(half_turns, &s, &c);
            if (!isfinite(f)) s = c = __int_as_float(0x7fc00000);
            cs[tk][0][j] = c * p.rope_scale;
            cs[tk][1][j] = s * p.rope_scale;
        }
        __syncthreads();
    }

    const bool norms = p.q_norm || p.k_norm;
    for (int tk = 0; tk < ntok; ++tk) {
        const RowInfo r = info[tk];
        float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turns) {                                     // frequencies 4 l .. 4 l + 3, in either layout
            c4 = *reinterpret_cast<const float4*>(&cs[tk][0][4 * l]);
            s4 = *reinterpret_cast<const float4*>(&cs[tk][1][4 * l]);
        }
        for (int h0 = h_lo; h0 < h_hi; h0 += U * GRP) {
            Chunks<T> cur[U];
#pragma unroll
            for (int u = 0; u < U; ++u) cur[u] = in[u];
            if (h0 + U * GRP < h_hi) fetch(tk, h0 + U * GRP);
            else if (tk + 1 < ntok) fetch(tk + 1, h_lo);
            if (r.slot < 0) continue;                    // the same for the whole CTA
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h0 + u * GRP >= h_hi) break;         // the same for the whole CTA
                const int h = h0 + u * GRP + grp;
                const bool have = h < h_hi;
                const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
                float x[8];
                cur[u].get(x);
                if (norms && __any_sync(0xffffffffu, !is_v)) {
                    float a0 = 0.f, a1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; i += 2) fma2(a0, a1, x[i], x[i + 1], x[i], x[i + 1], a0, a1);
                    float ss = a0 + a1;
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float* w = is_v ? nullptr : is_q ? p.q_norm : p.k_norm;
                    if (w) {
                        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                        const float4 wa = __ldg(reinterpret_cast<const float4*>(w + ca));
                        const float4 wb = __ldg(reinterpret_cast<const float4*>(w + cb));
#pragma unroll
                        for (int i = 0; i < 8; i += 2) mul2(x[i], x[i + 1], x[i], x[i + 1], inv, inv);
                        mul2(x[0], x[1], x[0], x[1], wa.x, wa.y);
                        mul2(x[2], x[3], x[2], x[3], wa.z, wa.w);
                        mul2(x[4], x[5], x[4], x[5], wb.x, wb.y);
                        mul2(x[6], x[7], x[6], x[7], wb.z, wb.w);
                    }
                }
                if (turns && !is_v) {
                    if (half) {                          // (x[i], x[i + 4])
                        float y[4], z[4];
                        mul2(y[0], y[1], x[4], x[5], -s4.x, -s4.y);
                        mul2(y[2], y[3], x[6], x[7], -s4.z, -s4.w);
                        mul2(z[0], z[1], x[0], x[1], s4.x, s4.y);
                        mul2(z[2], z[3], x[2], x[3], s4.z, s4.w);
                        fma2(x[0], x[1], x[0], x[1], c4.x, c4.y, y[0], y[1]);
                        fma2(x[2], x[3], x[2], x[3], c4.z, c4.w, y[2], y[3]);
                        fma2(x[4], x[5], x[4], x[5], c4.x, c4.y, z[0], z[1]);
                        fma2(x[6], x[7], x[6], x[7], c4.z, c4.w, z[2], z[3]);
                    } else {                             // (x[2 i], x[2 i + 1])
                        const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a = x[2 * i], b = x[2 * i + 1];
                            x[2 * i] = fmaf(a, cc[i], -(b * sn[i]));
                            x[2 * i + 1] = fmaf(b, cc[i], a * sn[i]);
                        }
                    }
                }
                const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
                if constexpr (E4M3) {
                    if (__any_sync(0xffffffffu, have && !is_q)) {
                        float mx = max_abs(max_abs(max_abs(x[0], x[1]), max_abs(x[2], x[3])),
                                           max_abs(max_abs(x[4], x[5]), max_abs(x[6], x[7])));
#pragma unroll
                        for (int o = LPH / 2; o > 0; o >>= 1) mx = max_abs(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        if (have && !is_q) {
                            float sc = mx * (1.f / 448.f);
                            if (sc < kScaleMin) sc = kScaleMin;
                            const float inv = 1.f / sc;  // at most 2^100; 0 for a head with an infinity
#pragma unroll
                            for (int i = 0; i < 8; i += 2) mul2(x[i], x[i + 1], x[i], x[i + 1], inv, inv);
                            unsigned char* dst = static_cast<unsigned char*>(is_v ? p.v_pages : p.k_pages) +
                                                 (r.slot * p.Hkv + hk) * D;
                            *reinterpret_cast<uint32_t*>(dst + ca) =
                                uint32_t(f32x2_to_e4m3x2(x[0], x[1])) | uint32_t(f32x2_to_e4m3x2(x[2], x[3])) << 16;
                            *reinterpret_cast<uint32_t*>(dst + cb) =
                                uint32_t(f32x2_to_e4m3x2(x[4], x[5])) | uint32_t(f32x2_to_e4m3x2(x[6], x[7])) << 16;
                            if (l == 0)
                                (is_v ? p.v_scales : p.k_scales)[((r.slot >> 4) * p.Hkv + hk) * kPage + (r.slot & 15)] = sc;
                        }
                    }
                    if (have && is_q) store_chunks(static_cast<T*>(p.q_out) + ((t0 + tk) * p.Hq + h) * D, ca, cb, x);
                } else if (have) {
                    T* dst = is_q ? static_cast<T*>(p.q_out) + ((t0 + tk) * p.Hq + h) * D
                                  : static_cast<T*>(is_v ? p.v_pages : p.k_pages) + (r.slot * p.Hkv + hk) * D;
                    store_chunks(dst, ca, cb, x);
                }
            }
        }
    }
}

// Launch shapes, three heads per thread at a time in all but the first (five measured
// slower nearly everywhere: 2048 tokens x 80 heads 28.7 us against 24.6, 13114 tokens x 36 heads
// into 8 bits 60.1 against 52.6; faster by 3% for 13114 x 80 in bf16):
//   few tokens: one CTA per token and group of heads, so that the latency is that of one head
//   (1 token x 48 heads: 6.3 us with its status word's clearing, 2 us of it the kernel's own chain);
//   up to 32 tokens per SM: CTAs of 256 threads, 2 tokens each once there are 8 per SM (2048 tokens x
//   80 heads 22.6 us; 4 tokens 24.6, 4 tokens by 128 threads 26.7, 8 tokens 27.0);
//   more: CTAs of 128 threads, 4 tokens each, which leave more of an SM's registers in use at once (13114
//   tokens x 48 heads, 8-bit: 63.5 us = 4.7 TB/s, 68.6 with 256 threads).
template <typename T, bool E4M3, int D>
cudaError_t launch_typed(const AppendParams& p, cudaStream_t s) {
    const int H = p.Hq + 2 * p.Hkv;
    constexpr int GRP = 256 / (D / 8);
    const int rounds = (H + GRP - 1) / GRP;              // of GRP heads by 256 threads
    if ((long long)p.T * rounds <= 2ll * p.sms)
        chunk_append_kernel<T, E4M3, D, 1, 1, 256><<<dim3(unsigned(p.T), unsigned(rounds)), 256, 0, s>>>(p, GRP);
    else if (p.T < 8 * p.sms)
        chunk_append_kernel<T, E4M3, D, 1, 3, 256><<<dim3(unsigned(p.T)), 256, 0, s>>>(p, H);
    else if (p.T < 32 * p.sms)
        chunk_append_kernel<T, E4M3, D, 2, 3, 256><<<dim3(unsigned((p.T + 1ll) / 2)), 256, 0, s>>>(p, H);
    else
        chunk_append_kernel<T, E4M3, D, 4, 3, 128><<<dim3(unsigned((p.T + 3ll) / 4)), 128, 0, s>>>(p, H);
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
