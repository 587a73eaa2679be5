// Shared device helpers and launch parameter blocks of libtreespec.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "treespec.h"

namespace treespec {

// Tree nodes per sequence.  A node's ancestor-or-self set is kAncWords 64-bit words
// (word w holds nodes 64w .. 64w+63): one word covers the 64-node trees of the radar
// page's single-word mask, two cover trees of up to 128 nodes.
constexpr int kMaxNodes = 128;
constexpr int kStreamMaxBatch = 256;   // persistent two-tile attention: sequences per call
constexpr int kStreamMaxCtas = 1024;   // persistent two-tile attention: CTAs (one per SM)
constexpr int kAncWords = 2;
constexpr int kAbsent = TREESPEC_ABSENT;   // parent entry of a padding slot past the end of a smaller tree
constexpr size_t kWsAlign = 256;
// Every wait inside a kernel gives up after this long (nanoseconds), sets
// TREESPEC_STATUS_TIMEOUT and winds the CTA down.
constexpr uint64_t kDefaultWaitNs = 2000000000ull;

__host__ __device__ inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Programmatic dependent launch between the tree prologue and the attention kernel that
// follows it on the stream.  The prologue lets the next grid launch at once; the
// attention kernel, launched with the programmatic-serialisation attribute, waits at its
// first instruction until the prologue has finished and its writes are visible, so only
// the launch and the CTAs' start overlap the prologue.  Launched without the attribute,
// the wait returns at once.
__device__ __forceinline__ void grid_dep_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// bf16 <-> f32 on raw bit patterns (bf16 is the high half of an f32).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) {
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return uint16_t((u >> 16) | 0x40u);   // NaN stays NaN
    u += 0x7fffu + ((u >> 16) & 1u);
    return uint16_t(u >> 16);
}

// Bits sh .. sh+31 of a 128-bit ancestor set {a0, a1} (bit j of the set = node j), as one
// 32-bit word; positions outside 0..127 read as 0.  sh may be negative (down to -31).
__device__ __forceinline__ uint32_t anc_bits32(uint64_t a0, uint64_t a1, int sh) {
    if (sh <= -32 || sh >= 128) return 0u;
    if (sh < 0) return uint32_t(a0 << (-sh));
    if (sh >= 64) return uint32_t(a1 >> (sh - 64));
    uint64_t w = a0 >> sh;
    if (sh > 32) w |= a1 << (64 - sh);
    return uint32_t(w);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------------------------ attention

// Workspace of tree_attn_verify (offsets in bytes from the workspace base).
struct AttnLayout {
    size_t status, anc, lens, nn, ml, acc, flags, total;
};

struct AttnPlan {
    int kernel;          // TREESPEC_KERNEL_SIMT / _TC / _TC_PAIR / _TC_2SM / _TC_STREAM
    int num_splits;
    int split_tokens;
    int rows_per_block;
    int row_blocks;
    int merge;
    int stream_ctas;     // _TC_STREAM: persistent CTAs (one per SM)
};

struct AttnParams {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* page_table;
    const int32_t* prefix_lens;   // caller's array (read by the prologue only)
    const int32_t* parents;       // caller's array (read by the prologue only)
    void* out;
    uint32_t* status;
    uint64_t* anc;                // [B][N][kAncWords] ancestor-or-self sets
    int32_t* lens;                // [B] validated prefix lengths, -1 = invalid sequence
    int32_t* nn;                  // [B] nodes of each tree: parent entries before the first kAbsent
    float* part_ml;               // [B][Hkv][splits][R][2]  (m in log2 units, l)
    float* part_acc;              // [B][Hkv][splits][R][D]
    int B, N, Hq, Hkv, G, R, D, ps, max_pages, num_pool_pages;
    int num_splits, split_tokens, rows_per_block, row_blocks, merge;
    float scale_log2;             // log2(e) / sqrt(D)
    int stream_ctas;              // persistent two-tile kernel: CTAs (one per SM)
    int32_t* stream_flags;        // persistent two-tile kernel: [2 * CTAs][2] a piece's partial is written
                                  // (slot, query tile); zeroed by the prologue
    uint64_t wait_ns;             // bound of the tensor-core kernels' pipeline waits (kDefaultWaitNs unless a test shortens it)
};

// ------------------------------------------------------------------ accept

struct AcceptLayout {
    size_t status, amax, stats, izs, total;
};

struct AcceptParams {
    const float* logits;
    const int32_t* tokens;
    const float* probs;
    const int32_t* parents;
    const float* uniforms;
    int32_t* path;
    int32_t* len;
    int32_t* bonus;
    uint32_t* status;
    int32_t* amax;    // [B][N]   lowest argmax of each target row
    float* stats;     // [B][N][2] (M2, S): max of logits*c and sum of 2^(logits*c - M2)
    float* izs;       // [B][N][64] 1/Z_1.. of the sibling residual chain of each row (0: Z = 0)
    int B, N, V;
    float temperature;
    float c;          // log2(e) / temperature
    int sms;          // SMs of the device (the cluster size of the walk depends on B / sms)
    int probs_on_host;  // draft_probs is host memory read over the CPU-GPU link: fetch a draft
                        // row only where a child is rejected, never ahead
};

// A kernel's dynamic shared-memory limit, set at its first launch on each device (the
// attribute belongs to the function and the device; setting it again costs a microsecond).
// `done`: a bit per device, one such word for each kernel.
template <class Kernel>
inline cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Kernel launchers (each returns cudaGetLastError() of its launch).
cudaError_t launch_tree_prologue(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_simt(const AttnParams& p, int dtype, cudaStream_t s);
cudaError_t launch_attn_tc(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_tc_2sm(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_tc_pair(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_tc_stream(const AttnParams& p, cudaStream_t s);
bool attn_tc_supported(int dtype, int D);
// TMA map of a K or V page pool [P][16][Hkv][D] bf16, one page x 64 head dims per box
bool make_pool_map(CUtensorMap* map, const void* base, int Hkv, long long pool_tokens, int D = 128);
// TMA map of an 8-bit pool of codes [P][16][Hkv][D], one page of one head per box, not swizzled
bool make_code_map(CUtensorMap* map, const void* base, int Hkv, long long pool_tokens, int D);
cudaError_t launch_attn_merge(const AttnParams& p, int dtype, cudaStream_t s);
cudaError_t launch_accept(const AcceptParams& p, int mode, cudaStream_t s, int* kernels);

// KV commit (tree_kv_commit)
struct CommitParams {
    void* k;
    void* v;
    const int32_t* page_table;
    const int32_t* prefix_lens;
    const int32_t* path;
    const int32_t* len;
    int32_t* new_lens;
    uint32_t* status;
    float* k_scales;   // [P][Hkv][16] of 8-bit pools, else NULL
    float* v_scales;
    int B, N, Hkv, D, ps, max_pages, num_pool_pages, elem;   // elem: bytes per element
};
cudaError_t launch_kv_commit(const CommitParams& p, cudaStream_t s);

// Appending new tokens (tree_chunk_append)
struct AppendParams {
    const void* q;
    const void* k;
    const void* v;
    long long q_stride, k_stride, v_stride;   // elements from one token to the next
    void* q_out;
    void* k_pages;
    void* v_pages;
    float* k_scales;
    float* v_scales;
    const int32_t* page_table;
    const int32_t* prefix_lens;
    const int32_t* offsets;
    const int32_t* positions;                 // or NULL: logical positions
    const float* q_norm;
    const float* k_norm;
    const float* inv_freq;
    uint32_t* status;
    int B, T, Hq, Hkv, D, max_pages, num_pool_pages, rot, layout;
    float eps, rope_scale;
    int sms;
};
cudaError_t launch_chunk_append(const AppendParams& p, int dtype, int kv_dtype, cudaStream_t s);

// Attention of packed chunks, or of a batch of trees over 8-bit pools
constexpr int kPage = 16;                     // tokens per page
constexpr int kChunkMaxBatch = 1024;          // persistent tensor-core form: sequences per call
constexpr int kChunkMaxCtas = 1024;           // persistent tensor-core form: CTAs
struct ChunkLayout {
    size_t status, cleared, anc, lens, nn, ml, acc, total;   // [status, cleared): zeroed before every call
};
struct ChunkParams {
    const void* q;
    const void* k;
    const void* v;
    const float* k_scales;
    const float* v_scales;
    const int32_t* page_table;
    const int32_t* prefix_lens;
    const int32_t* offsets;                   // [B + 1]; NULL: a batch of trees
    const uint64_t* anc;                      // trees: ancestor sets, checked lengths and node counts
    const int32_t* lens;                      //        of the prologue
    const int32_t* nn;
    void* out;
    uint32_t* status;
    float* part_ml;                           // SIMT: [splits][T][Hq][2], acc [splits][T][Hq][D]
    float* part_acc;                          // persistent: [2 CTAs][256][2] and [2 CTAs][256][D]
    int32_t* counters;                        // persistent: [CTAs][8] warps that finished a piece of the unit that
                                              // the CTA cut, zero at launch
    int B, T, N, Hq, Hkv, G, D, ps, max_pages, num_pool_pages;
    int num_splits, split_tokens, rows_block; // SIMT
    int ctas, tpq, inv_g;                     // persistent: CTAs; tokens per 128-row query tile, 128 / G; ceil(2^16 / G)
    float scale_log2;
    uint64_t wait_ns;
};
cudaError_t launch_chunk_simt(const ChunkParams& p, int dtype, int kv_dtype, cudaStream_t s);
// the smallest row block whose CTA still has 8 warps, `elem` bytes per K/V element
int chunk_simt_min_rows(int D, int elem);
cudaError_t launch_chunk_tc(const ChunkParams& p, int kv_dtype, cudaStream_t s);
bool chunk_tc_supported(int dtype, int batch, long long pool_tokens);
cudaError_t launch_chunk_merge(const ChunkParams& p, int dtype, cudaStream_t s);

// Rows of a sequence's new tokens: the first row, the rows, those of them that hold a
// token (a padded tree's other rows are zeros), and the prefix length (-1: the sequence is
// invalid and its rows are zeros).  Offsets that decrease or leave [0, T] give no rows.
struct SeqRows {
    int row0, n, live, S;
};
__device__ __forceinline__ SeqRows seq_rows(const ChunkParams& p, int b) {
    SeqRows r;
    if (!p.offsets) {
        r.row0 = b * p.N;
        r.n = p.N;
        r.S = p.lens[b];
        r.live = p.nn[b];
        return r;
    }
    const int o0 = p.offsets[b], o1 = p.offsets[b + 1];
    const bool ok = o0 >= 0 && o1 >= o0 && o1 <= p.T;
    r.row0 = ok ? o0 : 0;
    r.n = r.live = ok ? o1 - o0 : 0;
    const int S = p.prefix_lens[b];
    r.S = S >= 0 && (long long)S + r.n <= (long long)p.max_pages * kPage ? S : -1;
    return r;
}
// Whether sequence b's lengths are what the call allows (trees: the prologue checks them).
__device__ __forceinline__ bool seq_ok(const ChunkParams& p, int b) {
    if (!p.offsets) return true;
    const int o0 = p.offsets[b], o1 = p.offsets[b + 1], S = p.prefix_lens[b];
    return o0 >= 0 && o1 >= o0 && o1 <= p.T && S >= 0 && (long long)S + (o1 - o0) <= (long long)p.max_pages * kPage;
}

// two e4m3 codes -> two floats (exact; NaN codes give NaN)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}
// two floats -> two e4m3 codes, to nearest even; `lo` in the low byte
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}

// Draft-tree construction (tree_draft_step, tree_rerank)
constexpr int kMaxTopk = 16;          // branching per step
constexpr int kMaxFrontier = 16;      // frontier rows per step (1 or topk)
constexpr int kMaxDraftNodes = 1024;  // node arrays of a sequence (root + steps * topk)
constexpr int kMaxDraftSplits = 16;   // CTAs that share one frontier row's vocabulary
struct DraftParams {
    const float* logprobs;            // [B][F][V]
    const int32_t* frontier_in;       // [B][F] node ids (unused at step 0)
    int32_t* frontier_out;            // [B][k]
    int32_t* node_parent;             // [B][M]
    int32_t* node_token;
    float* node_score;
    int32_t* tk_tok;                  // workspace: [B][F][S][k] top-k of each part of a row
    float* tk_lp;
    uint32_t* status;
    int B, F, V, k, step, M;
    int S, chunk;                     // a row's vocabulary in S parts of `chunk` tokens (one CTA each)
};
struct RerankParams {
    const int32_t* node_parent;
    const int32_t* node_token;
    const float* node_score;
    const int32_t* pool;              // [B][P] eligible node ids, or NULL: every node
    int P;
    int32_t* parents;                 // [B][N]
    int32_t* tokens;
    uint32_t* status;
    int B, M, N;
};
cudaError_t launch_draft_step(const DraftParams& p, cudaStream_t s);
cudaError_t launch_rerank(const RerankParams& p, cudaStream_t s);
size_t attn_simt_smem_bytes(int dtype, int D, int R_block);

}  // namespace treespec
