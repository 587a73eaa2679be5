// Host side of libtreespec: argument checks, the split planner, workspace layout and
// launches.  Every exported symbol is declared in include/treespec.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "common.cuh"

namespace treespec {
namespace {

std::atomic<uint64_t> g_launches{0};
std::atomic<uint64_t> g_wait_ns{kDefaultWaitNs};     // see treespec_set_wait_limit_ns
std::atomic<int> g_launch_error{0};                 // cudaError_t of the last rejected launch

// TREESPEC_ERR_LAUNCH for a launch (or memset, copy or wait) the runtime rejected, keeping the
// runtime's code.  The runtime also keeps it as the thread's last error, which the check after
// the next launch would take for that launch's own: it is cleared here.
int launch_failed(cudaError_t e) {
    cudaGetLastError();
    g_launch_error.store(int(e));
    return TREESPEC_ERR_LAUNCH;
}

constexpr int kDefaultSms = 152;
constexpr int kMaxDevices = 64;

struct DeviceInfo {
    int sms = 0;
    int cc_major = 0, cc_minor = 0;
};

// Per-device attributes, read once.  Returns false when no device is usable.
bool device_info(DeviceInfo* out) {
    static DeviceInfo cache[kMaxDevices];
    static std::mutex mu;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].sms == 0) {
        DeviceInfo d;
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        cache[dev] = d;
    }
    *out = cache[dev];
    return true;
}

int sm_count_or_default() {
    DeviceInfo d;
    return device_info(&d) ? d.sms : kDefaultSms;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The persistent two-tile kernel keeps the batch's 64-token tile offsets in shared memory
// and its tile positions (over row-block pairs, sequences and kv heads) as int32: at most
// kStreamMaxBatch sequences and fewer than 2^31 positions.
bool stream_fits(const treespec_attn_shape& s) {
    const long long tiles = ((long long)s.max_pages_per_seq * s.page_size + 63) / 64 + 3;   // + tree nodes
    const long long G = s.num_q_heads / s.num_kv_heads;
    const long long pairs = ((long long)s.num_nodes * G + 255) / 256;
    return s.batch <= kStreamMaxBatch && pairs * s.num_kv_heads * s.batch * tiles < (1ll << 31);
}

int check_attn_shape(const treespec_attn_shape* s) {
    if (!s) return TREESPEC_ERR_NULL_POINTER;
    if (s->dtype != TREESPEC_DTYPE_F32 && s->dtype != TREESPEC_DTYPE_BF16) return TREESPEC_ERR_DTYPE;
    if (s->batch < 1 || s->batch > 65535) return TREESPEC_ERR_SHAPE;
    if (s->num_nodes < 1 || s->num_nodes > kMaxNodes) return TREESPEC_ERR_SHAPE;
    if (s->num_kv_heads < 1 || s->num_q_heads < 1 || s->num_q_heads % s->num_kv_heads) return TREESPEC_ERR_SHAPE;
    if (s->head_dim != 64 && s->head_dim != 128) return TREESPEC_ERR_SHAPE;
    if (s->page_size != 16) return TREESPEC_ERR_SHAPE;
    if (s->max_pages_per_seq < 1 || s->num_pool_pages < 1) return TREESPEC_ERR_SHAPE;
    if ((long long)s->max_pages_per_seq * s->page_size > (1ll << 30)) return TREESPEC_ERR_SHAPE;
    const long long R = (long long)s->num_nodes * (s->num_q_heads / s->num_kv_heads);
    if (R > 4096 || (long long)s->num_kv_heads * ((R + 63) / 64) > 65535) return TREESPEC_ERR_SHAPE;
    if (s->kernel < TREESPEC_KERNEL_AUTO || s->kernel > TREESPEC_KERNEL_TC_STREAM) return TREESPEC_ERR_SHAPE;
    if (s->num_splits < 0) return TREESPEC_ERR_SHAPE;
    if (s->kernel >= TREESPEC_KERNEL_TC) {
        if (!attn_tc_supported(s->dtype, s->head_dim)) return TREESPEC_ERR_DTYPE;
        if ((long long)s->num_pool_pages * s->page_size >= (1ll << 31)) return TREESPEC_ERR_SHAPE;
    }
    if (s->kernel >= TREESPEC_KERNEL_TC_PAIR && ((R + 127) / 128) % 2 != 0) return TREESPEC_ERR_SHAPE;
    if (s->kernel == TREESPEC_KERNEL_TC_STREAM && !stream_fits(*s)) return TREESPEC_ERR_SHAPE;
    return TREESPEC_OK;
}

AttnPlan make_plan(const treespec_attn_shape& s, int sms) {
    AttnPlan p{};
    const int G = s.num_q_heads / s.num_kv_heads;
    const int R = s.num_nodes * G;
    const bool tc_ok = attn_tc_supported(s.dtype, s.head_dim) &&
                       (long long)s.num_pool_pages * s.page_size < (1ll << 31);
    // Tensor cores for every bf16 / head_dim 128 shape: measured faster than the CUDA-core
    // kernel from 16 rows per kv head up (rows are padded to the 128-row MMA tile).
    // Where the row blocks of a kv head pair up, a K/V tile should serve 256 rows: the
    // one-tile kernel's L2 reads bind first otherwise.  Of the two kernels that do that, the
    // CTA-pair kernel (256-row MMAs across two SMs) when the two-tile kernel's CTAs would
    // not fill the SMs once, the two-tile kernel (two 128-row tiles in one CTA) otherwise.
    // Measured at 64 q / 8 kv heads, 64 nodes, 8192-token prefixes (ms, CTA pair / two-tile /
    // one-tile): batch 2 0.080 / 0.088 / -, batch 8 0.149 / 0.169 / 0.169, batch 16
    // 0.279 / 0.243 / 0.315, batch 32 0.491 / 0.474 / 0.543.
    if (s.kernel >= TREESPEC_KERNEL_TC || (s.kernel == TREESPEC_KERNEL_AUTO && tc_ok)) {
        const long long rbs = (R + 127) / 128;
        const bool paired = rbs % 2 == 0;
        const long long pair_units = (long long)s.batch * s.num_kv_heads * (rbs / 2);
        const bool small = pair_units < sms;
        // the persistent form pays a merge of the cut units and a few us per unit change,
        // which two waves of two-tile CTAs or more amortise (measured: batch 32 0.460 ms
        // against 0.473, batch 16 0.255 against 0.250)
        const bool many = pair_units >= 2ll * sms;
        p.kernel = s.kernel != TREESPEC_KERNEL_AUTO ? s.kernel
                   : !paired                        ? TREESPEC_KERNEL_TC
                   : small                          ? TREESPEC_KERNEL_TC_2SM
                   : (many && stream_fits(s))       ? TREESPEC_KERNEL_TC_STREAM
                                                    : TREESPEC_KERNEL_TC_PAIR;
        p.rows_per_block = 128;
    } else {
        p.kernel = TREESPEC_KERNEL_SIMT;
        p.rows_per_block = R < 64 ? R : 64;
    }
    p.row_blocks = (R + p.rows_per_block - 1) / p.rows_per_block;
    const long long max_tokens = (long long)s.max_pages_per_seq * s.page_size;
    const int tile = 128;                       // split sizes are multiples of every tile size
    const bool tc = p.kernel != TREESPEC_KERNEL_SIMT;
    const long long units = (long long)s.batch * s.num_kv_heads *
                            (p.kernel == TREESPEC_KERNEL_TC_PAIR ? p.row_blocks / 2 : p.row_blocks);
    long long splits;
    if (s.num_splits > 0) {
        splits = s.num_splits;
    } else if (tc) {
        // One CTA fits an SM.  Split a sequence only as far as one wave of CTAs holds
        // (rounded down: a few CTAs past the SM count would run as a second wave), keep a
        // CTA's run at most 66 tiles (a ragged batch's longest sequences split into several
        // CTAs; an 8256-token one stays whole), and no chunk below two tiles: each split
        // costs a pipeline fill and its partials.  Measured against earlier rules: about two
        // CTAs per SM gave 32 x 8192 tokens at batch 8 0.192 ms against 0.147, 8 x 4096
        // tokens (32 kv heads) 0.131 against 0.116, 64 ragged sequences up to 32768 tokens
        // 0.774 against 0.751; rounding up gave the 64 q / 8 kv-head, 64-node shape 0.056 ms
        // at batch 1 (160 CTA-pair CTAs) against 0.044 (128) and 0.077 at batch 2 against 0.058.
        splits = units >= sms ? 1 : sms / units;
        const long long cap = 66ll * tile;
        splits = std::max(splits, (max_tokens + cap - 1) / cap);
        splits = std::min(splits, std::max(1ll, (max_tokens + 2 * tile - 1) / (2 * tile)));
        if (splits < 1) splits = 1;
    } else {
        const long long target = 2ll * sms;      // two waves of CTAs, then merge
        splits = (target + units - 1) / units;
        if (splits < 1) splits = 1;
    }
    long long chunk = (max_tokens + splits - 1) / splits;
    chunk = (chunk + tile - 1) / tile * tile;
    if (s.num_splits == 0 && !tc && chunk > 16384) chunk = 16384;   // bounded CTA length
    if (chunk < tile) chunk = tile;
    p.split_tokens = int(chunk);
    p.num_splits = int((max_tokens + chunk - 1) / chunk);
    if (p.num_splits > 65535) {
        p.num_splits = 65535;
        p.split_tokens = int((max_tokens + 65534) / 65535);
        p.split_tokens = (p.split_tokens + tile - 1) / tile * tile;
    }
    p.merge = p.num_splits > 1;
    if (p.kernel == TREESPEC_KERNEL_TC_STREAM) {   // no splits: the SMs share the tiles evenly
        p.num_splits = 1;
        p.split_tokens = int(std::min<long long>(max_tokens + 128, 1ll << 30));
        p.merge = 0;
        p.stream_ctas = std::min(sms, kStreamMaxCtas);
    }
    return p;
}

AttnLayout attn_layout(const treespec_attn_shape& s, const AttnPlan& p) {
    AttnLayout L{};
    const size_t R = size_t(s.num_nodes) * (s.num_q_heads / s.num_kv_heads);
    size_t off = 0;
    L.status = off;
    off += kWsAlign;
    L.anc = off;
    off = align_up(off + size_t(s.batch) * s.num_nodes * kAncWords * 8, kWsAlign);
    L.lens = off;
    off = align_up(off + size_t(s.batch) * 4, kWsAlign);
    L.nn = off;
    off = align_up(off + size_t(s.batch) * 4, kWsAlign);
    const size_t parts = p.merge ? size_t(s.batch) * s.num_kv_heads * p.num_splits * R : 0;
    L.ml = off;
    off = align_up(off + parts * 2 * 4, kWsAlign);
    L.acc = off;
    off = align_up(off + parts * s.head_dim * 4, kWsAlign);
    if (p.kernel == TREESPEC_KERNEL_TC_STREAM) {
        // two partial slots of 2 x 128 rows per CTA for the pieces of cut units, and their
        // ready flags
        const size_t rows = size_t(2) * p.stream_ctas * 256;
        L.ml = off;
        off = align_up(off + rows * 2 * 4, kWsAlign);
        L.acc = off;
        off = align_up(off + rows * s.head_dim * 4, kWsAlign);
        L.flags = off;
        off = align_up(off + size_t(2) * p.stream_ctas * 2 * 4, kWsAlign);
    }
    L.total = off;
    return L;
}

AcceptLayout accept_layout(int B, int N) {
    AcceptLayout L{};
    size_t off = 0;
    L.status = off;
    off += kWsAlign;
    L.amax = off;
    off = align_up(off + size_t(B) * N * 4, kWsAlign);
    L.stats = off;
    off = align_up(off + size_t(B) * N * 8, kWsAlign);
    L.izs = off;
    off = align_up(off + size_t(B) * N * kMaxNodes * 4, kWsAlign);
    L.total = off;
    return L;
}

int check_device() {
    DeviceInfo d;
    if (!device_info(&d)) return TREESPEC_ERR_DEVICE;
    if (d.cc_major != 10 || d.cc_minor != 3) return TREESPEC_ERR_DEVICE;
    return TREESPEC_OK;
}

}  // namespace
}  // namespace treespec

using namespace treespec;

extern "C" size_t treespec_attn_workspace_bytes(const treespec_attn_shape* shape) {
    if (check_attn_shape(shape) != TREESPEC_OK) return 0;
    return attn_layout(*shape, make_plan(*shape, sm_count_or_default())).total;
}

extern "C" int treespec_attn_plan_for(const treespec_attn_shape* shape, treespec_attn_plan* plan) {
    const int rc = check_attn_shape(shape);
    if (rc != TREESPEC_OK) return rc;
    if (!plan) return TREESPEC_ERR_NULL_POINTER;
    const AttnPlan p = make_plan(*shape, sm_count_or_default());
    plan->kernel = p.kernel;
    plan->num_splits = p.num_splits;
    plan->split_tokens = p.split_tokens;
    plan->rows_per_block = p.rows_per_block;
    plan->row_blocks = p.row_blocks;
    plan->merge = p.merge;
    return TREESPEC_OK;
}

extern "C" int tree_attn_verify(const void* q, const void* k_pages, const void* v_pages,
                                const int32_t* page_table, const int32_t* prefix_lens,
                                const int32_t* tree_parents, void* out,
                                const treespec_attn_shape* shape, void* workspace,
                                size_t workspace_bytes, treespec_stream_t stream) {
    int rc = check_attn_shape(shape);
    if (rc != TREESPEC_OK) return rc;
    if (!q || !k_pages || !v_pages || !page_table || !prefix_lens || !tree_parents || !out)
        return TREESPEC_ERR_NULL_POINTER;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
        return TREESPEC_ERR_ALIGNMENT;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign)) return TREESPEC_ERR_WORKSPACE;
    rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    const treespec_attn_shape& s = *shape;
    const AttnPlan plan = make_plan(s, sm_count_or_default());
    const AttnLayout lay = attn_layout(s, plan);
    if (workspace_bytes < lay.total) return TREESPEC_ERR_WORKSPACE;

    unsigned char* ws = static_cast<unsigned char*>(workspace);
    AttnParams p{};
    p.q = q;
    p.k = k_pages;
    p.v = v_pages;
    p.page_table = page_table;
    p.prefix_lens = prefix_lens;
    p.parents = tree_parents;
    p.out = out;
    p.status = reinterpret_cast<uint32_t*>(ws + lay.status);
    p.anc = reinterpret_cast<uint64_t*>(ws + lay.anc);
    p.lens = reinterpret_cast<int32_t*>(ws + lay.lens);
    p.nn = reinterpret_cast<int32_t*>(ws + lay.nn);
    p.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    p.part_acc = reinterpret_cast<float*>(ws + lay.acc);
    p.B = s.batch;
    p.N = s.num_nodes;
    p.Hq = s.num_q_heads;
    p.Hkv = s.num_kv_heads;
    p.G = s.num_q_heads / s.num_kv_heads;
    p.R = p.N * p.G;
    p.D = s.head_dim;
    p.ps = s.page_size;
    p.max_pages = s.max_pages_per_seq;
    p.num_pool_pages = s.num_pool_pages;
    p.num_splits = plan.num_splits;
    p.split_tokens = plan.split_tokens;
    p.rows_per_block = plan.rows_per_block;
    p.row_blocks = plan.row_blocks;
    p.merge = plan.merge;
    p.scale_log2 = float(1.4426950408889634 / std::sqrt(double(s.head_dim)));
    p.wait_ns = g_wait_ns.load();
    p.stream_ctas = plan.stream_ctas;
    p.stream_flags = plan.kernel == TREESPEC_KERNEL_TC_STREAM ? reinterpret_cast<int32_t*>(ws + lay.flags) : nullptr;

    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st); e != cudaSuccess) return launch_failed(e);
    if (const cudaError_t e = launch_tree_prologue(p, st); e != cudaSuccess) return launch_failed(e);
    g_launches++;
    const cudaError_t e = plan.kernel == TREESPEC_KERNEL_TC_STREAM ? launch_attn_tc_stream(p, st)
                          : plan.kernel == TREESPEC_KERNEL_TC_PAIR ? launch_attn_tc_pair(p, st)
                          : plan.kernel == TREESPEC_KERNEL_TC_2SM ? launch_attn_tc_2sm(p, st)
                          : plan.kernel == TREESPEC_KERNEL_TC    ? launch_attn_tc(p, st)
                                                                 : launch_attn_simt(p, s.dtype, st);
    if (e != cudaSuccess) return launch_failed(e);
    g_launches++;
    if (plan.merge) {
        if (const cudaError_t e = launch_attn_merge(p, s.dtype, st); e != cudaSuccess) return launch_failed(e);
        g_launches++;
    }
    return TREESPEC_OK;
}

extern "C" size_t treespec_accept_workspace_bytes(int32_t batch, int32_t num_nodes, int32_t vocab) {
    if (batch < 1 || num_nodes < 1 || num_nodes > kMaxNodes || vocab < 1 || vocab > (1 << 30)) return 0;
    return accept_layout(batch, num_nodes).total;
}

extern "C" int tree_accept_with_mode(const float* target_logits, const int32_t* draft_tokens,
                                     const float* draft_probs, const int32_t* tree_parents,
                                     const float* uniforms, float temperature, int32_t* accept_path,
                                     int32_t* accept_len, int32_t* bonus_token, int32_t batch,
                                     int32_t num_nodes, int32_t vocab, int32_t mode, void* workspace,
                                     size_t workspace_bytes, treespec_stream_t stream) {
    if (batch < 1 || num_nodes < 1 || num_nodes > kMaxNodes || vocab < 1 || vocab > (1 << 30))
        return TREESPEC_ERR_SHAPE;
    if ((long long)batch * num_nodes > 0x7fffffffll) return TREESPEC_ERR_SHAPE;
    if (mode < TREESPEC_ACCEPT_AUTO || mode > TREESPEC_ACCEPT_PATH_ONLY) return TREESPEC_ERR_SHAPE;
    if (!target_logits || !draft_tokens || !tree_parents || !accept_path || !accept_len || !bonus_token)
        return TREESPEC_ERR_NULL_POINTER;
    if (!(temperature >= 0.f) || std::isinf(temperature)) return TREESPEC_ERR_SAMPLING;
    const bool stoch = temperature > 0.f;
    if (stoch && (!draft_probs || !uniforms)) return TREESPEC_ERR_SAMPLING;
    if (!aligned16(target_logits) || (stoch && !aligned16(draft_probs))) return TREESPEC_ERR_ALIGNMENT;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign)) return TREESPEC_ERR_WORKSPACE;
    const AcceptLayout lay = accept_layout(batch, num_nodes);
    if (workspace_bytes < lay.total) return TREESPEC_ERR_WORKSPACE;
    const int rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    if (mode == TREESPEC_ACCEPT_AUTO) mode = TREESPEC_ACCEPT_PATH_ONLY;   // measured faster on every workload

    unsigned char* ws = static_cast<unsigned char*>(workspace);
    AcceptParams p{};
    p.logits = target_logits;
    p.tokens = draft_tokens;
    p.probs = draft_probs;
    p.parents = tree_parents;
    p.uniforms = uniforms;
    p.path = accept_path;
    p.len = accept_len;
    p.bonus = bonus_token;
    p.status = reinterpret_cast<uint32_t*>(ws + lay.status);
    p.amax = reinterpret_cast<int32_t*>(ws + lay.amax);
    p.stats = reinterpret_cast<float*>(ws + lay.stats);
    p.izs = reinterpret_cast<float*>(ws + lay.izs);
    p.B = batch;
    p.N = num_nodes;
    p.V = vocab;
    p.temperature = temperature;
    p.c = stoch ? float(1.4426950408889634 / double(temperature)) : 0.f;
    p.sms = sm_count_or_default();
    if (stoch) {
        cudaPointerAttributes at{};
        if (cudaPointerGetAttributes(&at, draft_probs) == cudaSuccess) p.probs_on_host = at.type == cudaMemoryTypeHost;
        else cudaGetLastError();                         // not a pointer CUDA knows: treat as device memory
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st); e != cudaSuccess) return launch_failed(e);
    int kernels = 0;
    if (const cudaError_t e = launch_accept(p, mode, st, &kernels); e != cudaSuccess) return launch_failed(e);
    g_launches += kernels;
    return TREESPEC_OK;
}

extern "C" int tree_accept(const float* target_logits, const int32_t* draft_tokens,
                           const float* draft_probs, const int32_t* tree_parents,
                           const float* uniforms, float temperature, int32_t* accept_path,
                           int32_t* accept_len, int32_t* bonus_token, int32_t batch,
                           int32_t num_nodes, int32_t vocab, void* workspace,
                           size_t workspace_bytes, treespec_stream_t stream) {
    return tree_accept_with_mode(target_logits, draft_tokens, draft_probs, tree_parents, uniforms, temperature,
                                 accept_path, accept_len, bonus_token, batch, num_nodes, vocab,
                                 TREESPEC_ACCEPT_AUTO, workspace, workspace_bytes, stream);
}

extern "C" size_t treespec_commit_workspace_bytes(void) { return kWsAlign; }

namespace {
// tree_kv_commit (k_scales NULL) and tree_kv_commit_e4m3
int commit(void* k_pages, void* v_pages, float* k_scales, float* v_scales, const int32_t* page_table,
           const int32_t* prefix_lens, const int32_t* accept_path, const int32_t* accept_len,
           int32_t* new_prefix_lens, const treespec_attn_shape* shape, void* workspace, size_t workspace_bytes,
           treespec_stream_t stream) {
    int rc = check_attn_shape(shape);
    if (rc != TREESPEC_OK) return rc;
    if (!k_pages || !v_pages || !page_table || !prefix_lens || !accept_path || !accept_len || !new_prefix_lens)
        return TREESPEC_ERR_NULL_POINTER;
    if (!aligned16(k_pages) || !aligned16(v_pages)) return TREESPEC_ERR_ALIGNMENT;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign) ||
        workspace_bytes < treespec_commit_workspace_bytes())
        return TREESPEC_ERR_WORKSPACE;
    rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    const treespec_attn_shape& s = *shape;
    CommitParams p{};
    p.k = k_pages;
    p.v = v_pages;
    p.page_table = page_table;
    p.prefix_lens = prefix_lens;
    p.path = accept_path;
    p.len = accept_len;
    p.new_lens = new_prefix_lens;
    p.status = static_cast<uint32_t*>(workspace);
    p.B = s.batch;
    p.N = s.num_nodes;
    p.Hkv = s.num_kv_heads;
    p.D = s.head_dim;
    p.ps = s.page_size;
    p.max_pages = s.max_pages_per_seq;
    p.num_pool_pages = s.num_pool_pages;
    p.elem = k_scales ? 1 : s.dtype == TREESPEC_DTYPE_BF16 ? 2 : 4;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st); e != cudaSuccess) return launch_failed(e);
    if (const cudaError_t e = launch_kv_commit(p, st); e != cudaSuccess) return launch_failed(e);
    g_launches++;
    return TREESPEC_OK;
}
}  // namespace

extern "C" int tree_kv_commit(void* k_pages, void* v_pages, const int32_t* page_table,
                              const int32_t* prefix_lens, const int32_t* accept_path,
                              const int32_t* accept_len, int32_t* new_prefix_lens,
                              const treespec_attn_shape* shape, void* workspace, size_t workspace_bytes,
                              treespec_stream_t stream) {
    return commit(k_pages, v_pages, nullptr, nullptr, page_table, prefix_lens, accept_path, accept_len,
                  new_prefix_lens, shape, workspace, workspace_bytes, stream);
}

extern "C" int tree_kv_commit_e4m3(void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                                   const int32_t* page_table, const int32_t* prefix_lens,
                                   const int32_t* accept_path, const int32_t* accept_len, int32_t* new_prefix_lens,
                                   const treespec_attn_shape* shape, void* workspace, size_t workspace_bytes,
                                   treespec_stream_t stream) {
    if (!k_scales || !v_scales) return TREESPEC_ERR_NULL_POINTER;
    if (!aligned16(k_scales) || !aligned16(v_scales)) return TREESPEC_ERR_ALIGNMENT;
    return commit(k_pages, v_pages, k_scales, v_scales, page_table, prefix_lens, accept_path, accept_len,
                  new_prefix_lens, shape, workspace, workspace_bytes, stream);
}

// ------------------------------------------------------------------ chunks, 8-bit cache

namespace {

int check_chunk_shape(const treespec_chunk_shape* s, bool attn) {
    if (!s) return TREESPEC_ERR_NULL_POINTER;
    if (s->dtype != TREESPEC_DTYPE_F32 && s->dtype != TREESPEC_DTYPE_BF16) return TREESPEC_ERR_DTYPE;
    if (s->kv_dtype != s->dtype && s->kv_dtype != TREESPEC_DTYPE_E4M3) return TREESPEC_ERR_DTYPE;
    if (s->batch < 1 || s->batch > 65535 || s->num_tokens < 1) return TREESPEC_ERR_SHAPE;
    if (s->num_kv_heads < 1 || s->num_q_heads < 1 || s->num_q_heads % s->num_kv_heads) return TREESPEC_ERR_SHAPE;
    if (s->num_q_heads > 65535 || s->num_q_heads / s->num_kv_heads > 128) return TREESPEC_ERR_SHAPE;
    if ((long long)s->num_tokens * s->num_q_heads >= (1ll << 31)) return TREESPEC_ERR_SHAPE;
    if (s->head_dim != 64 && s->head_dim != 128) return TREESPEC_ERR_SHAPE;
    if (s->page_size != kPage) return TREESPEC_ERR_SHAPE;
    if (s->max_pages_per_seq < 1 || s->num_pool_pages < 1) return TREESPEC_ERR_SHAPE;
    if ((long long)s->max_pages_per_seq * s->page_size > (1ll << 30)) return TREESPEC_ERR_SHAPE;
    if (s->kernel != TREESPEC_KERNEL_AUTO &&
        !(attn && (s->kernel == TREESPEC_KERNEL_SIMT || s->kernel == TREESPEC_KERNEL_TC_STREAM)))
        return TREESPEC_ERR_SHAPE;
    if (s->kernel == TREESPEC_KERNEL_TC_STREAM) {
        if (s->dtype != TREESPEC_DTYPE_BF16) return TREESPEC_ERR_DTYPE;
        if (!chunk_tc_supported(s->dtype, s->batch, (long long)s->num_pool_pages * kPage)) return TREESPEC_ERR_SHAPE;
    }
    return TREESPEC_OK;
}

struct ChunkPlan {
    int kernel, num_splits, split_tokens, rows_block, ctas;
};

// rows: query rows per kv head of the whole batch.  The lengths are on the device, so the
// plan goes by the page table's width and the mean rows of a sequence.
ChunkPlan chunk_plan(int kernel, int dtype, int kv_dtype, long long batch, long long rows, int Hkv, int D,
                     int max_pages, int pool_pages, int sms) {
    ChunkPlan c{};
    if (kernel != TREESPEC_KERNEL_SIMT && chunk_tc_supported(dtype, int(batch), (long long)pool_pages * kPage)) {
        c.kernel = TREESPEC_KERNEL_TC_STREAM;
        c.num_splits = 1;
        c.ctas = std::min(sms, kChunkMaxCtas);
        return c;
    }
    c.kernel = TREESPEC_KERNEL_SIMT;
    // Row blocks no larger than the mean sequence fills, and smaller ones where those and
    // splits of at least 128 tokens would leave SMs without a CTA: a block of 64 rows reads
    // K and V a quarter as often as one of 16, but a small problem is bound by one CTA's run
    // (5 sequences of up to 130 tokens x 4 heads over up to 830 tokens of 64, float32: 59 us
    // with blocks of 64 rows in splits of 256 tokens, 27 us with this rule).
    const long long mean = (rows + batch - 1) / batch;
    const long long tokens = (long long)max_pages * kPage;
    long long splits = 1;
    // No block smaller than leaves its CTA 8 warps: they share the loads even where only some
    // hold rows.
    const int least = chunk_simt_min_rows(D, kv_dtype == TREESPEC_DTYPE_E4M3 ? 1 : kv_dtype == TREESPEC_DTYPE_BF16 ? 2 : 4);
    for (int rb = 64; rb >= least; rb /= 2) {
        if (rb > least && mean <= rb / 2) continue;
        c.rows_block = rb;
        const long long units = ((rows + rb - 1) / rb) * Hkv;
        // two CTAs per SM where the row blocks alone do not give them
        splits = units >= 2ll * sms ? 1 : 2ll * sms / units;
        splits = std::min(std::max(1ll, std::min(splits, tokens / 128)), 256ll);
        if (units * splits >= sms) break;
    }
    long long chunk = (tokens + splits - 1) / splits;
    chunk = (chunk + 127) / 128 * 128;
    c.split_tokens = int(chunk);
    c.num_splits = int((tokens + chunk - 1) / chunk);
    return c;
}

ChunkLayout chunk_layout(const ChunkPlan& c, long long T, int Hq, int D, long long tree_rows, long long batch) {
    ChunkLayout L{};
    size_t off = 0;
    L.status = off;                                      // and the persistent kernel's counters behind it
    off += kWsAlign;
    off = align_up(off + size_t(c.ctas) * 8 * 4, kWsAlign);
    L.cleared = off;
    L.anc = off;
    off = align_up(off + size_t(tree_rows) * kAncWords * 8, kWsAlign);
    L.lens = off;
    off = align_up(off + (tree_rows ? size_t(batch) * 4 : 0), kWsAlign);
    L.nn = off;
    off = align_up(off + (tree_rows ? size_t(batch) * 4 : 0), kWsAlign);
    // SIMT: a row of each split; persistent: two slots of two tiles per CTA
    const size_t parts = c.ctas ? size_t(2) * c.ctas * 256 : c.num_splits > 1 ? size_t(c.num_splits) * T * Hq : 0;
    L.ml = off;
    off = align_up(off + parts * 2 * 4, kWsAlign);
    L.acc = off;
    off = align_up(off + parts * D * 4, kWsAlign);
    L.total = off;
    return L;
}

ChunkPlan plan_of(const treespec_chunk_shape& s) {
    return chunk_plan(s.kernel, s.dtype, s.kv_dtype, s.batch, (long long)s.num_tokens * (s.num_q_heads / s.num_kv_heads),
                      s.num_kv_heads, s.head_dim, s.max_pages_per_seq, s.num_pool_pages, sm_count_or_default());
}
ChunkLayout layout_of(const treespec_chunk_shape& s, const ChunkPlan& c) {
    return chunk_layout(c, s.num_tokens, s.num_q_heads, s.head_dim, 0, s.batch);
}

int check_e4m3_verify_shape(const treespec_attn_shape* s) {
    if (!s) return TREESPEC_ERR_NULL_POINTER;
    treespec_attn_shape t = *s;
    if (t.kernel != TREESPEC_KERNEL_AUTO && t.kernel != TREESPEC_KERNEL_SIMT && t.kernel != TREESPEC_KERNEL_TC_STREAM)
        return TREESPEC_ERR_SHAPE;
    if (t.kernel == TREESPEC_KERNEL_TC_STREAM) {
        if (t.dtype != TREESPEC_DTYPE_BF16) return TREESPEC_ERR_DTYPE;
        if (!chunk_tc_supported(t.dtype, t.batch, (long long)t.num_pool_pages * kPage)) return TREESPEC_ERR_SHAPE;
    }
    t.kernel = TREESPEC_KERNEL_SIMT;                     // the limits of the tensor-core kernels are checked by the plan
    const int rc = check_attn_shape(&t);
    if (rc != TREESPEC_OK) return rc;
    if (t.num_q_heads / t.num_kv_heads > 128) return TREESPEC_ERR_SHAPE;
    if ((long long)t.batch * t.num_nodes * t.num_q_heads >= (1ll << 31)) return TREESPEC_ERR_SHAPE;
    return TREESPEC_OK;
}
ChunkPlan plan_of(const treespec_attn_shape& s) {
    return chunk_plan(s.kernel, s.dtype, TREESPEC_DTYPE_E4M3, s.batch,
                      (long long)s.batch * s.num_nodes * (s.num_q_heads / s.num_kv_heads), s.num_kv_heads, s.head_dim,
                      s.max_pages_per_seq, s.num_pool_pages, sm_count_or_default());
}
ChunkLayout layout_of(const treespec_attn_shape& s, const ChunkPlan& c) {
    const long long rows = (long long)s.batch * s.num_nodes;
    return chunk_layout(c, rows, s.num_q_heads, s.head_dim, rows, s.batch);
}

// What the two attention calls share once their arguments are checked.
int run_chunk(ChunkParams& p, const ChunkPlan& c, const ChunkLayout& lay, unsigned char* ws, int dtype, int kv_dtype,
              cudaStream_t st) {
    p.status = reinterpret_cast<uint32_t*>(ws + lay.status);
    p.counters = reinterpret_cast<int32_t*>(ws + lay.status + kWsAlign);
    p.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    p.part_acc = reinterpret_cast<float*>(ws + lay.acc);
    p.ps = kPage;
    p.G = p.Hq / p.Hkv;
    p.num_splits = c.num_splits;
    p.split_tokens = c.split_tokens;
    p.rows_block = c.rows_block;
    p.ctas = c.ctas;
    p.tpq = 128 / p.G;
    p.inv_g = (65536 + p.G - 1) / p.G;
    p.scale_log2 = float(1.4426950408889634 / std::sqrt(double(p.D)));
    p.wait_ns = g_wait_ns.load();
    cudaError_t e = c.kernel == TREESPEC_KERNEL_TC_STREAM ? launch_chunk_tc(p, kv_dtype, st)
                                                          : launch_chunk_simt(p, dtype, kv_dtype, st);
    if (e != cudaSuccess) return launch_failed(e);
    g_launches++;
    if (c.num_splits > 1) {
        e = launch_chunk_merge(p, dtype, st);
        if (e != cudaSuccess) return launch_failed(e);
        g_launches++;
    }
    return TREESPEC_OK;
}

}  // namespace

extern "C" size_t treespec_append_workspace_bytes(void) { return kWsAlign; }

extern "C" int tree_chunk_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, void* q_out, void* k_pages, void* v_pages, float* k_scales,
                                 float* v_scales, const int32_t* page_table, const int32_t* prefix_lens,
                                 const int32_t* chunk_offsets, const treespec_chunk_shape* shape,
                                 const treespec_append_options* options, void* workspace, size_t workspace_bytes,
                                 treespec_stream_t stream) {
    int rc = check_chunk_shape(shape, false);
    if (rc != TREESPEC_OK) return rc;
    if (!options || !q || !k || !v || !q_out || !k_pages || !v_pages || !page_table || !prefix_lens || !chunk_offsets)
        return TREESPEC_ERR_NULL_POINTER;
    const treespec_chunk_shape& s = *shape;
    const treespec_append_options& o = *options;
    const bool q8 = s.kv_dtype == TREESPEC_DTYPE_E4M3;
    if (q8 && (!k_scales || !v_scales)) return TREESPEC_ERR_NULL_POINTER;
    if (o.rot_dim < 0 || o.rot_dim > s.head_dim || o.rot_dim % 16) return TREESPEC_ERR_SHAPE;
    if (o.layout != TREESPEC_ROPE_HALF && o.layout != TREESPEC_ROPE_INTERLEAVED) return TREESPEC_ERR_SHAPE;
    if (o.rot_dim > 0 && !o.inv_freq) return TREESPEC_ERR_NULL_POINTER;
    if ((o.q_norm || o.k_norm) && !(o.norm_eps >= 0.f)) return TREESPEC_ERR_SHAPE;
    if (!std::isfinite(o.rope_scale)) return TREESPEC_ERR_SHAPE;
    const long long e = s.dtype == TREESPEC_DTYPE_BF16 ? 2 : 4;
    const long long D = s.head_dim;
    if (q_stride < s.num_q_heads * D || k_stride < s.num_kv_heads * D || v_stride < s.num_kv_heads * D)
        return TREESPEC_ERR_SHAPE;
    if (q == q_out && q_stride != s.num_q_heads * D) return TREESPEC_ERR_SHAPE;
    if (q_stride * e % 16 || k_stride * e % 16 || v_stride * e % 16) return TREESPEC_ERR_ALIGNMENT;
    const void* all[] = {q, k, v, q_out, k_pages, v_pages, o.q_norm, o.k_norm};
    for (const void* x : all)
        if (!aligned16(x)) return TREESPEC_ERR_ALIGNMENT;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign) ||
        workspace_bytes < treespec_append_workspace_bytes())
        return TREESPEC_ERR_WORKSPACE;
    rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    AppendParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = q_out;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.page_table = page_table;
    p.prefix_lens = prefix_lens;
    p.offsets = chunk_offsets;
    p.positions = o.positions;
    p.q_norm = o.q_norm;
    p.k_norm = o.k_norm;
    p.inv_freq = o.inv_freq;
    p.status = static_cast<uint32_t*>(workspace);
    p.B = s.batch;
    p.T = s.num_tokens;
    p.Hq = s.num_q_heads;
    p.Hkv = s.num_kv_heads;
    p.D = s.head_dim;
    p.max_pages = s.max_pages_per_seq;
    p.num_pool_pages = s.num_pool_pages;
    p.rot = o.rot_dim;
    p.layout = o.layout;
    p.eps = o.norm_eps;
    p.rope_scale = o.rope_scale;
    p.sms = sm_count_or_default();
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st); e != cudaSuccess) return launch_failed(e);
    const cudaError_t err = launch_chunk_append(p, s.dtype, s.kv_dtype, st);
    if (err != cudaSuccess) return launch_failed(err);
    g_launches++;
    return TREESPEC_OK;
}

extern "C" size_t treespec_chunk_attn_workspace_bytes(const treespec_chunk_shape* shape) {
    if (check_chunk_shape(shape, true) != TREESPEC_OK) return 0;
    return layout_of(*shape, plan_of(*shape)).total;
}

extern "C" int tree_chunk_attn(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                               const float* v_scales, const int32_t* page_table, const int32_t* prefix_lens,
                               const int32_t* chunk_offsets, void* out, const treespec_chunk_shape* shape,
                               void* workspace, size_t workspace_bytes, treespec_stream_t stream) {
    int rc = check_chunk_shape(shape, true);
    if (rc != TREESPEC_OK) return rc;
    if (!q || !k_pages || !v_pages || !page_table || !prefix_lens || !chunk_offsets || !out)
        return TREESPEC_ERR_NULL_POINTER;
    const treespec_chunk_shape& s = *shape;
    const bool q8 = s.kv_dtype == TREESPEC_DTYPE_E4M3;
    if (q8 && (!k_scales || !v_scales)) return TREESPEC_ERR_NULL_POINTER;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
        (q8 && (!aligned16(k_scales) || !aligned16(v_scales))))
        return TREESPEC_ERR_ALIGNMENT;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign)) return TREESPEC_ERR_WORKSPACE;
    rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    const ChunkPlan plan = plan_of(s);
    const ChunkLayout lay = layout_of(s, plan);
    if (workspace_bytes < lay.total) return TREESPEC_ERR_WORKSPACE;
    ChunkParams p{};
    p.q = q;
    p.k = k_pages;
    p.v = v_pages;
    p.k_scales = q8 ? k_scales : nullptr;
    p.v_scales = q8 ? v_scales : nullptr;
    p.page_table = page_table;
    p.prefix_lens = prefix_lens;
    p.offsets = chunk_offsets;
    p.out = out;
    p.B = s.batch;
    p.T = s.num_tokens;
    p.Hq = s.num_q_heads;
    p.Hkv = s.num_kv_heads;
    p.D = s.head_dim;
    p.max_pages = s.max_pages_per_seq;
    p.num_pool_pages = s.num_pool_pages;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaMemsetAsync(ws + lay.status, 0, lay.cleared, st); e != cudaSuccess) return launch_failed(e);
    return run_chunk(p, plan, lay, ws, s.dtype, s.kv_dtype, st);
}

extern "C" size_t treespec_attn_e4m3_workspace_bytes(const treespec_attn_shape* shape) {
    if (check_e4m3_verify_shape(shape) != TREESPEC_OK) return 0;
    return layout_of(*shape, plan_of(*shape)).total;
}

extern "C" int tree_attn_verify_e4m3(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                                     const float* v_scales, const int32_t* page_table, const int32_t* prefix_lens,
                                     const int32_t* tree_parents, void* out, const treespec_attn_shape* shape,
                                     void* workspace, size_t workspace_bytes, treespec_stream_t stream) {
    int rc = check_e4m3_verify_shape(shape);
    if (rc != TREESPEC_OK) return rc;
    if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !page_table || !prefix_lens || !tree_parents || !out)
        return TREESPEC_ERR_NULL_POINTER;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) || !aligned16(k_scales) ||
        !aligned16(v_scales))
        return TREESPEC_ERR_ALIGNMENT;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign)) return TREESPEC_ERR_WORKSPACE;
    rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    const treespec_attn_shape& s = *shape;
    const ChunkPlan plan = plan_of(s);
    const ChunkLayout lay = layout_of(s, plan);
    if (workspace_bytes < lay.total) return TREESPEC_ERR_WORKSPACE;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    ChunkParams p{};
    p.q = q;
    p.k = k_pages;
    p.v = v_pages;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.page_table = page_table;
    p.anc = reinterpret_cast<uint64_t*>(ws + lay.anc);
    p.lens = reinterpret_cast<int32_t*>(ws + lay.lens);
    p.nn = reinterpret_cast<int32_t*>(ws + lay.nn);
    p.out = out;
    p.B = s.batch;
    p.T = s.batch * s.num_nodes;
    p.N = s.num_nodes;
    p.Hq = s.num_q_heads;
    p.Hkv = s.num_kv_heads;
    p.D = s.head_dim;
    p.max_pages = s.max_pages_per_seq;
    p.num_pool_pages = s.num_pool_pages;
    AttnParams a{};                                      // what the tree prologue reads and writes
    a.parents = tree_parents;
    a.prefix_lens = prefix_lens;
    a.status = reinterpret_cast<uint32_t*>(ws + lay.status);
    a.anc = reinterpret_cast<uint64_t*>(ws + lay.anc);
    a.lens = reinterpret_cast<int32_t*>(ws + lay.lens);
    a.nn = reinterpret_cast<int32_t*>(ws + lay.nn);
    a.B = s.batch;
    a.N = s.num_nodes;
    a.max_pages = s.max_pages_per_seq;
    a.ps = kPage;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaMemsetAsync(ws + lay.status, 0, lay.cleared, st); e != cudaSuccess) return launch_failed(e);
    const cudaError_t e = launch_tree_prologue(a, st);
    if (e != cudaSuccess) return launch_failed(e);
    g_launches++;
    return run_chunk(p, plan, lay, ws, s.dtype, TREESPEC_DTYPE_E4M3, st);
}

extern "C" size_t treespec_draft_workspace_bytes(int32_t batch, int32_t frontier, int32_t topk) {
    if (batch < 1 || batch > 65535 || frontier < 1 || frontier > kMaxFrontier || topk < 1 || topk > kMaxTopk)
        return 0;
    const size_t per = size_t(batch) * frontier * kMaxDraftSplits * topk;
    return kWsAlign + align_up(per * 4, kWsAlign) * 2;
}

extern "C" int tree_draft_step(const float* logprobs, int32_t batch, int32_t frontier, int32_t vocab,
                               int32_t topk, int32_t step, const int32_t* frontier_in, int32_t* node_parent,
                               int32_t* node_token, float* node_score, int32_t max_nodes, int32_t* frontier_out,
                               void* workspace, size_t workspace_bytes, treespec_stream_t stream) {
    if (batch < 1 || batch > 65535 || topk < 1 || topk > kMaxTopk || step < 0) return TREESPEC_ERR_SHAPE;
    if (frontier != (step == 0 ? 1 : topk)) return TREESPEC_ERR_SHAPE;
    if (vocab < topk || vocab > (1 << 30)) return TREESPEC_ERR_SHAPE;
    const long long base = step == 0 ? 1 : 1 + topk + (long long)(step - 1) * topk * topk;
    if (max_nodes > kMaxDraftNodes || base + (long long)frontier * topk > max_nodes) return TREESPEC_ERR_SHAPE;
    if ((long long)batch * frontier * vocab > (1ll << 40)) return TREESPEC_ERR_SHAPE;
    if (!logprobs || !node_parent || !node_token || !node_score || !frontier_out || (step > 0 && !frontier_in))
        return TREESPEC_ERR_NULL_POINTER;
    if (vocab % 4 == 0 && !aligned16(logprobs)) return TREESPEC_ERR_ALIGNMENT;
    const size_t need = treespec_draft_workspace_bytes(batch, frontier, topk);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign) || workspace_bytes < need)
        return TREESPEC_ERR_WORKSPACE;
    int rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    const size_t per = size_t(batch) * frontier * kMaxDraftSplits * topk;
    DraftParams p{};
    p.logprobs = logprobs;
    p.frontier_in = frontier_in;
    p.frontier_out = frontier_out;
    p.node_parent = node_parent;
    p.node_token = node_token;
    p.node_score = node_score;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.tk_tok = reinterpret_cast<int32_t*>(ws + kWsAlign);
    p.tk_lp = reinterpret_cast<float*>(ws + kWsAlign + align_up(per * 4, kWsAlign));
    p.B = batch;
    p.F = frontier;
    p.V = vocab;
    p.k = topk;
    p.step = step;
    p.M = max_nodes;
    // A row's vocabulary is cut into S parts (one CTA each) only where the rows alone would
    // leave SMs idle: a CTA's lists filter best over a long stream (the floor rises and
    // fewer groups pass the vote), so parts cost more than they save once every SM has a
    // row (measured per step over 128256 tokens: 256 rows 36 us in one part, 41 in two;
    // 64 rows 23 us in one, 19 in two, 21 in four).  No part below 8192 tokens, parts a
    // multiple of 1024 tokens.
    {
        const long long rows = (long long)batch * frontier;
        long long S = sm_count_or_default() / rows;
        S = std::min<long long>(S, std::max<long long>(1, vocab / 8192));
        S = std::max<long long>(1, std::min<long long>(S, kMaxDraftSplits));
        long long chunk = (vocab + S - 1) / S;
        chunk = (chunk + 1023) / 1024 * 1024;
        p.S = int((vocab + chunk - 1) / chunk);
        p.chunk = int(chunk);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // the top-k kernel clears the status word (no memset: one stream operation fewer a step)
    if (const cudaError_t e = launch_draft_step(p, st); e != cudaSuccess) return launch_failed(e);
    g_launches += 2;
    return TREESPEC_OK;
}

extern "C" int tree_rerank(const int32_t* node_parent, const int32_t* node_token, const float* node_score,
                           int32_t batch, int32_t max_nodes, int32_t num_nodes, int32_t* tree_parents,
                           int32_t* draft_tokens, void* workspace, size_t workspace_bytes,
                           treespec_stream_t stream) {
    return tree_rerank_pool(node_parent, node_token, node_score, nullptr, 0, batch, max_nodes, num_nodes,
                            tree_parents, draft_tokens, workspace, workspace_bytes, stream);
}

extern "C" int tree_rerank_pool(const int32_t* node_parent, const int32_t* node_token, const float* node_score,
                                const int32_t* pool, int32_t pool_size, int32_t batch, int32_t max_nodes,
                                int32_t num_nodes, int32_t* tree_parents, int32_t* draft_tokens, void* workspace,
                                size_t workspace_bytes, treespec_stream_t stream) {
    if (batch < 1 || batch > 65535 || max_nodes < 1 || max_nodes > kMaxDraftNodes) return TREESPEC_ERR_SHAPE;
    if (pool ? (pool_size < 1 || pool_size > kMaxDraftNodes) : pool_size != 0) return TREESPEC_ERR_SHAPE;
    if (num_nodes < 1 || num_nodes > kMaxNodes || num_nodes > max_nodes) return TREESPEC_ERR_SHAPE;
    if (!node_parent || !node_token || !node_score || !tree_parents || !draft_tokens)
        return TREESPEC_ERR_NULL_POINTER;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kWsAlign) || workspace_bytes < kWsAlign)
        return TREESPEC_ERR_WORKSPACE;
    int rc = check_device();
    if (rc != TREESPEC_OK) return rc;
    RerankParams p{};
    p.node_parent = node_parent;
    p.node_token = node_token;
    p.node_score = node_score;
    p.pool = pool;
    p.P = pool_size;
    p.parents = tree_parents;
    p.tokens = draft_tokens;
    p.status = static_cast<uint32_t*>(workspace);
    p.B = batch;
    p.M = max_nodes;
    p.N = num_nodes;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st); e != cudaSuccess) return launch_failed(e);
    if (const cudaError_t e = launch_rerank(p, st); e != cudaSuccess) return launch_failed(e);
    g_launches++;
    return TREESPEC_OK;
}

extern "C" int treespec_read_status(const void* workspace, uint32_t* status, treespec_stream_t stream) {
    if (!workspace || !status) return TREESPEC_ERR_NULL_POINTER;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = cudaStreamSynchronize(st); e != cudaSuccess) return launch_failed(e);
    if (const cudaError_t e = cudaMemcpy(status, workspace, sizeof(uint32_t), cudaMemcpyDeviceToHost); e != cudaSuccess)
        return launch_failed(e);
    return TREESPEC_OK;
}

extern "C" const char* treespec_error_string(int code) {
    switch (code) {
        case TREESPEC_OK: return "ok";
        case TREESPEC_ERR_NULL_POINTER: return "a required pointer is NULL";
        case TREESPEC_ERR_SHAPE: return "a size is outside the supported range";
        case TREESPEC_ERR_DTYPE: return "unsupported dtype or kernel for this dtype";
        case TREESPEC_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case TREESPEC_ERR_SAMPLING: return "invalid temperature, or sampling inputs missing";
        case TREESPEC_ERR_ALIGNMENT: return "a tensor is not 16-byte aligned";
        case TREESPEC_ERR_DEVICE: return "no usable sm_103 CUDA device";
        case TREESPEC_ERR_LAUNCH: return "the CUDA runtime rejected a launch";
        default: return "unknown error code";
    }
}

extern "C" int treespec_version(void) { return 100; }

extern "C" uint64_t treespec_launch_count(void) { return g_launches.load(); }

extern "C" void treespec_set_wait_limit_ns(uint64_t ns) { g_wait_ns.store(ns ? ns : kDefaultWaitNs); }

extern "C" int treespec_last_launch_error(const char** name) {
    const int e = g_launch_error.load();
    if (name) *name = cudaGetErrorName(cudaError_t(e));
    return e;
}
