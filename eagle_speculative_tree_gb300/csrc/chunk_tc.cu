// Attention of packed chunks on tensor cores without a window or shared prefixes.
#include "chunk_tc.cuh"

namespace treespec {

template cudaError_t launch_chunk_tc<kChunkPlain>(const ChunkParams& p, int kv_dtype, cudaStream_t s);

bool chunk_tc_supported(int dtype, int entries, long long pool_tokens) {
    return dtype == TREESPEC_DTYPE_BF16 && entries <= kChunkMaxBatch && pool_tokens < (1ll << 31);
}

}  // namespace treespec
