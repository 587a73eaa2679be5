// Attention of packed chunks and trees on tensor cores with a sliding window and sinks.
#include "chunk_tc.cuh"

namespace treespec {

template cudaError_t launch_chunk_tc<kChunkWindow>(const ChunkParams& p, int kv_dtype, cudaStream_t s);

}  // namespace treespec
