// Attention of few rows per sequence with a sliding window and sinks.
#include "chunk_few.cuh"

namespace treespec {

template cudaError_t launch_chunk_few<kChunkWindow>(const ChunkParams& p, int kv_dtype, cudaStream_t s);

}  // namespace treespec
