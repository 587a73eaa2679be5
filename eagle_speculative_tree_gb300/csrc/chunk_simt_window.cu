// Attention of packed chunks and trees on CUDA cores with a sliding window and sinks.
#include "chunk_simt.cuh"

namespace treespec {

template cudaError_t launch_chunk_simt<kChunkWindow>(const ChunkParams& p, int dtype, int kv_dtype, cudaStream_t s);

}  // namespace treespec
