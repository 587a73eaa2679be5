// Attention of packed chunks and trees on CUDA cores of sequences that share prefixes.
#include "chunk_simt.cuh"

namespace treespec {

template cudaError_t launch_chunk_simt<kChunkShared>(const ChunkParams& p, int dtype, int kv_dtype, cudaStream_t s);

}  // namespace treespec
