// Attention of few rows per sequence of sequences that share prefixes.
#include "chunk_few.cuh"

namespace treespec {

template cudaError_t launch_chunk_few<kChunkShared>(const ChunkParams& p, int kv_dtype, cudaStream_t s);

}  // namespace treespec
