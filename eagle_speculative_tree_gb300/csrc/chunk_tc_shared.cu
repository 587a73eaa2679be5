// Attention of packed chunks and trees on tensor cores of sequences that share prefixes.
#include "chunk_tc.cuh"

namespace treespec {

template cudaError_t launch_chunk_tc<kChunkShared>(const ChunkParams& p, int kv_dtype, cudaStream_t s);

}  // namespace treespec
