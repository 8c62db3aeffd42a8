// tree_mma.cu -- chunk attention on warp-level matrix instructions over trees of
// new tokens (chunk_mma.cuh).
#include "chunk_mma.cuh"

namespace fp8kv {

cudaError_t launch_tree_mma(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  return launch_mma<true>(p, dtype, tiles, st);
}

}  // namespace fp8kv
