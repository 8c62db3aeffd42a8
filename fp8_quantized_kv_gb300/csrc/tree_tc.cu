// tree_tc.cu -- chunk attention on the tcgen05 tensor cores, over trees of new tokens (chunk_tc.cuh).
#include "chunk_tc.cuh"

namespace fp8kv {

cudaError_t launch_tree_tc(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  return launch_tc<true>(p, dtype, tiles, st);
}

}  // namespace fp8kv
