// tree_rows.cu -- the few-row kernel over trees of new tokens (chunk_rows.cuh).
#include "chunk_rows.cuh"

namespace fp8kv {

cudaError_t launch_tree_rows(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  return launch_rows<true>(p, dtype, tiles, st);
}

}  // namespace fp8kv
