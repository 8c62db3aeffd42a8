// chunk_rows.cu -- the few-row kernel of chunk attention, causal (chunk_rows.cuh).
#include "chunk_rows.cuh"

namespace fp8kv {

cudaError_t launch_chunk_rows(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  return launch_rows<false>(p, dtype, tiles, st);
}

}  // namespace fp8kv
