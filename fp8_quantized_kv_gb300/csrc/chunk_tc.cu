// chunk_tc.cu -- chunk attention on the tcgen05 tensor cores, causal (chunk_tc.cuh).
#include "chunk_tc.cuh"

namespace fp8kv {

cudaError_t launch_chunk_tc(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  return launch_tc<false>(p, dtype, tiles, st);
}

}  // namespace fp8kv
