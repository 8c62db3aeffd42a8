// api_linear.cu -- the extern "C" boundary of the matrix products: argument checks
// and status codes.
#include <cstdint>

#include "params.cuh"

using namespace fp8kv;

extern "C" {

fp8kv_status fp8kv_block_matmul(const uint8_t* a_codes, const float* a_scales, const uint8_t* b_codes,
                                const float* b_scales, const float* bias, int64_t m, int64_t n, int64_t k, void* out,
                                int32_t out_dtype, fp8kv_stream_t stream) {
  if (m < 0 || n < 0 || k < 1) return FP8KV_ERR_INVALID_ARG;
  if (out_dtype != FP8KV_OUT_BF16 && out_dtype != FP8KV_OUT_F32) return FP8KV_ERR_INVALID_ARG;
  // (rows of codes start on 16 bytes; coordinates and tile numbers are 32-bit)
  constexpr int64_t most = 1 << 30;
  if (k % 16 != 0 || m > most || n > most || k > most) return FP8KV_ERR_UNSUPPORTED;
  if ((m + 127) / 128 * ((n + 127) / 128) > INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return FP8KV_OK;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !out) return FP8KV_ERR_INVALID_ARG;
  if (misaligned(a_codes, 16) || misaligned(b_codes, 16) || misaligned(out, 16)) return FP8KV_ERR_INVALID_ARG;
  if (misaligned(a_scales, 4) || misaligned(b_scales, 4) || misaligned(bias, 4)) return FP8KV_ERR_INVALID_ARG;
  const size_t M = (size_t)m, N = (size_t)n, K = (size_t)k, KB = (K + 127) / 128;
  const Range result = {out, M * N * (out_dtype == FP8KV_OUT_F32 ? 4 : 2)};
  for (const Range& r : {Range{a_codes, M * K}, Range{a_scales, 4 * M * KB}, Range{b_codes, N * K},
                         Range{b_scales, 4 * ((N + 127) / 128) * KB}, Range{bias, 4 * N}})
    if (overlap(r, result)) return FP8KV_ERR_INVALID_ARG;
  MatmulArgs a;
  a.a = a_codes;
  a.b = b_codes;
  a.sa = a_scales;
  a.sb = b_scales;
  a.bias = bias;
  a.out = out;
  a.M = (int)m;
  a.N = (int)n;
  a.K = (int)k;
  a.out_f32 = out_dtype == FP8KV_OUT_F32;
  a.err = device_error_ptr();
  if (!a.err) return FP8KV_ERR_CUDA;
  return cuda_status(launch_block_matmul(a, (cudaStream_t)stream));
}

}  // extern "C"
