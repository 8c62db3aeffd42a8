// chunk_mma.cu -- chunk attention on warp-level matrix instructions, causal
// (chunk_mma.cuh), and the kernel that joins the splits of all chunk kernels.
#include "chunk_mma.cuh"

namespace fp8kv {

// Joins the splits of each row of out.  Rows that no tile holds (padding, and
// those of a sequence with bad offsets) have no shares and stay as they were.
// Many rows or few splits: a warp a row (W 1); few rows of more than three splits:
// the eight warps of a CTA take every eighth split each and add their sums in
// order.  A chain of loads bounds it: one token of 32 heads over 24,000 tokens in
// 76 splits takes 33 us with a warp a row, 17 us so; 3,000 rows of 12 splits 34 us
// with a warp a row, 38 us with eight.  It is launched as a programmatic dependent,
// set up while the kernel before it drains (1 us); at 32 registers 1,024 rows are
// one wave (at 39 two, 1.5 us more).
template <int D, int W>
__global__ void __launch_bounds__(256, 8) chunk_merge(const ChunkParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, S = p.num_splits;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 8 + warp : blockIdx.x;
  const int tok = (int)(row / p.q_heads);
  // padding in front of and behind the sequences (the offsets are an input of the
  // kernel before as well: they can be read now); an end before the start has its
  // rows marked (chunk_mark_rows)
  bool live = row < (int64_t)p.total_q * p.q_heads;
  if (live && p.cu_q != nullptr) {
    const int start = p.cu_q[0], end = p.cu_q[p.c.batch];
    live = tok >= start && (tok < end || end < start);
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");    // the shares are written
  if (!live) return;
  const float* pm = p.part_m + row * S;
  const float* pl = p.part_l + row * S;
  constexpr int E = D / 32;
  float M = -INFINITY, L = 0.f, x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.f;
  const bool marked = pl[0] == kChunkNoRow;
  for (int s = lane; s < S; s += 32) M = fmaxf(M, pm[s]);
  M = warp_max(M);
  if (marked) return;
  bool minus = false;                          // no finite score: did a share see some (its sum is -0)?
  if (M == -INFINITY)
    for (int s = 0; s < S; ++s) minus = minus || __float_as_uint(pl[s]) == 0x80000000u;
  // splits k W + warp (W 1: all)
  for (int k0 = 0; k0 * W < S; k0 += 32) {
    const int s = W == 1 ? k0 + lane : (k0 + lane) * W + warp;
    float w = 0.f;
    if (s < S) {
      w = chunk_weight(pm[s], pl[s], M);
      L = fmaf(w, pl[s], L);
    }
    const int n = min(32, (S - k0 * W + W - 1 - (W == 1 ? 0 : warp)) / W);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* po = p.part_o + (row * S + (W == 1 ? k0 + k : (k0 + k) * W + warp)) * D + lane * E;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(po);
        x[0] = fmaf(wk, v.x, x[0]); x[1] = fmaf(wk, v.y, x[1]);
        x[2] = fmaf(wk, v.z, x[2]); x[3] = fmaf(wk, v.w, x[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(po);
        x[0] = fmaf(wk, v.x, x[0]); x[1] = fmaf(wk, v.y, x[1]);
      }
    }
  }
  L = warp_sum(L);
  if constexpr (W > 1) {                       // the warps' shares, added in their order
    __shared__ float sx[W][D], sl[W];
#pragma unroll
    for (int e = 0; e < E; ++e) sx[warp][lane * E + e] = x[e];
    if (lane == 0) sl[warp] = L;
    __syncthreads();
    if (warp > 0) return;
    for (int k = 1; k < W; ++k) {
      L += sl[k];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] += sx[k][lane * E + e];
    }
  }
  const float inv = chunk_inverse(L, minus);
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] *= inv;
  if (p.out_f32) {
    float* dst = reinterpret_cast<float*>(p.out) + row * D + lane * E;
    if constexpr (E == 4) *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.out) + row * D + lane * E);
    if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<true>(x[0], x[1]), pack16<true>(x[2], x[3]));
    else *dst = pack16<true>(x[0], x[1]);
  }
}

cudaError_t launch_chunk_merge(const ChunkParams& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.total_q * p.q_heads;
  const bool many = p.num_splits > 3 && rows <= 16 * sm_count();
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(many ? rows : (rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (p.c.head_dim == 128) return cudaLaunchKernelEx(&cfg, many ? chunk_merge<128, 8> : chunk_merge<128, 1>, p);
  return cudaLaunchKernelEx(&cfg, many ? chunk_merge<64, 8> : chunk_merge<64, 1>, p);
}

cudaError_t launch_chunk_mma(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  return launch_mma<false>(p, dtype, tiles, st);
}

}  // namespace fp8kv
