// rope_append.cu -- rotary positions and the write into the cache in one pass:
// queries and keys are rotated, keys and values quantised as fp8kv_append
// does, and the rows stored in the slots of a step's slot map.
//
// Pair (a, b) of a row at position t becomes (a cos - b sin, b cos + a sin),
// each product rounded to fp32 once and the sum once, so the result depends
// on the inputs alone and not on how a compiler contracts the expression.
// The rotated key is quantised from fp32: it is rounded to the cache's type
// only, not to bf16 before.
//
// What bounds it: memory.  7,940 tokens of 28 query and 4 KV heads (143 MB)
// take 26.8 us on the device, 5.3 TB/s (79 % of the measured copy rate); 64
// tokens take 2.7 us, a launch and two dependent loads.  One row pass a warp
// took 73 us, eight behind the token's slot 41 us, eight loaded before it this.
//
// A row of D values takes D / 8 lanes; lane s holds two groups of four
// elements that contain both sides of its pairs, so a rotation needs no
// exchange between lanes:
//   half layout         dims 4s..4s+3 and R/2 + 4s..R/2 + 4s+3   (s < R/8)
//   interleaved layout  dims 8s..8s+3 and 8s+4..8s+7             (s < R/8)
//   behind the rotated part (s >= R/8): dims 8s..8s+3, 8s+4..8s+7, as they are
#include "params.cuh"
#include "tc_common.cuh"

namespace fp8kv {

__device__ __forceinline__ void unpack4(uint2 u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x << 16);
  x[1] = __uint_as_float(u.x & 0xFFFF0000u);
  x[2] = __uint_as_float(u.y << 16);
  x[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(__nv_bfloat16* dst, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void rotate1(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// Maximum over the LPR lanes of a row (LPR consecutive lanes of the warp).
template <int LPR>
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float amax4(const float (&x)[4]) {
  return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
}
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float scale) {
  return e4m3x2_rn(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
         (e4m3x2_rn(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)) << 16);
}

// One row side (K or V), held by its lanes as the groups x (dims d0..) and y
// (dims d1..), into cache row `dst`.  Every lane of the warp takes part;
// lanes with `live` false store nothing.
template <int D, int KIND>
__device__ __forceinline__ void store_row(uint8_t* base, float* scales, int64_t dst, int d0, int d1, float (&x)[4],
                                          float (&y)[4], bool live) {
  constexpr int LPR = D / 8;
  if constexpr (KIND == ELEM_BF16) {
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(base) + dst * D;
    if (live) { store4(out + d0, x); store4(out + d1, y); }
  } else if constexpr (KIND == ELEM_E4M3) {
    const float amax = row_max<LPR>(fmaxf(amax4(x), amax4(y)));
    const float scale = __fdiv_rn(amax, 448.0f);
    uint32_t a = 0, b = 0;
    if (amax != 0.f) { a = codes4(x, scale); b = codes4(y, scale); }
    if (live) {
      *reinterpret_cast<uint32_t*>(base + dst * D + d0) = a;
      *reinterpret_cast<uint32_t*>(base + dst * D + d1) = b;
      if ((threadIdx.x & (LPR - 1)) == 0) scales[dst] = scale;
    }
  } else {
    // a lane's two groups can lie in any two of the row's 32-element blocks
    // (a partly rotated head shifts the second group): one maximum per block
    const int b0 = d0 >> 5, b1 = d1 >> 5;
    const float a0 = amax4(x), a1 = amax4(y);
    int e0 = 0, e1 = 0;
    uint32_t packed = 0;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const int e = mx_block_exp(row_max<LPR>(fmaxf(b0 == k ? a0 : 0.f, b1 == k ? a1 : 0.f)));
      if (b0 == k) e0 = e;
      if (b1 == k) e1 = e;
      packed |= (uint32_t)(e + 127) << (8 * k);
    }
    const float i0 = pow2_exact(-e0), i1 = pow2_exact(-e1);
    if (live) {
      *reinterpret_cast<uint32_t*>(base + dst * D + d0) =
          e4m3x2_rn(x[0] * i0, x[1] * i0) | (e4m3x2_rn(x[2] * i0, x[3] * i0) << 16);
      *reinterpret_cast<uint32_t*>(base + dst * D + d1) =
          e4m3x2_rn(y[0] * i1, y[1] * i1) | (e4m3x2_rn(y[2] * i1, y[3] * i1) << 16);
      if ((threadIdx.x & (LPR - 1)) == 0) reinterpret_cast<uint32_t*>(scales)[dst] = packed;
    }
  }
}

// A pass is 256 / D rows of one kind; a warp takes up to QU passes of a token's
// queries, or up to KU of its keys or of its values.  All its rows are loaded
// before the token's slot and position have arrived (a padding row is loaded
// and dropped): two memory latencies a warp, the second for the table row.
template <int D, int KE, int VE, int QU, int KU>
__global__ void __launch_bounds__(256) rope_append_kernel(const RopeAppendParams p) {
  constexpr int LPR = D / 8, RPP = 32 / LPR;      // lanes per row, rows per pass
  const int lane = threadIdx.x & 31, s = lane & (LPR - 1), sub = lane / LPR;
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t tok = w / p.groups;
  if (tok >= p.n) return;
  const CacheView& c = p.c;
  // which rows: groups of queries, then of keys, then of values
  int grp = (int)(w - tok * p.groups);
  const int kind = grp < p.q_groups ? 0 : grp < p.q_groups + p.k_groups ? 1 : 2;
  if (kind > 0) grp -= p.q_groups + (kind - 1) * p.k_groups;
  const int heads = kind == 0 ? p.q_heads : c.kv_heads;
  const int h0 = grp * (kind == 0 ? p.q_per : p.k_per) * RPP + sub;              // first row of this lane
  const int h1 = min(heads, (grp + 1) * (kind == 0 ? p.q_per : p.k_per) * RPP);   // rows of the group end here
  const __nv_bfloat16* src = (kind == 0 ? p.q + tok * p.q_stride : kind == 1 ? p.k + tok * p.k_stride
                                                                             : p.v + tok * p.v_stride) + h0 * D;
  const int R8 = p.rot >> 3;
  const bool turn = s < R8 && kind < 2;
  const int d0 = turn && !p.interleaved ? 4 * s : 8 * s;
  const int d1 = turn && !p.interleaved ? 4 * s + (p.rot >> 1) : 8 * s + 4;
  constexpr int U = QU > KU ? QU : KU;
  uint2 raw[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool in = h0 + u * RPP < h1;
    raw[u][0] = in ? *reinterpret_cast<const uint2*>(src + u * RPP * D + d0) : make_uint2(0, 0);
    raw[u][1] = in ? *reinterpret_cast<const uint2*>(src + u * RPP * D + d1) : make_uint2(0, 0);
  }
  const int64_t slot = p.slots[tok];
  const int t = p.pos[tok];
  if (slot < 0) return;                            // padding
  // (a cache has fewer than 2^31 rows, so a slot inside it fits 32 bits)
  const int64_t slots = c.paged ? (int64_t)c.num_pages << c.page_shift : (int64_t)c.batch * c.max_tokens;
  const bool bad_slot = slot >= slots;
  if (t < 0 || t >= p.positions || bad_slot) {
    if (lane == 0) raise_error(p.err, bad_slot ? FP8KV_DEVERR_BAD_PAGE : FP8KV_DEVERR_SEQ_TOO_LONG);
    return;
  }
  float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turn) {
    const int64_t at = (int64_t)t * (p.rot >> 1) + 4 * s;
    cs = *reinterpret_cast<const float4*>(p.cos + at);
    sn = *reinterpret_cast<const float4*>(p.sin + at);
  }
  auto row = [&](int u, float (&x)[4], float (&y)[4]) {
    unpack4(raw[u][0], x);
    unpack4(raw[u][1], y);
    if (!turn) return;
    if (p.interleaved) {
      rotate1(x[0], x[1], cs.x, sn.x);
      rotate1(x[2], x[3], cs.y, sn.y);
      rotate1(y[0], y[1], cs.z, sn.z);
      rotate1(y[2], y[3], cs.w, sn.w);
    } else {
      rotate1(x[0], y[0], cs.x, sn.x);
      rotate1(x[1], y[1], cs.y, sn.y);
      rotate1(x[2], y[2], cs.z, sn.z);
      rotate1(x[3], y[3], cs.w, sn.w);
    }
  };
  if (kind == 0) {
    // (q_out may be q itself: a lane writes the elements that it read)
    __nv_bfloat16* dst = p.q_out + (tok * p.q_heads + h0) * D;
#pragma unroll
    for (int u = 0; u < QU; ++u)
      if (h0 + u * RPP < h1) {
        float x[4], y[4];
        row(u, x, y);
        store4(dst + u * RPP * D + d0, x);
        store4(dst + u * RPP * D + d1, y);
      }
    return;
  }
  const unsigned span = c.paged ? c.page_size : c.max_tokens;
  const unsigned unit = c.paged ? (unsigned)slot >> c.page_shift : (unsigned)slot / span;
  const unsigned off = (unsigned)slot - unit * span;
  // every lane of the warp takes part in a row's maximum
#pragma unroll
  for (int u = 0; u < KU; ++u) {
    const int h = h0 + u * RPP;
    if (h - sub >= h1) break;
    const bool live = h < h1;
    const int64_t dst = ((int64_t)unit * c.kv_heads + h) * span + off;
    float x[4], y[4];
    row(u, x, y);
    if (kind == 1) {
      if (KE == ELEM_E4M3 && c.k_bias != nullptr && live) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] -= c.rope_cos != nullptr ? rope_bias(c, h, t, d0 + i) : c.k_bias[h * D + d0 + i];
          y[i] -= c.rope_cos != nullptr ? rope_bias(c, h, t, d1 + i) : c.k_bias[h * D + d1 + i];
        }
      }
      store_row<D, KE>(const_cast<uint8_t*>(c.k), const_cast<float*>(c.k_scale), dst, d0, d1, x, y, live);
    } else {
      store_row<D, VE>(const_cast<uint8_t*>(c.v), const_cast<float*>(c.v_scale), dst, d0, d1, x, y, live);
    }
  }
}

template <int D, int KE, int VE>
static cudaError_t launch_one(const RopeAppendParams& p, unsigned grid, cudaStream_t s) {
  if (p.q_per == 1 && p.k_per == 1) rope_append_kernel<D, KE, VE, 1, 1><<<grid, 256, 0, s>>>(p);
  else rope_append_kernel<D, KE, VE, 8, 2><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t dispatch(const RopeAppendParams& p, int dtype, unsigned grid, cudaStream_t s) {
  if constexpr (D == 128)
    if (dtype == FP8KV_MXK8V8) return launch_one<D, ELEM_MX, ELEM_E4M3>(p, grid, s);
  if (dtype == FP8KV_K8V8) return launch_one<D, ELEM_E4M3, ELEM_E4M3>(p, grid, s);
  if (dtype == FP8KV_K16V8) return launch_one<D, ELEM_BF16, ELEM_E4M3>(p, grid, s);
  if (dtype == FP8KV_K8V16) return launch_one<D, ELEM_E4M3, ELEM_BF16>(p, grid, s);
  return launch_one<D, ELEM_BF16, ELEM_BF16>(p, grid, s);
}

cudaError_t launch_rope_append(RopeAppendParams& p, int dtype, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  const int rpp = 256 / p.c.head_dim;
  const int pq = (p.q_heads + rpp - 1) / rpp, pk = (p.c.kv_heads + rpp - 1) / rpp;
  // few tokens: a warp per pass, as many warps as there is work; many: up to
  // eight query passes or two key or value passes a warp
  const bool few = p.n * (pq + 2 * pk) <= 64 * (int64_t)sm_count();
  p.q_groups = few ? pq : (pq + 7) / 8;
  p.k_groups = few ? pk : (pk + 1) / 2;
  p.q_per = (pq + p.q_groups - 1) / p.q_groups;
  p.k_per = (pk + p.k_groups - 1) / p.k_groups;
  p.groups = p.q_groups + 2 * p.k_groups;
  const int64_t warps = p.n * p.groups;
  if (warps > (int64_t)INT32_MAX * 8) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  return p.c.head_dim == 128 ? dispatch<128>(p, dtype, grid, s) : dispatch<64>(p, dtype, grid, s);
}

}  // namespace fp8kv
