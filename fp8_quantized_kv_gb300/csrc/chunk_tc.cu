// chunk_tc.cu -- ragged chunk attention over the cache on the tcgen05 tensor
// cores (head_dim 128): the form for tiles with many query rows, where the
// two matrix products and the softmax between them bound the time.
//
// A CTA owns up to 128 query rows of one KV head (tokens x heads of the
// group: the heads share the K and V tiles) and walks the 64-key tiles that
// any of them sees.  Per tile:
//   S[128 x 64]   = Q . K^T        e4m3 keys: kind::f8f6f4 on the codes as they
//                                  landed, the bf16 query as two e4m3 terms
//                                  (hi, and what hi leaves over) after a
//                                  power-of-two scaling of the row; bf16 keys:
//                                  kind::f16 in bf16
//   p = 2^(s - m), l += p          a quad of threads per two rows, running
//                                  maximum m moved only when it grows by
//                                  more than 2^8
//   O[128 x 128] += P . V          kind::f16; P is the A operand and stays in
//                                  TMEM, written over the scores it came from;
//                                  e4m3 values converted to f16 (exact), bf16
//                                  values as they landed
// P carries the value scale and a power of two 2^-kp per row, as in
// chunk_rows.cu: 16 bits, the one rounding of the softmax (f16 beside e4m3
// values; bf16 beside bf16 ones, since the instruction takes one 16-bit type).
//
// The CTA keeps to 256 TMEM columns (two score buffers, one O) and at most 113
// KB of shared memory, so two CTAs share an SM: one's softmax runs while the
// other's products, prologue or epilogue do.
//
// Warp roles (384 threads, 80 registers each at two CTAs):
//   warps 0-7   softmax of 16 query rows (TMEM lanes) each; epilogue
//   warps 8-9   preparation, one key per thread: per-key scales; e4m3 V codes
//               -> f16 operand; in a tile that not every query sees whole,
//               rows nobody sees are zeroed, and a row with non-finite values
//               is cleared of them and its key scale set to NaN: queries that
//               see it get NaN, the others nothing
//   warp 10     TMA producer: K ring and V ring
//   warp 11     TMEM owner and MMA issuer
// Every wait is bounded; one that runs out raises FP8KV_DEVERR_TIMEOUT, and the
// tile's rows come out as if they saw no key (an empty share, a row of zeros).
//
// Measured on one GB300: 3,727 queries over 2,000-8,000 tokens (28 query / 4 KV
// heads, e4m3, 16-token pages) 280 us, 693 TFLOP/s, 36 % of the measured bf16
// peak; 6,642 queries under a 512-token window (16 / 2 heads, bf16) 73 us.  What
// bounds it: the chain of a tile through a softmax warp (TMEM load, scales,
// maximum, exponentials, P store: about 2,500 cycles with two CTAs on the SM,
// issue slots 60 % busy, tensor pipe 44 %, shared-memory port 49 %).  On the way:
//   one warpgroup more with setmaxnreg (3 x 80 registers)  spills, 447 us
//   256 threads at 128 registers, a whole row per thread    324 us
//   fragment-shaped TMEM loads, 16 rows a warp (this)       321 us, the base of
//   the rest: copies issued by a converged warp with uniform row numbers, scale
//   rows read by the preparation warps                      295 us
//   maxima joined only when a reference moves               281 us
// Measured and not kept: four preparation warps (72 registers, spills: 351 us),
// preparation warps on alternate tiles (315 us), scores of two tiles by one
// 128-key product (fewer reads of Q, but the pair waits for both P.V: 309 us),
// key scales loaded while the scores arrive (287 us), waits with a suspend hint
// (as fast).
#include <cfloat>

#include "chunk_common.cuh"
#include "tc_common.cuh"

namespace fp8kv {

constexpr int kCtRows = 128, kCtThreads = 384;

template <int KE, int VE>
struct CtCfg {
  static constexpr bool K16 = KE == ELEM_BF16, V16 = VE == ELEM_BF16;
  static constexpr int D = 128;
  static constexpr int QOP = kCtRows * 2 * D;                       // [hi, lo][128][128 B], or [2 halves of D][128][128 B]
  static constexpr int KT = kChunkKeys * D * (K16 ? 2 : 1);         // K tile
  static constexpr int VT = kChunkKeys * D * (V16 ? 2 : 1);         // V tile as stored
  static constexpr int KN = K16 ? 2 : 3, VN = K16 && !V16 ? 1 : 2;  // ring depths
  static constexpr int NOP = V16 ? 0 : 2;                           // f16 V operand buffers
  static constexpr int OPT = kChunkKeys * D * 2;
  static constexpr int CST = 2 * kChunkKeys + 4;                    // floats: k, v column scales, largest v scale of each half
  static constexpr int NCOL = 4;
  static constexpr int MISC = 512;
  static constexpr int BYTES = 1024 + QOP + KN * KT + VN * VT + NOP * OPT + NCOL * CST * 4 + MISC;
  static_assert(2 * (BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
};

struct ChunkTcParams {
  CUtensorMap tmk, tmv;
  ChunkParams p;
};

// D[tmem] (+)= A[tmem] x B[smem]^T, 16-bit operands; one thread issues.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(id), "r"(accumulate));
}
// TMEM access of 16 lanes (rows) in the fragment shape of a matrix product:
// thread 4 g + c of the warp holds rows g and g + 8.  256-bit columns (8 fp32):
// registers 4 n .. 4 n + 3 are columns 8 n + 2 c, + 1 of row g, then of row
// g + 8; 128-bit columns (4 words): registers 2 n, 2 n + 1 are word 4 n + c of
// row g and of row g + 8.  A thread then meets only a quarter of the keys, and
// loads a quarter of their scales: with a whole row per thread, bringing 64 key
// and 64 value scales to every thread took half of the shared-memory bandwidth.
__device__ __forceinline__ void tmem_ld_256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_256b_x2(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// One lane of the (converged) warp, the same at every call.  The issuing warps
// run their loops with all lanes, and only the instruction itself belongs to
// the elected one: addresses and descriptors are then uniform for the compiler.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e != 0;
}
// OR of `pred` over the 256 softmax threads (named barrier 1).
__device__ __forceinline__ bool softmax_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}
// Two bf16 elements times zero: 0, or NaN for one that is infinite or NaN.
__device__ __forceinline__ uint32_t times_zero(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0x7FFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0x7FFF0000u : 0u);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int KE, int VE>
__global__ void __launch_bounds__(kCtThreads, 2) chunk_tc(const __grid_constant__ ChunkTcParams tp) {
  using C = CtCfg<KE, VE>;
  constexpr int D = 128;
  const ChunkParams& p = tp.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qop = smem;
  uint8_t* kring = qop + C::QOP;
  uint8_t* vring = kring + C::KN * C::KT;
  uint8_t* vop = C::V16 ? vring : vring + C::VN * C::VT;
  float* cols = reinterpret_cast<float*>(vring + C::VN * C::VT + C::NOP * C::OPT);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(cols) + C::NCOL * C::CST * 4);
  constexpr int OPN = C::V16 ? C::VN : C::NOP;                // operand buffers of P.V
  uint64_t* kfull = bars;                                     // [KN] K tile landed
  uint64_t* kfree = kfull + C::KN;                            // [KN] QK has read it
  uint64_t* vfull = kfree + C::KN;                            // [VN] V tile landed
  uint64_t* vfree = vfull + C::VN;                            // [VN] converted (bf16: read by P.V)
  uint64_t* op_full = vfree + C::VN;                          // [OPN] operand of P.V ready
  uint64_t* op_free = op_full + OPN;                          // [OPN] P.V has read it
  uint64_t* col_full = op_free + OPN;                         // [NCOL] column scales written
  uint64_t* s_full = col_full + C::NCOL;                      // [2] scores ready
  // P written, one barrier a buffer: a warp may be done with tile j + 1 before
  // another is with tile j
  uint64_t* p_full = s_full + 2;                              // [2]
  uint64_t* pv_done = p_full + 2;                             // P.V finished
  uint64_t* drained = pv_done + 1;                            // every product finished
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int8_t* kq_sh = reinterpret_cast<int8_t*>(bars) + 256;      // [128] exponent of each row's query operand
  int8_t* own_sh = kq_sh + kCtRows;               // [128] is the row's own key in this share?
  static_assert(8 * (2 * C::KN + 2 * C::VN + 2 * OPN + C::NCOL + 6) + 8 <= 256 && 256 + 2 * kCtRows <= C::MISC, "they fit");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.y, split = blockIdx.z;
  ChunkTile t;
  if (!chunk_tile(p, gridDim.x - 1 - blockIdx.x, hk == 0 && split == 0, t)) return;
  const int per = (t.n + p.num_splits - 1) / p.num_splits;
  const int j0 = min(t.n, split * per), n = min(t.n, j0 + per) - j0;
  const CacheView& c = p.c;
  const int G = p.group;

  const int64_t cont0 = ((int64_t)t.b * c.kv_heads + hk) * c.max_tokens;
  auto page_needed = [&](int k0, int len) {                   // is any key of [k0, k0 + len) seen by a query?
    return k0 < t.kv_end && (k0 + len > t.lo || k0 < p.sinks);
  };
  // The producer warp loads the K tiles and the V tiles.  Paged: lane 4 i + k
  // keeps the first cache row of page k of tile 8 q + i (-1: a page nobody
  // sees, which may be gone), fetched for eight tiles at once and one group
  // ahead, so no copy waits for the page table.
  const int pages = c.paged ? kChunkKeys / c.page_size : 0;
  auto fetch_ids = [&](int group) {
    const int j = 8 * group + (lane >> 2), k = lane & 3;
    int row = -1;
    if (k < pages && j < n) {
      const int key = chunk_key0(t, j0 + j) + k * c.page_size;
      if (page_needed(key, c.page_size)) {
        int page = c.page_table[(int64_t)t.b * c.max_pages_per_seq + (key >> c.page_shift)];
        if (page < 0 || page >= c.num_pages) {
          raise_error(p.err, FP8KV_DEVERR_BAD_PAGE);
          page = 0;
        }
        row = (page * c.kv_heads + hk) * c.page_size;          // (rows of a cache fit 31 bits)
      }
    }
    return row;
  };
  auto load_tile = [&](int j, bool is_v, int ids) {
    const int key0 = chunk_key0(t, j0 + j);
    uint8_t* st = is_v ? vring + (j % C::VN) * C::VT : kring + (j % C::KN) * C::KT;
    uint64_t* bar = is_v ? &vfull[j % C::VN] : &kfull[j % C::KN];
    const CUtensorMap* map = is_v ? &tp.tmv : &tp.tmk;
    const bool wide = is_v ? C::V16 : C::K16;
    const uint32_t half = kChunkKeys * 128;                   // bf16: dims 64..127 behind dims 0..63
    if (!c.paged) {
      const int row = (int)(cont0 + key0);
      if (elect_one()) {
        tma::arrive_expect_tx(bar, half * (wide ? 2 : 1));
        tma::load_2d(st, map, 0, row, bar);
        if (wide) tma::load_2d(st + half, map, 64, row, bar);
      }
    } else {
      const int P = c.page_size;
      int row[4], np = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {                           // (four pages of 16 tokens at most)
        // a reduction, not a shuffle: its result is uniform for the compiler,
        // and a copy with uniform operands issues twice as fast
        row[k] = __reduce_max_sync(0xffffffffu, lane == (j & 7) * 4 + k ? ids : -1);
        np += row[k] >= 0;
      }
      if (elect_one()) {
        tma::arrive_expect_tx(bar, np * (uint32_t)P * 128 * (wide ? 2 : 1));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row[k] >= 0) {
            tma::load_2d(st + k * P * 128, map, 0, row[k], bar);
            if (wide) tma::load_2d(st + half + k * P * 128, map, 64, row[k], bar);
          }
      }
      __syncwarp();
    }
  };

  // ---------------------------------------------------------------- setup
  int ids = 0, next_ids = 0;                      // page ids of this group of eight tiles and of the next
  if (warp == 10) {
    ids = fetch_ids(0);
    next_ids = fetch_ids(1);
  }
  if (warp == 10 && lane == 0) {
    tma::prefetch_map(&tp.tmk);
    tma::prefetch_map(&tp.tmv);
    for (int i = 0; i < C::KN; ++i) { umma::mbar_init(&kfull[i], 1); umma::mbar_init(&kfree[i], 1); }
    for (int i = 0; i < C::VN; ++i) { umma::mbar_init(&vfull[i], 1); umma::mbar_init(&vfree[i], C::V16 ? 1 : 2); }
    for (int i = 0; i < OPN; ++i) { umma::mbar_init(&op_full[i], 2); umma::mbar_init(&op_free[i], 1); }
    for (int i = 0; i < C::NCOL; ++i) umma::mbar_init(&col_full[i], 2);
    umma::mbar_init(&s_full[0], 1);
    umma::mbar_init(&s_full[1], 1);
    umma::mbar_init(&p_full[0], 8);
    umma::mbar_init(&p_full[1], 8);
    umma::mbar_init(pv_done, 1);
    umma::mbar_init(drained, 1);
    *abort_flag = 0;
    umma::mbar_fence_init();
  }
  // the first tiles' copies start before the query operand is made
  constexpr int LEAD = C::KN - C::VN;
  const int first_k = min(n, C::KN), first_v = min(n, C::VN);
  if (warp == 10) {
    __syncwarp();
    for (int j = 0; j < first_k; ++j) load_tile(j, false, ids);
    for (int j = 0; j < first_v; ++j) load_tile(j, true, ids);
  }
  if (warp == 11) {
    umma::tmem_alloc(tslot, 256);
    umma::tmem_relinquish();
  }
  // softmax warps: query rows -> QK operand, 16 lanes a row (16 bytes each), so
  // that a row is read in one piece; all eight loads of a thread in flight
  const int hf = (tid >> 7) & 1;                  // softmax warps: which half of its lanes, and of O's dims
  if (warp < 8) {
    const int ch = tid & 15;
    if (tid < kCtRows) own_sh[tid] = chunk_own(t, t.pos0 + tid / G, j0, j0 + n);
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 16 * i + (tid >> 4), tk = row / G;
      x[i] = make_uint4(0, 0, 0, 0);
      if (tk < t.ntok && row < p.tile_tokens * G)
        x[i] = reinterpret_cast<const uint4*>(p.q + ((int64_t)(t.row0 + tk) * p.q_heads + hk * G + (row - tk * G)) * D)[ch];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 16 * i + (tid >> 4);
      if constexpr (C::K16) {
        uint4 w = x[i];
        if (p.scale_log2 < 0.f) w = make_uint4(w.x ^ 0x80008000u, w.y ^ 0x80008000u, w.z ^ 0x80008000u, w.w ^ 0x80008000u);
        if (p.scale_log2 == 0.f) w = make_uint4(times_zero(w.x), times_zero(w.y), times_zero(w.z), times_zero(w.w));
        *reinterpret_cast<uint4*>(qop + (ch >> 3) * (kCtRows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = w;
      } else {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float f[8], amax = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float f2[2];
          bf16x2_to_f32(w[u], f2);
          f[2 * u] = f2[0];
          f[2 * u + 1] = f2[1];
          amax = fmaxf(amax, fmaxf(fabsf(f2[0]), fabsf(f2[1])));
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // smallest power of two that brings the row within 448 = 1.75 * 2^8; e4m3
        // has no infinity: a row with one becomes NaN, as its softmax is
        const int ab = __float_as_int(amax);
        const int kq = ab < 0x7F800000 ? max(-100, min(120, (ab >> 23) - 127 - 8 + ((ab & 0x7FFFFF) > 0x600000))) : 0;
        if (ch == 0) kq_sh[row] = (int8_t)kq;
        const float qsc = ab < 0x7F800000 ? pow2i(-kq) : NAN;
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float x0 = f[4 * u] * qsc, x1 = f[4 * u + 1] * qsc, x2 = f[4 * u + 2] * qsc, x3 = f[4 * u + 3] * qsc;
          float hv[4];
          hi[u] = e4m3x2_rn(x0, x1) | (e4m3x2_rn(x2, x3) << 16);
          e4m3x4_to_f32_scaled(hi[u], hv);
          lo[u] = e4m3x2_rn(x0 - hv[0] * kTwoPow120, x1 - hv[1] * kTwoPow120) |
                  (e4m3x2_rn(x2 - hv[2] * kTwoPow120, x3 - hv[3] * kTwoPow120) << 16);
        }
        const int off = row * 128 + (((ch >> 1) ^ (row & 7)) << 4) + (ch & 1) * 8;
        *reinterpret_cast<uint2*>(qop + off) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(qop + kCtRows * 128 + off) = make_uint2(lo[0], lo[1]);
      }
    }
    umma::fence_proxy_async_smem();
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tslot;
  const uint32_t o_col = tmem + 128;              // S and P: columns 0-63 and 64-127; O: 128-255

  if (warp >= 10) {
    if (warp == 10) {
      // ---------------------------------------------------------- producer
      // V tile j goes out behind K tile j + KN - VN (the K ring is the deeper
      // one); a V tile's page ids may be those of the group before
      int old_ids = ids, kdone = first_k, vdone = first_v;
      for (int i = first_k; i < n + LEAD; ++i) {
        if (i < n) {
          const bool ok = wait_fast(&kfree[i % C::KN], (i / C::KN - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) break;
          if ((i & 7) == 0) {
            old_ids = ids;
            ids = next_ids;
            next_ids = fetch_ids((i >> 3) + 1);
          }
          load_tile(i, false, ids);
          kdone = i + 1;
        }
        const int j = i - LEAD;
        if (j >= first_v) {
          const bool ok = wait_fast(&vfree[j % C::VN], (j / C::VN - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) break;
          load_tile(j, true, (j >> 3) == (min(i, n - 1) >> 3) ? ids : old_ids);
          vdone = j + 1;
        }
      }
      // no copy is in flight when the CTA ends (matters when a wait gave up)
      if (lane == 0) {
        for (int j = max(0, kdone - C::KN); j < kdone; ++j)
          (void)umma::mbar_wait(&kfull[j % C::KN], (j / C::KN) & 1, 100000000ull);
        for (int j = max(0, vdone - C::VN); j < vdone; ++j)
          (void)umma::mbar_wait(&vfull[j % C::VN], (j / C::VN) & 1, 100000000ull);
      }
    } else {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t ID_QK = C::K16 ? umma::idesc(umma::FMT_BF16, umma::FMT_BF16, umma::MAJOR_K, umma::MAJOR_K, 128, 64)
                                        : umma::idesc(umma::FMT_E4M3, umma::FMT_E4M3, umma::MAJOR_K, umma::MAJOR_K, 128, 64);
      constexpr uint32_t FV = C::V16 ? umma::FMT_BF16 : umma::FMT_F16;
      constexpr uint32_t ID_PV = umma::idesc(FV, FV, umma::MAJOR_K, umma::MAJOR_MN, 128, 128);
      const uint32_t qa = umma::smem_u32(qop);
      auto issue_qk = [&](int j) {
        const bool in = wait_fast(&kfull[j % C::KN], (j / C::KN) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, in)) return false;
        umma::fence_after_sync();
        const uint32_t ka = umma::smem_u32(kring + (j % C::KN) * C::KT), sd = tmem + 64 * (j & 1);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // e4m3: 32 dims a step, the four steps of hi and of lo meet the same
            // K; bf16: 16 dims a step, halves of 64 dims behind each other
            const uint64_t a = umma::sdesc(qa + (kk >> 2) * (kCtRows * 128) + (kk & 3) * 32, 16, 1024, umma::SWIZZLE_128B);
            const uint64_t b = umma::sdesc(ka + (C::K16 ? (kk >> 2) * (kChunkKeys * 128) : 0) + (kk & 3) * 32, 16, 1024,
                                           umma::SWIZZLE_128B);
            if constexpr (C::K16) umma::mma_f16_ss(sd, a, b, ID_QK, kk > 0);
            else umma::mma_f8_ss(sd, a, b, ID_QK, kk > 0);
          }
          umma::mma_commit(&s_full[j & 1]);
          umma::mma_commit(&kfree[j % C::KN]);
        }
        __syncwarp();
        return true;
      };
      bool ok = n > 0 && issue_qk(0);
      if (ok && n > 1) ok = issue_qk(1);
      for (int j = 0; ok && j < n; ++j) {
        const int ob = j % OPN;
        bool in = wait_fast(&op_full[ob], (j / OPN) & 1, abort_flag);
        in = in && wait_fast(&p_full[j & 1], (j >> 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, in)) break;
        umma::fence_after_sync();
        const uint32_t va = umma::smem_u32(vop + ob * (C::V16 ? C::VT : C::OPT)), pa = tmem + 64 * (j & 1);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ts(o_col, pa + 8 * kk, umma::sdesc(va + kk * 2048, kChunkKeys * 128, 1024, umma::SWIZZLE_128B), ID_PV,
                       (j > 0 || kk > 0) ? 1u : 0u);
          umma::mma_commit(pv_done);
          if constexpr (C::V16) umma::mma_commit(&vfree[ob]);
          else umma::mma_commit(&op_free[ob]);
        }
        __syncwarp();
        if (j + 2 < n) {
          // the scores of tile j + 2 go where P of tile j was
          in = wait_fast(pv_done, j & 1, abort_flag);
          if (!__all_sync(0xffffffffu, in)) break;
          ok = issue_qk(j + 2);
        }
      }
      // all issued MMAs complete before TMEM is released
      __syncwarp();
      if (elect_one()) umma::mma_commit(drained);
      (void)umma::mbar_wait(drained, 0, 100000000ull);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ preparation
    const int kr = tid - 256;                     // this thread's key of the tile
    // its scales come straight from the cache, a tile ahead, and the page id
    // (paged) two tiles ahead
    float next_k = 0.f, next_v = 0.f;
    auto key_seen = [&](int j) {
      const int key = j < n ? chunk_key0(t, j0 + j) + kr : INT32_MAX;
      return key < t.kv_end && (key >= t.lo || key < p.sinks) ? key : -1;
    };
    auto fetch_page = [&](int j) {
      const int key = c.paged ? key_seen(j) : -1;
      return key < 0 ? 0 : c.page_table[(int64_t)t.b * c.max_pages_per_seq + (key >> c.page_shift)];
    };
    auto fetch_scales = [&](int j, int page) {
      const int key = C::K16 && C::V16 ? -1 : key_seen(j);
      if (key < 0) return;
      if (page < 0 || page >= c.num_pages) page = 0;          // (reported by the producer)
      const int64_t row = c.paged ? ((int64_t)page * c.kv_heads + hk) * c.page_size + (key & (c.page_size - 1)) : cont0 + key;
      if constexpr (!C::K16) next_k = c.k_scale[row];
      if constexpr (!C::V16) next_v = c.v_scale[row];
    };
    fetch_scales(0, fetch_page(0));
    int page = fetch_page(1);
    for (int j = 0; j < n; ++j) {
      const int vs = j % C::VN, cb = j % C::NCOL, key0 = chunk_key0(t, j0 + j);
      bool ok = wait_fast(&vfull[vs], (j / C::VN) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t* st = vring + vs * C::VT;
      const float k_scale = next_k, v_scale = next_v;
      fetch_scales(j + 1, page);
      page = fetch_page(j + 2);
      const bool part = !chunk_all_seen(p, t, key0);
      float* cc = cols + cb * C::CST;
      auto seen = [&](int k) { return !part || (key0 + k < t.kv_end && (key0 + k >= t.lo || key0 + k < p.sinks)); };
      const bool vis = seen(kr);
      // per-key scales; in a tile that not every query sees whole they wait
      // for the values: a row with one that is not finite marks its key's score
      auto publish = [&](bool aside) {
        const float vv = C::V16 || !vis ? 0.f : v_scale;
        aside = (aside || !(fabsf(vv) < INFINITY)) && part && vis;
        cc[kr] = aside ? NAN : C::K16 ? 1.f : vis ? k_scale * p.scale_log2 : 0.f;
        if constexpr (!C::V16) cc[kChunkKeys + kr] = aside ? 0.f : vv;
        if constexpr (!C::V16) {                   // the largest finite value scale of these 32 keys
          const float vm = warp_max_f32(vv < INFINITY ? vv : 0.f);
          if (lane == 0) cc[2 * kChunkKeys + warp - 8] = vm;
        }
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&col_full[cb]);
      };
      if (!part) publish(false);
      if constexpr (C::V16) {
        if (part) {
          bool aside = false;
          for (int ch = 0; ch < 16; ++ch) {
            uint4* at = reinterpret_cast<uint4*>(st + (ch >> 3) * (kChunkKeys * 128) + kr * 128 + (((ch & 7) ^ (kr & 7)) << 4));
            const uint4 w = *at;
            uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            bool bad = false;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const bool b0 = (ww[u] & 0x7F80u) == 0x7F80u, b1 = (ww[u] & 0x7F800000u) == 0x7F800000u;
              if (b0 || !vis) ww[u] &= 0xFFFF0000u;
              if (b1 || !vis) ww[u] &= 0x0000FFFFu;
              bad = bad || b0 || b1;
            }
            aside = aside || bad;
            if (bad || !vis) *at = make_uint4(ww[0], ww[1], ww[2], ww[3]);
          }
          umma::fence_proxy_async_smem();
          publish(aside);
        }
        if (lane == 0) umma::mbar_arrive(&op_full[vs]);
      }
      if constexpr (!C::V16) {
        const int ob = j % C::NOP, ou = j / C::NOP;
        uint32_t w[32];                            // the key's 128 codes
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 x = *reinterpret_cast<const uint4*>(st + kr * 128 + ((ch ^ (kr & 7)) << 4));
          w[4 * ch] = x.x; w[4 * ch + 1] = x.y; w[4 * ch + 2] = x.z; w[4 * ch + 3] = x.w;
        }
        if (part) {
          bool aside = false;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t nan = (((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;   // 1 per NaN code
            aside = aside || nan != 0;
            w[k] = vis ? w[k] & ~(nan * 0xFFu) : 0u;
          }
          publish(aside);
        }
        if (ou > 0) {
          ok = wait_fast(&op_free[ob], (ou - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        uint8_t* dst = vop + ob * C::OPT + kr * 128;
#pragma unroll
        for (int ch = 0; ch < 16; ++ch)            // 8 dims each; 64 dims a half
          *reinterpret_cast<uint4*>(dst + (ch >> 3) * (kChunkKeys * 128) + (((ch & 7) ^ (kr & 7)) << 4)) =
              make_uint4(e4m3x2_to_f16x2((uint16_t)(w[2 * ch] & 0xFFFF)), e4m3x2_to_f16x2((uint16_t)(w[2 * ch] >> 16)),
                         e4m3x2_to_f16x2((uint16_t)(w[2 * ch + 1] & 0xFFFF)), e4m3x2_to_f16x2((uint16_t)(w[2 * ch + 1] >> 16)));
        umma::fence_proxy_async_smem();
        __syncwarp();
        // The stage is handed back only here, when the codes have been used.
        // (Handed back right behind the reads, it could be overwritten while
        // some were still pending: results differed from run to run.)
        if (lane == 0) {
          umma::mbar_arrive(&op_full[ob]);
          umma::mbar_arrive(&vfree[vs]);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // a warp reaches the 32 TMEM lanes of its quarter: warps w and w + 4 share
    // them, 16 rows each; this thread's rows are row0 + g + 8 i, with its quad
    const int row0 = 32 * (warp & 3) + 16 * hf;
    const uint32_t lane_off = (uint32_t)row0 << 16;
    const int g = lane >> 2, c2 = 2 * (lane & 3);
    int qpos[2];                                  // position (-1: no query)
    float s2[2], m_used[2], l[2], neg_m[2];
    float up[2];                                  // 2^kp
    float vm_top[2];                              // value scales below it need no larger kp
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + g + 8 * i, tk = row / G;
      qpos[i] = tk < t.ntok && row < p.tile_tokens * G ? t.pos0 + tk : -1;
      // what is left of the score's scale, positive (bf16 keys: the query
      // operand carries the sign, and is zero for a scale of zero)
      s2[i] = !C::K16 ? pow2i(kq_sh[row]) : p.scale_log2 != 0.f ? fabsf(p.scale_log2) : 1.f;
      up[i] = 1.f;
      m_used[i] = -INFINITY;
      l[i] = neg_m[i] = 0.f;
      vm_top[i] = FLT_MIN;
    }
    bool failed = false;
    for (int j = 0; j < n; ++j) {
      const int cb = j % C::NCOL, key0 = chunk_key0(t, j0 + j);
      const uint32_t s_col = tmem + 64 * (j & 1) + lane_off;
      bool ok = wait_fast(&col_full[cb], (j / C::NCOL) & 1, abort_flag);
      ok = ok && wait_fast(&s_full[j & 1], (j >> 1) & 1, abort_flag);
      ok = ok && !*abort_flag;
      if (!__all_sync(0xffffffffu, ok)) { failed = true; break; }
      umma::fence_after_sync();
      float2 sv[2][8];                            // row i, keys 8 k + c2, + 1
      {
        uint32_t rr[32];
        tmem_ld_256b_x8(s_col, rr);
        umma::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sv[i][k] = make_float2(__uint_as_float(rr[4 * k + 2 * i]), __uint_as_float(rr[4 * k + 2 * i + 1]));
      }
      const float* kc = cols + cb * C::CST + c2;
      const float* vc = kc + kChunkKeys;
      if constexpr (!C::K16) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 x = *reinterpret_cast<const float2*>(kc + 8 * k);
#pragma unroll
          for (int i = 0; i < 2; ++i) sv[i][k] = __fmul2_rn(sv[i][k], x);
        }
      }
      const float vmt = C::V16 ? 0.f : fmaxf(cols[cb * C::CST + 2 * kChunkKeys], cols[cb * C::CST + 2 * kChunkKeys + 1]);
      float vm[2] = {vmt, vmt};                   // largest value scale that the row sees
      if (!chunk_all_seen(p, t, key0)) {          // some query of the tile does not see all of its keys
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const unsigned long long seen = chunk_seen_mask(p, qpos[i], key0) >> c2;
          const uint32_t bits[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
          vm[i] = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 x = C::K16 ? *reinterpret_cast<const float2*>(kc + 8 * k) : make_float2(1.f, 1.f);
            const float2 v = C::V16 ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2*>(vc + 8 * k);
            const bool a = bits[k >> 2] & (1u << (8 * (k & 3))), b = bits[k >> 2] & (2u << (8 * (k & 3)));
            sv[i][k].x = a ? sv[i][k].x * x.x : -INFINITY;
            sv[i][k].y = b ? sv[i][k].y * x.y : -INFINITY;
            if constexpr (!C::V16) vm[i] = fmaxf(vm[i], fmaxf(a ? v.x : 0.f, b ? v.y : 0.f));
          }
        }
        if constexpr (!C::V16) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            vm[i] = fmaxf(vm[i], __shfl_xor_sync(0xffffffffu, vm[i], 1));
            vm[i] = fmaxf(vm[i], __shfl_xor_sync(0xffffffffu, vm[i], 2));
          }
        }
      }
      // the maximum of this thread's part of each row, by three-input max
      float mt[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mt[i] = max3(max3(max3(sv[i][0].x, sv[i][0].y, sv[i][1].x), max3(sv[i][1].y, sv[i][2].x, sv[i][2].y),
                          max3(sv[i][3].x, sv[i][3].y, sv[i][4].x)),
                     max3(sv[i][4].y, sv[i][5].x, sv[i][5].y), max3(max3(sv[i][6].x, sv[i][6].y, sv[i][7].x), sv[i][7].y, -INFINITY));
#pragma unroll
      for (int i = 0; i < 2; ++i) mt[i] *= s2[i];
      // The reference maximum moves only when it grows by more than 2^8 (P stays
      // within 2^8 of it), kp only up; l (in units of 2^m) and O (2^(m + kp))
      // move with them.  Rare behind the first tile: one vote on what each
      // thread sees skips it, and the row's maximum is joined only then.
      bool moved = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) moved = moved || mt[i] > m_used[i] + 8.f || (!C::V16 && vm[i] >= vm_top[i]);
      moved = __any_sync(0xffffffffu, moved);
      float alpha[2] = {1.f, 1.f};
      if (moved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 1));
          mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 2));
          if (mt[i] > m_used[i] + 8.f) {
            alpha[i] = ex2(m_used[i] - mt[i]);    // (0 for the first)
            m_used[i] = mt[i];
            l[i] *= alpha[i];
          }
          if (!C::V16 && vm[i] >= vm_top[i]) {
            const int need = max(-100, min(100, ((__float_as_int(vm[i]) >> 23) & 0xFF) - 127 - 6));   // vm 2^-need < 2^7
            alpha[i] *= pow2i(max(-126, (__float_as_int(up[i]) >> 23) - 127 - need));
            up[i] = pow2i(need);
            vm_top[i] = pow2i(need + 7);
          }
          neg_m[i] = (m_used[i] == -INFINITY ? 0.f : -m_used[i]) - (float)((__float_as_int(up[i]) >> 23) - 127);
        }
      }
      float2 la[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t ph[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 v = C::V16 ? make_float2(1.f, 1.f) : *reinterpret_cast<const float2*>(vc + 8 * k);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 a = __ffma2_rn(sv[i][k], make_float2(s2[i], s2[i]), make_float2(neg_m[i], neg_m[i]));
          float2 x = make_float2(ex2_ftz(a.x), ex2_ftz(a.y));
          la[i] = __fadd2_rn(la[i], x);
          uint32_t& w = ph[2 * k + i];
          if constexpr (C::V16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
            w = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            x = __fmul2_rn(x, v);
            const __half2 h = __floats2half2_rn(x.x, x.y);
            w = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) l[i] = fmaf(la[i].x + la[i].y, up[i], l[i]);
      tmem_st_128b_x8(s_col, ph);
      if (moved && j > 0) {
        // O may be rescaled only when the previous P.V is done.  (The parity is
        // unambiguous: the scores of this tile were issued behind the P.V before
        // that one, and the next P.V waits for this warp.)
        const bool done = wait_fast(pv_done, (j - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, done)) { failed = true; break; }
        umma::fence_after_sync();
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {             // 16 columns (head dims)
          const uint32_t at = o_col + lane_off + 16 * k;
          uint32_t rr[8];
          tmem_ld_256b_x2(at, rr);
          umma::tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u) rr[u] = __float_as_uint(__uint_as_float(rr[u]) * (u & 2 ? alpha[1] : alpha[0]));
          tmem_st_256b_x2(at, rr);
        }
      }
      tmem_wait_st();
      umma::fence_before_sync();
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&p_full[j & 1]);
    }
    // ---------------------------------------------------------------- epilogue
    if (!failed && n > 0) {
      // (a barrier of its own: a late warp cannot tell by pv_done's parity
      // whether the last phase or the one before it is over)
      const bool done = wait_fast(drained, 0, abort_flag) && !*abort_flag;
      failed = !__all_sync(0xffffffffu, done);
    }
    // one row and half of its dims per thread: the quads leave their rows'
    // (m, l, 2^kp) in the query operand's place, which no product reads any more
    float* st = reinterpret_cast<float*>(qop);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int row = row0 + g + 8 * i;
      if (c2 == 0 && !failed) {
        st[row] = m_used[i];
        st[kCtRows + row] = l[i];
        st[2 * kCtRows + row] = up[i];
      }
    }
    failed = softmax_any(failed);                 // (a barrier of the eight warps)
    if (failed && tid == 0) raise_error(p.err, FP8KV_DEVERR_TIMEOUT);
    const bool empty = failed || n == 0;          // O and the quads' values are not read
    umma::fence_after_sync();
    const int r = tid & 127, tok = r / G;          // row of the tile, TMEM lane
    const bool live = tok < t.ntok && r < p.tile_tokens * G;
    const int64_t qrow = live ? (int64_t)(t.row0 + tok) * p.q_heads + hk * G + (r - tok * G) : -1;
    const uint32_t lane_q = (uint32_t)(32 * (warp & 3)) << 16;
    const float mr = empty ? -INFINITY : st[r], lr = empty ? 0.f : st[kCtRows + r], of = empty ? 0.f : st[2 * kCtRows + r];
    const bool whole = p.num_splits == 1;
    const bool own = !failed && own_sh[r];
    const float f = whole ? of * chunk_inverse(lr, own) : of;
    const int64_t at = whole ? qrow : qrow * p.num_splits + split;
    if (!whole && live && hf == 0) { p.part_m[at] = mr; p.part_l[at] = chunk_share_sum(lr, own); }
#pragma unroll 1
    for (int k = 4 * hf; k < 4 * hf + 4; ++k) {
      uint32_t rr[16];
      if (!empty) {
        umma::tmem_ld16_nowait(o_col + lane_q + 16 * k, rr);
        umma::tmem_wait_ld();
      } else {
#pragma unroll
        for (int u = 0; u < 16; ++u) rr[u] = 0u;
      }
      if (!live) continue;
      float o[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) o[u] = __uint_as_float(rr[u]) * f;
      if (!whole || p.out_f32) {
        float4* dst = reinterpret_cast<float4*>((whole ? reinterpret_cast<float*>(p.out) : p.part_o) + at * D + 16 * k);
#pragma unroll
        for (int u = 0; u < 4; ++u) dst[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
      } else {
        uint32_t h[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(o[2 * u], o[2 * u + 1]);
          h[u] = *reinterpret_cast<const uint32_t*>(&x);
        }
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at * D + 16 * k);
        dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
        dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == 11) umma::tmem_dealloc(tmem, 256);
}

template <int KE, int VE>
static cudaError_t launch_one_tc(const ChunkParams& p, int tiles, cudaStream_t st) {
  using C = CtCfg<KE, VE>;
  const cudaError_t e = ensure_smem_optin((const void*)chunk_tc<KE, VE>, C::BYTES);
  if (e != cudaSuccess) return e;
  ChunkTcParams tp;
  const CacheView& c = p.c;
  const int64_t rows = c.paged ? (int64_t)c.num_pages * c.kv_heads * c.page_size
                               : (int64_t)c.batch * c.kv_heads * c.max_tokens;
  const int box = c.paged ? c.page_size : kChunkKeys;
  if (!make_map(&tp.tmk, c.k, C::K16, rows, box) || !make_map(&tp.tmv, c.v, C::V16, rows, box)) return cudaErrorInvalidValue;
  tp.p = p;
  chunk_tc<KE, VE><<<dim3(tiles, c.kv_heads, p.num_splits), kCtThreads, C::BYTES, st>>>(tp);
  return cudaGetLastError();
}

cudaError_t launch_chunk_tc(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  if (dtype == FP8KV_K8V8) return launch_one_tc<ELEM_E4M3, ELEM_E4M3>(p, tiles, st);
  if (dtype == FP8KV_K16V8) return launch_one_tc<ELEM_BF16, ELEM_E4M3>(p, tiles, st);
  if (dtype == FP8KV_K8V16) return launch_one_tc<ELEM_E4M3, ELEM_BF16>(p, tiles, st);
  return launch_one_tc<ELEM_BF16, ELEM_BF16>(p, tiles, st);
}

}  // namespace fp8kv
