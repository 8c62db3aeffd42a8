// chunk_mma.cuh -- ragged chunk attention over the cache on warp-level matrix
// instructions, for head dim 64 and many query rows (more than 32 a sequence).
//
// One pass over the keys with a running maximum m, sum l and output O:
//   s = (q . k) k_scale sm_scale log2(e),  m' = max(m, max s),
//   l = l 2^(m - m') + sum 2^(s - m'),     O = O 2^(m - m') + 2^(s - m') V
// 128 threads; a CTA owns 64 query rows of one KV head (rows = tokens x heads of
// the group), a warp 16 of them, and walks 64-key tiles through a ring of three
// cp.async stages.
//
// Operands.  e4m3 codes convert to f16 exactly, so QK runs in f16 with each
// bf16 query row scaled by a power of two to put its largest element in
// [2^14, 2^15): elements 2^-29 and more below it lose bits, an error of 2^-39
// of the largest.  The scale comes back in fp32.  bf16 keys meet the bf16
// query as they are.  The order of a row's elements inside a dot product is
// free, so a lane takes the 16 bytes that lie together and the query fragments
// use the same order: no shuffles, no transposition of K.
// P (16 bits, the one rounding of the softmax) is f16 next to e4m3 values,
// with the value scale folded in and a power of two 2^-kp that follows the
// largest value scale the row sees (to [2^14, 2^15): the step below 2^-28 of that is
// 2^-39 of the largest value; O is rescaled when it rises), and bf16 next to bf16
// values, since the instruction takes one 16-bit type.  m, l and O are fp32.
//
// What bounds it: instruction issue (conversions of codes are repeated by each
// of a tile's four warps).  The few-row kernel's 16-row tiles read the cache four times
// as often; at head dim 128 with block-scaled keys it is ahead all the same (128 fp32 of
// O and wider fragments leave two CTAs an SM here), so that form is gone.
//
// Keys that a query does not see get no weight, whatever their rows hold:
// rows that no query of the tile sees are not read at all, and in a tile that
// only some of the queries see, non-finite values are set aside and added
// to the queries that see them (a zero weight times NaN would not be zero).
//
// Measured on one GB300 (256-512 tokens x 8 heads of 4 sequences of 4K-8K tokens, 4 KV
// heads, e4m3): 394 us, issue slots bound it; 490 us while one form of the loop served
// tiles that every query sees and others alike.  Trees of 33-64 nodes x 8 heads, 16
// sequences of 2K-8K tokens: 217 us whole in that shape (290), 181 with the plan's shares;
// two CTAs an SM at 255 registers beside e4m3 values (three at 168 with spills 221), three
// beside bf16 ones and in chunk calls.
#pragma once

#include <type_traits>

#include "chunk_common.cuh"

namespace fp8kv {

template <int KE, int VE>
struct ChunkCfg {
  static constexpr int D = 64;
  static constexpr int KB = KE == ELEM_BF16 ? 2 * D : D;       // bytes of a K row
  static constexpr int VB = VE == ELEM_BF16 ? 2 * D : D;
  static constexpr int SC = KE == ELEM_BF16 && VE == ELEM_BF16 ? 0 : 2 * kChunkKeys * 4;
  static constexpr int STAGE = kChunkKeys * (KB + VB) + SC;
  static constexpr int NS = 3;
  static constexpr int BYTES = NS * STAGE + 4 * kChunkKeys * 4;
};

template <bool TREE, int KE, int VE>
__global__ void __launch_bounds__(kChunkThreads) chunk_mma(const ChunkParams p) {
  using C = ChunkCfg<KE, VE>;
  constexpr int D = C::D, NT = kChunkKeys / 8; // 8-key score tiles
  constexpr bool KB16 = KE == ELEM_BF16, VB16 = VE == ELEM_BF16;
  extern __shared__ __align__(128) uint8_t csm[];
  int* rows_sh = reinterpret_cast<int*>(csm + (C::BYTES - 4 * kChunkKeys * 4));   // [4][64] cache rows of coming tiles

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c4 = lane & 3;
  ChunkTile t;
  ChunkPlace place;
  if (!chunk_tile<TREE>(p, place, t)) return;
  const int hk = place.hk, split = place.split;
  const int per = (t.n + p.num_splits - 1) / p.num_splits;
  const int j0 = min(t.n, split * per), nt = min(t.n, j0 + per) - j0;
  const int G = p.group;

  // threads 0..63: this thread's key of tile `it`, its page and its cache row
  auto tile_key = [&](int it) { return chunk_key0(t, j0 + it) + tid; };
  auto find_page = [&](int it) { return tid < kChunkKeys && it < nt ? chunk_page(p, t, tile_key(it)) : 0; };
  auto find_row = [&](int it, int page) { return it < nt ? chunk_row(p, t, hk, tile_key(it), page) : -1; };
  auto issue = [&](int it) {
    if (it < nt) {
      uint8_t* st = csm + (it % C::NS) * C::STAGE;
      const uint32_t ks = umma::smem_u32(st), vs = ks + kChunkKeys * C::KB, sc = vs + kChunkKeys * C::VB;
      const int* rows = rows_sh + (it & 3) * kChunkKeys;
      constexpr int KC = C::KB / 16, VC = C::VB / 16;
#pragma unroll
      for (int i = 0; i < kChunkKeys * KC / kChunkThreads; ++i) {
        const int e = tid + i * kChunkThreads, r = e / KC, ch = e % KC, row = rows[r];
        cp_async16_z(ks + r * C::KB + k_chunk<KE, C::KB>(ch, r) * 16, p.c.k + (row < 0 ? 0 : (int64_t)row * C::KB + ch * 16),
                     row >= 0);
      }
#pragma unroll
      for (int i = 0; i < kChunkKeys * VC / kChunkThreads; ++i) {
        const int e = tid + i * kChunkThreads, r = e / VC, ch = e % VC, row = rows[r];
        cp_async16_z(vs + r * C::VB + v_chunk<C::VB>(ch, r) * 16, p.c.v + (row < 0 ? 0 : (int64_t)row * C::VB + ch * 16),
                     row >= 0);
      }
      if constexpr (C::SC > 0) {
        const int r = tid & 63, row = rows[r];
        const float* src = tid < 64 ? p.c.k_scale : p.c.v_scale;
        if (tid < 64 ? !KB16 : !VB16) cp_async4_z(sc + tid * 4, src + (row < 0 ? 0 : row), row >= 0);
      }
    }
    cp_async_commit();
  };

  // prologue: cache rows of the first NS tiles, loads of the first NS - 1
  if (tid < kChunkKeys)
    for (int it = 0; it < C::NS; ++it) rows_sh[(it & 3) * kChunkKeys + tid] = find_row(it, find_page(it));
  __syncthreads();
  for (int it = 0; it < C::NS - 1; ++it) issue(it);

  // the warp's 16 query rows as A fragments: rows g and g + 8
  int qpos[2];
  int64_t qrow[2];                             // row of out (query row x heads + head), -1: none
  const uint4* qsrc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = warp * 16 + g + 8 * i, tok = r / G;
    const bool live = tok < t.ntok && r < p.tile_tokens * G;
    qpos[i] = live ? t.pos0 + tok : -1;
    qrow[i] = live ? (int64_t)(t.row0 + tok) * p.q_heads + hk * G + (r - tok * G) : -1;
    qsrc[i] = reinterpret_cast<const uint4*>(p.q + (live ? qrow[i] : 0) * D);
  }
  constexpr int KS = D / 16;                   // k steps
  uint32_t qa[KS][4];
  float qf[2] = {1.f, 1.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[KS][2];                         // four elements of each step
    constexpr bool WIDE = KE == ELEM_E4M3;     // 16 elements together per lane (else 8)
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const int at = WIDE ? 8 * (u >> 1) + 2 * c4 + (u & 1) : 4 * u + c4;
      const uint4 x = qrow[i] >= 0 ? qsrc[i][at] : make_uint4(0, 0, 0, 0);
      w[2 * u][0] = x.x; w[2 * u][1] = x.y; w[2 * u + 1][0] = x.z; w[2 * u + 1][1] = x.w;
    }
    float sc = 1.f;
    if constexpr (!KB16) {
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float f[2];
          bf16x2_to_f32(w[k][u], f);
          amax = fmaxf(amax, fmaxf(fabsf(f[0]), fabsf(f[1])));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = ((__float_as_int(amax) >> 23) & 0xFF) - 127;       // amax in [2^e, 2^(e+1))
      const int up = min(14 - e, 126);
      if (amax > 0.f && e < 128) { sc = pow2i(up); qf[i] = pow2i(-up); }
    }
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t v = w[k][u];
        if constexpr (!KB16) {
          float f[2];
          bf16x2_to_f32(v, f);
          v = pack16<false>(f[0] * sc, f[1] * sc);
        }
        qa[k][2 * u + i] = v;
      }
  }

  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int kp[2] = {-1000, -1000};                  // exponent of P of each row (e4m3 values; none yet)

#pragma unroll 1
  for (int it = 0; it < nt; ++it) {
    cp_async_wait<C::NS - 2>();
    __syncthreads();                           // tile `it` has landed; every warp is done with tile it - 1
    issue(it + C::NS - 1);
    const int next_page = find_page(it + C::NS);
    const uint8_t* st = csm + (it % C::NS) * C::STAGE;
    const uint8_t* vst = st + kChunkKeys * C::KB;
    const float* ksc = reinterpret_cast<const float*>(vst + kChunkKeys * C::VB);
    const float* vsc = ksc + kChunkKeys;
    const int key0 = chunk_key0(t, j0 + it);

    // scores: s[n] holds rows g, g + 8 and keys 8 n + 2 c4, + 1
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int kr = 8 * n + g, kc = 8 * n + 2 * c4;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
      if constexpr (KE == ELEM_E4M3) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 w = *reinterpret_cast<const uint4*>(st + kr * C::KB + k_chunk<KE, C::KB>(4 * h + c4, kr) * 16);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mma16816<false>(s[n], qa[4 * h + u], e4m3x2_to_f16x2((uint16_t)ww[u]), e4m3x2_to_f16x2((uint16_t)(ww[u] >> 16)));
        }
        const float2 sc = *reinterpret_cast<const float2*>(ksc + kc);
        const float s0 = sc.x * p.scale_log2, s1 = sc.y * p.scale_log2;
        s[n][0] *= s0 * qf[0]; s[n][1] *= s1 * qf[0];
        s[n][2] *= s0 * qf[1]; s[n][3] *= s1 * qf[1];
      } else {
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          const uint4 w = *reinterpret_cast<const uint4*>(st + kr * C::KB + k_chunk<KE, C::KB>(4 * u + c4, kr) * 16);
          mma16816<true>(s[n], qa[2 * u], w.x, w.y);
          mma16816<true>(s[n], qa[2 * u + 1], w.z, w.w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] *= p.scale_log2;
      }
    }
    // `part`: not every query sees all 64 keys (a form of its own: the other tiles then
    // neither ask who sees what nor for values that must be set aside)
    auto weigh = [&](auto cut) {
      constexpr bool part = decltype(cut)::value;
      unsigned long long bits[2] = {0, 0};
      if (TREE && part) {
#pragma unroll
        for (int i = 0; i < 2; ++i) bits[i] = tree_seen_mask(p, t, qpos[i], key0);
      }
      auto sees = [&](int i, int key) {          // row i, key `key` of the tile (asked where it is seen in part)
        return TREE ? (bool)(bits[i] >> key & 1) : chunk_sees(p, qpos[i], key0 + key);
      };
      if (part) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!sees(e >> 1, 8 * n + 2 * c4 + (e & 1))) s[n][e] = -INFINITY;
      }
      // running maximum and weights
      float alpha[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mt = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) mt = fmaxf(mt, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
        const float mn = fmaxf(m[i], mt), ref = mn == -INFINITY ? 0.f : mn;
        alpha[i] = m[i] == -INFINITY ? 1.f : ex2_ftz(m[i] - ref);   // (nothing yet: O and l are zero)
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[n][2 * i] = ex2_ftz(s[n][2 * i] - ref);
          s[n][2 * i + 1] = ex2_ftz(s[n][2 * i + 1] - ref);
          sum += s[n][2 * i] + s[n][2 * i + 1];
        }
        l[i] = l[i] * alpha[i] + sum;
      }
      if constexpr (!VB16) {
        // the largest value scale among the keys that the row sees
        auto finite = [](float v) { return v < INFINITY ? v : 0.f; };
        float vm[2];
        if (!part) {
          vm[0] = vm[1] = warp_max_f32(fmaxf(finite(vsc[lane]), finite(vsc[lane + 32])));
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            vm[i] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int kc = 8 * n + 2 * c4 + e;
                if (sees(i, kc)) vm[i] = fmaxf(vm[i], finite(vsc[kc]));
              }
            vm[i] = fmaxf(vm[i], __shfl_xor_sync(0xffffffffu, vm[i], 1));
            vm[i] = fmaxf(vm[i], __shfl_xor_sync(0xffffffffu, vm[i], 2));
          }
        }
        float vf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int need = max(-100, min(100, ((__float_as_int(vm[i]) >> 23) & 0xFF) - 127 - 14));   // vm 2^-need < 2^15
          if (vm[i] > 0.f && need > kp[i]) {
            if (kp[i] > -1000) alpha[i] *= pow2_diff((float)(kp[i] - need), 0);
            kp[i] = need;
          }
          vf[i] = kp[i] > -1000 ? pow2i(-kp[i]) : 1.f;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 v = *reinterpret_cast<const float2*>(vsc + 8 * n + 2 * c4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = s[n][e] * ((e & 1 ? v.y : v.x) * vf[e >> 1]);
            // a scale that is not finite would turn an unseen key's zero into NaN
            s[n][e] = part && !sees(e >> 1, 8 * n + 2 * c4 + (e & 1)) ? 0.f : w;
          }
        }
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][0] *= alpha[0]; o[n][1] *= alpha[0];
          o[n][2] *= alpha[1]; o[n][3] *= alpha[1];
        }
      }
      // a tile seen by some of its queries only: are there values that must not
      // meet the others' zero weights?
      bool aside = false;
      if (part && (TREE || t.ntok > 1)) {
        constexpr int VC = C::VB / 16;
        for (int e = lane; e < kChunkKeys * VC; e += 32) {
          const uint4 w = *reinterpret_cast<const uint4*>(vst + e / VC * C::VB + (e % VC) * 16);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if constexpr (VB16)
              aside = aside || (ww[u] & 0x7F800000u) == 0x7F800000u || (ww[u] & 0x7F80u) == 0x7F80u;
            else
              aside = aside || ((((ww[u] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0);
          }
        }
        aside = __any_sync(0xffffffffu, aside);
      }
      // O += P V: 16 keys at a time
      const uint32_t vaddr = umma::smem_u32(vst);
#pragma unroll
      for (int j = 0; j < kChunkKeys / 16; ++j) {
        const uint32_t pa[4] = {pack16<VB16>(s[2 * j][0], s[2 * j][1]), pack16<VB16>(s[2 * j][2], s[2 * j][3]),
                                pack16<VB16>(s[2 * j + 1][0], s[2 * j + 1][1]), pack16<VB16>(s[2 * j + 1][2], s[2 * j + 1][3])};
        const int vr = 16 * j + (lane & 15);       // row this lane addresses for ldmatrix
#pragma unroll
        for (int u = 0; u < C::VB / 32; ++u) {
          uint32_t r[4];
          ldsm_x4_trans(vaddr + vr * C::VB + v_chunk<C::VB>(2 * u + (lane >> 4), vr) * 16, r);
          if constexpr (VB16) {
            if (aside) {
#pragma unroll
              for (int k = 0; k < 4; ++k) r[k] = SetAside<true>(r[k]).clean;
            }
            mma16816<true>(o[2 * u], pa, r[0], r[1]);
            mma16816<true>(o[2 * u + 1], pa, r[2], r[3]);
          } else {
            // two keys x two dims of e4m3 codes -> the two keys' pairs of each dim
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = __byte_perm(r[k], 0, 0x3120);
            uint32_t b[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              b[2 * k] = e4m3x2_to_f16x2((uint16_t)r[k]);
              b[2 * k + 1] = e4m3x2_to_f16x2((uint16_t)(r[k] >> 16));
            }
            if (aside) {
#pragma unroll
              for (int k = 0; k < 8; ++k) b[k] = SetAside<false>(b[k]).clean;
            }
            mma16816<false>(o[4 * u], pa, b[0], b[2]);
            mma16816<false>(o[4 * u + 1], pa, b[1], b[3]);
            mma16816<false>(o[4 * u + 2], pa, b[4], b[6]);
            mma16816<false>(o[4 * u + 3], pa, b[5], b[7]);
          }
        }
      }
      if (aside) {                               // rare: which queries see the values set aside
#pragma unroll
        for (int j = 0; j < kChunkKeys / 16; ++j) {
          uint32_t see[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = 16 * j + 8 * (k >> 1) + 2 * c4;
            see[k] = pack16<VB16>(sees(k & 1, key) ? 1.f : 0.f, sees(k & 1, key + 1) ? 1.f : 0.f);
          }
          auto add = [&](float (&acc)[4], uint32_t b0, uint32_t b1) {
            const SetAside<VB16> x(b0), y(b1);
            float nan[4] = {0.f, 0.f, 0.f, 0.f}, pinf[4] = {0.f, 0.f, 0.f, 0.f}, ninf[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<VB16>(nan, see, x.nan, y.nan);
            mma16816<VB16>(pinf, see, x.pinf, y.pinf);
            mma16816<VB16>(ninf, see, x.ninf, y.ninf);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (pinf[e] > 0.f) acc[e] += INFINITY;
              if (ninf[e] > 0.f) acc[e] -= INFINITY;
              if (nan[e] > 0.f) acc[e] = NAN;
            }
          };
          const int vr = 16 * j + (lane & 15);
#pragma unroll
          for (int u = 0; u < C::VB / 32; ++u) {
            uint32_t r[4];
            ldsm_x4_trans(vaddr + vr * C::VB + v_chunk<C::VB>(2 * u + (lane >> 4), vr) * 16, r);
            if constexpr (VB16) {
              add(o[2 * u], r[0], r[1]);
              add(o[2 * u + 1], r[2], r[3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) r[k] = __byte_perm(r[k], 0, 0x3120);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                add(o[4 * u + 2 * k], e4m3x2_to_f16x2((uint16_t)r[2 * k]), e4m3x2_to_f16x2((uint16_t)r[2 * k + 1]));
                add(o[4 * u + 2 * k + 1], e4m3x2_to_f16x2((uint16_t)(r[2 * k] >> 16)),
                    e4m3x2_to_f16x2((uint16_t)(r[2 * k + 1] >> 16)));
              }
            }
          }
        }
      }
    };
    if (chunk_all_seen<TREE>(p, t, key0)) weigh(std::false_type());
    else weigh(std::true_type());
    if (tid < kChunkKeys) rows_sh[((it + C::NS) & 3) * kChunkKeys + tid] = find_row(it + C::NS, next_page);
  }

#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }
  if constexpr (!VB16) {
    const float f[2] = {kp[0] > -1000 ? pow2i(kp[0]) : 1.f, kp[1] > -1000 ? pow2i(kp[1]) : 1.f};
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] *= f[e >> 1];
  }
  // four neighbouring elements of row g + 8 i: e4m3 values interleave two
  // accumulator tiles; bf16 values have two neighbours in each, and lanes 2 c
  // and 2 c + 1 swap a pair
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int u = 0; u < D / 16; ++u) {
      float x[4] = {o[2 * u][2 * i], o[2 * u + 1][2 * i], o[2 * u][2 * i + 1], o[2 * u + 1][2 * i + 1]};
      int d = 16 * u + 4 * c4;
      if constexpr (VB16) {
        const bool odd = c4 & 1;
        const float a = __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[1], 1);
        const float b = __shfl_xor_sync(0xffffffffu, odd ? x[2] : x[3], 1);
        const float own[2] = {odd ? x[1] : x[0], odd ? x[3] : x[2]};
        x[0] = odd ? a : own[0]; x[1] = odd ? b : own[1];
        x[2] = odd ? own[0] : a; x[3] = odd ? own[1] : b;
        d = 16 * u + (odd ? 8 : 0) + 4 * (c4 >> 1);
      }
      if (qrow[i] >= 0) chunk_store(p, qrow[i], split, D, d, x, m[i], l[i], chunk_own(t, qpos[i], j0, j0 + nt));
    }
}

template <bool TREE, int KE, int VE>
static cudaError_t launch_mma_one(const ChunkParams& p, dim3 grid, cudaStream_t st) {
  constexpr int smem = ChunkCfg<KE, VE>::BYTES;
  const cudaError_t e = ensure_smem_optin((const void*)chunk_mma<TREE, KE, VE>, smem);
  if (e != cudaSuccess) return e;
  chunk_mma<TREE, KE, VE><<<grid, kChunkThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <bool TREE>
static cudaError_t launch_mma(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  const dim3 grid(tiles, p.c.kv_heads, p.num_splits);
  if (dtype == FP8KV_K8V8) return launch_mma_one<TREE, ELEM_E4M3, ELEM_E4M3>(p, grid, st);
  if (dtype == FP8KV_K16V8) return launch_mma_one<TREE, ELEM_BF16, ELEM_E4M3>(p, grid, st);
  if (dtype == FP8KV_K8V16) return launch_mma_one<TREE, ELEM_E4M3, ELEM_BF16>(p, grid, st);
  return launch_mma_one<TREE, ELEM_BF16, ELEM_BF16>(p, grid, st);
}

}  // namespace fp8kv
