// chunk_rows.cuh -- ragged chunk attention in tiles of at most sixteen query
// rows, for single tokens of a group of heads and a few drafted tokens: the cache
// is read once and nothing else takes as long, so the kernel is built around
// keeping loads in flight.  Also the form of block-scaled keys at any length
// (256-512 tokens x 8 heads, 4 sequences of 4K-8K: 0.71 ms, conversions and the
// four fp32 partial products of a score).
//
// The products are turned around so that the queries are the narrow side of the
// matrix instruction: S^T = K Q^T (16 keys x 8 queries per instruction) and
// O^T = V^T P^T (16 head dims x 8 queries).  A tile has one or two sets of eight
// queries (QT); two share the loads and conversions of K and V.  A warp owns
// groups of 16 keys: it copies their K and V rows and scales into its own ring
// (cp.async, no barrier between warps), and keeps its own running maximum m, sum
// l and O^T; the four warps of a CTA, and the splits of a long sequence, are
// joined at the end.  A group never crosses a page (pages hold 16 tokens or
// more), so a page id is looked up once per group, an iteration before its copy.
//
// Arithmetic as in chunk_mma.cuh: f16 operands for e4m3 sides (codes exact,
// query scaled by a power of two, P by 2^-kp and the value scale), bf16 for
// bf16 sides, m, l and O in fp32.  Here kp puts the largest value scale a row sees
// in [2^6, 2^7) (the reference may lag by 2^8), so a weight of 1 on a key whose
// value scale is 2^-20 of that is the smallest normal f16 number, and from there
// the step is 2^-31 of the largest seen value.  Block-scaled keys: the four
// 32-element partial products are scaled in fp32 and added.
//
// Measured on one GB300 (64 sequences, 32 query / 8 KV heads, head dim 128,
// e4m3, 16-token pages, device time): a 1,024-token window 30 us (140 MB: 4.6
// TB/s, 68 % of the measured copy rate); whole contexts of 1K-16K tokens, 2-4 tokens
// each, 181 us of a call's 189 (1.06 GB: 5.8 TB/s, 86 %).  What is left is the fixed
// part (about 5 us to find the tile, load the first groups and join) and latency: three
// to four warps a scheduler, 470 instructions a group of sixteen rows, 64 of them the
// conversion of 4,096 codes.  On the way there (the window): 58 us with
// a reference that moves at every new maximum and checked row copies; 46 us with
// one vote for both and whole-group copies, three CTAs an SM at four ring stages;
// 40 us with five CTAs at two; 36.5 us with four at three; 30.5 us with groups that
// every query sees in a form of their own (`weigh`: 33 instructions less, and the
// registers of the other form) and copies whose addresses take 32-bit row numbers
// (100 instructions instead of 158; sixteen rows 217 -> 194 us).  QK on e4m3
// instructions without conversion (mma.sync m16n8k32) was slower.  Two groups
// a step, which share the vote and the loop: slower too (67 KB of rings, three CTAs an
// SM, one wave and a bit).
//
// Sixteen rows (two tokens x 8 heads, 4 KV heads, 64 sequences of 2K-4K tokens,
// 210 MB): 56 us, three CTAs an SM at 168 registers (four at 128 registers leave 9 KB
// of first-level cache, where spilled registers and scales are lost: 25 % slower);
// 45 us for one token.  The second set costs its products, exponentials and transposes,
// not the codes' conversion.  The query's fragments in shared memory take 8 loads a
// group and give back 32 registers: 0.7 % faster, not kept.  16 heads on one KV head at
// head dim 64 (64 sequences of 4K-8K tokens) take 24 us.
#pragma once

#include <cfloat>
#include <type_traits>

#include "chunk_common.cuh"

namespace fp8kv {

constexpr int kRowKeys = 16;       // keys of a group

// QT: tiles of eight query rows (1 or 2)
template <int D, int KE, int VE, int QT>
struct RowsCfg {
  static constexpr int KB = KE == ELEM_BF16 ? 2 * D : D;
  static constexpr int VB = VE == ELEM_BF16 ? 2 * D : D;
  static constexpr int STAGE = kRowKeys * (KB + VB) + 2 * kRowKeys * 4;    // rows, key scales, value scales
  static constexpr int NS = KB + VB > 256 ? 2 : 3;
  static constexpr int OS = D + 4;
  static constexpr int JOIN = 32 * QT * OS * 4 + 2 * 32 * QT * 4;
  static constexpr int RING = 4 * NS * STAGE;
  static constexpr int BYTES = RING > JOIN ? RING : JOIN;
};

// 8x8 transposition of 16-bit elements held as a matrix fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void cp_async16_u(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4_u(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

template <bool TREE, int D, int KE, int VE, int QT>
__global__ void __launch_bounds__(kChunkThreads, QT == 1 ? 4 : 3) chunk_rows(const ChunkParams p) {
  using C = RowsCfg<D, KE, VE, QT>;
  constexpr int QC = 2 * QT;                   // score columns (queries) of a thread
  constexpr int QR = 8 * QT;                   // query rows of the tile
  constexpr bool KB16 = KE == ELEM_BF16, VB16 = VE == ELEM_BF16;
  constexpr int KS = D / 16;                   // k steps of QK, m tiles of PV
  extern __shared__ __align__(128) uint8_t rsm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c4 = lane & 3;
  ChunkTile t;
  ChunkPlace place;
  if (!chunk_tile<TREE>(p, place, t)) return;
  const int hk = place.hk, split = place.split;
  const CacheView& c = p.c;
  const int G = p.group;
  // groups of 16 keys: those of the first tokens, then the window's
  const int first = t.lo / kRowKeys;
  const int n_sink = p.window > 0 ? min((min(p.sinks, t.kv_end) + kRowKeys - 1) / kRowKeys, first) : 0;
  const int all = n_sink + max(0, (t.kv_end + kRowKeys - 1) / kRowKeys - first);
  const int per = (all + p.num_splits - 1) / p.num_splits;
  const int j0 = min(all, split * per) + warp, j1 = min(all, (split + 1) * per);      // this warp's groups j0, j0 + 4, ...
  const int skip = first - n_sink;
  auto group_key0 = [&](int j) { return (j < n_sink ? j : j + skip) * kRowKeys; };
  // The copies of a group take a third of the loop's instructions unless their addresses
  // are little work: rows are 31-bit numbers (of a page: page * row_step + row0 + its
  // token; contiguous: row0 + key), and a lane's three pointers to row 0 are kept.
  const unsigned row_step = c.kv_heads * c.page_size, num_pages = c.paged ? c.num_pages : 1;
  const unsigned row0 = c.paged ? hk * c.page_size : (unsigned)(t.b * c.kv_heads + hk) * c.max_tokens;
  const int key_mask = c.paged ? c.page_size - 1 : INT32_MAX;
  const int32_t* table = c.paged ? c.page_table + (int64_t)t.b * c.max_pages_per_seq : nullptr;
  int jf = j0;                                 // next group whose page is fetched
  auto fetch = [&](int& key0, int& page) {     // its first key (-1: none) and page
    key0 = -1;
    page = 0;
    if (jf < j1) {
      key0 = group_key0(jf);
      if (c.paged) page = table[key0 >> c.page_shift];
    }
    jf += 4;
  };
  uint8_t* ring = rsm + warp * C::NS * C::STAGE;
  const uint32_t ring_at = umma::smem_u32(ring);
  // Where a lane's chunks of a group go: chunk lane + 32 i lies 512 i bytes
  // behind chunk lane, with one placement (K) or two that alternate (V), since
  // 512 bytes hold a whole number of the rows after which the placement repeats
  constexpr int KC = C::KB / 16, VC = C::VB / 16, VALT = 32 / VC < 8 ? 8 / (32 / VC) : 1;
  static_assert(VALT <= 4, "rows of 64 bytes or more");
  const uint32_t kdst = (lane / KC) * C::KB + k_chunk<KE, C::KB>(lane % KC, lane / KC) * 16;
  uint32_t vdst[VALT];
#pragma unroll
  for (int i = 0; i < VALT; ++i)
    vdst[i] = ((lane + 32 * i) / VC) * C::VB + v_chunk<C::VB>(lane % VC, (lane + 32 * i) / VC) * 16 - 512 * i;
  auto issue = [&](uint32_t stage, int key0, int page) {      // stage: byte offset in the ring
    if (key0 >= 0) {
      const bool ok = (unsigned)page < num_pages;
      if (!ok && lane == 0) raise_error(p.err, FP8KV_DEVERR_BAD_PAGE);
      const unsigned row = (ok ? page : 0) * row_step + row0 + (unsigned)(key0 & key_mask);
      const uint32_t ks = ring_at + stage, vs = ks + kRowKeys * C::KB, sc = vs + kRowKeys * C::VB;
      // the 16 rows lie together: chunk e of the group is 16 e bytes from its start
      const uint8_t* ksrc = c.k + ((uint64_t)row * C::KB + lane * 16);
      const uint8_t* vsrc = c.v + ((uint64_t)row * C::VB + lane * 16);
      const float* ssrc = (lane < 16 ? c.k_scale : c.v_scale) + ((uint64_t)row + (lane & 15));
      // rows nobody sees are zero-filled, not read: they may hold anything
      const bool whole = ok && key0 + kRowKeys <= t.kv_end && (key0 >= t.lo || key0 + kRowKeys <= p.sinks);
      if (whole) {
#pragma unroll
        for (int i = 0; i < KC / 2; ++i) cp_async16_u(ks + kdst + 512 * i, ksrc + 512 * i);
#pragma unroll
        for (int i = 0; i < VC / 2; ++i) cp_async16_u(vs + vdst[i % VALT] + 512 * i, vsrc + 512 * i);
        if (lane < 16 ? !KB16 : !VB16) cp_async4_u(sc + lane * 4, ssrc);
      } else {
        auto live = [&](int r) { return ok && key0 + r < t.kv_end && (key0 + r >= t.lo || key0 + r < p.sinks); };
#pragma unroll
        for (int i = 0; i < KC / 2; ++i) cp_async16_z(ks + kdst + 512 * i, ksrc + 512 * i, live((lane + 32 * i) / KC));
#pragma unroll
        for (int i = 0; i < VC / 2; ++i)
          cp_async16_z(vs + vdst[i % VALT] + 512 * i, vsrc + 512 * i, live((lane + 32 * i) / VC));
        if (lane < 16 ? !KB16 : !VB16) cp_async4_z(sc + lane * 4, ssrc, live(lane & 15));
      }
    }
    cp_async_commit();
  };
  {
    int key0[C::NS - 1], page[C::NS - 1];
#pragma unroll
    for (int it = 0; it < C::NS - 1; ++it) fetch(key0[it], page[it]);
#pragma unroll
    for (int it = 0; it < C::NS - 1; ++it) issue(it * C::STAGE, key0[it], page[it]);
  }
  int next_key, next_page;
  fetch(next_key, next_page);

  // query rows g and g + 8 as B fragments; positions of this thread's score
  // columns, queries col(i)
  auto col = [&](int i) { return 8 * (i >> 1) + 2 * c4 + (i & 1); };
  uint32_t qb[QT][KS][2];
  float qf[QC];                                // what the scaled query leaves to undo, per score column
#pragma unroll
  for (int w = 0; w < QT; ++w) {
    const int r = g + 8 * w, tokr = r / G;
    const bool live = tokr < t.ntok && r < p.tile_tokens * G;
    const uint4* qsrc = reinterpret_cast<const uint4*>(
        p.q + (live ? (int64_t)(t.row0 + tokr) * p.q_heads + hk * G + (r - tokr * G) : 0) * D);
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const int at = KE == ELEM_E4M3 ? 8 * (u >> 1) + 2 * c4 + (u & 1) : 4 * u + c4;
      const uint4 x = live ? qsrc[at] : make_uint4(0, 0, 0, 0);
      qb[w][2 * u][0] = x.x; qb[w][2 * u][1] = x.y; qb[w][2 * u + 1][0] = x.z; qb[w][2 * u + 1][1] = x.w;
    }
    qf[2 * w] = qf[2 * w + 1] = 1.f;
    if constexpr (!KB16) {
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float f[2];
          bf16x2_to_f32(qb[w][k][u], f);
          amax = fmaxf(amax, fmaxf(fabsf(f[0]), fabsf(f[1])));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = ((__float_as_int(amax) >> 23) & 0xFF) - 127;
      const int up = amax > 0.f && e < 128 ? min(14 - e, 126) : 0;   // amax 2^up in [2^14, 2^15)
      const float sc = pow2i(up), down = pow2i(-up);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float f[2];
          bf16x2_to_f32(qb[w][k][u], f);
          qb[w][k][u] = pack16<false>(f[0] * sc, f[1] * sc);
        }
      qf[2 * w] = __shfl_sync(0xffffffffu, down, 8 * c4);
      qf[2 * w + 1] = __shfl_sync(0xffffffffu, down, 8 * c4 + 4);
    }
  }
  auto qpos = [&](int i) {                     // (asked in the few groups that are seen in part)
    const int r = col(i), tk = r / G;
    return tk < t.ntok && r < p.tile_tokens * G ? t.pos0 + tk : -1;
  };
#pragma unroll
  for (int i = 0; i < QC; ++i) qf[i] *= p.scale_log2;

  float o[QT][KS][4];
#pragma unroll
  for (int w = 0; w < QT; ++w)
#pragma unroll
    for (int u = 0; u < KS; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[w][u][e] = 0.f;
  // the reference maximum, the sum in units of 2^m, -m - kp, and 2^kp (a value scale
  // of 2^(kp + 7) or more lets it rise)
  float m[QC], l[QC], neg_m[QC], up2[QC];
#pragma unroll
  for (int i = 0; i < QC; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    neg_m[i] = VB16 ? 0.f : 100.f;
    up2[i] = VB16 ? 1.f : pow2i(-100);
  }

  uint32_t stage = 0;                          // byte offset of the group's place in the ring
#pragma unroll 1
  for (int jr = j0; jr < j1; jr += 4) {
    cp_async_wait<C::NS - 2>();
    __syncwarp();
    issue(stage == 0 ? (C::NS - 1) * C::STAGE : stage - C::STAGE, next_key, next_page);
    fetch(next_key, next_page);
    const uint8_t* st = ring + stage;
    stage = stage == (C::NS - 1) * C::STAGE ? 0 : stage + C::STAGE;
    const uint8_t* vst = st + kRowKeys * C::KB;
    const float* ksc = reinterpret_cast<const float*>(vst + kRowKeys * C::VB);
    const float* vsc = ksc + kRowKeys;
    const int key0 = group_key0(jr);
    // s[w][e]: key g + 8 (e >> 1), query col(2 w + (e & 1)); two chains of products
    float s[QT][4], s1[QT][4];
#pragma unroll
    for (int w = 0; w < QT; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[w][e] = s1[w][e] = 0.f;
    if constexpr (KE == ELEM_E4M3) {
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + g * C::KB + k_chunk<KE, C::KB>(4 * h + c4, g) * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(st + (g + 8) * C::KB + k_chunk<KE, C::KB>(4 * h + c4, g + 8) * 16);
        const uint32_t xx[4] = {x.x, x.y, x.z, x.w}, yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)xx[u]), e4m3x2_to_f16x2((uint16_t)yy[u]),
                                 e4m3x2_to_f16x2((uint16_t)(xx[u] >> 16)), e4m3x2_to_f16x2((uint16_t)(yy[u] >> 16))};
#pragma unroll
          for (int w = 0; w < QT; ++w)
            mma16816<false>(u & 1 ? s1[w] : s[w], a, qb[w][4 * h + u][0], qb[w][4 * h + u][1]);
        }
      }
      const float k0 = ksc[g], k1 = ksc[g + 8];
#pragma unroll
      for (int w = 0; w < QT; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[w][e] = (s[w][e] + s1[w][e]) * ((e >> 1 ? k1 : k0) * qf[2 * w + (e & 1)]);
    } else if constexpr (KE == ELEM_MX) {
      const uint32_t e0 = reinterpret_cast<const uint32_t*>(ksc)[g], e1 = reinterpret_cast<const uint32_t*>(ksc)[g + 8];
#pragma unroll
      for (int blk = 0; blk < D / 32; ++blk) {
        const int ch = 2 * blk + (c4 >> 1), in = (c4 & 1) * 8;
        const uint2 x = *reinterpret_cast<const uint2*>(st + g * C::KB + k_chunk<KE, C::KB>(ch, g) * 16 + in);
        const uint2 y = *reinterpret_cast<const uint2*>(st + (g + 8) * C::KB + k_chunk<KE, C::KB>(ch, g + 8) * 16 + in);
        const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)x.x), e4m3x2_to_f16x2((uint16_t)y.x),
                               e4m3x2_to_f16x2((uint16_t)(x.x >> 16)), e4m3x2_to_f16x2((uint16_t)(y.x >> 16))};
        const uint32_t b[4] = {e4m3x2_to_f16x2((uint16_t)x.y), e4m3x2_to_f16x2((uint16_t)y.y),
                               e4m3x2_to_f16x2((uint16_t)(x.y >> 16)), e4m3x2_to_f16x2((uint16_t)(y.y >> 16))};
        const float f0 = pow2_exact((int)((e0 >> (8 * blk)) & 0xFF) - 127), f1 = pow2_exact((int)((e1 >> (8 * blk)) & 0xFF) - 127);
#pragma unroll
        for (int w = 0; w < QT; ++w) {
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816<false>(part, a, qb[w][2 * blk][0], qb[w][2 * blk][1]);
          mma16816<false>(part, b, qb[w][2 * blk + 1][0], qb[w][2 * blk + 1][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[w][e] = fmaf(part[e], e >> 1 ? f1 : f0, s[w][e]);
        }
      }
#pragma unroll
      for (int w = 0; w < QT; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[w][e] *= qf[2 * w + (e & 1)];
    } else {
#pragma unroll
      for (int u = 0; u < D / 32; ++u) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + g * C::KB + k_chunk<KE, C::KB>(4 * u + c4, g) * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(st + (g + 8) * C::KB + k_chunk<KE, C::KB>(4 * u + c4, g + 8) * 16);
        const uint32_t a[4] = {x.x, y.x, x.y, y.y}, b[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
        for (int w = 0; w < QT; ++w) {
          mma16816<true>(s[w], a, qb[w][2 * u][0], qb[w][2 * u][1]);
          mma16816<true>(s1[w], b, qb[w][2 * u + 1][0], qb[w][2 * u + 1][1]);
        }
      }
#pragma unroll
      for (int w = 0; w < QT; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[w][e] = (s[w][e] + s1[w][e]) * qf[2 * w + (e & 1)];
    }
    // `part`: not every query sees all 16 keys
    auto weigh = [&](auto cut) {
      constexpr bool part = decltype(cut)::value;
      bool see[QT][4];
#pragma unroll
      for (int w = 0; w < QT; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) see[w][e] = true;
      if (part) {
        unsigned bits[QC];
#pragma unroll
        for (int i = 0; i < QC; ++i) bits[i] = TREE ? (unsigned)tree_seen_mask(p, t, qpos(i), key0) >> g : 0u;
#pragma unroll
        for (int w = 0; w < QT; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (TREE) see[w][e] = bits[2 * w + (e & 1)] >> (8 * (e >> 1)) & 1;
            else see[w][e] = chunk_sees(p, qpos(2 * w + (e & 1)), key0 + g + 8 * (e >> 1));
            if (!see[w][e]) s[w][e] = -INFINITY;
          }
      }
      // The reference moves only when the maximum grows by more than 2^8, kp only
      // up, and O with them: rare behind the first groups, one vote on what each
      // lane sees skips it, and the query's maximum is joined only then.
      [[maybe_unused]] const float v0 = VB16 ? 0.f : vsc[g], v1 = VB16 ? 0.f : vsc[g + 8];
      bool moved = false;
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        moved = moved || fmaxf(s[i >> 1][i & 1], s[i >> 1][2 + (i & 1)]) > m[i] + 8.f;
        if constexpr (!VB16) moved = moved || fmaxf(v0, v1) * 0.0078125f >= up2[i];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < QC; ++i) {
          const int w = i >> 1, j = i & 1;
          float alpha = 1.f, mt = fmaxf(s[w][j], s[w][2 + j]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
          if (mt > m[i] + 8.f) {
            alpha = ex2(m[i] - mt);              // (0 for the first)
            m[i] = mt;
            l[i] *= alpha;
          }
          if constexpr (!VB16) {                 // the largest finite value scale among the keys the query sees
            float vm = fmaxf(see[w][j] && v0 < INFINITY ? v0 : 0.f, see[w][2 + j] && v1 < INFINITY ? v1 : 0.f);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, x));
            if (vm * 0.0078125f >= up2[i]) {
              const int need = max(-100, min(100, ((__float_as_int(vm) >> 23) & 0xFF) - 127 - 6));   // vm 2^-need < 2^7
              alpha *= pow2i(max(-126, (__float_as_int(up2[i]) >> 23) - 127 - need));
              up2[i] = pow2i(need);
            }
          }
          neg_m[i] = (m[i] == -INFINITY ? 0.f : -m[i]) - (float)((__float_as_int(up2[i]) >> 23) - 127);
#pragma unroll
          for (int u = 0; u < KS; ++u) {
            o[w][u][j] *= alpha;
            o[w][u][2 + j] *= alpha;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        const int w = i >> 1, j = i & 1;
        s[w][j] = ex2_ftz(s[w][j] + neg_m[i]);
        s[w][2 + j] = ex2_ftz(s[w][2 + j] + neg_m[i]);
        l[i] = fmaf(s[w][j] + s[w][2 + j], up2[i], l[i]);
        if constexpr (!VB16) {
          s[w][j] *= v0;
          s[w][2 + j] *= v1;
          if (part) {                            // an unseen key's scale may be anything
            s[w][j] = see[w][j] ? s[w][j] : 0.f;
            s[w][2 + j] = see[w][2 + j] ? s[w][2 + j] : 0.f;
          }
        }
      }
      // P^T as B fragments: keys 2 c4, + 1 (and + 8) of queries g (and g + 8)
      uint32_t pb[QT][2];
#pragma unroll
      for (int w = 0; w < QT; ++w) {
        pb[w][0] = transpose8(pack16<VB16>(s[w][0], s[w][1]));
        pb[w][1] = transpose8(pack16<VB16>(s[w][2], s[w][3]));
      }
      bool aside = false;                        // values that must not meet an unseeing query's zero weight
      if (part && (TREE || t.ntok > 1)) {
        constexpr int VC = C::VB / 16;
        for (int e = lane; e < kRowKeys * VC; e += 32) {
          const uint4 w = *reinterpret_cast<const uint4*>(vst + e * 16);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if constexpr (VB16)
              aside = aside || (ww[u] & 0x7F800000u) == 0x7F800000u || (ww[u] & 0x7F80u) == 0x7F80u;
            else
              aside = aside || (((ww[u] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
          }
        }
        aside = __any_sync(0xffffffffu, aside);
      }
      const uint32_t vaddr = umma::smem_u32(vst);
      const int vr = lane & 15;
      // the two 16-dim A fragments of 32 bytes of V rows
      auto load_v = [&](int u, uint32_t (&a)[2][4]) {
        uint32_t r[4];
        ldsm_x4_trans(vaddr + vr * C::VB + v_chunk<C::VB>(2 * u + (lane >> 4), vr) * 16, r);
        if constexpr (VB16) {
          a[0][0] = r[0]; a[0][1] = r[2]; a[0][2] = r[1]; a[0][3] = r[3];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // two keys x two dims of codes -> the two keys of each dim
            const uint32_t w = __byte_perm(r[k], 0, 0x3120);
            a[k >> 1][2 * (k & 1)] = e4m3x2_to_f16x2((uint16_t)w);
            a[k >> 1][2 * (k & 1) + 1] = e4m3x2_to_f16x2((uint16_t)(w >> 16));
          }
        }
      };
      constexpr int MT = VB16 ? 1 : 2;           // m tiles per 32 bytes of a row
#pragma unroll
      for (int u = 0; u < C::VB / 32; ++u) {
        uint32_t a[2][4];
        load_v(u, a);
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          if (aside) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[k][e] = SetAside<VB16>(a[k][e]).clean;
          }
#pragma unroll
          for (int w = 0; w < QT; ++w) mma16816<VB16>(o[w][MT * u + k], a[k], pb[w][0], pb[w][1]);
        }
      }
      if (aside) {                               // rare: which queries see the values set aside
#pragma unroll
        for (int w = 0; w < QT; ++w) {
          const uint32_t z0 = transpose8(pack16<VB16>(see[w][0] ? 1.f : 0.f, see[w][1] ? 1.f : 0.f));
          const uint32_t z1 = transpose8(pack16<VB16>(see[w][2] ? 1.f : 0.f, see[w][3] ? 1.f : 0.f));
#pragma unroll
          for (int u = 0; u < C::VB / 32; ++u) {
            uint32_t a[2][4];
            load_v(u, a);
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              uint32_t an[4], ap[4], am[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const SetAside<VB16> x(a[k][e]);
                an[e] = x.nan; ap[e] = x.pinf; am[e] = x.ninf;
              }
              float nan[4] = {0.f, 0.f, 0.f, 0.f}, pinf[4] = {0.f, 0.f, 0.f, 0.f}, ninf[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<VB16>(nan, an, z0, z1);
              mma16816<VB16>(pinf, ap, z0, z1);
              mma16816<VB16>(ninf, am, z0, z1);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float& acc = o[w][MT * u + k][e];
                if (pinf[e] > 0.f) acc += INFINITY;
                if (ninf[e] > 0.f) acc -= INFINITY;
                if (nan[e] > 0.f) acc = NAN;
              }
            }
          }
        }
      }
    };
    if (chunk_all_seen<TREE, kRowKeys>(p, t, key0)) weigh(std::false_type());
    else weigh(std::true_type());
  }

#pragma unroll
  for (int i = 0; i < QC; ++i)
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
  // The kernel that joins the splits may be set up from here on: it waits for
  // this one's end.  Without splits the next kernel is a stranger, which may
  // count on this one's results as soon as it starts.
  if (p.num_splits > 1) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  // the four warps meet: [warp][query][D] in the rings' place
  cp_async_wait<0>();
  __syncthreads();
  float* osh = reinterpret_cast<float*>(rsm);
  float* msh = osh + 4 * QR * C::OS;
  float* lsh = msh + 4 * QR;
#pragma unroll
  for (int i = 0; i < QC; ++i) {
    const int r = warp * QR + col(i), w = i >> 1, j = i & 1;
    const float f = up2[i];
    if (g == 0) { msh[r] = m[i]; lsh[r] = l[i]; }
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      if constexpr (VB16) {
        osh[r * C::OS + 16 * u + g] = o[w][u][j];      // (2^kp is 1)
        osh[r * C::OS + 16 * u + 8 + g] = o[w][u][2 + j];
      } else {
        *reinterpret_cast<float2*>(osh + r * C::OS + 16 * u + 2 * g) = make_float2(o[w][u][j] * f, o[w][u][2 + j] * f);
      }
    }
  }
  __syncthreads();
  for (int e = tid; e < QR * (D / 4); e += kChunkThreads) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4, tk = r / G;
    if (tk >= t.ntok || r >= p.tile_tokens * G) continue;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) M = fmaxf(M, msh[QR * k + r]);
    float L = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float w = chunk_weight(msh[QR * k + r], lsh[QR * k + r], M);
      const float4 v = *reinterpret_cast<const float4*>(osh + (QR * k + r) * C::OS + d);
      L = fmaf(w, lsh[QR * k + r], L);
      x[0] = fmaf(w, v.x, x[0]); x[1] = fmaf(w, v.y, x[1]);
      x[2] = fmaf(w, v.z, x[2]); x[3] = fmaf(w, v.w, x[3]);
    }
    const int pos = t.pos0 + tk, jpos = pos / kRowKeys - first + n_sink;         // the group of the row's own key
    const bool own = pos >= 0 && jpos >= split * per && jpos < (split + 1) * per;
    chunk_store(p, (int64_t)(t.row0 + tk) * p.q_heads + hk * G + (r - tk * G), split, D, d, x, M, L, own);
  }
}

template <bool TREE, int D, int KE, int VE, int QT>
static cudaError_t launch_rows_one(const ChunkParams& p, dim3 grid, cudaStream_t st) {
  constexpr int smem = RowsCfg<D, KE, VE, QT>::BYTES;
  const cudaError_t e = ensure_smem_optin((const void*)chunk_rows<TREE, D, KE, VE, QT>, smem);
  if (e != cudaSuccess) return e;
  chunk_rows<TREE, D, KE, VE, QT><<<grid, kChunkThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <bool TREE, int D, int QT>
static cudaError_t launch_rows_types(const ChunkParams& p, int dtype, dim3 grid, cudaStream_t st) {
  if constexpr (D == 128)     // (MXFP8 keys are built for head_dim 128)
    if (dtype == FP8KV_MXK8V8) return launch_rows_one<TREE, D, ELEM_MX, ELEM_E4M3, QT>(p, grid, st);
  if (dtype == FP8KV_K8V8) return launch_rows_one<TREE, D, ELEM_E4M3, ELEM_E4M3, QT>(p, grid, st);
  if (dtype == FP8KV_K16V8) return launch_rows_one<TREE, D, ELEM_BF16, ELEM_E4M3, QT>(p, grid, st);
  if (dtype == FP8KV_K8V16) return launch_rows_one<TREE, D, ELEM_E4M3, ELEM_BF16, QT>(p, grid, st);
  return launch_rows_one<TREE, D, ELEM_BF16, ELEM_BF16, QT>(p, grid, st);
}

template <bool TREE>
static cudaError_t launch_rows(const ChunkParams& p, int dtype, int tiles, cudaStream_t st) {
  const dim3 grid(tiles, p.c.kv_heads, p.num_splits);
  if (p.tile_tokens * p.group > 8)
    return p.c.head_dim == 128 ? launch_rows_types<TREE, 128, 2>(p, dtype, grid, st) : launch_rows_types<TREE, 64, 2>(p, dtype, grid, st);
  return p.c.head_dim == 128 ? launch_rows_types<TREE, 128, 1>(p, dtype, grid, st) : launch_rows_types<TREE, 64, 1>(p, dtype, grid, st);
}

}  // namespace fp8kv
