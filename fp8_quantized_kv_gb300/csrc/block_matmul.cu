// block_matmul.cu -- matrix product of e4m3 codes with an fp32 scale for each block
// of 128, on the tcgen05 tensor cores:
//   y[m][n] = sum_j sa[m][j] sb[n / 128][j] sum_{k in block j} a[m][k] b[n][k]  (+ bias[n])
// a: one scale per row and block of 128 elements of K (activations); b: one per
// block of 128 x 128 (weights).
//
// The scales change with every block of K, so the tensor core sums one block at a
// time (four kind::f8f6f4 products of 32 elements into a fresh TMEM buffer) and
// fp32 registers sum the blocks: acc = fma(d, sa sb, acc), one rounding of the pair
// of scales and one of each sum.  While one buffer is read the tensor core fills
// another.  Three kernels: a few rows of a are bound by the bytes of b (fragments
// straight from memory, or shares of K in clusters), many by the products and by the
// hand-over of each block's sums (pairs of CTAs).  Measured on one GB300, device time:
// 1 x 2560 x 2048 2.5 us; 64 x 6144 x 4096 10.8 us (25 MB: 2.4 TB/s; 4.9 TB/s at 32,768
// columns); 997 x 4608 x 3584 17.7 us (1,860 TFLOP/s); 7940 x 6144 x 4096 170 us (2,350
// TFLOP/s, 1.23 times the measured bf16 rate); 8192^3 412 us (2,670 TFLOP/s).
#include <type_traits>

#include "params.cuh"
#include "tc_common.cuh"

namespace fp8kv {

constexpr int kMmBlock = 128;            // elements of a block of K: one 128-byte swizzled row
// A CTA's last wait for what another of its cluster sends, in ns: longer than the other
// takes to give up where its waits run out (kWaitLimitCycles, about 2 s) and send.
constexpr uint64_t kMmLastWait = 5000000000ull;

struct MatmulParams {
  CUtensorMap ta, tb, to;
  CUtensorMap th;                        // b for half tiles
  MatmulArgs a;
  int kb;                                // blocks of K
  int tiles_m, tiles_n;
  int whole;                             // pairs of CTAs: tiles before the first that is cut into halves
  int bulk_out;                          // rows of out start on 16 bytes: stored by TMA (map `to`)
};

// 32 columns of TMEM into registers, and the wait for this thread's loads: the values
// are named there, so that nothing that uses them moves in front.
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// Columns n0 .. n0 + 63 of row m of out, as far as there are any: for widths whose rows do
// not start on 16 bytes, element by element, 32 rows an instruction (others are stored by
// TMA).  997 x 4609 x 3584: 63 us in bf16, 39 in fp32, where 4608 columns take 17.1 and 18.5.
__device__ __forceinline__ void store_row64(const MatmulArgs& a, int m, int n0, float2* acc) {
  const int cols = min(64, a.N - n0);
  if (cols <= 0) return;
  if (a.bias != nullptr) {
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      if (2 * c < cols) acc[c].x += a.bias[n0 + 2 * c];
      if (2 * c + 1 < cols) acc[c].y += a.bias[n0 + 2 * c + 1];
    }
  }
  const int64_t out = (int64_t)m * a.N + n0;
  if (a.out_f32) {
    float* y = reinterpret_cast<float*>(a.out) + out;
#pragma unroll
    for (int c = 0; c < 64; ++c)
      if (c < cols) y[c] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
  } else {
    __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(a.out) + out;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(acc[c].x, acc[c].y);
      if (2 * c < cols) y[2 * c] = h.x;
      if (2 * c + 1 < cols) y[2 * c + 1] = h.y;
    }
  }
}
// Columns n .. n + 3 of row m of out (n a multiple of 4), as far as there are any.
__device__ __forceinline__ void store_row4(const MatmulArgs& a, int m, int n, float4 y) {
  const int cols = a.N - n;
  if (a.bias != nullptr) {
    y.x += a.bias[n];
    if (cols > 1) y.y += a.bias[n + 1];
    if (cols > 2) y.z += a.bias[n + 2];
    if (cols > 3) y.w += a.bias[n + 3];
  }
  const int64_t at = (int64_t)m * a.N + n;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
  if (a.N % 4 == 0) {
    if (a.out_f32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = y;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    return;
  }
  const float v[4] = {y.x, y.y, y.z, y.w};
  const __nv_bfloat16 w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u < cols) {
      if (a.out_f32) reinterpret_cast<float*>(a.out)[at + u] = v[u];
      else reinterpret_cast<__nv_bfloat16*>(a.out)[at + u] = w[u];
    }
}
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }

// A warp's 32 rows of out from row m0 on, HC columns from n0 on (lane: row), staged in
// `buf` (8 KB, two boxes of 32 rows x 128 bytes, swizzled) and stored by TMA, which
// cuts what lies outside.  (Stored by the threads, 16 bytes of 32 rows an
// instruction, a tile's end took 2.5 us.)  The warp goes on while the stores run.
template <int HC>
__device__ __forceinline__ void store_rows(const MatmulParams& p, uint8_t* buf, int lane, int m0, int n0, float2* acc) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");     // the last stores have read the buffer
  __syncwarp();
  if (p.a.bias != nullptr) {                                  // (in the buffer for as long as it is added)
    float* b = reinterpret_cast<float*>(buf);
#pragma unroll
    for (int c = 0; c < HC / 32; ++c) b[32 * c + lane] = n0 + 32 * c + lane < p.a.N ? p.a.bias[n0 + 32 * c + lane] : 0.f;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < HC / 4; ++c) {
      const float4 x = reinterpret_cast<const float4*>(b)[c];
      acc[2 * c].x += x.x; acc[2 * c].y += x.y; acc[2 * c + 1].x += x.z; acc[2 * c + 1].y += x.w;
    }
    __syncwarp();
  }
  auto put = [&](int box, int chunk, uint4 v) { *reinterpret_cast<uint4*>(buf + box * 4096 + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = v; };
  auto send = [&](int box, int n) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(
                     reinterpret_cast<uint64_t>(&p.to)),
                 "r"(n), "r"(m0), "r"(umma::smem_u32(buf + box * 4096))
                 : "memory");
  };
  if (!p.a.out_f32) {
#pragma unroll
    for (int c = 0; c < HC / 8; ++c) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) h[u] = __floats2bfloat162_rn(acc[4 * c + u].x, acc[4 * c + u].y);
      put(c / 8, c % 8, *reinterpret_cast<const uint4*>(h));
    }
    umma::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && m0 < p.a.M) {
#pragma unroll
      for (int b = 0; b < HC / 64; ++b)
        if (n0 + 64 * b < p.a.N) send(b, n0 + 64 * b);
      asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
    }
  } else {
#pragma unroll
    for (int q = 0; q < HC / 64; ++q) {                       // two boxes of 32 columns at a time
      if (q > 0) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
        __syncwarp();
      }
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float2 x = acc[32 * q + 2 * c], y = acc[32 * q + 2 * c + 1];
        const float4 v = make_float4(x.x, x.y, y.x, y.y);
        put(c / 8, c % 8, *reinterpret_cast<const uint4*>(&v));
      }
      umma::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && m0 < p.a.M) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          if (n0 + 64 * q + 32 * b < p.a.N) send(b, n0 + 64 * q + 32 * b);
        asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
      }
    }
  }
}

// ---------------------------------------------------------- many rows of a --
// A pair of CTAs (cta_group::2) owns tiles of 256 rows of a x BN rows of b, one after
// the other: each CTA loads and keeps 128 rows of a and half of b's, the products read
// b from both, and each CTA's TMEM holds its own 128 rows of the sums.
//   warp 0      TMA producer: ring of a and b blocks; every copy counts on the first
//               CTA's barrier
//   warp 1      TMEM owner; the first CTA's issues the products
//   warps 4-11  sums: a thread keeps one row of the tile and half of its columns
// Where the last wave would leave half of the pairs or more without a tile, its tiles
// are cut into halves of 128 columns (launch_pair).
//
// The end.  Arrivals on the other CTA's barriers and copies that count there may still
// be under way when a CTA has nothing left to do, and the cluster barrier alone (relaxed:
// a release would wait for the stores of out) orders none of them.  So each CTA first
// waits for everything that is sent to it: the producer for its last `empty` phases and
// `drained`, the issuer for the last `d_free` phases, the warps of sums have seen every
// `d_full`, and the products every `full`.  Where a wait gave up, either CTA tells the
// other, and the first one then waits for the copies of both before the pair ends.
//
// What bounds 256 columns: a block's products take about 640 cycles back to back, but
// with two TMEM buffers a block also waits for half of the way round a buffer: products
// until their sums are seen (820 cycles), reading (450), hand-back to the issuer (250).
// On the way (997 x 4608 x 3584 and 8192^3, us):
//   one CTA, 128 x 256, sums of a whole row's half in pieces of 32       23.5   572
//   pairs (8192^3 without any hand-over: 302)                            21.3   461
//   output by TMA instead of 16-byte stores of 32 rows                   18.7   430
//   two pieces on their way at once, hand-back before the last products  18.0   425
//   one thread each for copies and products                              18.0   412
// Measured and not kept: sixteen warps of sums with 64 columns each (22.1, 571: twice the
// instructions around the sums), buffers of 128 columns (26.4, 610: products of 128
// columns take 116 cycles instead of 160 for 256), scalar sums instead of packed pairs
// (23.6, 623), barriers tested without suspension (18.6, 437), a release at cluster scope
// for the hand-back (36, 1150).
template <int BN>
struct MmCfg {
  static constexpr int STAGE = (128 + BN / 2) * kMmBlock;     // of one CTA
  static constexpr int NS = BN == 256 ? 5 : 6;
  static constexpr int NB = 512 / BN;                         // TMEM buffers
  static constexpr int THREADS = 384;
  static constexpr int OUT = 8 * 8192;                        // staged output, 8 KB a warp of sums
  static constexpr int BYTES = 1024 + NS * STAGE + OUT + 512;
  static_assert(BYTES <= 227 * 1024, "shared memory of an SM");
};

namespace pair {
__device__ __forceinline__ void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(umma::smem_u32(dst_smem)), "r"(ncols));
}
__device__ __forceinline__ void tmem_relinquish() { asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::); }
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols));
}
// D (both CTAs' TMEM) (+)= A x B^T, 256 rows; one thread of the first CTA issues.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
// Arrive on the barrier at this place in both CTAs when all products issued before are complete.
__device__ __forceinline__ void mma_commit(uint64_t* mbar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                   umma::smem_u32(mbar)),
               "h"((uint16_t)3)
               : "memory");
}
// Tile load into this CTA; its bytes count on the barrier of the first CTA, given
// by its shared::cluster address.
__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n" ::"r"(umma::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrive on a barrier of either CTA (shared::cluster address).  It orders reads of
// TMEM, which the tcgen05 fence in front covers, and no shared memory: at cluster
// scope the release costs a microsecond.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// A word of either CTA's shared memory (this CTA's address of it).
__device__ __forceinline__ void store_word(volatile int* at, uint32_t rank, int value) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(mapa_u32(umma::smem_u32(const_cast<int*>(at)), rank)), "r"(value) : "memory");
}
// Count `bytes` that never arrive as arrived.
__device__ __forceinline__ void complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(umma::smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cluster_arrive_release() { asm volatile("barrier.cluster.arrive.release;\n" ::: "memory"); }
}  // namespace pair

// The tiles of a pair: tile first, first + step, ... of the whole ones, then (CUT) a half.
template <bool CUT>
struct MmTile {
  int m0, n0;
  bool half;
  __device__ __forceinline__ bool get(const MatmulParams& p, int bn, int i) {
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1, tiles = p.tiles_m * p.tiles_n;
    int t = first + i * step, side = 0;
    half = CUT && t >= p.whole;
    if (half) {
      t -= p.whole;
      side = t & 1;
      t = p.whole + (t >> 1);
    }
    if (t >= tiles) return false;
    m0 = t % p.tiles_m * 256;
    n0 = t / p.tiles_m * bn + 128 * side;
    return true;
  }
};

template <int BN, bool CUT>
__global__ void __launch_bounds__(MmCfg<BN>::THREADS, 1) block_matmul_pair(const __grid_constant__ MatmulParams p) {
  using C = MmCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staged = smem + C::NS * C::STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staged + C::OUT);
  uint64_t* full = bars;                                      // [NS] first CTA: both CTAs' blocks landed
  uint64_t* empty = full + C::NS;                             // [NS] products have read them
  uint64_t* d_full = empty + C::NS;                           // [NB] a block's sums are in TMEM
  uint64_t* d_free = d_full + C::NB;                          // [NB] first CTA: both CTAs have read them
  uint64_t* drained = d_free + C::NB;                         // every product finished
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile int* issued = abort_flag + 1;                      // [2] blocks that each CTA has copied, in both
  static_assert(8 * (2 * C::NS + 2 * C::NB + 1) + 4 * 4 <= 512, "they fit");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  MmTile<CUT> tile;
  if (tid == 0) {
    tma::prefetch_map(&p.ta);
    tma::prefetch_map(&p.tb);
    for (int i = 0; i < C::NS; ++i) { umma::mbar_init(&full[i], 1); umma::mbar_init(&empty[i], 1); }
    for (int i = 0; i < C::NB; ++i) { umma::mbar_init(&d_full[i], 1); umma::mbar_init(&d_free[i], 16); }
    umma::mbar_init(drained, 1);
    *abort_flag = 0;
    umma::mbar_fence_init();
  }
  cluster_arrive_relaxed();                                   // (thread 0's barriers are initialised: fence above)
  cluster_wait();
  // TMEM is there before it is used, not before the first copies
  uint32_t tmem = 0;
  if (warp == 1) {
    pair::tmem_alloc(tslot, 512);
    pair::tmem_relinquish();
    umma::fence_before_sync();
  }
  if (warp == 1 || warp >= 4) {
    asm volatile("bar.sync 1, 288;\n" ::: "memory");
    umma::fence_after_sync();
    tmem = *tslot;
  }

  if (warp < 4) {
    regs_dec<40>();
    if (warp == 0) {
      if (elect_one()) {                                      // (one thread: see the issuer below)
        const uint32_t full0 = mapa_u32(umma::smem_u32(full), 0);
        int it = 0;
        bool ok = true;
        for (int i = 0; ok && tile.get(p, BN, i); ++i) {
          const bool half = CUT && tile.half;
          const int m0 = tile.m0 + 128 * rank, n0 = tile.n0 + (half ? 64 : BN / 2) * rank;
          for (int j = 0; j < p.kb; ++j, ++it) {
            const int s = it % C::NS;
            if (it >= C::NS) ok = wait_fast(&empty[s], (it / C::NS - 1) & 1, abort_flag);
            if (!ok) break;
            uint8_t* st = smem + s * C::STAGE;
            const uint32_t bar = full0 + 8 * s;
            if (rank == 0) tma::arrive_expect_tx(&full[s], half ? 2 * (128 + 64) * kMmBlock : 2 * C::STAGE);
            pair::load_2d(st, &p.ta, j * kMmBlock, m0, bar);
            pair::load_2d(st + 128 * kMmBlock, half ? &p.th : &p.tb, j * kMmBlock, n0, bar);
          }
        }
#pragma unroll 1
        for (int i = max(0, it - C::NS); ok && i < it; ++i) ok = wait_fast(&empty[i % C::NS], (i / C::NS) & 1, abort_flag);
        (void)umma::mbar_wait(drained, 0, kMmLastWait);
        pair::store_word(issued + rank, 0, it);
        pair::store_word(issued + rank, 1, it);
      }
    } else if (warp == 1 && rank == 0) {
      constexpr uint32_t ID = umma::idesc(umma::FMT_E4M3, umma::FMT_E4M3, umma::MAJOR_K, umma::MAJOR_K, 256, BN);
      // One thread: a converged warp that elects one for each instruction takes longer
      // from block to block (200 x 6144 x 4096: 15.5 us; the issuer so 13.5, the producer
      // too 12.8).
      if (elect_one()) {
        int it = 0;
        bool ok = true, full_ok = false, free_ok = true;
        for (int i = 0; ok && tile.get(p, BN, i); ++i) {
          const uint32_t id = CUT && tile.half ? umma::idesc(umma::FMT_E4M3, umma::FMT_E4M3, umma::MAJOR_K, umma::MAJOR_K, 256, 128) : ID;
          for (int j = 0; j < p.kb; ++j, ++it) {
            const int s = it % C::NS, d = it % C::NB;
            const int next = it + 1;
            if (!full_ok) ok = wait_fast(&full[s], (it / C::NS) & 1, abort_flag);
            if (!free_ok) ok = ok && wait_fast(&d_free[d], (it / C::NB - 1) & 1, abort_flag);
            if (!ok) break;
            umma::fence_after_sync();
            const uint32_t aa = umma::smem_u32(smem + s * C::STAGE), ba = aa + 128 * kMmBlock;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k == 2) {
                free_ok = next < C::NB || umma::mbar_test(&d_free[next % C::NB], (next / C::NB - 1) & 1);
                full_ok = umma::mbar_test(&full[next % C::NS], (next / C::NS) & 1);
              }
              pair::mma_f8(tmem + d * BN, umma::sdesc(aa + 32 * k, 16, 1024, umma::SWIZZLE_128B),
                           umma::sdesc(ba + 32 * k, 16, 1024, umma::SWIZZLE_128B), id, k > 0);
            }
            pair::mma_commit(&d_full[d]);
            pair::mma_commit(&empty[s]);
          }
        }
        // all issued products complete before TMEM is released
        pair::mma_commit(drained);
        (void)umma::mbar_wait(drained, 0, 100000000ull);
#pragma unroll 1
        for (int i = max(0, it - C::NB); ok && i < it; ++i) ok = wait_fast(&d_free[i % C::NB], (i / C::NB) & 1, abort_flag);
      }
    }
  } else {
    regs_inc<232>();
    const int part = (warp - 4) >> 2, row_in = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t free0 = mapa_u32(umma::smem_u32(d_free), 0);
    int it = 0;
    bool ok = true, ready = false;
    // a tile of which a thread keeps HC columns
    auto run = [&](auto columns) {
      constexpr int HC = decltype(columns)::value, PC = HC / 32;             // in pieces of 32
      const int m = tile.m0 + 128 * rank + row_in, n0 = tile.n0 + HC * part;
      const uint32_t base = lanes + HC * part;
      const float* sa = p.a.sa + (int64_t)min(m, p.a.M - 1) * p.kb;
      const float* sb = p.a.sb + (int64_t)(n0 < p.a.N ? n0 / 128 : 0) * p.kb;
      float2 acc[HC / 2];
#pragma unroll
      for (int c = 0; c < HC / 2; ++c) acc[c] = make_float2(0.f, 0.f);
      float next_a = sa[0], next_b = sb[0];
      for (int j = 0; j < p.kb; ++j, ++it) {
        const int d = it % C::NB, next = it + 1;
        const uint32_t at = base + BN * d;
        if (!ready) ok = wait_fast(&d_full[d], (it / C::NB) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; return; }
        umma::fence_after_sync();
        // The buffer is handed back as soon as it is read: two pieces of 32 columns are
        // on their way at once, and the last two are multiplied behind the hand-back.
        uint32_t r[2][32];
        tmem_ld32_nowait(at, r[0]);
        tmem_ld32_nowait(at + 32, r[1]);
        const float2 s2 = make_float2(next_a * next_b, next_a * next_b);
        if (j + 1 < p.kb) { next_a = sa[j + 1]; next_b = sb[j + 1]; }
        auto sum = [&](int c) {
#pragma unroll
          for (int u = 0; u < 16; ++u)
            acc[16 * c + u] = __ffma2_rn(make_float2(__uint_as_float(r[c & 1][2 * u]), __uint_as_float(r[c & 1][2 * u + 1])), s2,
                                         acc[16 * c + u]);
        };
        tmem_wait_ld32(r[0]);
        tmem_wait_ld32(r[1]);
        if constexpr (PC == 4) {
          sum(0);
          tmem_ld32_nowait(at + 64, r[0]);
          sum(1);
          tmem_ld32_nowait(at + 96, r[1]);
          tmem_wait_ld32(r[0]);
          tmem_wait_ld32(r[1]);
        }
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) pair::arrive_remote(free0 + 8 * d);
        ready = umma::mbar_test(&d_full[next % C::NB], (next / C::NB) & 1);
        sum(PC - 2);
        sum(PC - 1);
      }
      if (p.bulk_out) {
        store_rows<HC>(p, staged + (warp - 4) * 8192, lane, m - lane, n0, acc);
      } else if (m < p.a.M) {
#pragma unroll
        for (int c = 0; c < HC / 64; ++c) store_row64(p.a, m, n0 + 64 * c, acc + 32 * c);
      }
    };
    for (int i = 0; ok && tile.get(p, BN, i); ++i) {
      if constexpr (CUT) {
        if (tile.half) {
          run(std::integral_constant<int, 64>());
          continue;
        }
      }
      run(std::integral_constant<int, BN / 2>());
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
    if (!ok && lane == 0) raise_error(p.a.err, FP8KV_DEVERR_TIMEOUT);
  }
  // neither CTA's shared memory or TMEM is in use by the other any more
  umma::fence_before_sync();
  __syncwarp();
  const bool gave_up = *abort_flag;
  if (gave_up && lane == 0) pair::store_word(abort_flag, cluster_rank() ^ 1, 1);
  if (gave_up || warp == 0) pair::cluster_arrive_release();   // (warp 0 has stored no rows of out)
  else cluster_arrive_relaxed();
  cluster_wait();
  if (*abort_flag) {                                          // (in both CTAs alike)
    if (cluster_rank() == 0 && threadIdx.x == 0) {
      const int n0 = issued[0], n1 = issued[1], top = max(n0, n1);
#pragma unroll 1
      for (int i = max(0, top - C::NS); i < top; ++i) {
        const int s = i % C::NS;
        (void)tile.get(p, BN, i / p.kb);
        const uint32_t bytes = CUT && tile.half ? (128 + 64) * kMmBlock : C::STAGE;    // of one CTA
        if (i >= n0) tma::arrive_expect_tx(&full[s], bytes);
        else if (i >= n1) pair::complete_tx(&full[s], bytes);
        (void)umma::mbar_wait(&full[s], (i / C::NS) & 1, 100000000ull);
      }
    }
    __syncwarp();
    pair::cluster_arrive_release();
    cluster_wait();
  }
  umma::fence_after_sync();
  if (warp == 1) pair::tmem_dealloc(tmem, 512);
}

// --------------------------------------------------- at most sixteen rows of a --
// The weights are read once and nothing else takes as long, so no operand is staged:
// a warp takes 16 rows of b and every eighth block of K, and its lanes load their
// matrix fragments straight from memory (mma.sync, b's rows on the long side, a's
// as the eight columns; NT sets of those).  The order of a dot product's elements is
// free, so a lane takes 16 bytes that lie together, of b and of a alike.  The eight
// warps of a CTA join in shared memory in their order.  8 x 6144 x 4096 take 6.7 us (3.8
// TB/s): three CTAs an SM, two blocks of K in flight a warp; with four blocks and fewer
// CTAs, or CTAs of four warps, 7 to 8.4 us.
constexpr int kMwRows = 16, kMwWarps = 8;

__device__ __forceinline__ void mma16832_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 x;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}

template <int NT>
__global__ void __launch_bounds__(32 * kMwWarps, NT == 1 ? 3 : 2) block_matmul_warp(const MatmulArgs a, int kb) {
  constexpr int U = NT == 1 ? 2 : 1;                          // blocks of K loaded at once
  __shared__ float part[kMwWarps][8 * NT][kMwRows + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c4 = lane & 3;
  const int n0 = blockIdx.x * kMwRows;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint8_t* brow[2];
  const uint8_t* arow[NT];
  bool blive[2], alive[NT];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = n0 + g + 8 * i;
    blive[i] = n < a.N;
    brow[i] = a.b + (int64_t)(blive[i] ? n : 0) * a.K + 16 * c4;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = 8 * t + g;
    alive[t] = m < a.M;
    arow[t] = a.a + (int64_t)(alive[t] ? m : 0) * a.K + 16 * c4;
  }
  const float* sb = a.sb + (int64_t)(n0 / 128) * kb;
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
  for (int j0 = warp; j0 < kb; j0 += U * kMwWarps) {
    uint4 bx[U][2][2], ax[U][NT][2];                          // [block][row][64-byte half]
    float s[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kMwWarps;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = (int64_t)j * kMmBlock + 64 * h;
        const bool in = j < kb && k + 16 * c4 < a.K;          // (K is a multiple of 16)
#pragma unroll
        for (int i = 0; i < 2; ++i) bx[u][i][h] = in && blive[i] ? load_once(brow[i] + k) : zero;
#pragma unroll
        for (int t = 0; t < NT; ++t) ax[u][t][h] = in && alive[t] ? *reinterpret_cast<const uint4*>(arow[t] + k) : zero;
      }
      const float b = j < kb ? sb[j] : 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int m = 8 * t + 2 * c4 + i;
          s[u][t][i] = j < kb && m < a.M ? a.sa[(int64_t)m * kb + j] * b : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma16832_e4m3(d, bx[u][0][h].x, bx[u][1][h].x, bx[u][0][h].y, bx[u][1][h].y, ax[u][t][h].x, ax[u][t][h].y);
          mma16832_e4m3(d, bx[u][0][h].z, bx[u][1][h].z, bx[u][0][h].w, bx[u][1][h].w, ax[u][t][h].z, ax[u][t][h].w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(d[e], s[u][t][e & 1], acc[t][e]);
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][8 * t + 2 * c4 + (e & 1)][g + 8 * (e >> 1)] = acc[t][e];
  __syncthreads();
  if (tid < 8 * NT * kMwRows) {
    const int m = tid / kMwRows, n = n0 + tid % kMwRows;
    if (m >= a.M || n >= a.N) return;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kMwWarps; ++w) y += part[w][m][tid % kMwRows];
    if (a.bias != nullptr) y += a.bias[n];
    if (a.out_f32) reinterpret_cast<float*>(a.out)[(int64_t)m * a.N + n] = y;
    else reinterpret_cast<__nv_bfloat16*>(a.out)[(int64_t)m * a.N + n] = __float2bfloat16_rn(y);
  }
}

// ----------------------------------------------------------- few rows of a --
// The weights' bytes bound it, so they are spread over all SMs: a CTA takes 128
// rows of b (the tensor core's 128 lanes), up to MT rows of a (its columns), and a
// share of the blocks of K; the CTAs of a cluster hold the shares of one tile.  Each
// sums its blocks in registers, copies every column's sums to the CTA that owns the
// column (one bulk copy a CTA through distributed shared memory), and the owner adds
// the shares in rank order.  Of the 10.8 us of 64 x 6144 x 4096 about 2.5 pass until the
// first blocks land, 4.3 with them (25 MB at the measured copy rate: 3.9) and 3 with the
// join and the stores.  One CTA an SM with a deeper ring is slower (12.0 us), and so are
// eight shares (64 x 2560 x 2048: 8.1 us, 6.7 in four) and clusters of three (a cluster
// takes whole pairs of SMs: 26 us), and sums sent from registers 16 bytes at a time
// (st.async: 11.8 us).
template <int MT>
struct MfCfg {
  static constexpr int STAGE = (128 + MT) * kMmBlock;
  static constexpr int CTAS = 2;                              // of an SM
  static constexpr int NB = 256 / MT;                         // TMEM buffers
  static constexpr int NS = MT == 64 ? 3 : 4;
  static constexpr int SK = 16;                               // blocks whose scales are held
  static constexpr int SUMS = MT * 128 * 4;                   // a tile's sums, as they are sent
  static constexpr int BYTES = 1024 + NS * STAGE + SUMS + SK * MT * 4 + 512;
  static constexpr int TCOLS = NB * MT;
  static constexpr int THREADS = 192;
  static_assert(SUMS <= NS * STAGE, "sums to send take the ring's place");
  static_assert(CTAS * (BYTES + 1024) <= 228 * 1024, "shared memory of an SM");
};

template <int MT>
__global__ void __launch_bounds__(MfCfg<MT>::THREADS, MfCfg<MT>::CTAS) block_matmul_few(const __grid_constant__ MatmulParams p) {
  using C = MfCfg<MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sent = reinterpret_cast<float*>(smem);               // sums, [column][row of b], in the ring's place
  float* got = reinterpret_cast<float*>(smem + C::NS * C::STAGE);        // received, [rank][own column][row of b]
  float* scol = got + C::SUMS / 4;                            // [SK][MT] scales of the columns
  uint64_t* bars = reinterpret_cast<uint64_t*>(scol + C::SK * MT);
  uint64_t* full = bars;
  uint64_t* empty = full + C::NS;
  uint64_t* d_full = empty + C::NS;                           // [NB]
  uint64_t* d_free = d_full + C::NB;                          // [NB]
  uint64_t* drained = d_free + C::NB;                         // every product finished
  uint64_t* landed = drained + 1;                             // the other shares of this CTA's columns
  uint32_t* tslot = reinterpret_cast<uint32_t*>(landed + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int S;
  asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(S));
  const int rank = (int)cluster_rank(), per = MT / S;         // columns of a rank (S is 1, 2 or 4)
  const int n0 = blockIdx.x / S * 128, m0 = blockIdx.y * MT;
  const int j0 = (int)((int64_t)p.kb * rank / S), j1 = (int)((int64_t)p.kb * (rank + 1) / S);
  auto load = [&](int it) {                                   // block j0 + it
    const int s = it % C::NS;
    uint8_t* st = smem + s * C::STAGE;
    tma::arrive_expect_tx(&full[s], C::STAGE);
    tma::load_2d(st, &p.tb, (j0 + it) * kMmBlock, n0, &full[s]);
    tma::load_2d(st + 128 * kMmBlock, &p.ta, (j0 + it) * kMmBlock, m0, &full[s]);
  };
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) { umma::mbar_init(&full[i], 1); umma::mbar_init(&empty[i], 1); }
    for (int i = 0; i < C::NB; ++i) { umma::mbar_init(&d_full[i], 1); umma::mbar_init(&d_free[i], 4); }
    umma::mbar_init(drained, 1);
    umma::mbar_init(landed, 1);
    *abort_flag = 0;
    umma::mbar_fence_init();
    if (S > 1) tma::arrive_expect_tx(landed, (S - 1) * per * 512);
    for (int it = 0; it < C::NS && it < j1 - j0; ++it) load(it);         // the first copies do not wait for the rest
  }
  if (warp == 1) {
    umma::tmem_alloc(tslot, C::TCOLS);
    umma::tmem_relinquish();
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  cluster_arrive_relaxed();                                   // every CTA runs, its barriers ready, before sums are sent to it
  const uint32_t tmem = *tslot;
  float2 acc[MT / 2];
  bool ok = true;
  if (warp == 0) {
    if (elect_one()) {
      int it = min(C::NS, j1 - j0);
      for (; it < j1 - j0; ++it) {
        if (!wait_fast(&empty[it % C::NS], (it / C::NS - 1) & 1, abort_flag)) break;
        load(it);
      }
      // no copy is in flight when the ring is used for the sums (matters when a wait gave up)
      for (int i = max(0, it - C::NS); i < it; ++i) (void)umma::mbar_wait(&full[i % C::NS], (i / C::NS) & 1, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t ID = umma::idesc(umma::FMT_E4M3, umma::FMT_E4M3, umma::MAJOR_K, umma::MAJOR_K, 128, MT);
    if (elect_one()) {
      for (int it = 0; it < j1 - j0; ++it) {
        const int s = it % C::NS, d = it % C::NB;
        bool go = wait_fast(&full[s], (it / C::NS) & 1, abort_flag);
        if (it >= C::NB) go = go && wait_fast(&d_free[d], (it / C::NB - 1) & 1, abort_flag);
        if (!go) break;
        umma::fence_after_sync();
        const uint32_t wa = umma::smem_u32(smem + s * C::STAGE), xa = wa + 128 * kMmBlock;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma::mma_f8_ss(tmem + d * MT, umma::sdesc(wa + 32 * k, 16, 1024, umma::SWIZZLE_128B),
                          umma::sdesc(xa + 32 * k, 16, 1024, umma::SWIZZLE_128B), ID, k > 0);
        umma::mma_commit(&empty[s]);
        umma::mma_commit(&d_full[d]);
      }
    }
    __syncwarp();
    if (elect_one()) umma::mma_commit(drained);               // complete before TMEM and the ring are used otherwise
    (void)umma::mbar_wait(drained, 0, 100000000ull);
  } else {
    const int t = tid - 64;
    const uint32_t base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float* sb = p.a.sb + (int64_t)(n0 / 128) * p.kb;
#pragma unroll
    for (int c = 0; c < MT / 2; ++c) acc[c] = make_float2(0.f, 0.f);
    for (int j = j0; j < j1; ++j) {
      const int it = j - j0, d = it % C::NB;
      if (it % C::SK == 0) {                                  // scales of the next blocks: both factors multiplied once
        asm volatile("bar.sync 1, 128;\n" ::: "memory");      // (the others are done with the last ones)
        constexpr int EACH = C::SK * MT / 128;                // of a thread: loaded at once, one block of K
        const int i = t % C::SK;
        const float b = j + i < j1 ? sb[j + i] : 0.f;
        float x[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
          const int m = min(m0 + t / C::SK + e * (128 / C::SK), p.a.M - 1);
          x[e] = j + i < j1 ? p.a.sa[(int64_t)m * p.kb + j + i] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) scol[i * MT + t / C::SK + e * (128 / C::SK)] = x[e] * b;
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
      }
      ok = ok && wait_fast(&d_full[d], (it / C::NB) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;                                      // (the barriers' other warps go on as well)
      umma::fence_after_sync();
      const float4* sc = reinterpret_cast<const float4*>(scol + it % C::SK * MT);
#pragma unroll
      for (int c = 0; c < MT / 32; c += 2) {                  // two pieces of 32 columns in flight
        uint32_t r[2][32];
        tmem_ld32_nowait(base + d * MT + 32 * c, r[0]);
        if (c + 1 < MT / 32) tmem_ld32_nowait(base + d * MT + 32 * (c + 1), r[1]);
        tmem_wait_ld32(r[0]);
        if (c + 1 < MT / 32) tmem_wait_ld32(r[1]);
        if (c + 2 >= MT / 32) {
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) umma::mbar_arrive(&d_free[d]);
        }
#pragma unroll
        for (int k = 0; k < 2 && c + k < MT / 32; ++k)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float4 x = sc[8 * (c + k) + u];
            float2* y = acc + 16 * (c + k) + 2 * u;
            y[0] = __ffma2_rn(make_float2(__uint_as_float(r[k][4 * u]), __uint_as_float(r[k][4 * u + 1])), make_float2(x.x, x.y), y[0]);
            y[1] = __ffma2_rn(make_float2(__uint_as_float(r[k][4 * u + 2]), __uint_as_float(r[k][4 * u + 3])), make_float2(x.z, x.w), y[1]);
          }
      }
    }
  }
  // every product is complete and every copy has landed: the sums take the ring's place
  __syncthreads();
  if (warp >= 2) {
    const int row = 32 * (warp & 3) + lane;                   // of b, TMEM lane
    if (!ok && lane == 0) raise_error(p.a.err, FP8KV_DEVERR_TIMEOUT);
#pragma unroll
    for (int c = 0; c < MT; ++c) sent[c * 128 + row] = !ok ? NAN : c & 1 ? acc[c / 2].y : acc[c / 2].x;
    umma::fence_proxy_async_smem();
  }
  cluster_wait();
  __syncthreads();
  if (S > 1) {
    if (tid < S && tid != rank)
      asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                       mapa_u32(umma::smem_u32(got + rank * per * 128), tid)),
                   "r"(umma::smem_u32(sent + tid * per * 128)), "r"(per * 512), "r"(mapa_u32(umma::smem_u32(landed), tid))
                   : "memory");
    ok = wait_cluster(landed, 0, abort_flag);
    if (!ok) {                                                // (and nothing lands behind this CTA's end)
      raise_error(p.a.err, FP8KV_DEVERR_TIMEOUT);
      (void)umma::mbar_wait(landed, 0, kMmLastWait);
    }
  }
  // this rank's columns (rows of out), four neighbouring columns of out a thread; the
  // warps of sums have each four of them at once
  if (warp >= 2 && (S == 1 || ok)) {
    const int l = 4 * lane, n = n0 + l, c0 = warp - 2;        // columns c0, c0 + 4, ...
    for (int c = c0; c < per; c += 16) {
      float4 y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c + 4 * u >= per) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {                         // (four ranks at most)
          if (r >= S) continue;
          const float4 x = *reinterpret_cast<const float4*>((r == rank ? sent : got) + (r * per + c + 4 * u) * 128 + l);
          y[u].x += x.x; y[u].y += x.y; y[u].z += x.z; y[u].w += x.w;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int m = m0 + rank * per + c + 4 * u;
        if (c + 4 * u < per && m < p.a.M && n < p.a.N) store_row4(p.a, m, n, y[u]);
      }
    }
  }
  // the copies out of this CTA have arrived when their readers are here
  umma::fence_before_sync();
  if (S > 1) {
    __syncwarp();
    cluster_arrive_relaxed();                                 // (a release would wait for the stores of out)
    cluster_wait();
  } else {
    __syncthreads();
  }
  umma::fence_after_sync();
  if (warp == 1) umma::tmem_dealloc(tmem, C::TCOLS);
}

// Codes viewed as [rows][K], boxes of `box` rows x 128 bytes; what lies outside
// reads as zero codes.
static bool make_codes_map(CUtensorMap* m, const uint8_t* base, int rows, int K, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {kMmBlock, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// out viewed as [rows][N], boxes of 32 rows x 128 bytes.
static bool make_out_map(CUtensorMap* m, const MatmulArgs& a) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int size = a.out_f32 ? 4 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.M};
  const cuuint64_t strides[1] = {(cuuint64_t)a.N * size};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32}, estr[2] = {1, 1};
  return fn(m, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.out, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool CUT>
static cudaError_t launch_pair_one(const MatmulParams& p, unsigned pairs, cudaStream_t st) {
  using C = MmCfg<BN>;
  const cudaError_t e = ensure_smem_optin((const void*)block_matmul_pair<BN, CUT>, C::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::BYTES;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t r = cudaLaunchKernelEx(&cfg, block_matmul_pair<BN, CUT>, p);
  if (r != cudaSuccess) (void)cudaGetLastError();
  return r;
}

template <int BN>
static cudaError_t launch_pair(MatmulParams& p, cudaStream_t st) {
  p.tiles_m = (p.a.M + 255) / 256;
  p.tiles_n = (p.a.N + BN - 1) / BN;
  if (!make_codes_map(&p.ta, p.a.a, p.a.M, p.a.K, 128) || !make_codes_map(&p.tb, p.a.b, p.a.N, p.a.K, BN / 2)) return cudaErrorInvalidValue;
  p.bulk_out = p.a.N % (p.a.out_f32 ? 4 : 8) == 0;
  if (p.bulk_out && !make_out_map(&p.to, p.a)) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, pairs = sm_count() / 2, rest = tiles % pairs;
  p.whole = (int)tiles;
  if constexpr (BN == 256) {
    // Half tiles in the last wave: 1000 x 6144 x 4096 (96 tiles) 33.8 -> 30.1 us, 4000 x 2560 x
    // 2048 (160) 28.4 -> 26.5, 5000 x 6144 x 4096 (480) 109.5 -> 108; the form that can cut
    // takes 2.5 % more a tile, so from eight waves on nothing is won (768 tiles: 169 us both).
    if (tiles > pairs && tiles < 8 * pairs && rest > 0 && 2 * rest <= pairs) {
      p.whole = (int)(tiles - rest);
      if (!make_codes_map(&p.th, p.a.b, p.a.N, p.a.K, 64)) return cudaErrorInvalidValue;
      return launch_pair_one<256, true>(p, (unsigned)pairs, st);
    }
  }
  return launch_pair_one<BN, false>(p, (unsigned)(tiles < pairs ? tiles : pairs), st);
}

template <int MT>
static cudaError_t launch_few(MatmulParams& p, cudaStream_t st) {
  const cudaError_t e = ensure_smem_optin((const void*)block_matmul_few<MT>, MfCfg<MT>::BYTES);
  if (e != cudaSuccess) return e;
  p.tiles_m = (p.a.M + MT - 1) / MT;
  p.tiles_n = (p.a.N + 127) / 128;
  if (!make_codes_map(&p.ta, p.a.a, p.a.M, p.a.K, MT) || !make_codes_map(&p.tb, p.a.b, p.a.N, p.a.K, 128)) return cudaErrorInvalidValue;
  const int64_t units = (int64_t)p.tiles_m * p.tiles_n;
  int S = 1;                                                  // shares while every CTA runs at once
  while (S < 4 && 2 * S * units <= MfCfg<MT>::CTAS * sm_count() && 2 * S <= p.kb) S *= 2;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = S;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.tiles_n * S, p.tiles_m);
  cfg.blockDim = dim3(MfCfg<MT>::THREADS);
  cfg.dynamicSmemBytes = MfCfg<MT>::BYTES;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t r = cudaLaunchKernelEx(&cfg, block_matmul_few<MT>, p);
  if (r != cudaSuccess) (void)cudaGetLastError();
  return r;
}

// Which kernel, by the rows of a (times in us on one GB300, inputs from memory):
//   up to 8      fragments from memory (8 x 6144 x 4096: 6.7, in clusters 8.5; 8 x 1000 x
//                2048: 2.2 and 4.9; from 20,000 columns on clusters are 8 % faster)
//   up to 16     the same while the strips of 16 columns fill the SMs once (12 x 4608 x
//                3584: 6.4, in clusters 7.5), beyond it clusters (16 x 6144 x 4096: 8.9, 10.7)
//   up to 64     clusters (64 x 6144 x 4096: 10.8, on pairs 12.6)
//   up to 128    clusters while four shares of every tile run at once (100 x 4608 x 3584:
//                10.7, on pairs 11.7), else pairs (128 x 6144 x 4096: 12.9, 14.9)
//   more         pairs, 128 columns a tile while those fit the SMs at once (200 x 6144 x
//                4096: 12.4, 256 columns 20; 512 x 2560 x 2048: 8.1 and 12.3), else 256
//                (512 x 6144 x 4096: 19.4, 128 columns 26.7; 2000 x 2560 x 2048: 21.1, 21.7)
cudaError_t launch_block_matmul(const MatmulArgs& a, cudaStream_t st) {
  MatmulParams p;
  p.a = a;
  p.kb = (a.K + kMmBlock - 1) / kMmBlock;
  const int64_t strips = ((int64_t)a.N + kMwRows - 1) / kMwRows;
  if (a.M <= 8 || (a.M <= 16 && strips <= 2 * sm_count())) {
    if (a.M <= 8) block_matmul_warp<1><<<(unsigned)strips, 32 * kMwWarps, 0, st>>>(a, p.kb);
    else block_matmul_warp<2><<<(unsigned)strips, 32 * kMwWarps, 0, st>>>(a, p.kb);
    return cudaGetLastError();
  }
  if (a.M <= 32) return launch_few<32>(p, st);
  const int64_t units = 2 * (((int64_t)a.N + 127) / 128);
  if (a.M <= 64 || (a.M <= 128 && 4 * units <= 2 * sm_count())) return launch_few<64>(p, st);
  const int64_t wide = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
  return 2 * wide > sm_count() / 2 ? launch_pair<256>(p, st) : launch_pair<128>(p, st);
}

}  // namespace fp8kv
