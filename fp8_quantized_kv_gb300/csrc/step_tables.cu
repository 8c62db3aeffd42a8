// step_tables.cu -- what a serving step needs before its attention runs: the
// page tables and slot maps of a ragged batch, built on the GPU from the
// requests' lengths, and the rotary tables.
//
// Page tables and slot maps.  Sequence b holds c_b tokens and gets n_b more:
//   cu_b    = sum of n_b' over b' < b              first row of the sequence
//   first_b = ceil(c_b / P), last_b = ceil((c_b + n_b) / P)
//   base_b  = sum of (last_b' - first_b') over b' < b
//   page i of [first_b, last_b) = free_pages[head + base_b + i - first_b]
//   row cu_b + j: position t = c_b + j, slot = page(t / P) P + t mod P
// A row's page is either one that the sequence had before (read from the
// table, at an entry this call does not write) or a fresh one (read from the
// free list), so no thread reads what another writes and one launch does it
// all.  Every CTA scans the lengths itself: 8 bytes a sequence, against the
// second launch (about 2 us) that sharing one scan would take.  Latency bounds
// it: 3.6 us for 64 sequences of one token, 5.6 us for 300 sequences and 127,000
// rows (2 MB written), on the device.
#include "params.cuh"

namespace fp8kv {

constexpr int kTablesThreads = 256;

// Inclusive sums over the CTA of two values per thread.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long* wa, long long* wb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o);
    const long long y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) { a += x; b += y; }
  }
  if (lane == 31) { wa[warp] = a; wb[warp] = b; }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTablesThreads / 32; ++w)
    if (w < warp) { a += wa[w]; b += wb[w]; }
}

struct TablesParams {
  const int32_t *cached, *fresh, *free_pages, *free_head;
  int32_t* table;              // page table, written in place (null: contiguous cache)
  int32_t *cu, *seq_lens, *seq_idx, *pos, *head_out;
  int64_t* slots;
  unsigned int* err;
  int batch, num_free, rows, page_shift, num_pages, max_pages, max_tokens;
};

// Thread i places fresh page i (a fresh page holds at least one new row, so
// there are no more of them than rows) and writes row i's entries.
__global__ void __launch_bounds__(kTablesThreads) build_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t tsm[];
  int32_t* cu = tsm;                                   // [batch + 1] first row of each sequence
  int32_t* base = cu + p.batch + 1;                    // [batch + 1] first fresh page of each sequence
  int32_t* cached = base + p.batch + 1;                // [batch] tokens before the step, -1: not placed
  __shared__ long long wa[kTablesThreads / 32];
  __shared__ long long wb[kTablesThreads / 32];
  __shared__ long long tot_rows, tot_pages;
  const int tid = threadIdx.x;
  const bool paged = p.table != nullptr;
  const int P1 = (1 << p.page_shift) - 1;
  const long long cap = paged ? (long long)p.max_pages << p.page_shift : p.max_tokens;
  const int head = paged ? *p.free_head : 0;
  const int avail = paged ? (head < 0 || head > p.num_free ? 0 : p.num_free - head) : 0;
  const bool lead = blockIdx.x == 0;
  unsigned int bad = 0;
  if (tid == 0) { tot_rows = 0; tot_pages = 0; cu[0] = 0; base[0] = 0; }
  if (paged && (head < 0 || head > p.num_free)) bad |= FP8KV_DEVERR_NO_PAGES;
  __syncthreads();
  for (int b0 = 0; b0 < p.batch; b0 += kTablesThreads) {
    const int b = b0 + tid;
    int c = 0, n = 0, need = 0;
    bool fits = true;
    if (b < p.batch) {
      c = p.cached[b];
      n = p.fresh[b];
      // a length below 0 or past the cache's capacity: the sequence keeps its
      // rows (so that the others' rows stay where the caller has them) and
      // gets no page
      fits = c >= 0 && n >= 0 && (long long)c + n <= cap;
      if (!fits) bad |= FP8KV_DEVERR_SEQ_TOO_LONG;
      if (n < 0) n = 0;
      if (fits && paged) need = ((c + n + P1) >> p.page_shift) - ((c + P1) >> p.page_shift);
    }
    long long a = n, f = need;
    block_scan2(a, f, wa, wb);
    const long long rows_end = tot_rows + a, pages_end = tot_pages + f;
    if (b < p.batch) {
      if (fits && need > 0 && pages_end > avail) { fits = false; bad |= FP8KV_DEVERR_NO_PAGES; }
      cu[b + 1] = (int)min(rows_end, (long long)INT32_MAX);
      base[b + 1] = (int)min(pages_end, (long long)INT32_MAX);
      cached[b] = fits ? c : -1;
      if (lead) p.seq_lens[b] = fits ? c + n : max(c, 0);
      if (b == p.batch - 1 && rows_end > p.rows) bad |= FP8KV_DEVERR_SEQ_TOO_LONG;
    }
    __syncthreads();
    if (tid == kTablesThreads - 1) { tot_rows = rows_end; tot_pages = pages_end; }
    __syncthreads();
  }
  if (lead) {
    for (int b = tid; b <= p.batch; b += kTablesThreads) p.cu[b] = cu[b];
    if (tid == 0 && paged) {
      // pages placed: sequences take them in order, so those that got theirs
      // are the ones whose range ends within the list
      int lo = 0, hi = p.batch;                        // largest b with base[b] <= avail
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= avail) lo = mid; else hi = mid - 1;
      }
      *p.head_out = head + base[lo];
    }
  }
  const int i = blockIdx.x * kTablesThreads + tid;
  // fresh page f (placed sequences' pages end within the list)
  const int pages = min(base[p.batch], avail);
  for (long long f = i; paged && f < pages; f += (long long)gridDim.x * kTablesThreads) {
    int lo = 0, hi = p.batch - 1;                      // sequence with base[b] <= f < base[b + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (base[mid + 1] > f) hi = mid; else lo = mid + 1;
    }
    const int c = cached[lo];
    if (c >= 0) {
      int page = p.free_pages[head + f];
      if (page < 0 || page >= p.num_pages) { page = -1; bad |= FP8KV_DEVERR_BAD_PAGE; }
      p.table[(int64_t)lo * p.max_pages + ((c + P1) >> p.page_shift) + (f - base[lo])] = page;
    }
  }
  // row i
  if (i < p.rows) {
    int b = -1, t = -1;
    long long slot = -1;
    if (i < cu[p.batch]) {
      int lo = 0, hi = p.batch - 1;                    // sequence with cu[b] <= i < cu[b + 1]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > i) hi = mid; else lo = mid + 1;
      }
      b = lo;
      const int c = cached[lo];
      if (c >= 0) {
        t = c + (i - cu[lo]);
        if (!paged) {
          slot = (long long)lo * p.max_tokens + t;
        } else {
          const int pi = t >> p.page_shift, first = (c + P1) >> p.page_shift;
          const int page = pi < first ? p.table[(int64_t)lo * p.max_pages + pi]
                                      : p.free_pages[head + base[lo] + pi - first];
          if (page < 0 || page >= p.num_pages) bad |= FP8KV_DEVERR_BAD_PAGE;
          else slot = ((long long)page << p.page_shift) + (t & P1);
        }
      }
    }
    p.seq_idx[i] = b;
    p.pos[i] = t;
    p.slots[i] = slot;
  }
  if (bad) raise_error(p.err, bad);
}

cudaError_t launch_build_tables(const CacheView& c, const int32_t* cached, const int32_t* fresh,
                                const int32_t* free_pages, int num_free, const int32_t* free_head, int rows,
                                int32_t* cu, int32_t* seq_lens, int32_t* seq_idx, int32_t* pos, int64_t* slots,
                                int32_t* head_out, unsigned int* err, cudaStream_t s) {
  TablesParams p;
  p.cached = cached;
  p.fresh = fresh;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.table = const_cast<int32_t*>(c.page_table);
  p.cu = cu;
  p.seq_lens = seq_lens;
  p.seq_idx = seq_idx;
  p.pos = pos;
  p.slots = slots;
  p.head_out = head_out;
  p.err = err;
  p.batch = c.batch;
  p.num_free = num_free;
  p.rows = rows;
  p.page_shift = c.page_shift;
  p.num_pages = c.num_pages;
  p.max_pages = c.max_pages_per_seq;
  p.max_tokens = c.max_tokens;
  constexpr int most = (3 * kTablesMaxBatch + 2) * (int)sizeof(int32_t);
  const int bytes = (3 * c.batch + 2) * (int)sizeof(int32_t);
  if (bytes > 40 * 1024) {
    const cudaError_t e = ensure_smem_optin((const void*)build_tables_kernel, most);
    if (e != cudaSuccess) return e;
  }
  const int grid = rows > 0 ? (rows - 1) / kTablesThreads + 1 : 1;
  build_tables_kernel<<<grid, kTablesThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

// Rotary tables.  cos and sin of theta = t w_i for positions t and pairs i.
// With w_i in turns as a 64-bit binary fraction W_i (host, fp64), the phase
// t W_i mod 2^64 is exact integer arithmetic: far positions lose nothing but
// t times the rounding of W_i itself.  Its top two bits (after adding an eighth
// of a turn) pick the quadrant; the rest is an angle x in [-pi/4, pi/4], turned
// to fp32 in two 32-bit parts, so that a small angle keeps its leading digits (a
// small negative one loses 2^-56 of a turn to their sum).  There the Taylor polynomials through x^9 and x^10 are
// within 2^-28 and 2^-31 of sine and cosine, so rounding to fp32 is what is
// left.  A thread keeps VEC pairs and walks down the positions: the tables are
// written once, 16 bytes a thread, and nothing is read.  131,072 positions of 32
// pairs (34 MB) take 7.1 us on the device, 4.7 TB/s (69 % of the measured copy
// rate; 6.8 us with the upper 32 bits of the phase alone, which left a sine of a
// millionth with two digits; one pair a thread, a 64-bit division each and CUDA's sincosf: 35 us).
struct RopeTablesParams {
  unsigned long long w[kRopeMaxPairs];
  float *cos, *sin;
  float amplitude;
  int positions, pairs;
};

// (phase: a 64-bit binary fraction of a turn)
__device__ __forceinline__ void sincos_phase(unsigned long long phase, float amplitude, float& c, float& s) {
  const unsigned int top = (unsigned int)(phase >> 32), quad = (top + 0x20000000u) >> 30;
  const float x = fmaf((float)(unsigned int)phase, 3.4061215800865545e-19f,      // 2 pi / 2^64, 2 pi / 2^32
                       (float)(int)(top - (quad << 30)) * 1.4629180792671596e-09f);
  const float z = x * x;
  const float sn = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -1.6666667e-1f), x);
  const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f), 4.1666667e-2f), -0.5f), 1.f);
  const float a = quad & 1 ? sn : cs, b = quad & 1 ? cs : sn;
  c = (quad == 1 || quad == 2 ? -a : a) * amplitude;
  s = (quad & 2 ? -b : b) * amplitude;
}

template <int VEC>
__global__ void __launch_bounds__(256) rope_tables_kernel(const __grid_constant__ RopeTablesParams p) {
  const int cols = p.pairs / VEC;                  // threads along a position
  const int col = threadIdx.x % cols, rows = blockDim.x / cols;
  if (threadIdx.x >= cols * rows) return;
  unsigned long long w[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) w[k] = p.w[VEC * col + k];
  for (long long t = (long long)blockIdx.x * rows + threadIdx.x / cols; t < p.positions; t += (long long)gridDim.x * rows) {
    float c[VEC], s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) sincos_phase((unsigned long long)t * w[k], p.amplitude, c[k], s[k]);
    const long long at = t * p.pairs + VEC * col;
    if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(p.cos + at) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(p.sin + at) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      p.cos[at] = c[0];
      p.sin[at] = s[0];
    }
  }
}

cudaError_t launch_rope_tables(int positions, int pairs, const unsigned long long* w, float amplitude, float* cos,
                               float* sin, cudaStream_t s) {
  if (positions == 0) return cudaSuccess;
  RopeTablesParams p;
  for (int i = 0; i < kRopeMaxPairs; ++i) p.w[i] = i < pairs ? w[i] : 0;
  p.cos = cos;
  p.sin = sin;
  p.amplitude = amplitude;
  p.positions = positions;
  p.pairs = pairs;
  // 16-byte stores where every row of the tables starts on one
  const bool vec = pairs % 4 == 0 && (((uintptr_t)cos | (uintptr_t)sin) & 15) == 0;
  const int rows = 256 / (vec ? pairs / 4 : pairs);
  const long long blocks = ((long long)positions + rows - 1) / rows, most = 8LL * sm_count();
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  if (vec) rope_tables_kernel<4><<<grid, 256, 0, s>>>(p);
  else rope_tables_kernel<1><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8kv
