// chunk_common.cuh -- what the kernels of ragged chunk attention share: the
// tile of queries a CTA takes, the cache tokens that tile can see, and how
// partial results of several splits are laid out.
//
// Queries are ragged: rows cu_q[b] .. cu_q[b+1] - 1 belong to sequence b, the
// last one at position seq_lens[b] - 1.  A tile is `tile_tokens` consecutive
// queries of one sequence times the `group` query heads of one KV head, so
// that the heads of a group share the K and V tiles they read.  Query
// position p sees key j if j <= p and, under a window W, j > p - W or
// j < sinks.
//
// Trees (the kernels' TREE forms): the new tokens of a sequence are the nodes of a
// tree, in the cache behind its ctx = seq_lens[b] - nodes cached tokens, node i
// as key ctx + i.  Node i sees the cached tokens (under a window those with
// j > pos - W or j < sinks, pos its position in the text, ctx + its depth), the
// nodes of its row of bits, and itself.  So every KV tile that holds a node, or
// whose first keys some node's window misses, is seen in part, and the bits are
// looked up there alone: the context's tiles run as in the causal form.
#pragma once

#include "params.cuh"
#include "tc_common.cuh"

namespace fp8kv {

constexpr int kChunkKeys = 64;     // keys per KV tile
constexpr int kChunkThreads = 128; // of the kernels on warp-level matrix instructions

struct ChunkTile {
  int b;           // sequence
  int row0;        // first query row of the tile
  int ntok;        // queries (tokens) in the tile
  int pos0;        // position of the first query (negative: it sees nothing)
  int kv_end;      // keys 0 .. kv_end - 1 can be visible to the tile
  int lo;          // first key of the first query's window
  int n_sink;      // KV tiles that hold first tokens, before the window's
  int first;       // first KV tile of the window
  int n;           // KV tiles in all
  int ctx;         // trees: tokens before the first node (negative: not all nodes are in the cache)
};

// KV tiles that `keys` keys (>= 0, up to 2^31 - 16) take.
__device__ __forceinline__ int chunk_tiles(int keys) { return (int)(((unsigned)keys + kChunkKeys - 1) / kChunkKeys); }

// Whether KV tiles j0 .. j1 - 1 of the tile's list hold the key at position `pos`.
__device__ __forceinline__ bool chunk_own(const ChunkTile& t, int pos, int j0, int j1) {
  const int j = pos / kChunkKeys - t.first + t.n_sink;
  return pos >= 0 && j >= j0 && j < j1;
}

// The first key of KV tile j of the tile's list.
__device__ __forceinline__ int chunk_key0(const ChunkTile& t, int j) {
  return (j < t.n_sink ? j : t.first + j - t.n_sink) * kChunkKeys;
}

// Tiles are numbered so that a CTA finds its own without a scan over the
// batch: sequence b owns the numbers from start(b) = cu_q[b] / T + b on,
// because it has at most (cu_q[b+1] / T - cu_q[b] / T) + 1 tiles of T tokens.
//
// The last sequence b with start(b) <= x, found by a 32-way search of the warp;
// its offsets and its length.  Offsets that decrease give some sequence of the
// batch (the right one, up to 32 sequences, before the first that decreases: the
// lanes in front count, not all).
__device__ __forceinline__ int chunk_search(const ChunkParams& p, int x, int& q0, int& q1, int& len) {
  const int lane = threadIdx.x & 31;
  auto last_of = [](unsigned m) { return max(__clz(__brev(~m)), 1) - 1; };     // last lane of those in front
  auto before = [&](int b, int first) { return (long long)first / p.tile_tokens + b <= x; };
  int lo = 0, n = p.c.batch;
  while (n > 32) {
    const int step = (n + 31) >> 5, at = lane * step;
    const bool le = at < n && (at == 0 || before(lo + at, p.cu_q[lo + at]));
    const int k = last_of(__ballot_sync(0xffffffffu, le));
    lo += k * step;
    n = min(step, n - k * step);
  }
  // the last step's lanes hold all there is to know of their sequence
  const int at = min(lane, n - 1) + lo;
  const int c0 = p.cu_q[at], c1 = p.cu_q[at + 1], ln = p.seq_lens[at];
  const bool le = lane < n && (lane == 0 || before(at, c0));
  const int k = last_of(__ballot_sync(0xffffffffu, le));
  q0 = __shfl_sync(0xffffffffu, c0, k);
  q1 = __shfl_sync(0xffffffffu, c1, k);
  len = __shfl_sync(0xffffffffu, ln, k);
  return lo + k;
}
__device__ __forceinline__ bool chunk_offsets_ok(const ChunkParams& p, int q0, int q1) {
  return q0 >= 0 && q1 >= q0 && q1 <= p.total_q;
}

// Splits: rows of a sequence with bad offsets have no shares.  The whole CTA that
// looks at them (pair x) marks those rows for the joining kernel, in the sum of
// their first share, which is never below zero otherwise.  Where the pair
// decreases, any row from the largest offset so far on may be without shares, and
// in a batch past one step of the search any row at all: all of these are marked,
// and a tile that holds some writes its sum over the mark, or has it marked.
constexpr float kChunkNoRow = -1.f;
static __device__ __noinline__ void chunk_mark_rows(const int32_t* cu_q, float* part_l, int batch, int total_q, int q_heads,
                                                    int num_splits, int x, int a0, int a1) {
  int first = max(a0, 0);
  if (a0 < 0 || a1 < a0) {
    first = 0;
    if (batch <= 32)
      for (int i = 0; i <= x; ++i) first = max(first, cu_q[i]);
  }
  const int64_t rows = (int64_t)total_q * q_heads;
  for (int64_t r = (int64_t)first * q_heads + threadIdx.x; r < rows; r += blockDim.x) part_l[r * num_splits] = kChunkNoRow;
}

// What a CTA works at: tile number, KV head, share.  The last tiles of a sequence see
// the most keys (trees: all see as many): they start first, or, for trees, with
// `longest_first`, those of long sequences in all their heads and shares.
struct ChunkPlace {
  int x, hk, split;
  int b, q0, q1, len, i0;      // the sequence, where it is known already (else b is -1), and the tile's first query
};

// Trees: the tile that comes `at`-th when those of long sequences go first.  Up to 32
// sequences: in the order of their lengths, a lane each (16 sequences of 2K-8K tokens x
// 33-64 nodes on tcgen05: 121 us, in four classes by length 124.5, as they come 150).
// More: in four classes; each lane counts the tiles of batch / 32 sequences (eight at
// most) in 16 bits a class (the host sees to it that they fit).  Returns false where no
// tile has the number; bad offsets: as the search finds them.
__device__ __forceinline__ bool tree_order(const ChunkParams& p, int at, ChunkPlace& a) {
  const int lane = threadIdx.x & 31, B = p.c.batch, T = p.tile_tokens, each = (B + 31) / 32, b0 = lane * each;
  int cu[9], len[8], longest = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= each) break;
    cu[k] = p.cu_q[min(b0 + k, B)];
    len[k] = b0 + k < B ? p.seq_lens[b0 + k] : 0;
    cu[k + 1] = p.cu_q[min(b0 + k + 1, B)];
  }
  bool ok = true;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= each) break;
    ok = ok && chunk_offsets_ok(p, cu[k], cu[k + 1]);
    longest = max(longest, len[k]);
  }
  if (!__all_sync(0xffffffffu, ok)) {
    a.x = at;
    return true;
  }
  if (each == 1) {                                     // up to 32 sequences: in their order
    const bool in = b0 < B;
    const int start = cu[0] / T + b0, n = in ? cu[1] / T + b0 + 1 - start : 0, mylen = in ? len[0] : -1;
    int pos = 0;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const int lj = __shfl_sync(0xffffffffu, mylen, j), nj = __shfl_sync(0xffffffffu, n, j);
      if (lj > mylen || (lj == mylen && j < lane)) pos += nj;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at >= pos && at < pos + n);
    if (hit == 0) return false;
    const int from = __ffs(hit) - 1;
    a.b = __shfl_sync(0xffffffffu, b0, from);
    a.q0 = __shfl_sync(0xffffffffu, cu[0], from);
    a.q1 = __shfl_sync(0xffffffffu, cu[1], from);
    a.len = __shfl_sync(0xffffffffu, len[0], from);
    a.i0 = __shfl_sync(0xffffffffu, at - pos, from) * T;
    return a.i0 < a.q1 - a.q0;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  const int l1 = longest >> 2, l2 = longest >> 1, l3 = l1 + l2;
  auto shift = [&](int k) { return len[k] > l3 ? 0 : len[k] > l2 ? 16 : len[k] > l1 ? 32 : 48; };
  unsigned long long own = 0;
  int first = cu[0] / T + b0;
  auto tiles = [&](int k, int& start) {                // of sequence b0 + k, whose first number is `start`
    const int end = cu[k + 1] / T + b0 + k + 1, n = b0 + k < B ? end - start : 0;
    start = end;
    return n;
  };
  int start = first;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= each) break;
    own += (unsigned long long)(unsigned)tiles(k, start) << shift(k);
  }
  unsigned long long upto = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += x;
  }
  const unsigned long long all = __shfl_sync(0xffffffffu, upto, 31);
  int y = at, sh = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int n = (int)(all >> sh & 0xFFFF);
    if (sh == 16 * k && y >= n) { y -= n; sh += 16; }
  }
  if (y >= (int)(all >> sh & 0xFFFF)) return false;    // numbers in front of the first sequence, and behind the last
  int e = (int)((upto - own) >> sh & 0xFFFF), mine = -1, i = 0;
  start = first;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= each) break;
    const int n = tiles(k, start);
    if (shift(k) == sh) {
      if (y >= e && y < e + n) { mine = k; i = y - e; a.q0 = cu[k]; a.q1 = cu[k + 1]; a.len = len[k]; }
      e += n;
    }
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, mine >= 0)) - 1;
  a.b = __shfl_sync(0xffffffffu, b0 + mine, from);
  a.q0 = __shfl_sync(0xffffffffu, a.q0, from);
  a.q1 = __shfl_sync(0xffffffffu, a.q1, from);
  a.len = __shfl_sync(0xffffffffu, a.len, from);
  a.i0 = __shfl_sync(0xffffffffu, i, from) * T;
  return a.i0 < a.q1 - a.q0;
}

// The CTA's place and tile.  Returns false for a number that no tile has.  The same
// CTA of a tile reports errors (KV head 0, share 0).
template <bool TREE>
__device__ __forceinline__ bool chunk_tile(const ChunkParams& p, ChunkPlace& a, ChunkTile& t) {
  const int T = p.tile_tokens;
  a = {(int)(gridDim.x - 1 - blockIdx.x), (int)blockIdx.y, (int)blockIdx.z, -1, 0, 0, 0, 0};
  if (TREE && p.longest_first) {
    const unsigned i = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z), each = gridDim.y * gridDim.z, r = i % each;
    a.hk = (int)(r % gridDim.y);
    a.split = (int)(r / gridDim.y);
    if (!tree_order(p, (int)(i / each), a)) return false;
  }
  const bool lead = a.hk == 0 && a.split == 0;
  const int x = a.x;
  int b = x, q0 = x, q1 = x + 1, i0 = 0;           // one query per sequence
  if (p.cu_q == nullptr && x >= p.c.batch) return false;
  int len = 0;
  if (TREE && a.b >= 0) {
    b = a.b;
    q0 = a.q0;
    q1 = a.q1;
    len = a.len;
    i0 = a.i0;
  } else if (p.cu_q != nullptr) {
    // there are as many tile numbers as sequences, or more: each looks at one pair of
    // offsets, so that every bad one is reported, found by the search or not
    int a0 = 0, a1 = 0;
    if (lead && x < p.c.batch) { a0 = p.cu_q[x]; a1 = p.cu_q[x + 1]; }
    b = chunk_search(p, x, q0, q1, len);
    if (!chunk_offsets_ok(p, a0, a1)) {
      if (threadIdx.x == 0) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
      if (p.num_splits > 1) chunk_mark_rows(p.cu_q, p.part_l, p.c.batch, p.total_q, p.q_heads, p.num_splits, x, a0, a1);
    }
    if (!chunk_offsets_ok(p, q0, q1)) return false;
    const long long i = ((long long)x - ((long long)q0 / T + b)) * T;
    if (i < 0 || i >= q1 - q0) return false;
    i0 = (int)i;
  } else {
    len = p.seq_lens[b];
  }
  // reported; the sequence's queries see nothing
  if (len < 0 || len > cache_capacity(p.c) || (TREE && q1 - q0 > 32 * p.mask_words)) {
    if (lead && threadIdx.x == 0) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
    len = 0;
  }
  t.b = b;
  t.row0 = q0 + i0;
  t.ntok = min(T, q1 - q0 - i0);
  t.pos0 = len - (q1 - q0) + i0;
  t.kv_end = max(0, t.pos0 + t.ntok);
  t.ctx = 0;
  int first_pos = t.pos0;                          // no query's window starts before this position's
  if constexpr (TREE) {
    t.ctx = first_pos = len - (q1 - q0);
    if (t.kv_end > 0) t.kv_end = len;              // bits may name any node
  }
  t.lo = 0;
  t.n_sink = 0;
  if (p.window > 0) {
    const long long lo = (long long)first_pos - p.window + 1;
    t.lo = lo > 0 ? (int)lo : 0;
    t.n_sink = min(chunk_tiles(min(p.sinks, t.kv_end)), t.lo / kChunkKeys);
  }
  t.first = t.lo / kChunkKeys;
  t.n = t.n_sink + max(0, chunk_tiles(t.kv_end) - t.first);
  return true;
}

// Whether every query of the tile sees all keys of the KV tile from key0 on.
// (Trees: a node's position is below the end of its sequence.)
template <bool TREE = false, int KEYS = kChunkKeys>
__device__ __forceinline__ bool chunk_all_seen(const ChunkParams& p, const ChunkTile& t, int key0) {
  const int last = key0 + KEYS - 1;
  if constexpr (TREE)
    return last < t.ctx && (p.window <= 0 || key0 > t.kv_end - 1 - p.window || last < p.sinks);
  return last <= t.pos0 && (p.window <= 0 || key0 > t.pos0 + t.ntok - 1 - p.window || last < p.sinks);
}
__device__ __forceinline__ bool chunk_sees(const ChunkParams& p, int pos, int key) {
  return key <= pos && (p.window <= 0 || key > pos - p.window || key < p.sinks);
}

// The 64 keys from key0 on that a query sees, as bits.
__device__ __forceinline__ unsigned long long chunk_seen_mask(const ChunkParams& p, int pos, int key0) {
  const int hi = min(pos - key0, 63);              // last key in reach
  if (hi < 0) return 0;
  const unsigned long long upto = ~0ull >> (63 - hi);
  if (p.window <= 0) return upto;
  const int lo = pos - p.window + 1 - key0, first = p.sinks - key0;
  unsigned long long out = lo > 63 ? 0ull : ~0ull << max(lo, 0);
  if (first > 0) out |= ~0ull >> (64 - min(first, 64));
  return out & upto;
}

// Trees: the 64 keys from key0 on that the node at cache position `own` (-1: no
// query) sees, as bits.  Its position in the text is taken within its sequence.
__device__ __forceinline__ unsigned long long tree_seen_mask(const ChunkParams& p, const ChunkTile& t, int own, int key0) {
  const int live = min(t.kv_end - key0, 64);       // keys in the cache
  if (own < 0 || live <= 0) return 0;
  const int64_t row = t.row0 + (own - t.pos0);
  const int cached = t.ctx - key0;                 // keys before the first node
  unsigned long long out = 0;
  if (cached > 0) {
    out = ~0ull >> (64 - min(cached, 64));
    if (p.window > 0) {
      const int pos = max(t.ctx, min(p.tree_pos[row], t.kv_end - 1));
      const int lo = pos - p.window + 1 - key0, first = p.sinks - key0;
      unsigned long long in = lo > 63 ? 0ull : ~0ull << max(lo, 0);
      if (first > 0) in |= ~0ull >> (64 - min(first, 64));
      out &= in;
    }
  }
  if (cached < 64) {                               // bits -cached .. -cached + 63 of the node's row
    const uint32_t* bits = p.masks + row * p.mask_words;
    unsigned long long nodes;
    if (cached > 0) {
      nodes = bits[0];
      if (p.mask_words > 1) nodes |= (unsigned long long)bits[1] << 32;
      nodes <<= cached;
    } else {
      const int w = -cached >> 5, sh = -cached & 31;
      auto word = [&](int i) { return i < p.mask_words ? bits[i] : 0u; };
      const uint32_t a = word(w), b = word(w + 1), c = word(w + 2);
      nodes = __funnelshift_r(a, b, sh) | (unsigned long long)__funnelshift_r(b, c, sh) << 32;
    }
    const int self = own - key0;
    if (self >= 0 && self < 64) nodes |= 1ull << self;
    out |= nodes & (~0ull >> (64 - live));
  }
  return out;
}

// Cache row of a key of the tile's sequence, or -1: a key that no query of
// the tile can see (its row is never read: it may hold anything) or a bad
// page (reported).  In two steps, so that the page id's latency can be spent
// on other work: chunk_page fetches it, chunk_row makes the row of it.
__device__ __forceinline__ bool chunk_wanted(const ChunkParams& p, const ChunkTile& t, int key) {
  return key < t.kv_end && (key >= t.lo || key < p.sinks);
}
__device__ __forceinline__ int chunk_page(const ChunkParams& p, const ChunkTile& t, int key) {
  if (!p.c.paged || !chunk_wanted(p, t, key)) return 0;
  return p.c.page_table[(int64_t)t.b * p.c.max_pages_per_seq + (key >> p.c.page_shift)];
}
__device__ __forceinline__ int chunk_row(const ChunkParams& p, const ChunkTile& t, int hk, int key, int page) {
  if (!chunk_wanted(p, t, key)) return -1;
  const CacheView& c = p.c;
  if (!c.paged) return (t.b * c.kv_heads + hk) * c.max_tokens + key;      // (rows of a cache fit 31 bits)
  if (page < 0 || page >= c.num_pages) {
    raise_error(p.err, FP8KV_DEVERR_BAD_PAGE);
    return -1;
  }
  return (page * c.kv_heads + hk) * c.page_size + (key & (c.page_size - 1));
}

// Weight of a split's (m, l): zero for a split that saw nothing, NaN for one
// whose scores were all NaN.
__device__ __forceinline__ float chunk_weight(float m, float l, float M) {
  if (m == -INFINITY) return l == l ? 0.f : l;
  return exp2f(m - M);
}

// ------------------------------------- warp-level matrix instructions --
// 16-byte chunk of a K row in shared memory.  A lane reads 16 (MX: 8) bytes of
// row lane / 4, four lanes side by side: neighbouring rows swap their 64-byte
// (MX: 32-byte) parts so that a quarter warp (half warp) meets every bank once.
template <int KE, int KB>
__device__ __forceinline__ int k_chunk(int ch, int row) {
  if constexpr (KE == ELEM_MX) return ch ^ ((row & 3) << 1);
  return KB >= 128 ? ch ^ ((row & 1) << 2) : ch;
}
// 16-byte chunk of a V row: eight rows' chunks of the same column lie in
// different banks (ldmatrix).
template <int VB>
__device__ __forceinline__ int v_chunk(int ch, int row) {
  return VB >= 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3);
}

__device__ __forceinline__ void cp_async16_z(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_z(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Non-finite 16-bit values of a B fragment register: `clean` has zeros in
// their place, the others 1.0 at each NaN, +inf or -inf.
template <bool BF16>
struct SetAside {
  uint32_t clean, nan, pinf, ninf;
  __device__ __forceinline__ explicit SetAside(uint32_t w) : clean(w), nan(0), pinf(0), ninf(0) {
    constexpr uint32_t INF = BF16 ? 0x7F80u : 0x7C00u, ONE = BF16 ? 0x3F80u : 0x3C00u;
#pragma unroll
    for (int sh = 0; sh < 32; sh += 16) {
      const uint32_t h = (w >> sh) & 0xFFFFu, m = h & 0x7FFFu;
      if (m < INF) continue;
      clean &= ~(0xFFFFu << sh);
      if (m > INF) nan |= ONE << sh;
      else if (h & 0x8000u) ninf |= ONE << sh;
      else pinf |= ONE << sh;
    }
  }
};


// A row that sees no key is zero.  One whose seen keys all score -inf (an infinite
// query or key) has a sum of zero too, but the softmax of such scores is NaN.  The
// two are told apart by the row's own key, the one at its position, which it sees
// whatever the window: a share that holds that key (`own`) and has a sum of zero
// keeps it as -0.  (Once a finite score has been seen the sum is at least 1.)
//
// Factor from a whole row's unnormalised O to out, from its sum.
__device__ __forceinline__ float chunk_inverse(float l, bool own) {
  return l > 0.f ? 1.f / l : l == 0.f && !own ? 0.f : NAN;
}
__device__ __forceinline__ float chunk_share_sum(float l, bool own) { return l == 0.f && own ? -0.f : l; }

// Elements d .. d + 3 of an unnormalised row of out with its maximum and sum:
// normalised into out, or kept as this split's share.
__device__ __forceinline__ void chunk_store(const ChunkParams& p, int64_t row, int split, int D, int d, const float (&x)[4],
                                            float m, float l, bool own) {
  if (p.num_splits > 1) {
    const int64_t at = row * p.num_splits + split;
    *reinterpret_cast<float4*>(p.part_o + at * D + d) = make_float4(x[0], x[1], x[2], x[3]);
    if (d == 0) { p.part_m[at] = m; p.part_l[at] = chunk_share_sum(l, own); }
    return;
  }
  const float inv = chunk_inverse(l, own);
  if (p.out_f32)
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + row * D + d) =
        make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  else
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + row * D + d) =
        make_uint2(pack16<true>(x[0] * inv, x[1] * inv), pack16<true>(x[2] * inv, x[3] * inv));
}

}  // namespace fp8kv
