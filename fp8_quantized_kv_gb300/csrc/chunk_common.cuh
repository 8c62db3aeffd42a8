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
#pragma once

#include "params.cuh"

namespace fp8kv {

constexpr int kChunkKeys = 64;     // keys per KV tile

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
};

// The first key of KV tile j of the tile's list.
__device__ __forceinline__ int chunk_key0(const ChunkTile& t, int j) {
  return (j < t.n_sink ? j : t.first + j - t.n_sink) * kChunkKeys;
}

// Tiles are numbered so that a CTA finds its own without a scan over the
// batch: sequence b owns the numbers from start(b) = cu_q[b] / T + b on,
// because it has at most (cu_q[b+1] / T - cu_q[b] / T) + 1 tiles of T tokens.
// The last sequence with start(b) <= x is found by a 32-way search of the
// warp.  Returns false for a number that no tile has.  `lead`: raise errors.
__device__ __forceinline__ bool chunk_tile(const ChunkParams& p, int x, bool lead, ChunkTile& t) {
  const int T = p.tile_tokens, lane = threadIdx.x & 31;
  int b = x, q0 = x, q1 = x + 1, i0 = 0;           // one query per sequence
  if (p.cu_q == nullptr && x >= p.c.batch) return false;
  if (p.cu_q != nullptr) {
    int lo = 0, n = p.c.batch;
    while (n > 1) {
      const int step = (n + 31) >> 5, at = lane * step;
      const bool le = at < n && (at == 0 || (long long)p.cu_q[lo + at] / T + lo + at <= x);
      // le is monotone for offsets that do not decrease; for others the
      // count still lands on a sequence of the batch
      const int k = max(__popc(__ballot_sync(0xffffffffu, le)), 1) - 1;
      lo += k * step;
      n = min(step, n - k * step);
    }
    b = lo;
    q0 = p.cu_q[b];
    q1 = p.cu_q[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.total_q) {
      if (lead) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
      return false;
    }
    const long long i = ((long long)x - ((long long)q0 / T + b)) * T;
    if (i < 0 || i >= q1 - q0) return false;
    i0 = (int)i;
  }
  int len = p.seq_lens[b];
  if (len < 0 || len > cache_capacity(p.c)) {      // reported; the sequence's queries see nothing
    if (lead) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
    len = 0;
  }
  t.b = b;
  t.row0 = q0 + i0;
  t.ntok = min(T, q1 - q0 - i0);
  t.pos0 = len - (q1 - q0) + i0;
  t.kv_end = max(0, t.pos0 + t.ntok);
  t.lo = 0;
  t.n_sink = 0;
  if (p.window > 0) {
    const long long lo = (long long)t.pos0 - p.window + 1;
    t.lo = lo > 0 ? (int)lo : 0;
    t.n_sink = min((min(p.sinks, t.kv_end) + kChunkKeys - 1) / kChunkKeys, t.lo / kChunkKeys);
  }
  t.first = t.lo / kChunkKeys;
  t.n = t.n_sink + max(0, (t.kv_end + kChunkKeys - 1) / kChunkKeys - t.first);
  return true;
}

// Whether every query of the tile sees all keys of the KV tile from key0 on.
__device__ __forceinline__ bool chunk_all_seen(const ChunkParams& p, const ChunkTile& t, int key0) {
  const int last = key0 + kChunkKeys - 1;
  return last <= t.pos0 && (p.window <= 0 || key0 > t.pos0 + t.ntok - 1 - p.window || last < p.sinks);
}
__device__ __forceinline__ bool chunk_sees(const ChunkParams& p, int pos, int key) {
  return key <= pos && (p.window <= 0 || key > pos - p.window || key < p.sinks);
}

// Cache row of a key of the tile's sequence, or -1: a key that no query of
// the tile can see (its row is never read: it may hold anything) or a bad
// page (reported).
__device__ __forceinline__ int chunk_row(const ChunkParams& p, const ChunkTile& t, int hk, int key) {
  if (key >= t.kv_end || (key < t.lo && key >= p.sinks)) return -1;
  return (int)cache_row(p.c, t.b, hk, key, p.err);
}

// Weight of a split's (m, l): zero for a split that saw nothing, NaN for one
// whose scores were all NaN.
__device__ __forceinline__ float chunk_weight(float m, float l, float M) {
  if (m == -INFINITY) return l == l ? 0.f : l;
  return exp2f(m - M);
}

}  // namespace fp8kv
