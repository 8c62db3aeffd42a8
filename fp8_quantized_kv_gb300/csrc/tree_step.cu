// tree_step.cu -- what surrounds the attention of a step that verifies trees of
// drafted tokens: each node's ancestors and position from the parents, and, once
// the model has chosen a token at every node, the walk along the accepted nodes
// with the move of their cache rows.
#include "params.cuh"

namespace fp8kv {

// Masks and positions.  Row i of sequence b: bits of node i and of its ancestors (under
// a window W those less than W positions above it or among the first `sinks` tokens),
// and ctx + depth.  A thread walks up from its node in shared memory (parents come
// before their children, so the walk ends) and writes its words from the highest
// down: ancestors only get lower.  Latency bounds it: offsets, parents, then the
// steps of the walk, which read four ancestors at once (300 trees of up to 256 nodes
// on 40 levels: 5.8 us, one at a time 6.6; 64 trees of 24-64 nodes: 2.5 and 2.3).
constexpr int kTreeThreads = 256;

template <bool WINDOW>
__global__ void __launch_bounds__(kTreeThreads) tree_tables_kernel(const TreeTablesParams p) {
  __shared__ int16_t up[kTreeMaxNodes];
  __shared__ short2 two[kTreeMaxNodes];            // parent and its parent, -1: none
  __shared__ short4 four[kTreeMaxNodes];
  const int tid = threadIdx.x;
  if (blockIdx.x >= p.batch) {                     // rows that belong to no sequence
    const int first = min(max(p.cu[0], 0), p.rows), end = min(max(p.cu[p.batch], first), p.rows);
    for (int64_t i = (int64_t)(blockIdx.x - p.batch) * kTreeThreads + tid; i < (int64_t)first + p.rows - end;
         i += (int64_t)(gridDim.x - p.batch) * kTreeThreads) {
      const int64_t r = i < first ? i : end + (i - first);
      p.pos[r] = -1;
      for (int w = 0; w < p.words; ++w) p.masks[r * p.words + w] = 0;
    }
    return;
  }
  const int b = blockIdx.x, q0 = p.cu[b], q1 = p.cu[b + 1], len = p.seq_lens[b];
  if (q0 < 0 || q1 < q0 || q1 > p.rows) {
    if (tid == 0) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
    return;
  }
  const int n = q1 - q0;
  const bool fits = n <= 32 * p.words && len >= n;
  if (!fits) {
    if (tid == 0) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
    for (int i = tid; i < n; i += kTreeThreads) p.pos[q0 + i] = -1;
    for (int64_t i = tid; i < (int64_t)n * p.words; i += kTreeThreads) p.masks[(int64_t)q0 * p.words + i] = 0;
    return;
  }
  bool bad = false;
  for (int i = tid; i < n; i += kTreeThreads) {
    int u = p.parents[q0 + i];
    if (u < -1 || u >= i) { bad = true; u = -1; }
    up[i] = (int16_t)u;
  }
  if (bad) raise_error(p.err, FP8KV_DEVERR_BAD_TREE);
  __syncthreads();
  for (int i = tid; i < n; i += kTreeThreads) {
    const int16_t a = up[i];
    two[i] = make_short2(a, a >= 0 ? up[a] : -1);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kTreeThreads) {
    const short2 a = two[i], b = a.y >= 0 ? two[a.y] : make_short2(-1, -1);
    four[i] = make_short4(a.x, a.y, b.x, b.y);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kTreeThreads) {
    uint32_t* row = p.masks + (int64_t)(q0 + i) * p.words;
    int w = p.words - 1, depth = -1;
    uint32_t bits = 0;
    auto climb = [&](auto&& sees) {                // (-1: no more)
      sees(i);
      for (short4 a = four[i]; sees(a.x) && sees(a.y) && sees(a.z) && sees(a.w); a = four[a.w]) {}
    };
    // under a window: ancestors at depths from `reach` on, or below `early`, are seen
    int reach = 0, early = 0;
    if constexpr (WINDOW) {                        // (the node's own depth first)
      climb([&](int a) { depth += a >= 0; return a >= 0; });
      reach = depth - p.window + 1;
      early = p.sinks - (len - n);
    }
    [[maybe_unused]] const int own = depth;
    depth = -1;
    climb([&](int a) {
      if (a < 0) return false;
      ++depth;                                     // steps above the node
      if (WINDOW && own - depth < reach && own - depth >= early) return true;
      for (; w > a >> 5; --w) { row[w] = bits; bits = 0; }
      bits |= 1u << (a & 31);
      return true;
    });
    for (; w >= 0; --w) { row[w] = bits; bits = 0; }
    p.pos[q0 + i] = len - n + depth;
  }
}

cudaError_t launch_tree_tables(const TreeTablesParams& p, cudaStream_t st) {
  const int pad = p.rows / 1024 < 8 ? p.rows / 1024 + 1 : 8;
  (p.window > 0 ? tree_tables_kernel<true> : tree_tables_kernel<false>)<<<p.batch + pad, kTreeThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// Acceptance.  Node i continues node u = parents[i] if its drafted token is the
// choice at u; best[u] is the lowest such child, so the walk from node 0 takes one
// shared-memory read a step.  A CTA owns a sequence in one layer (each repeats the
// walk: two dependent loads, against a second launch).
//
// The move: accepted node path[k] of depth k goes from key ctx + path[k] to key
// ctx + k.  The path rises, so path[k] >= k, and a row that is written has been
// read if rows are taken in order, kTreeMove at a time: those of one group are all
// loaded before any is stored, and later groups read keys behind the stored ones.
constexpr int kTreeMove = 8;
constexpr int kAcceptThreads = 256;

__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const __grid_constant__ TreeAcceptParams p) {
  __shared__ int best[kTreeMaxNodes];
  __shared__ int16_t path[kTreeMaxNodes];
  __shared__ int64_t from[kTreeMaxNodes], to[kTreeMaxNodes];    // rows of KV head 0, -1: stays
  __shared__ int taken_sh;
  const int tid = threadIdx.x, b = blockIdx.x;
  const bool lead = blockIdx.y == 0 && p.first;
  const int q0 = p.cu[b], q1 = p.cu[b + 1], len = p.seq_lens[b];
  const bool offsets = q0 >= 0 && q1 >= q0 && q1 <= p.rows;
  const int n = offsets ? q1 - q0 : 0;
  const bool fits = offsets && n <= kTreeMaxNodes && len >= n;
  if (!fits && lead && tid == 0) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
  const int nodes = fits ? n : 0, ctx = fits ? len - n : 0;
  for (int i = tid; i < nodes; i += kAcceptThreads) best[i] = INT32_MAX;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < nodes; i += kAcceptThreads) {
    const int u = p.parents[q0 + i];
    if (u < -1 || u >= i) bad = true;
    else if (u >= 0 && p.tokens[q0 + i] == p.choices[q0 + u]) atomicMin(&best[u], i);
  }
  if (bad && lead) raise_error(p.err, FP8KV_DEVERR_BAD_TREE);
  __syncthreads();
  if (tid == 0) {
    int k = 0;
    if (nodes > 0) {
      const int most = min(p.max_path, nodes);
      for (int at = 0; at < nodes && k < most; at = best[at]) path[k++] = (int16_t)at;
    }
    taken_sh = k;
  }
  __syncthreads();
  const int taken = taken_sh;
  if (lead) {
    for (int k = tid; k < p.max_path; k += kAcceptThreads) p.path[(int64_t)b * p.max_path + k] = k < taken ? path[k] : -1;
    if (tid == 0) {
      p.accepted[b] = taken;
      p.new_lens[b] = fits ? ctx + taken : len;
      p.next[b] = taken > 0 ? p.choices[q0 + path[taken - 1]] : -1;
    }
  }
  if (blockIdx.y >= p.layers || taken <= 1) return;
  const TreeLayer& c = p.layer[blockIdx.y];
  const int P1 = (1 << p.page_shift) - 1;
  const int64_t cap = p.paged ? (int64_t)c.max_pages << p.page_shift : c.max_tokens;
  if (len > cap) {
    if (tid == 0) raise_error(p.err, FP8KV_DEVERR_SEQ_TOO_LONG);
    return;
  }
  auto row_of = [&](int key) -> int64_t {
    if (!p.paged) return (int64_t)b * p.kv_heads * c.max_tokens + key;
    const int page = c.page_table[(int64_t)b * c.max_pages + (key >> p.page_shift)];
    if (page < 0 || page >= c.num_pages) {
      raise_error(p.err, FP8KV_DEVERR_BAD_PAGE);
      return -1;
    }
    return ((int64_t)page * p.kv_heads << p.page_shift) + (key & P1);
  };
  for (int k = tid; k < taken; k += kAcceptThreads) {
    int64_t f = -1, t = -1;
    if (path[k] != k) {
      f = row_of(ctx + path[k]);
      t = row_of(ctx + k);
    }
    from[k] = t < 0 ? -1 : f;
    to[k] = t;
  }
  __syncthreads();
  // items of a row: 16-byte pieces of its K and V, then its two scale slots
  const int kc = p.k_bytes / 16, vc = p.v_bytes / 16, per = kc + vc + 2;
  const int64_t head_rows = p.paged ? (int64_t)1 << p.page_shift : c.max_tokens;
  for (int k0 = 0; k0 < taken; k0 += kTreeMove) {
    const int m = min(kTreeMove, taken - k0);
    for (int e0 = 0; e0 < p.kv_heads * per; e0 += kAcceptThreads) {
      const int e = e0 + tid, h = e / per, x = e - h * per;
      const bool live = e < p.kv_heads * per;
      uint8_t* base = nullptr;                       // of this item in row 0, and its distance from row to row
      int64_t stride = 0;
      bool word = false;
      if (live) {
        if (x < kc) { base = c.k + 16 * x; stride = p.k_bytes; }
        else if (x < kc + vc) { base = c.v + 16 * (x - kc); stride = p.v_bytes; }
        else { base = reinterpret_cast<uint8_t*>(x == kc + vc ? c.k_scale : c.v_scale); stride = 4; word = true; }
      }
      uint4 r[kTreeMove];
      const int64_t hr = h * head_rows;
#pragma unroll
      for (int i = 0; i < kTreeMove; ++i) {
        r[i] = make_uint4(0, 0, 0, 0);
        if (base == nullptr || i >= m || from[k0 + i] < 0) continue;
        const uint8_t* src = base + (from[k0 + i] + hr) * stride;
        if (word) r[i].x = *reinterpret_cast<const uint32_t*>(src);
        else r[i] = *reinterpret_cast<const uint4*>(src);
      }
      // (an item is one thread's, in all rows: no other thread reads what this one stores)
#pragma unroll
      for (int i = 0; i < kTreeMove; ++i) {
        if (base == nullptr || i >= m || from[k0 + i] < 0) continue;
        uint8_t* dst = base + (to[k0 + i] + hr) * stride;
        if (word) *reinterpret_cast<uint32_t*>(dst) = r[i].x;
        else *reinterpret_cast<uint4*>(dst) = r[i];
      }
    }
  }
}

cudaError_t launch_tree_accept(const TreeAcceptParams& p, cudaStream_t st) {
  tree_accept_kernel<<<dim3(p.batch, p.layers > 0 ? p.layers : 1), kAcceptThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8kv
