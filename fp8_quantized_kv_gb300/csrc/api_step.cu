// api_step.cu -- the extern "C" boundary of the serving-step calls: argument
// checks, launch plans, status codes.  As in api.cu, every entry validates on
// the host, launches on the caller's stream and allocates nothing.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "params.cuh"

using namespace fp8kv;

namespace {

// Positions are 32-bit: a page table row may not hold more tokens.
bool capacity_fits(const fp8kv_cache* c) {
  return c->layout != FP8KV_LAYOUT_PAGED || (int64_t)c->max_pages_per_seq * c->page_size <= INT32_MAX;
}

// The rows and scales of a cache, up to four ranges; returns how many.
int cache_rows_of(const fp8kv_cache* c, Range* out) {
  const size_t per = c->layout == FP8KV_LAYOUT_PAGED ? (size_t)c->num_pages * c->page_size : (size_t)c->batch * c->max_tokens;
  const size_t rows = c->kv_heads * per;
  int n = 0;
  out[n++] = {c->k, rows * c->head_dim * (c->k_scale ? 1 : 2)};
  out[n++] = {c->v, rows * c->head_dim * (c->v_scale ? 1 : 2)};
  if (c->k_scale) out[n++] = {c->k_scale, 4 * rows};
  if (c->v_scale) out[n++] = {c->v_scale, 4 * rows};
  return n;
}
Range cache_table_of(const fp8kv_cache* c) {
  if (c->layout != FP8KV_LAYOUT_PAGED) return {nullptr, 0};
  return {c->page_table, 4 * (size_t)c->batch * (size_t)c->max_pages_per_seq};
}

struct ChunkPlan { int kernel, tile_rows, tile_tokens, tiles, splits; };

// How a chunk call runs, from its sizes (lengths are on the device).
// Kernel, by the average number of query rows (queries x heads of a group) a
// sequence has: up to 16 rows the few-row kernel, in tiles of 8 or 16 (one token
// of 64 sequences under a 1,024-token window: 30 us, against 81 us on tcgen05; two
// tokens x 8 heads of 64 sequences of 2K-4K tokens: 56 us, against 101 us);
// above, tcgen05 where it is built, which far above is ahead (256 x 4 over 16,000: 107
// against 323).  Between 17 and 32 rows the few-row kernel is, beside e4m3 values (8
// tokens x 4 heads over 8,000 tokens, 4 sequences: 33 us against 39 us at the best
// split counts; 2-4 x 8 over 4K-8K, 16 sequences: 45 against 61; trees of 3-4 x 8 over
// 100-2,000, 300 sequences: 179 against 227; but 50 against 46 under a window of 1,024
// of 64), beside bf16 ones either (188 against 180, 127 against 159): trees take it
// there, chunk calls stay with tcgen05 and its roundings.  The average counts idle sequences
// and rows of padding, and one kernel runs the whole call: batches of unlike
// sequences (a prompt in many idle slots, or beside many single tokens) get the
// form that suits only some of them.  Lengths of queries are on the device, so the
// host knows no better.  Block-scaled keys stay on the few-row kernel (2-4 x 8 over
// 4K-8K, 16 sequences: 49 us, 88 us on the form that the warp-level kernel had for
// them; 256-512 x 8, 4 sequences: 0.71 ms against 1.33), head dim 64 does up to 32
// rows (2-4 x 8 of 64 sequences of 2K-4K, bf16: 56 us against 71 on 64-row tiles at
// the best split count), with more it runs on the warp-level kernel (256-512 x 8 over
// 4K-8K, 4 sequences: 0.39 ms; before both were made faster 0.56 against 0.70, and around
// 64 rows either could be ahead).
//
// Splits of the few-row kernel: an SM holds four of its CTAs (three of 16 rows,
// or of 32 KiB stages), and a call takes as many waves of them as they need,
// each as long as one share and the 8 tiles' time that a CTA spends on its
// start and end.  So the counts that fill one, two or three waves are compared:
// 256 units of 32-64 tiles (16 rows) take 72 us whole, 62 us in 2 shares (1.1
// waves), 56 us in 3 (1.7), 60 us in 4.  Shares are 192 keys or longer (one token of
// 32 / 8 heads over 6,200: 9.4 us in 32 shares, 9.7 in 24 and in 64).
// Without a window lengths can differ widely: shares of about 4,096 keys at most
// then even them out (64 sequences of 1K-16K tokens, 32 / 8 heads: 200 us in 4
// shares, 246 us whole; sequences of 700 tokens in the same cache pay 34 us instead of 19), as
// long as that makes no more than 16 CTAs an SM.
//
// Splits of the others: tiles are few -> one wave.  tcgen05: two CTAs an SM,
// shares of 512 keys or longer.  Warp-level kernel: three an SM (by their
// registers) and 128 keys (32-64 x 8 of 2 sequences of 2K-4K tokens, when it was slower:
// 36 us in 4 shares, 31 us in 6, 37 us in 9, past one wave).
// Trees on tcgen05: tiles see whole contexts, and two CTAs of an SM slow each other
// down, so one CTA an SM with shares of 256 keys or longer, or two with 1,024 or
// longer, whichever is more shares (5-31 nodes x 8 heads, 2 KV heads, 16 sequences,
// window 1,024: 32 us whole, 26 in 2 shares, 29 in 4; of 4 sequences 32, 25 and 20;
// 64 x 4, 8 KV heads, 4 sequences of 8,000 tokens: 138 whole, 80 in 2, 71 in 4, 91 in
// 5, past one wave).  Without a window lengths can differ, and shares even them out: two
// where whole tiles fit one wave (12-24 x 4, 8 KV heads, 32 sequences of 1K-8K: 156 us
// whole, 132 in 2; past one wave, 33-64 x 7 of 32 sequences of 2K-8K, 197 and 221), three
// from 2.5 CTAs a tile on (33-64 x 8, 8 sequences of 1K-16K: 177 in 2, 138 in 3; with 1.5
// CTAs a tile, 33-64 x 7 of 16 sequences of 2K-8K, 168 whole, 120 in 2, 126 in 3).  Shares
// of 1,024 to 3,000 keys or more, so that only long sequences have several, were no better.
// Trees on the warp-level kernel, no window: up to four shares while that makes no more
// than eight CTAs an SM, for the same reason (33-64 x 8, 4 KV heads, 2K-8K: 16 sequences
// 200 us whole, 169 in 2; 8 sequences 93 in 2, 82 in 4).
fp8kv_status plan_chunk(const fp8kv_cache* c, int64_t total_q, int q_heads, int window, int sinks, int num_splits,
                        int kernel, bool tree, ChunkPlan* plan) {
  if (total_q < 0 || q_heads <= 0 || q_heads % c->kv_heads != 0 || window < 0 || sinks < 0 || num_splits < 0)
    return FP8KV_ERR_INVALID_ARG;
  if (kernel != FP8KV_KERNEL_AUTO && kernel != FP8KV_KERNEL_WARP_MMA && kernel != FP8KV_KERNEL_TENSOR_CORES)
    return FP8KV_ERR_INVALID_ARG;
  const int G = q_heads / c->kv_heads;
  if (!capacity_fits(c) || G > 16 || c->rope_cos != nullptr || c->kv_heads > 65535 || num_splits > 4096) return FP8KV_ERR_UNSUPPORTED;
  if (total_q > INT32_MAX || (double)total_q * q_heads > 8.0 * INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
  const int64_t B = c->batch > 0 ? c->batch : 1;
  // (an idle step, total_q 0, plans like one of single tokens: a tile holds one at least)
  const int64_t rows = total_q > 0 ? (total_q + B - 1) / B * G : G;
  const bool tc_built = c->head_dim == 128 && c->dtype != FP8KV_MXK8V8;
  if (kernel == FP8KV_KERNEL_TENSOR_CORES && !tc_built) return FP8KV_ERR_UNSUPPORTED;
  const int cap = capacity_of(c);
  // (a cache without room has no tensor map; its calls only write zero rows)
  const int few = tree && (c->dtype == FP8KV_K8V8 || c->dtype == FP8KV_K16V8) ? 32 : 16;
  const bool tc = cap > 0 && (kernel == FP8KV_KERNEL_TENSOR_CORES || (kernel == FP8KV_KERNEL_AUTO && tc_built && rows > few));
  plan->kernel = tc ? FP8KV_KERNEL_TENSOR_CORES : FP8KV_KERNEL_WARP_MMA;
  plan->tile_rows = tc ? 128 : rows <= 8 ? 8 : c->head_dim == 128 || rows <= 32 ? 16 : 64;
  plan->tile_tokens = plan->tile_rows / G;
  const int64_t tiles = total_q / plan->tile_tokens + c->batch;      // at most (chunk_common.cuh)
  if (tiles > INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
  plan->tiles = (int)tiles;
  // KV tiles that a tile of queries sees: under a window those of its queries, or of all
  // nodes of its tree, whatever part of them the tile holds (on average; a call's largest
  // tree can have all rows)
  auto seen_by = [&](int64_t queries) {
    const int64_t seen = window > 0 && window < cap ? (int64_t)window + queries + (sinks < cap ? sinks : cap) : cap;
    return seen < cap ? seen : cap;
  };
  const int64_t seen = seen_by(tree ? (total_q + B - 1) / B : plan->tile_tokens);
  const int64_t kv_tiles = (seen + 63) / 64 + 1;
  const int64_t most_tiles = tree ? (seen_by(total_q < kTreeMaxNodes ? total_q : kTreeMaxNodes) + 63) / 64 + 1 : kv_tiles;
  int64_t want = num_splits;
  if (want == 0) {
    // tiles if every sequence had the average number of queries, or, if that is
    // not a whole number, as many more or fewer of them as it says
    // (trees are rarely of one size: half a tile more each, and a little over, since a
    // wave that is just missed costs as much as a whole one)
    const int64_t T = plan->tile_tokens, even_q = (total_q / B + T - 1) / T * B;
    const int64_t some_q = tree ? (total_q / T + B / 2) * 21 / 20 : (total_q + T - 1) / T;
    const int64_t units = (total_q % B == 0 ? even_q : some_q > B ? some_q : B) * c->kv_heads;
    const int64_t sms = sm_count();
    if (plan->tile_rows > 16) {
      auto shares = [&](int64_t held, int64_t tiles) {        // fill `held` CTAs with shares of `tiles` KV tiles or more
        const int64_t s = units > 0 ? held / units : 1;
        return s < kv_tiles / tiles ? s : kv_tiles / tiles;
      };
      if (tc && tree) {
        want = shares(sms, 4);
        if (shares(2 * sms, 16) > want) want = shares(2 * sms, 16);
        if (window == 0 && want <= 1 && kv_tiles >= 32 && units <= 2 * sms) want = 2;
        if (window == 0 && want == 2 && kv_tiles >= 48 && 5 * units <= 2 * 2 * sms) want = 3;
      } else {
        want = tc ? shares(2 * sms, 8) : shares(3 * sms, 2);
        if (tree && window == 0 && kv_tiles >= 32) {
          const int64_t more = shares(8 * sms, 2) < 4 ? shares(8 * sms, 2) : 4;
          if (more > want) want = more;
        }
      }
    } else if (units > 0) {
      const bool wide = c->head_dim == 128 && c->dtype == FP8KV_K16V16;
      const int64_t held = (plan->tile_rows == 8 && !wide ? 4 : 3) * sms, most = kv_tiles / 3;
      int64_t even = seen == cap ? (kv_tiles + 63) / 64 : 1;
      if (even > 16 * sms / units) even = 16 * sms / units;
      if (even < 1) even = 1;
      want = even;
      auto cost = [&](int64_t s) { return (double)((units * s + held - 1) / held) * ((double)kv_tiles / s + 8); };
      for (int64_t waves = 1; waves <= 3; ++waves) {
        int64_t s = waves * held / units;
        if (s > most) s = most;
        if (s > want && cost(s) < cost(want)) want = s;
      }
    }
  }
  if (want > (num_splits > 0 ? most_tiles : kv_tiles)) want = num_splits > 0 ? most_tiles : kv_tiles;
  if (want > 4096) want = 4096;
  plan->splits = want < 1 ? 1 : (int)want;
  return FP8KV_OK;
}

// The fp32 partials (O, m, l) of every (row, split); nothing without splits.
size_t share_bytes(const fp8kv_cache* c, int64_t total_q, int q_heads, int splits) {
  return splits <= 1 ? 0 : (size_t)total_q * q_heads * splits * ((size_t)c->head_dim + 2) * sizeof(float);
}

// The chunk and the tree call: causal without masks (null), else over trees.
struct TreeArgs { const uint32_t* masks; const int32_t* pos; int32_t words; };

fp8kv_status run_chunk(const void* q, const fp8kv_cache* cache, const int32_t* cu_q, const int32_t* seq_lens,
                       const TreeArgs* tree, int64_t total_q, int32_t q_heads, float sm_scale, int32_t window,
                       int32_t sinks, int32_t num_splits, int32_t kernel, void* workspace, size_t workspace_bytes,
                       void* out, int32_t out_dtype, fp8kv_stream_t stream) {
  ChunkParams p;
  fp8kv_status st = check_cache(cache, &p.c);
  if (st != FP8KV_OK) return st;
  ChunkPlan plan;
  st = plan_chunk(cache, total_q, q_heads, window, sinks, num_splits, kernel, tree != nullptr, &plan);
  if (st != FP8KV_OK) return st;
  if (out_dtype != FP8KV_OUT_BF16 && out_dtype != FP8KV_OUT_F32) return FP8KV_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale)) return FP8KV_ERR_INVALID_ARG;
  if (cu_q == nullptr && (tree != nullptr || total_q != cache->batch)) return FP8KV_ERR_INVALID_ARG;
  if (tree != nullptr) {
    if (tree->words < 1) return FP8KV_ERR_INVALID_ARG;
    if (tree->words > kTreeMaxNodes / 32) return FP8KV_ERR_UNSUPPORTED;
  }
  if (cache->batch == 0 || total_q == 0) return FP8KV_OK;
  if (!q || !seq_lens || !out || misaligned(q, 16) || misaligned(out, 16)) return FP8KV_ERR_INVALID_ARG;
  if (misaligned(cu_q, 4) || misaligned(seq_lens, 4)) return FP8KV_ERR_INVALID_ARG;
  const int64_t rows = total_q * q_heads;
  const size_t values = (size_t)rows * cache->head_dim;
  if (overlap({q, 2 * values}, {out, (out_dtype == FP8KV_OUT_F32 ? 4 : 2) * values})) return FP8KV_ERR_INVALID_ARG;
  const size_t need = share_bytes(cache, total_q, q_heads, plan.splits);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FP8KV_ERR_WORKSPACE;
  if (need > 0 && misaligned(workspace, 16)) return FP8KV_ERR_INVALID_ARG;
  const Range result = {out, (out_dtype == FP8KV_OUT_F32 ? 4 : 2) * values};
  const Range shares = {workspace, need};
  if (overlap(result, shares) || overlap({q, 2 * values}, shares)) return FP8KV_ERR_INVALID_ARG;
  // (the joining kernel reads the offsets again, behind the first rows of out)
  Range read[7];
  int reads = cache_rows_of(cache, read);
  read[reads++] = cache_table_of(cache);
  read[reads++] = {seq_lens, 4 * (size_t)cache->batch};
  read[reads++] = {cu_q, cu_q ? 4 * ((size_t)cache->batch + 1) : 0};
  for (int i = 0; i < reads; ++i)
    if (overlap(read[i], result) || overlap(read[i], shares)) return FP8KV_ERR_INVALID_ARG;
  p.window = window < capacity_of(cache) ? window : 0;
  p.masks = nullptr;
  p.tree_pos = nullptr;
  p.mask_words = 0;
  if (tree != nullptr) {
    if (!tree->masks || misaligned(tree->masks, 4) || misaligned(tree->pos, 4)) return FP8KV_ERR_INVALID_ARG;
    if (p.window > 0 && !tree->pos) return FP8KV_ERR_INVALID_ARG;
    for (const Range& r : {Range{tree->masks, 4 * (size_t)total_q * tree->words}, Range{tree->pos, 4 * (size_t)total_q}})
      if (overlap(r, result) || overlap(r, shares)) return FP8KV_ERR_INVALID_ARG;
    p.masks = tree->masks;
    p.tree_pos = tree->pos;
    p.mask_words = tree->words;
  }
  p.err = device_error_ptr();
  if (!p.err) return FP8KV_ERR_CUDA;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cu_q = cu_q;
  p.seq_lens = seq_lens;
  p.out = out;
  p.part_o = plan.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  p.part_m = plan.splits > 1 ? p.part_o + rows * plan.splits * cache->head_dim : nullptr;
  p.part_l = plan.splits > 1 ? p.part_m + rows * plan.splits : nullptr;
  p.total_q = (int)total_q;
  p.q_heads = q_heads;
  p.group = q_heads / cache->kv_heads;
  p.out_f32 = out_dtype == FP8KV_OUT_F32;
  p.sinks = sinks;
  p.num_splits = plan.splits;
  p.tile_tokens = plan.tile_tokens;
  p.scale_log2 = sm_scale * kLog2e;
  cudaStream_t s = (cudaStream_t)stream;
  const int tiles = cu_q ? plan.tiles : cache->batch;
  // (one wave starts at once anyway; under a window sequences are alike)
  const int64_t ctas = (int64_t)tiles * cache->kv_heads * plan.splits;
  p.longest_first = tree && p.window == 0 && cache->batch > 1 && cache->batch <= 256 && tiles <= 65535 && ctas <= INT32_MAX &&
                    ctas > 2 * sm_count();
  auto* launch = plan.kernel == FP8KV_KERNEL_TENSOR_CORES ? (tree ? launch_tree_tc : launch_chunk_tc)
                 : plan.tile_rows <= 16 ? (tree ? launch_tree_rows : launch_chunk_rows)
                                        : (tree ? launch_tree_mma : launch_chunk_mma);
  cudaError_t e = launch(p, cache->dtype, tiles, s);
  if (e == cudaSuccess && plan.splits > 1) e = launch_chunk_merge(p, s);
  return cuda_status(e);
}

}  // namespace

extern "C" {

fp8kv_status fp8kv_build_tables(const fp8kv_cache* cache, const int32_t* cached_lens, const int32_t* new_lens,
                                const int32_t* free_pages, int32_t num_free, const int32_t* free_head,
                                int64_t n_rows, int32_t* cu_new, int32_t* seq_lens, int32_t* seq_idx, int32_t* pos,
                                int64_t* slots, int32_t* free_head_out, fp8kv_stream_t stream) {
  CacheView view;
  const fp8kv_status st = check_cache(cache, &view);
  if (st != FP8KV_OK) return st;
  if (n_rows < 0 || num_free < 0 || cu_new == nullptr) return FP8KV_ERR_INVALID_ARG;
  if (!capacity_fits(cache) || cache->batch > kTablesMaxBatch || n_rows > INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
  if (cache->batch > 0 && (!cached_lens || !new_lens || !seq_lens)) return FP8KV_ERR_INVALID_ARG;
  if (n_rows > 0 && (!seq_idx || !pos || !slots)) return FP8KV_ERR_INVALID_ARG;
  if (view.paged) {
    if (!free_head || !free_head_out || (num_free > 0 && !free_pages)) return FP8KV_ERR_INVALID_ARG;
  } else if (free_pages || num_free || free_head || free_head_out) {
    return FP8KV_ERR_INVALID_ARG;
  }
  for (const void* a : {(const void*)cached_lens, (const void*)new_lens, (const void*)free_pages, (const void*)free_head,
                        (const void*)cu_new, (const void*)seq_lens, (const void*)seq_idx, (const void*)pos,
                        (const void*)free_head_out})
    if (misaligned(a, 4)) return FP8KV_ERR_INVALID_ARG;
  if (misaligned(slots, 8)) return FP8KV_ERR_INVALID_ARG;
  const size_t B = (size_t)cache->batch, N = (size_t)n_rows;
  const Range in[] = {{cached_lens, 4 * B}, {new_lens, 4 * B}, {free_pages, 4 * (size_t)num_free}, {free_head, 4},
                      {view.page_table, 4 * B * (size_t)view.max_pages_per_seq}};
  const Range out[] = {{cu_new, 4 * (B + 1)}, {seq_lens, 4 * B}, {seq_idx, 4 * N},
                       {pos, 4 * N}, {slots, 8 * N}, {free_head_out, 4}};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : in)
      if (overlap(r, out[i])) return FP8KV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[j], out[i])) return FP8KV_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 4; ++i)
    if (overlap(in[i], in[4])) return FP8KV_ERR_INVALID_ARG;      // the page table is written in place
  unsigned int* err = device_error_ptr();
  if (!err) return FP8KV_ERR_CUDA;
  return cuda_status(launch_build_tables(view, cached_lens, new_lens, free_pages, num_free, free_head, (int)n_rows,
                                         cu_new, seq_lens, seq_idx, pos, slots, free_head_out, err,
                                         (cudaStream_t)stream));
}

fp8kv_status fp8kv_rope_tables(int64_t positions, int32_t rot_dim, double base, double factor,
                               int32_t original_positions, double ramp_low, double ramp_high, double amplitude,
                               float* cos, float* sin, fp8kv_stream_t stream) {
  if (positions < 0 || rot_dim <= 0 || original_positions < 0) return FP8KV_ERR_INVALID_ARG;
  if (!(base > 0) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor) || !(std::fabs(amplitude) <= FLT_MAX))
    return FP8KV_ERR_INVALID_ARG;
  if (original_positions > 0 && !(std::isfinite(ramp_low) && std::isfinite(ramp_high) && ramp_low < ramp_high))
    return FP8KV_ERR_INVALID_ARG;
  if (rot_dim % 2 != 0 || rot_dim > 2 * kRopeMaxPairs || positions > INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
  constexpr double kTwoPi = 6.283185307179586476925, kMostRadians = 1048576.0;
  unsigned long long w[kRopeMaxPairs];
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (original_positions > 0) {
      double g = (original_positions * f / kTwoPi - ramp_low) / (ramp_high - ramp_low);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f *= g + (1 - g) / factor;
    } else {
      f /= factor;
    }
    // (a 64-bit float has no fraction of a turn left where the turns are many)
    if (!(f <= kMostRadians)) return FP8KV_ERR_INVALID_ARG;
    // the frequency in turns per position, modulo one turn (positions are
    // whole numbers), as a 64-bit binary fraction
    double turns = f / kTwoPi;
    turns -= std::floor(turns);
    const double scaled = std::ldexp(turns, 64);
    w[i] = scaled >= 18446744073709551616.0 ? 0 : (unsigned long long)scaled;
  }
  if (positions == 0) return FP8KV_OK;
  if (!cos || !sin || misaligned(cos, 4) || misaligned(sin, 4)) return FP8KV_ERR_INVALID_ARG;
  const size_t bytes = (size_t)positions * (rot_dim / 2) * sizeof(float);
  if (overlap({cos, bytes}, {sin, bytes})) return FP8KV_ERR_INVALID_ARG;
  return cuda_status(launch_rope_tables((int)positions, rot_dim / 2, w, (float)amplitude, cos, sin,
                                        (cudaStream_t)stream));
}

fp8kv_status fp8kv_rope_append(const fp8kv_cache* cache, const void* q, int64_t q_stride, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, int32_t q_heads,
                               const int32_t* pos, const int64_t* slots, int64_t n_tokens, const float* cos,
                               const float* sin, int32_t positions, int32_t rot_dim, int32_t layout, void* q_out,
                               fp8kv_stream_t stream) {
  RopeAppendParams p;
  const fp8kv_status st = check_cache(cache, &p.c);
  if (st != FP8KV_OK) return st;
  if (n_tokens < 0 || q_heads <= 0 || positions < 0 || rot_dim <= 0) return FP8KV_ERR_INVALID_ARG;
  if (layout != FP8KV_ROPE_HALF && layout != FP8KV_ROPE_INTERLEAVED) return FP8KV_ERR_INVALID_ARG;
  if (rot_dim > cache->head_dim) return FP8KV_ERR_INVALID_ARG;
  if (rot_dim % 8 != 0 || n_tokens > INT32_MAX || q_heads > 65535) return FP8KV_ERR_UNSUPPORTED;
  if (n_tokens == 0) return FP8KV_OK;
  if (!q || !k || !v || !pos || !slots || !cos || !sin || !q_out) return FP8KV_ERR_INVALID_ARG;
  const int64_t qw = (int64_t)q_heads * cache->head_dim, kw = (int64_t)cache->kv_heads * cache->head_dim;
  if (q_stride < qw || k_stride < kw || v_stride < kw) return FP8KV_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8) return FP8KV_ERR_INVALID_ARG;
  for (const void* a : {q, k, v, (const void*)cos, (const void*)sin, (const void*)q_out})
    if (misaligned(a, 16)) return FP8KV_ERR_INVALID_ARG;
  if (misaligned(slots, 8) || misaligned(pos, 4)) return FP8KV_ERR_INVALID_ARG;
  // q_out: a buffer of its own, or q rotated in place
  const int64_t N = n_tokens;
  const Range out = {q_out, (size_t)(2 * N * qw)};
  if (!(q_out == q && q_stride == qw) && overlap(out, {q, (size_t)(2 * ((N - 1) * q_stride + qw))}))
    return FP8KV_ERR_INVALID_ARG;
  if (overlap(out, {k, (size_t)(2 * ((N - 1) * k_stride + kw))}) ||
      overlap(out, {v, (size_t)(2 * ((N - 1) * v_stride + kw))}))
    return FP8KV_ERR_INVALID_ARG;
  p.err = device_error_ptr();
  if (!p.err) return FP8KV_ERR_CUDA;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.pos = pos;
  p.slots = slots;
  p.cos = cos;
  p.sin = sin;
  p.n = n_tokens;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_heads = q_heads;
  p.rot = rot_dim;
  // a turning key bias has its own table, one row per position of the cache
  p.positions = cache->rope_cos != nullptr && cache->rope_positions < positions ? cache->rope_positions : positions;
  p.interleaved = layout == FP8KV_ROPE_INTERLEAVED;
  return cuda_status(launch_rope_append(p, cache->dtype, (cudaStream_t)stream));
}

int32_t fp8kv_chunk_num_splits(const fp8kv_cache* cache, int64_t total_q, int32_t q_heads, int32_t window,
                               int32_t sinks, int32_t num_splits, int32_t kernel) {
  CacheView view;
  ChunkPlan plan;
  if (check_cache(cache, &view) != FP8KV_OK) return 0;
  if (plan_chunk(cache, total_q, q_heads, window, sinks, num_splits, kernel, false, &plan) != FP8KV_OK) return 0;
  return plan.splits;
}

size_t fp8kv_chunk_workspace_bytes(const fp8kv_cache* cache, int64_t total_q, int32_t q_heads, int32_t window,
                                   int32_t sinks, int32_t num_splits, int32_t kernel) {
  return share_bytes(cache, total_q, q_heads, fp8kv_chunk_num_splits(cache, total_q, q_heads, window, sinks, num_splits, kernel));
}

fp8kv_status fp8kv_chunk_attention(const void* q, const fp8kv_cache* cache, const int32_t* cu_q,
                                   const int32_t* seq_lens, int64_t total_q, int32_t q_heads, float sm_scale,
                                   int32_t window, int32_t sinks, int32_t num_splits, int32_t kernel,
                                   void* workspace, size_t workspace_bytes, void* out, int32_t out_dtype,
                                   fp8kv_stream_t stream) {
  return run_chunk(q, cache, cu_q, seq_lens, nullptr, total_q, q_heads, sm_scale, window, sinks, num_splits, kernel,
                   workspace, workspace_bytes, out, out_dtype, stream);
}

size_t fp8kv_tree_workspace_bytes(const fp8kv_cache* cache, int64_t total_q, int32_t q_heads, int32_t window,
                                  int32_t sinks, int32_t num_splits, int32_t kernel) {
  CacheView view;
  ChunkPlan plan;
  if (check_cache(cache, &view) != FP8KV_OK) return 0;
  if (plan_chunk(cache, total_q, q_heads, window, sinks, num_splits, kernel, true, &plan) != FP8KV_OK) return 0;
  return share_bytes(cache, total_q, q_heads, plan.splits);
}

fp8kv_status fp8kv_tree_attention(const void* q, const fp8kv_cache* cache, const int32_t* cu_q,
                                  const int32_t* seq_lens, const uint32_t* masks, int32_t mask_words,
                                  const int32_t* pos, int64_t total_q, int32_t q_heads, float sm_scale, int32_t window,
                                  int32_t sinks, int32_t num_splits, int32_t kernel, void* workspace,
                                  size_t workspace_bytes, void* out, int32_t out_dtype, fp8kv_stream_t stream) {
  const TreeArgs tree = {masks, pos, mask_words};
  return run_chunk(q, cache, cu_q, seq_lens, &tree, total_q, q_heads, sm_scale, window, sinks, num_splits, kernel,
                   workspace, workspace_bytes, out, out_dtype, stream);
}

fp8kv_status fp8kv_tree_tables(const int32_t* parents, const int32_t* cu_new, const int32_t* seq_lens, int32_t batch,
                               int64_t n_rows, int32_t mask_words, uint32_t* masks, int32_t* pos,
                               fp8kv_stream_t stream) {
  return fp8kv_tree_tables_window(parents, cu_new, seq_lens, batch, n_rows, mask_words, 0, 0, masks, pos, stream);
}

fp8kv_status fp8kv_tree_tables_window(const int32_t* parents, const int32_t* cu_new, const int32_t* seq_lens,
                                      int32_t batch, int64_t n_rows, int32_t mask_words, int32_t window, int32_t sinks,
                                      uint32_t* masks, int32_t* pos, fp8kv_stream_t stream) {
  if (batch < 0 || n_rows < 0 || mask_words < 1 || window < 0 || sinks < 0 || !cu_new) return FP8KV_ERR_INVALID_ARG;
  if (mask_words > kTreeMaxNodes / 32 || n_rows > INT32_MAX || batch > INT32_MAX - 64) return FP8KV_ERR_UNSUPPORTED;
  if (batch > 0 && !seq_lens) return FP8KV_ERR_INVALID_ARG;
  if (n_rows == 0) return FP8KV_OK;
  if (!parents || !masks || !pos) return FP8KV_ERR_INVALID_ARG;
  const size_t N = (size_t)n_rows, B = (size_t)batch;
  const Range in[] = {{parents, 4 * N}, {cu_new, 4 * (B + 1)}, {seq_lens, 4 * B}};
  const Range out[] = {{masks, 4 * N * mask_words}, {pos, 4 * N}};
  for (const Range& o : out) {
    if (misaligned(o.p, 4)) return FP8KV_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (misaligned(r.p, 4) || overlap(r, o)) return FP8KV_ERR_INVALID_ARG;
  }
  if (overlap(out[0], out[1])) return FP8KV_ERR_INVALID_ARG;
  TreeTablesParams p;
  p.err = device_error_ptr();
  if (!p.err) return FP8KV_ERR_CUDA;
  p.parents = parents;
  p.cu = cu_new;
  p.seq_lens = seq_lens;
  p.masks = masks;
  p.pos = pos;
  p.batch = batch;
  p.rows = (int)n_rows;
  p.words = mask_words;
  p.window = window;
  p.sinks = sinks;
  return cuda_status(launch_tree_tables(p, (cudaStream_t)stream));
}

fp8kv_status fp8kv_tree_accept(const fp8kv_cache* const* caches, int32_t num_caches, const int32_t* parents,
                               const int64_t* tokens, const int64_t* choices, const int32_t* cu_new,
                               const int32_t* seq_lens, int32_t batch, int64_t n_rows, int32_t max_path, int32_t* path,
                               int32_t* accepted, int64_t* next_tokens, int32_t* new_lens, fp8kv_stream_t stream) {
  if (num_caches < 0 || batch < 0 || n_rows < 0 || max_path < 1 || (num_caches > 0 && !caches))
    return FP8KV_ERR_INVALID_ARG;
  if (num_caches > kTreeMostCaches || n_rows > INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
  TreeAcceptParams p;
  const size_t N = (size_t)n_rows, B = (size_t)batch;
  const Range out[] = {{path, 4 * B * max_path}, {accepted, 4 * B}, {next_tokens, 8 * B}, {new_lens, 4 * B}};
  const Range in[] = {{parents, 4 * N}, {tokens, 8 * N}, {choices, 8 * N}, {cu_new, 4 * (B + 1)}, {seq_lens, 4 * B}};
  // what the call moves rows of: no cache twice, none that shares memory with another, or with the other arguments
  Range held[4 * kTreeMostCaches];
  int n_held = 0;
  const fp8kv_cache* c0 = nullptr;
  for (int i = 0; i < num_caches; ++i) {
    const fp8kv_cache* c = caches[i];
    CacheView view;
    const fp8kv_status st = check_cache(c, &view);
    if (st != FP8KV_OK) return st;
    if (!capacity_fits(c)) return FP8KV_ERR_UNSUPPORTED;
    if (i == 0) c0 = c;
    if (c->batch != batch || c->dtype != c0->dtype || c->layout != c0->layout || c->kv_heads != c0->kv_heads ||
        c->head_dim != c0->head_dim || c->page_size != c0->page_size)
      return FP8KV_ERR_INVALID_ARG;
    n_held += cache_rows_of(c, held + n_held);
    for (const Range& o : out)
      if (overlap(o, cache_table_of(c))) return FP8KV_ERR_INVALID_ARG;
  }
  if (batch == 0) return FP8KV_OK;
  if (!cu_new || !seq_lens || !path || !accepted || !next_tokens || !new_lens) return FP8KV_ERR_INVALID_ARG;
  if (n_rows > 0 && (!parents || !tokens || !choices)) return FP8KV_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i) {
    if (misaligned(out[i].p, i == 2 ? 8 : 4)) return FP8KV_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (overlap(r, out[i])) return FP8KV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[j], out[i])) return FP8KV_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 5; ++i)
    if (misaligned(in[i].p, i == 1 || i == 2 ? 8 : 4)) return FP8KV_ERR_INVALID_ARG;
  // in the order of their addresses only neighbours can overlap
  std::sort(held, held + n_held, [](const Range& a, const Range& b) { return (uintptr_t)a.p < (uintptr_t)b.p; });
  for (int i = 0; i < n_held; ++i) {
    if (i > 0 && overlap(held[i - 1], held[i])) return FP8KV_ERR_INVALID_ARG;
    for (const Range& o : out)
      if (overlap(o, held[i])) return FP8KV_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (overlap(r, held[i])) return FP8KV_ERR_INVALID_ARG;
  }
  // a page table among rows would be written over while another layer's CTAs read it (the
  // layers of a model share one table: looked at once)
  for (int i = 0; i < num_caches; ++i) {
    const fp8kv_cache* c = caches[i];
    if (c->layout != FP8KV_LAYOUT_PAGED || (i > 0 && c->page_table == caches[i - 1]->page_table &&
                                            c->max_pages_per_seq == caches[i - 1]->max_pages_per_seq)) continue;
    const Range table = cache_table_of(c);
    const Range* next = std::upper_bound(held, held + n_held, table, [](const Range& a, const Range& b) { return (uintptr_t)a.p < (uintptr_t)b.p; });
    if (next != held && overlap(next[-1], table)) return FP8KV_ERR_INVALID_ARG;
    if (next != held + n_held && overlap(*next, table)) return FP8KV_ERR_INVALID_ARG;
  }
  p.err = device_error_ptr();
  if (!p.err) return FP8KV_ERR_CUDA;
  p.parents = parents;
  p.cu = cu_new;
  p.seq_lens = seq_lens;
  p.tokens = tokens;
  p.choices = choices;
  p.path = path;
  p.accepted = accepted;
  p.new_lens = new_lens;
  p.next = next_tokens;
  p.batch = batch;
  p.rows = (int)n_rows;
  p.max_path = max_path;
  p.kv_heads = p.k_bytes = p.v_bytes = p.page_shift = p.paged = 0;
  if (c0 != nullptr) {
    p.kv_heads = c0->kv_heads;
    p.k_bytes = c0->head_dim * (c0->k_scale ? 1 : 2);
    p.v_bytes = c0->head_dim * (c0->v_scale ? 1 : 2);
    p.paged = c0->layout == FP8KV_LAYOUT_PAGED;
    while (p.paged && (1 << p.page_shift) < c0->page_size) ++p.page_shift;
  }
  int at = 0;
  do {
    p.first = at == 0;
    p.layers = num_caches - at < kTreeMaxLayers ? num_caches - at : kTreeMaxLayers;
    for (int i = 0; i < p.layers; ++i) {
      const fp8kv_cache* c = caches[at + i];
      p.layer[i] = {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), reinterpret_cast<uint32_t*>(c->k_scale),
                    reinterpret_cast<uint32_t*>(c->v_scale), c->page_table, c->num_pages, c->max_pages_per_seq,
                    c->max_tokens};
    }
    const cudaError_t e = launch_tree_accept(p, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_status(e);
    at += p.layers;
  } while (at < num_caches);
  return FP8KV_OK;
}

}  // extern "C"
