// api_step.cu -- the extern "C" boundary of the serving-step calls: argument
// checks, launch plans, status codes.  As in api.cu, every entry validates on
// the host, launches on the caller's stream and allocates nothing.
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "params.cuh"

using namespace fp8kv;

namespace {

struct Range { const void* p; size_t bytes; };

bool overlap(const Range& a, const Range& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.bytes && y < x + a.bytes;
}

bool misaligned(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) != 0; }

// Positions are 32-bit: a page table row may not hold more tokens.
bool capacity_fits(const fp8kv_cache* c) {
  return c->layout != FP8KV_LAYOUT_PAGED || (int64_t)c->max_pages_per_seq * c->page_size <= INT32_MAX;
}

struct ChunkPlan { int kernel, tile_rows, tile_tokens, tiles, splits; };

// How a chunk call runs, from its sizes (lengths are on the device).
// Kernel, by the average number of query rows (queries x heads of a group) a
// sequence has: up to 16 rows the few-row kernel, in tiles of 8 or 16 (one token
// of 64 sequences under a 1,024-token window: 35 us, against 81 us on tcgen05; two
// tokens x 8 heads of 64 sequences of 2K-4K tokens: 74 us, against 101 us);
// above, tcgen05 where it is built.  Between 17 and 32 rows neither is clearly ahead
// (8 tokens x 4 heads over 8,000 tokens, 4 sequences: 40 us against 45 us at the best
// split counts; 2-4 x 8 over 4K-8K, 16 sequences: 62 against 58 to 71), far above
// it is (256 x 4 over 16,000: 108 against 447).  The average counts idle sequences
// and rows of padding, and one kernel runs the whole call: batches of unlike
// sequences (a prompt in many idle slots, or beside many single tokens) get the
// form that suits only some of them.  Lengths of queries are on the device, so the
// host knows no better.  Block-scaled keys stay on the few-row kernel (2-4 x 8 over
// 4K-8K, 16 sequences: 63 us, 88 us on the form that the warp-level kernel had for
// them; 256-512 x 8, 4 sequences: 1.15 ms against 1.33), head dim 64 does up to 32
// rows (2-4 x 8 of 64 sequences of 2K-4K, bf16: 64 us against 71 on 64-row tiles at
// the best split count), with more it runs on the warp-level kernel (256-512 x 8 over
// 4K-8K, 4 sequences: 0.56 ms against 0.70; around 64 rows either can be faster).
//
// Splits of the few-row kernel: an SM holds four of its CTAs (three of 16 rows,
// or of 32 KiB stages), and a call takes as many waves of them as they need,
// each as long as one share and the 8 tiles' time that a CTA spends on its
// start and end.  So the counts that fill one, two or three waves are compared:
// 256 units of 32-64 tiles (16 rows) take 100 us whole, 84 us in 2 shares (1.1
// waves), 75 us in 3 (1.7), 79 us in 4.  Shares are 192 keys or longer (one token of
// 32 / 8 heads over 6,200: 10.6 us in 32 shares, 11.1 in 24, 12.1 in 64).
// Without a window lengths can differ widely: shares of about 4,096 keys at most
// then even them out (64 sequences of 1K-16K tokens, 32 / 8 heads: 249 us in 4
// shares, 355 us whole; sequences of 700 tokens in the same cache pay 35 us instead of 23), as
// long as that makes no more than 16 CTAs an SM.
//
// Splits of the others: tiles are few -> one wave.  tcgen05: two CTAs an SM,
// shares of 512 keys or longer.  Warp-level kernel: three an SM (by their
// registers) and 128 keys (32-64 x 8 of 2 sequences of 2K-4K tokens: 36 us in 4
// shares, 31 us in 6, 37 us in 9, past one wave).
fp8kv_status plan_chunk(const fp8kv_cache* c, int64_t total_q, int q_heads, int window, int sinks, int num_splits,
                        int kernel, ChunkPlan* plan) {
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
  const bool tc = cap > 0 && (kernel == FP8KV_KERNEL_TENSOR_CORES || (kernel == FP8KV_KERNEL_AUTO && tc_built && rows > 16));
  plan->kernel = tc ? FP8KV_KERNEL_TENSOR_CORES : FP8KV_KERNEL_WARP_MMA;
  plan->tile_rows = tc ? 128 : rows <= 8 ? 8 : c->head_dim == 128 || rows <= 32 ? 16 : 64;
  plan->tile_tokens = plan->tile_rows / G;
  const int64_t tiles = total_q / plan->tile_tokens + c->batch;      // at most (chunk_common.cuh)
  if (tiles > INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
  plan->tiles = (int)tiles;
  const int64_t seen = window > 0 && window < cap ? (int64_t)window + plan->tile_tokens + (sinks < cap ? sinks : cap) : cap;
  const int64_t kv_tiles = ((seen < cap ? seen : cap) + 63) / 64 + 1;
  int64_t want = num_splits;
  if (want == 0) {
    // tiles if every sequence had the average number of queries, or, if that is
    // not a whole number, as many more or fewer of them as it says
    const int64_t T = plan->tile_tokens, even_q = (total_q / B + T - 1) / T * B, some_q = (total_q + T - 1) / T;
    const int64_t units = (total_q % B == 0 ? even_q : some_q > B ? some_q : B) * c->kv_heads;
    const int64_t sms = sm_count();
    if (plan->tile_rows > 16) {
      want = units > 0 ? (tc ? 2 : 3) * sms / units : 1;
      const int64_t most = kv_tiles / (tc ? 8 : 2);
      if (want > most) want = most;
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
  if (want > kv_tiles) want = kv_tiles;
  if (want > 4096) want = 4096;
  plan->splits = want < 1 ? 1 : (int)want;
  return FP8KV_OK;
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
  if (plan_chunk(cache, total_q, q_heads, window, sinks, num_splits, kernel, &plan) != FP8KV_OK) return 0;
  return plan.splits;
}

size_t fp8kv_chunk_workspace_bytes(const fp8kv_cache* cache, int64_t total_q, int32_t q_heads, int32_t window,
                                   int32_t sinks, int32_t num_splits, int32_t kernel) {
  const int S = fp8kv_chunk_num_splits(cache, total_q, q_heads, window, sinks, num_splits, kernel);
  if (S <= 1) return 0;
  return (size_t)total_q * q_heads * S * ((size_t)cache->head_dim + 2) * sizeof(float);
}

fp8kv_status fp8kv_chunk_attention(const void* q, const fp8kv_cache* cache, const int32_t* cu_q,
                                   const int32_t* seq_lens, int64_t total_q, int32_t q_heads, float sm_scale,
                                   int32_t window, int32_t sinks, int32_t num_splits, int32_t kernel,
                                   void* workspace, size_t workspace_bytes, void* out, int32_t out_dtype,
                                   fp8kv_stream_t stream) {
  ChunkParams p;
  fp8kv_status st = check_cache(cache, &p.c);
  if (st != FP8KV_OK) return st;
  ChunkPlan plan;
  st = plan_chunk(cache, total_q, q_heads, window, sinks, num_splits, kernel, &plan);
  if (st != FP8KV_OK) return st;
  if (out_dtype != FP8KV_OUT_BF16 && out_dtype != FP8KV_OUT_F32) return FP8KV_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale)) return FP8KV_ERR_INVALID_ARG;
  if (cu_q == nullptr && total_q != cache->batch) return FP8KV_ERR_INVALID_ARG;
  if (cache->batch == 0 || total_q == 0) return FP8KV_OK;
  if (!q || !seq_lens || !out || misaligned(q, 16) || misaligned(out, 16)) return FP8KV_ERR_INVALID_ARG;
  if (misaligned(cu_q, 4) || misaligned(seq_lens, 4)) return FP8KV_ERR_INVALID_ARG;
  const int64_t rows = total_q * q_heads;
  const size_t values = (size_t)rows * cache->head_dim;
  if (overlap({q, 2 * values}, {out, (out_dtype == FP8KV_OUT_F32 ? 4 : 2) * values})) return FP8KV_ERR_INVALID_ARG;
  const size_t need = fp8kv_chunk_workspace_bytes(cache, total_q, q_heads, window, sinks, num_splits, kernel);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FP8KV_ERR_WORKSPACE;
  if (need > 0 && misaligned(workspace, 16)) return FP8KV_ERR_INVALID_ARG;
  for (const Range& r : {Range{q, 2 * values}, Range{out, (out_dtype == FP8KV_OUT_F32 ? 4 : 2) * values}})
    if (overlap(r, {workspace, need})) return FP8KV_ERR_INVALID_ARG;
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
  p.window = window < capacity_of(cache) ? window : 0;
  p.sinks = sinks;
  p.num_splits = plan.splits;
  p.tile_tokens = plan.tile_tokens;
  p.scale_log2 = sm_scale * kLog2e;
  cudaStream_t s = (cudaStream_t)stream;
  const int tiles = cu_q ? plan.tiles : cache->batch;
  cudaError_t e = plan.kernel == FP8KV_KERNEL_TENSOR_CORES ? launch_chunk_tc(p, cache->dtype, tiles, s)
                  : plan.tile_rows <= 16 ? launch_chunk_rows(p, cache->dtype, tiles, s)
                                        : launch_chunk_mma(p, cache->dtype, tiles, s);
  if (e == cudaSuccess && plan.splits > 1) e = launch_chunk_merge(p, s);
  return cuda_status(e);
}

}  // extern "C"
