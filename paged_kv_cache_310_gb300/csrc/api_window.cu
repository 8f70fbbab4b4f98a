// api_window.cu -- the extern "C" entry points of attention over sliding windows (declared in
// include/pagedkv.h): argument checks, the choice of a kernel, launches.
#include <algorithm>
#include <cmath>

#include "api_util.h"
#include "launch.h"

using namespace pkv;

namespace {

constexpr float kLog2e = 1.4426950408889634f;  // softmax is evaluated with exp2
constexpr int kMaxGroup = 16;

// The arguments of both calls; query_start is NULL for one new token per sequence.
struct Args {
  const void *q, *k_cache, *v_cache;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t *context_lens, *query_start;
  int32_t num_seqs, num_q_heads, num_query_tokens, max_context_len, window, sinks;
  float scale;
  void* out;
  int32_t out_dtype;
  const pkv_cache_desc* cache;
};

// What can be refused for either call whatever the pointers are.
pkv_status check_sizes(const Args& a) {
  if (pkv_status st = check_cache(a.cache)) return st;
  if (a.window < 1) return fail(PKV_ERR_INVALID_ARG, "window %d < 1", a.window);
  if (a.sinks < 0) return fail(PKV_ERR_INVALID_ARG, "sinks %d < 0", a.sinks);
  if (a.num_q_heads <= 0 || a.num_q_heads % a.cache->num_kv_heads)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of num_kv_heads %d", a.num_q_heads,
                a.cache->num_kv_heads);
  if (a.num_q_heads / a.cache->num_kv_heads > kMaxGroup)
    return fail(PKV_ERR_UNSUPPORTED, "query-head groups of %d (at most %d)", a.num_q_heads / a.cache->num_kv_heads, kMaxGroup);
  if (a.num_query_tokens < 0 || a.max_context_len < 0) return fail(PKV_ERR_INVALID_ARG, "negative size");
  if (a.max_context_len > (1 << 30)) return fail(PKV_ERR_UNSUPPORTED, "max_context_len %d above 2^30", a.max_context_len);
  if (static_cast<int64_t>(a.num_query_tokens) * a.num_q_heads > INT32_MAX)
    return fail(PKV_ERR_UNSUPPORTED, "more than 2^31 - 1 query rows");
  return PKV_OK;
}

pkv_status check_pointers(const Args& a) {
  if (!a.q || !a.k_cache || !a.v_cache || !a.context_lens || !a.out) return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (a.max_context_len > 0 && !a.block_tables) return fail(PKV_ERR_INVALID_ARG, "block_tables is NULL");
  if (!aligned16(a.q) || !aligned16(a.k_cache) || !aligned16(a.v_cache) || !aligned16(a.out))
    return fail(PKV_ERR_INVALID_ARG, "q, out and the caches must be 16-byte aligned");
  if (a.out_dtype != a.cache->dtype && a.out_dtype != PKV_F32)
    return fail(PKV_ERR_UNSUPPORTED, "out dtype %d (must be the cache dtype or f32)", a.out_dtype);
  if (!std::isfinite(a.scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  const int64_t need_blocks = (static_cast<int64_t>(a.max_context_len) + a.cache->block_size - 1) / a.cache->block_size;
  if (a.max_blocks_per_seq < need_blocks)
    return fail(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d < ceil(max_context_len / block_size) = %lld",
                a.max_blocks_per_seq, static_cast<long long>(need_blocks));
  return PKV_OK;
}

// A window past every sequence's start and sinks past its end change nothing.
int32_t held_window(const Args& a) { return std::min(a.window, std::max(a.max_context_len, 1)); }
int32_t held_sinks(const Args& a) { return std::min(a.sinks, a.max_context_len); }
int32_t blocks_of(int32_t tokens, int32_t block_size) { return tokens > 0 ? (tokens - 1) / block_size + 1 : 0; }

WindowRowsParams rows_params(const Args& a, int cluster, int* flag) {
  WindowRowsParams p{};
  p.q = a.q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  p.out = a.out;
  p.err = flag;
  p.num_seqs = a.num_seqs;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.cache->num_kv_heads;
  p.group = a.num_q_heads / a.cache->num_kv_heads;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.block_size = a.cache->block_size;
  p.num_blocks = a.cache->num_blocks;
  p.head_dim = a.cache->head_dim;
  p.num_query_tokens = a.num_query_tokens;
  p.max_len = a.max_context_len;
  p.window = held_window(a);
  p.sinks = held_sinks(a);
  p.sink_blocks = blocks_of(p.sinks, p.block_size);
  p.cluster = cluster;
  p.out_f32 = a.out_dtype == PKV_F32 ? 1 : 0;
  p.scale_log2 = a.scale * kLog2e;
  return p;
}

WindowPrefillParams prefill_params(const Args& a) {
  WindowPrefillParams p{};
  p.q = a.q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  p.out = a.out;
  p.num_seqs = a.num_seqs;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.cache->num_kv_heads;
  p.group = a.num_q_heads / a.cache->num_kv_heads;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.block_size = a.cache->block_size;
  p.num_blocks = a.cache->num_blocks;
  p.max_context_len = a.max_context_len;
  p.num_query_tokens = a.num_query_tokens;
  p.tile_tokens = prefill_tile_tokens(p.group);
  p.head_dim = a.cache->head_dim;
  p.out_f32 = a.out_dtype == PKV_F32 ? 1 : 0;
  p.scale_log2 = a.scale * kLog2e;
  p.wait_limit_ns = wait_limit_ns();
  p.window = held_window(a);
  p.sinks = held_sinks(a);
  p.sink_blocks = blocks_of(p.sinks, p.block_size);
  return p;
}

// The tokens that `span` new tokens of one sequence attend to at most.
int64_t keys_of(const Args& a, int64_t span) {
  return std::min<int64_t>(a.max_context_len, static_cast<int64_t>(a.window) + a.sinks + span);
}

constexpr int64_t kSms = 152;

// CTAs that share the tokens of one of `items` (columns, KV head) in the kernels of
// window_rows.cuh: up to three an SM in all, of 64 tokens or more each.
// Clusters start slowly -- about 20 ns each at 2 CTAs, 200 at 8 -- so many items go unshared
// (64 sequences, 64/8 heads, D 64, window 128: 10 us with one CTA, 25 with two).  Three whatever an SM
// holds: at four of the 16-bit kernel at D 64, which it does hold, 19 sequences, 64/8 heads, window
// 1,020 take 25 us instead of 18; at two of the f32 kernel with 16 heads at D 128, the most that it
// holds, 28 sequences, 96/8 heads take 264 us instead of 213 under a window of 4,092, though 31 instead
// of 41 under one of 252.
int rows_cluster(int64_t items, int64_t tokens) {
  int size = 1;
  while (size < 8 && 2 * size * items <= 3 * kSms && tokens > 64 * size) size *= 2;
  return size;
}

struct PrefillPlan {
  pkv_window_kernel kernel;
  int cluster;  // CTAs that share an item (rows; 1 for the others)
};

// Which kernel a windowed prefill takes: the one with the shortest estimate, for sequences that
// share the new tokens out evenly (the host knows no more of them).  Only the estimates' order
// matters; on calls of 1 to 64 sequences with 4 to 2,400 new tokens each, windows of 128 to 4,096,
// head_dim 64 and 128, it was right or within a tenth but for one (32 sequences of 5, D 64, window
// 4,096: 114 us with rows, 101 with shared tiles).  In us:
//  * rows: 10 + 0.85 (D 128) or 0.65 (D 64) per 1,000 tiles of 16 tokens for 16 query rows (1
//    sequence of 4 new tokens, 64/8 heads, window 4,096: 21 against 51 with shared tiles; 64 of 4, D 64,
//    window 256: 29 against 36);
//  * shared tiles: 12 + 2.1 a step of 128 tokens for one tile (64 sequences of 8, window 1,024: 82 against
//    133 with rows, 103 with pairs; 32 of 5, window 4,096: 110 against 160 and 166);
//  * pairs: 10 + 1.55 a step of 64 tokens for two tiles (4 sequences of 256, window 1,024: 53 against 72
//    with shared tiles, 240 with rows).
PrefillPlan plan_prefill(const Args& a) {
  const int64_t S = a.num_seqs, H = a.cache->num_kv_heads, T = a.num_query_tokens;
  const int group = a.num_q_heads / a.cache->num_kv_heads;
  auto groups = [&](int64_t span) { return S * ((T + S * span - 1) / (S * span)); };
  auto rounds = [&](int64_t items) { return (items + kSms - 1) / kSms; };
  const int64_t per = kRowsPerGroup / group, tq = prefill_tile_tokens(group);
  const int64_t row_groups = groups(per);
  const double rows = 10. + (a.cache->head_dim == 64 ? 0.65e-3 : 0.85e-3) * static_cast<double>(row_groups * H * (keys_of(a, per) / 16 + 1));
  const double shared = 12. + 2.1 * static_cast<double>(rounds(groups(tq) * H) * (keys_of(a, tq) / 128 + 1));
  const double pairs = 10. + 1.55 * static_cast<double>(rounds(groups(2 * tq) * H) * (keys_of(a, 2 * tq) / 64 + 1));
  PrefillPlan plan{shared < pairs ? PKV_WINDOW_SHARED_TILES : PKV_WINDOW_TILE_PAIRS, 1};
  if (rows < std::min(shared, pairs) && T / per + S <= 65535) {  // a grid's third dimension
    plan.kernel = PKV_WINDOW_ROWS;
    plan.cluster = rows_cluster(row_groups * H, keys_of(a, per));
  }
  return plan;
}

// What a windowed prefill refuses by its sizes: before those that leave nothing to do return, and after.
pkv_status check_prefill(const Args& a) {
  if (a.num_seqs < 0 || a.num_seqs > (1 << 20)) return fail(PKV_ERR_INVALID_ARG, "num_seqs %d", a.num_seqs);
  if (pkv_status st = check_sizes(a)) return st;
  if (a.cache->dtype == PKV_F32) return fail(PKV_ERR_UNSUPPORTED, "windowed prefill needs f16 or bf16 caches");
  if (a.cache->num_kv_heads > 4095)  // an item packs the KV head into 12 bits
    return fail(PKV_ERR_UNSUPPORTED, "prefill supports at most 4095 KV heads (%d)", a.cache->num_kv_heads);
  return PKV_OK;
}
pkv_status check_prefill_counts(const Args& a) {
  if (static_cast<int64_t>(a.cache->num_blocks) * a.cache->num_kv_heads * a.cache->block_size > (int64_t{1} << 30))
    return fail(PKV_ERR_UNSUPPORTED, "pool too large for 32-bit row coordinates");
  if (window_prefill_items(prefill_params(a), true) > (int64_t{1} << 30))
    return fail(PKV_ERR_UNSUPPORTED, "too many (new tokens, KV head) items");
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status paged_attention_decode_window(const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t max_context_len, int32_t window, int32_t sinks, float scale, void* out,
                                         int32_t out_dtype, const pkv_cache_desc* cache, void* stream) {
  const Args a{q,           k_cache,  v_cache,         block_tables, max_blocks_per_seq, context_lens, nullptr, num_seqs,
               num_q_heads, num_seqs, max_context_len, window,       sinks,              scale,        out,     out_dtype,
               cache};
  if (num_seqs < 0 || num_seqs > 65535) return fail(PKV_ERR_INVALID_ARG, "num_seqs %d outside [0, 65535]", num_seqs);
  if (pkv_status st = check_sizes(a)) return st;
  if (num_seqs == 0) return PKV_OK;
  if (pkv_status st = check_pointers(a)) return st;
  int* flag = nullptr;
  if (pkv_status st = device_flag(&flag)) return st;
  const int cluster = rows_cluster(static_cast<int64_t>(num_seqs) * cache->num_kv_heads, keys_of(a, 1));
  cudaError_t e = launch_window_rows(rows_params(a, cluster, flag), cache->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "windowed decode launch");
}

pkv_status paged_attention_prefill_window(const void* q, const void* k_cache, const void* v_cache,
                                          const int32_t* block_tables, int32_t max_blocks_per_seq,
                                          const int32_t* context_lens, const int32_t* query_start, int32_t num_seqs,
                                          int32_t num_q_heads, int32_t num_query_tokens, int32_t max_context_len,
                                          int32_t window, int32_t sinks, float scale, void* out, int32_t out_dtype,
                                          const pkv_cache_desc* cache, void* stream) {
  const Args a{q,           k_cache,          v_cache,         block_tables, max_blocks_per_seq, context_lens, query_start,
               num_seqs,    num_q_heads,      num_query_tokens, max_context_len, window,         sinks,        scale,
               out,         out_dtype,        cache};
  if (pkv_status st = check_prefill(a)) return st;
  if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
  if (!query_start) return fail(PKV_ERR_INVALID_ARG, "query_start is NULL");
  if (pkv_status st = check_pointers(a)) return st;
  if (pkv_status st = check_prefill_counts(a)) return st;
  WindowPrefillParams p = prefill_params(a);
  if (pkv_status st = device_flag(&p.err)) return st;
  const PrefillPlan plan = plan_prefill(a);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = plan.kernel == PKV_WINDOW_ROWS
                            ? launch_window_rows(rows_params(a, plan.cluster, p.err), cache->dtype, s)
                            : launch_window_prefill(p, plan.kernel == PKV_WINDOW_SHARED_TILES, cache->dtype, s);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "windowed prefill launch");
}

pkv_status paged_attention_prefill_window_plan(int32_t num_seqs, int32_t num_q_heads, int32_t num_query_tokens,
                                               int32_t max_context_len, int32_t window, int32_t sinks,
                                               const pkv_cache_desc* cache, pkv_window_plan* out) {
  if (!out) return fail(PKV_ERR_INVALID_ARG, "plan output is NULL");
  Args a{};
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_query_tokens = num_query_tokens;
  a.max_context_len = max_context_len;
  a.window = window;
  a.sinks = sinks;
  a.cache = cache;
  if (pkv_status st = check_prefill(a)) return st;
  *out = pkv_window_plan{PKV_WINDOW_ROWS, 0, 0};
  if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
  if (pkv_status st = check_prefill_counts(a)) return st;
  const PrefillPlan plan = plan_prefill(a);
  const int per_tile = prefill_tile_tokens(num_q_heads / cache->num_kv_heads);
  out->kernel = plan.kernel;
  out->tokens_per_item = plan.kernel == PKV_WINDOW_ROWS           ? kRowsPerGroup / (num_q_heads / cache->num_kv_heads)
                         : plan.kernel == PKV_WINDOW_SHARED_TILES ? per_tile
                                                                  : 2 * per_tile;
  out->ctas_per_item = plan.cluster;
  return PKV_OK;
}

}  // extern "C"
