// api_kv4.cu -- the extern "C" entry points of the cache-compression calls (declared in
// include/pagedkv.h): 4-bit caches and eviction by attention weight.
#include <cmath>

#include "api_util.h"
#include "launch.h"

using namespace pkv;

namespace {

bool is_wide(int dtype) { return dtype >= PKV_F32 && dtype <= PKV_BF16; }

pkv_status check_kv4(const pkv_cache_desc* c) {
  if (pkv_status st = check_cache(c, true)) return st;
  if (c->dtype != PKV_KV4) return fail(PKV_ERR_UNSUPPORTED, "cache dtype %d (this call takes PKV_KV4 pools)", c->dtype);
  // rows of a block are indexed in 32 bits
  if (static_cast<int64_t>(c->num_kv_heads) * c->block_size * c->head_dim > (int64_t{1} << 30))
    return fail(PKV_ERR_UNSUPPORTED, "%d KV heads of %d tokens: block too large", c->num_kv_heads, c->block_size);
  return PKV_OK;
}

struct Kv4Plan {
  int ctas;
  bool whole;
  size_t ml_at, o_at, workspace;  // offsets of the workspace's parts; 0 bytes: no item is ever split
};

pkv_status plan_kv4(int32_t num_seqs, int32_t num_q_heads, int32_t max_len, int32_t q_dtype, const pkv_cache_desc* c,
                    Kv4Plan* plan) {
  if (pkv_status st = check_kv4(c)) return st;
  if (num_seqs < 0 || num_seqs > 65535) return fail(PKV_ERR_INVALID_ARG, "num_seqs %d outside [0, 65535]", num_seqs);
  if (num_q_heads <= 0 || num_q_heads % c->num_kv_heads)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of num_kv_heads %d", num_q_heads,
                c->num_kv_heads);
  const int group = num_q_heads / c->num_kv_heads;
  if (group > kKv4MaxGroup)
    return fail(PKV_ERR_UNSUPPORTED, "4-bit decode supports query-head groups <= %d (group %d)", kKv4MaxGroup, group);
  if (!is_wide(q_dtype)) return fail(PKV_ERR_UNSUPPORTED, "q dtype %d", q_dtype);
  if (max_len < 0) return fail(PKV_ERR_INVALID_ARG, "max_context_len %d < 0", max_len);
  if (max_len > (1 << 30)) return fail(PKV_ERR_UNSUPPORTED, "max_context_len %d above 2^30", max_len);
  const int64_t units = (static_cast<int64_t>(max_len) + kKv4Unit - 1) / kKv4Unit;
  const int64_t most = units * num_seqs * c->num_kv_heads;
  if (most > (int64_t{1} << 50)) return fail(PKV_ERR_UNSUPPORTED, "%lld units of work", static_cast<long long>(most));
  const int64_t items = static_cast<int64_t>(num_seqs) * c->num_kv_heads;
  plan->ctas = kv4_decode_ctas(c->head_dim, group, q_dtype, most, items < 1 ? 1 : items);
  plan->ml_at = plan->o_at = plan->workspace = 0;
  plan->whole = max_len <= kKv4Whole && items <= kv4_decode_ctas(c->head_dim, group, q_dtype, int64_t{1} << 50, 1);
  if (plan->whole) {
    plan->ctas = items < 1 ? 1 : static_cast<int>(items);
    return PKV_OK;
  }
  if (units > 1 && plan->ctas > 1 && num_seqs > 0) {
    const size_t rows = static_cast<size_t>(2) * plan->ctas * group;
    plan->ml_at = (plan->ctas * 32 + 255) / 256 * 256;
    plan->o_at = plan->ml_at + (rows * 8 + 255) / 256 * 256;
    plan->workspace = plan->o_at + rows * c->head_dim * sizeof(float);
  }
  return PKV_OK;
}

pkv_status check_workspace(const void* workspace, size_t given, size_t need) {
  if (need == 0) return PKV_OK;
  if (!workspace || given < need)
    return fail(PKV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? given : 0);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return PKV_OK;
}

bool overlap(const float* x, const float* y, size_t floats) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y), bytes = floats * sizeof(float);
  return a < b + bytes && b < a + bytes;
}

pkv_status check_table_width(int32_t max_blocks, int32_t tokens, int32_t block_size, const char* what) {
  const int64_t need = (static_cast<int64_t>(tokens) + block_size - 1) / block_size;
  if (max_blocks < need)
    return fail(PKV_ERR_INVALID_ARG, "%s %d < %lld blocks needed", what, max_blocks, static_cast<long long>(need));
  return PKV_OK;
}

// Scores that would take more go in turns of as many sequences as fit: of 65,535 sequences with
// 64 heads, one of 128 Ki tokens, they would be 2.2 TB at once, whatever the others' lengths.
// A turn costs its two kernels' latency, some 10 us (256 sequences of 200 to 400 tokens and one of
// them 128 Ki, 64/8 heads, 4-bit pool: 212 us at once in 8.6 GB, 240 us in the three turns that
// this limit makes, 302 us in nine of 1 GiB; uniform batches of 1.3 and 0.8 GB: no difference).
constexpr size_t kScoresBytes = size_t{4} << 30;

struct WeightsPlan {
  int part_tokens, max_parts;
  int seqs;  // a turn's sequences
  int64_t ld;  // of a query head's row of scores: whole 128-byte lines
  size_t ml_bytes, workspace;
};

// Partitions of the scores kernel: about six CTAs per SM (two to six are resident), of 256 to 4,096 tokens.
pkv_status plan_weights(int32_t num_seqs, int32_t num_q_heads, int32_t max_len, const pkv_cache_desc* c,
                        WeightsPlan* plan) {
  if (pkv_status st = check_cache(c, true)) return st;
  if (num_seqs < 0 || num_seqs > 65535) return fail(PKV_ERR_INVALID_ARG, "num_seqs %d outside [0, 65535]", num_seqs);
  if (num_q_heads <= 0 || num_q_heads % c->num_kv_heads)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of num_kv_heads %d", num_q_heads,
                c->num_kv_heads);
  if (num_q_heads / c->num_kv_heads > kWeightsMaxGroup)
    return fail(PKV_ERR_UNSUPPORTED, "attention weights support query-head groups <= %d (group %d)", kWeightsMaxGroup,
                num_q_heads / c->num_kv_heads);
  if (max_len < 0) return fail(PKV_ERR_INVALID_ARG, "max_context_len %d < 0", max_len);
  if (max_len > (1 << 30)) return fail(PKV_ERR_UNSUPPORTED, "max_context_len %d above 2^30", max_len);
  const int64_t work = static_cast<int64_t>(num_seqs) * c->num_kv_heads * (max_len / 2 + 1);
  const int64_t per_cta = work / (6 * 152) + 1;
  plan->part_tokens = static_cast<int>(per_cta < 256 ? 256 : per_cta > 4096 ? 4096 : (per_cta + 127) / 128 * 128);
  plan->max_parts = max_len == 0 ? 1 : (max_len + plan->part_tokens - 1) / plan->part_tokens;
  plan->ld = (static_cast<int64_t>(max_len) + 31) / 32 * 32;
  const size_t head_bytes = (plan->max_parts * 2 + plan->ld) * sizeof(float);
  const size_t fit = kScoresBytes / (head_bytes * num_q_heads);  // sequences a turn has room for
  const size_t most = fit < 1 ? 1 : fit, turns = (num_seqs + most - 1) / most;
  plan->seqs = num_seqs == 0 ? 0 : static_cast<int>((num_seqs + turns - 1) / turns);
  const size_t heads = static_cast<size_t>(plan->seqs) * num_q_heads;
  plan->ml_bytes = (heads * plan->max_parts * 2 * sizeof(float) + 255) / 256 * 256;
  plan->workspace = num_seqs == 0 || max_len == 0 ? 0 : plan->ml_bytes + heads * plan->ld * sizeof(float);
  if (max_len <= kWeightsOne) {
    plan->seqs = num_seqs;
    plan->part_tokens = max_len < 128 ? 128 : (max_len + 127) / 128 * 128;
    plan->max_parts = 1;
    plan->ld += 4;  // rows of scores in shared memory: eight tokens of four heads in different banks
    plan->workspace = 0;
  }
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status paged_kv4_append(const void* k, const void* v, int32_t kv_dtype, const int64_t* slot_mapping,
                            int32_t num_tokens, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                            void* stream) {
  if (pkv_status st = check_kv4(cache)) return st;
  if (!is_wide(kv_dtype)) return fail(PKV_ERR_UNSUPPORTED, "k/v dtype %d", kv_dtype);
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(PKV_ERR_INVALID_ARG, "k, v and the caches must be 16-byte aligned");
  int* flag = nullptr;
  if (pkv_status st = device_flag(&flag)) return st;
  Kv4AppendParams p{};
  p.k = k;
  p.v = v;
  p.slots = slot_mapping;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.err = flag;
  p.num_slots = static_cast<int64_t>(cache->num_blocks) * cache->block_size;
  p.num_tokens = num_tokens;
  p.num_kv_heads = cache->num_kv_heads;
  p.block_size = cache->block_size;
  p.head_dim = cache->head_dim;
  cudaError_t e = launch_kv4_append(p, kv_dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "4-bit append launch");
}

pkv_status paged_kv4_expand(const int64_t* src_dst_pairs, int32_t num_pairs, const void* k_cache,
                            const void* v_cache, const pkv_cache_desc* cache, void* k_out, void* v_out,
                            const pkv_cache_desc* out_cache, void* stream) {
  if (pkv_status st = check_kv4(cache)) return st;
  if (pkv_status st = check_cache(out_cache)) return st;
  if (out_cache->block_size != cache->block_size || out_cache->num_kv_heads != cache->num_kv_heads ||
      out_cache->head_dim != cache->head_dim)
    return fail(PKV_ERR_INVALID_ARG, "the pools' block_size, num_kv_heads and head_dim must be equal");
  if (num_pairs < 0) return fail(PKV_ERR_INVALID_ARG, "num_pairs %d < 0", num_pairs);
  if (num_pairs == 0) return PKV_OK;
  if (!src_dst_pairs || !k_cache || !v_cache || !k_out || !v_out)
    return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out))
    return fail(PKV_ERR_INVALID_ARG, "the pools must be 16-byte aligned");
  int* flag = nullptr;
  if (pkv_status st = device_flag(&flag)) return st;
  Kv4ExpandParams p{};
  p.pairs = src_dst_pairs;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_out = k_out;
  p.v_out = v_out;
  p.err = flag;
  p.num_pairs = num_pairs;
  p.num_blocks = cache->num_blocks;
  p.num_out_blocks = out_cache->num_blocks;
  p.num_kv_heads = cache->num_kv_heads;
  p.block_size = cache->block_size;
  p.head_dim = cache->head_dim;
  cudaError_t e = launch_kv4_expand(p, out_cache->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "4-bit expand launch");
}

size_t paged_attention_decode_kv4_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t max_context_len,
                                                  int32_t q_dtype, const pkv_cache_desc* cache) {
  Kv4Plan plan;
  if (plan_kv4(num_seqs, num_q_heads, max_context_len, q_dtype, cache, &plan) != PKV_OK) return 0;
  return plan.workspace;
}

pkv_status paged_attention_decode_kv4(const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                      int32_t max_context_len, float scale, void* out, int32_t out_dtype,
                                      void* workspace, size_t workspace_bytes, const pkv_cache_desc* cache,
                                      void* stream) {
  Kv4Plan plan;
  if (pkv_status st = plan_kv4(num_seqs, num_q_heads, max_context_len, q_dtype, cache, &plan)) return st;
  if (out_dtype != q_dtype && out_dtype != PKV_F32)
    return fail(PKV_ERR_UNSUPPORTED, "out dtype %d (must be q's dtype or f32)", out_dtype);
  if (num_seqs == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !context_lens || !out) return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (max_context_len > 0 && !block_tables) return fail(PKV_ERR_INVALID_ARG, "block_tables is NULL");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return fail(PKV_ERR_INVALID_ARG, "q, out and the caches must be 16-byte aligned");
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (pkv_status st = check_table_width(max_blocks_per_seq, max_context_len, cache->block_size, "max_blocks_per_seq"))
    return st;
  if (pkv_status st = check_workspace(workspace, workspace_bytes, plan.workspace)) return st;
  int* flag = nullptr;
  if (pkv_status st = device_flag(&flag)) return st;

  Kv4DecodeParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.out = out;
  if (plan.workspace > 0) {
    char* base = static_cast<char*>(workspace);
    p.desc = reinterpret_cast<int4*>(base);
    p.ws_ml = reinterpret_cast<float2*>(base + plan.ml_at);
    p.ws_o = reinterpret_cast<float*>(base + plan.o_at);
  }
  p.err = flag;
  p.q_dtype = q_dtype;
  p.out_dtype = out_dtype;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.group = num_q_heads / cache->num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.block_size = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.head_dim = cache->head_dim;
  p.max_len = max_context_len;
  p.ctas = plan.ctas;
  p.whole = plan.whole;
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaError_t e = launch_decode_kv4(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "4-bit decode launch");
}

size_t paged_attention_weights_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t max_context_len,
                                               const pkv_cache_desc* cache) {
  WeightsPlan plan;
  if (plan_weights(num_seqs, num_q_heads, max_context_len, cache, &plan) != PKV_OK) return 0;
  return plan.workspace;
}

pkv_status paged_attention_weights(const void* q, int32_t q_dtype, const void* k_cache, const int32_t* block_tables,
                                   int32_t max_blocks_per_seq, const int32_t* context_lens,
                                   const int32_t* tracked_lens, int32_t num_seqs, int32_t num_q_heads,
                                   int32_t max_context_len, float scale, const float* weights, float* weights_out,
                                   int64_t weights_width, void* workspace, size_t workspace_bytes,
                                   const pkv_cache_desc* cache, void* stream) {
  WeightsPlan plan;
  if (pkv_status st = plan_weights(num_seqs, num_q_heads, max_context_len, cache, &plan)) return st;
  if (!is_wide(q_dtype)) return fail(PKV_ERR_UNSUPPORTED, "q dtype %d", q_dtype);
  if (cache->dtype != PKV_KV4 && q_dtype != cache->dtype)
    return fail(PKV_ERR_INVALID_ARG, "q dtype %d differs from the cache's %d", q_dtype, cache->dtype);
  if (num_seqs == 0 || max_context_len == 0) return PKV_OK;
  if (!q || !k_cache || !block_tables || !context_lens || !weights || !weights_out)
    return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(k_cache)) return fail(PKV_ERR_INVALID_ARG, "q and the cache must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(weights_out)) & 3u)
    return fail(PKV_ERR_INVALID_ARG, "weights must be 4-byte aligned");
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (weights_width < max_context_len)
    return fail(PKV_ERR_INVALID_ARG, "weights_width %lld < max_context_len %d", static_cast<long long>(weights_width),
                max_context_len);
  if (weights != weights_out &&
      overlap(weights, weights_out, static_cast<size_t>(num_seqs) * cache->num_kv_heads * weights_width))
    return fail(PKV_ERR_INVALID_ARG, "weights_out overlaps weights without being it");
  if (pkv_status st = check_table_width(max_blocks_per_seq, max_context_len, cache->block_size, "max_blocks_per_seq"))
    return st;
  if (pkv_status st = check_workspace(workspace, workspace_bytes, plan.workspace)) return st;
  int* flag = nullptr;
  if (pkv_status st = device_flag(&flag)) return st;
  WeightsParams p{};
  p.k_cache = k_cache;
  if (plan.workspace > 0) {
    p.ws_ml = static_cast<float*>(workspace);
    p.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.ml_bytes);
  }
  p.err = flag;
  p.width = weights_width;
  p.scores_ld = plan.ld;
  p.q_dtype = q_dtype;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.group = num_q_heads / cache->num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.block_size = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.head_dim = cache->head_dim;
  p.max_len = max_context_len;
  p.part_tokens = plan.part_tokens;
  p.max_parts = plan.max_parts;
  p.scale_log2 = scale * 1.4426950408889634f;
  for (int32_t s = 0; s < num_seqs; s += plan.seqs) {  // turns follow each other in the workspace
    p.num_seqs = num_seqs - s < plan.seqs ? num_seqs - s : plan.seqs;
    p.q = static_cast<const char*>(q) + static_cast<size_t>(s) * num_q_heads * cache->head_dim * elem_bytes(q_dtype);
    p.block_tables = block_tables + static_cast<size_t>(s) * max_blocks_per_seq;
    p.context_lens = context_lens + s;
    p.tracked_lens = tracked_lens ? tracked_lens + s : nullptr;
    const size_t row = static_cast<size_t>(s) * cache->num_kv_heads * weights_width;
    p.weights = weights + row;
    p.weights_out = weights_out + row;
    const cudaError_t e = launch_weights(p, cache->dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attention weights launch");
  }
  return PKV_OK;
}

pkv_status paged_kv_evict(const float* weights, float* weights_out, int64_t weights_width, const int32_t* block_tables,
                          int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* keep_lens,
                          int32_t recent, const int32_t* new_tables, int32_t max_new_blocks, int32_t num_seqs,
                          int32_t max_context_len, int32_t max_keep, int32_t* kept, void* k_cache, void* v_cache,
                          const pkv_cache_desc* cache, void* stream) {
  if (pkv_status st = check_cache(cache, true)) return st;
  if (num_seqs < 0 || num_seqs > 65535) return fail(PKV_ERR_INVALID_ARG, "num_seqs %d outside [0, 65535]", num_seqs);
  if (max_context_len < 0 || max_keep < 0 || recent < 0)
    return fail(PKV_ERR_INVALID_ARG, "max_context_len %d, max_keep %d, recent %d: none may be negative", max_context_len,
                max_keep, recent);
  if (max_context_len > (1 << 30)) return fail(PKV_ERR_UNSUPPORTED, "max_context_len %d above 2^30", max_context_len);
  if (num_seqs == 0 || max_context_len == 0) return PKV_OK;
  if (!weights || !weights_out || !block_tables || !context_lens || !keep_lens || !k_cache || !v_cache ||
      (max_keep > 0 && (!new_tables || !kept)))
    return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(PKV_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  if (weights_width < max_context_len)
    return fail(PKV_ERR_INVALID_ARG, "weights_width %lld < max_context_len %d", static_cast<long long>(weights_width),
                max_context_len);
  if ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(weights_out)) & 3u)
    return fail(PKV_ERR_INVALID_ARG, "weights must be 4-byte aligned");
  if (overlap(weights, weights_out, static_cast<size_t>(num_seqs) * cache->num_kv_heads * weights_width))
    return fail(PKV_ERR_INVALID_ARG, "weights_out overlaps weights");
  if (pkv_status st = check_table_width(max_blocks_per_seq, max_context_len, cache->block_size, "max_blocks_per_seq"))
    return st;
  const int32_t most = max_keep < max_context_len ? max_keep : max_context_len;  // rows a sequence may keep
  if (pkv_status st = check_table_width(max_new_blocks, most, cache->block_size, "max_new_blocks")) return st;
  int* flag = nullptr;
  if (pkv_status st = device_flag(&flag)) return st;
  EvictParams p{};
  p.weights = weights;
  p.weights_out = weights_out;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.keep_lens = keep_lens;
  p.new_tables = new_tables;
  p.kept = kept;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.err = flag;
  p.width = weights_width;
  p.num_seqs = num_seqs;
  p.num_kv_heads = cache->num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_new_blocks = max_new_blocks;
  p.block_size = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.row_bytes = static_cast<int32_t>(row_bytes(cache));
  p.max_len = max_context_len;
  p.max_keep = max_keep;
  p.recent = recent;
  cudaError_t e = launch_evict(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "evict launch");
}

}  // extern "C"
