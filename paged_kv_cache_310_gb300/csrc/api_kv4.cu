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

}  // extern "C"
