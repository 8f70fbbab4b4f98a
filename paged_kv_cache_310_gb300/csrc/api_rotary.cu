// api_rotary.cu -- the extern "C" entry points of norms and position rotation (declared in
// include/pagedkv.h): argument checks, launches, and the frequencies of scaled rotations.
#include <cmath>

#include "api_util.h"
#include "launch.h"

using namespace pkv;

namespace {

// A call's rows of one tensor: `tokens` rows of `len` elements, `stride` apart.
struct Rows {
  const char* what;
  const void* base;
  int64_t stride, len;
};

// Whether two sets of rows share memory.  With one stride the rows are columns of one table,
// which may lie beside each other (the parts of a fused projection); with two, sets whose
// ranges meet count as sharing.
bool overlap(const Rows& a, const Rows& b, int64_t tokens, int64_t size) {
  const int64_t a0 = reinterpret_cast<intptr_t>(a.base), b0 = reinterpret_cast<intptr_t>(b.base);
  const int64_t a1 = a0 + ((tokens - 1) * a.stride + a.len) * size, b1 = b0 + ((tokens - 1) * b.stride + b.len) * size;
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.stride != b.stride || tokens == 1) return true;
  const int64_t s = a.stride * size, d = ((b0 - a0) % s + s) % s;
  return d < a.len * size || d + b.len * size > s;
}

pkv_status check_rows(const Rows& r, int64_t tokens, int64_t size) {
  if (!r.base) return fail(PKV_ERR_INVALID_ARG, "%s is NULL", r.what);
  if (!aligned16(r.base)) return fail(PKV_ERR_INVALID_ARG, "%s must be 16-byte aligned", r.what);
  if (tokens > 1 && (r.stride < r.len || r.stride * size % 16 || r.stride > (int64_t{1} << 28)))
    return fail(PKV_ERR_INVALID_ARG, "%s: token stride %lld (at least %lld elements, a multiple of 16 bytes, at most 2^28)", r.what,
                static_cast<long long>(r.stride), static_cast<long long>(r.len));
  return PKV_OK;
}

// What both calls ask of the rotation, the sizes and the queries; fills those parameters in.
pkv_status check_rotary(const pkv_rotary* rot, int32_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                        RotaryParams* p) {
  if (!rot) return fail(PKV_ERR_INVALID_ARG, "rotary is NULL");
  if (tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens %d < 0", tokens);
  if (q_heads < 0 || q_heads > 65535 || kv_heads < 0 || kv_heads > 65535)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d, num_kv_heads %d outside [0, 65535]", q_heads, kv_heads);
  if (rot->rotary_dim < 0 || rot->rotary_dim > head_dim || rot->rotary_dim % 16)
    return fail(PKV_ERR_UNSUPPORTED, "rotary_dim %d (a multiple of 16 up to head_dim %d)", rot->rotary_dim, head_dim);
  if (rot->layout != PKV_ROTARY_HALF && rot->layout != PKV_ROTARY_INTERLEAVED)
    return fail(PKV_ERR_INVALID_ARG, "rotary layout %d", rot->layout);
  if (!std::isfinite(rot->factor)) return fail(PKV_ERR_INVALID_ARG, "rotary factor is not finite");
  if ((rot->q_weight || rot->k_weight) && !(rot->eps >= 0.f && std::isfinite(rot->eps)))
    return fail(PKV_ERR_INVALID_ARG, "eps is negative or not finite");
  if (!aligned16(rot->q_weight) || !aligned16(rot->k_weight))
    return fail(PKV_ERR_INVALID_ARG, "the norm weights must be 16-byte aligned");
  if (rot->rotary_dim > 0 && !rot->inv_freq && tokens > 0) return fail(PKV_ERR_INVALID_ARG, "inv_freq is NULL");
  if (reinterpret_cast<uintptr_t>(rot->inv_freq) & 7u) return fail(PKV_ERR_INVALID_ARG, "inv_freq must be 8-byte aligned");
  p->inv_freq = rot->inv_freq;
  p->q_weight = rot->q_weight;
  p->k_weight = rot->k_weight;
  p->num_tokens = tokens;
  p->num_q_heads = q_heads;
  p->num_kv_heads = kv_heads;
  p->head_dim = head_dim;
  p->rotary_dim = rot->rotary_dim;
  p->interleaved = rot->layout == PKV_ROTARY_INTERLEAVED;
  p->factor = rot->factor;
  p->eps = rot->eps;
  return PKV_OK;
}

pkv_status check_apart(const Rows& out, const Rows& in, int64_t tokens, int64_t size, bool in_place) {
  if (in_place && out.base == in.base && (tokens == 1 || out.stride == in.stride)) return PKV_OK;
  if (overlap(out, in, tokens, size)) return fail(PKV_ERR_INVALID_ARG, "%s overlaps %s", out.what, in.what);
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status paged_kv_append_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                                  int32_t num_tokens, int32_t num_q_heads, const pkv_rotary* rotary, void* q_out,
                                  int64_t q_out_stride, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                                  void* stream) {
  if (pkv_status st = check_cache(cache)) return st;
  RotaryParams p{};
  if (pkv_status st = check_rotary(rotary, num_tokens, num_q_heads, cache->num_kv_heads, cache->head_dim, &p)) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!positions || !slot_mapping || !k_cache || !v_cache) return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(PKV_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  const int64_t size = elem_bytes(cache->dtype), d = cache->head_dim;
  const Rows rq{"q", q, q_stride, num_q_heads * d}, rk{"k", k, k_stride, cache->num_kv_heads * d};
  const Rows rv{"v", v, v_stride, cache->num_kv_heads * d}, ro{"q_out", q_out, q_out_stride, num_q_heads * d};
  if (pkv_status st = check_rows(rk, num_tokens, size)) return st;
  if (pkv_status st = check_rows(rv, num_tokens, size)) return st;
  if (num_q_heads > 0) {
    if (pkv_status st = check_rows(rq, num_tokens, size)) return st;
    if (pkv_status st = check_rows(ro, num_tokens, size)) return st;
    if (pkv_status st = check_apart(ro, rq, num_tokens, size, true)) return st;
    if (pkv_status st = check_apart(ro, rk, num_tokens, size, false)) return st;
    if (pkv_status st = check_apart(ro, rv, num_tokens, size, false)) return st;
  }
  if (pkv_status st = device_flag(&p.err)) return st;
  p.q = q;
  p.k = k;
  p.v = v;
  p.positions = positions;
  p.slots = slot_mapping;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.num_slots = static_cast<int64_t>(cache->num_blocks) * cache->block_size;
  p.block_size = cache->block_size;
  cudaError_t e = launch_rotary(p, cache->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "rotary append launch");
}

pkv_status paged_qk_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
                           int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                           const pkv_rotary* rotary, void* q_out, int64_t q_out_stride, void* k_out,
                           int64_t k_out_stride, void* stream) {
  if (dtype < PKV_F32 || dtype > PKV_BF16) return fail(PKV_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (head_dim != 64 && head_dim != 128) return fail(PKV_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  RotaryParams p{};
  if (pkv_status st = check_rotary(rotary, num_tokens, num_q_heads, num_kv_heads, head_dim, &p)) return st;
  if (num_tokens == 0 || num_q_heads + num_kv_heads == 0) return PKV_OK;
  if (!positions) return fail(PKV_ERR_INVALID_ARG, "positions is NULL");
  const int64_t size = elem_bytes(dtype), d = head_dim;
  const Rows rq{"q", q, q_stride, num_q_heads * d}, rk{"k", k, k_stride, num_kv_heads * d};
  const Rows qo{"q_out", q_out, q_out_stride, num_q_heads * d}, ko{"k_out", k_out, k_out_stride, num_kv_heads * d};
  if (num_q_heads > 0) {
    if (pkv_status st = check_rows(rq, num_tokens, size)) return st;
    if (pkv_status st = check_rows(qo, num_tokens, size)) return st;
    if (pkv_status st = check_apart(qo, rq, num_tokens, size, true)) return st;
  }
  if (num_kv_heads > 0) {
    if (pkv_status st = check_rows(rk, num_tokens, size)) return st;
    if (pkv_status st = check_rows(ko, num_tokens, size)) return st;
    if (pkv_status st = check_apart(ko, rk, num_tokens, size, true)) return st;
  }
  if (num_q_heads > 0 && num_kv_heads > 0) {
    if (pkv_status st = check_apart(qo, rk, num_tokens, size, false)) return st;
    if (pkv_status st = check_apart(ko, rq, num_tokens, size, false)) return st;
    if (pkv_status st = check_apart(qo, ko, num_tokens, size, false)) return st;
  }
  if (pkv_status st = device_flag(&p.err)) return st;
  p.q = q;
  p.k = k;
  p.positions = positions;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  cudaError_t e = launch_rotary(p, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "rotary launch");
}

pkv_status paged_rotary_frequencies(double* inv_freq, int32_t rotary_dim, double base, const pkv_rotary_scaling* scaling,
                                    float* factor) {
  if (!inv_freq || !factor) return fail(PKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (rotary_dim <= 0 || rotary_dim % 2) return fail(PKV_ERR_INVALID_ARG, "rotary_dim %d is not even and positive", rotary_dim);
  if (!(base > 1.) || !std::isfinite(base)) return fail(PKV_ERR_INVALID_ARG, "base %g: finite and above 1 needed", base);
  const int rule = scaling ? scaling->rule : PKV_ROTARY_UNSCALED;
  if (rule < PKV_ROTARY_UNSCALED || rule > PKV_ROTARY_PARTS) return fail(PKV_ERR_INVALID_ARG, "scaling rule %d", rule);
  const double by = rule == PKV_ROTARY_UNSCALED ? 1. : scaling->factor;
  if (!(by >= 1.) || !std::isfinite(by)) return fail(PKV_ERR_INVALID_ARG, "scaling factor %g: finite and at least 1 needed", by);
  if (rule == PKV_ROTARY_BASE) {
    if (rotary_dim == 2) return fail(PKV_ERR_INVALID_ARG, "a base cannot scale the one frequency of rotary_dim 2");
    base *= std::pow(by, rotary_dim / (rotary_dim - 2.));
    if (!std::isfinite(base)) return fail(PKV_ERR_INVALID_ARG, "the base scaled by a factor of %g is not finite", by);
  }
  if (rule == PKV_ROTARY_PARTS &&
      !(scaling->original_len > 0. && std::isfinite(scaling->original_len) && scaling->slow_turns >= 0. &&
        scaling->fast_turns > scaling->slow_turns && std::isfinite(scaling->fast_turns)))
    return fail(PKV_ERR_INVALID_ARG, "scaling by parts needs original_len > 0 and fast_turns > slow_turns >= 0");
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2. * i / rotary_dim);
    if (rule == PKV_ROTARY_LINEAR) f /= by;
    if (rule == PKV_ROTARY_PARTS) {
      const double turns = scaling->original_len * f / 6.283185307179586477;
      double keep = (turns - scaling->slow_turns) / (scaling->fast_turns - scaling->slow_turns);
      keep = keep < 0. ? 0. : keep > 1. ? 1. : keep;
      f = f / by * (1. - keep) + f * keep;
    }
    inv_freq[i] = f;
  }
  *factor = rule == PKV_ROTARY_PARTS ? static_cast<float>(0.1 * std::log(by) + 1.) : 1.f;
  return PKV_OK;
}

}  // extern "C"
