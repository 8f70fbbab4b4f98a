// kv4_ops.cu -- data movement of the 4-bit K/V cache (format: kv4.cuh):
//  * append: round each new token's K/V rows to 4 bits and write them into their slots;
//  * expand: widen whole 4-bit blocks into blocks of an f32/f16/bf16 pool.
// Append reads D * e and writes 5 D / 8 bytes per row, expand the reverse.  Expand is bound by
// HBM (16,384 blocks of 16 tokens, 8 heads, D 128, to bf16: 217 us, 6.5 TB/s, 0.96 of copy
// bandwidth).  A large append is bound by the instructions of the rounding, 25 a value: while it
// runs, 70 % of the issue slots are taken and HBM is at 22 % (8,191 tokens of 8 heads: f16 16.7 us,
// 0.39 of copy bandwidth, bf16 19.1, f32, twice the bytes, 15.5 and 0.74).  A small one is bound
// by its launch.
#include "kv4.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Raw8 {
  static constexpr int kVecs = static_cast<int>(8 * sizeof(T) / 16);
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; i += Elem<T>::kVec) Elem<T>::load16(&v[i / Elem<T>::kVec], x + i);
  }
};

// One thread per eight values of one (token, KV head) row, of K and of V; four
// neighbouring lanes share a group's minimum and maximum.  blockIdx.x takes
// tokens_per_cta tokens (several when a token has few values), blockIdx.y a part of a
// token's (when it has many).  Threads past the end or with a padding slot work on what
// they have and store nothing, so the shuffles always see whole warps.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const __grid_constant__ Kv4AppendParams p) {
  grid_dependency_wait();    // of the kernel before: only this one's launch overlaps it
  grid_dependents_launch();  // the next kernel's launch may overlap this one; it waits before it writes
  const int row_log2 = p.head_dim == 128 ? 4 : 3;  // threads per row
  const int per_token = p.num_kv_heads << row_log2;
  const int x = blockIdx.y * kThreads + threadIdx.x;
  const int in_cta = x / per_token, rem = x - in_cta * per_token;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * p.tokens_per_cta + in_cta;
  const int h = rem >> row_log2, c = rem & ((1 << row_log2) - 1);
  const bool have = in_cta < p.tokens_per_cta && t < p.num_tokens;
  Raw8<T> rk, rv;
  int64_t slot = -1;
  if (have) {
    const int64_t at = (t * per_token + rem) * 8;
    rk.load(static_cast<const T*>(p.k) + at);
    rv.load(static_cast<const T*>(p.v) + at);
    slot = p.slots[t];
  } else {
    rk.zero();
    rv.zero();
  }
  float xs[8];
  __half2 pk, pv;
  rk.widen(xs);
  const uint32_t wk = kv4_quantise8<T>(rk.v, xs, &pk);
  rv.widen(xs);
  const uint32_t wv = kv4_quantise8<T>(rv.v, xs, &pv);
  if (slot >= p.num_slots) {
    set_error(p.err, kErrIndex);
  } else if (slot >= 0) {
    const int bs_log2 = 31 - __clz(p.block_size);
    const int64_t row = ((slot >> bs_log2) * p.num_kv_heads + h) * p.block_size + (slot & (p.block_size - 1));
    const int words = p.head_dim * 5 / 32;  // 32-bit words of a row
    uint32_t* dst_k = static_cast<uint32_t*>(p.k_cache) + row * words;
    uint32_t* dst_v = static_cast<uint32_t*>(p.v_cache) + row * words;
    dst_k[c] = wk;
    dst_v[c] = wv;
    if ((c & 3) == 0) {
      const int at = p.head_dim / 8 + c / 4;  // the pairs follow the codes
      dst_k[at] = as_u32(pk);
      dst_v[at] = as_u32(pv);
    }
  }
}

// Stores eight fp16 values, given as (i, i + 4) pairs, in order and in type T.
__device__ __forceinline__ void store8(__half* out, const uint32_t (&v)[4]) {
  uint4 o;
  o.x = __byte_perm(v[0], v[1], 0x5410);
  o.y = __byte_perm(v[2], v[3], 0x5410);
  o.z = __byte_perm(v[0], v[1], 0x7632);
  o.w = __byte_perm(v[2], v[3], 0x7632);
  *reinterpret_cast<uint4*>(out) = o;
}
__device__ __forceinline__ void store8(float* out, const uint32_t (&v)[4]) {
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __half22float2(as_half2(v[i]));
  reinterpret_cast<float4*>(out)[0] = make_float4(f[0].x, f[1].x, f[2].x, f[3].x);
  reinterpret_cast<float4*>(out)[1] = make_float4(f[0].y, f[1].y, f[2].y, f[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16* out, const uint32_t (&v)[4]) {
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __half22float2(as_half2(v[i]));
  uint4 o;
  __nv_bfloat162 b[4] = {__floats2bfloat162_rn(f[0].x, f[1].x), __floats2bfloat162_rn(f[2].x, f[3].x),
                         __floats2bfloat162_rn(f[0].y, f[1].y), __floats2bfloat162_rn(f[2].y, f[3].y)};
  o.x = *reinterpret_cast<uint32_t*>(&b[0]);
  o.y = *reinterpret_cast<uint32_t*>(&b[1]);
  o.z = *reinterpret_cast<uint32_t*>(&b[2]);
  o.w = *reinterpret_cast<uint32_t*>(&b[3]);
  *reinterpret_cast<uint4*>(out) = o;
}

// One thread per word of codes (eight values) of K and of V.  A CTA along x takes
// pairs_per_cta pairs (several when blocks are small), the CTAs along y share a block.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_expand_kernel(const __grid_constant__ Kv4ExpandParams p) {
  grid_dependency_wait();    // of the kernel before: only this one's launch overlaps it
  grid_dependents_launch();  // the next kernel's launch may overlap this one; it waits before it writes
  const int words_log2 = p.head_dim == 128 ? 4 : 3, words = 1 << words_log2, row_words = words * 5 / 4;
  const int rows = p.num_kv_heads * p.block_size, total = rows * words;  // of one block
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.pairs_per_cta;
  const int items = static_cast<int>(min(static_cast<int64_t>(p.pairs_per_cta), p.num_pairs - first)) * total;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < items; i += gridDim.y * kThreads) {
    const int which = p.pairs_per_cta == 1 ? 0 : i / total, rem = i - which * total;
    const int64_t src = p.pairs[2 * (first + which)], dst = p.pairs[2 * (first + which) + 1];
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_out_blocks) {
      set_error(p.err, kErrIndex);
      continue;
    }
    const int row = rem >> words_log2, c = rem & (words - 1);
    const int64_t base = src * rows * row_words;
    const int64_t at = base + row * row_words + c, pair = base + row * row_words + words + c / 4;
    const uint32_t wk = static_cast<const uint32_t*>(p.k_cache)[at], wv = static_cast<const uint32_t*>(p.v_cache)[at];
    const __half2 pk = as_half2(static_cast<const uint32_t*>(p.k_cache)[pair]);
    const __half2 pv = as_half2(static_cast<const uint32_t*>(p.v_cache)[pair]);
    const int64_t to = (dst * rows + row) * p.head_dim + c * 8;
    uint32_t out[4];
    kv4_word(wk, __low2half2(pk), __high2half2(pk), p.bits, out);
    store8(static_cast<T*>(p.k_out) + to, out);
    kv4_word(wv, __low2half2(pv), __high2half2(pv), p.bits, out);
    store8(static_cast<T*>(p.v_out) + to, out);
  }
}

}  // namespace

cudaError_t launch_kv4_append(Kv4AppendParams p, int dtype, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const int per_token = p.num_kv_heads * (p.head_dim / 8);
  p.tokens_per_cta = per_token >= kThreads ? 1 : kThreads / per_token;
  const dim3 grid((p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta,
                  per_token > kThreads ? (per_token + kThreads - 1) / kThreads : 1);
  switch (dtype) {
    case PKV_F32: return launch_dependent(kv4_append_kernel<float>, grid, kThreads, 0, stream, p);
    case PKV_F16: return launch_dependent(kv4_append_kernel<__half>, grid, kThreads, 0, stream, p);
    default: return launch_dependent(kv4_append_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, p);
  }
}

cudaError_t launch_kv4_expand(Kv4ExpandParams p, int dtype, cudaStream_t stream) {
  if (p.num_pairs == 0) return cudaSuccess;
  constexpr int kPerCta = 4 * kThreads;  // words a CTA takes: four rounds of its threads
  const int total = p.num_kv_heads * p.block_size * (p.head_dim / 8);
  p.pairs_per_cta = total >= kPerCta ? 1 : kPerCta / total;
  const int parts = total > kPerCta ? (total + kPerCta - 1) / kPerCta : 1;  // CTAs that share a block
  const dim3 grid((p.num_pairs + p.pairs_per_cta - 1) / p.pairs_per_cta, parts < 1024 ? parts : 1024);
  switch (dtype) {
    case PKV_F32: return launch_dependent(kv4_expand_kernel<float>, grid, kThreads, 0, stream, p);
    case PKV_F16: return launch_dependent(kv4_expand_kernel<__half>, grid, kThreads, 0, stream, p);
    default: return launch_dependent(kv4_expand_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, p);
  }
}

}  // namespace pkv
