// kv4_ops.cu -- data movement of the 4-bit K/V cache (format: kv4.cuh):
//  * append: round each new token's K/V rows to 4 bits and write them into their slots;
//  * expand: widen whole 4-bit blocks into blocks of an f32/f16/bf16 pool.
// Both are bound by HBM: append reads D * e and writes 5 D / 8 bytes per row, expand the
// reverse.
#include "kv4.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += Elem<T>::kVec) Elem<T>::load16(p + i, x + i);
}

// One thread per eight values of one (token, KV head) row, of K and of V; four
// neighbouring lanes share a group's minimum and maximum.  The thread count is a
// multiple of 32 and whole warps take whole groups, so the shuffles see full warps: a
// thread past the end or with a padding slot computes on zeros and stores nothing.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const __grid_constant__ Kv4AppendParams p) {
  grid_dependents_launch();  // a following decode's work may start; it waits for this grid before reading
  const int per_row = p.head_dim / 8;
  const int64_t per_token = static_cast<int64_t>(p.num_kv_heads) * per_row;
  const int64_t total = per_token * p.num_tokens;
  const int row_bytes = p.head_dim * 5 / 8;
  const int64_t first = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
  for (int64_t i = first; i - (threadIdx.x & 31) < total; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    float k[8], v[8];
    unsigned char* dst_k = nullptr;
    unsigned char* dst_v = nullptr;
    int c = 0;
    if (i < total) {
      const int64_t t = i / per_token;
      const int rem = static_cast<int>(i - t * per_token);
      const int h = rem / per_row;
      c = rem - h * per_row;
      load8(static_cast<const T*>(p.k) + i * 8, k);
      load8(static_cast<const T*>(p.v) + i * 8, v);
      const int64_t slot = p.slots[t];
      if (slot >= p.num_slots) {
        set_error(p.err, kErrIndex);
      } else if (slot >= 0) {
        const int64_t b = slot / p.block_size;
        const int64_t row = (b * p.num_kv_heads + h) * p.block_size + (slot - b * p.block_size);
        dst_k = static_cast<unsigned char*>(p.k_cache) + row * row_bytes;
        dst_v = static_cast<unsigned char*>(p.v_cache) + row * row_bytes;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = v[e] = 0.f;
    }
    __half2 pk, pv;
    const uint32_t wk = kv4_quantise8(k, &pk), wv = kv4_quantise8(v, &pv);
    if (dst_k) {
      reinterpret_cast<uint32_t*>(dst_k)[c] = wk;
      reinterpret_cast<uint32_t*>(dst_v)[c] = wv;
      if ((c & 3) == 0) {
        const int at = p.head_dim / 8 + c / 4;  // in words: the pairs follow the codes
        reinterpret_cast<uint32_t*>(dst_k)[at] = as_u32(pk);
        reinterpret_cast<uint32_t*>(dst_v)[at] = as_u32(pv);
      }
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
  const int words = p.head_dim / 8, row_words = words * 5 / 4;
  const int rows = p.num_kv_heads * p.block_size, total = rows * words;  // of one block
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.pairs_per_cta;
  const int items = static_cast<int>(min(static_cast<int64_t>(p.pairs_per_cta), p.num_pairs - first)) * total;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < items; i += gridDim.y * kThreads) {
    const int which = i / total, rem = i - which * total;
    const int64_t src = p.pairs[2 * (first + which)], dst = p.pairs[2 * (first + which) + 1];
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_out_blocks) {
      set_error(p.err, kErrIndex);
      continue;
    }
    const int row = rem / words, c = rem - row * words;
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

int grid_for(int64_t work, int cap) {
  const int64_t g = (work + kThreads - 1) / kThreads;
  return static_cast<int>(g < 1 ? 1 : (g > cap ? cap : g));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams& p, int dtype, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const int64_t work = static_cast<int64_t>(p.num_tokens) * p.num_kv_heads * (p.head_dim / 8);
  const int grid = grid_for(work, 152 * 16);
  switch (dtype) {
    case PKV_F32: kv4_append_kernel<float><<<grid, kThreads, 0, stream>>>(p); break;
    case PKV_F16: kv4_append_kernel<__half><<<grid, kThreads, 0, stream>>>(p); break;
    default: kv4_append_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_expand(Kv4ExpandParams p, int dtype, cudaStream_t stream) {
  if (p.num_pairs == 0) return cudaSuccess;
  constexpr int kPerCta = 4 * kThreads;  // words a CTA takes: four rounds of its threads
  const int total = p.num_kv_heads * p.block_size * (p.head_dim / 8);
  p.pairs_per_cta = total >= kPerCta ? 1 : kPerCta / total;
  const dim3 grid((p.num_pairs + p.pairs_per_cta - 1) / p.pairs_per_cta, total > kPerCta ? (total + kPerCta - 1) / kPerCta : 1);
  switch (dtype) {
    case PKV_F32: kv4_expand_kernel<float><<<grid, kThreads, 0, stream>>>(p); break;
    case PKV_F16: kv4_expand_kernel<__half><<<grid, kThreads, 0, stream>>>(p); break;
    default: kv4_expand_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace pkv
