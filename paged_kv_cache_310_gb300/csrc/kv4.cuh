// kv4.cuh -- the 4-bit row format (PKV_KV4) on the device.
//
// A row holds D values in 5 D / 8 bytes: D/2 bytes of codes (byte i: value 2i in the low
// half, 2i + 1 in the high half; as a little-endian 32-bit word, half-byte i of word w is
// value 8w + i), then D/32 pairs (step, lo) of fp16, one for each group of 32 values.  A
// code c stands for fp16(lo + c * step), ONE rounding: exactly what a half-precision fused
// multiply-add of the exact integer c gives.  So a stored value is a fixed fp16 number,
// every kernel that widens a row agrees bit for bit, and fp16 tensor-core products of it
// are exact.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pkv {

constexpr int kKv4Group = 32;  // values that share one (step, lo) pair
// Values beyond this are stored as this: with the roundings of lo (at most 16) and of
// step (at most 4, times 15) lo + 15 step stays below the 65,520 that rounds to infinity.
constexpr float kKv4Largest = 65408.f;

template <int D>
struct Kv4Row {
  static constexpr int kBytes = D * 5 / 8;
  static constexpr int kCodes = D / 2;  // bytes of codes; the (step, lo) pairs follow
};

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(bits));
  return d;
}

// The exact integers of half-bytes 0 and 4 (bits 0-3 and 16-19) of w as fp16.
__device__ __forceinline__ __half2 low_codes(uint32_t w, const Kv4Bits& k) {
  return __hsub2(as_half2(and_or(w, k.low, k.one)), as_half2(0x64006400u));
}
// ... of half-bytes 1 and 5 (bits 4-7 and 20-23): 1024 + 16 c, times 1/16, minus 64 (exact).
__device__ __forceinline__ __half2 high_codes(uint32_t w, const Kv4Bits& k) {
  return __hfma2(as_half2(and_or(w, k.high, k.one)), as_half2(0x2c002c00u), as_half2(0xd400d400u));
}

// The eight values of a word of codes: out[i] = (value i, value i + 4).
__device__ __forceinline__ void kv4_word(uint32_t w, __half2 step, __half2 lo, const Kv4Bits& k, uint32_t (&out)[4]) {
  out[0] = as_u32(__hfma2(low_codes(w, k), step, lo));
  out[1] = as_u32(__hfma2(high_codes(w, k), step, lo));
  w >>= 8;
  out[2] = as_u32(__hfma2(low_codes(w, k), step, lo));
  out[3] = as_u32(__hfma2(high_codes(w, k), step, lo));
}

// Eight values of one group, held by four neighbouring lanes with eight each: returns the
// lane's word of codes and the group's (step, lo) pair.
//   lo = fp16(min), step = fp16(fp32(max(0, max - lo) / 15)), each operation rounded once;
//   code = the integer nearest to fp32(x - lo) / step (exact quotient, ties to even),
//   held within 0..15; step 0 gives code 0.  A NaN or infinity makes step = lo = NaN.
// The quotient's integer comes from a product with 1/step, off by at most one near a tie,
// and is settled by the remainder d - c step, which one fma gives exactly (c step has at
// most 15 bits, and the remainder no more than d or step): no division, no fp64.
__device__ __forceinline__ uint32_t kv4_quantise8(float (&x)[8], __half2* pair) {
  float mn = INFINITY, mx = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bad |= !(fabsf(x[i]) < INFINITY);
    x[i] = fminf(fmaxf(x[i], -kKv4Largest), kKv4Largest);
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
  }
  uint32_t any_bad = bad;
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    any_bad |= __shfl_xor_sync(0xffffffffu, any_bad, off);
  }
  if (any_bad) {
    *pair = as_half2(0x7e007e00u);
    return 0u;
  }
  const __half lo16 = __float2half_rn(mn + 0.f);  // -0 becomes +0
  const float lo = __half2float(lo16);
  const __half step16 = __float2half_rn(__fdiv_rn(fmaxf(0.f, mx - lo), 15.f));
  const float step = __half2float(step16);
  *pair = __halves2half2(step16, lo16);
  if (step == 0.f) return 0u;
  const float inverse = __frcp_rn(step);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = x[i] - lo;
    float c = fminf(fmaxf(rintf(d * inverse), 0.f), 15.f);
    const float r2 = 2.f * fmaf(-c, step, d);
    const bool odd = static_cast<int>(c) & 1;
    if (r2 > step || (r2 == step && odd)) c += 1.f;
    if (r2 < -step || (r2 == -step && odd)) c -= 1.f;
    c = fminf(fmaxf(c, 0.f), 15.f);
    word |= static_cast<uint32_t>(c) << (4 * i);
  }
  return word;
}

}  // namespace pkv
