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

// ---- rounding to 4 bits
// Eight values of one group, held by four neighbouring lanes with eight each, become the
// lane's word of codes and the group's (step, lo) pair:
//   lo = fp16(min), step = fp16(fp32(max(0, max - lo) / 15)), each operation rounded once;
//   code = the integer nearest to fp32(x - lo) / step (exact quotient, ties to even),
//   held within 0..15; step 0 gives code 0.  A NaN or infinity makes step = lo = NaN.

// Minimum, maximum and a NaN-or-infinity mark (not 0) of a lane's eight values.
template <typename T>
__device__ __forceinline__ void kv4_stats(const uint4* raw, const float (&x)[8], float* mn, float* mx, float* mark) {
  *mn = *mx = x[0];
  *mark = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    *mn = fminf(*mn, x[i]);
    *mx = fmaxf(*mx, x[i]);
    *mark = fmaf(x[i], 0.f, *mark);
  }
}
// 16-bit values two at a time: their minimum and maximum are exact.
template <typename H2, typename ToFloat2>
__device__ __forceinline__ void kv4_stats_pairs(const uint4& raw, float* mn, float* mx, float* mark, H2 zero, ToFloat2 widen) {
  const H2* h = reinterpret_cast<const H2*>(&raw);
  H2 lo = h[0], hi = h[0], nan = __hfma2(h[0], zero, zero);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    lo = __hmin2(lo, h[i]);
    hi = __hmax2(hi, h[i]);
    nan = __hfma2(h[i], zero, nan);
  }
  const float2 a = widen(lo), b = widen(hi), c = widen(nan);
  *mn = fminf(a.x, a.y);
  *mx = fmaxf(b.x, b.y);
  *mark = c.x + c.y;
}
template <>
__device__ __forceinline__ void kv4_stats<__half>(const uint4* raw, const float (&)[8], float* mn, float* mx, float* mark) {
  kv4_stats_pairs<__half2>(*raw, mn, mx, mark, __half2half2(__ushort_as_half(0)), [](__half2 v) { return __half22float2(v); });
}
template <>
__device__ __forceinline__ void kv4_stats<__nv_bfloat16>(const uint4* raw, const float (&)[8], float* mn, float* mx,
                                                         float* mark) {
  kv4_stats_pairs<__nv_bfloat162>(*raw, mn, mx, mark, __bfloat162bfloat162(__ushort_as_bfloat16(0)),
                                  [](__nv_bfloat162 v) { return __bfloat1622float2(v); });
}

// raw: the eight values in T (one uint4, or two for f32); x: the same as floats.
template <typename T>
__device__ __forceinline__ uint32_t kv4_quantise8(const uint4* raw, float (&x)[8], __half2* pair) {
  float mn, mx, mark;
  kv4_stats<T>(raw, x, &mn, &mx, &mark);
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    mark += __shfl_xor_sync(0xffffffffu, mark, off);
  }
  if (!(mark == 0.f)) {  // 0 * infinity and 0 * NaN are NaN
    *pair = as_half2(0x7e007e00u);
    return 0u;
  }
  if (mx > kKv4Largest || mn < -kKv4Largest) {  // all four lanes of the group
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -kKv4Largest), kKv4Largest);
    mn = fminf(fmaxf(mn, -kKv4Largest), kKv4Largest);
    mx = fminf(fmaxf(mx, -kKv4Largest), kKv4Largest);
  }
  const __half lo16 = __float2half_rn(mn + 0.f);  // -0 becomes +0
  const float lo = __half2float(lo16);
  // spread / 15, rounded once, by Markstein's method: a first quotient, its exact remainder by
  // fma, and the correction (compared with a division for every mantissa: always equal)
  const float spread = fmaxf(0.f, mx - lo);
  constexpr float kFifteenth = 1.f / 15.f;
  const float q0 = spread * kFifteenth;
  const __half step16 = __float2half_rn(fmaf(fmaf(-15.f, q0, spread), kFifteenth, q0));
  const float step = __half2float(step16);
  *pair = __halves2half2(step16, lo16);
  if (step == 0.f) return 0u;

  // The quotient over 15, held within 0..1, then its integer by adding 2^23, which rounds to
  // nearest even at units; c = integer + 2^23.  Off by less than 2^-17 before the rounding
  // (15 times a few 2^-23), so right unless the quotient is that near a tie.
  const float inverse = __fdividef(1.f, 15.f * step);
  constexpr float kUnits = 8388608.f;
  const float2 minus_lo = make_float2(-lo, -lo), fifteen = make_float2(15.f, 15.f), units = make_float2(kUnits, kUnits);
  uint32_t word = 0;
  float off_tie = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 d = __fadd2_rn(make_float2(x[i], x[i + 1]), minus_lo);
    const float2 y = make_float2(__saturatef(d.x * inverse), __saturatef(d.y * inverse));
    const float2 c = __ffma2_rn(y, fifteen, units);
    const float2 off = __ffma2_rn(y, fifteen, __fadd2_rn(units, make_float2(-c.x, -c.y)));
    off_tie = fmaxf(off_tie, fmaxf(fabsf(off.x), fabsf(off.y)));
    word += (__float_as_uint(c.x) << (4 * i)) + (__float_as_uint(c.y) << (4 * i + 4));
  }
  word -= 0x4b000000u;  // the bits of 2^23: those of the other seven left the word with the shifts
  word -= 0x4b000000u << 4;
  if (off_tie < 0.49999f) return word;

  // Near a tie the remainder d - c step settles it, which one fma gives exactly (c step has at
  // most 15 bits, and the remainder no more than d or step).
  word = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    float xi = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e == i) xi = x[e];
    const float d = xi - lo;
    float c = rintf(15.f * __saturatef(d * inverse));
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
