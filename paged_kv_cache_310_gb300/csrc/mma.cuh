// mma.cuh -- warp-level matrix instructions and asynchronous copies (inline PTX) of the
// kernels that widen operands in registers (4-bit rows) or read few rows per query.
//
// m16n8k16 fragments, lane = 4 g + t (g = 0..7, t = 0..3):
//   A (16 x 16): a0 = row g, columns 2t, 2t+1; a1 = row g+8, same; a2 = row g, columns
//                2t+8, 2t+9; a3 = row g+8, same.
//   B (16 x 8):  b0 = rows 2t, 2t+1 of column g; b1 = rows 2t+8, 2t+9.
//   C (16 x 8):  c0, c1 = row g, columns 2t, 2t+1; c2, c3 = row g+8.
// The 16 products of a step may be summed in any order, so a lane may bring any 4 of a
// step's 16 contracted values as long as A and B agree.
#pragma once

#include "common.cuh"

namespace pkv {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with C = 0: the first product of a sum.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%10, %10, %10, %10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held as one C-shaped row per lane group.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes global -> shared, asynchronously; `bytes` (16 or 0) are read, the rest is zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The same with an L2 policy (policy_evict_first: read once).
__device__ __forceinline__ void cp_async16_hint(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x, relative error up to 2^-22; results below the smallest normal number become 0.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// p rounded to fp16 pairs: (a, b) and what the rounding left of them.
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_half2_rest(float a, float b, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_half2(a - f.x, b - f.y);
}

// Eight consecutive elements of an f32, f16 or bf16 array (16-byte aligned) as floats.
__device__ __forceinline__ void load8_any(const void* p, int dtype, size_t at, float* out) {
  if (dtype == PKV_F32) {
    Elem<float>::load16(static_cast<const float*>(p) + at, out);
    Elem<float>::load16(static_cast<const float*>(p) + at + 4, out + 4);
  } else if (dtype == PKV_F16) {
    Elem<__half>::load16(static_cast<const __half*>(p) + at, out);
  } else {
    Elem<__nv_bfloat16>::load16(static_cast<const __nv_bfloat16*>(p) + at, out);
  }
}

// 4-bit K rows are multiplied with queries in fp16: a row of q is scaled by the power of two
// that puts its largest element, amax, in [2^14, 2^15).  bf16 and f16 elements are then exact
// (those 2^31 and 2^28 below the largest may lose bits, worth 2^-39 of it), f32 ones good to
// 2^-22 in two parts.  The power is at most 126, so that its inverse stays a normal number; a
// row of zeros, and one with a NaN or an infinity, which poisons its scores, is not scaled.
__device__ __forceinline__ int query_power(float amax, bool bad) {
  const int up = 141 - static_cast<int>(__float_as_uint(amax) >> 23);  // 14 less amax's exponent
  return bad || amax == 0.f ? 0 : (up > 126 ? 126 : up);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Query fragments against 4-bit K rows, one column (query head) per lane group g.
//
// Lane t of a K row brings the D/4 consecutive values from t D/4 on: word w of its codes
// gives steps 2w (values 0, 4 | 1, 5 of the word) and 2w + 1 (2, 6 | 3, 7).  q is scaled
// (query_power) and held in fp16 parts hi and, with kSplit, lo.  Returns what undoes the scale.
template <int D, bool kSplit>
__device__ __forceinline__ float load_q_kv4(const void* q, int dtype, size_t row, bool valid, int t,
                                            uint32_t (&hi)[D / 16][2], uint32_t (&lo)[kSplit ? D / 16 : 1][2]) {
  float f[D / 4];
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    if (valid) {
      load8_any(q, dtype, row * D + t * (D / 4) + 8 * w, f + 8 * w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[8 * w + i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, fabsf(f[8 * w + i]));
      bad |= !(fabsf(f[8 * w + i]) < INFINITY);
    }
  }
  uint32_t any_bad = bad;
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    any_bad |= __shfl_xor_sync(0xffffffffu, any_bad, off);
  }
  const int up = query_power(amax, any_bad);
  const float factor = power_of_two(up);
#pragma unroll
  for (int i = 0; i < D / 4; ++i) f[i] *= factor;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = f[8 * w + i], b = f[8 * w + i + 4];
      const uint32_t h = pack_half2(a, b);
      hi[2 * w + i / 2][i % 2] = h;
      if (kSplit) lo[2 * w + i / 2][i % 2] = pack_half2_rest(a, b, h);
    }
  }
  return power_of_two(-up);
}

}  // namespace pkv
