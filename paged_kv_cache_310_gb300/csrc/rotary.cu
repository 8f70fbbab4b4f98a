// rotary.cu -- new tokens' queries and keys normed per head and rotated by their
// positions, on the way into the cache (paged_kv_append_rotary) or into buffers
// (paged_qk_rotary).
//
// Per row x of D values (one token, one head), all in fp32, one rounding at the end:
//   y = x * w / sqrt(mean(x^2) + eps)                 (where a weight is given)
//   a pair (y_a, y_b) of rotated dimensions, i < R/2, angle t = position * inv_freq[i]:
//     (y_a c - y_b s, y_b c + y_a s), c = factor cos t, s = factor sin t
//   with (a, b) = (i, i + R/2), or (2i, 2i + 1) interleaved; dimensions from R on stay y.
//
// Angles.  Whole turns do not matter, so a position's angle is kept as a fraction of a turn
// in 64-bit fixed point: F = inv_freq / 2 pi as a multiple of 2^-64, and position * F
// modulo 2^64 drops the whole turns exactly.  What is lost is F's last bit (2^-53 of it, from
// the double product) times the position: below 2^-33 turns up to position 2^20 and inv_freq 1.
// The nearest quarter turn goes off as an integer too, so that only the rest, at most 1/8
// turn, is rounded to fp32.  No range reduction of large arguments, no table of positions
// (a table is a dependent load of 512 bytes a token).
//
// Layout.  A row is L = D / (2 V) lanes of two 16-byte vectors (V values each).  A lane
// holds both halves of its pairs: half layout: vectors l and l + R/2V, interleaved: 2l and
// 2l + 1; lanes past the rotated dimensions take vectors 2l and 2l + 1 either way (R/V + 2 (l -
// R/2V) = 2l).  So rotation needs no exchange between lanes, and pair j of lane l is number
// V l + j in both layouts.  A warp has 32 / L rows, whose sums of squares take log2 L shuffles.
//
// Bound: HBM, each value read once and written once, for prompts; the chain launch ->
// position -> angle -> store for a few tokens, so rows are loaded before angles are computed.
#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens a CTA takes at most
constexpr int kAhead = 3;      // rows a thread loads before it works on the first

// A vector of T as floats, and back (one rounding to nearest even).
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__half>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// inv_freq (radians per position) as a fraction of a turn, in units of 2^-64.
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
  const double turns = inv_freq * 0.15915494309189533577;  // 1 / 2 pi
  return __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}

// cos and sin of position * inv_freq.
__device__ __forceinline__ float2 cos_sin(uint64_t turns, uint32_t position) {
  const uint64_t at = turns * position + 0x80000000ull;
  const uint32_t turn = static_cast<uint32_t>(at >> 32);     // of 2^32 to the turn, whole turns gone
  const uint32_t quarter = (turn + (1u << 29)) >> 30;        // the nearest quarter turn, 0 .. 3 (4 is 0 again)
  const int32_t rest = static_cast<int32_t>(turn - (quarter << 30));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);    // half turns
  const float cc = (quarter & 1) ? s : c, ss = (quarter & 1) ? c : s;
  return make_float2(((quarter + 1) & 2) ? -cc : cc, (quarter & 2) ? -ss : ss);
}

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int L = D / (2 * V);  // lanes of a row
  // pair j of lane l: floats 2 (j % 2) of piece [j / 2][l], so that a warp reads a piece without bank conflicts
  __shared__ __align__(16) float4 angles[kMaxTokens][V / 2][L];
  __shared__ int64_t place[kMaxTokens];  // row of the token's first KV head in the pools; 0 in buffers; -1: skipped
  grid_dependency_wait();
  grid_dependents_launch();
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const bool pools = p.slots != nullptr;
  const int rows = hq + (pools ? 2 : 1) * hkv;  // rows of a token: queries, keys, values
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tokens_per_cta;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tokens_per_cta), p.num_tokens - first));
  const int total = tokens * rows * L;
  const int lane = threadIdx.x % L;
  const int turned = p.rotary_dim / (2 * V);  // lanes that hold rotated pairs
  const int v0 = !kInterleaved && lane < turned ? lane : 2 * lane;
  const int v1 = !kInterleaved && lane < turned ? lane + turned : 2 * lane + 1;

  for (int base = 0; base < total; base += kAhead * kThreads) {
    uint4 x[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = base + u * kThreads + threadIdx.x;
      if (i >= total) continue;
      const int row = i / L, tk = row / rows, r = row - tk * rows;
      const T* src = r < hq         ? static_cast<const T*>(p.q) + (first + tk) * p.q_stride + r * D
                     : r < hq + hkv ? static_cast<const T*>(p.k) + (first + tk) * p.k_stride + (r - hq) * D
                                    : static_cast<const T*>(p.v) + (first + tk) * p.v_stride + (r - hq - hkv) * D;
      x[u][0] = reinterpret_cast<const uint4*>(src)[v0];
      x[u][1] = reinterpret_cast<const uint4*>(src)[v1];
    }
    if (base == 0) {
      for (int i = threadIdx.x; i < tokens; i += kThreads) {
        int64_t at = p.positions[first + i] < 0 ? -1 : 0;
        if (pools && at == 0) {
          const int64_t slot = p.slots[first + i];
          if (slot >= p.num_slots) set_error(p.err, kErrIndex);
          at = slot < 0 || slot >= p.num_slots ? -1 : slot / p.block_size * p.block_size * hkv + slot % p.block_size;
        }
        place[i] = at;
      }
      const int pairs = p.rotary_dim / 2;
      for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
        const int tk = i / pairs, n = i - tk * pairs;
        const double freq = p.inv_freq[n];
        float2 cs = cos_sin(turns_of(freq), static_cast<uint32_t>(p.positions[first + tk]));
        if (!isfinite(freq)) cs = make_float2(NAN, NAN);
        reinterpret_cast<float2*>(&angles[tk][(n % V) / 2][n / V])[n % 2] = make_float2(cs.x * p.factor, cs.y * p.factor);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = base + u * kThreads + threadIdx.x;
      if (i - static_cast<int>(threadIdx.x % 32) >= total) break;  // a warp's lanes stay together for the shuffles
      const bool live = i < total;
      const int row = live ? i / L : 0, tk = row / rows, r = row - tk * rows;
      const void* weight = r < hq ? p.q_weight : r < hq + hkv ? p.k_weight : nullptr;
      float f[2 * V];
      if (!live) x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      Elem<T>::load16(&x[u][0], f);
      Elem<T>::load16(&x[u][1], f + V);
      if (p.q_weight || p.k_weight) {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 2 * V; e += 2) {
          const float2 y = make_float2(f[e], f[e + 1]);
          sum = __ffma2_rn(y, y, sum);
        }
        const float mean = group_sum<L>(sum.x + sum.y) * (1.f / D);
        if (weight) {
          const float norm = rsqrtf(mean + p.eps);
          float w[2 * V];
          Elem<T>::load16(static_cast<const uint4*>(weight) + v0, w);
          Elem<T>::load16(static_cast<const uint4*>(weight) + v1, w + V);
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) f[e] = f[e] * norm * w[e];
        }
      }
      const int64_t at = place[tk];
      if (!live || at < 0) continue;
      const bool value = r >= hq + hkv;
      if (lane < turned && !value) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const float4 cs = angles[tk][j / 2][lane];
          float* a0 = kInterleaved ? f + 2 * j : f + j;
          float* b0 = kInterleaved ? f + 2 * j + 1 : f + V + j;
          float* a1 = kInterleaved ? f + 2 * j + 2 : f + j + 1;
          float* b1 = kInterleaved ? f + 2 * j + 3 : f + V + j + 1;
          const float y0 = *a0, z0 = *b0, y1 = *a1, z1 = *b1;
          *a0 = y0 * cs.x - z0 * cs.y;
          *b0 = z0 * cs.x + y0 * cs.y;
          *a1 = y1 * cs.z - z1 * cs.w;
          *b1 = z1 * cs.z + y1 * cs.w;
        }
      }
      T* dst;
      if (r < hq)
        dst = static_cast<T*>(p.q_out) + (first + tk) * p.q_out_stride + r * D;
      else if (!pools)
        dst = static_cast<T*>(p.k_out) + (first + tk) * p.k_out_stride + (r - hq) * D;
      else
        dst = static_cast<T*>(value ? p.v_cache : p.k_cache) +
              (at + static_cast<int64_t>(value ? r - hq - hkv : r - hq) * p.block_size) * D;
      // values are copied as they came: a NaN keeps its bits
      reinterpret_cast<uint4*>(dst)[v0] = value ? x[u][0] : pack16<T>(f);
      reinterpret_cast<uint4*>(dst)[v1] = value ? x[u][1] : pack16<T>(f + V);
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(const RotaryParams& p, int grid, cudaStream_t stream) {
  return p.interleaved ? launch_dependent(rotary_kernel<T, D, true>, grid, kThreads, 0, stream, p)
                       : launch_dependent(rotary_kernel<T, D, false>, grid, kThreads, 0, stream, p);
}

template <typename T>
cudaError_t launch_d(RotaryParams p, cudaStream_t stream) {
  const int lanes = (p.num_q_heads + (p.slots ? 2 : 1) * p.num_kv_heads) * (p.head_dim / (2 * Elem<T>::kVec));
  p.tokens_per_cta = 1;
  while (p.tokens_per_cta < kMaxTokens && 2 * p.tokens_per_cta * lanes <= kAhead * kThreads &&
         p.num_tokens / (2 * p.tokens_per_cta) >= 2 * 152)
    p.tokens_per_cta *= 2;
  const int grid = (p.num_tokens - 1) / p.tokens_per_cta + 1;
  return p.head_dim == 64 ? launch_t<T, 64>(p, grid, stream) : launch_t<T, 128>(p, grid, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int dtype, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  switch (dtype) {
    case PKV_F32: return launch_d<float>(p, stream);
    case PKV_F16: return launch_d<__half>(p, stream);
    default: return launch_d<__nv_bfloat16>(p, stream);
  }
}

}  // namespace pkv
