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
// modulo 2^64 drops the whole turns exactly.  What is lost is F's last bit times the position:
// below 2^-32 turns up to position 2^31 (for frequencies up to 1; larger ones lose as many bits
// more as they are larger).
// The nearest quarter turn goes off as an integer too, so that only the rest, at most 1/8
// turn, is rounded to fp32: by 2^-28 turns at most (half a step of 2^-27 from 1/16 turn on).  No
// range reduction of large arguments, no table of positions (a table is a dependent load of 512
// bytes a token).
//
// Layout.  A row is L = D / (2 V) lanes of two 16-byte vectors (V values each).  A lane
// holds both halves of its pairs: half layout: vectors l and l + R/2V, interleaved: 2l and
// 2l + 1; lanes past the rotated dimensions take vectors 2l and 2l + 1 either way (R/V + 2 (l -
// R/2V) = 2l).  So rotation needs no exchange between lanes, and pair j of lane l is number
// V l + j in both layouts.  A warp has 32 / L rows, whose sums of squares take log2 L shuffles.
//
// Work.  A token belongs to 1 to 8 warps, each of which computes the token's cosines and sines,
// multiplies them with the norm's weights once, and then runs over its share of the heads with
// those factors in registers: out_a = r (x_a w_a c - x_b w_b s), r the norm.  Four rows are
// loaded ahead.
//
// Bound: HBM, each value read once and written once, for prompts (append of 16,384 tokens, 64/8
// heads, D 128, bf16, norms: 107 us, 0.92 of copy bandwidth); the chain launch -> position -> angle
// -> store for a few tokens (64 tokens: 3.8 us in a graph), so rows are loaded before angles are computed.
#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kAhead = 4;  // rows of a lane in flight

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

// inv_freq (radians per position) as a fraction of a turn, in units of 2^-64: its 53-bit
// mantissa times 2^64 / 2 pi, shifted by its exponent, whole turns dropped.  In integers: the
// GPU's FP64 rate is low.
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
  const int exponent = static_cast<int>(bits >> 52) & 0x7ff;
  const uint64_t mantissa = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  const uint64_t kInvTwoPi = 0x28be60db9391054aull;
  const uint64_t low = mantissa * kInvTwoPi, high = __umul64hi(mantissa, kInvTwoPi);
  const int down = 1075 - exponent;  // the product's places below 2^-64 turns
  uint64_t turns = 0;                // frequencies below 2^-75 do not turn in 2^31 positions
  if (down >= 64) turns = down < 128 ? high >> (down - 64) : 0;
  else if (down > 0) turns = high << (64 - down) | low >> down;
  else if (down > -64) turns = low << -down;
  return bits >> 63 ? 0 - turns : turns;
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

// A lane's factors for the heads of one tensor, for outputs a and b of its V pairs (half: the
// elements of its two vectors; interleaved: the first and the second of each pair):
//   a' = a ca - b sb,  b' = b cb + a sa.
template <int V>
struct Factors {
  float ca[V], sb[V], cb[V], sa[V];
};

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 2) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int L = D / (2 * V);        // lanes of a row
  constexpr int kRows = 32 / L;         // rows of a warp
  __shared__ __align__(16) float2 angles[kWarps][D / 2];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per = p.warps_per_token;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kWarps / per) + warp / per;
  if (t >= p.num_tokens) return;
  const int l = lane % L;
  const int first = warp % per * kRows + lane / L, step = per * kRows;  // this lane's heads
  const int turned = p.rotary_dim / (2 * V);  // lanes of a row that hold rotated pairs
  const int v0 = (!kInterleaved && l < turned ? l : 2 * l) * V;
  const int v1 = !kInterleaved && l < turned ? v0 + turned * V : v0 + V;
  const bool turns = l < turned;

  // the first rows of queries, before anything that takes a while
  uint4 ahead[kAhead][2];
  const T* src = static_cast<const T*>(p.q) + t * p.q_stride;
  auto load = [&](int u, int head, int heads) {
    if (head < heads) {
      ahead[u][0] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(head) * D + v0);
      ahead[u][1] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(head) * D + v1);
    }
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, first + u * step, p.num_q_heads);

  const int position = p.positions[t];
  const int64_t slot = p.slots ? p.slots[t] : 0;
  if (position < 0 || slot < 0) return;  // padding
  int64_t place = 0;  // in the pools: the row of the token's first KV head
  if (p.slots) {
    if (slot >= p.num_slots) {
      set_error(p.err, kErrIndex);
      return;
    }
    place = slot / p.block_size * p.block_size * p.num_kv_heads + slot % p.block_size;
  }
  for (int n = lane; n < p.rotary_dim / 2; n += 32) {
    const double freq = p.inv_freq[n];
    const float2 cs = cos_sin(turns_of(freq), static_cast<uint32_t>(position));
    angles[warp][n] = isfinite(freq) ? make_float2(cs.x * p.factor, cs.y * p.factor) : make_float2(NAN, NAN);
  }
  __syncwarp();

  Factors<V> f;
  auto factors = [&](const void* weight) {
    float w[2 * V];  // of vector 0, of vector 1
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) w[e] = 1.f;
    if (weight) {
      Elem<T>::load16(static_cast<const T*>(weight) + v0, w);
      Elem<T>::load16(static_cast<const T*>(weight) + v1, w + V);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float wa = kInterleaved ? w[2 * j] : w[j], wb = kInterleaved ? w[2 * j + 1] : w[V + j];
      const float2 cs = turns ? angles[warp][l * V + j] : make_float2(1.f, 0.f);
      f.ca[j] = wa * cs.x;
      f.sb[j] = wb * cs.y;
      f.cb[j] = wb * cs.x;
      f.sa[j] = wa * cs.y;
    }
  };
  // heads first, first + step, ... of src, whose first kAhead are loaded, to dst; `apart` rows
  // of D from a head to the next there
  auto run = [&](int heads, bool norm, T* dst, int apart) {
    for (int base = first - lane / L; base < heads; base += kAhead * step) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (base + u * step >= heads) break;  // a warp's lanes stay together for the shuffles
        const int head = base + u * step + lane / L;
        const bool live = head < heads;
        if (!live) ahead[u][0] = ahead[u][1] = make_uint4(0, 0, 0, 0);
        float x[2 * V];
        Elem<T>::load16(&ahead[u][0], x);
        Elem<T>::load16(&ahead[u][1], x + V);
        load(u, head + kAhead * step, heads);
        if (norm) {
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 2 * V; e += 2) {
            const float2 y = make_float2(x[e], x[e + 1]);
            sum = __ffma2_rn(y, y, sum);
          }
          const float r = rsqrtf(group_sum<L>(sum.x + sum.y) * (1.f / D) + p.eps);
          const float2 r2 = make_float2(r, r);
#pragma unroll
          for (int e = 0; e < 2 * V; e += 2) {
            const float2 y = __fmul2_rn(make_float2(x[e], x[e + 1]), r2);
            x[e] = y.x;
            x[e + 1] = y.y;
          }
        }
        if (!live) continue;
        if (turns) {
#pragma unroll
          for (int j = 0; j < V; j += (kInterleaved ? 1 : 2)) {
            if (kInterleaved) {
              const float2 y = make_float2(x[2 * j], x[2 * j + 1]);
              const float2 z = __ffma2_rn(make_float2(y.y, y.x), make_float2(-f.sb[j], f.sa[j]),
                                          __fmul2_rn(y, make_float2(f.ca[j], f.cb[j])));
              x[2 * j] = z.x;
              x[2 * j + 1] = z.y;
            } else {
              const float2 a = make_float2(x[j], x[j + 1]), b = make_float2(x[V + j], x[V + j + 1]);
              const float2 ya = __ffma2_rn(b, make_float2(-f.sb[j], -f.sb[j + 1]),
                                           __fmul2_rn(a, make_float2(f.ca[j], f.ca[j + 1])));
              const float2 yb = __ffma2_rn(a, make_float2(f.sa[j], f.sa[j + 1]),
                                           __fmul2_rn(b, make_float2(f.cb[j], f.cb[j + 1])));
              x[j] = ya.x;
              x[j + 1] = ya.y;
              x[V + j] = yb.x;
              x[V + j + 1] = yb.y;
            }
          }
        } else {  // factors of 1 times the weights (a product with a sine of 0 would turn infinities into NaN)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            x[kInterleaved ? 2 * j : j] *= f.ca[j];
            x[kInterleaved ? 2 * j + 1 : V + j] *= f.cb[j];
          }
        }
        T* row = dst + static_cast<int64_t>(head) * apart * D;
        *reinterpret_cast<uint4*>(row + v0) = pack16<T>(x);
        *reinterpret_cast<uint4*>(row + v1) = pack16<T>(x + V);
      }
    }
  };
  if (p.num_q_heads > 0) {
    factors(p.q_weight);
    run(p.num_q_heads, p.q_weight != nullptr, static_cast<T*>(p.q_out) + t * p.q_out_stride, 1);
  }
  if (p.num_kv_heads > 0) {
    src = static_cast<const T*>(p.k) + t * p.k_stride;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u, first + u * step, p.num_kv_heads);
    factors(p.k_weight);
    if (p.slots) run(p.num_kv_heads, p.k_weight != nullptr, static_cast<T*>(p.k_cache) + place * D, p.block_size);
    else run(p.num_kv_heads, p.k_weight != nullptr, static_cast<T*>(p.k_out) + t * p.k_out_stride, 1);
  }
  if (p.slots) {  // values as they came, bit for bit
    src = static_cast<const T*>(p.v) + t * p.v_stride;
    for (int head = first; head < p.num_kv_heads; head += kAhead * step) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load(u, head + u * step, p.num_kv_heads);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (head + u * step >= p.num_kv_heads) break;
        T* row = static_cast<T*>(p.v_cache) + (place + static_cast<int64_t>(head + u * step) * p.block_size) * D;
        *reinterpret_cast<uint4*>(row + v0) = ahead[u][0];
        *reinterpret_cast<uint4*>(row + v1) = ahead[u][1];
      }
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
  // As many warps a token as it takes for 16 warps an SM: every warp computes its token's angles
  // (1,000 tokens of 64/8 heads: 12 us with 2 warps a token, 23 with 8).
  p.warps_per_token = 8;
  while (p.warps_per_token > 1 && static_cast<int64_t>(p.num_tokens) * p.warps_per_token > 16 * 152) p.warps_per_token /= 2;
  const int tokens = kWarps / p.warps_per_token;
  const int grid = (p.num_tokens - 1) / tokens + 1;
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
