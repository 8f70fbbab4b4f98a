// window_rows_f32.cu -- single-token attention over a sliding window and the first tokens for f32
// caches, in fp32 on CUDA cores; head_dim 64 or 128, up to 16 query heads per KV head.
//
// What it computes, its work and its join are those of window_rows.cu (see window_rows.cuh); tiles
// have 8 tokens.  Per tile and warp:
//   scores: lane = (token, quarter of the dimensions).  A K row's piece is read once, a query's
//   pieces are broadcast from shared memory, and the four quarters of a token's dot products are
//   added by a reduce-scatter, which leaves each lane the totals of a quarter of the heads (2 + 1
//   shuffles at 4 heads instead of 8).
//   products: lane = 4 dimensions (at head_dim 64 of one of two tokens at once); a token's weights
//   are broadcast from shared memory, O stays in registers.
// A K/V byte takes GM / 2 packed FMAs a lane per 4 bytes.  (A row spread over all lanes, as in
// decode_simt.cu, spends a shuffle per two FMAs on the sums: 113 us against 50 on 32 sequences,
// 64/8 heads, window 1,024.)
//
// Bound: HBM with up to 8 heads (32 sequences of 0 to 6,000 tokens, window 1,021, 32/8 heads: 44 us, copy
// bandwidth would take 36); instructions with 16 (32 sequences, 128/8 heads, window 1,024: 76 us,
// 40); for few sequences the chain launch -> length -> block table -> K/V -> join.
#include "window_rows.cuh"

namespace pkv {
namespace {

constexpr int kTile = 8;

template <int D, int GM>
struct RowsF32 {
  static constexpr int kStages = D == 128 ? 2 : 4;          // 16 KB a warp
  static constexpr int kRing = 2 * kStages * kTile * D * 4;
  static constexpr int kHeads = GM < 4 ? 1 : GM / 4;        // whose totals a lane has
  static constexpr int kQuarter = D / 4 + 4;                // floats of a query's quarter: four lie in different banks
  static constexpr int kPitch = D + 4;
  static constexpr int kJoin = kWarps * GM * kPitch * 4;
  static constexpr int kMain = kWarps * kRing > kJoin ? kWarps * kRing : kJoin;
  static constexpr int kOffStats = kMain;                                  // [kWarps][GM]
  static constexpr int kOffFactor = kOffStats + kWarps * GM * 8;           // [GM][8 kWarps]
  static constexpr int kOffQ = (kOffFactor + GM * 8 * kWarps * 4 + 15) / 16 * 16;  // [GM][4][kQuarter]
  static constexpr int kOffWeights = kOffQ + GM * 4 * kQuarter * 4;        // [kWarps][kTile][GM]
  static constexpr int kBytes = kOffWeights + kWarps * kTile * GM * 4;
  // CTAs of an SM, by shared memory: two of 16 heads at head_dim 128, three else.  (Registers for three
  // there, 168 instead of 248: 86 us against 80 on 32 sequences, 128/8 heads, window 1,020; 135
  // against 117 on 57; 471 against 401 on 57, 96/8 heads, window 4,092.)
  static constexpr int kCtas = 3 * (kBytes + kCtaReserve) <= kSmShared ? 3 : 2;
  static_assert(kCtas * (kBytes + kCtaReserve) <= kSmShared, "shared memory");
};

// Totals of each v[h] over the four lanes that differ in bits 3 and 4 of their number; returns those
// of heads first .. first + kHeads - 1, first = quarter_head<GM>(quarter).
template <int GM>
__device__ __forceinline__ int quarter_head(int quarter) {
  return GM >= 4 ? ((quarter & 2) ? GM / 2 : 0) + ((quarter & 1) ? GM / 4 : 0) : GM == 2 ? quarter / 2 : 0;
}
template <int GM, int kHeads>
__device__ __forceinline__ void quarter_sums(float (&v)[GM], float (&out)[kHeads]) {
  const int lane = threadIdx.x % 32;
  float a[GM > 1 ? GM / 2 : 1];
  if constexpr (GM > 1) {
    const bool upper = lane & 16;
#pragma unroll
    for (int h = 0; h < GM / 2; ++h) {
      const float send = upper ? v[h] : v[h + GM / 2], keep = upper ? v[h + GM / 2] : v[h];
      a[h] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
  } else {
    a[0] = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
  }
  if constexpr (GM > 2) {
    const bool upper = lane & 8;
#pragma unroll
    for (int h = 0; h < GM / 4; ++h) {
      const float send = upper ? a[h] : a[h + GM / 4], keep = upper ? a[h + GM / 4] : a[h];
      out[h] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
    }
  } else {
    out[0] = a[0] + __shfl_xor_sync(0xffffffffu, a[0], 8);
  }
}

template <int D, int GM>
__global__ void __launch_bounds__(kThreads, (RowsF32<D, GM>::kCtas)) window_rows_f32_kernel(const __grid_constant__ WindowRowsParams p) {
  using R = RowsF32<D, GM>;
  using Stream = TileStream<float, D, kTile, R::kStages>;
  static_assert(Stream::kRing == R::kRing, "ring");
  constexpr int kHeads = R::kHeads, kTileBytes = Stream::kTileBytes;
  constexpr int kLanes = D / 4;             // lanes of a token's products
  constexpr int kAtOnce = 32 / kLanes;      // tokens whose products are added at once
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = p.group;
  grid_dependency_wait();
  grid_dependents_launch();
  RowsItem it;
  if (!find_item<float, D, true>(p, 1, it)) return;
  Stream stream(p, it, smem);
#pragma unroll
  for (int i = 0; i < R::kStages; ++i) stream.load(i, i);

  // queries, a quarter of each after the other with room between; heads past the group are zeros
  float* q_s = reinterpret_cast<float*>(smem + R::kOffQ);
  for (int i = threadIdx.x; i < GM * D / 4; i += kThreads) {
    const int h = i / (D / 4), piece = i % (D / 4), quarter = piece / (D / 16);
    const float* src = static_cast<const float*>(p.q) + (static_cast<size_t>(it.s) * p.num_q_heads + it.g * G + h) * D;
    reinterpret_cast<float4*>(q_s + (h * 4 + quarter) * R::kQuarter)[piece % (D / 16)] =
        h < G ? reinterpret_cast<const float4*>(src)[piece] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();

  const int token = lane % 8, quarter = lane / 8;
  const int first_head = quarter_head<GM>(quarter);
  const bool owner = GM >= 4 || (GM == 2 ? quarter % 2 == 0 : quarter == 0);  // one lane has each (token, head)
  float* weights = reinterpret_cast<float*>(smem + R::kOffWeights) + warp * kTile * GM;
  const float* q_mine = q_s + quarter * R::kQuarter;
  float m[kHeads], l[kHeads];
  float2 o[GM][2];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
  }
#pragma unroll
  for (int h = 0; h < GM; ++h) o[h][0] = o[h][1] = make_float2(0.f, 0.f);

  int stage = 0;
  for (int i = 0; i < stream.mine; ++i) {
    cp_async_wait<R::kStages - 1>();
    __syncwarp();
    const unsigned char* ks = smem + warp * R::kRing + stage * 2 * kTileBytes;
    const unsigned char* vs = ks + kTileBytes;
    const int place = stream.place_of(i);
    // ---- scores
    float2 dots[GM];
#pragma unroll
    for (int h = 0; h < GM; ++h) dots[h] = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const float4 k = *reinterpret_cast<const float4*>(ks + token * (D * 4) + (((quarter * (D / 16) + c) ^ token) * 16));
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        const float4 qv = reinterpret_cast<const float4*>(q_mine + h * 4 * R::kQuarter)[c];
        dots[h] = __ffma2_rn(make_float2(k.x, k.y), make_float2(qv.x, qv.y), dots[h]);
        dots[h] = __ffma2_rn(make_float2(k.z, k.w), make_float2(qv.z, qv.w), dots[h]);
      }
    }
    float part[GM], x[kHeads];
#pragma unroll
    for (int h = 0; h < GM; ++h) part[h] = dots[h].x + dots[h].y;
    quarter_sums<GM, kHeads>(part, x);
    // ---- weights of this lane's token and heads
    const bool seen = stream.counts(place + token);
    bool rises = false;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      x[h] = seen ? x[h] * p.scale_log2 : -INFINITY;
      rises |= x[h] > m[h] + 8.f;
    }
    if (__any_sync(0xffffffffu, rises)) {
      // new maxima over the tile's tokens, and the factors of O for all heads by way of the weights' room
      float* factors = weights;
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        float top = x[h];
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = fmaxf(top, m[h]);
        const float factor = top > m[h] ? exp2f(m[h] - top) : 1.f;  // 0 from -inf
        m[h] = top;
        l[h] *= factor;
        if (owner && token == 0) factors[first_head + h] = factor;
      }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        const float2 f = make_float2(factors[h], factors[h]);
        o[h][0] = __fmul2_rn(o[h][0], f);
        o[h][1] = __fmul2_rn(o[h][1], f);
      }
      __syncwarp();
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const float w = seen ? exp2f(x[h] - (m[h] == -INFINITY ? 0.f : m[h])) : 0.f;
      l[h] += w;
      if (owner) weights[token * GM + first_head + h] = w;
    }
    __syncwarp();
    // ---- products
#pragma unroll
    for (int t = 0; t < kTile; t += kAtOnce) {
      const int tk = t + lane / kLanes;
      const float4 v = *reinterpret_cast<const float4*>(vs + tk * (D * 4) + (((lane % kLanes) ^ tk) * 16));
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        const float w = weights[tk * GM + h];
        o[h][0] = __ffma2_rn(make_float2(w, w), make_float2(v.x, v.y), o[h][0]);
        o[h][1] = __ffma2_rn(make_float2(w, w), make_float2(v.z, v.w), o[h][1]);
      }
    }
    __syncwarp();
    stream.load(i + R::kStages, stage);
    if (++stage == R::kStages) stage = 0;
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings become the warps' products

  float2* stats = reinterpret_cast<float2*>(smem + R::kOffStats);
  float* prod = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float sum = l[h];
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (owner && token == 0) stats[warp * GM + first_head + h] = make_float2(m[h], sum);
  }
#pragma unroll
  for (int h = 0; h < GM; ++h) {
    float4 sum = make_float4(o[h][0].x, o[h][0].y, o[h][1].x, o[h][1].y);
    if (kAtOnce == 2) {  // the tokens of the other half of the lanes
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, 16);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, 16);
      sum.z += __shfl_xor_sync(0xffffffffu, sum.z, 16);
      sum.w += __shfl_xor_sync(0xffffffffu, sum.w, 16);
    }
    if (lane < kLanes) *reinterpret_cast<float4*>(prod + (warp * GM + h) * R::kPitch + lane * 4) = sum;
  }
  join_rows<float, D, GM, R::kPitch, true>(p, it, stats, prod, reinterpret_cast<float*>(smem + R::kOffFactor));
}

template <int D, int GM>
cudaError_t launch_t(const WindowRowsParams& p, cudaStream_t stream) {
  constexpr int smem = RowsF32<D, GM>::kBytes;
  static std::atomic<unsigned long long> configured{0};  // devices whose limit is raised
  cudaError_t e = ensure_smem_limit(window_rows_f32_kernel<D, GM>, smem, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = rows_config(p, p.num_seqs, smem, stream, attr);
  return cudaLaunchKernelEx(&cfg, window_rows_f32_kernel<D, GM>, p);
}

template <int D>
cudaError_t launch_g(const WindowRowsParams& p, cudaStream_t stream) {
  if (p.group <= 1) return launch_t<D, 1>(p, stream);
  if (p.group <= 2) return launch_t<D, 2>(p, stream);
  if (p.group <= 4) return launch_t<D, 4>(p, stream);
  if (p.group <= 8) return launch_t<D, 8>(p, stream);
  return launch_t<D, 16>(p, stream);
}

}  // namespace

cudaError_t launch_window_rows_f32(const WindowRowsParams& p, cudaStream_t stream) {
  return p.head_dim == 64 ? launch_g<64>(p, stream) : launch_g<128>(p, stream);
}

}  // namespace pkv
