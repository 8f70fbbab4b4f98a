// window_rows.cu -- attention of few query rows over a sliding window and the first tokens, in
// one launch and without a workspace; f16/bf16, head_dim 64 or 128.
//
// What it computes: softmax(scale * q . K_j) V_j over the tokens j that a new token at position p
// attends to (j <= p with j > p - window or j < sinks; see window.cuh), for the query heads of one
// KV head and one or a few new tokens of a sequence.
//
// Mathematics, per tile of 16 tokens and columns = (new token, query head), 8 NT of them:
//   S[16 tokens x 8 NT] = K[16 x D] . Q^T          (m16n8k16 MMAs, tokens are rows)
//   O^T[D x 8 NT] += V^T[D x 16] . P[16 x 8 NT]    (twice: P as a rounded part and what is left)
// S comes out with tokens on lane groups and columns on the lanes of a group, P goes in with
// tokens on the lanes: one 8 x 8 transpose per word (movmatrix).  O^T has columns where S has
// them, so that running maxima and rescales need no exchange.  Columns keep a maximum that moves
// only when a score passes it by 8 (log2 units), so most tiles have one vote and no reduction.
//
// Work and join: see window_rows.cuh.
//
// Bound: for few sequences the chain launch -> length -> block table -> K/V -> join (one, window
// 1,024: 7.0 us in a graph); for many, HBM (128 of 512 to 32,768 tokens, window 4,096, 64/8 heads,
// D 128, bf16: 298 to 306 us, 6.8 to 7.0 TB/s).
#include "window_rows.cuh"

namespace pkv {
namespace {

constexpr int kTile = 16;  // tokens of a tile

template <int D, int NT>
struct Rows {
  static constexpr int kCols = 8 * NT;
  static constexpr int kStages = D == 128 ? 2 : 3;          // 16 or 12 KB a warp
  // CTAs of an SM, by registers and shared memory.  (Rings half as deep again and two CTAs: 14.4 us
  // against 10.3 on 64 sequences, 64/8 heads, D 64, window 128; 90 against 88 on 128, D 128, 1,024.
  // Three instead of four at D 64 with 16 columns: 38 against 31 on 64 sequences, 128/8 heads, 1,024.)
  static constexpr int kCtas = D == 64 ? 4 : 3;
  static constexpr int kRing = 2 * kStages * kTile * D * 2;  // of a warp
  static constexpr int kPitch = D + 4;                      // floats of a column's products
  static constexpr int kJoin = kWarps * kCols * kPitch * 4; // the warps' products, over the rings
  static constexpr int kMain = kWarps * kRing > kJoin ? kWarps * kRing : kJoin;
  static constexpr int kOffStats = kMain;                   // [kWarps][kCols] maxima and sums
  static constexpr int kOffFactor = kOffStats + kWarps * kCols * 8;  // [kCols][8 kWarps] factors of the parts
  static constexpr int kOffQ = kOffFactor + kCols * 8 * kWarps * 4;
  static constexpr bool kSharedQ = NT > 1;                  // queries in shared memory, not in registers
  static constexpr int kBytes = kOffQ + (kSharedQ ? kCols * D * 2 : 0);
  static_assert(kCtas * (kBytes + kCtaReserve) <= kSmShared, "shared memory");
};

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
}

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void load_matrices_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// Two weights rounded to T, and what the rounding left of them rounded to T.
template <typename T>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo);
template <>
__device__ __forceinline__ void split_pair<__half>(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_half2(a, b);
  lo = pack_half2_rest(a, b, hi);
}
template <>
__device__ __forceinline__ void split_pair<__nv_bfloat16>(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 l =
      __floats2bfloat162_rn(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// kOne: one new token per sequence (query_start is not read); the columns are its query heads.
template <typename T, int D, int NT, bool kOne>
__global__ void __launch_bounds__(kThreads, (Rows<D, NT>::kCtas)) window_rows_kernel(const __grid_constant__ WindowRowsParams p) {
  using R = Rows<D, NT>;
  using Stream = TileStream<T, D, kTile, R::kStages>;
  static_assert(Stream::kRing == R::kRing, "ring");
  constexpr int kCols = R::kCols, kTileBytes = Stream::kTileBytes;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = p.group;
  grid_dependency_wait();
  grid_dependents_launch();
  RowsItem it;
  if (!find_item<T, D, kOne>(p, kOne ? 1 : kCols / G, it)) return;
  const int len = it.len;
  Stream stream(p, it, smem);
#pragma unroll
  for (int i = 0; i < R::kStages; ++i) stream.load(i, i);

  // queries: column c is query head c % G of new token c / G
  const int gid = lane / 4, tid = lane % 4;
  uint32_t q[R::kSharedQ ? 1 : NT][D / 16][2];
  auto query_row = [&](int c) -> const T* {
    const int tk = kOne ? 0 : c / G, h = kOne ? c : c - tk * G;
    if (kOne ? c >= G : tk >= it.tokens) return nullptr;
    return static_cast<const T*>(p.q) + ((static_cast<size_t>(it.row0) + tk) * p.num_q_heads + it.g * G + h) * D;
  };
  if constexpr (R::kSharedQ) {
    for (int i = threadIdx.x; i < kCols * Stream::kChunks; i += kThreads) {
      const int c = i / Stream::kChunks, piece = i % Stream::kChunks;
      const T* src = query_row(c);
      *reinterpret_cast<uint4*>(smem + R::kOffQ + c * (D * 2) + ((piece ^ (c & 7)) * 16)) =
          src ? reinterpret_cast<const uint4*>(src)[piece] : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const T* src = query_row(8 * n + gid);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        q[n][kk][0] = src ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 2 * tid) : 0u;
        q[n][kk][1] = src ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + 2 * tid) : 0u;
      }
    }
  }
  // the last place that a column sees, and the first of its window
  int last[kOne ? 1 : NT][2];
  if constexpr (!kOne) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) last[n][e] = it.first_place + min((8 * n + 2 * tid + e) / G, it.tokens - 1);
  }

  float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
  }

  // ldmatrix: this lane's matrix (of four) and its row of it.  Rows start on multiples of 2 D
  // bytes, so pieces 2 kk and 2 kk + 1 of a row differ from pieces 0 and 1 by an xor.
  const int mat = lane / 8, mrow = lane % 8;
  const uint32_t k_at = ((mat & 1) * 8 + mrow) * (D * 2) + ((mat / 2) ^ mrow) * 16;
  const uint32_t v_at = ((mat / 2) * 8 + mrow) * (D * 2) + ((mat & 1) ^ mrow) * 16;
  const uint32_t q_at = smem_addr(smem + R::kOffQ) + ((mat / 2) * 8 + mrow) * (D * 2) + ((mat & 1) ^ mrow) * 16;
  int stage = 0;
  for (int i = 0; i < stream.mine; ++i) {
    cp_async_wait<R::kStages - 1>();
    __syncwarp();
    const uint32_t ks = stream.ring + stage * 2 * kTileBytes, vs = ks + kTileBytes;
    const int place = stream.place_of(i);
    // ---- scores
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4];
      load_matrices(a, (ks + k_at) ^ (kk * 32));
      if constexpr (R::kSharedQ) {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {  // both halves of two groups of eight columns
          uint32_t b[4];
          load_matrices(b, (q_at + n * 8 * (D * 2)) ^ (kk * 32));
          mma16<T>(x[n], a, b[0], b[1]);
          mma16<T>(x[n + 1], a, b[2], b[3]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16<T>(x[n], a, q[n][kk][0], q[n][kk][1]);
      }
    }
    // ---- weights: this lane has tokens gid and gid + 8 of columns 2 tid and 2 tid + 1 of each group
    // (a new token after the first has a later window: rows before it are cut as well)
    const bool whole = kOne ? place + kTile <= len && (place + kTile <= p.sinks || place >= p.sinks + it.view.gap)
                            : place + kTile - 1 <= it.first_place && (place + kTile <= p.sinks || place > len - 1 - p.window);
    uint32_t hidden = 0;  // bit 4 n + e: x[n][e] is masked
    if (!whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = place + gid + (e < 2 ? 0 : 8), to = kOne ? len - 1 : last[n][e & 1];
          const bool seen = at <= to && (at < p.sinks || (kOne ? at >= p.sinks + it.view.gap : at > to - p.window));
          if (!seen) hidden |= 1u << (4 * n + e);
        }
      }
    }
    float y[NT][4];  // log2 of the weights: scores less their column's maximum (nothing seen yet: 0)
    bool rises = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool none = m[n][e & 1] == -INFINITY;
        y[n][e] = fmaf(x[n][e], p.scale_log2, none ? 0.f : -m[n][e & 1]);
        rises |= y[n][e] > (none ? -INFINITY : 8.f) && !(hidden >> (4 * n + e) & 1);
      }
    }
    if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = hidden >> (4 * n + e) & 1 ? -INFINITY : x[n][e] * p.scale_log2;
          const float b = hidden >> (4 * n + e + 2) & 1 ? -INFINITY : x[n][e + 2] * p.scale_log2;
          float top = fmaxf(a, b);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          if (top > m[n][e]) {
            const float factor = exp2_approx(m[n][e] - top);  // 0 from -inf
            m[n][e] = top;
            l[n][e] *= factor;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              o[n][d][e] *= factor;
              o[n][d][e + 2] *= factor;
            }
          }
          const float base = m[n][e] == -INFINITY ? 0.f : m[n][e];
          y[n][e] = a - base;
          y[n][e + 2] = b - base;
        }
      }
    }
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = exp2_approx(y[n][e]);
        if (!whole && (hidden >> (4 * n + e) & 1)) w[e] = 0.f;
      }
      l[n][0] += w[0] + w[2];
      l[n][1] += w[1] + w[3];
      split_pair<T>(w[0], w[1], hi[n][0], lo[n][0]);
      split_pair<T>(w[2], w[3], hi[n][1], lo[n][1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        hi[n][h] = movmatrix_trans(hi[n][h]);
        lo[n][h] = movmatrix_trans(lo[n][h]);
      }
    }
    // ---- products
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      uint32_t a[4];
      load_matrices_trans(a, (vs + v_at) ^ (d * 32));
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16<T>(o[n][d], a, hi[n][0], hi[n][1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16<T>(o[n][d], a, lo[n][0], lo[n][1]);
    }
    __syncwarp();
    stream.load(i + R::kStages, stage);
    if (++stage == R::kStages) stage = 0;
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings become the warps' products

  // every warp leaves maxima, sums and products
  float2* stats = reinterpret_cast<float2*>(smem + R::kOffStats);   // [kWarps][kCols]
  float* prod = reinterpret_cast<float*>(smem);                     // [kWarps][kCols][kPitch]
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[n][e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const int c = 8 * n + 2 * tid + e;
      if (gid == 0) stats[warp * kCols + c] = make_float2(m[n][e], sum);
      float* dst = prod + (warp * kCols + c) * R::kPitch + gid;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        dst[16 * d] = o[n][d][e];
        dst[16 * d + 8] = o[n][d][e + 2];
      }
    }
  }
  join_rows<T, D, kCols, R::kPitch, kOne>(p, it, stats, prod, reinterpret_cast<float*>(smem + R::kOffFactor));
}

template <typename T, int D, int NT, bool kOne>
cudaError_t launch_t(const WindowRowsParams& p, cudaStream_t stream) {
  constexpr int smem = Rows<D, NT>::kBytes;
  static std::atomic<unsigned long long> configured{0};  // devices whose limit is raised
  cudaError_t e = ensure_smem_limit(window_rows_kernel<T, D, NT, kOne>, smem, configured);
  if (e != cudaSuccess) return e;
  const int per = Rows<D, NT>::kCols / p.group;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      rows_config(p, kOne ? p.num_seqs : p.num_query_tokens / per + p.num_seqs, smem, stream, attr);
  return cudaLaunchKernelEx(&cfg, window_rows_kernel<T, D, NT, kOne>, p);
}

template <typename T, int D>
cudaError_t launch_d(const WindowRowsParams& p, cudaStream_t stream) {
  if (p.query_start) return launch_t<T, D, 2, false>(p, stream);
  return p.group <= 8 ? launch_t<T, D, 1, true>(p, stream) : launch_t<T, D, 2, true>(p, stream);
}

template <typename T>
cudaError_t launch_dtype(const WindowRowsParams& p, cudaStream_t stream) {
  return p.head_dim == 64 ? launch_d<T, 64>(p, stream) : launch_d<T, 128>(p, stream);
}

}  // namespace

cudaError_t launch_window_rows(const WindowRowsParams& p, int dtype, cudaStream_t stream) {
  if (dtype == PKV_F32) return launch_window_rows_f32(p, stream);
  return dtype == PKV_F16 ? launch_dtype<__half>(p, stream) : launch_dtype<__nv_bfloat16>(p, stream);
}

}  // namespace pkv
