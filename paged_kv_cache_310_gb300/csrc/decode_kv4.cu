// decode_kv4.cu -- single-token attention over a 4-bit paged cache (format: kv4.cuh).
//
// For sequence s, KV head g and each query head h of g's group:
//   out = sum_j softmax_j(scale * q_h . K_j) V_j,  j < context_lens[s],
// with K_j, V_j the fp16 numbers that the rows stand for.
//
// Bound: HBM.  A token and KV head is 2 * 5 D / 8 bytes (160 at D = 128, against 512 in
// 16 bits), so at copy bandwidth an SM must widen about 37 values per clock: the 4-bit
// codes cannot go through shared memory again as 16-bit operands.  They are widened in
// registers, straight into the fragments of warp-level MMAs (m16n8k16, fp32 accumulators):
//   scores  S[16 tokens x 8 heads] = K[16 x D] q^T      A = K,    B = q^T
//   output  O^T[D x 8 heads]      += V^T[D x 16] P^T    A = V^T,  B = P^T
// Both products take the 4-bit operand as A, whose fragment covers 16 x 16 values; B's
// eight columns are the query heads.
//  * K: lane (g, t) takes the t-th quarter of rows g and g + 8 -- one group's (step, lo)
//    per row -- and pairs of one word's codes become the contracted pairs of a step.
//  * V: lane (g, t) takes the g-th eighth of rows 2t, 2t+1, 2t+8, 2t+9; a byte permute
//    pairs two tokens' codes of one dimension, as the contraction over tokens wants them.
//  * P goes from the score layout to the B layout by 8 x 8 transposes, in two fp16 parts
//    (p rounded, and the rest), so a weight is good to 2^-22.  Up to four heads per KV
//    head the second part takes columns 4..7 (q's columns are doubled, so the lanes there
//    hold the same p); above, a second MMA.
//
// Work: one CTA per (partition, KV head, sequence); its warps take every fourth tile of 16
// tokens and run alone: each has its own ring of cp.async stages (K and V of a tile, 16
// bytes per lane and copy), its own running maximum (raised only when a score exceeds it by
// 8, log2 domain), sum and O, combined through shared memory at the end in a fixed order.
// Waits are cp.async.wait_group only.  Partitions are merged as for the other caches.
#include "kv4.cuh"
#include "launch.h"
#include "mma.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;          // tokens per warp tile
constexpr float kSlack = 8.f;      // a score may exceed the running maximum by this much
constexpr float kLift = 6.f;       // p = 2^(x - m + 6): small weights stay normal fp16 numbers

// NB blocks of eight columns; kDup: at most four heads, in columns 0..3 and again in 4..7;
// kSplit: f32 queries, in two fp16 parts.
template <int D, int NB, bool kDup, bool kSplit>
struct Kv4 {
  static constexpr int kRow = Kv4Row<D>::kBytes;
  static constexpr int kHalf = 8 * kRow;             // eight rows: never more than one block
  static constexpr int kStage = 4 * kHalf;           // K rows 0-7, 8-15, V rows 0-7, 8-15
  static constexpr int kChunks = kStage / 16;
  static constexpr int kPerLane = (kChunks + 31) / 32;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kRingBytes = kWarps * kStages * kStage;
  static constexpr int kCols = 8 * NB;
  static constexpr int kReduceBytes = kWarps * kCols * (D + 2) * 4;
  static constexpr int kMainBytes = (kRingBytes > kReduceBytes ? kRingBytes : kReduceBytes);
};

__device__ __forceinline__ void store_any(void* out, size_t i, float x, int dtype) {
  if (dtype == PKV_F32)
    static_cast<float*>(out)[i] = x;
  else if (dtype == PKV_F16)
    static_cast<__half*>(out)[i] = __float2half_rn(x);
  else
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
}

template <int D, int NB, bool kDup, bool kSplit>
__global__ void __launch_bounds__(kThreads) decode_kv4_kernel(const __grid_constant__ DecodeParams p, int q_dtype,
                                                              int out_dtype) {
  using C = Kv4<D, NB, kDup, kSplit>;
  extern __shared__ __align__(128) unsigned char smem[];
  if (p.max_parts > 1) grid_dependents_launch();  // the merge, which waits for this grid

  const int part = blockIdx.x, kvh = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int G = p.group;
  const int L = p.context_lens[s];
  if (L < 0 || L > p.max_parts * p.part_tokens) {
    if (part == 0 && threadIdx.x == 0) set_error(p.err, kErrLength);
    return;
  }
  const size_t out_row = static_cast<size_t>(s) * p.num_q_heads + static_cast<size_t>(kvh) * G;
  if (L == 0) {  // empty context: the neutral output
    if (part == 0)
      for (int i = threadIdx.x; i < G * D; i += kThreads) store_any(p.out, out_row * D + i, 0.f, out_dtype);
    return;
  }
  const int t0 = part * p.part_tokens;
  if (t0 >= L) return;
  const int ntok = min(p.part_tokens, L - t0);
  const int ntiles = (ntok + kTile - 1) / kTile;
  const int nparts = (L + p.part_tokens - 1) / p.part_tokens;

  int* ids = reinterpret_cast<int*>(smem + C::kMainBytes);
  const int bs_log2 = 31 - __clz(p.block_size);
  {
    const int first = t0 >> bs_log2, nblk = (ntok + p.block_size - 1) >> bs_log2;
    const int32_t* row = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    for (int i = threadIdx.x; i < nblk; i += kThreads) {
      int b = first + i < p.max_blocks_per_seq ? row[first + i] : -1;
      if (b < 0 || b >= p.num_blocks) {
        set_error(p.err, kErrIndex);
        b = 0;  // keep the copy in bounds; the flag reports the bad table
      }
      ids[i] = b;
    }
  }
  __syncthreads();

  // ---- this lane's share of a tile's copies: 16-byte piece `lane + 32 i` of the stage
  unsigned char* ring = smem + warp * (C::kStages * C::kStage);
  const uint32_t ring_addr = smem_addr(ring) + lane * 16;
  const unsigned char* base[C::kPerLane];
  bool second[C::kPerLane];  // of the tile's two halves
#pragma unroll
  for (int i = 0; i < C::kPerLane; ++i) {
    const int ch = lane + 32 * i, quarter = ch / (C::kHalf / 16);
    base[i] = static_cast<const unsigned char*>(quarter < 2 ? p.k_cache : p.v_cache) +
              (ch - quarter * (C::kHalf / 16)) * 16;
    second[i] = quarter & 1;
  }
  const int64_t tile_bytes = static_cast<int64_t>(p.block_size) * C::kRow;
  const int64_t block_bytes = tile_bytes * p.num_kv_heads;
  const int64_t head_off = tile_bytes * kvh;
  auto issue = [&](int tile, int stage) {
    if (tile < ntiles) {
      const int tok0 = tile * kTile, tok1 = tok0 + 8;
      const bool have1 = tok1 < ntok;
      const int at1 = have1 ? tok1 : tok0;
      const int64_t off0 = ids[tok0 >> bs_log2] * block_bytes + head_off + (tok0 & (p.block_size - 1)) * C::kRow;
      const int64_t off1 = ids[at1 >> bs_log2] * block_bytes + head_off + (at1 & (p.block_size - 1)) * C::kRow;
#pragma unroll
      for (int i = 0; i < C::kPerLane; ++i)
        if (C::kChunks % 32 == 0 || i + 1 < C::kPerLane || lane + 32 * i < C::kChunks)
          cp_async16(ring_addr + stage * C::kStage + i * 512, base[i] + (second[i] ? off1 : off0),
                     second[i] && !have1 ? 0u : 16u);
    }
    cp_async_commit();  // one group per call, empty past the end: the waits below count them
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) issue(warp + i * kWarps, i);

  // ---- queries
  uint32_t qh[NB][D / 16][2], ql[NB][kSplit ? D / 16 : 1][2];
  float sc[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int h = kDup ? (g & 3) : nb * 8 + g;
    const float undo = load_q_kv4<D, kSplit>(p.q, q_dtype, out_row + h, h < G, t, qh[nb], ql[nb]) * p.scale_log2;
    sc[nb][0] = __shfl_sync(0xffffffffu, undo, 8 * t);
    sc[nb][1] = __shfl_sync(0xffffffffu, undo, 8 * t + 4);
  }

  float m[NB][2], l[NB][2], o[NB][D / 16][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
  }

  int stage = 0;
  for (int tile = warp; tile < ntiles; tile += kWarps) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();  // the other lanes' copies too; and everybody has left the stage refilled next
    {
      const int refill = stage == 0 ? C::kStages - 1 : stage - 1;
      issue(tile + (C::kStages - 1) * kWarps, refill);
    }
    const unsigned char* ks = ring + stage * C::kStage;
    const unsigned char* vs = ks + 2 * C::kHalf;
    stage = stage + 1 == C::kStages ? 0 : stage + 1;
    const int left = ntok - tile * kTile;  // tokens of this tile and after it

    // ---- scores
    float c[NB][2][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[nb][0][i] = c[nb][1][i] = 0.f;
    {
      constexpr int kWords = D / 32;
      uint32_t w0[kWords], w1[kWords];
      const unsigned char* r0 = ks + g * C::kRow;
#pragma unroll
      for (int i = 0; i < kWords; i += 2) {  // 8-byte loads: rows of 40 bytes are 8-byte aligned
        const uint2 a = *reinterpret_cast<const uint2*>(r0 + t * (D / 8) + 4 * i);
        const uint2 b = *reinterpret_cast<const uint2*>(r0 + C::kHalf + t * (D / 8) + 4 * i);
        w0[i] = a.x; w0[i + 1] = a.y;
        w1[i] = b.x; w1[i + 1] = b.y;
      }
      const int pair = D / 2 + 4 * (t * D / 128);
      const __half2 p0 = *reinterpret_cast<const __half2*>(r0 + pair);
      const __half2 p1 = *reinterpret_cast<const __half2*>(r0 + C::kHalf + pair);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t a[4], b[4];
        kv4_word(w0[i], __low2half2(p0), __high2half2(p0), a);
        kv4_word(w1[i], __low2half2(p1), __high2half2(p1), b);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma_f16(c[nb][0], a[0], b[0], a[1], b[1], qh[nb][2 * i][0], qh[nb][2 * i][1]);
          mma_f16(c[nb][1], a[2], b[2], a[3], b[3], qh[nb][2 * i + 1][0], qh[nb][2 * i + 1][1]);
          if (kSplit) {
            mma_f16(c[nb][0], a[0], b[0], a[1], b[1], ql[nb][2 * i][0], ql[nb][2 * i][1]);
            mma_f16(c[nb][1], a[2], b[2], a[3], b[3], ql[nb][2 * i + 1][0], ql[nb][2 * i + 1][1]);
          }
        }
      }
    }

    // ---- softmax; tokens past the end get -inf
    uint32_t ph[NB][2], pl[NB][2];  // P^T fragments: tokens 0-7 and 8-15
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (c[nb][0][i] + c[nb][1][i]) * sc[nb][i & 1];
      if (left < kTile) {
        if (g >= left) x[0] = x[1] = -INFINITY;
        if (g + 8 >= left) x[2] = x[3] = -INFINITY;
      }
      const bool over = x[0] > m[nb][0] + kSlack || x[2] > m[nb][0] + kSlack || x[1] > m[nb][1] + kSlack ||
                        x[3] > m[nb][1] + kSlack;
      if (__any_sync(0xffffffffu, over)) {
        float a = fmaxf(x[0], x[2]), b = fmaxf(x[1], x[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
          b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
        }
        a = fmaxf(a, m[nb][0]);
        b = fmaxf(b, m[nb][1]);
        // a column that saw nothing but NaN yet keeps m = -inf, and its NaN sum
        const float fa = a == m[nb][0] ? 1.f : exp2f(m[nb][0] - a), fb = b == m[nb][1] ? 1.f : exp2f(m[nb][1] - b);
        m[nb][0] = a;
        m[nb][1] = b;
        l[nb][0] *= fa;
        l[nb][1] *= fb;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[nb][i][0] *= fa;
          o[nb][i][1] *= fb;
          o[nb][i][2] *= fa;
          o[nb][i][3] *= fb;
        }
      }
      const float ma = m[nb][0] - kLift, mb = m[nb][1] - kLift;
      const float e0 = exp2f(x[0] - ma), e1 = exp2f(x[1] - mb), e2 = exp2f(x[2] - ma), e3 = exp2f(x[3] - mb);
      l[nb][0] += e0 + e2;
      l[nb][1] += e1 + e3;
      uint32_t h0 = pack_half2(e0, e1), h1 = pack_half2(e2, e3);
      const uint32_t r0 = pack_half2_rest(e0, e1, h0), r1 = pack_half2_rest(e2, e3, h1);
      if (kDup) {
        if (t >= 2) {
          h0 = r0;
          h1 = r1;
        }
      } else {
        pl[nb][0] = movmatrix_trans(r0);
        pl[nb][1] = movmatrix_trans(r1);
      }
      ph[nb][0] = movmatrix_trans(h0);
      ph[nb][1] = movmatrix_trans(h1);
    }

    // ---- output
    {
      constexpr int kWords = D / 64;  // of codes per row and lane
      uint32_t w[4][kWords];
      uint32_t pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1) + (i & 2) * 4;
        const unsigned char* row = vs + r * C::kRow;
        if (kWords == 2) {
          const uint2 a = *reinterpret_cast<const uint2*>(row + g * 8);
          w[i][0] = a.x;
          w[i][kWords - 1] = a.y;
        } else {
          w[i][0] = *reinterpret_cast<const uint32_t*>(row + g * 4);
        }
        pr[i] = *reinterpret_cast<const uint32_t*>(row + D / 2 + 4 * (g * D / 256));
        // past the end a row holds anything, NaN too: step = lo = 0 makes it zero
        if (left < kTile && r >= left) pr[i] = 0u;
      }
      const __half2 step0 = as_half2(__byte_perm(pr[0], pr[1], 0x5410)), lo0 = as_half2(__byte_perm(pr[0], pr[1], 0x7632));
      const __half2 step1 = as_half2(__byte_perm(pr[2], pr[3], 0x5410)), lo1 = as_half2(__byte_perm(pr[2], pr[3], 0x7632));
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t sel = 0x4400u + 0x1111u * j;  // byte j of both words, twice each
          const uint32_t x0 = __byte_perm(w[0][i], w[1][i], sel), x1 = __byte_perm(w[2][i], w[3][i], sel);
          const uint32_t a0 = as_u32(__hfma2(low_codes(x0), step0, lo0)), a1 = as_u32(__hfma2(high_codes(x0), step0, lo0));
          const uint32_t a2 = as_u32(__hfma2(low_codes(x1), step1, lo1)), a3 = as_u32(__hfma2(high_codes(x1), step1, lo1));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_f16(o[nb][4 * i + j], a0, a1, a2, a3, ph[nb][0], ph[nb][1]);
            if (!kDup) mma_f16(o[nb][4 * i + j], a0, a1, a2, a3, pl[nb][0], pl[nb][1]);
          }
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // every warp has left its ring: the sums take its place

  // ---- combine the warps in a fixed order
  float* red_m = reinterpret_cast<float*>(smem);       // [warps][cols]
  float* red_l = red_m + kWarps * C::kCols;            // [warps][cols]
  float* red_o = red_l + kWarps * C::kCols;            // [warps][cols][D]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l[nb][0] += __shfl_xor_sync(0xffffffffu, l[nb][0], off);
      l[nb][1] += __shfl_xor_sync(0xffffffffu, l[nb][1], off);
    }
    const int col = warp * C::kCols + nb * 8 + 2 * t;
    if (g == 0) {
      red_m[col] = m[nb][0];
      red_m[col + 1] = m[nb][1];
      red_l[col] = l[nb][0];
      red_l[col + 1] = l[nb][1];
    }
    // lane (g, t): dimensions g D/8 + 2i and + 2i + 1 of columns 2t and 2t + 1
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int d = g * (D / 8) + 2 * i;
      *reinterpret_cast<float2*>(red_o + col * D + d) = make_float2(o[nb][i][0], o[nb][i][2]);
      *reinterpret_cast<float2*>(red_o + (col + 1) * D + d) = make_float2(o[nb][i][1], o[nb][i][3]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += kThreads) {
    const int h = i / D, d = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w * C::kCols + h]);
    float lsum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int col = w * C::kCols + h;
      if (red_l[col] == 0.f) continue;  // the warp saw no token
      const float cf = exp2f(red_m[col] - M);
      lsum = fmaf(cf, red_l[col], lsum);
      acc = fmaf(cf, red_o[col * D + d] + (kDup ? red_o[(col + 4) * D + d] : 0.f), acc);
    }
    if (nparts == 1) {
      store_any(p.out, (out_row + h) * D + d, acc / lsum, out_dtype);
    } else {
      const size_t k = (out_row + h) * p.max_parts + part;
      p.ws_o[k * D + d] = acc;
      if (d == 0) {
        p.ws_ml[2 * k] = M;
        p.ws_ml[2 * k + 1] = lsum;
      }
    }
  }
}

template <int D, int NB, bool kDup, bool kSplit>
cudaError_t launch_t(const DecodeParams& p, int q_dtype, int out_dtype, cudaStream_t stream) {
  using C = Kv4<D, NB, kDup, kSplit>;
  const size_t smem = C::kMainBytes + static_cast<size_t>(p.part_tokens / p.block_size) * 4;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem_limit(decode_kv4_kernel<D, NB, kDup, kSplit>, 100 * 1024, configured);
  if (e != cudaSuccess) return e;
  dim3 grid(p.max_parts, p.num_kv_heads, p.num_seqs);
  decode_kv4_kernel<D, NB, kDup, kSplit><<<grid, kThreads, smem, stream>>>(p, q_dtype, out_dtype);
  return cudaGetLastError();
}

template <int D, bool kSplit>
cudaError_t launch_g(const DecodeParams& p, int q_dtype, int out_dtype, cudaStream_t stream) {
  if (p.group <= 4) return launch_t<D, 1, true, kSplit>(p, q_dtype, out_dtype, stream);
  if (p.group <= 8) return launch_t<D, 1, false, kSplit>(p, q_dtype, out_dtype, stream);
  return launch_t<D, 2, false, kSplit>(p, q_dtype, out_dtype, stream);
}

}  // namespace

cudaError_t launch_decode_kv4(const DecodeParams& p, int q_dtype, int out_dtype, cudaStream_t stream) {
  if (q_dtype == PKV_F32)
    return p.head_dim == 64 ? launch_g<64, true>(p, q_dtype, out_dtype, stream) : launch_g<128, true>(p, q_dtype, out_dtype, stream);
  return p.head_dim == 64 ? launch_g<64, false>(p, q_dtype, out_dtype, stream) : launch_g<128, false>(p, q_dtype, out_dtype, stream);
}

}  // namespace pkv
