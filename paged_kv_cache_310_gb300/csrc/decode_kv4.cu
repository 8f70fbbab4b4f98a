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
// tokens and run alone: each has its own ring of cp.async stages (lanes 0-15 bring the
// tile's first eight rows of K and V, lanes 16-31 the others), its own running maximum
// (raised only when a score exceeds it by 8, log2 domain), sum and O, combined through
// shared memory at the end in a fixed order.  Waits are cp.async.wait_group only.
// Partitions are merged as for the other caches.
#include <type_traits>

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
  static constexpr int kStage = 4 * kHalf;           // K then V of rows 0-7, K then V of rows 8-15
  static constexpr int kHalfPieces = kHalf / 16;
  static constexpr int kCopies = (2 * kHalfPieces + 15) / 16;  // per lane: 16 lanes bring K and V of a half
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRingBytes = kWarps * kStages * kStage;
  static constexpr int kCols = 8 * NB;
  // the sums at the end take the ring's place: per warp (max, sum) of the columns, O fragments
  static constexpr int kReduceBytes = kWarps * (kCols * 8 + NB * (D / 16) * 32 * 16);
  static constexpr int kMainBytes = kRingBytes > kReduceBytes ? kRingBytes : kReduceBytes;
  static constexpr int kQueryBytes = NB * (kSplit ? 2 : 1) * (D / 32) * 32 * 16 + kCols * 4;
};

// Query fragments of 4-bit K rows in shared memory: piece [w][4 g + t] (16 bytes) is lane
// (g, t)'s B fragment of steps 2w and 2w + 1 for query head g of a block of eight columns.
//
// Lane t of a K row brings the D/4 consecutive values from t D/4 on: word w of its codes
// gives steps 2w (values 0, 4 | 1, 5 of the word) and 2w + 1 (2, 6 | 3, 7).  q is scaled by
// a power of two that puts its largest element in [2^14, 2^15): bf16 and f16 queries are
// then exact in fp16 (elements 2^38 below the largest lose bits, f16's none), f32 ones in
// two parts (hi, and lo with kSplit) to 2^-22.  undo[h] takes the power of two back.
// D/8 neighbouring threads work on one head; whole warps take part.
template <int D, int NB, bool kSplit>
__device__ __forceinline__ void stage_queries(const void* q, int dtype, size_t row, int heads, uint4* frag, float* undo) {
  constexpr int kPer = D / 8;  // threads per head
  for (int i = threadIdx.x; i < NB * 8 * kPer; i += kThreads) {
    const int h = i / kPer, word = i % kPer;  // values 8 word .. 8 word + 7
    float f[8];
    if (h < heads) {
      load8_any(q, dtype, (row + h) * D + 8 * word, f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
    }
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      amax = fmaxf(amax, fabsf(f[e]));
      bad |= !(fabsf(f[e]) < INFINITY);
    }
    if (bad) amax = INFINITY;
#pragma unroll
    for (int off = 1; off < kPer; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    // 2^up with up = 14 - exponent(amax), at most 126 (its inverse stays a normal number);
    // a query with a NaN or an infinity keeps its scale and poisons its scores
    int up = 141 - static_cast<int>(__float_as_uint(amax) >> 23);
    up = amax == INFINITY || amax == 0.f ? 0 : (up > 126 ? 126 : up);
    const float factor = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = f[e] * factor, b = f[e + 4] * factor;
      hi[e] = pack_half2(a, b);
      if (kSplit) lo[e] = pack_half2_rest(a, b, hi[e]);
    }
    const int t = word / (D / 32), w = word % (D / 32);
    uint4* to = frag + (((h / 8) * (kSplit ? 2 : 1)) * (D / 32) + w) * 32 + (h % 8) * 4 + t;
    *to = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (kSplit) to[(D / 32) * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (word == 0) undo[h] = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
  }
}

__device__ __forceinline__ void store_any(void* out, size_t i, float x, int dtype) {
  if (dtype == PKV_F32)
    static_cast<float*>(out)[i] = x;
  else if (dtype == PKV_F16)
    static_cast<__half*>(out)[i] = __float2half_rn(x);
  else
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
}

// Two neighbouring outputs.
__device__ __forceinline__ void store_pair(void* out, size_t i, float x, float y, int dtype) {
  if (dtype == PKV_F32) {
    *reinterpret_cast<float2*>(static_cast<float*>(out) + i) = make_float2(x, y);
  } else if (dtype == PKV_F16) {
    *reinterpret_cast<__half2*>(static_cast<__half*>(out) + i) = __floats2half2_rn(x, y);
  } else {
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(out) + i) = __floats2bfloat162_rn(x, y);
  }
}

template <int D, int NB, bool kDup, bool kSplit>
__global__ void __launch_bounds__(kThreads) decode_kv4_kernel(const __grid_constant__ DecodeParams p, int q_dtype,
                                                              int out_dtype, const Kv4Bits bits) {
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
  const int nparts = (L + p.part_tokens - 1) / p.part_tokens;

  uint4* q_frag = reinterpret_cast<uint4*>(smem + C::kMainBytes);
  float* q_undo = reinterpret_cast<float*>(smem + C::kMainBytes + C::kQueryBytes - C::kCols * 4);
  // ---- where each eight tokens' rows of this KV head start in the pools, in bytes
  int64_t* offs = reinterpret_cast<int64_t*>(smem + C::kMainBytes + C::kQueryBytes);
  {
    const int bs_log2 = 31 - __clz(p.block_size);
    const int64_t tile_bytes = static_cast<int64_t>(p.block_size) * C::kRow;
    const int32_t* row = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    for (int i = threadIdx.x; i < (ntok + 7) / 8; i += kThreads) {
      const int tok = t0 + 8 * i, col = tok >> bs_log2;
      int b = col < p.max_blocks_per_seq ? row[col] : -1;
      if (b < 0 || b >= p.num_blocks) {
        set_error(p.err, kErrIndex);
        b = 0;  // keep the copy in bounds; the flag reports the bad table
      }
      offs[i] = (static_cast<int64_t>(b) * p.num_kv_heads + kvh) * tile_bytes + (tok & (p.block_size - 1)) * C::kRow;
    }
  }
  __syncthreads();

  // ---- this lane's share of a tile's copies: pieces (lane & 15) + 16 i of its half
  unsigned char* ring = smem + warp * (C::kStages * C::kStage);
  const int half = lane >> 4, piece = lane & 15;
  const uint32_t ring_addr = smem_addr(ring) + half * 2 * C::kHalf + piece * 16;
  constexpr int kMixed = C::kHalfPieces / 16;  // the copy that brings the end of K and the start of V
  const unsigned char* kbase = static_cast<const unsigned char*>(p.k_cache) + piece * 16;
  const unsigned char* vbase = static_cast<const unsigned char*>(p.v_cache) + piece * 16 - C::kHalf;
  const unsigned char* mbase = 16 * kMixed + piece < C::kHalfPieces ? kbase : vbase;
  auto issue = [&](int tile, uint32_t to) {
    if (tile * kTile + kTile <= ntok) {
      const int64_t off = offs[2 * tile + half];
#pragma unroll
      for (int i = 0; i < C::kCopies; ++i)
        if (16 * (i + 1) <= 2 * C::kHalfPieces || 16 * i + piece < 2 * C::kHalfPieces)
          cp_async16(to + i * 256, (i < kMixed ? kbase : i == kMixed ? mbase : vbase) + off + i * 256);
    } else if (tile * kTile < ntok) {  // the last tile: a half past the end is filled with zeros
      const bool have = tile * kTile + 8 * half < ntok;
      const int64_t off = offs[have ? 2 * tile + half : 2 * tile];
#pragma unroll
      for (int i = 0; i < C::kCopies; ++i)
        if (16 * (i + 1) <= 2 * C::kHalfPieces || 16 * i + piece < 2 * C::kHalfPieces)
          cp_async16(to + i * 256, (i < kMixed ? kbase : i == kMixed ? mbase : vbase) + off + i * 256, have ? 16u : 0u);
    }
    cp_async_commit();  // one group per call, empty past the end: the waits below count them
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) issue(warp + i * kWarps, ring_addr + i * C::kStage);

  // ---- queries
  stage_queries<D, NB, kSplit>(p.q, q_dtype, out_row, G, q_frag, q_undo);
  __syncthreads();
  uint4 qh[NB][D / 32], ql[NB][kSplit ? D / 32 : 1];
  float sc[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int at = kDup ? (g & 3) * 4 + t : lane;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      qh[nb][w] = q_frag[(nb * (kSplit ? 2 : 1) * (D / 32) + w) * 32 + at];
      if (kSplit) ql[nb][w] = q_frag[((nb * 2 + 1) * (D / 32) + w) * 32 + at];
    }
    const int col = kDup ? 2 * (t & 1) : nb * 8 + 2 * t;
    sc[nb][0] = q_undo[col] * p.scale_log2;
    sc[nb][1] = q_undo[col + 1] * p.scale_log2;
  }

  float m[NB][2], l[NB][2], o[NB][D / 16][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
  }

  uint32_t at = 0, refill = (C::kStages - 1) * C::kStage;  // stages, as offsets into the ring
  auto step = [&](int tile, auto last) {
    constexpr bool kLast = decltype(last)::value;  // the tile may end past the context
    cp_async_wait<C::kStages - 2>();
    __syncwarp();  // the other lanes' copies too; and everybody has left the stage refilled next
    issue(tile + (C::kStages - 1) * kWarps, ring_addr + refill);
    refill = at;
    const unsigned char* ks = ring + at;
    at = at == (C::kStages - 1) * C::kStage ? 0 : at + C::kStage;
    const int left = kLast ? ntok - tile * kTile : kTile;  // tokens of this tile

    // ---- scores
    float c[NB][2][4];
    {
      constexpr int kWords = D / 32;
      uint32_t w0[kWords], w1[kWords];
      const unsigned char* r0 = ks + g * C::kRow;
      if constexpr (kWords == 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(r0 + t * 16);
        const uint4 b = *reinterpret_cast<const uint4*>(r0 + 2 * C::kHalf + t * 16);
        w0[0] = a.x; w0[1] = a.y; w0[2] = a.z; w0[3] = a.w;
        w1[0] = b.x; w1[1] = b.y; w1[2] = b.z; w1[3] = b.w;
      } else {
        const uint2 a = *reinterpret_cast<const uint2*>(r0 + t * 8);
        const uint2 b = *reinterpret_cast<const uint2*>(r0 + 2 * C::kHalf + t * 8);
        w0[0] = a.x; w0[1] = a.y;
        w1[0] = b.x; w1[1] = b.y;
      }
      const int pair = D / 2 + 4 * (t * D / 128);
      const __half2 p0 = *reinterpret_cast<const __half2*>(r0 + pair);
      const __half2 p1 = *reinterpret_cast<const __half2*>(r0 + 2 * C::kHalf + pair);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t a[4], b[4];
        kv4_word(w0[i], __low2half2(p0), __high2half2(p0), bits, a);
        kv4_word(w1[i], __low2half2(p1), __high2half2(p1), bits, b);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (i == 0) {
            mma_f16_first(c[nb][0], a[0], b[0], a[1], b[1], qh[nb][i].x, qh[nb][i].y);
            mma_f16_first(c[nb][1], a[2], b[2], a[3], b[3], qh[nb][i].z, qh[nb][i].w);
          } else {
            mma_f16(c[nb][0], a[0], b[0], a[1], b[1], qh[nb][i].x, qh[nb][i].y);
            mma_f16(c[nb][1], a[2], b[2], a[3], b[3], qh[nb][i].z, qh[nb][i].w);
          }
          if (kSplit) {
            mma_f16(c[nb][0], a[0], b[0], a[1], b[1], ql[nb][i].x, ql[nb][i].y);
            mma_f16(c[nb][1], a[2], b[2], a[3], b[3], ql[nb][i].z, ql[nb][i].w);
          }
        }
      }
    }

    // ---- softmax; tokens past the end get -inf
    uint32_t ph[NB][2], pl[NB][2];  // P^T fragments: tokens 0-7 and 8-15
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x[4];  // score - m + 6
      const float ma = kLift - m[nb][0], mb = kLift - m[nb][1];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fmaf(c[nb][0][i] + c[nb][1][i], sc[nb][i & 1], i & 1 ? mb : ma);
      if (kLast) {
        if (g >= left) x[0] = x[1] = -INFINITY;
        if (g + 8 >= left) x[2] = x[3] = -INFINITY;
      }
      if (__any_sync(0xffffffffu, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) > kLift + kSlack)) {
        // raise both columns' maxima: scores again (m = -inf makes x = inf), their largest
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[i] = kLast && g + (i & 2) * 4 >= left ? -INFINITY : (c[nb][0][i] + c[nb][1][i]) * sc[nb][i & 1];
        float a = fmaxf(y[0], y[2]), b = fmaxf(y[1], y[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
          b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
        }
        a = fmaxf(a, m[nb][0]);
        b = fmaxf(b, m[nb][1]);
        // a column that saw nothing but NaN yet keeps m = -inf, and its NaN sum
        const float fa = a == m[nb][0] ? 1.f : exp2_approx(m[nb][0] - a);
        const float fb = b == m[nb][1] ? 1.f : exp2_approx(m[nb][1] - b);
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
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i] - (i & 1 ? b : a) + kLift;
      }
      const float e0 = exp2_approx(x[0]), e1 = exp2_approx(x[1]), e2 = exp2_approx(x[2]), e3 = exp2_approx(x[3]);
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
        const int r = 2 * t + (i & 1) + (i & 2) * 4;  // rows 2t, 2t+1 of either half
        const unsigned char* row = ks + (i & 2 ? 3 : 1) * C::kHalf + (2 * t + (i & 1)) * C::kRow;
        if (kWords == 2) {
          const uint2 a = *reinterpret_cast<const uint2*>(row + g * 8);
          w[i][0] = a.x;
          w[i][kWords - 1] = a.y;
        } else {
          w[i][0] = *reinterpret_cast<const uint32_t*>(row + g * 4);
        }
        pr[i] = *reinterpret_cast<const uint32_t*>(row + D / 2 + 4 * (g * D / 256));
        // past the end a row holds anything, NaN too: step = lo = 0 makes it zero
        if (kLast && r >= left) pr[i] = 0u;
      }
      const __half2 step0 = as_half2(__byte_perm(pr[0], pr[1], 0x5410)), lo0 = as_half2(__byte_perm(pr[0], pr[1], 0x7632));
      const __half2 step1 = as_half2(__byte_perm(pr[2], pr[3], 0x5410)), lo1 = as_half2(__byte_perm(pr[2], pr[3], 0x7632));
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t sel = 0x4400u + 0x1111u * j;  // byte j of both words, twice each
          const uint32_t x0 = __byte_perm(w[0][i], w[1][i], sel), x1 = __byte_perm(w[2][i], w[3][i], sel);
          const uint32_t a0 = as_u32(__hfma2(low_codes(x0, bits), step0, lo0));
          const uint32_t a1 = as_u32(__hfma2(high_codes(x0, bits), step0, lo0));
          const uint32_t a2 = as_u32(__hfma2(low_codes(x1, bits), step1, lo1));
          const uint32_t a3 = as_u32(__hfma2(high_codes(x1, bits), step1, lo1));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_f16(o[nb][4 * i + j], a0, a1, a2, a3, ph[nb][0], ph[nb][1]);
            if (!kDup) mma_f16(o[nb][4 * i + j], a0, a1, a2, a3, pl[nb][0], pl[nb][1]);
          }
        }
      }
    }
  };
  int tile = warp;
  for (; (tile + 1) * kTile <= ntok; tile += kWarps) step(tile, std::false_type{});
  if (tile * kTile < ntok) step(tile, std::true_type{});
  cp_async_wait<0>();
  __syncthreads();  // every warp has left its ring: the sums take its place

  // ---- combine the warps in a fixed order.  O is exchanged as fragments, 16 bytes per lane:
  // lane (g, t), fragment i: dimensions d = g D/8 + 2i and d + 1 of columns 2t and 2t + 1
  float2* red_ml = reinterpret_cast<float2*>(smem);                     // [warps][cols]: (max, sum)
  float4* red_o = reinterpret_cast<float4*>(red_ml + kWarps * C::kCols);  // [warps][NB][D/16][32]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l[nb][0] += __shfl_xor_sync(0xffffffffu, l[nb][0], off);
      l[nb][1] += __shfl_xor_sync(0xffffffffu, l[nb][1], off);
    }
    if (g == 0) {
      red_ml[warp * C::kCols + nb * 8 + 2 * t] = make_float2(m[nb][0], l[nb][0]);
      red_ml[warp * C::kCols + nb * 8 + 2 * t + 1] = make_float2(m[nb][1], l[nb][1]);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      red_o[((warp * NB + nb) * (D / 16) + i) * 32 + lane] = make_float4(o[nb][i][0], o[nb][i][1], o[nb][i][2], o[nb][i][3]);
  }
  __syncthreads();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float f[2][kWarps], M[2], lsum[2];  // factors of the warps' sums, per column
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 ml[kWarps];
      M[e] = -INFINITY;
      lsum[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = red_ml[w * C::kCols + nb * 8 + 2 * t + e];
        M[e] = fmaxf(M[e], ml[w].x);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[e][w] = ml[w].y == 0.f ? 0.f : exp2_approx(ml[w].x - M[e]);  // 0: the warp saw no token
        lsum[e] = fmaf(f[e][w], ml[w].y, lsum[e]);
      }
    }
    const int h = kDup ? 2 * (t & 1) : nb * 8 + 2 * t;  // heads h and h + 1
#pragma unroll
    for (int i = warp; i < D / 16; i += kWarps) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = red_o[((w * NB + nb) * (D / 16) + i) * 32 + lane];
        acc.x = fmaf(f[0][w], x.x, acc.x);
        acc.y = fmaf(f[1][w], x.y, acc.y);
        acc.z = fmaf(f[0][w], x.z, acc.z);
        acc.w = fmaf(f[1][w], x.w, acc.w);
      }
      if (kDup) {  // the weights' second parts are in columns 4..7
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 2);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 2);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 2);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 2);
      }
      const int d = g * (D / 8) + 2 * i;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if ((kDup && t >= 2) || h + e >= G) continue;
        const float a = e ? acc.y : acc.x, b = e ? acc.w : acc.z;
        const size_t row = out_row + h + e;
        if (nparts == 1) {
          store_pair(p.out, row * D + d, a / lsum[e], b / lsum[e], out_dtype);
        } else {
          const size_t k = row * p.max_parts + part;
          *reinterpret_cast<float2*>(p.ws_o + k * D + d) = make_float2(a, b);
          if (i == 0 && g == 0) {
            p.ws_ml[2 * k] = M[e];
            p.ws_ml[2 * k + 1] = lsum[e];
          }
        }
      }
    }
  }
}

template <int D, int NB, bool kDup, bool kSplit>
cudaError_t launch_t(const DecodeParams& p, int q_dtype, int out_dtype, cudaStream_t stream) {
  using C = Kv4<D, NB, kDup, kSplit>;
  const size_t smem = C::kMainBytes + C::kQueryBytes + static_cast<size_t>(p.part_tokens / 8) * 8;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem_limit(decode_kv4_kernel<D, NB, kDup, kSplit>, 100 * 1024, configured);
  if (e != cudaSuccess) return e;
  dim3 grid(p.max_parts, p.num_kv_heads, p.num_seqs);
  decode_kv4_kernel<D, NB, kDup, kSplit><<<grid, kThreads, smem, stream>>>(p, q_dtype, out_dtype, Kv4Bits{});
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
