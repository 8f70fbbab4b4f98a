// weights.cu -- attention weights of a decode step, accumulated per cached token.
//
// For sequence s, KV head g and token j < n = context_lens[s]:
//   out[s][g][j] = (j < tracked[s] ? w[s][g][j] : 0) + sum_h softmax_j(scale * q_h . K_j),
// h over g's query heads.  The softmax needs its sum before any weight is known, so the
// scores are looked at twice:
//  * scores_kernel reads K once, a CTA per (partition, KV head, sequence): 16 tokens (32 of
//    a 4-bit pool) per warp and step from a ring of cp.async stages; scores (fp32, log2
//    domain) go to the workspace, a row of tokens per query head, and each partition's
//    (maximum, sum) beside them;
//  * weights_kernel joins the partitions' (maximum, sum) and adds up each token's weights.
// Up to kWeightsOne tokens one CTA sees a (sequence, KV head) whole: the scores stay in its
// shared memory, it adds the weights up itself, and there is no second kernel or workspace
// (one sequence of 512 tokens, 64/8 heads, 4-bit: 5.6 us on the GPU in place of 7.7; at 1,000
// tokens a second kernel is ahead: 64 sequences, 32/8 heads, bf16, 25 us against 28).
// Floor: HBM: K's row (2 D bytes in 16 bits, 5 D / 8 in four), 8 bytes of accumulator.  The
// scores' 8 G bytes more stay in L2 between the kernels while a batch's are well below its
// 129 MB (K is read with an evict-first policy for that); a larger batch's go through HBM.
//
// Measured: 64 sequences of 128 to 2,048 tokens, 32/8 heads, bf16: 28.5 us a call, 0.76 of
// copy bandwidth (the rest: the second kernel's launch and latency).  8 of 20,000 to 32,768,
// 64/8 heads, 4-bit: 46.4 us, of which scores_kernel 36 at 4.0 TB/s, bound by instructions
// (220 per 16 tokens and eight heads, 104 of them widening), and weights_kernel 10; 32 of them,
// whose scores (216 MB) pass L2: 190 us; f32 queries: 53.  f32 pools, the first batch: 56 us, 0.79.
//
// 16-bit pools go to m16n8k16 MMAs as they are, 4-bit ones are widened in registers
// (kv4.cuh), f32 ones are multiplied on CUDA cores in fp32.
#include <cfloat>
#include <type_traits>

#include "kv4.cuh"
#include "launch.h"
#include "mma.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kFinishThreads = 256;
constexpr int kFinishTokens = 1024;  // tokens per CTA of weights_kernel

// Kinds of pool: PKV_F32, PKV_F16, PKV_BF16, PKV_KV4 (f16 and bf16 queries), kKv4Split
// (4-bit pool, f32 queries in two fp16 parts).
constexpr int kKv4Split = 4;

template <int KIND, int D>
struct KPool {
  static constexpr bool kIsKv4 = KIND >= PKV_KV4;
  static constexpr int kSub = KIND >= PKV_KV4 ? 2 : 1;  // MMA tiles of 16 tokens per step
  static constexpr int kTile = 16 * kSub;
  static constexpr int kEighths = 2 * kSub;  // groups of eight rows: never more than one block each
  static constexpr int kRow = kIsKv4 ? D * 5 / 8 : D * (KIND == PKV_F32 ? 4 : 2);
  static constexpr int kHalf = 8 * kRow;
  static constexpr int kPieces = kHalf / 16;
  static constexpr int kLanes = 32 / kEighths;  // lanes that bring eight rows
  static constexpr int kCopies = (kPieces + kLanes - 1) / kLanes;
  static constexpr int kStage = kEighths * kHalf;
  static constexpr int kStages = kStage >= 8192 ? 2 : 3;
  static constexpr int kRingBytes = kWarps * kStages * kStage;
  static constexpr int kRowPieces = kIsKv4 ? kPieces : kRow / 16;
  // Wide rows are a multiple of 128 bytes: odd rows swap the halves of each 128 bytes, so the
  // eight lanes of two rows that load together never share banks.
  static_assert(kIsKv4 || kLanes % kRowPieces == 0 || kRowPieces % kLanes == 0, "a copy's rows");
  __host__ __device__ static constexpr int swap(int row) { return kIsKv4 ? 0 : (row & 1) << 2; }
};

template <int KIND, int D, int NB>
__global__ void __launch_bounds__(kThreads) scores_kernel(const __grid_constant__ WeightsParams p) {
  using C = KPool<KIND, D>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ volatile uint32_t bit_patterns[3];
  __shared__ float2 join[kWeightsMaxGroup];  // (maximum, 1 / sum) of a query head
  grid_dependency_wait();    // of the kernel before: only this one's launch overlaps it
  grid_dependents_launch();  // weights_kernel, or another call's: it waits for this grid before it writes

  const int part = blockIdx.x, kvh = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int G = p.group;
  const int L = p.context_lens[s];
  if (L < 0 || L > p.max_len) {
    if (part == 0 && threadIdx.x == 0) set_error(p.err, kErrLength);
    return;
  }
  const int t0 = part * p.part_tokens;
  if (t0 >= L) return;
  const int ntok = min(p.part_tokens, L - t0);
  const size_t q_row = static_cast<size_t>(s) * p.num_q_heads + static_cast<size_t>(kvh) * G;

  float* q_smem = reinterpret_cast<float*>(smem + C::kRingBytes);  // f32 pools: [G][D]
  // where each eight tokens' rows of this KV head start in the pool, in bytes
  int64_t* offs = reinterpret_cast<int64_t*>(smem + C::kRingBytes + (KIND == PKV_F32 ? NB * 8 * D * 4 : 0));
  {
    const int bs_log2 = 31 - __clz(p.block_size);
    const int32_t* row = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    for (int i = threadIdx.x; i < (ntok + 7) / 8; i += kThreads) {
      const int tok = t0 + 8 * i, col = tok >> bs_log2;
      int b = col < p.max_blocks_per_seq ? row[col] : -1;
      if (b < 0 || b >= p.num_blocks) {
        set_error(p.err, kErrIndex);
        b = 0;  // keep the copy in bounds; the flag reports the bad table
      }
      offs[i] = ((static_cast<int64_t>(b) * p.num_kv_heads + kvh) * p.block_size + (tok & (p.block_size - 1))) * C::kRow;
    }
    if (KIND == PKV_F32)
      for (int i = threadIdx.x; i < NB * 8 * D; i += kThreads)
        q_smem[i] = i < G * D ? static_cast<const float*>(p.q)[q_row * D + i] : 0.f;
    if (threadIdx.x == 0) {  // in registers from here on: constant memory's port is slower
      bit_patterns[0] = p.bits.low;
      bit_patterns[1] = p.bits.high;
      bit_patterns[2] = p.bits.one;
    }
  }
  __syncthreads();
  Kv4Bits bits;
  bits.low = bit_patterns[0];
  bits.high = bit_patterns[1];
  bits.one = bit_patterns[2];

  unsigned char* ring = smem + warp * (C::kStages * C::kStage);
  const int eighth = lane / C::kLanes, piece = lane % C::kLanes;
  const uint32_t ring_addr = smem_addr(ring) + eighth * C::kHalf;
  const unsigned char* pool = static_cast<const unsigned char*>(p.k_cache) + piece * 16;
  const uint64_t policy = policy_evict_first();  // K is read once; the scores should stay in L2
  auto issue = [&](int tile, uint32_t stage) {
    const int tok = tile * C::kTile + 8 * eighth;
    if (tile * C::kTile < ntok) {
      const uint32_t bytes = tok < ntok ? 16u : 0u;  // eight rows past the end: zeros
      const unsigned char* src = pool + offs[(tok < ntok ? tok : tile * C::kTile) / 8];
#pragma unroll
      for (int i = 0; i < C::kCopies; ++i)
        if (C::kLanes * (i + 1) <= C::kPieces || C::kLanes * i + piece < C::kPieces) {
          // the piece's row: one for all lanes, or two where a row has fewer pieces than there are lanes
          const int row = C::kLanes * i / C::kRowPieces + (C::kLanes > C::kRowPieces ? piece / C::kRowPieces : 0);
          cp_async16_hint(ring_addr + stage + ((piece ^ C::swap(row)) + C::kLanes * i) * 16, src + i * C::kLanes * 16,
                          bytes, policy);
        }
    }
    cp_async_commit();  // one group per call, empty past the end: the waits below count them
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) issue(warp + i * kWarps, i * C::kStage);

  // ---- queries
  constexpr bool kMma = KIND != PKV_F32;
  constexpr bool kSplit = KIND == kKv4Split;
  uint32_t qh[NB][kMma ? D / 16 : 1][2], ql[NB][kSplit ? D / 16 : 1][2];
  float sc[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int h = nb * 8 + g;
    sc[nb][0] = sc[nb][1] = p.scale_log2;
    if constexpr (C::kIsKv4) {
      const float undo = load_q_kv4<D, kSplit>(p.q, p.q_dtype, q_row + h, h < G, t, qh[nb], ql[nb]) * p.scale_log2;
      sc[nb][0] = __shfl_sync(0xffffffffu, undo, 8 * t);
      sc[nb][1] = __shfl_sync(0xffffffffu, undo, 8 * t + 4);
    } else if constexpr (kMma) {
      // lane t brings the 16-byte pieces t, t + 4, ... of a row: piece t + 4 i gives steps 2i, 2i + 1
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (h < G) x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (q_row + h) * D)[t + 4 * i];
        qh[nb][2 * i][0] = x.x;
        qh[nb][2 * i][1] = x.y;
        qh[nb][2 * i + 1][0] = x.z;
        qh[nb][2 * i + 1][1] = x.w;
      }
    }
  }

  float m[NB][2], l[NB][2];  // the warp's maximum, this lane's rows' sum
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -FLT_MAX;  // not -infinity: -infinity less it is no NaN
    l[nb][0] = l[nb][1] = 0.f;
  }
  const bool one = p.scores == nullptr;  // one CTA sees all tokens: its scores stay in shared memory
  float* held = reinterpret_cast<float*>(offs + p.part_tokens / 8);
  float* column[NB][2];  // this lane's heads' rows of scores, and whether they are heads
  bool first_in[NB], second_in[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int h = nb * 8 + 2 * t;
    column[nb][0] = (one ? held + h * p.scores_ld : p.scores + (q_row + h) * p.scores_ld + t0) + g;
    column[nb][1] = column[nb][0] + p.scores_ld;
    first_in[nb] = h < G;
    second_in[nb] = h + 1 < G;
  }

  uint32_t at = 0, refill = (C::kStages - 1) * C::kStage;  // stages, as offsets into the ring
  auto step = [&](int tile, auto last) {
    constexpr bool kLast = decltype(last)::value;  // the tile may end past the context
    cp_async_wait<C::kStages - 2>();
    __syncwarp();  // the other lanes' copies too; and everybody has left the stage refilled next
    issue(tile + (C::kStages - 1) * kWarps, refill);
    refill = at;
    const unsigned char* ks = ring + at;
    at = at == (C::kStages - 1) * C::kStage ? 0 : at + C::kStage;
    const int left = kLast ? ntok - tile * C::kTile : C::kTile;

    float x[NB][C::kSub][4];  // rows g, g + 8 of each tile of 16; columns 2t, 2t + 1
#pragma unroll
    for (int u = 0; u < C::kSub; ++u) {
      const unsigned char* r0 = ks + 2 * u * C::kHalf + g * C::kRow;  // row g; row g + 8 is kHalf on
      if constexpr (kMma) {
        float c[NB][4];
        [[maybe_unused]] uint32_t w0[D / 32], w1[D / 32];
        [[maybe_unused]] __half2 p0, p1;
        if constexpr (C::kIsKv4) {
#pragma unroll
          for (int i = 0; i < D / 32; i += D / 32 > 2 ? 4 : 2) {
            if constexpr (D == 128) {
              const uint4 a = *reinterpret_cast<const uint4*>(r0 + t * 16);
              const uint4 b = *reinterpret_cast<const uint4*>(r0 + C::kHalf + t * 16);
              w0[0] = a.x; w0[1] = a.y; w0[D / 32 - 2] = a.z; w0[D / 32 - 1] = a.w;
              w1[0] = b.x; w1[1] = b.y; w1[D / 32 - 2] = b.z; w1[D / 32 - 1] = b.w;
            } else {
              const uint2 a = *reinterpret_cast<const uint2*>(r0 + t * 8);
              const uint2 b = *reinterpret_cast<const uint2*>(r0 + C::kHalf + t * 8);
              w0[0] = a.x; w0[1] = a.y;
              w1[0] = b.x; w1[1] = b.y;
            }
          }
          const int pair = D / 2 + 4 * (t * D / 128);
          p0 = *reinterpret_cast<const __half2*>(r0 + pair);
          p1 = *reinterpret_cast<const __half2*>(r0 + C::kHalf + pair);
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t a[4], b[4];  // rows g and g + 8: step 2i (0, 1), step 2i + 1 (2, 3)
          if constexpr (C::kIsKv4) {
            kv4_word(w0[i], __low2half2(p0), __high2half2(p0), bits, a);
            kv4_word(w1[i], __low2half2(p1), __high2half2(p1), bits, b);
          } else {
            const int off = ((t + 4 * i) ^ C::swap(g)) * 16;
            const uint4 v0 = *reinterpret_cast<const uint4*>(r0 + off);
            const uint4 v1 = *reinterpret_cast<const uint4*>(r0 + C::kHalf + off);
            a[0] = v0.x; a[1] = v0.y; a[2] = v0.z; a[3] = v0.w;
            b[0] = v1.x; b[1] = v1.y; b[2] = v1.z; b[3] = v1.w;
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint32_t *h0 = qh[nb][2 * i], *h1 = qh[nb][2 * i + 1];
            if constexpr (KIND == PKV_BF16) {
              if (i == 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) c[nb][e] = 0.f;
              }
              mma_bf16(c[nb], a[0], b[0], a[1], b[1], h0[0], h0[1]);
              mma_bf16(c[nb], a[2], b[2], a[3], b[3], h1[0], h1[1]);
            } else {
              if (i == 0)
                mma_f16_first(c[nb], a[0], b[0], a[1], b[1], h0[0], h0[1]);
              else
                mma_f16(c[nb], a[0], b[0], a[1], b[1], h0[0], h0[1]);
              mma_f16(c[nb], a[2], b[2], a[3], b[3], h1[0], h1[1]);
            }
            if constexpr (kSplit) {
              mma_f16(c[nb], a[0], b[0], a[1], b[1], ql[nb][2 * i][0], ql[nb][2 * i][1]);
              mma_f16(c[nb], a[2], b[2], a[3], b[3], ql[nb][2 * i + 1][0], ql[nb][2 * i + 1][1]);
            }
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[nb][u][i] = c[nb][i] * sc[nb][i & 1];
      } else {
        // fp32: lane t multiplies its quarter of rows g and g + 8 with every head's, then the
        // four lanes add up and each keeps its two columns
        float4 v0[D / 16], v1[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int off = ((t + 4 * i) ^ C::swap(g)) * 16;
          v0[i] = *reinterpret_cast<const float4*>(r0 + off);
          v1[i] = *reinterpret_cast<const float4*>(r0 + C::kHalf + off);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          x[nb][u][0] = x[nb][u][1] = x[nb][u][2] = x[nb][u][3] = 0.f;
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            if (nb * 8 + h >= G) break;  // warp-uniform
            float2 a = make_float2(0.f, 0.f), b = a;  // even and odd elements
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const float4 qv = *reinterpret_cast<const float4*>(q_smem + (nb * 8 + h) * D + (t + 4 * i) * 4);
              const float2 q0 = make_float2(qv.x, qv.y), q1 = make_float2(qv.z, qv.w);
              a = __ffma2_rn(make_float2(v0[i].x, v0[i].y), q0, a);
              b = __ffma2_rn(make_float2(v1[i].x, v1[i].y), q0, b);
              a = __ffma2_rn(make_float2(v0[i].z, v0[i].w), q1, a);
              b = __ffma2_rn(make_float2(v1[i].z, v1[i].w), q1, b);
            }
            const float sa = group_sum<4>(a.x + a.y), sb = group_sum<4>(b.x + b.y);
            if (t == h / 2) {
              x[nb][u][h & 1] = sa * p.scale_log2;
              x[nb][u][2 + (h & 1)] = sb * p.scale_log2;
            }
          }
        }
      }
    }

    // ---- store the scores; the warp's (maximum, sum) of its columns: the maximum is raised only
    // when a score exceeds it by 8 (log2 domain), so sums hold powers up to 2^8.  Columns past
    // the group come along (scores 0) and are used by nobody.
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float d[2][2 * C::kSub], top = -INFINITY;  // scores less the maximum
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* to = column[nb][e] + tile * C::kTile;
#pragma unroll
        for (int i = 0; i < 2 * C::kSub; ++i) {
          float& y = x[nb][i / 2][2 * (i & 1) + e];
          const bool in = !kLast || 8 * i + g < left;
          if (!in) y = -INFINITY;
          if (in && (e == 0 ? first_in[nb] : second_in[nb])) to[8 * i] = y;
          d[e][i] = y - m[nb][e];
          top = fmaxf(top, d[e][i]);
        }
      }
      if (__any_sync(0xffffffffu, top > 8.f)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = m[nb][e];
#pragma unroll
          for (int u = 0; u < C::kSub; ++u) M = fmaxf(M, fmaxf(x[nb][u][e], x[nb][u][2 + e]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
          if (M != m[nb][e]) l[nb][e] *= exp2_approx(m[nb][e] - M);
          m[nb][e] = M;
#pragma unroll
          for (int i = 0; i < 2 * C::kSub; ++i) d[e][i] = x[nb][i / 2][2 * (i & 1) + e] - M;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int u = 0; u < C::kSub; ++u) l[nb][e] += exp2_approx(d[e][2 * u]) + exp2_approx(d[e][2 * u + 1]);
    }
  };
  int tile = warp;
  for (; (tile + 1) * C::kTile <= ntok; tile += kWarps) step(tile, std::false_type{});
  if (tile * C::kTile < ntok) step(tile, std::true_type{});
  cp_async_wait<0>();
  __syncthreads();

  // ---- (maximum, sum) of the partition, in a fixed order
  float* red = reinterpret_cast<float*>(smem);  // [warps][columns][2]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float M = m[nb][e];
      float sum = l[nb][e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (g == 0) {
        float* r = red + (warp * NB * 8 + nb * 8 + 2 * t + e) * 2;
        r[0] = M;
        r[1] = sum;
      }
    }
  __syncthreads();
  if (threadIdx.x < G) {
    float M = -FLT_MAX, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[(w * NB * 8 + threadIdx.x) * 2]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* r = red + (w * NB * 8 + threadIdx.x) * 2;
      if (r[1] != 0.f) sum += r[1] * exp2_approx(r[0] - M);
    }
    if (one) {
      join[threadIdx.x] = make_float2(M, 1.f / sum);
    } else {
      float* ml = p.ws_ml + ((q_row + threadIdx.x) * p.max_parts + part) * 2;
      ml[0] = M;
      ml[1] = sum;
    }
  }
  if (one) {
    __syncthreads();
    const size_t row = (static_cast<size_t>(s) * p.num_kv_heads + kvh) * p.width;
    const int tracked = p.tracked_lens ? p.tracked_lens[s] : L;
    for (int j = threadIdx.x; j < L; j += kThreads) {
      const float before = j < tracked ? p.weights[row + j] : 0.f;
      float w = 0.f;
      for (int h = 0; h < G; ++h) w = fmaf(exp2_approx(held[h * p.scores_ld + j] - join[h].x), join[h].y, w);
      p.weights_out[row + j] = before + w;
    }
  }
}

// One CTA per (1,024 tokens, KV head, sequence); a thread adds up four tokens, 256 apart, so
// that every load and store is a whole line per warp whatever the rows' alignment.
// kWhole: all of the CTA's tokens are within the context (no test per load).
template <bool kWhole>
__device__ __forceinline__ void sum_weights(const WeightsParams& p, int s, int kvh, int L, float2* join) {
  const int G = p.group, j0 = blockIdx.x * kFinishTokens + threadIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const size_t row = static_cast<size_t>(s) * p.num_kv_heads + kvh;
  const int tracked = p.tracked_lens ? p.tracked_lens[s] : L;
  constexpr int kEach = kFinishTokens / kFinishThreads, kHeads = 4;
  // the first heads' scores and the accumulators are asked for before the partitions are joined
  float w[kEach], before[kEach], x[kHeads][kEach];
  const float* from = p.scores + row * G * p.scores_ld + j0;
  auto load = [&](int heads) {
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < heads) {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
          x[h][i] = kWhole || j0 + i * kFinishThreads < L ? from[i * kFinishThreads] : 0.f;
        from += p.scores_ld;
      }
  };
  load(G);
  const float* acc = p.weights + row * p.width + j0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = j0 + i * kFinishThreads;
    w[i] = 0.f;
    before[i] = (kWhole || j < L) && j < tracked ? acc[i * kFinishThreads] : 0.f;
  }
  const int np = (L + p.part_tokens - 1) / p.part_tokens;
  for (int h = warp; h < G; h += kFinishThreads / 32) {
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + (row * G + h) * p.max_parts;
    float M = -INFINITY, sum = 0.f;
    for (int i = lane; i < np; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int i = lane; i < np; i += 32)
      if (ml[i].y != 0.f) sum += ml[i].y * exp2_approx(ml[i].x - M);
    sum = group_sum<32>(sum);
    if (lane == 0) join[h] = make_float2(M, 1.f / sum);
  }
  __syncthreads();
  for (int h0 = 0; h0 < G; h0 += kHeads) {
    if (h0 > 0) load(G - h0);
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h0 + h < G) {
        const float2 ml = join[h0 + h];
#pragma unroll
        for (int i = 0; i < kEach; ++i) w[i] = fmaf(exp2_approx(x[h][i] - ml.x), ml.y, w[i]);
      }
  }
  float* out = p.weights_out + row * p.width + j0;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (kWhole || j0 + i * kFinishThreads < L) out[i * kFinishThreads] = before[i] + w[i];
}

__global__ void __launch_bounds__(kFinishThreads) weights_kernel(const __grid_constant__ WeightsParams p) {
  __shared__ float2 join[kWeightsMaxGroup];  // (maximum, 1 / sum) of a query head
  grid_dependency_wait();
  const int kvh = blockIdx.y, s = blockIdx.z;
  const int L = p.context_lens[s];
  const int j0 = blockIdx.x * kFinishTokens;
  if (L < 0 || L > p.max_len || j0 >= L) return;
  if (j0 + kFinishTokens <= L)
    sum_weights<true>(p, s, kvh, L, join);
  else
    sum_weights<false>(p, s, kvh, L, join);
}

template <int KIND, int D, int NB>
cudaError_t launch_t(const WeightsParams& p, cudaStream_t stream) {
  using C = KPool<KIND, D>;
  const size_t smem = C::kRingBytes + (KIND == PKV_F32 ? NB * 8 * D * 4 : 0) +
                      static_cast<size_t>(p.part_tokens) +  // 8 bytes per eight tokens
                      (p.scores ? 0 : p.group * p.scores_ld * sizeof(float));
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem_limit(scores_kernel<KIND, D, NB>, 160 * 1024, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(scores_kernel<KIND, D, NB>, dim3(p.max_parts, p.num_kv_heads, p.num_seqs), kThreads,
                          static_cast<int>(smem), stream, p);
}

template <int KIND>
cudaError_t launch_k(const WeightsParams& p, cudaStream_t stream) {
  if (p.group <= 8)
    return p.head_dim == 64 ? launch_t<KIND, 64, 1>(p, stream) : launch_t<KIND, 128, 1>(p, stream);
  return p.head_dim == 64 ? launch_t<KIND, 64, 2>(p, stream) : launch_t<KIND, 128, 2>(p, stream);
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, int dtype, cudaStream_t stream) {
  cudaError_t e;
  switch (dtype) {
    case PKV_F32: e = launch_k<PKV_F32>(p, stream); break;
    case PKV_F16: e = launch_k<PKV_F16>(p, stream); break;
    case PKV_BF16: e = launch_k<PKV_BF16>(p, stream); break;
    default: e = p.q_dtype == PKV_F32 ? launch_k<kKv4Split>(p, stream) : launch_k<PKV_KV4>(p, stream); break;
  }
  if (e != cudaSuccess || !p.scores) return e;
  return launch_dependent(weights_kernel,
                          dim3((p.max_len + kFinishTokens - 1) / kFinishTokens, p.num_kv_heads, p.num_seqs),
                          kFinishThreads, 0, stream, p);
}

}  // namespace pkv
