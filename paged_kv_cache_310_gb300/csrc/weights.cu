// weights.cu -- attention weights of a decode step, accumulated per cached token.
//
// For sequence s, KV head g and token j < n = context_lens[s]:
//   out[s][g][j] = (j < tracked[s] ? w[s][g][j] : 0) + sum_h softmax_j(scale * q_h . K_j),
// h over g's query heads.  The softmax needs its sum before any weight is known, so the
// scores are looked at twice:
//  * scores_kernel reads K once, a CTA per (partition, KV head, sequence): 16 tokens per
//    warp and step, as in the decode kernels; scores (fp32, log2 domain) go to the
//    workspace as [s][g][j][h] and each partition's (maximum, sum) beside them;
//  * weights_kernel joins the partitions' (maximum, sum) and adds up each token's weights.
// Bound: HBM: K's row (2 D bytes in 16 bits, 5 D / 8 in four), 8 bytes of accumulator and
// the scores' 8 G bytes, which mostly stay in L2 between the kernels.
//
// 16-bit pools go to m16n8k16 MMAs as they are, 4-bit ones are widened in registers
// (kv4.cuh), f32 ones are multiplied on CUDA cores in fp32.
#include "kv4.cuh"
#include "launch.h"
#include "mma.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;
constexpr int kFinishThreads = 256;
constexpr int kFinishTokens = 1024;  // tokens per CTA of weights_kernel

// Kinds of pool: PKV_F32, PKV_F16, PKV_BF16, PKV_KV4 (f16 and bf16 queries), kKv4Split
// (4-bit pool, f32 queries in two fp16 parts).
constexpr int kKv4Split = 4;

template <int KIND, int D>
struct KPool {
  static constexpr bool kIsKv4 = KIND >= PKV_KV4;
  static constexpr int kRow = kIsKv4 ? D * 5 / 8 : D * (KIND == PKV_F32 ? 4 : 2);
  static constexpr int kHalf = 8 * kRow;
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kChunks = kStage / 16;
  static constexpr int kPerLane = (kChunks + 31) / 32;
  static constexpr int kRowChunks = kRow / 16;  // wide kinds
  static constexpr int kStages = kStage >= 8192 ? 3 : kStage >= 4096 ? 4 : 8;
  static constexpr int kRingBytes = kWarps * kStages * kStage;
  // shared offset of 16-byte piece c of a stage: wide rows are a multiple of 128 bytes, so
  // odd rows swap the halves of each 128 bytes and eight lanes of two rows never share banks
  __device__ static int place(int c) {
    return (kIsKv4 ? c : c ^ (((c / (kIsKv4 ? 1 : kRowChunks)) & 1) << 2)) * 16;
  }
};

template <int KIND, int D, int NB>
__global__ void __launch_bounds__(kThreads) scores_kernel(const __grid_constant__ WeightsParams p) {
  using C = KPool<KIND, D>;
  extern __shared__ __align__(128) unsigned char smem[];
  grid_dependents_launch();  // weights_kernel, which waits for this grid

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
  const int ntiles = (ntok + kTile - 1) / kTile;
  const size_t q_row = static_cast<size_t>(s) * p.num_q_heads + static_cast<size_t>(kvh) * G;

  float* q_smem = reinterpret_cast<float*>(smem + C::kRingBytes);  // f32 pools: [G][D]
  int* ids = reinterpret_cast<int*>(smem + C::kRingBytes + (KIND == PKV_F32 ? NB * 8 * D * 4 : 0));
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
    if (KIND == PKV_F32)
      for (int i = threadIdx.x; i < NB * 8 * D; i += kThreads)
        q_smem[i] = i < G * D ? static_cast<const float*>(p.q)[q_row * D + i] : 0.f;
  }
  __syncthreads();

  unsigned char* ring = smem + warp * (C::kStages * C::kStage);
  const uint32_t ring_addr = smem_addr(ring);
  const int64_t tile_bytes = static_cast<int64_t>(p.block_size) * C::kRow;
  const int64_t block_bytes = tile_bytes * p.num_kv_heads;
  const unsigned char* pool = static_cast<const unsigned char*>(p.k_cache) + tile_bytes * kvh;
  auto issue = [&](int tile, int stage) {
    if (tile < ntiles) {
      const int tok0 = tile * kTile, tok1 = tok0 + 8;
      const bool have1 = tok1 < ntok;
      const int at1 = have1 ? tok1 : tok0;
      const unsigned char* src0 = pool + ids[tok0 >> bs_log2] * block_bytes + (tok0 & (p.block_size - 1)) * C::kRow;
      const unsigned char* src1 = pool + ids[at1 >> bs_log2] * block_bytes + (at1 & (p.block_size - 1)) * C::kRow;
#pragma unroll
      for (int i = 0; i < C::kPerLane; ++i) {
        const int c = lane + 32 * i;
        if (C::kChunks % 32 == 0 || c < C::kChunks) {
          const bool second = c >= C::kChunks / 2;
          const unsigned char* src = (second ? src1 : src0) + (c - (second ? C::kChunks / 2 : 0)) * 16;
          cp_async16(ring_addr + stage * C::kStage + C::place(c), src, second && !have1 ? 0u : 16u);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) issue(warp + i * kWarps, i);

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

  float m[NB][2], l[NB][2];  // this lane's rows of its columns only
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.f;
  }
  float* scores = p.scores + ((static_cast<size_t>(s) * p.num_kv_heads + kvh) * p.max_len + t0) * G;

  int stage = 0;
  for (int tile = warp; tile < ntiles; tile += kWarps) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();
    issue(tile + (C::kStages - 1) * kWarps, stage == 0 ? C::kStages - 1 : stage - 1);
    const unsigned char* ks = ring + stage * C::kStage;
    stage = stage + 1 == C::kStages ? 0 : stage + 1;
    const int left = ntok - tile * kTile;

    float x[NB][4];  // rows g, g + 8; columns 2t, 2t + 1
    if constexpr (kMma) {
      float c[NB][2][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[nb][0][i] = c[nb][1][i] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t a[4], b[4];  // rows g and g + 8: step 2i (0, 1), step 2i + 1 (2, 3)
        if constexpr (C::kIsKv4) {
          const unsigned char* r0 = ks + g * C::kRow;
          const int pair = D / 2 + 4 * (t * D / 128), word = t * (D / 8) + 4 * i;
          const __half2 p0 = *reinterpret_cast<const __half2*>(r0 + pair);
          const __half2 p1 = *reinterpret_cast<const __half2*>(r0 + C::kHalf + pair);
          kv4_word(*reinterpret_cast<const uint32_t*>(r0 + word), __low2half2(p0), __high2half2(p0), p.bits, a);
          kv4_word(*reinterpret_cast<const uint32_t*>(r0 + C::kHalf + word), __low2half2(p1), __high2half2(p1), p.bits, b);
        } else {
          const uint4 v0 = *reinterpret_cast<const uint4*>(ks + C::place(g * C::kRowChunks + t + 4 * i));
          const uint4 v1 = *reinterpret_cast<const uint4*>(ks + C::place((g + 8) * C::kRowChunks + t + 4 * i));
          a[0] = v0.x; a[1] = v0.y; a[2] = v0.z; a[3] = v0.w;
          b[0] = v1.x; b[1] = v1.y; b[2] = v1.z; b[3] = v1.w;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (KIND == PKV_BF16) {
            mma_bf16(c[nb][0], a[0], b[0], a[1], b[1], qh[nb][2 * i][0], qh[nb][2 * i][1]);
            mma_bf16(c[nb][1], a[2], b[2], a[3], b[3], qh[nb][2 * i + 1][0], qh[nb][2 * i + 1][1]);
          } else {
            mma_f16(c[nb][0], a[0], b[0], a[1], b[1], qh[nb][2 * i][0], qh[nb][2 * i][1]);
            mma_f16(c[nb][1], a[2], b[2], a[3], b[3], qh[nb][2 * i + 1][0], qh[nb][2 * i + 1][1]);
          }
          if constexpr (kSplit) {
            mma_f16(c[nb][0], a[0], b[0], a[1], b[1], ql[nb][2 * i][0], ql[nb][2 * i][1]);
            mma_f16(c[nb][1], a[2], b[2], a[3], b[3], ql[nb][2 * i + 1][0], ql[nb][2 * i + 1][1]);
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nb][i] = c[nb][0][i] + c[nb][1][i];
    } else {
      // fp32: lane t multiplies its quarter of rows g and g + 8 with every head's, then the
      // four lanes add up and each keeps its two columns
      float4 v0[D / 16], v1[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        v0[i] = *reinterpret_cast<const float4*>(ks + C::place(g * C::kRowChunks + t + 4 * i));
        v1[i] = *reinterpret_cast<const float4*>(ks + C::place((g + 8) * C::kRowChunks + t + 4 * i));
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          if (nb * 8 + h >= G) break;  // warp-uniform
          float a = 0.f, b = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const float4 qv = *reinterpret_cast<const float4*>(q_smem + (nb * 8 + h) * D + (t + 4 * i) * 4);
            a = fmaf(v0[i].x, qv.x, a); b = fmaf(v1[i].x, qv.x, b);
            a = fmaf(v0[i].y, qv.y, a); b = fmaf(v1[i].y, qv.y, b);
            a = fmaf(v0[i].z, qv.z, a); b = fmaf(v1[i].z, qv.z, b);
            a = fmaf(v0[i].w, qv.w, a); b = fmaf(v1[i].w, qv.w, b);
          }
          a = group_sum<4>(a);
          b = group_sum<4>(b);
          if (t == h / 2) {
            x[nb][h & 1] = a;
            x[nb][2 + (h & 1)] = b;
          }
        }
      }
    }

#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int col = nb * 8 + 2 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = g + (i & 2) * 4, h = col + (i & 1), e = i & 1;
        if (r < left && h < G) {
          const float y = x[nb][i] * sc[nb][e];
          scores[static_cast<size_t>(tile * kTile + r) * G + h] = y;
          if (y > m[nb][e]) {
            l[nb][e] *= exp2f(m[nb][e] - y);
            m[nb][e] = y;
          }
          // nothing seen yet but -inf: no weight (a NaN stays)
          l[nb][e] += y == -INFINITY && m[nb][e] == -INFINITY ? 0.f : exp2f(y - m[nb][e]);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---- (maximum, sum) of the partition, in a fixed order
  float* red = reinterpret_cast<float*>(smem);  // [warps][columns][2]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float M = m[nb][e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      float sum = l[nb][e] == 0.f ? 0.f : l[nb][e] * exp2f(m[nb][e] - M);
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
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[(w * NB * 8 + threadIdx.x) * 2]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* r = red + (w * NB * 8 + threadIdx.x) * 2;
      if (r[1] != 0.f) sum += r[1] * exp2f(r[0] - M);
    }
    float* ml = p.ws_ml + ((q_row + threadIdx.x) * p.max_parts + part) * 2;
    ml[0] = M;
    ml[1] = sum;
  }
}

// One CTA per (1,024 tokens, KV head, sequence).
__global__ void __launch_bounds__(kFinishThreads) weights_kernel(const __grid_constant__ WeightsParams p) {
  __shared__ float top[16], inverse[16];
  grid_dependency_wait();
  const int kvh = blockIdx.y, s = blockIdx.z, G = p.group;
  const int L = p.context_lens[s];
  const int j0 = blockIdx.x * kFinishTokens;
  if (L < 0 || L > p.max_len || j0 >= L) return;
  const int np = (L + p.part_tokens - 1) / p.part_tokens;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int h = warp; h < G; h += kFinishThreads / 32) {
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) +
                       (static_cast<size_t>(s) * p.num_q_heads + static_cast<size_t>(kvh) * G + h) * p.max_parts;
    float M = -INFINITY, sum = 0.f;
    for (int i = lane; i < np; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int i = lane; i < np; i += 32)
      if (ml[i].y != 0.f) sum += ml[i].y * exp2f(ml[i].x - M);
    sum = group_sum<32>(sum);
    if (lane == 0) {
      top[h] = M;
      inverse[h] = 1.f / sum;
    }
  }
  __syncthreads();
  const size_t row = static_cast<size_t>(s) * p.num_kv_heads + kvh;
  const float* scores = p.scores + row * p.max_len * G;
  const int end = min(L, j0 + kFinishTokens);
  const int tracked = p.tracked_lens ? p.tracked_lens[s] : L;
  for (int j = j0 + threadIdx.x; j < end; j += kFinishThreads) {
    float w = 0.f;
    for (int h = 0; h < G; ++h) w = fmaf(exp2f(scores[static_cast<size_t>(j) * G + h] - top[h]), inverse[h], w);
    const size_t at = row * p.width + j;
    p.weights_out[at] = (j < tracked ? p.weights[at] : 0.f) + w;
  }
}

template <int KIND, int D, int NB>
cudaError_t launch_t(const WeightsParams& p, cudaStream_t stream) {
  using C = KPool<KIND, D>;
  const size_t smem = C::kRingBytes + (KIND == PKV_F32 ? NB * 8 * D * 4 : 0) +
                      static_cast<size_t>(p.part_tokens / p.block_size) * 4;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem_limit(scores_kernel<KIND, D, NB>, 160 * 1024, configured);
  if (e != cudaSuccess) return e;
  scores_kernel<KIND, D, NB><<<dim3(p.max_parts, p.num_kv_heads, p.num_seqs), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
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
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.max_len + kFinishTokens - 1) / kFinishTokens, p.num_kv_heads, p.num_seqs);
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_kernel, p);
}

}  // namespace pkv
