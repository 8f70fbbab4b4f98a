// evict.cu -- eviction by accumulated attention weight.
//
// Of a sequence's n rows, each KV head keeps k = min(keep, n): the last r = min(recent, k)
// and, of the others, the k - r with the largest accumulated weight (NaN counts as
// -infinity; equal weights: the lowest row first).  Kept rows keep their order.
//  * select_kernel, one CTA per (KV head, sequence): the (k - r)-th largest weight by radix
//    selection (up to four passes of eight bits over order-preserving integer keys, held in
//    shared memory up to 48 Ki rows), then one ordered pass that writes the kept rows'
//    indices and weights.  A row's place is the number of heavier rows before it plus the
//    number of equal ones, the latter held at how many of them are kept: one prefix sum of
//    two packed counts.  Bound: the latency of its passes, not bytes.
//  * move_kernel copies the kept rows of K and V into the sequence's new blocks, 16 bytes
//    (8 where rows are 40) per thread.  Bound: HBM; each kept row is read and written once.
#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kPerThread = 4;  // rows per thread and step of the ordered pass
constexpr int kMaxKeys = 48 * 1024;  // rows whose keys fit in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;  // kept rows per CTA

// Larger weight, larger key; -0 as +0; NaN as -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w != w ? -INFINITY : w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t found[3];  // digit, rows still to take among it, rows that have it
  extern __shared__ uint32_t keys[];
  grid_dependency_wait();    // of the kernel before: only this one's launch overlaps it
  grid_dependents_launch();  // move_kernel, which waits for this grid
  const int kvh = blockIdx.x, s = blockIdx.y;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int n = p.context_lens[s], keep = p.keep_lens[s];
  if (n < 0 || n > p.max_len || keep < 0 || min(keep, n) > p.max_keep) {
    if (kvh == 0 && tid == 0) set_error(p.err, kErrLength);
    return;
  }
  const int k = min(keep, n), r = min(p.recent, k);
  const int candidates = n - r;
  const size_t row = static_cast<size_t>(s) * p.num_kv_heads + kvh;
  const float* w = p.weights + row * p.width;

  // ---- the threshold: keys above it are kept, and the first `ties` of those equal to it
  uint32_t threshold = 0, ties = 0;
  if (k - r == 0) {
    threshold = 0xffffffffu;  // no key is above it
  } else if (k - r < candidates) {
    const bool held = candidates <= p.key_room;
    if (held) {
      constexpr int kBatch = 8;  // loads in flight per thread
      for (int j0 = tid; j0 < candidates; j0 += kSelectThreads * kBatch) {
        float x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) x[i] = j0 + i * kSelectThreads < candidates ? w[j0 + i * kSelectThreads] : 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (j0 + i * kSelectThreads < candidates) keys[j0 + i * kSelectThreads] = weight_key(x[i]);
      }  // each thread reads back only what it wrote
    }
    uint32_t need = k - r;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = tid; j < candidates; j += kSelectThreads) {
        const uint32_t key = held ? keys[j] : weight_key(w[j]);
        if (shift == 24 || (key >> (shift + 8)) == (threshold >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1u);
      }
      __syncthreads();
      if (warp == 0) {
        // lane 0 holds the eight largest digits: the digit whose rows from the top reach `need`
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = hist[255 - (lane * 8 + i)];
          sum += c[i];
        }
        uint32_t above = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, above, off);
          if (lane >= off) above += x;
        }
        above -= sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < need && above + c[i] >= need) {
            found[0] = 255 - (lane * 8 + i);
            found[1] = need - above;
            found[2] = c[i];
          }
          above += c[i];
        }
      }
      __syncthreads();
      threshold |= found[0] << shift;
      need = found[1];
      const bool all = found[2] == need;  // every row with these digits is kept: no need to look further
      __syncthreads();
      if (all) {
        threshold -= 1;  // >= 0x007fffff here, the key of -infinity
        need = 0;
        break;
      }
    }
    ties = need;
  }

  // ---- the kept rows in order
  int32_t* kept = p.kept + row * p.max_keep;
  float* out = p.weights_out + row * p.width;
  uint32_t above_before = 0, ties_before = 0;  // in the steps done
  float x[kPerThread], ahead[kPerThread];
  auto load = [&](int j0, float (&to)[kPerThread]) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int j = j0 + tid * kPerThread + i;
      to[i] = j < n ? w[j] : 0.f;
    }
  };
  load(0, ahead);
  for (int j0 = 0; j0 < n; j0 += kSelectThreads * kPerThread) {
    const int j = j0 + tid * kPerThread;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) x[i] = ahead[i];
    load(j0 + kSelectThreads * kPerThread, ahead);
    uint32_t count = 0, flag[kPerThread];  // rows above the threshold, and ties << 16
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const uint32_t key = weight_key(x[i]);
      flag[i] = j + i >= n ? 0u : j + i >= candidates || key > threshold ? 1u : key == threshold && ties ? 0x10000u : 0u;
      count += flag[i];
    }
    uint32_t scan = count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, scan, off);
      if (lane >= off) scan += y;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    uint32_t total = warp_sum[lane], before = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += y;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, before, 31);
    before = __shfl_sync(0xffffffffu, before - total, warp) + scan - count;
    __syncthreads();  // warp_sum is written again
    uint32_t a = above_before + (before & 0xffffu), e = ties_before + (before >> 16);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (flag[i] == 1u || (flag[i] && e < ties)) {
        const uint32_t at = a + min(e, ties);
        kept[at] = j + i;
        out[at] = x[i];
      }
      a += flag[i] & 0xffffu;
      e += flag[i] >> 16;
    }
    above_before += all & 0xffffu;
    ties_before += all >> 16;
  }
}

template <typename V>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictParams p) {
  grid_dependency_wait();
  const int kvh = blockIdx.y, s = blockIdx.z;
  const int n = p.context_lens[s], keep = p.keep_lens[s];
  if (n < 0 || n > p.max_len || keep < 0 || min(keep, n) > p.max_keep) return;
  const int k = min(keep, n), i0 = blockIdx.x * kMoveRows;
  if (i0 >= k) return;
  const int rows = min(kMoveRows, k - i0);
  const int bs_log2 = 31 - __clz(p.block_size), bs_mask = p.block_size - 1;
  const int32_t* kept = p.kept + (static_cast<size_t>(s) * p.num_kv_heads + kvh) * p.max_keep;
  const int32_t* from = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
  const int32_t* to = p.new_tables + static_cast<size_t>(s) * p.max_new_blocks;
  const int vecs = p.row_bytes / static_cast<int>(sizeof(V));
  V* kc = static_cast<V*>(p.k_cache);
  V* vc = static_cast<V*>(p.v_cache);
  for (int x = threadIdx.x; x < rows * vecs; x += kMoveThreads) {
    const int i = i0 + x / vecs, c = x % vecs;
    const int j = kept[i];
    const int src = (j >> bs_log2) < p.max_blocks_per_seq ? from[j >> bs_log2] : -1;
    const int dst = (i >> bs_log2) < p.max_new_blocks ? to[i >> bs_log2] : -1;
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
      set_error(p.err, kErrIndex);
      continue;
    }
    const int64_t a = ((static_cast<int64_t>(src) * p.num_kv_heads + kvh) * p.block_size + (j & bs_mask)) * vecs + c;
    const int64_t b = ((static_cast<int64_t>(dst) * p.num_kv_heads + kvh) * p.block_size + (i & bs_mask)) * vecs + c;
    const V kx = kc[a], vx = vc[a];
    kc[b] = kx;
    vc[b] = vx;
  }
}

template <typename V>
cudaError_t launch_move(const EvictParams& p, cudaStream_t stream) {
  const int most = p.max_keep < p.max_len ? p.max_keep : p.max_len;  // rows a sequence may keep
  if (most == 0) return cudaSuccess;
  return launch_dependent(move_kernel<V>, dim3((most + kMoveRows - 1) / kMoveRows, p.num_kv_heads, p.num_seqs),
                          kMoveThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_evict(EvictParams p, cudaStream_t stream) {
  p.key_room = p.max_len < kMaxKeys ? p.max_len : kMaxKeys;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem_limit(select_kernel, kMaxKeys * 4, configured);
  if (e != cudaSuccess) return e;
  e = launch_dependent(select_kernel, dim3(p.num_kv_heads, p.num_seqs), kSelectThreads, p.key_room * 4, stream, p);
  if (e != cudaSuccess) return e;
  return p.row_bytes % 16 == 0 ? launch_move<uint4>(p, stream) : launch_move<uint2>(p, stream);
}

}  // namespace pkv
