// evict.cu -- eviction by accumulated attention weight.
//
// Of a sequence's n rows, each KV head keeps k = min(keep, n): the last r = min(recent, k)
// and, of the others, the k - r with the largest accumulated weight (NaN counts as
// -infinity; equal weights: the lowest row first).  Kept rows keep their order.
//  * select_kernel, one CTA or a cluster of them per (KV head, sequence): the (k - r)-th
//    largest weight by radix selection (up to four passes of eight bits over
//    order-preserving integer keys, held in shared memory up to 48 Ki rows a CTA; a cluster
//    shares its rows out and adds up its CTAs' counts), then one ordered pass that writes the kept rows'
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
constexpr int kMoveRows = 32;  // kept rows per CTA

// Cluster-wide barrier, and a word of another CTA's shared memory.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* mine, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Larger weight, larger key; -0 as +0; NaN as -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w != w ? -INFINITY : w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[2][256];  // this CTA's counts, of even and odd passes
  __shared__ uint32_t counts[256];   // the cluster's
  __shared__ uint32_t totals[2];     // this CTA's rows above the threshold, and ties
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t found[3];  // digit, rows still to take among it, rows that have it
  extern __shared__ uint32_t keys[];
  grid_dependency_wait();    // of the kernel before: only this one's launch overlaps it
  grid_dependents_launch();  // move_kernel, which waits for this grid
  const int kvh = blockIdx.y, s = blockIdx.z;
  const uint32_t size = gridDim.x, rank = blockIdx.x;  // the cluster spans x
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int n = p.context_lens[s], keep = p.keep_lens[s];
  if (n < 0 || n > p.max_len || keep < 0 || min(keep, n) > p.max_keep) {
    if (kvh == 0 && rank == 0 && tid == 0) set_error(p.err, kErrLength);
    return;
  }
  const int k = min(keep, n), r = min(p.recent, k);
  const int candidates = n - r;
  const size_t row = static_cast<size_t>(s) * p.num_kv_heads + kvh;
  const float* w = p.weights + row * p.width;
  // this CTA's rows
  const int each = (n + static_cast<int>(size) - 1) / static_cast<int>(size);
  const int first = min(n, static_cast<int>(rank) * each), last = min(n, first + each);
  const int own = max(0, min(last, candidates) - first);  // of them, those chosen by weight

  // ---- the threshold: keys above it are kept, and the first `ties` of those equal to it
  uint32_t threshold = 0, ties = 0;
  if (k - r == 0) {
    threshold = 0xffffffffu;  // no key is above it
  } else if (k - r < candidates) {
    const bool held = own <= p.key_room;
    if (held) {
      constexpr int kBatch = 8;  // loads in flight per thread
      for (int j0 = tid; j0 < own; j0 += kSelectThreads * kBatch) {
        float x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) x[i] = j0 + i * kSelectThreads < own ? w[first + j0 + i * kSelectThreads] : 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (j0 + i * kSelectThreads < own) keys[j0 + i * kSelectThreads] = weight_key(x[i]);
      }  // each thread reads back only what it wrote
    }
    uint32_t need = k - r;
    if (tid < 256) hist[0][tid] = 0;
    for (int shift = 24, pass = 0; shift >= 0; shift -= 8, ++pass) {
      uint32_t* mine = hist[pass & 1];
      __syncthreads();
#pragma unroll 4
      for (int j = tid; j < own; j += kSelectThreads) {
        const uint32_t key = held ? keys[j] : weight_key(w[first + j]);
        if (shift == 24 || (key >> (shift + 8)) == (threshold >> (shift + 8))) atomicAdd(&mine[(key >> shift) & 255], 1u);
      }
      if (size > 1)
        cluster_barrier();
      else
        __syncthreads();
      if (tid < 256) {
        // the other buffer is free: everybody read it before arriving at the barrier
        hist[(pass & 1) ^ 1][tid] = 0;
        uint32_t c = mine[tid];
        for (uint32_t i = 1; i < size; ++i) c += cluster_load(mine + tid, (rank + i) % size);
        counts[tid] = c;
      }
      __syncthreads();
      if (warp == 0) {
        // lane 0 holds the eight largest digits: the digit whose rows from the top reach `need`
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = counts[255 - (lane * 8 + i)];
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
  auto flag_of = [&](int j, float x) {  // 1 above the threshold or recent, 1 << 16 a tie
    const uint32_t key = weight_key(x);
    return j >= last ? 0u : j >= candidates || key > threshold ? 1u : key == threshold && ties ? 0x10000u : 0u;
  };
  uint32_t above_before = 0, ties_before = 0;  // in the CTAs and steps before
  if (size > 1) {
    // count this CTA's first: their numbers tell the others where to begin
    if (tid < 2) totals[tid] = 0;
    __syncthreads();
    uint32_t above = 0, equal = 0;
    for (int j = first + tid; j < last; j += kSelectThreads) {
      const uint32_t f = flag_of(j, w[j]);
      above += f & 0xffffu;
      equal += f >> 16;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
      atomicAdd(&totals[0], above);
      atomicAdd(&totals[1], equal);
    }
    cluster_barrier();
    for (uint32_t i = 0; i < rank; ++i) {
      above_before += cluster_load(&totals[0], i);
      ties_before += cluster_load(&totals[1], i);
    }
  }
  int32_t* kept = p.kept + row * p.max_keep;
  float* out = p.weights_out + row * p.width;
  float x[kPerThread], ahead[kPerThread];
  auto load = [&](int j0, float (&to)[kPerThread]) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int j = j0 + tid * kPerThread + i;
      to[i] = j < last ? w[j] : 0.f;
    }
  };
  load(first, ahead);
  for (int j0 = first; j0 < last; j0 += kSelectThreads * kPerThread) {
    const int j = j0 + tid * kPerThread;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) x[i] = ahead[i];
    load(j0 + kSelectThreads * kPerThread, ahead);
    uint32_t count = 0, flag[kPerThread];  // rows above the threshold, and ties << 16
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      flag[i] = flag_of(j + i, x[i]);
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
  if (size > 1) cluster_barrier();  // nobody leaves while its counts may be read
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
  // A selection's passes are bound by its CTA's instructions (one of 32,767 rows: 20 us), so
  // few long ones are shared by up to eight CTAs each, as many as leave two CTAs per SM and
  // 4,096 rows each; a batch that fills the GPU by itself gains nothing (its barriers cost).
  const int64_t items = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads;
  int size = 1;
  while (size < 8 && items * size * 2 <= 2 * 152 && p.max_len / (size * 2) >= 4096) size *= 2;
  const int most = (p.max_len + size - 1) / size;
  p.key_room = most < kMaxKeys ? most : kMaxKeys;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem_limit(select_kernel, kMaxKeys * 4, configured);
  if (e != cudaSuccess) return e;
  const dim3 grid(size, p.num_kv_heads, p.num_seqs);
  if (size == 1) {
    e = launch_dependent(select_kernel, grid, kSelectThreads, p.key_room * 4, stream, p);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = p.key_room * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, select_kernel, p);
  }
  if (e != cudaSuccess) return e;
  return p.row_bytes % 16 == 0 ? launch_move<uint4>(p, stream) : launch_move<uint2>(p, stream);
}

}  // namespace pkv
