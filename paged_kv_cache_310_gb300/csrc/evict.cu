// evict.cu -- eviction by accumulated attention weight.
//
// Of a sequence's n rows, each KV head keeps k = min(keep, n): the last r = min(recent, k)
// and, of the others, the k - r with the largest accumulated weight (NaN counts as
// -infinity; equal weights: the lowest row first).  Kept rows keep their order.
//  * select_kernel, one CTA or a cluster of them per (KV head, sequence): the (k - r)-th
//    largest weight by radix selection (up to three passes of eleven bits over
//    order-preserving integer keys; weights are held in shared memory up to 48 Ki rows a CTA;
//    a cluster shares its rows out and adds up its CTAs' counts), then one ordered pass that
//    writes the kept rows' indices and weights.  A row's place is the number of heavier rows
//    before it plus the number of equal ones, the latter held at how many of them are kept:
//    ballots within a warp's 32 rows, one sum of two packed counts over the warps.  Bound: the
//    latency of its passes, not bytes: of 13 us for 32,767 rows in a cluster, 1.4 are the
//    load, 2 each pass, 1 the counts for the other CTAs, 4 the ordered pass.  Digits of eleven
//    bits (four passes of eight before) spread accumulators of similar size over more
//    counters (32 sequences of 512 to 4,096 rows, 8 heads: 81 us a call).
//  * move_kernel copies the kept rows of K and V into the sequence's new blocks, 16 bytes
//    (8 where rows are 40) per thread.  Bound: HBM; each kept row is read and written once:
//    69 us of that call, 413 MB, 6.0 TB/s (0.88 of copy bandwidth; the call with the selection
//    0.86 of its 70 us).  4-bit pools, whose rows are short: 38 us at D = 128 (floor 22), 32 at
//    D = 64 (12).
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kPerLane = 8;  // rows per lane and step of the ordered pass: a warp takes 32 at a time
constexpr int kDigits = 2048;  // eleven bits a pass
constexpr int kMaxKeys = 48 * 1024;  // rows whose weights fit in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;  // kept rows per CTA (that batch: 81 us; with 16, 86; with 64, 82)

// Cluster-wide barrier, and words of another CTA's shared memory.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_address(const void* mine, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(mine)), "r"(rank));
  return at;
}
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* mine, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_address(mine, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint2 cluster_load(const uint2* mine, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(cluster_address(mine, rank)) : "memory");
  return v;
}

__device__ __forceinline__ uint4 cluster_load(const uint4* mine, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_address(mine, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void unpack(const uint2& v, uint32_t (&x)[2]) { x[0] = v.x, x[1] = v.y; }
__device__ __forceinline__ void unpack(const uint4& v, uint32_t (&x)[4]) { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }

// Larger weight, larger key; -0 as +0; NaN as -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w != w ? -INFINITY : w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// kSize CTAs per (KV head, sequence): a cluster along x.
template <int kSize, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) select_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kBins = kDigits / kThreads;  // digits of a thread
  using Bins = std::conditional_t<kBins % 4 == 0, uint4, uint2>;  // read at once
  constexpr int kAtOnce = sizeof(Bins) / 4;
  static_assert(kBins % 2 == 0 && kWarps <= 32, "bins are read in pairs; one warp adds up the warps' sums");
  __shared__ __align__(16) uint32_t hist[2][kDigits];  // this CTA's counts, of even and odd passes
  __shared__ uint32_t totals[2];                       // this CTA's rows above the threshold, and ties
  __shared__ uint32_t warp_sum[kWarps];
  __shared__ uint32_t found[3];  // digit, rows still to take among it, rows that have it
  extern __shared__ float held_weights[];
  grid_dependency_wait();    // of the kernel before: only this one's launch overlaps it
  grid_dependents_launch();  // move_kernel, which waits for this grid
  const int kvh = blockIdx.y, s = blockIdx.z;
  const uint32_t rank = kSize > 1 ? blockIdx.x : 0;
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
  const int each = (n + kSize - 1) / kSize;
  const int first = min(n, static_cast<int>(rank) * each), last = min(n, first + each);
  const int own = max(0, min(last, candidates) - first);  // of them, those chosen by weight

  // ---- the threshold: keys above it are kept, and the first `ties` of those equal to it
  uint32_t threshold = k - r == 0 ? 0xffffffffu : 0, ties = 0;  // no key is above it, or every key
  bool held = false;
  if (k - r > 0 && k - r < candidates) {
    held = own <= p.key_room;
#pragma unroll
    for (int i = 0; i < kBins; ++i) hist[0][tid + i * kThreads] = 0;
    __syncthreads();
    constexpr int kBatch = 8;  // loads in flight per thread
    for (int j0 = tid; j0 < own; j0 += kThreads * kBatch) {
      float x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) x[i] = j0 + i * kThreads < own ? w[first + j0 + i * kThreads] : 0.f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (j0 + i * kThreads < own) {
          if (held) held_weights[j0 + i * kThreads] = x[i];
          atomicAdd(&hist[0][weight_key(x[i]) >> 21], 1u);
        }
    }
    uint32_t need = k - r;
    for (int pass = 0; pass < 3; ++pass) {  // bits 31..21, 20..10, 9..0
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      uint32_t* mine = hist[pass & 1];
      if (pass > 0) {
        const int above_bits = pass == 1 ? 21 : 10;
        const uint32_t mask = pass == 1 ? 2047u : 1023u;
#pragma unroll 4
        for (int j = tid; j < own; j += kThreads) {
          const uint32_t key = weight_key(held ? held_weights[j] : w[first + j]);  // what this thread put there
          if ((key >> above_bits) == (threshold >> above_bits)) atomicAdd(&mine[(key >> shift) & mask], 1u);
        }
      }
      if (kSize > 1)
        cluster_barrier();
      else
        __syncthreads();
      // the other buffer is free: everybody read it before arriving at the barrier
#pragma unroll
      for (int i = 0; i < kBins; ++i) hist[(pass & 1) ^ 1][tid + i * kThreads] = 0;
      // thread 0 holds the largest digits: the digit whose rows from the top reach `need`
      const int lowest = (kThreads - 1 - tid) * kBins;
      const Bins* bins = reinterpret_cast<const Bins*>(mine + lowest);
      uint32_t count[kBins], sum = 0;  // from its largest digit down
#pragma unroll
      for (int u = 0; u < kBins / kAtOnce; ++u) {
        Bins theirs[kSize];
        theirs[0] = bins[u];
#pragma unroll
        for (int i = 1; i < kSize; ++i) theirs[i] = cluster_load(bins + u, (rank + i) % kSize);
        uint32_t c[kAtOnce] = {};
#pragma unroll
        for (int i = 0; i < kSize; ++i) {
          uint32_t y[kAtOnce];
          unpack(theirs[i], y);
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) c[e] += y[e];
        }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          count[kBins - 1 - kAtOnce * u - e] = c[e];
          sum += c[e];
        }
      }
      uint32_t above = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, above, off);
        if (lane >= off) above += x;
      }
      if (lane == 31) warp_sum[warp] = above;
      __syncthreads();
      above += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u) - sum;
#pragma unroll
      for (int i = 0; i < kBins; ++i) {
        if (above < need && above + count[i] >= need) {
          found[0] = lowest + kBins - 1 - i;
          found[1] = need - above;
          found[2] = count[i];
        }
        above += count[i];
      }
      __syncthreads();
      threshold |= found[0] << shift;
      need = found[1];
      if (found[2] == need) {  // every row with these digits is kept: no need to look further
        threshold -= 1;        // >= 0x005fffff here: the key of -infinity is 0x007fffff
        need = 0;
        break;
      }
    }
    ties = need;
  }

  // ---- the kept rows in order
  uint32_t above_before = 0, ties_before = 0;  // in the CTAs and steps before
  if (kSize > 1) {
    // count this CTA's first: their numbers tell the others where to begin
    if (tid < 2) totals[tid] = 0;
    __syncthreads();
    uint32_t above = 0, equal = 0;
    if (k - r > 0) {
#pragma unroll 4
      for (int j = tid; j < own; j += kThreads) {
        const uint32_t key = weight_key(held ? held_weights[j] : w[first + j]);
        above += key > threshold;
        equal += key == threshold;
      }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
      atomicAdd(&totals[0], above);
      atomicAdd(&totals[1], equal);
    }
    cluster_barrier();
    const bool before = lane < static_cast<int>(rank);  // the recent rows come behind every other
    above = before ? cluster_load(&totals[0], lane) : 0u;
    equal = before ? cluster_load(&totals[1], lane) : 0u;
    above_before = __reduce_add_sync(0xffffffffu, above) + max(0, first - candidates);
    ties_before = ties ? __reduce_add_sync(0xffffffffu, equal) : 0u;
  }
  int32_t* kept = p.kept + row * p.max_keep;
  float* out = p.weights_out + row * p.width;
  constexpr int kStep = kThreads * kPerLane;
  for (int j0 = first; j0 < last; j0 += kStep) {
    const int j = j0 + warp * 32 * kPerLane + lane;
    float x[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int at = j + 32 * i;
      x[i] = at >= last ? 0.f : held && at - first < own ? held_weights[at - first] : w[at];
    }
    uint32_t heavy[kPerLane], equal[kPerLane], count = 0;  // masks of the warp's rows; their numbers, ties << 16
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int at = j + 32 * i;
      const uint32_t key = weight_key(x[i]);
      heavy[i] = __ballot_sync(0xffffffffu, at < last && (at >= candidates || key > threshold));
      equal[i] = __ballot_sync(0xffffffffu, at < last && at < candidates && key == threshold && ties);
      count += __popc(heavy[i]) + (__popc(equal[i]) << 16);
    }
    if (lane == 0) warp_sum[warp] = count;
    __syncthreads();
    const uint32_t theirs = lane < kWarps ? warp_sum[lane] : 0u;
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0u);
    const uint32_t all = __reduce_add_sync(0xffffffffu, theirs);
    uint32_t a = above_before + (before & 0xffffu), e = ties_before + (before >> 16);
    const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const uint32_t above = a + __popc(heavy[i] & lower), tied = e + __popc(equal[i] & lower);
      if ((heavy[i] >> lane & 1u) || ((equal[i] >> lane & 1u) && tied < ties)) {
        const uint32_t at = above + min(tied, ties);
        kept[at] = j + 32 * i;
        out[at] = x[i];
      }
      a += __popc(heavy[i]);
      e += __popc(equal[i]);
    }
    above_before += all & 0xffffu;
    ties_before += all >> 16;
    __syncthreads();  // warp_sum is written again
  }
  if (kSize > 1) cluster_barrier();  // nobody leaves while its counts may be read
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

template <int kSize, int kThreads>
cudaError_t launch_select(const EvictParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = ensure_smem_limit(select_kernel<kSize, kThreads>, kMaxKeys * 4, configured);
  if (e != cudaSuccess) return e;
  const dim3 grid(kSize, p.num_kv_heads, p.num_seqs);
  if (kSize == 1) return launch_dependent(select_kernel<kSize, kThreads>, grid, kThreads, p.key_room * 4, stream, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.key_room * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSize;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<kSize, kThreads>, p);
}

template <int kThreads>
cudaError_t launch_cluster(const EvictParams& p, int size, cudaStream_t stream) {
  return size == 2   ? launch_select<2, kThreads>(p, stream)
         : size == 4 ? launch_select<4, kThreads>(p, stream)
                     : launch_select<8, kThreads>(p, stream);
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
  // A selection's passes are bound by its CTA's instructions, so few long ones are shared by up
  // to eight CTAs each, as many as leave two CTAs per SM and 4,096 rows each (one sequence of
  // 32,767 rows, 4 heads: 16.1 us a call with four CTAs, 22.4 with two); a batch that fills the
  // GPU by itself gains nothing, and with fewer rows the barriers cost more than they save (16
  // sequences of 4,096 rows, 8 heads: 30.4 us with one CTA each, 33.6 with two).  Clusters of
  // sixteen lose: 83 us in place of 72 for 131,072 rows.
  const int64_t items = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads;
  int size = 1;
  while (size < 8 && items * size * 2 <= 2 * 152 && p.max_len / (size * 2) >= 4096) size *= 2;
  const int most = (p.max_len + size - 1) / size;
  p.key_room = most < kMaxKeys ? most : kMaxKeys;
  // Threads: enough CTAs for every SM side by side (256 sequences of 1,024 rows, 8 heads: 100 us
  // a call with 128, 120 with 512; 32 of 4,096: 52 with 512, 54 with 256, 65 with 128); a
  // thousand where clusters leave a CTA an SM and many rows (one of 131,072, 8 heads: 69 us
  // against 72; four of 32,768, which are two CTAs per SM: 81 against 66).
  const cudaError_t e = size > 1 && items * size <= 152 && most > 4096 ? launch_cluster<1024>(p, size, stream)
                        : size > 1                                     ? launch_cluster<512>(p, size, stream)
                        : p.max_len <= 1024                            ? launch_select<1, 128>(p, stream)
                        : p.max_len <= 2048                            ? launch_select<1, 256>(p, stream)
                                                                       : launch_select<1, 512>(p, stream);
  if (e != cudaSuccess) return e;
  return p.row_bytes % 16 == 0 ? launch_move<uint4>(p, stream) : launch_move<uint2>(p, stream);
}

}  // namespace pkv
