// window_rows.cuh -- what the kernels for few query rows over a sliding window share
// (window_rows.cu: f16/bf16 on tensor cores, window_rows_f32.cu: f32 on CUDA cores): which
// tokens a CTA and its warps take, how tiles of K and V come into shared memory, and how the
// warps' results are joined.
//
// A window bounds what a sequence costs and the host knows it, so there is no work list.  A
// cluster of CTAs takes one (columns, KV head), columns = (new token, query head); its warps take
// the tiles of tokens in turn, each with a ring of its own in shared memory (cp.async; masked
// rows are filled with zeros and not read), and nothing waits for another warp until the end,
// when each CTA joins its share of the columns' values from all warps' maxima, sums and products
// through the cluster's shared memory, in a fixed order.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "mma.cuh"
#include "window.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSmShared = 228 * 1024;  // shared memory of an SM, and what a CTA takes of it beyond its own
constexpr int kCtaReserve = 1024;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_at(uint32_t mine, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(rank));
  return at;
}
__device__ __forceinline__ float cluster_load(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// A CTA's new tokens and the places (window.cuh) that they attend to.
struct RowsItem {
  int s, g;          // sequence, KV head
  int row0, tokens;  // its first new token's row of q and out, new tokens
  int first_place;   // place of the first new token
  int len;           // places that count
  WindowView view;   // of the first new token
};

// This CTA's item, of up to `per` new tokens; false: nothing to do (an empty context's zeros are
// written here).  kOne: one new token per sequence (query_start is not read).
template <typename T, int D, bool kOne>
__device__ __forceinline__ bool find_item(const WindowRowsParams& p, int per, RowsItem& it) {
  const int size = gridDim.x, rank = blockIdx.x, G = p.group;
  int oldest_pos;
  it.s = blockIdx.z;
  it.g = blockIdx.y;
  it.tokens = 1;
  if (kOne) {
    const int L = p.context_lens[it.s];
    it.row0 = it.s;
    if (L <= 0 || L > p.max_len) {
      if (L != 0) {
        if (rank == 0 && threadIdx.x == 0) set_error(p.err, kErrLength);
      } else {
        for (int i = rank * kThreads + threadIdx.x; i < G * D; i += size * kThreads) {
          const size_t at = (static_cast<size_t>(it.s) * p.num_q_heads + it.g * G) * D + i;
          if (p.out_f32) static_cast<float*>(p.out)[at] = 0.f;
          else static_cast<T*>(p.out)[at] = Elem<T>::from_float(0.f);
        }
      }
      return false;
    }
    oldest_pos = L - 1;
  } else {
    // group z of the batch is group z - base(s) of sequence s, base(s) = query_start[s] / per + s:
    // bases rise by at least a sequence's groups
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.query_start[mid] / per + mid <= static_cast<int>(blockIdx.z)) lo = mid;
      else hi = mid - 1;
    }
    it.s = lo;
    const int q0 = p.query_start[lo], n = p.query_start[lo + 1] - q0, L = p.context_lens[lo];
    const int at = (static_cast<int>(blockIdx.z) - q0 / per - lo) * per;
    if (q0 < 0 || n < 0 || n > p.num_query_tokens - q0 || L < n || L > p.max_len) {
      if (at == 0 && rank == 0 && threadIdx.x == 0) set_error(p.err, kErrLength);
      return false;
    }
    if (at < 0 || at >= n) return false;
    it.row0 = q0 + at;
    it.tokens = min(per, n - at);
    oldest_pos = L - n + at;
  }
  it.view = window_view(max(0, oldest_pos - p.window + 1), p.sinks, p.sink_blocks, p.block_size);
  it.first_place = oldest_pos - it.view.shift * p.block_size;
  it.len = it.first_place + it.tokens;
  return true;
}

// A warp's tiles of kTile tokens (8 or 16) of an item, copied into its ring.
//
// A tile in shared memory: rows of D values, 16-byte piece c of row r at place c ^ (r & 7), so
// that the same piece of eight rows lies in different banks.  Row r + row_in of a copy, r a
// multiple of the rows that it takes at once: its place is (chunk ^ row_in) ^ (r & 7).
template <typename T, int D, int kTile, int kStages>
struct TileStream {
  static constexpr int kRowBytes = D * static_cast<int>(sizeof(T));
  static constexpr int kTileBytes = kTile * kRowBytes;        // K or V of a tile
  static constexpr int kRing = 2 * kStages * kTileBytes;      // of a warp
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kRowsAtOnce = 32 / kChunks;
  const WindowRowsParams& p;
  const RowsItem& it;
  const int32_t* table;
  int me, step, mine;   // this warp's number among the cluster's, their count, this warp's tiles
  int skip0, skipped;   // tiles from skip0 on that lie in the gap as a whole: left out
  int shift;            // log2 of the block size
  bool two;             // a tile is in two blocks
  int id0, id1;         // block ids of tile i % 32 of this warp, lane i % 32 (two ids: of its halves)
  uint32_t ring, copy_to, copy_piece;
  int chunk, row_in;
  uint64_t policy;

  __device__ __forceinline__ TileStream(const WindowRowsParams& params, const RowsItem& item, unsigned char* smem)
      : p(params), it(item) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    table = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks_per_seq;
    step = gridDim.x * kWarps;
    me = blockIdx.x * kWarps + warp;
    skip0 = (p.sinks + kTile - 1) / kTile;
    skipped = max(0, (p.sinks + it.view.gap) / kTile - skip0);
    const int tiles = (it.len + kTile - 1) / kTile - skipped;
    mine = me < tiles ? (tiles - me + step - 1) / step : 0;
    shift = 31 - __clz(p.block_size);  // a power of two
    two = p.block_size < kTile;
    id0 = id1 = 0;
    ring = smem_addr(smem + warp * kRing);
    chunk = lane % kChunks;
    row_in = lane / kChunks;
    copy_to = ring + row_in * kRowBytes;
    copy_piece = (chunk ^ row_in) * 16;
    policy = policy_evict_first();
  }
  // the first place of the warp's tile i
  __device__ __forceinline__ int place_of(int i) const {
    const int t = me + i * step;
    return (t < skip0 ? t : t + skipped) * kTile;
  }
  __device__ __forceinline__ bool counts(int at) const {  // (of at least one new token)
    return at < it.len && (at < p.sinks || at >= p.sinks + it.view.gap);
  }
  __device__ __forceinline__ int block_of(int place) const {
    int lb = place >> shift;
    if (lb >= p.sink_blocks) lb += it.view.shift;
    int b = lb < p.max_blocks_per_seq ? table[lb] : -1;
    if (b < 0 || b >= p.num_blocks) {
      set_error(p.err, kErrIndex);
      b = -1;
    }
    return b;
  }
  __device__ __forceinline__ void load_ids(int i) {
    const int lane = threadIdx.x % 32;
    if (i + lane < mine) {
      const int place = place_of(i + lane);
      // rows past the newest token, and rows in the gap, need no block
      auto needed = [&](int at) { return at < it.len && !(at >= p.sinks && at + (two ? 8 : kTile) <= p.sinks + it.view.gap); };
      id0 = needed(place) ? block_of(place) : -1;
      if (two) id1 = needed(place + 8) ? block_of(place + 8) : -1;
    }
  }
  // the warp's tile i into a stage of its ring, as one group of copies
  __device__ __forceinline__ void load(int i, int stage) {
    if (i < mine) {
      if (i % 32 == 0) load_ids(i);
      const int place = place_of(i);
      const int b0 = __shfl_sync(0xffffffffu, id0, i % 32), b1 = two ? __shfl_sync(0xffffffffu, id1, i % 32) : b0;
      const uint32_t dst = copy_to + stage * 2 * kTileBytes;
      // rows 0 to 7 and 8 to 15 (of one block, but where a tile is in two)
      const int64_t head = static_cast<int64_t>(p.num_kv_heads) * p.block_size;
      const int64_t in_pool = (static_cast<int64_t>(it.g) * p.block_size + (place & (p.block_size - 1)) + row_in) * D +
                              chunk * (16 / static_cast<int>(sizeof(T)));
      const int64_t src0 = b0 * head * D + in_pool;
      const int64_t src1 = two ? b1 * head * D + in_pool : src0 + 8 * D;
      const bool full = b0 >= 0 && b1 >= 0 && place + kTile <= it.len && (place + kTile <= p.sinks || place >= p.sinks + it.view.gap);
      if (full) {
#pragma unroll
        for (int r = 0; r < kTile; r += kRowsAtOnce) {
          const int64_t src = (r < 8 ? src0 : src1) + (r & 7) * D;
          const uint32_t to = dst + r * kRowBytes + (copy_piece ^ ((r & 7) * 16));
          cp_async16_hint(to, static_cast<const T*>(p.k_cache) + src, 16, policy);
          cp_async16_hint(to + kTileBytes, static_cast<const T*>(p.v_cache) + src, 16, policy);
        }
      } else {
#pragma unroll
        for (int r = 0; r < kTile; r += kRowsAtOnce) {
          const bool row_counts = (r < 8 ? b0 : b1) >= 0 && counts(place + r + row_in);
          const int64_t src = row_counts ? (r < 8 ? src0 : src1) + (r & 7) * D : 0;
          const uint32_t to = dst + r * kRowBytes + (copy_piece ^ ((r & 7) * 16));
          cp_async16_hint(to, static_cast<const T*>(p.k_cache) + src, row_counts ? 16 : 0, policy);
          cp_async16_hint(to + kTileBytes, static_cast<const T*>(p.v_cache) + src, row_counts ? 16 : 0, policy);
        }
      }
    }
    cp_async_commit();
  }
};

// Joins what the cluster's warps left in each CTA's shared memory: stats[warp][column] (maximum,
// sum) and prod[warp][column][kPitch] products; factors: room for [column][8 kWarps].  Column c
// is query head c % G of new token c / G.  All of a cluster's threads call it.
template <typename T, int D, int kCols, int kPitch, bool kOne>
__device__ __forceinline__ void join_rows(const WindowRowsParams& p, const RowsItem& it, const float2* stats,
                                          const float* prod, float* factors) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, size = gridDim.x, rank = blockIdx.x, G = p.group;
  if (size > 1) cluster_sync();
  else __syncthreads();
  const int cols = it.tokens * G;             // that hold a query
  const int parts = size * kWarps;            // of each column, a lane's each
  for (int c = warp; c < cols; c += kWarps) {
    float top = -INFINITY, sum = 0.f;
    if (lane < parts) {
      const uint32_t at = cluster_at(smem_addr(stats + (lane % kWarps) * kCols + c), lane / kWarps);
      top = cluster_load(at);
      sum = cluster_load(at + 4);
    }
    float most = top;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
    // a warp that saw nothing of the column has a maximum of -inf and no sum
    const float w = sum == 0.f ? 0.f : exp2f(top - most);
    const float total = group_sum<32>(w * sum);
    if (lane < parts) factors[c * 8 * kWarps + lane] = w / total;
  }
  __syncthreads();
  for (int i = rank * kThreads + threadIdx.x; i < cols * D; i += size * kThreads) {
    const int c = i / D, d = i % D;
    const float* f = factors + c * 8 * kWarps;
    float acc = 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k)
      acc = fmaf(f[k], cluster_load(cluster_at(smem_addr(prod + ((k % kWarps) * kCols + c) * kPitch + d), k / kWarps)), acc);
    const int tk = kOne ? 0 : c / G, h = kOne ? c : c - tk * G;
    const size_t at = ((static_cast<size_t>(it.row0) + tk) * p.num_q_heads + it.g * G + h) * D + d;
    if (p.out_f32) static_cast<float*>(p.out)[at] = acc;
    else static_cast<T*>(p.out)[at] = Elem<T>::from_float(acc);
  }
  if (size > 1) cluster_sync();  // nobody leaves while its products may be read
}

// A grid of clusters over KV heads and `groups` (sequences, or groups of new tokens).
inline cudaLaunchConfig_t rows_config(const WindowRowsParams& p, int groups, int smem, cudaStream_t stream,
                                      cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.cluster, p.num_kv_heads, groups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

}  // namespace
}  // namespace pkv
