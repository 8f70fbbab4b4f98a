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
// Work: a window bounds what a sequence costs and the host knows it, so there is no work list.  A
// cluster of CTAs takes one (columns, KV head); its warps take the tiles in turn, each with a ring
// of its own in shared memory (cp.async; masked rows are filled with zeros and not read), and
// nothing waits for another warp until the end, when each CTA joins its share of the columns'
// values from all warps' maxima, sums and products through the cluster's shared memory, in a
// fixed order.
//
// Bound: for few sequences the chain launch -> length -> block table -> K/V -> join; for many, HBM.
#include "common.cuh"
#include "launch.h"
#include "mma.cuh"
#include "window.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;  // tokens of a tile

template <int D, int NT>
struct Rows {
  static constexpr int kCols = 8 * NT;
  static constexpr int kTileBytes = kTile * D * 2;          // K or V of a tile: 2 or 4 KB
  static constexpr int kStages = D == 128 ? 2 : 3;          // 16 or 12 KB a warp
  // CTAs of an SM, by registers and shared memory.  (Rings half as deep again and two CTAs: 14.4 us
  // against 10.3 on 64 sequences, 64/8 heads, D 64, window 128; 90 against 88 on 128, D 128, 1,024.)
  static constexpr int kCtas = D == 64 && NT == 1 ? 4 : 3;
  static constexpr int kRing = 2 * kStages * kTileBytes;    // of a warp
  static constexpr int kPitch = D + 4;                      // floats of a column's products
  static constexpr int kJoin = kWarps * kCols * kPitch * 4; // the warps' products, over the rings
  static constexpr int kMain = kWarps * kRing > kJoin ? kWarps * kRing : kJoin;
  static constexpr int kOffStats = kMain;                   // [kWarps][kCols] maxima and sums
  static constexpr int kOffFactor = kOffStats + kWarps * kCols * 8;  // [kCols][8 kWarps] factors of the parts
  static constexpr int kOffQ = kOffFactor + kCols * 8 * kWarps * 4;
  static constexpr bool kSharedQ = NT > 1;                  // queries in shared memory, not in registers
  static constexpr int kBytes = kOffQ + (kSharedQ ? kCols * D * 2 : 0);
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

// kOne: one new token per sequence (query_start is not read); the columns are its query heads.
template <typename T, int D, int NT, bool kOne>
__global__ void __launch_bounds__(kThreads, (Rows<D, NT>::kCtas)) window_rows_kernel(const __grid_constant__ WindowRowsParams p) {
  using R = Rows<D, NT>;
  constexpr int kCols = R::kCols;
  constexpr int kChunks = D / 8;              // 16-byte pieces of a row
  constexpr int kRowsAtOnce = 32 / kChunks;   // rows that a warp copies with one instruction
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int size = gridDim.x, rank = blockIdx.x, g = blockIdx.y;  // the grid's x is one cluster
  const int G = p.group;
  grid_dependency_wait();
  grid_dependents_launch();

  // the sequence, its new tokens from `first` on that are this CTA's, and their columns
  int s = blockIdx.z, row0, tokens = 1, oldest_pos, newest_pos;
  const int per = kOne ? 1 : kCols / G;       // new tokens of a CTA
  if (kOne) {
    const int L = p.context_lens[s];
    row0 = s;
    if (L <= 0 || L > p.max_len) {
      if (L != 0) {
        if (rank == 0 && threadIdx.x == 0) set_error(p.err, kErrLength);
      } else {  // an empty context: zeros
        for (int i = rank * kThreads + threadIdx.x; i < G * D; i += size * kThreads) {
          const size_t at = (static_cast<size_t>(s) * p.num_q_heads + g * G) * D + i;
          if (p.out_f32) static_cast<float*>(p.out)[at] = 0.f;
          else static_cast<T*>(p.out)[at] = Elem<T>::from_float(0.f);
        }
      }
      return;
    }
    oldest_pos = newest_pos = L - 1;
  } else {
    // group z of the batch is group z - base(s) of sequence s, base(s) = query_start[s] / per + s:
    // bases rise by at least a sequence's groups
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.query_start[mid] / per + mid <= static_cast<int>(blockIdx.z)) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    const int q0 = p.query_start[s], n = p.query_start[s + 1] - q0, L = p.context_lens[s];
    const int at = (static_cast<int>(blockIdx.z) - q0 / per - s) * per;
    if (q0 < 0 || n < 0 || n > p.num_query_tokens - q0 || L < n || L > p.max_len) {
      if (at == 0 && rank == 0 && threadIdx.x == 0) set_error(p.err, kErrLength);
      return;
    }
    if (at < 0 || at >= n) return;
    row0 = q0 + at;
    tokens = min(per, n - at);
    oldest_pos = L - n + at;
    newest_pos = oldest_pos + tokens - 1;
  }
  const WindowView view = window_view(max(0, oldest_pos - p.window + 1), p.sinks, p.sink_blocks, p.block_size);
  const int first_place = oldest_pos - view.shift * p.block_size;      // of the first new token
  const int len = newest_pos - view.shift * p.block_size + 1;          // places that count
  // tiles that lie in the gap as a whole are left out
  const int skip0 = (p.sinks + kTile - 1) / kTile;
  const int skipped = max(0, (p.sinks + view.gap) / kTile - skip0);
  const int tiles = (len + kTile - 1) / kTile - skipped;
  const int step = size * kWarps, me = rank * kWarps + warp;
  const int mine = me < tiles ? (tiles - me + step - 1) / step : 0;
  auto tile_of = [&](int i) {
    const int t = me + i * step;
    return t < skip0 ? t : t + skipped;
  };

  const int shift = 31 - __clz(p.block_size);  // a power of two
  // block ids of 32 of this warp's tiles at a time (two ids a tile at block size 8)
  const int32_t* table = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
  const bool two = p.block_size == 8;
  int id0 = 0, id1 = 0;
  auto block_of = [&](int place) {
    int lb = place >> shift;
    if (lb >= p.sink_blocks) lb += view.shift;
    int b = lb < p.max_blocks_per_seq ? table[lb] : -1;
    if (b < 0 || b >= p.num_blocks) {
      set_error(p.err, kErrIndex);
      b = -1;
    }
    return b;
  };
  auto load_ids = [&](int i) {
    if (i + lane < mine) {
      const int place = tile_of(i + lane) * kTile;
      // a tile's last rows past the newest token, and rows in the gap, need no block
      auto needed = [&](int at) { return at < len && !(at >= p.sinks && at + (two ? 8 : kTile) <= p.sinks + view.gap); };
      id0 = needed(place) ? block_of(place) : -1;
      if (two) id1 = needed(place + 8) ? block_of(place + 8) : -1;
    }
  };

  // A tile in shared memory: rows of 2 D bytes, piece c of row r at place c ^ (r & 7), so that
  // the eight rows that ldmatrix reads at once lie in different banks.  Row r + row_in of a
  // copy, r a multiple of the rows that it takes at once: its place is (chunk ^ row_in) ^ (r & 7).
  const uint32_t ring = smem_addr(smem + warp * R::kRing);
  const int chunk = lane % kChunks, row_in = lane / kChunks;
  const uint32_t copy_to = ring + row_in * (D * 2), copy_piece = (chunk ^ row_in) * 16;
  const uint64_t policy = policy_evict_first();
  auto load_tile = [&](int i, int stage) {  // the warp's tile i
    if (i < mine) {
      if (i % 32 == 0) load_ids(i);
      const int place = tile_of(i) * kTile;
      const int b0 = __shfl_sync(0xffffffffu, id0, i % 32), b1 = two ? __shfl_sync(0xffffffffu, id1, i % 32) : b0;
      const uint32_t dst = copy_to + stage * 2 * R::kTileBytes;
      // rows 0 to 7 and 8 to 15 (of one block, but at block size 8)
      const int64_t head = static_cast<int64_t>(p.num_kv_heads) * p.block_size;
      const int64_t in_pool = (static_cast<int64_t>(g) * p.block_size + (place & (p.block_size - 1)) + row_in) * D + chunk * 8;
      const int64_t src0 = b0 * head * D + in_pool;
      const int64_t src1 = two ? b1 * head * D + in_pool : src0 + 8 * D;
      const bool full = b0 >= 0 && b1 >= 0 && place + kTile <= len && (place + kTile <= p.sinks || place >= p.sinks + view.gap);
      if (full) {
#pragma unroll
        for (int r = 0; r < kTile; r += kRowsAtOnce) {
          const int64_t src = (r < 8 ? src0 : src1) + (r & 7) * D;
          const uint32_t to = dst + r * (D * 2) + (copy_piece ^ ((r & 7) * 16));
          cp_async16_hint(to, static_cast<const T*>(p.k_cache) + src, 16, policy);
          cp_async16_hint(to + R::kTileBytes, static_cast<const T*>(p.v_cache) + src, 16, policy);
        }
      } else {
#pragma unroll
        for (int r = 0; r < kTile; r += kRowsAtOnce) {
          const int at = place + r + row_in;
          const bool counts = (r < 8 ? b0 : b1) >= 0 && at < len && (at < p.sinks || at >= p.sinks + view.gap);
          const int64_t src = counts ? (r < 8 ? src0 : src1) + (r & 7) * D : 0;
          const uint32_t to = dst + r * (D * 2) + (copy_piece ^ ((r & 7) * 16));
          cp_async16_hint(to, static_cast<const T*>(p.k_cache) + src, counts ? 16 : 0, policy);
          cp_async16_hint(to + R::kTileBytes, static_cast<const T*>(p.v_cache) + src, counts ? 16 : 0, policy);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < R::kStages; ++i) load_tile(i, i);

  // queries: column c is query head c % G of new token c / G
  const int gid = lane / 4, tid = lane % 4;
  uint32_t q[R::kSharedQ ? 1 : NT][D / 16][2];
  auto query_row = [&](int c) -> const T* {
    const int tk = kOne ? 0 : c / G, h = kOne ? c : c - tk * G;
    if (kOne ? c >= G : tk >= tokens) return nullptr;
    return static_cast<const T*>(p.q) + ((static_cast<size_t>(row0) + tk) * p.num_q_heads + g * G + h) * D;
  };
  if constexpr (R::kSharedQ) {
    for (int i = threadIdx.x; i < kCols * kChunks; i += kThreads) {
      const int c = i / kChunks, piece = i % kChunks;
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
      for (int e = 0; e < 2; ++e) last[n][e] = first_place + min((8 * n + 2 * tid + e) / G, tokens - 1);
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
  for (int i = 0; i < mine; ++i) {
    cp_async_wait<R::kStages - 1>();
    __syncwarp();
    const uint32_t ks = ring + stage * 2 * R::kTileBytes, vs = ks + R::kTileBytes;
    const int place = tile_of(i) * kTile;
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
    const bool whole = kOne ? place + kTile <= len && (place + kTile <= p.sinks || place >= p.sinks + view.gap)
                            : place + kTile - 1 <= first_place && (place + kTile <= p.sinks || place > len - 1 - p.window);
    uint32_t hidden = 0;  // bit 4 n + e: x[n][e] is masked
    if (!whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = place + gid + (e < 2 ? 0 : 8), to = kOne ? len - 1 : last[n][e & 1];
          const bool seen = at <= to && (at < p.sinks || (kOne ? at >= p.sinks + view.gap : at > to - p.window));
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
    load_tile(i + R::kStages, stage);
    if (++stage == R::kStages) stage = 0;
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings become the warps' products

  // ---- join: every warp of the cluster leaves maxima, sums and products
  float2* stats = reinterpret_cast<float2*>(smem + R::kOffStats);   // [kWarps][kCols]
  float* prod = reinterpret_cast<float*>(smem);                     // [kWarps][kCols][kPitch]
  float* factor = reinterpret_cast<float*>(smem + R::kOffFactor);   // [kCols][8 kWarps]
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
  if (size > 1) cluster_sync();
  else __syncthreads();
  const int cols = tokens * G;                // that hold a query
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
    const float w = sum == 0.f ? 0.f : exp2_approx(top - most);
    const float total = group_sum<32>(w * sum);
    if (lane < parts) factor[c * 8 * kWarps + lane] = w / total;
  }
  __syncthreads();
  for (int i = rank * kThreads + threadIdx.x; i < cols * D; i += size * kThreads) {
    const int c = i / D, d = i % D;
    const float* f = factor + c * 8 * kWarps;
    float acc = 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k)
      acc = fmaf(f[k], cluster_load(cluster_at(smem_addr(prod + ((k % kWarps) * kCols + c) * R::kPitch + d), k / kWarps)), acc);
    const int tk = kOne ? 0 : c / G, h = kOne ? c : c - tk * G;
    const size_t at = ((static_cast<size_t>(row0) + tk) * p.num_q_heads + g * G + h) * D + d;
    if (p.out_f32) static_cast<float*>(p.out)[at] = acc;
    else static_cast<T*>(p.out)[at] = Elem<T>::from_float(acc);
  }
  if (size > 1) cluster_sync();  // nobody leaves while its products may be read
}

template <typename T, int D, int NT, bool kOne>
cudaError_t launch_t(const WindowRowsParams& p, cudaStream_t stream) {
  constexpr int smem = Rows<D, NT>::kBytes;
  static std::atomic<unsigned long long> configured{0};  // devices whose limit is raised
  cudaError_t e = ensure_smem_limit(window_rows_kernel<T, D, NT, kOne>, smem, configured);
  if (e != cudaSuccess) return e;
  const int per = Rows<D, NT>::kCols / p.group;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.cluster, p.num_kv_heads, kOne ? p.num_seqs : p.num_query_tokens / per + p.num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
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
  return dtype == PKV_F16 ? launch_dtype<__half>(p, stream) : launch_dtype<__nv_bfloat16>(p, stream);
}

}  // namespace pkv
