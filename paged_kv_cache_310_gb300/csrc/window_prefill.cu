// window_prefill.cu -- several new tokens per sequence over sliding windows, on the tcgen05 tensor
// cores; f16/bf16, head_dim 64 or 128, up to 16 query heads per KV head.
//
// What it computes: new token i of sequence s sits at position p = context_lens[s] - n_s + i and
// attends to the positions j <= p with j > p - window or j < sinks, through the block table.
//
// Tiles, chunks and products are those of prefill_tc.cu: a tile is 128 query rows of one KV
// head, its G query heads times TQ = 8 * floor(16 / G) consecutive new tokens, token by token; per
// 64-key chunk and tile
//   S[128 rows x 64 keys] = Q . K^T             (M=128, N=64, K=D dims)
//   O[128 rows x D dims] += P . V               (M=128, N=D,  K=64 keys), twice: P as a rounded
// part and what is left; S (double-buffered), P over it, and O in TMEM; one thread per row, a
// maximum that moves only when a chunk passes it by 8 (log2 units).  What differs:
//  * An item runs over its sinks' and its window's blocks as one sequence and masks the rest (see
//    window.cuh).  A row's mask is 64 bits per chunk; scores are scaled and masked once, so that
//    weights need no test (a test at each weight: 323 us instead of 297 on four prompts of 1,000
//    to 2,000 new tokens, window 1,024, 64/8 heads).  A row may see nothing of its item's first
//    chunks: its maximum stays at -inf, its weights at 0.
//  * A window bounds what an item costs, so there is no work list: item i is group i / Hkv of the
//    batch's new tokens for KV head i % Hkv (WindowCursor), dealt out in turn.  (The list kernel
//    took 20 us for 2,300 new tokens.)  The kernel starts while the one before on the stream may
//    still run, and waits for it after its own setup.
//  * Pairs of tiles (kShared false) read each chunk once for both.  With kShared an item is one tile
//    and both softmax warpgroups work on it, each on every other chunk, with sums and O of its own
//    that are joined at the item's end: half the steps for tiles that have no partner (a few new
//    tokens per sequence), twice the items for short batches.
//
//  * Rows of a tile are its tokens one after the other, G query heads each, as they lie in memory: one
//    box of 64 dimensions brings a tile's queries, and a few new tokens leave whole warps without
//    rows, which skip their weights.
//
// Roles (384 threads, persistent CTAs): warps 0-3 and 4-7 the softmax warpgroups (thread = query
// row = TMEM lane), warp 8 the producer of Q and K, warp 9 of V (4-D TMA boxes, one per block;
// places past the item's last come from outside the tensor: zeros), warps 10 and 11 the MMA issuers
// of the two warpgroups.
//
// Measured (64/8 heads, D 128, bf16): four prompts of 1,000 to 2,000 new tokens, window 1,024:
// 224 to 235 us; 32 sequences with 3 to 8 new tokens, window 4,096: 107 to 109 us.
// Bound: pairs: 2,150 clocks a chunk, of which the softmax's dependent instructions take 1,900 and the
// tensor cores' products 1,800 (QK with 64 keys runs at 2/3 of their rate: shared memory feeds the
// 128 query rows), and 3 to 4 us between items.  Shared tiles: the K producer's turns and the
// softmax, 2,600 clocks a step, and the second round of CTAs.
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "tc_util.cuh"
#include "tcgen05.cuh"
#include "window.cuh"

namespace pkv {
namespace {

constexpr int kGroups = 2;                 // tiles per item, one softmax warpgroup each
constexpr int kThreads = (5 * kGroups + 2) * 32;
constexpr int kProducerWarp = 4 * kGroups, kVWarp = kProducerWarp + 1, kMmaWarp = kProducerWarp + 2;  // and the next
constexpr int kRows = 128;                 // query rows per tile (M)
constexpr int kKC = 64;                    // keys per chunk
constexpr uint32_t kTmemCols = 512;        // per tile g: S[2] at 256g + 0/64, O at 256g + 128 (D columns)
constexpr float kRescaleSlack = 8.f;       // log2 units a row's max may grow before O is rescaled

constexpr int kQBlock = kRows * 128;       // 64 dimensions of a tile's queries
constexpr int kQBufs = 2;                  // query buffers: an item's queries load while the previous one runs

// Shared-memory layout for head_dim D (64 or 128): K and V tiles as [8-row group]
// [64-column block][8 rows][128 B], Q tiles (and outputs in their place) as [64-column block][128
// rows][128 B], 128-byte swizzled.
template <int D, bool kShared>
struct Layout {
  static constexpr int kBlocks = D / 64;                  // 64-column blocks of a row
  static constexpr int kGroup = 8 * D * 2;                // one 8-row group: all its blocks
  static constexpr int kKVTile = kKC * D * 2;             // K (or V) of one chunk: 8 or 16 KB
  // stages per ring (K and V have one each); shared tiles: two steps of two chunks
  static constexpr int kStages = kShared ? 4 : 3 * 128 / D;
  static constexpr int kQBytes = kRows * D * 2;           // one tile's queries: 16 or 32 KB
  static constexpr int kQItem = (kShared ? 1 : kGroups) * kQBytes;  // an item's tiles
  static constexpr int kOffV = kStages * kKVTile;
  static constexpr int kOffQ = 2 * kStages * kKVTile;
  static constexpr int kOffBar = kOffQ + kQBufs * kQItem;
  // K ring full/empty, V ring full/empty, qfull[2], qempty[2], then per tile: sfull[2],
  // pfull[2], pvdone[2]; turn, staged and drain of each
  // shared tiles: joined halves full, empty
  static constexpr int kNumBars = 4 * kStages + 4 + kGroups * 9 + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  // shared tiles: the second warpgroup's O on its way to the first, 64 dimensions at a time, and
  // its rows' maxima and sums
  static constexpr int kOffJoin = (kOffMisc + 64 + 127) / 128 * 128;
  static constexpr int kSmemBytes = kShared ? kOffJoin + kRows * (64 + 2) * 4 : kOffMisc + 64;
  static_assert(D == 64 || D == 128, "head_dim 64 or 128");
  static_assert(kOffQ % 1024 == 0 && kSmemBytes <= 232448, "shared memory");
};

struct Bars {
  uint64_t *kfull, *kempty, *vfull, *vempty, *qfull, *qempty, *grp, *turn, *staged, *drain, *jfull, *jempty;
  // per tile g (addresses computed, so a runtime tile index needs no local-memory table)
  __device__ __forceinline__ uint64_t* sfull(int g, int i) const { return grp + 6 * g + i; }
  __device__ __forceinline__ uint64_t* pfull(int g, int i) const { return grp + 6 * g + 2 + i; }
  __device__ __forceinline__ uint64_t* pvdone(int g, int i) const { return grp + 6 * g + 4 + i; }
};

template <typename L>
__device__ __forceinline__ Bars carve(unsigned char* smem) {
  constexpr int kStages = L::kStages;
  uint64_t* b = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  Bars r;
  r.kfull = b;
  r.kempty = b + kStages;
  r.vfull = b + 2 * kStages;
  r.vempty = b + 3 * kStages;
  r.qfull = b + 4 * kStages;
  r.qempty = r.qfull + 2;
  r.grp = r.qempty + 2;
  r.turn = r.grp + 6 * kGroups;
  r.staged = r.turn + kGroups;
  r.drain = r.staged + kGroups;
  r.jfull = r.drain + kGroups;
  r.jempty = r.jfull + 1;
  return r;
}

struct PrefillArgs {
  CUtensorMap tk;  // pool 4-D views: one box = one block's tile for one KV head
  CUtensorMap tv;
  CUtensorMap tq;  // queries (head_dim, heads, tokens): one box = 64 dimensions of a tile
  CUtensorMap to;  // 16-bit outputs, the same
  WindowPrefillParams p;
};

// {s, g | ntile_a << 12 | ntile_b << 20, first query token of tile a, position of that token}
struct Item {
  int s, g, na, nb, qrow0, pos0, last, nchunks;  // na, nb: tokens in tile a, tile b
  int shift, gap;  // blocks left out, masked places from `sinks` on
  __device__ __forceinline__ int ntok(int tile) const { return tile ? nb : na; }
};

// Positions become places (see window.cuh) of the item's first token's view.
template <bool kShared>
__device__ __forceinline__ Item unpack_item(int4 e, const WindowPrefillParams& p) {
  const int tq = p.tile_tokens;
  Item t;
  t.s = e.x;
  t.g = e.y & 0xfff;
  t.na = (e.y >> 12) & 0xff;
  t.nb = (static_cast<unsigned>(e.y) >> 20) & 0xff;
  t.qrow0 = e.z;
  t.pos0 = e.w;
  const WindowView v = window_view(max(0, t.pos0 - p.window + 1), p.sinks, p.sink_blocks, p.block_size);
  t.shift = v.shift;
  t.gap = v.gap;
  t.pos0 -= v.shift * p.block_size;
  t.last = t.pos0 + (t.nb ? tq + t.nb : t.na) - 1;  // place of the item's last token
  t.nchunks = (t.last + kKC) / kKC;
  if (kShared) t.nchunks = (t.nchunks + 1) / 2 * 2;  // steps of two; the odd one's is masked
  return t;
}

// This CTA's items, one after the other from blockIdx.x on in steps of
// the grid.  The batch's new tokens go in groups of a `span` (the tokens of an item), a
// sequence's after the one before's; item i is group i / Hkv for KV head i % Hkv.  Up to 1,024
// sequences a warp counts their groups, 32 shares of up to 32 sequences, and finds a group's
// share and then its sequence by a vote each (shares of one stay in the lanes' registers).
// Beyond, where there are many more items than CTAs anyway, group z is group z - base(s) of
// sequence s, base(s) = query_start[s] / span + s: bases rise by at least a sequence's groups,
// and some numbers have no group.  (Numbering so always left up to half of the CTAs idle on 128
// items: 80 us against 49.)  A warp's lanes call together.
struct WindowCursor {
  const WindowPrefillParams* p;
  int count, k, idx, span;
  int share, before, upto;  // sequences of a lane's share, groups before it and up to its end (share 0: not counted)
  int lane_q0, lane_n, lane_len;  // shares of one sequence: its first new token, new tokens, length
  int4 cur;

  // groups of n new tokens from q0 on; a sequence out of bounds has none
  __device__ __forceinline__ int groups(int q0, int n) const {
    return q0 >= 0 && n > 0 && n <= p->num_query_tokens - q0 ? (n - 1) / span + 1 : 0;
  }
  __device__ __forceinline__ int groups(int s) const {
    return groups(p->query_start[s], p->query_start[s + 1] - p->query_start[s]);
  }
  // the sum of v over the lanes up to this one
  __device__ static __forceinline__ int sum_upto(int v) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += u;
    }
    return v;
  }
  // the entry of item i: no tokens in tile a where there are none
  __device__ __forceinline__ int4 entry(int item) const {
    const int lane = threadIdx.x % 32, H = p->num_kv_heads, z = item / H, g = item - z * H, S = p->num_seqs;
    int s, t0, q0, n, L;
    if (share == 1) {
      s = __popc(__ballot_sync(0xffffffffu, upto <= z)) & 31;
      t0 = (z - __shfl_sync(0xffffffffu, before, s)) * span;
      q0 = __shfl_sync(0xffffffffu, lane_q0, s);
      n = __shfl_sync(0xffffffffu, lane_n, s);
      L = __shfl_sync(0xffffffffu, lane_len, s);
    } else if (share > 0) {
      const int j = __popc(__ballot_sync(0xffffffffu, upto <= z));
      const int rest = z - __shfl_sync(0xffffffffu, before, j & 31);
      const int at = j * share + lane, mine = lane < share && at < S ? groups(at) : 0, sum = sum_upto(mine);
      const int i = __popc(__ballot_sync(0xffffffffu, sum <= rest)) & 31;
      s = j * share + i;
      t0 = (rest - __shfl_sync(0xffffffffu, sum - mine, i)) * span;
    } else {
      int hi = S - 1;
      s = 0;
      while (s < hi) {
        const int mid = (s + hi + 1) / 2;
        if (p->query_start[mid] / span + mid <= z) s = mid;
        else hi = mid - 1;
      }
      t0 = (z - p->query_start[s] / span - s) * span;
    }
    if (share != 1) {
      q0 = p->query_start[s];
      n = p->query_start[s + 1] - q0;
      L = p->context_lens[s];
    }
    if (t0 < 0 || t0 >= n || !sequence_ok(*p, q0, n, L)) return make_int4(0, 0, 0, 0);
    const int tq = p->tile_tokens;
    const int na = min(tq, n - t0), nb = span > tq ? max(0, min(tq, n - t0 - tq)) : 0;
    return make_int4(s, g | (na << 12) | (nb << 20), q0 + t0, L - n + t0);
  }
  __device__ static __forceinline__ bool sequence_ok(const WindowPrefillParams& p, int q0, int n, int L) {
    return q0 >= 0 && n >= 0 && n <= p.num_query_tokens - q0 && L >= n && L <= p.max_context_len;
  }
  // from item idx on, the first that has tokens
  __device__ __forceinline__ void settle() {
    for (; idx < count; idx += gridDim.x) {
      cur = entry(idx);
      if (cur.y >> 12) break;
    }
  }
  __device__ __forceinline__ void init(const WindowPrefillParams& params, int span_) {
    p = &params;
    span = span_;
    const int S = p->num_seqs;
    share = S <= 1024 ? (S + 31) / 32 : 0;
    if (share > 0) {
      const int first = static_cast<int>(threadIdx.x % 32) * share;
      int mine = 0;
      if (share == 1) {
        lane_q0 = first < S ? p->query_start[first] : 0;
        lane_n = first < S ? p->query_start[first + 1] - lane_q0 : 0;
        lane_len = first < S ? p->context_lens[first] : 0;
        mine = groups(lane_q0, lane_n);
      } else {
        for (int s = first; s < min(S, first + share); ++s) mine += groups(s);
      }
      upto = sum_upto(mine);
      before = upto - mine;
      count = __shfl_sync(0xffffffffu, upto, 31) * p->num_kv_heads;
    } else {
      count = (p->num_query_tokens / span + S) * p->num_kv_heads;
    }
    k = 0;
    idx = blockIdx.x;
    settle();
  }
  __device__ __forceinline__ bool valid() const { return idx < count; }
  __device__ __forceinline__ void advance() {
    ++k;
    idx += gridDim.x;
    settle();
  }
};

// The lowest n bits (none below 0, all from 64 on).
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// A box of 64 dimensions x 1 head x 8 tokens from shared memory to its place in the outputs, and the
// waits for a thread's boxes: their reads done, all done.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
               "r"(z), "r"(smem_addr(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Branches that a chunk rarely takes: their code goes out of the loop's straight line (instruction
// fetches past them were a tenth of a chunk's time).
__device__ __forceinline__ bool rare(bool taken) { return __builtin_expect(taken, 0); }

// The maximum of a row's 64 scores. Where the mask cuts the chunk, keys past `lim`, and those
// before `low` from `sink` on, become -inf in place, so that their weights come out as 0 without
// another test.
__device__ __forceinline__ float masked_maximum(float* sv, bool cut, int lim, int low, int sink) {
  if (rare(cut)) {
    const uint64_t seen = low_bits(lim + 1) & (~low_bits(low) | low_bits(sink));
    const uint32_t lower = static_cast<uint32_t>(seen), upper = static_cast<uint32_t>(seen >> 32);
#pragma unroll
    for (int i = 0; i < 64; ++i) sv[i] = ((i < 32 ? lower : upper) & (1u << (i % 32))) ? sv[i] : -INFINITY;
  }
  float e0 = -INFINITY, e1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    e0 = fmax3(e0, sv[i], sv[i + 1]);
    e1 = fmax3(e1, sv[i + 2], sv[i + 3]);
  }
  return fmaxf(e0, e1);
}

// p minus its rounding h, exact: a mixed-precision h * -1 + p, one instruction for taking the 16-bit
// value apart and for the difference.
template <typename T>
__device__ __forceinline__ float rest_of(uint32_t h, float p) {
  float d;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(static_cast<uint16_t>(h)), "h"(static_cast<uint16_t>(0xBF80)), "f"(p));
  else
    asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(static_cast<uint16_t>(h)), "h"(static_cast<uint16_t>(0xBC00)), "f"(p));
  return d;
}

// One producer warp's copies of an item's chunks of K (or V) into its ring: per chunk
// one 4-D box per block (blocks past the pair's last position from outside the tensor:
// zero fill).  `c` counts the warp's chunks over all items.  Returns false on abort.
template <int D, bool kShared>
__device__ __forceinline__ bool load_chunks(const WindowPrefillParams& p, const Item& it, const CUtensorMap* map,
                                            unsigned char* ring, uint64_t* full, uint64_t* empty, int& c,
                                            int* issued_slot, uint64_t policy, volatile int* abort_flag) {
  constexpr int kStages = Layout<D, kShared>::kStages, kKVTile = Layout<D, kShared>::kKVTile;
  const int lane = threadIdx.x % 32;
  const int bs = p.block_size;
  const int blocks_per_chunk = kKC / bs;
  const int oob_group = p.num_blocks * p.num_kv_heads * bs / 8;  // first row group outside the pool
  const int32_t* table = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks_per_seq;
  for (int k = 0; k < it.nchunks; ++k, ++c) {
    const int st = c % kStages;
    const int lb = k * blocks_per_chunk + lane;  // logical block of this lane
    const bool live = lane < blocks_per_chunk && lb * bs <= it.last;
    const int tb = lb >= p.sink_blocks ? lb + it.shift : lb;  // its table entry
    int b = live ? (tb < p.max_blocks_per_seq ? table[tb] : -1) : 0;
    bool ok = true;
    if (lane == 0) {
      ok = c < kStages || wait_role(&empty[st], ((c / kStages) - 1) & 1, abort_flag, p.err, p.wait_limit_ns);
      if (ok) mbar_arrive_expect_tx(&full[st], kKVTile);
    }
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    __syncwarp();
    if (lane < blocks_per_chunk) {
      int grp = oob_group;
      if (live) {
        if (b < 0 || b >= p.num_blocks) {
          set_error(p.err, kErrIndex);
          b = 0;
        }
        grp = (b * p.num_kv_heads + it.g) * bs / 8;
      }
      tma_load_4d(ring + st * kKVTile + lane * bs * (D * 2), map, grp, &full[st], policy);
    }
    if (lane == 0) *issued_slot = c + 1;
  }
  return true;
}

template <typename T, int D, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) window_prefill_kernel(const __grid_constant__ PrefillArgs a) {
  using L = Layout<D, kShared>;
  constexpr int kStages = L::kStages, kGroup = L::kGroup, kKVTile = L::kKVTile;
  constexpr int kQBytes = L::kQBytes, kQItem = L::kQItem, kOffV = L::kOffV, kOffQ = L::kOffQ;
  constexpr int kOffMisc = L::kOffMisc;
  extern __shared__ __align__(1024) unsigned char smem[];
  const WindowPrefillParams& p = a.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Bars bars = carve<L>(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* kissued_slot = reinterpret_cast<int*>(smem + kOffMisc + 8);
  int* vissued_slot = reinterpret_cast<int*>(smem + kOffMisc + 12);
  int* qissued_slot = reinterpret_cast<int*>(smem + kOffMisc + 16);
  const int G = p.group, TQ = p.tile_tokens;
  constexpr int kTiles = kShared ? 1 : kGroups;  // of an item
  const int span = kTiles * TQ;                  // new tokens of an item

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.kfull[i], 1);
      mbar_init(&bars.kempty[i], kShared ? 1 : kGroups);
      mbar_init(&bars.vfull[i], 1);
      mbar_init(&bars.vempty[i], kShared ? 1 : kGroups);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.qfull[i], 1);
      mbar_init(&bars.qempty[i], kShared ? kGroups : 5 * kGroups);  // the issuers, and the softmax's warps
    }
    for (int g = 0; g < kGroups; ++g) {
      mbar_init(&bars.turn[g], 1);
      mbar_init(&bars.staged[g], 4);
      for (int i = 0; i < 2; ++i) {
        mbar_init(bars.sfull(g, i), 1);
        mbar_init(bars.pfull(g, i), 4);
        mbar_init(bars.pvdone(g, i), 1);
      }
    }
    if (kShared) {
      mbar_init(bars.jfull, 4);
      mbar_init(bars.jempty, 4);
    }
    *abort_flag = 0;
    *kissued_slot = 0;
    *vissued_slot = 0;
    *qissued_slot = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // launched while the kernel before may still run; everything above touches this CTA alone
  grid_dependency_wait();
  grid_dependents_launch();

  if (warp == kProducerWarp) {
    // ============================ producer: Q and K ============================
    if (lane == 0) {
      prefetch_tensormap(&a.tk);
      prefetch_tensormap(&a.tq);
    }
    const uint64_t pol_kv = policy_evict_normal();  // K/V: re-read by the sequence's other items
    const uint64_t pol_q = policy_evict_first();    // Q: read once
    int c = 0, j = 0;
    bool ok = true;
    WindowCursor cur;
    for (cur.init(p, span); cur.valid() && ok; cur.advance(), ++j) {
      const Item it = unpack_item<kShared>(cur.cur, p);
      // ---- both tiles' queries into buffer j % kQBufs (free once item j - kQBufs's QKs completed) ----
      const int qb = j % kQBufs;
      if (lane == 0) {
        ok = j < kQBufs || wait_role(&bars.qempty[qb], ((j / kQBufs) - 1) & 1, abort_flag, p.err, p.wait_limit_ns);
        if (ok) mbar_arrive_expect_tx(&bars.qfull[qb], kTiles * L::kBlocks * G * TQ * 128);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      __syncwarp();
      if (lane < kTiles * L::kBlocks) {
        const int tile = lane / L::kBlocks, half = lane % L::kBlocks;
        tma_load_3d(smem + kOffQ + qb * kQItem + tile * kQBytes + half * kQBlock, &a.tq, half * 64, it.g * G,
                    it.qrow0 + tile * TQ, &bars.qfull[qb], pol_q);
      }
      if (lane == 0) *qissued_slot = j + 1;
      // ---- K chunks (a stage is free once both tiles' QKs of its chunk completed) ----
      ok = load_chunks<D, kShared>(p, it, &a.tk, smem, bars.kfull, bars.kempty, c, kissued_slot, pol_kv, abort_flag);
    }
  } else if (warp == kVWarp) {
    // ============================ producer: V ============================
    if (lane == 0) prefetch_tensormap(&a.tv);
    // sequences out of bounds are skipped; this flags them
    for (int s = blockIdx.x * 32 + lane; s < p.num_seqs; s += gridDim.x * 32)
      if (!WindowCursor::sequence_ok(p, p.query_start[s], p.query_start[s + 1] - p.query_start[s], p.context_lens[s]))
        set_error(p.err, kErrLength);
    const uint64_t pol_kv = policy_evict_normal();
    int c = 0;
    bool ok = true;
    WindowCursor cur;
    for (cur.init(p, span); cur.valid() && ok; cur.advance()) {
      // a stage is free once both tiles' PVs of its chunk completed
      ok = load_chunks<D, kShared>(p, unpack_item<kShared>(cur.cur, p), &a.tv, smem + kOffV, bars.vfull, bars.vempty, c,
                          vissued_slot, pol_kv, abort_flag);
    }
  } else if (warp >= kMmaWarp) {
    // ============================ MMA issuers ============================
    // One per softmax warpgroup, each with a fixed schedule: PV of chunk c, then QK of
    // chunk c + 2 (whose S buffer held the probabilities of chunk c).  (One issuer for both left
    // the tensor cores idle for 600 of a step's 3,050 clocks: an issuer's own instructions between
    // its products take as long as the 9 products that the hardware queues.)  The whole warp runs it
    // with warp-uniform control flow (descriptors and counters stay in uniform registers); one
    // elected lane issues.
    // The tiles of a pair take turns: a PV goes out only after the other tile's last one and the
    // first product of its QK, so that one's products run while the other's issuer and
    // softmax are between theirs.  (Without turns 267 us against 248 on four prompts of 1,000 to
    // 2,000 new tokens, window 1,024, 64/8 heads, head_dim 128; 199 against 203 at head_dim 64.
    // Shared tiles, whose steps have more room: 109 without, 111 with, on 32 sequences with 3 to 8
    // new tokens, window 4,096.  PV and QK of a tile from warps of their own, with 184 and 72
    // registers a thread: 257 and 118: 16 warps slow the softmax.)
    constexpr bool kTurns = !kShared;
    const int g = warp - kMmaWarp;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t idesc_qk = instr_desc_f16(kBf16, false, false, kRows, kKC);
    constexpr uint32_t idesc_pv = instr_desc_f16(kBf16, false, true, kRows, D);
    // Shared tiles: a step has a chunk for each warpgroup, in stages st and st + 1; chunks,
    // items' counts and the stages' turns below are then in steps.
    constexpr int kPer = kShared ? 2 : 1;  // chunks, and stages, of a step
    const int st0 = kShared ? g : 0;       // this issuer's stage of a step
    // descriptor bases; adding (byte offset >> 4) moves a descriptor's start address
    const uint64_t dq0 = smem_desc(smem_addr(smem + kOffQ + (kShared ? 0 : g * kQBytes)), 16, 1024, kLayoutSwizzle128);
    const uint64_t dk0 = smem_desc(smem_addr(smem + st0 * kKVTile), 16, kGroup, kLayoutSwizzle128);
    const uint64_t dv0 = smem_desc(smem_addr(smem + kOffV + st0 * kKVTile), 1024, kGroup, kLayoutSwizzle128);
    const uint32_t sd = tmem + g * 256, od = sd + 128;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_role(bar, parity, abort_flag, p.err, p.wait_limit_ns));
    };
    auto steps_of = [&](const WindowCursor& c) { return c.valid() ? unpack_item<kShared>(c.cur, p).nchunks / kPer : 0; };
    // QK side: next chunk qc (global), its stage / phase, its place in the item
    WindowCursor qcur;
    qcur.init(p, span);
    int qc = 0, qst = 0, qph = 0, qk = 0, qn = steps_of(qcur);
    uint32_t starts = 0;  // bit sb: the chunk in S buffer sb is its item's first, whose PV overwrites O
    // PV side
    int pc = 0, pst = 0, pph = 0;
    bool ok = true;
    auto issue_qk = [&](bool k_seen, bool pass) -> bool {  // k_seen: the K stage was already seen landed; pass: the turn
      const int qj = qcur.k, qb = qj % kQBufs, sb = qc & 1;
      const bool first = qk == 0, last = qk == qn - 1;
      // pairs: the item's queries wait for the outputs, and so for the other tile's last PV, of the item
      // before the last: the turn goes first
      if (kTurns && first && pass && lane == 0) mbar_arrive(&bars.turn[g]);
      if (first && !wait_all(&bars.qfull[qb], (qj / kQBufs) & 1)) return false;
      if (!k_seen && !wait_all(&bars.kfull[qst + st0], qph)) return false;
      const uint64_t dk = dk0 + ((qst * kKVTile) >> 4);
      const uint64_t dq = dq0 + ((qb * kQItem) >> 4);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
          mma_f16(sd + sb * 64, dq + (((kk >> 2) * kQBlock + (kk & 3) * 32) >> 4), dk + off, idesc_qk, kk > 0);
          if (kTurns && kk == 0 && pass && !first) mbar_arrive(&bars.turn[g]);
        }
        mma_commit(bars.sfull(g, sb));
        mma_commit(&bars.kempty[qst + st0]);
        if (last) mma_commit(&bars.qempty[qb]);  // this issuer is done with the item's queries
      }
      __syncwarp();
      starts = (starts & ~(1u << sb)) | (static_cast<uint32_t>(first) << sb);
      ++qc;
      if ((qst += kPer) == kStages) {
        qst = 0;
        qph ^= 1;
      }
      if (++qk == qn) {
        qk = 0;
        qcur.advance();
        qn = steps_of(qcur);
      }
      return true;
    };
    for (int i = 0; i < 2 && ok && qcur.valid(); ++i) ok = issue_qk(false, false);
    for (; ok && pc < qc; ++pc) {
      const int sb = pc & 1;
      uint64_t* turn = &bars.turn[g ^ 1];
      const uint32_t turn_parity = (pc & 1) ^ (g ^ 1);
      // one round trip probes everything this step needs; only what is not ready yet is waited for
      const uint32_t seen = __shfl_sync(0xffffffffu,
          mbar_test_wait4(&bars.vfull[pst + st0], pph, bars.pfull(g, sb), (pc >> 1) & 1, turn, turn_parity,
                          &bars.kfull[qst + st0], qph), 0);
      if (!(seen & 1) && !wait_all(&bars.vfull[pst + st0], pph)) break;
      if (!(seen & 2) && !wait_all(bars.pfull(g, sb), (pc >> 1) & 1)) break;
      if (kTurns && !(seen & 4) && !wait_all(turn, turn_parity)) break;
      const uint64_t dv = dv0 + ((pst * kKVTile) >> 4);
      const bool acc0 = !(starts >> sb & 1);
      tc_fence_after();
      if (elect_one()) {
        const uint32_t pa = sd + sb * 64;  // probabilities: [hi 8 | lo 8] columns per 16 keys
#pragma unroll
        for (int kk = 0; kk < kKC / 16; ++kk) {
          const uint64_t bd = dv + ((kk * 2 * kGroup) >> 4);
          mma_f16_tmem_a(od, pa + kk * 16, bd, idesc_pv, acc0 || kk > 0);
          mma_f16_tmem_a(od, pa + kk * 16 + 8, bd, idesc_pv, true);
        }
        mma_commit(&bars.vempty[pst + st0]);
        mma_commit(bars.pvdone(g, sb));
      }
      __syncwarp();
      if ((pst += kPer) == kStages) {
        pst = 0;
        pph ^= 1;
      }
      if (qcur.valid()) ok = issue_qk((seen & 8) != 0, true);
      else if (kTurns && lane == 0) mbar_arrive(&bars.turn[g]);
    }
    __syncwarp();
  } else {
    // ============================ softmax warpgroups ============================
    const int grp = warp / 4;                 // which tile of the pair
    const int t = threadIdx.x % 128;          // query row of the tile = TMEM lane
    const int wq = warp % 4;                  // lane quarter
    const int head = t % G, tok = t / G;
    const uint32_t lane_base = tmem + grp * 256 + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t obuf = lane_base + 128;
    // scores are multiplied where the maximum is subtracted; by a scale that is not positive, which
    // does not keep their order, before
    const bool ordered = p.scale_log2 > 0.f;
    const float scale = ordered ? p.scale_log2 : 1.f;
    const float2 sc2 = make_float2(scale, scale);
    int c = 0;
    bool ok = true;
    int prev_row = -1, prev_c = -1;
    bool prev_full = false;
    float prev_l = 1.f, prev_m = 0.f;
    int tiles_out = 0;  // tiles that left by TMA
    int joins = 0;  // shared tiles: hand-overs so far
    // this row's O, 16 vectors, the i-th at i ^ (t & 7): eight rows at once lie in different banks
    float4* join = reinterpret_cast<float4*>(smem + L::kOffJoin) + t * 16;
    float* join_stats = reinterpret_cast<float*>(smem + L::kOffJoin) + kRows * 64 + 2 * t;

    // Warp-uniform: has this tile's PV of chunk cc completed?
    auto pv_done = [&](int cc) -> bool {
      return __all_sync(0xffffffffu, wait_role(bars.pvdone(grp, cc & 1), (cc >> 1) & 1, abort_flag, p.err, p.wait_limit_ns));
    };
    // Shared tiles: 32 of a finished row's values from dimension q * 32 on, times inv, to its output.
    auto store_row = [&](int row, int q, const float* o, float inv) {
      if (p.out_f32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + static_cast<size_t>(row) * D + q * 32);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[i] = make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + static_cast<size_t>(row) * D + q * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_uint4(pack2<T>(o[8 * i] * inv, o[8 * i + 1] * inv),
                              pack2<T>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                              pack2<T>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                              pack2<T>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
      }
    };
    // Pairs of tiles: piece q of a finished tile's rows, 32 values from dimension 32 q on, times inv. They go out
    // through the place of the tile's queries, which lie there done with, in the same layout and in
    // as many bytes a row (fp32: half a row at a time). A full tile of 16-bit rows leaves by TMA under the
    // next item's chunks; others are stored by the warps, a row's 16-byte pieces side by side.
    // (A lane storing its own row touches 32 lines at an instruction, 5,000 clocks an item: 238 us
    // against 225 on four prompts of 1,000 to 2,000 new tokens, window 1,024, 64/8 heads. Shared
    // tiles, whose few tokens fill no tile: 109 against 114 on 32 sequences with 3 to 8 new tokens.)
    auto store_piece = [&](unsigned char* stage, int row, bool full, int q, const float* o, float inv) {
      constexpr int kPieces = D * 2 / 16;  // 16-byte pieces of a staged row
      auto place = [&](int r, int i) {     // piece i of row r of this warp
        return reinterpret_cast<uint4*>(stage + i / 8 * kQBlock + (32 * wq + r) * 128 + ((i ^ r) & 7) * 16);
      };
      auto copy_out = [&](int skip, int bytes) {  // staged rows to `skip` of a row of `bytes`
        __syncwarp();
#pragma unroll 4
        for (int r = lane / kPieces; r < 32; r += 32 / kPieces) {
          const int to = __shfl_sync(0xffffffffu, row, r);
          const int i = lane % kPieces;
          const uint4 v = *place(r, i);
          if (to >= 0) *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p.out) + static_cast<size_t>(to) * bytes + skip + 16 * i) = v;
        }
        __syncwarp();
      };
      if (p.out_f32) {
        const int at = q % (D / 64) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *place(lane, at + i) = make_uint4(__float_as_uint(o[4 * i] * inv), __float_as_uint(o[4 * i + 1] * inv),
                                            __float_as_uint(o[4 * i + 2] * inv), __float_as_uint(o[4 * i + 3] * inv));
        if ((q + 1) % (D / 64) == 0) copy_out(q / (D / 64) * D * 2, D * 4);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *place(lane, 4 * q + i) = make_uint4(pack2<T>(o[8 * i] * inv, o[8 * i + 1] * inv), pack2<T>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                               pack2<T>(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack2<T>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        if (q < D / 32 - 1) return;
        if (full) {
          fence_proxy_async_smem();  // for the TMA's reads
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.staged[grp]);
          const uint32_t parity = tiles_out++ & 1;
          if (t == 0 && wait_role(&bars.staged[grp], parity, abort_flag, p.err, p.wait_limit_ns)) {  // row 0: the tile's first token and head
#pragma unroll
            for (int half = 0; half < L::kBlocks; ++half)
              tma_store_3d(&a.to, half * 64, row % p.num_q_heads, row / p.num_q_heads, stage + half * kQBlock);
            bulk_commit();
          }
        } else {
          copy_out(0, D * 2);
        }
      }
    };
    // The staged rows have left for good: the place is the producer's.
    auto release = [&](int item) {
      bulk_wait_read();
      fence_proxy_async_smem();  // its next writes are the TMA's
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.qempty[item % kQBufs]);
    };
    // A finished item's output rows: O / l (O is final: its last PV was waited for).  Shared
    // tiles: the second warpgroup hands its rows' O, maxima and sums to the first, which joins
    // the two.  False: a wait ran out.
    auto finish = [&](int item, int row, bool full, float lsum, float top) -> bool {
      tc_fence_after();
      if constexpr (kShared) {
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h, ++joins) {
          if (grp == 1) {
            if (joins > 0 && !__all_sync(0xffffffffu, wait_role(bars.jempty, (joins - 1) & 1, abort_flag, p.err, p.wait_limit_ns)))
              return false;
            join_stats[0] = top;
            join_stats[1] = lsum;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
              float o[32];
              tmem_load32(obuf + h * 64 + q * 32, o);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                join[(8 * q + i) ^ (t & 7)] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.jfull);
          } else {
            if (!__all_sync(0xffffffffu, wait_role(bars.jfull, joins & 1, abort_flag, p.err, p.wait_limit_ns))) return false;
            // a half that saw none of a row's keys has a maximum of -inf, a sum of 0 and an O of 0
            const float most = fmaxf(top, join_stats[0]);
            const float mine = lsum == 0.f ? 0.f : exp2f(top - most), theirs = join_stats[1] == 0.f ? 0.f : exp2f(join_stats[0] - most);
            const float inv = 1.f / (mine * lsum + theirs * join_stats[1]);
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
              float o[32];
              tmem_load32(obuf + h * 64 + q * 32, o);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 b = join[(8 * q + i) ^ (t & 7)];
                o[4 * i] = fmaf(theirs, b.x, mine * o[4 * i]);
                o[4 * i + 1] = fmaf(theirs, b.y, mine * o[4 * i + 1]);
                o[4 * i + 2] = fmaf(theirs, b.z, mine * o[4 * i + 2]);
                o[4 * i + 3] = fmaf(theirs, b.w, mine * o[4 * i + 3]);
              }
              if (row >= 0) store_row(row, 2 * h + q, o, inv);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.jempty);
          }
        }
      } else {
        unsigned char* stage = smem + kOffQ + item % kQBufs * kQItem + grp * kQBytes;
        const float inv = 1.f / lsum;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          float o[32];
          tmem_load32(obuf + q * 32, o);
          store_piece(stage, row, full, q, o, inv);
        }
      }
      tc_fence_before();
      return true;
    };

    int j = 0;
    WindowCursor cur;
    for (cur.init(p, span); cur.valid() && ok; cur.advance(), ++j) {
      const Item it = unpack_item<kShared>(cur.cur, p);
      const int tile = kShared ? 0 : grp;
      const bool row_valid = tok < it.ntok(tile);
      const int qpos = row_valid ? it.pos0 + tile * TQ + tok : it.last;  // padding rows act as the last token
      const int out_row = row_valid ? (it.qrow0 + tile * TQ + tok) * p.num_q_heads + it.g * G + head : -1;
      // shared tiles: a warp of padding rows has no scores to weigh (its rows of O are never read)
      const bool idle = kShared && !__any_sync(0xffffffffu, row_valid);
      float m = -INFINITY, l = 0.f;  // max used for this row's probabilities, running row sum
      const int steps = it.nchunks / (kShared ? 2 : 1);
      for (int k = 0; k < steps; ++k, ++c) {
        const int sb = c & 1;
        const uint32_t sbuf = lane_base + sb * 64;
        if (rare(!__all_sync(0xffffffffu, mbar_test_wait(bars.sfull(grp, sb), (c >> 1) & 1))) &&
            !__all_sync(0xffffffffu, wait_role(bars.sfull(grp, sb), (c >> 1) & 1, abort_flag, p.err, p.wait_limit_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int kbase = (kShared ? 2 * k + grp : k) * kKC;
        // the chunk's stage in the V ring, and the turn of it
        const int vst = kShared ? 2 * (c & 1) + grp : c % kStages, vturn = kShared ? (c >> 1) & 1 : (c / kStages) & 1;
        // keys of the chunk past lim are masked, and those before its window but for the sinks
        const int lim = qpos - kbase, low = lim - p.window + 1, sink = p.sinks - kbase;
        const bool cut = lim < kKC - 1 || low > max(0, sink);  // only then does the mask cut this row
        // the row's 64 scores, held in registers for both passes
        float sv[64], cm = -INFINITY;
        // pass 1: the row's chunk maximum of scale * score under the mask
        if (!kShared || !idle) {
          tmem_load64(sbuf, sv);
          if (rare(!ordered)) {
#pragma unroll
            for (int i = 0; i < 64; ++i) sv[i] *= p.scale_log2;
          }
          cm = scale * masked_maximum(sv, cut, lim, low, sink);
        }
        // lazy rescale: keep m unless the chunk brings a score more than the slack above
        // (a chunk that the mask leaves nothing of gives cm = -inf and changes nothing)
        // While the maximum is -inf (the row's window starts in a later chunk) the row's sum and O
        // are zeros, which need no rescale.
        const bool grow = cm > m + kRescaleSlack;
        const float alpha = grow && m != -INFINITY ? exp2_approx(m - cm) : 1.f;
        m = grow ? cm : m;
        l *= alpha;
        // O is read out (at an item's first chunk) or rescaled only after the PVs that
        // accumulate it have completed
        if (rare(k == 0 && prev_c >= 0)) {
          if (!pv_done(prev_c)) {
            ok = false;
            break;
          }
          ok = finish(j - 1, prev_row, prev_full, prev_l, prev_m);
          if (!ok) break;
          prev_c = -1;
        }
        if (rare(k > 0 && __any_sync(0xffffffffu, alpha != 1.f))) {
          if (!pv_done(c - 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            float o[16];
            tmem_load16(obuf + q * 16, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_store16(obuf + q * 16, o);
          }
        }
        // pass 2: probabilities as hi + lo parts, written over the 16 S columns they
        // came from: [hi of 16 keys | lo of 16 keys]
        if (!kShared || !idle) {
          float2 acc = make_float2(0.f, 0.f);
          const float used = m == -INFINITY ? 0.f : m;  // nothing seen yet: every score is -inf
          const float2 nm2 = make_float2(-used, -used);
#pragma unroll
          for (int q = 0; q < kKC / 16; ++q) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 s = make_float2(sv[q * 16 + 2 * i], sv[q * 16 + 2 * i + 1]);
              const float2 x = __ffma2_rn(s, sc2, nm2);
              const float p0 = exp2_approx(x.x), p1 = exp2_approx(x.y);
              const float2 pr = make_float2(p0, p1);
              w[i] = pack2<T>(p0, p1);  // rounded pair
              w[8 + i] = pack2<T>(rest_of<T>(w[i] & 0xffff, p0), rest_of<T>(w[i] >> 16, p1));
              acc = __fadd2_rn(acc, pr);
            }
            tmem_store16_words(sbuf + q * 16, w);
          }
          l += acc.x + acc.y;
          tmem_store_wait();
        }
        tc_fence_before();
        // V rows past the pair's last position inside loaded blocks, and those of a window's
        // gap: zero them (a NaN there would survive a zero weight).  Both groups write the
        // same zeros, but for shared tiles, where each has its own chunk.
        const int rows_needed = it.last + 1 - kbase;
        const int gap0 = max(0, p.sinks - kbase);
        const int gap1 = min(kKC, p.sinks + it.gap - kbase);
        const bool unseen = rows_needed < kKC || gap0 < gap1;
        if (rare(unseen)) {  // warp-uniform; V of this chunk must have landed first
          if (!__all_sync(0xffffffffu, wait_role(&bars.vfull[vst], vturn, abort_flag, p.err, p.wait_limit_ns))) {
            ok = false;
            break;
          }
        }
        if (rare(t < kKC && unseen)) {
          const int rows_loaded = min(kKC, (rows_needed + p.block_size - 1) / p.block_size * p.block_size);
          if ((t >= rows_needed && t < rows_loaded) || (t >= gap0 && t < gap1)) {
            unsigned char* vrow = smem + kOffV + vst * kKVTile + (t >> 3) * kGroup + (t & 7) * 128;
#pragma unroll
            for (int q = 0; q < 8 * L::kBlocks; ++q)  // 128 bytes per 64-column block, 1 KB apart
              reinterpret_cast<uint4*>(vrow + (q >> 3) * 1024)[q & 7] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.pfull(grp, sb));
        // the item before's outputs have had two chunks' time to leave
        if (!kShared && rare(k == min(1, steps - 1) && j > 0)) release(j - 1);
      }
      if (!ok) break;
      prev_row = out_row;
      prev_full = it.ntok(tile) == TQ;
      prev_c = c - 1;
      prev_l = l;
      prev_m = m;
    }
    if (ok && prev_c >= 0 && pv_done(prev_c)) finish(j - 1, prev_row, prev_full, prev_l, prev_m);
    if (!kShared) bulk_wait();
    __syncwarp();
  }

  // ---------------- teardown ----------------
  __syncthreads();
  if (*abort_flag) {
    // copies still in flight land before the CTA exits: the last chunk issued on each
    // stage (and the last query buffers) -- a phase already completed returns at once
    if (warp == kProducerWarp && lane == 0) {
      for (int c = max(0, *kissued_slot - kStages); c < *kissued_slot; ++c)
        if (!mbar_wait(&bars.kfull[c % kStages], (c / kStages) & 1)) break;
      for (int jj = max(0, *qissued_slot - kQBufs); jj < *qissued_slot; ++jj)
        if (!mbar_wait(&bars.qfull[jj % kQBufs], (jj / kQBufs) & 1)) break;
    }
    if (warp == kVWarp && lane == 0) {
      for (int c = max(0, *vissued_slot - kStages); c < *vissued_slot; ++c)
        if (!mbar_wait(&bars.vfull[c % kStages], (c / kStages) & 1)) break;
    }
    if (warp >= kMmaWarp) {
      // every lane commits (the MMAs went out from whichever lane was elected; a lane
      // that issued none arrives at once), so the barrier completes only when all of
      // the warp's MMAs have
      uint64_t* drain = bars.drain + (warp - kMmaWarp);
      if (lane == 0) {
        mbar_init(drain, 32);
        fence_barrier_init();
      }
      __syncwarp();
      mma_commit(drain);
      mbar_wait(drain, 0);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Queries, or 16-bit outputs, [tokens][heads][head_dim] seen as 3-D (head_dim, heads, tokens); a box is
// 64 dimensions of a tile: its KV head's `group` query heads and `tile_tokens` tokens.
bool make_query_map(CUtensorMap* m, const void* q, uint32_t heads, uint32_t tokens, uint32_t group, uint32_t tile_tokens, bool bf16,
                    int head_dim) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(head_dim) * 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), heads, tokens};
  cuuint64_t strides[2] = {row, static_cast<cuuint64_t>(heads) * row};
  cuuint32_t box[3] = {64, group, tile_tokens};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(q),
            dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool kShared>
cudaError_t launch_t(const PrefillArgs& args, int grid, cudaStream_t stream) {
  constexpr int smem = Layout<D, kShared>::kSmemBytes;
  static std::atomic<unsigned long long> configured{0};  // devices whose limit is raised
  cudaError_t e = ensure_smem_limit(window_prefill_kernel<T, D, kShared>, smem, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(window_prefill_kernel<T, D, kShared>, grid, kThreads, smem, stream, args);
}

template <typename T>
cudaError_t launch_d(const PrefillArgs& args, bool shared, int grid, cudaStream_t stream) {
  if (args.p.head_dim == 64)
    return shared ? launch_t<T, 64, true>(args, grid, stream) : launch_t<T, 64, false>(args, grid, stream);
  return shared ? launch_t<T, 128, true>(args, grid, stream) : launch_t<T, 128, false>(args, grid, stream);
}

// The kernel's maps, of the pools and the queries: encoded for each call, which a call of 20 us and
// more hides.
bool make_maps(PrefillArgs* args, bool bf16) {
  const WindowPrefillParams& p = args->p;
  const uint64_t pool_rows = static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * p.block_size;
  return make_pool_map_uncached(&args->tk, p.k_cache, pool_rows, p.block_size, bf16, p.head_dim) &&
         make_pool_map_uncached(&args->tv, p.v_cache, pool_rows, p.block_size, bf16, p.head_dim) &&
         make_query_map(&args->tq, p.q, p.num_q_heads, p.num_query_tokens, p.group, p.tile_tokens, bf16, p.head_dim) &&
         (p.out_f32 || make_query_map(&args->to, p.out, p.num_q_heads, p.num_query_tokens, p.group, p.tile_tokens, bf16, p.head_dim));
}

}  // namespace

cudaError_t launch_window_prefill(const WindowPrefillParams& p, bool shared, int dtype, cudaStream_t stream) {
  PrefillArgs args{};
  args.p = p;
  const bool bf16 = dtype == PKV_BF16;
  if (!make_maps(&args, bf16)) return cudaErrorInvalidValue;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t items = window_prefill_items(p, shared);
  const int grid = static_cast<int>(items < sms ? items : sms);
  return bf16 ? launch_d<__nv_bfloat16>(args, shared, grid, stream)
              : launch_d<__half>(args, shared, grid, stream);
}

int64_t window_prefill_items(const WindowPrefillParams& p, bool shared) {
  const int span = (shared ? 1 : kGroups) * p.tile_tokens;
  return (static_cast<int64_t>(p.num_query_tokens) / span + p.num_seqs) * p.num_kv_heads;
}

}  // namespace pkv
