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
//    (p rounded, and the rest), so a weight is good to 2^-22 of itself, and to 2^-36 of the
//    largest that the warp has met where that is more (kLift).  Up to four heads per KV
//    head the second part takes columns 4..7 (q's columns are doubled, so the lanes there
//    hold the same p); above, a second MMA.  (One part would be 11 bits of a weight, 2^-11 of
//    it, which a bf16 output shows next to its own 2^-8.)
//
// Work: a unit is 128 tokens of one (sequence, KV head), an item all units of one.  The
// batch's items, in order of sequence and head, each with its units and kItemCost more for
// itself, are cut into spans of equal cost, one per CTA, whatever the lengths are; a CTA
// works through its span item by item.  An item that lies in one span is written out at
// once; of one that does not, each CTA leaves (maximum, sum, O) in the workspace -- at most
// two per CTA, its first and its last item -- and a second kernel joins them.  (A grid over
// (partition, head, sequence) instead kept an SM busy for 0.83 of the time: the last wave's
// CTAs end at different times.)
//
// Each of a CTA's four warps takes 32 of a unit's 128 tokens and runs alone: it has its own
// ring of cp.async stages (lanes 0-7 bring K and V of the tile's first eight rows, 8-15 of
// the next, ...), its own running maximum (raised only when a score exceeds it by 4,
// log2 domain), sum and O, combined through shared memory at the item's end in a fixed
// order.  Waits are cp.async.wait_group only.
//
// Measured (128 sequences of 512 to 4,096 tokens, 64/8 heads, bf16): 88 us a call, 0.64 of
// copy bandwidth (80 us with one fp16 part of the weights), 9 of them the join.  About 365
// instructions per 16 tokens, 216 of them widening.  No one unit is full: while the first kernel
// runs, 60 % of the issue slots are taken, the FMA pipe (fp16 and fp32) is busy 48 % of the time,
// the integer pipe 41 %, the tensor pipe 31 %, HBM 58 %; a warp mostly waits for a pipe or its turn.
#include <type_traits>

#include "kv4.cuh"
#include "launch.h"
#include "mma.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 2;            // MMA tiles of 16 tokens per step: two independent chains of work
constexpr int kTile = 16 * kSub;   // tokens per warp and step
constexpr int kEighths = kTile / 8;  // groups of eight rows: never more than one block each
constexpr int kUnit = kWarps * kTile;  // tokens per unit of work
static_assert(kUnit == kKv4Unit, "the host sizes the grid by it");
constexpr int kItemCost = 2;       // an item's queries, first copies and sums cost about this many units
constexpr int kMinCost = 3;        // per CTA at least
constexpr int kOffs = 16;          // tiles whose block offsets a warp holds at a time
constexpr float kSlack = 4.f;      // a score may exceed the running maximum by this much
// p = 2^(x - m + 11), at most 2^15: as large as fp16 takes, since its numbers end at 2^-24, so the
// second part of a small p, or all of it, is off by up to 2^-25.  (With a slack of 8 and a lift
// of 6 that was 2^-31 of the largest weight: 2^-15 of weights that are 2^-16 of a sink's.  Raising
// the maximum more often costs nothing that shows: 88 us and 73 us as before for 128 sequences of
// 512 to 4,096 tokens and two of 128 Ki.)
constexpr float kLift = 11.f;

// NB blocks of eight columns; kDup: at most four heads, in columns 0..3 and again in 4..7;
// kSplit: f32 queries, in two fp16 parts.
// The kernel's kRound, for f32 outputs: a step's products are summed by MMAs that start from
// zero and added to O by additions that round to nearest.  The MMA truncates its sums; O kept
// in its accumulator shrank by half a unit in the last place per MMA, 2.7e-6 of itself over
// 128 Ki tokens (1.2e-7 with kRound), which a 16-bit output does not show, and adding costs
// registers and instructions (6 % of a batch with 64/8 heads).
template <int D, int NB, bool kDup, bool kSplit>
struct Kv4 {
  static constexpr int kRow = Kv4Row<D>::kBytes;
  static constexpr int kHalf = 8 * kRow;             // bytes of eight rows
  static constexpr int kStage = kEighths * 2 * kHalf;  // K then V of rows 0-7, of rows 8-15, ...
  static constexpr int kHalfPieces = kHalf / 16;
  static constexpr int kLanes = 32 / kEighths;       // lanes that bring K and V of eight rows
  static constexpr int kCopies = (2 * kHalfPieces + kLanes - 1) / kLanes;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kRingBytes = kWarps * kStages * kStage;
  static constexpr int kCols = 8 * NB;
  // the sums at the end take the ring's place: per warp (max, sum) of the columns, O fragments
  static constexpr int kReduceBytes = kWarps * (kCols * 8 + NB * (D / 16) * 32 * 16);
  static constexpr int kMainBytes = kRingBytes > kReduceBytes ? kRingBytes : kReduceBytes;
  static constexpr int kCtasPerSm = NB == 2 ? (D == 128 && kSplit ? 2 : 3) : 4;
  static constexpr int kQueryBytes = NB * (kSplit ? 2 : 1) * (D / 32) * 32 * 16 + kCols * 4;
  static constexpr int kSmemBytes = kMainBytes + kQueryBytes + kWarps * kOffs * kEighths * 8;
};

// What a sequence costs per KV head, in units: its units and what an item costs of its own
// (none where the length is 0 or out of range).
// whole: one, so that each of as many spans is an item (kKv4Whole).
__device__ __forceinline__ int cost_of(int len, int max_len, bool whole) {
  return len <= 0 || len > max_len ? 0 : whole ? 1 : (len + kUnit - 1) / kUnit + kItemCost;
}

// Query fragments of 4-bit K rows in shared memory: piece [w][4 g + t] (16 bytes) is lane
// (g, t)'s B fragment of steps 2w and 2w + 1 for query head g of a block of eight columns.
//
// Lane t of a K row brings the D/4 consecutive values from t D/4 on: word w of its codes
// gives steps 2w (values 0, 4 | 1, 5 of the word) and 2w + 1 (2, 6 | 3, 7).  q is scaled
// (query_power) and held in fp16 parts hi and, with kSplit, lo.  undo[h] takes the scale back.
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
    const int up = query_power(amax, amax == INFINITY);
    const float factor = power_of_two(up);
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
    if (word == 0) undo[h] = power_of_two(-up);
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

template <int D, int NB, bool kDup, bool kSplit, bool kRound>
__global__ void __launch_bounds__(kThreads, Kv4<D, NB, kDup, kSplit>::kCtasPerSm)
decode_kv4_kernel(const __grid_constant__ Kv4DecodeParams p) {
  using C = Kv4<D, NB, kDup, kSplit>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t scan[kThreads / 32 + 1];
  __shared__ int64_t start_before;  // cost of a KV head in the sequences before start_seq
  __shared__ int start_seq;
  __shared__ volatile uint32_t bit_patterns[3];
  grid_dependency_wait();    // of the kernel before: only this one's launch overlaps it
  if (p.desc) grid_dependents_launch();  // the join, which waits for this grid

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int G = p.group;

  // The bit patterns of widening in registers: the compiler would read them from constant
  // memory at every use, and that port is slower (128 sequences, 64/8 heads: 3 us of 90).
  if (threadIdx.x == 0) {
    bit_patterns[0] = p.bits.low;
    bit_patterns[1] = p.bits.high;
    bit_patterns[2] = p.bits.one;
  }
  __syncthreads();
  Kv4Bits bits;
  bits.low = bit_patterns[0];
  bits.high = bit_patterns[1];
  bits.one = bit_patterns[2];

  // ---- empty sequences get the neutral output; lengths out of range are reported
  for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
    const int L = p.context_lens[s];
    if (L == 0) {
      for (int i = threadIdx.x; i < p.num_q_heads * D; i += kThreads)
        store_any(p.out, static_cast<size_t>(s) * p.num_q_heads * D + i, 0.f, p.out_dtype);
    } else if ((L < 0 || L > p.max_len) && threadIdx.x == 0) {
      set_error(p.err, kErrLength);
    }
  }

  // ---- this CTA's span of the batch's units
  int64_t total = 0;
  for (int s = threadIdx.x; s < p.num_seqs; s += kThreads) total += cost_of(p.context_lens[s], p.max_len, p.whole);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  if (lane == 0) scan[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += scan[w];
  __syncthreads();
  const int64_t units = total * p.num_kv_heads;  // the batch's cost
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), p.whole ? units : (units + kMinCost - 1) / kMinCost);
  if (threadIdx.x < 2 && p.desc) p.desc[2 * blockIdx.x + threadIdx.x] = make_int4(-1, 0, 0, 0);
  if (static_cast<int64_t>(blockIdx.x) >= ctas) return;
  int64_t begin = blockIdx.x * units / ctas, end = (blockIdx.x + 1) * units / ctas;

  // ---- the sequence it starts in: the last one with (cost before it) * heads <= begin
  {
    int64_t before = 0;
    for (int base = 0; base < p.num_seqs; base += kThreads) {
      const int s = base + threadIdx.x;
      const int mine = s < p.num_seqs ? cost_of(p.context_lens[s], p.max_len, p.whole) : 0;
      int64_t incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
      }
      if (lane == 31) scan[warp] = incl;
      __syncthreads();
      int64_t all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += scan[w];
        all += scan[w];
      }
      incl += before;
      if (mine > 0 && (incl - mine) * p.num_kv_heads <= begin && begin < incl * p.num_kv_heads) {
        start_seq = s;
        start_before = incl - mine;
      }
      before += all;
      __syncthreads();
      if (begin < before * p.num_kv_heads) break;  // found: begin < units, so it always is
    }
  }
  int s = start_seq, L = p.context_lens[s], cost = cost_of(L, p.max_len, false);
  int kvh, at_cost;  // KV head of the item, and where in its cost the span begins
  {
    const int64_t r = begin - start_before * p.num_kv_heads;
    if (p.whole) {  // the span is item r of the sequence
      kvh = static_cast<int>(r);
      at_cost = 0;
      begin = 0;
      end = cost;
    } else {
      kvh = static_cast<int>(r / cost);
      at_cost = static_cast<int>(r - static_cast<int64_t>(kvh) * cost);
    }
  }

  uint4* q_frag = reinterpret_cast<uint4*>(smem + C::kMainBytes);
  float* q_undo = reinterpret_cast<float*>(smem + C::kMainBytes + C::kQueryBytes - C::kCols * 4);
  // where each eight rows of this warp's next tiles start in the pools, in bytes
  int64_t* offs = reinterpret_cast<int64_t*>(smem + C::kMainBytes + C::kQueryBytes) + warp * kOffs * kEighths;
  const int bs_log2 = 31 - __clz(p.block_size);
  const int64_t block_rows = static_cast<int64_t>(p.block_size) * C::kRow;

  // this lane's share of a tile's copies: pieces piece + kLanes i of its eight rows
  unsigned char* ring = smem + warp * (C::kStages * C::kStage);
  const int eighth = lane / C::kLanes, piece = lane % C::kLanes;
  const uint32_t ring_addr = smem_addr(ring) + eighth * 2 * C::kHalf + piece * 16;
  constexpr int kMixed = C::kHalfPieces / C::kLanes;  // the copy that brings the end of K and the start of V
  const unsigned char* kbase = static_cast<const unsigned char*>(p.k_cache) + piece * 16;
  const unsigned char* vbase = static_cast<const unsigned char*>(p.v_cache) + piece * 16 - C::kHalf;
  const unsigned char* mbase = C::kLanes * kMixed + piece < C::kHalfPieces ? kbase : vbase;

  for (int64_t cur = begin; cur < end;) {
  // the part of the item here: its own cost comes first, then its units
  const int taken = static_cast<int>(min(static_cast<int64_t>(cost - at_cost), end - cur));
  const int n_units = cost - kItemCost, u0 = max(0, at_cost - kItemCost);
  const int count = at_cost + taken - kItemCost - u0;
  if (count > 0) {
  const size_t out_row = static_cast<size_t>(s) * p.num_q_heads + static_cast<size_t>(kvh) * G;
  // this warp's tiles: from token first + i * kUnit on, i < tiles
  const int first = u0 * kUnit + warp * kTile;
  const int tiles = min(count, (L - first + kUnit - 1) / kUnit);  // may be <= 0 in an item's last unit
  const int full = min(tiles, (L - first - kTile + kUnit) / kUnit);  // of them, tiles that end within the context

  auto locate = [&](int i0) {  // tiles i0 .. i0 + kOffs - 1
    __syncwarp();
#pragma unroll
    for (int e = lane; e < kOffs * kEighths; e += 32) {
      const int tok = first + (i0 + e / kEighths) * kUnit + e % kEighths * 8;
      int64_t off = 0;  // rows past the end are not read
      if (i0 + e / kEighths < tiles && tok < L) {
        const int col = tok >> bs_log2;
        int b = col < p.max_blocks_per_seq ? p.block_tables[static_cast<size_t>(s) * p.max_blocks_per_seq + col] : -1;
        if (b < 0 || b >= p.num_blocks) {
          set_error(p.err, kErrIndex);
          b = 0;  // keep the copy in bounds; the flag reports the bad table
        }
        off = (static_cast<int64_t>(b) * p.num_kv_heads + kvh) * block_rows + (tok & (p.block_size - 1)) * C::kRow;
      }
      offs[e] = off;
    }
    __syncwarp();
  };
  auto issue = [&](int i, uint32_t to) {
    if (i < tiles) {
      if (i % kOffs == 0) locate(i);
      const int64_t off = offs[(i % kOffs) * kEighths + eighth];
      const uint32_t bytes = i < full || first + i * kUnit + 8 * eighth < L ? 16u : 0u;  // past the end: zeros
#pragma unroll
      for (int e = 0; e < C::kCopies; ++e)
        if (C::kLanes * (e + 1) <= 2 * C::kHalfPieces || C::kLanes * e + piece < 2 * C::kHalfPieces)
          cp_async16(to + e * C::kLanes * 16,
                     (e < kMixed || C::kLanes * (e + 1) <= C::kHalfPieces ? kbase : e == kMixed ? mbase : vbase) + off +
                         e * C::kLanes * 16,
                     bytes);
    }
    cp_async_commit();  // one group per call, empty past the end: the waits below count them
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) issue(i, ring_addr + i * C::kStage);

  // ---- queries
  stage_queries<D, NB, kSplit>(p.q, p.q_dtype, out_row, G, q_frag, q_undo);
  __syncthreads();
  // (the fragments stay there: four 16-byte loads per step cost less than their registers)
  const uint4* q_lane = q_frag + (kDup ? (g & 3) * 4 + t : lane);
  float sc[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
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
  auto step = [&](int i_tile, auto last) {
    constexpr bool kLast = decltype(last)::value;  // the tile may end past the context
    cp_async_wait<C::kStages - 2>();
    __syncwarp();  // the other lanes' copies too; and everybody has left the stage refilled next
    issue(i_tile + C::kStages - 1, ring_addr + refill);
    refill = at;
    const unsigned char* ks = ring + at;
    at = at == (C::kStages - 1) * C::kStage ? 0 : at + C::kStage;
    const int left = kLast ? L - first - i_tile * kUnit : kTile;  // tokens of this tile

    // ---- scores
    float c[NB][kSub][4];
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      constexpr int kWords = D / 32;
      uint32_t w0[kWords], w1[kWords];
      const unsigned char* r0 = ks + u * 4 * C::kHalf + g * C::kRow;
      const unsigned char* r1 = r0 + 2 * C::kHalf;
      if constexpr (kWords == 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(r0 + t * 16);
        const uint4 b = *reinterpret_cast<const uint4*>(r1 + t * 16);
        w0[0] = a.x; w0[1] = a.y; w0[2] = a.z; w0[3] = a.w;
        w1[0] = b.x; w1[1] = b.y; w1[2] = b.z; w1[3] = b.w;
      } else {
        const uint2 a = *reinterpret_cast<const uint2*>(r0 + t * 8);
        const uint2 b = *reinterpret_cast<const uint2*>(r1 + t * 8);
        w0[0] = a.x; w0[1] = a.y;
        w1[0] = b.x; w1[1] = b.y;
      }
      const int pair = D / 2 + 4 * (t * D / 128);
      const __half2 p0 = *reinterpret_cast<const __half2*>(r0 + pair);
      const __half2 p1 = *reinterpret_cast<const __half2*>(r1 + pair);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t a[4], b[4];
        kv4_word(w0[i], __low2half2(p0), __high2half2(p0), bits, a);
        kv4_word(w1[i], __low2half2(p1), __high2half2(p1), bits, b);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint4 q = q_lane[(nb * (kSplit ? 2 : 1) * (D / 32) + i) * 32];
          if (i == 0) {
            mma_f16_first(c[nb][u], a[0], b[0], a[1], b[1], q.x, q.y);
            mma_f16(c[nb][u], a[2], b[2], a[3], b[3], q.z, q.w);
          } else {
            mma_f16(c[nb][u], a[0], b[0], a[1], b[1], q.x, q.y);
            mma_f16(c[nb][u], a[2], b[2], a[3], b[3], q.z, q.w);
          }
          if (kSplit) {
            const uint4 r = q_lane[((nb * 2 + 1) * (D / 32) + i) * 32];
            mma_f16(c[nb][u], a[0], b[0], a[1], b[1], r.x, r.y);
            mma_f16(c[nb][u], a[2], b[2], a[3], b[3], r.z, r.w);
          }
        }
      }
    }

    // V's codes and pairs of rows 2t, 2t + 1 of a tile's first eight and of its last, asked for
    // before the softmax (its vote keeps the compiler from doing so)
    constexpr int kVWords = D / 64;  // of codes per row and lane
    uint32_t vw[kSub][4][kVWords], pr[kSub][4];
    auto load_v = [&](int u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned char* row = ks + (u * 4 + (i & 2) + 1) * C::kHalf + (2 * t + (i & 1)) * C::kRow;
        if constexpr (kVWords == 2) {
          const uint2 a = *reinterpret_cast<const uint2*>(row + g * 8);
          vw[u][i][0] = a.x;
          vw[u][i][1] = a.y;
        } else {
          vw[u][i][0] = *reinterpret_cast<const uint32_t*>(row + g * 4);
        }
        pr[u][i] = *reinterpret_cast<const uint32_t*>(row + D / 2 + 4 * (g * D / 256));
        // past the end a row holds anything, NaN too: step = lo = 0 makes it zero
        if (kLast && u * 16 + 2 * t + (i & 1) + (i & 2) * 4 >= left) pr[u][i] = 0u;
      }
    };
    load_v(0);

    // ---- softmax; tokens past the end get -inf
    uint32_t ph[NB][kSub][2];                   // P^T fragments: tokens 0-7 and 8-15
    [[maybe_unused]] uint32_t pl[NB][kSub][2];  // their second parts (kDup: in ph's columns 4..7)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x[kSub][4];  // score - m + kLift
      const float ma = kLift - m[nb][0], mb = kLift - m[nb][1];
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[u][i] = fmaf(c[nb][u][i], sc[nb][i & 1], i & 1 ? mb : ma);
          if (kLast && u * 16 + g + (i & 2) * 4 >= left) x[u][i] = -INFINITY;
          top = fmaxf(top, x[u][i]);
        }
      if (__any_sync(0xffffffffu, top > kLift + kSlack)) {
        // raise both columns' maxima: scores again (m = -inf makes x = inf), their largest
        float top2[2] = {m[nb][0], m[nb][1]};
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[u][i] = c[nb][u][i] * sc[nb][i & 1];
            if (kLast && u * 16 + g + (i & 2) * 4 >= left) x[u][i] = -INFINITY;
            top2[i & 1] = fmaxf(top2[i & 1], x[u][i]);
          }
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top2[e] = fmaxf(top2[e], __shfl_xor_sync(0xffffffffu, top2[e], off));
          // a column that saw nothing but NaN yet keeps m = -inf, and its NaN sum
          f[e] = top2[e] == m[nb][e] ? 1.f : exp2_approx(m[nb][e] - top2[e]);
          m[nb][e] = top2[e];
          l[nb][e] *= f[e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[nb][i][0] *= f[0];
          o[nb][i][1] *= f[1];
          o[nb][i][2] *= f[0];
          o[nb][i][3] *= f[1];
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[u][i] = x[u][i] - m[nb][i & 1] + kLift;
      }
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = exp2_approx(x[u][i]);
        l[nb][0] += e[0] + e[2];
        l[nb][1] += e[1] + e[3];
        uint32_t h0 = pack_half2(e[0], e[1]), h1 = pack_half2(e[2], e[3]);
        const uint32_t r0 = pack_half2_rest(e[0], e[1], h0), r1 = pack_half2_rest(e[2], e[3], h1);
        if constexpr (kDup) {
          if (t >= 2) {
            h0 = r0;
            h1 = r1;
          }
        } else {
          pl[nb][u][0] = movmatrix_trans(r0);
          pl[nb][u][1] = movmatrix_trans(r1);
        }
        ph[nb][u][0] = movmatrix_trans(h0);
        ph[nb][u][1] = movmatrix_trans(h1);
      }
    }

    // ---- output
#pragma unroll
    for (int u = 1; u < kSub; ++u) load_v(u);
    auto pairs_of = [&](int u, __half2 (&step)[2], __half2 (&lo)[2]) {  // tokens (2t, 2t + 1), (2t + 8, 2t + 9)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        step[e] = as_half2(__byte_perm(pr[u][2 * e], pr[u][2 * e + 1], 0x5410));
        lo[e] = as_half2(__byte_perm(pr[u][2 * e], pr[u][2 * e + 1], 0x7632));
      }
    };
    auto widen_v = [&](int u, int i, int j, const __half2 (&step)[2], const __half2 (&lo)[2], uint32_t (&a)[4]) {
      const uint32_t sel = 0x4400u + 0x1111u * j;  // byte j of both words, twice each
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t x = __byte_perm(vw[u][2 * e][i], vw[u][2 * e + 1][i], sel);
        a[2 * e] = as_u32(__hfma2(low_codes(x, bits), step[e], lo[e]));
        a[2 * e + 1] = as_u32(__hfma2(high_codes(x, bits), step[e], lo[e]));
      }
    };
    if constexpr (kRound) {
      __half2 step[kSub][2], lo[kSub][2];
#pragma unroll
      for (int u = 0; u < kSub; ++u) pairs_of(u, step[u], lo[u]);
#pragma unroll
      for (int i = 0; i < kVWords; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float sum[NB][4];
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            uint32_t a[4];
            widen_v(u, i, j, step[u], lo[u], a);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if (u == 0)
                mma_f16_first(sum[nb], a[0], a[1], a[2], a[3], ph[nb][u][0], ph[nb][u][1]);
              else
                mma_f16(sum[nb], a[0], a[1], a[2], a[3], ph[nb][u][0], ph[nb][u][1]);
              if constexpr (!kDup) mma_f16(sum[nb], a[0], a[1], a[2], a[3], pl[nb][u][0], pl[nb][u][1]);
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nb][4 * i + j][e] += sum[nb][e];
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        __half2 step[2], lo[2];
        pairs_of(u, step, lo);
#pragma unroll
        for (int i = 0; i < kVWords; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a[4];
            widen_v(u, i, j, step, lo, a);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              mma_f16(o[nb][4 * i + j], a[0], a[1], a[2], a[3], ph[nb][u][0], ph[nb][u][1]);
              if constexpr (!kDup) mma_f16(o[nb][4 * i + j], a[0], a[1], a[2], a[3], pl[nb][u][0], pl[nb][u][1]);
            }
          }
        }
      }
    }
  };
  int i_tile = 0;
  for (; i_tile < full; ++i_tile) step(i_tile, std::false_type{});
  if (i_tile < tiles) step(i_tile, std::true_type{});
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
    const int slot = 2 * blockIdx.x + (u0 == 0);  // of an item that is not all here
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
        if (count == n_units) {
          store_pair(p.out, row * D + d, a / lsum[e], b / lsum[e], p.out_dtype);
        } else {
          const size_t k = static_cast<size_t>(slot) * G + h + e;
          *reinterpret_cast<float2*>(p.ws_o + k * D + d) = make_float2(a, b);
          if (i == 0 && g == 0) p.ws_ml[k] = make_float2(M[e], lsum[e]);
        }
      }
    }
  }
  if (threadIdx.x == 0 && count < n_units) {
    // place x of the batch's cost is in the span of the last CTA c with c * units / ctas <= x
    auto span_of = [&](int64_t x) {
      const int64_t y = (x + 1) * ctas + units - 1;
      return y < (int64_t{1} << 32) ? static_cast<int>(static_cast<uint32_t>(y) / static_cast<uint32_t>(units)) - 1
                                    : static_cast<int>(y / units - 1);
    };
    const int64_t at = cur - at_cost;  // the item's first place; its units begin kItemCost later
    p.desc[2 * blockIdx.x + (u0 == 0)] = make_int4(s, kvh, span_of(at + kItemCost), span_of(at + cost - 1));
  }
  __syncthreads();  // the sums have been read: the ring and the queries take their place
  }

  // ---- the next item
  cur += taken;
  at_cost = 0;
  if (cur < end && ++kvh == p.num_kv_heads) {
    kvh = 0;
    do {
      if (++s >= p.num_seqs) return;  // not reached: the span has cost left
      L = p.context_lens[s];
      cost = cost_of(L, p.max_len, false);
    } while (cost == 0);
  }
  }
}

// Joins the items that lie in several spans, a CTA per span.  An item's pieces are the last
// item of its first span (slot 2 start + 1) and the first ones of the others (slots 2c).  Its
// tasks are 64 dimensions of a head each: a lane takes a piece at a time for the factors
// 2^(m - M), then two dimensions for the sum.  Up to kFew pieces are joined by the first span's
// CTA, a warp per task, whose loads all leave at once.  The CTAs of more share out the tasks in
// turn, and one with fewer tasks than warps shares a task's pieces out among its warps (one
// sequence of 128 Ki tokens and one KV head is 342 pieces: joined by its first CTA alone, 16
// heads took 240 us behind 13 us of attention).
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kFew = 8;
__global__ void __launch_bounds__(kJoinThreads) join_kv4_kernel(const __grid_constant__ Kv4DecodeParams p) {
  __shared__ float2 partial[kJoinWarps][32];
  grid_dependency_wait();
  const int G = p.group, D = p.head_dim, parts = D / 64, tasks = G * parts;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int4 continued = p.desc[2 * blockIdx.x], begun = p.desc[2 * blockIdx.x + 1];
  auto first_row = [&](const int4& d) {
    return static_cast<size_t>(d.x) * p.num_q_heads + static_cast<size_t>(d.y) * G;
  };
  auto slot = [&](const int4& d, int i) { return static_cast<size_t>(2 * (d.z + i) + (i == 0)) * G; };

  if (begun.x >= 0 && begun.w - begun.z < kFew) {
    const int n = begun.w - begun.z + 1;
    for (int x = warp; x < tasks; x += kJoinWarps) {
      const int h = x / parts, e = x % parts * 64 + 2 * lane;
      float2 o[kFew];
#pragma unroll
      for (int i = 0; i < kFew; ++i)
        o[i] = i < n ? *reinterpret_cast<const float2*>(p.ws_o + (slot(begun, i) + h) * D + e) : make_float2(0.f, 0.f);
      const int mine = lane % kFew;
      const float2 ml = mine < n ? p.ws_ml[slot(begun, mine) + h] : make_float2(-INFINITY, 0.f);
      float M = ml.x;
#pragma unroll
      for (int off = 1; off < kFew; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      const float f = mine < n ? exp2_approx(ml.x - M) : 0.f;
      const float lsum = group_sum<kFew>(f * ml.y);
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        a = fmaf(w, o[i].x, a);
        b = fmaf(w, o[i].y, b);
      }
      store_pair(p.out, (first_row(begun) + h) * D + e, a / lsum, b / lsum, p.out_dtype);
    }
  }

#pragma unroll 1
  for (int role = 0; role < 2; ++role) {
    const int4 d = role ? begun : continued;
    if (d.x < 0 || d.w - d.z < kFew) continue;
    const int n = d.w - d.z + 1, rank = blockIdx.x - d.z;
    const int mine = rank < tasks ? (tasks - rank + n - 1) / n : 0;
    const int share = mine >= 8 ? 1 : mine >= 4 ? 2 : mine >= 2 ? 4 : 8;  // warps per task
    for (int k0 = 0; k0 < mine; k0 += kJoinWarps / share) {
      const int k = k0 + warp / share, sub = warp % share;
      const int x = rank + k * n, h = x / parts, e = x % parts * 64 + 2 * lane;
      float lsum = 0.f, a = 0.f, b = 0.f;
      if (k < mine) {
        float M = -INFINITY;
        for (int i = lane; i < n; i += 32) M = fmaxf(M, p.ws_ml[slot(d, i) + h].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        for (int i = lane; i < n; i += 32) {
          const float2 ml = p.ws_ml[slot(d, i) + h];
          lsum = fmaf(exp2_approx(ml.x - M), ml.y, lsum);
        }
        lsum = group_sum<32>(lsum);  // of all pieces, in every warp of the task
        for (int base = sub; base < n; base += 32 * share) {  // pieces base, base + share, ...
          const int at = base + lane * share;
          const float f = at < n ? exp2_approx(p.ws_ml[slot(d, at) + h].x - M) : 0.f;
          for (int i0 = 0; i0 < 32 && base + i0 * share < n; i0 += 16) {
            float2 o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int j = base + (i0 + i) * share;
              o[i] = j < n ? *reinterpret_cast<const float2*>(p.ws_o + (slot(d, j) + h) * D + e) : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float w = __shfl_sync(0xffffffffu, f, i0 + i);
              a = fmaf(w, o[i].x, a);
              b = fmaf(w, o[i].y, b);
            }
          }
        }
      }
      if (share > 1) {
        __syncthreads();  // the sums of the tasks before have been read
        partial[warp][lane] = make_float2(a, b);
        __syncthreads();
        if (sub == 0)
          for (int w = 1; w < share; ++w) {
            const float2 y = partial[warp + w][lane];
            a += y.x;
            b += y.y;
          }
      }
      if (sub == 0 && k < mine) store_pair(p.out, (first_row(d) + h) * D + e, a / lsum, b / lsum, p.out_dtype);
    }
  }
}

template <int D, int NB, bool kDup, bool kSplit, bool kRound>
cudaError_t launch_t(const Kv4DecodeParams& p, cudaStream_t stream) {
  using C = Kv4<D, NB, kDup, kSplit>;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem_limit(decode_kv4_kernel<D, NB, kDup, kSplit, kRound>, C::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(decode_kv4_kernel<D, NB, kDup, kSplit, kRound>, p.ctas, kThreads, C::kSmemBytes, stream, p);
}

template <int D, bool kSplit, bool kRound>
cudaError_t launch_g(const Kv4DecodeParams& p, cudaStream_t stream) {
  if (p.group <= 4) return launch_t<D, 1, true, kSplit, kRound>(p, stream);
  if (p.group <= 8) return launch_t<D, 1, false, kSplit, kRound>(p, stream);
  return launch_t<D, 2, false, kSplit, kRound>(p, stream);
}

template <int D>
cudaError_t launch_d(const Kv4DecodeParams& p, cudaStream_t stream) {
  if (p.q_dtype == PKV_F32) return launch_g<D, true, true>(p, stream);  // f32 out as well
  if (p.out_dtype == PKV_F32) return launch_g<D, false, true>(p, stream);
  return launch_g<D, false, false>(p, stream);
}

}  // namespace

int kv4_decode_ctas(int head_dim, int group, int q_dtype, int64_t max_units, int64_t items) {
  int per_sm;
  if (head_dim == 128)
    per_sm = group <= 8 ? Kv4<128, 1, false, false>::kCtasPerSm
                        : q_dtype == PKV_F32 ? Kv4<128, 2, false, true>::kCtasPerSm : Kv4<128, 2, false, false>::kCtasPerSm;
  else
    per_sm = group <= 8 ? Kv4<64, 1, false, false>::kCtasPerSm : Kv4<64, 2, false, false>::kCtasPerSm;
  const int64_t most = (max_units + items * kItemCost + kMinCost - 1) / kMinCost;
  return static_cast<int>(most < 152 * per_sm ? most : 152 * per_sm);
}

cudaError_t launch_decode_kv4(const Kv4DecodeParams& p, cudaStream_t stream) {
  const cudaError_t e = p.head_dim == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
  if (e != cudaSuccess || !p.desc) return e;
  return launch_dependent(join_kv4_kernel, p.ctas, kJoinThreads, 0, stream, p);
}

}  // namespace pkv
