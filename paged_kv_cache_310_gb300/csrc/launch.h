// launch.h -- host-side launchers shared between the translation units of
// libpagedkv (not part of the public ABI; see include/pagedkv.h for that).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pagedkv.h"

namespace pkv {

// Everything decode kernels need, by value (one __grid_constant__ struct).
struct DecodeParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* out;
  float* ws_o;   // [S][Hq][max_parts][D] un-normalised partition outputs (fp32)
  float* ws_ml;  // [S][Hq][max_parts][2] partition (max, sum) in the log2 domain
  int* err;      // device error flag
  int4* work_list;  // tensor-core path: items sorted longest first (work-list kernel)
  int* work_count;  // number of entries in work_list
  int* work_next;   // claims so far past the grid's first entries (reset by the work-list kernel)
  int32_t num_seqs, num_q_heads, num_kv_heads, group, max_blocks_per_seq;
  int32_t block_size, num_blocks, head_dim;
  int32_t part_tokens, max_parts;
  int32_t out_f32;   // 1: out is fp32, 0: out has the cache dtype
  float scale_log2;  // softmax scale * log2(e): scores live in the exp2 domain
  uint64_t wait_limit_ns;  // bound of every pipeline wait (kWaitLimitNs unless a test lowers it)
  int32_t heads_per_item;  // KV heads of one tensor-core work item: 1, or 2 (head_dim 64, paired heads)
};

// Multi-token causal (prefill) attention, tensor cores; f16/bf16, head_dim 64 or 128.
struct PrefillParams {
  const void* q;  // [T][Hq][head_dim]
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // [S+1]
  void* out;                   // [T][Hq][head_dim]
  int4* work_list;
  int* work_count;
  int* err;
  int32_t num_seqs, num_q_heads, num_kv_heads, group, max_blocks_per_seq;
  int32_t block_size, num_blocks, max_context_len, num_query_tokens, tile_tokens;
  int32_t head_dim;  // 64 or 128
  int32_t out_f32;
  float scale_log2;
  uint64_t wait_limit_ns;  // bound of every pipeline wait (kWaitLimitNs unless a test lowers it)
};
int prefill_tile_tokens(int group);
size_t prefill_max_items(int num_seqs, int num_query_tokens, int num_kv_heads, int group);
cudaError_t launch_prefill_tc(const PrefillParams& p, int dtype, cudaStream_t stream);

// CUDA-core split-K decode (any supported dtype, head_dim 64/128, group <= 8).
cudaError_t launch_decode_simt(const DecodeParams& p, int dtype, cudaStream_t stream);
// Tensor-core (tcgen05) decode: f16/bf16, head_dim 64/128, group <= 16, persistent CTAs
// fed by a work list that a one-CTA kernel builds first.  Partitions <= 4096 tokens.
constexpr int kTcMaxPartition = 4096;
bool tc_supported(int dtype, int head_dim, int group, int block_size);
// KV heads one work item of the 16-bit tensor-core decode covers (2: paired heads).
int tc_heads_per_item(int dtype, int head_dim, int num_kv_heads);
cudaError_t launch_decode_tc(const DecodeParams& p, int dtype, cudaStream_t stream);
// The f32 (tf32, split-operand) decode kernel over a work list already launched on the
// stream; head_dim 64/128, group <= 8.
cudaError_t launch_decode_tc32(const DecodeParams& p, int grid, cudaStream_t stream);
// Partition merge for sequences longer than one partition.
cudaError_t launch_merge(const DecodeParams& p, int dtype, cudaStream_t stream);

// Records a failure message for paged_kv_last_error() on this host thread.
pkv_status record_error(pkv_status status, const char* message);

// Swap whole blocks between the pools and a device-reachable staging buffer.
cudaError_t launch_swap(bool out, const int64_t* ids, int32_t n, void* k_cache, void* v_cache, void* stage_k,
                        void* stage_v, int64_t block_bytes, int32_t num_blocks, int* err, cudaStream_t stream);

// Diagnostic: one bounded wait that cannot complete (see paged_kv_selftest_wait_timeout).
cudaError_t launch_wait_timeout_selftest(uint64_t limit_ns, int* err, cudaStream_t stream);

cudaError_t launch_append(const void* k, const void* v, const int64_t* slots, int32_t num_tokens,
                          void* k_cache, void* v_cache, int32_t num_kv_heads, int32_t block_size,
                          int32_t row_bytes, int64_t num_slots, int* err, cudaStream_t stream);

cudaError_t launch_block_copy(const int64_t* pairs, int32_t num_pairs, void* k_cache,
                              void* v_cache, int64_t block_bytes, int32_t num_blocks, int* err,
                              cudaStream_t stream);

cudaError_t launch_gather(const void* k_cache, const void* v_cache, const int32_t* block_tables,
                          int32_t max_blocks_per_seq, const int32_t* context_lens,
                          int32_t num_seqs, int32_t max_len, void* k_out, void* v_out,
                          int32_t num_kv_heads, int32_t block_size, int32_t row_bytes,
                          int32_t num_blocks, int* err, cudaStream_t stream);

// ---- 4-bit caches (PKV_KV4 pools)

// The bit patterns that widening 4-bit codes uses.  Kernels get them as an argument: as
// literals the assembler splits (w & mask) | bits into two instructions (a lop3 takes one
// literal), and the integer pipe is what widening is bound by.
struct Kv4Bits {
  uint32_t low = 0x000f000fu;   // half-bytes 0 and 4 of a word
  uint32_t high = 0x00f000f0u;  // half-bytes 1 and 5
  uint32_t one = 0x64006400u;   // fp16 1024, whose last bits are units, twice
};

struct Kv4AppendParams {
  const void* k;
  const void* v;
  const int64_t* slots;
  void* k_cache;
  void* v_cache;
  int* err;
  int64_t num_slots;
  int32_t num_tokens, num_kv_heads, block_size, head_dim;
  int32_t tokens_per_cta;  // set by the launcher
};
cudaError_t launch_kv4_append(Kv4AppendParams p, int dtype, cudaStream_t stream);

struct Kv4ExpandParams {
  const int64_t* pairs;
  const void* k_cache;  // 4-bit pools
  const void* v_cache;
  void* k_out;  // pools of the wide dtype
  void* v_out;
  int* err;
  int32_t num_pairs, num_blocks, num_out_blocks, num_kv_heads, block_size, head_dim;
  int32_t pairs_per_cta;  // set by the launcher
  Kv4Bits bits;
};
cudaError_t launch_kv4_expand(Kv4ExpandParams p, int dtype, cudaStream_t stream);

// Single-token attention over 4-bit pools (head_dim 64/128, group <= 16).
struct Kv4DecodeParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* out;
  int4* desc;    // workspace [ctas][2]: the unfinished items a CTA continues and begins (sequence, KV head,
                 // first and last CTA; -1: none); NULL: none can be
  float2* ws_ml; // workspace [2 ctas][G]: (maximum, sum) of an unfinished item
  float* ws_o;   // workspace [2 ctas][G][D]: its un-normalised output
  int* err;
  int32_t q_dtype, out_dtype, num_seqs, num_q_heads, num_kv_heads, group, max_blocks_per_seq;
  int32_t block_size, num_blocks, head_dim, max_len, ctas;
  bool whole;  // a CTA takes whole items
  float scale_log2;
  Kv4Bits bits;
};
constexpr int kKv4MaxGroup = 16;
constexpr int kKv4Unit = 128;  // tokens of one unit of work
// Up to here items are not split if the GPU holds a CTA for each at once: no workspace and no
// second kernel, which cost more than splitting so few tokens saves (70 sequences of 512, 32/8
// heads: 14 us against 20; one: 8 against 9).
constexpr int kKv4Whole = 512;
// CTAs of a call over at most max_units units in `items` (sequence, KV head) items.
int kv4_decode_ctas(int head_dim, int group, int q_dtype, int64_t max_units, int64_t items);
cudaError_t launch_decode_kv4(const Kv4DecodeParams& p, cudaStream_t stream);

// ---- attention weights and eviction
struct WeightsParams {  // of one turn's sequences (all of the batch, or as many as the workspace has scores for)
  const void* q;
  const void* k_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* tracked_lens;  // NULL: every row has an accumulator
  const float* weights;         // [S][Hkv][width]
  float* weights_out;           // may be weights
  float* scores;                // workspace [S][Hq][scores_ld]: log2-domain scores; NULL: kept in shared memory
  float* ws_ml;                 // workspace [S][Hq][max_parts][2]
  int* err;
  int64_t width, scores_ld;
  int32_t q_dtype, num_seqs, num_q_heads, num_kv_heads, group, max_blocks_per_seq;
  int32_t block_size, num_blocks, head_dim, max_len, part_tokens, max_parts;
  float scale_log2;
  Kv4Bits bits;
};
constexpr int kWeightsMaxGroup = 16;
constexpr int kWeightsOne = 512;  // up to here one CTA sees all tokens of a (sequence, KV head)
cudaError_t launch_weights(const WeightsParams& p, int dtype, cudaStream_t stream);

struct EvictParams {
  const float* weights;  // [S][Hkv][width]
  float* weights_out;    // same shape
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* keep_lens;
  const int32_t* new_tables;
  int32_t* kept;  // [S][Hkv][max_keep]
  void* k_cache;
  void* v_cache;
  int* err;
  int64_t width;
  int32_t num_seqs, num_kv_heads, max_blocks_per_seq, max_new_blocks;
  int32_t block_size, num_blocks, row_bytes, max_len, max_keep, recent;
  int32_t key_room;  // rows whose keys a CTA holds in shared memory; set by the launcher
};
cudaError_t launch_evict(EvictParams p, cudaStream_t stream);

}  // namespace pkv
