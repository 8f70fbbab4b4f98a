/*
 * pagedkv.h -- C ABI of libpagedkv.so: the data-parallel hot path of PagedAttention
 * on one GB300 (sm_103a).
 *
 * The method (four web pages on PagedAttention / vLLM):
 *  - "anthology-of-the-sota note-023", Method: a sequence's KV cache is cut into
 *    fixed-size blocks of a fixed number of tokens; a per-sequence block table maps
 *    logical block i to a physical block; attention gathers K/V from those
 *    non-contiguous blocks; blocks are allocated as the sequence grows and shared
 *    between sequences, with copy-on-write when one of them diverges.
 *  - "Efficient Memory Management for Large Language Model Serving with
 *    PagedAttention", How It Works: blocks of e.g. 16 tokens; the block table plays
 *    the part of an OS page table; copy-on-write for parallel sampling / beam search.
 *  - "Paged Attention" glossary, paragraph 4: attention's arithmetic is unchanged,
 *    only the storage of K/V moves; GQA paragraph: several query heads share one
 *    key/value head (Llama 2 70B: 64 query heads, 8 KV heads).
 *
 * Layouts (the pages fix none; this library's reading):
 *  - k_cache, v_cache: [num_blocks][num_kv_heads][block_size][head_dim], row-major.
 *    One (block, kv head) tile is block_size*head_dim contiguous elements.
 *  - q, out: [num_seqs][num_q_heads][head_dim].  Query head h reads KV head
 *    h / (num_q_heads / num_kv_heads).
 *  - k, v of new tokens: [num_tokens][num_kv_heads][head_dim].
 *  - block_tables: int32 [num_seqs][max_blocks_per_seq]; entry i of row s is the
 *    physical block of logical block i of sequence s.  Entries at or past
 *    ceil(context_lens[s] / block_size) are never read.
 *  - context_lens: int32 [num_seqs], tokens each sequence attends over (>= 0).
 *  - slot_mapping: int64 [num_tokens]; slot = physical_block * block_size + row;
 *    a negative slot is padding and is skipped.
 *  - src_dst_pairs: int64 [num_pairs][2] of (source block, destination block).
 *
 * Conventions:
 *  - Ownership: the caller owns every buffer.  Apart from arguments documented as
 *    host memory, every pointer is device memory of the current device.  The
 *    library allocates no device memory and keeps no pointer after a call returns.
 *    Caller-provided workspace holds the tensor-core decode work list, split-K
 *    partials and the prefill work list (the *_workspace_bytes calls size it).
 *  - Streams: `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *    call only enqueues work and returns; results are ready when the stream is.
 *    The calls can be captured in a CUDA graph once each kind has run once outside
 *    the capture (the first call sets its kernels' shared-memory limits).
 *  - Early start: the tensor-core decode's first kernel (its work list) is launched
 *    as a programmatic dependent of the kernel before it on the stream, so that it
 *    overlaps paged_kv_append.  Before it waits for that kernel it reads
 *    context_lens and writes its workspace and the zero rows of out for empty
 *    sequences.  A kernel that only ends, or one of this library's kernels, is
 *    always safe before it.  A caller's own kernel that releases its dependents
 *    early (griddepcontrol.launch_dependents) must do so only after its last write
 *    to context_lens, and must not touch out or the workspace after that point.
 *  - Alignment: q, k, v, out, k_cache, v_cache must be 16-byte aligned, and
 *    head_dim * element size must be a multiple of 16 bytes.
 *  - Errors: a call returns PKV_OK or an error status and records a message that
 *    paged_kv_last_error() returns (per host thread).  Host checks cover shapes,
 *    scalars, pointers and alignment.  Device-side index faults never trap: a
 *    kernel that meets an out-of-range block id or slot, or a bounded wait that
 *    runs out, sets a device flag, skips the access and completes;
 *    paged_kv_device_error() reports and clears that flag.
 *  - Supported set: dtype f32, f16, bf16 (q, k, v, caches share it); out dtype
 *    either that dtype or f32; head_dim 64 or 128; block_size 8, 16, 32 or 64;
 *    num_q_heads a multiple of num_kv_heads.  Group size (query heads per KV head)
 *    up to 8 on the CUDA-core decode path; on the tensor-core decode path up to 16
 *    for f16/bf16 and up to 8 for f32 (tf32 MMAs on split operands: scores to about
 *    2^-21 relative, within the f32 tolerance for logits of a few units; for logits
 *    of tens of units choose PKV_PATH_CUDA_CORE, fp32 throughout); prefill on tensor
 *    cores for f16/bf16, groups up to 16.  4-bit pools (PKV_KV4), eviction, rotary positions and
 *    sliding windows have their own calls below; block copies and swaps take 4-bit pools too.
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* PKV_KV4: a 4-bit pool (see "4-bit caches" below); only the calls that say so take it. */
typedef enum { PKV_F32 = 0, PKV_F16 = 1, PKV_BF16 = 2, PKV_KV4 = 3 } pkv_dtype;

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,    /* bad pointer, shape, scalar or alignment */
  PKV_ERR_UNSUPPORTED = 2,    /* outside the supported set above */
  PKV_ERR_WORKSPACE = 3,      /* workspace missing or smaller than required */
  PKV_ERR_CUDA = 4,           /* a CUDA runtime call or launch failed */
  PKV_ERR_DEVICE_INDEX = 5,   /* a kernel met an out-of-range block id, slot or length */
  PKV_ERR_DEVICE_TIMEOUT = 6, /* a kernel's bounded wait ran out (copy never landed) */
  PKV_ERR_OUT_OF_BLOCKS = 7   /* block manager: not enough free physical blocks */
} pkv_status;

/* Geometry of one layer's block pool (both k_cache and v_cache). */
typedef struct {
  int32_t num_blocks;   /* physical blocks in the pool */
  int32_t block_size;   /* tokens per block: 8, 16, 32 or 64 */
  int32_t num_kv_heads;
  int32_t head_dim;     /* 64 or 128 */
  int32_t dtype;        /* pkv_dtype of the caches, q, k and v (PKV_KV4: of the caches) */
} pkv_cache_desc;

/* Decode path selection and split-K partition size (NULL config = automatic: tensor
 * cores for f16/bf16 with groups <= 16 and for f32 at head_dim 128 with groups 5 to 8,
 * CUDA cores otherwise). */
typedef enum { PKV_PATH_AUTO = 0, PKV_PATH_CUDA_CORE = 1, PKV_PATH_TENSOR_CORE = 2 } pkv_path;

typedef struct {
  int32_t path;              /* pkv_path */
  int32_t partition_tokens;  /* 0 = automatic, else a positive multiple of 128 */
} pkv_decode_config;

/*
 * paged_kv_append -- write new tokens' K and V into their cache slots.
 * Pages: "Efficient Memory Management ... with PagedAttention", How It Works (blocks
 * filled as tokens are generated, allocated on demand); note-023, Method.
 *
 * For each token t with slot_mapping[t] >= 0 and every KV head h:
 *   k_cache[slot / block_size][h][slot % block_size][:] = k[t][h][:], same for v.
 * Bit-exact copies.  Slots must be distinct (duplicates race).  A slot
 * >= num_blocks * block_size sets the device index flag and is skipped.
 * k, v: device [num_tokens][num_kv_heads][head_dim]; slot_mapping: device int64.
 */
pkv_status paged_kv_append(const void* k, const void* v, const int64_t* slot_mapping,
                           int32_t num_tokens, void* k_cache, void* v_cache,
                           const pkv_cache_desc* cache, void* stream);

/*
 * paged_block_copy -- copy-on-write divergence: block dst becomes a copy of block
 * src in both pools (all KV heads and rows).
 * Pages: note-023, Concepts (copy-on-write gives the writer its own copy of a shared
 * block); "Paged Attention" glossary, paragraph 2; "Efficient Memory Management ...",
 * How It Works (copy when a sequence sharing a prefix diverges).
 *
 * src_dst_pairs: device int64 [num_pairs][2].  host_pairs: optional host copy of the
 * same pairs; when given, the call checks every id is in [0, num_blocks), src != dst,
 * no dst repeats and no dst is also a src (PKV_ERR_INVALID_ARG otherwise).  Without
 * it, out-of-range ids set the device index flag and are skipped; overlapping pairs
 * are the caller's responsibility.  Bit-exact.
 */
pkv_status paged_block_copy(const int64_t* src_dst_pairs, const int64_t* host_pairs,
                            int32_t num_pairs, void* k_cache, void* v_cache,
                            const pkv_cache_desc* cache, void* stream);

/* What paged_attention_decode will do for these sizes and config. */
typedef struct {
  int32_t path;              /* pkv_path actually taken (never PKV_PATH_AUTO) */
  int32_t partition_tokens;  /* tokens per split-K partition */
  int32_t max_partitions;    /* partitions of the longest sequence (1 = no merge) */
  int32_t kernel_launches;   /* kernels one call enqueues */
  size_t workspace_bytes;    /* as paged_attention_workspace_bytes */
  int32_t kv_heads_per_item; /* tensor-core path: KV heads one work item covers; 2 for f16/bf16
                                at head_dim 64 with an even number of KV heads (their tiles of a
                                block are adjacent and load as one head_dim-128 tile), else 1 */
} pkv_decode_plan;

/*
 * paged_attention_plan -- fill *out with the plan paged_attention_decode follows for
 * these arguments (host only, no device work).  Automatic partitions: on CUDA cores
 * 512 to 2048 tokens, aiming at about 12 CTAs per SM; on tensor cores the largest
 * size up to 4096 that leaves about three (sequence, KV head, partition) items per SM
 * (lengths assumed to average half of max_context_len).  Errors as
 * paged_attention_decode's argument checks.
 */
pkv_status paged_attention_plan(int32_t num_seqs, int32_t num_q_heads, int32_t max_context_len,
                                const pkv_cache_desc* cache, const pkv_decode_config* config,
                                pkv_decode_plan* out);

/*
 * paged_block_swap_out / paged_block_swap_in -- preemption under memory pressure: move
 * whole blocks (all KV heads and rows of K and V) between the pools and CPU memory, so
 * a preempted sequence can be restored later and continue exactly where it stopped.
 * Pages: "Paged Attention" glossary, paragraphs 3 and 5 (blocks of preempted sequences
 * are evicted to CPU RAM and swapped back, generation resumes where it left off);
 * "Efficient Memory Management ...", How It Works (preemption and swapping).
 *
 * block_ids: device int64 [num_ids].  host_k, host_v: [num_ids][num_kv_heads]
 * [block_size][head_dim] in the cache dtype, in pinned (cudaHostAlloc /
 * cudaHostRegister) host memory, or device memory; pageable memory is refused with
 * PKV_ERR_INVALID_ARG.  swap_out copies pool block block_ids[i] to entry i; swap_in
 * copies entry i into pool block block_ids[i].  Bit-exact.  Out-of-range ids set the
 * device index flag and are skipped.  Stream-ordered like every other call: issue the
 * swap-out before anything reuses the blocks.
 */
pkv_status paged_block_swap_out(const int64_t* block_ids, int32_t num_ids, const void* k_cache,
                                const void* v_cache, void* host_k, void* host_v,
                                const pkv_cache_desc* cache, void* stream);
pkv_status paged_block_swap_in(const int64_t* block_ids, int32_t num_ids, const void* host_k,
                               const void* host_v, void* k_cache, void* v_cache,
                               const pkv_cache_desc* cache, void* stream);

/*
 * Bytes of workspace paged_attention_decode needs for these sizes and config.  The
 * CUDA-core path needs none when every sequence fits one partition; the tensor-core
 * path always needs room for its work list (16 bytes per (sequence, KV head,
 * partition) plus a 256-byte header holding the entry count and the counter from
 * which the CTAs claim entries) and, past one partition, the partition partials.
 * Two calls in flight at once (on different streams) need separate workspaces.
 * max_context_len: host upper bound on context_lens.  Returns 0 for invalid
 * arguments as well (then the decode call itself reports the error).
 */
size_t paged_attention_workspace_bytes(int32_t num_seqs, int32_t num_q_heads,
                                       int32_t max_context_len, const pkv_cache_desc* cache,
                                       const pkv_decode_config* config);

/*
 * paged_attention_decode -- single-token decode attention through block tables.
 * Pages: note-023, Method and Concepts (attention gathers K/V through the block
 * table from non-contiguous blocks); "Paged Attention" glossary, paragraph 4
 * (arithmetic unchanged) and GQA paragraph.
 *
 * For every sequence s and query head h, with n = context_lens[s], kv = h / G,
 * K_j / V_j = row j % block_size of physical block block_tables[s][j / block_size]:
 *   out[s][h][:] = sum_j softmax_j(scale * q[s][h] . K_j) V_j,   j < n;
 *   n == 0 gives zeros.  Accumulation in fp32; out rounded to out_dtype (RNE).
 * Sequences longer than the partition size are split into partitions whose
 * (max, sum, unnormalised output) go to the workspace and are merged by a second
 * kernel.  max_context_len: host upper bound on context_lens (a longer sequence
 * sets the device index flag).  workspace: device, at least
 * paged_attention_workspace_bytes(...) bytes, 256-byte aligned; NULL allowed when
 * that is 0.  out must not alias any input.
 */
pkv_status paged_attention_decode(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, int32_t max_blocks_per_seq,
                                  const int32_t* context_lens, int32_t num_seqs,
                                  int32_t num_q_heads, int32_t max_context_len, float scale,
                                  void* out, int32_t out_dtype, void* workspace,
                                  size_t workspace_bytes, const pkv_cache_desc* cache,
                                  const pkv_decode_config* config, void* stream);

/*
 * paged_attention_decode_no_alloc -- paged_attention_decode for callers that must not
 * allocate device memory (allocator or memory-pool callbacks, serving paths that may
 * not fail with out-of-memory once running, runtimes that only pass pre-registered
 * buffers).  The pages have no counterpart: this is a packaging of the same decode.
 *
 * Same arguments and result as paged_attention_decode, minus the workspace: the
 * scratch comes from a fixed array of paged_attention_no_alloc_limit() bytes
 * (32 MiB) that every GPU loading the library holds until the process exits.  The
 * call allocates nothing.  Sizes whose workspace would exceed the array return
 * PKV_ERR_WORKSPACE (pass a larger partition_tokens, or use paged_attention_decode).
 * The first call on a device looks up the array's device address (with that device
 * current) and caches it; make that first call before any stream capture.  All calls
 * share the one array: calls that overlap on the GPU (other streams, other threads)
 * race on it and must be serialised by the caller.  Nothing in the array needs to
 * start at zero; each call writes what it reads.
 */
pkv_status paged_attention_decode_no_alloc(const void* q, const void* k_cache, const void* v_cache,
                                           const int32_t* block_tables, int32_t max_blocks_per_seq,
                                           const int32_t* context_lens, int32_t num_seqs,
                                           int32_t num_q_heads, int32_t max_context_len, float scale,
                                           void* out, int32_t out_dtype, const pkv_cache_desc* cache,
                                           const pkv_decode_config* config, void* stream);

/* Bytes of the built-in array paged_attention_decode_no_alloc uses. */
size_t paged_attention_no_alloc_limit(void);

/*
 * paged_attention_prefill -- several new tokens per sequence (prefill, chunked prefill)
 * attending through block tables with a causal mask.
 * Pages: note-023, Method (attention gathers K/V through the block table) and Open
 * questions (chunked prefill); attention arithmetic unchanged ("Paged Attention"
 * glossary, paragraph 4).
 *
 * Sequence s brings n_s = query_start[s+1] - query_start[s] new tokens: rows
 * query_start[s] .. query_start[s+1]-1 of q and out ([num_query_tokens][Hq][D]),
 * the last n_s of its context_lens[s] tokens, whose K/V are already in the pool
 * (paged_kv_append first).  New token i at position p = context_lens[s] - n_s + i:
 *   out[row][h] = sum_{j <= p} softmax_j(scale * q[row][h] . K_j) V_j.
 * query_start: device int32 [num_seqs + 1], non-decreasing, query_start[0] = 0 and
 * query_start[num_seqs] = num_query_tokens.  A sequence with n_s > context_lens[s]
 * or context_lens[s] > max_context_len sets the device index flag and is skipped.
 * Tensor cores only: f16/bf16, head_dim 64 or 128, query-head groups <= 16, block size 8,
 * 16, 32 or 64, at most 4095 KV heads (else PKV_ERR_UNSUPPORTED); q, out and the pools
 * 16-byte aligned.  workspace: at least paged_attention_prefill_workspace_bytes(...)
 * bytes, 256-byte aligned.
 */
size_t paged_attention_prefill_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_query_tokens,
                                               const pkv_cache_desc* cache);
pkv_status paged_attention_prefill(const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int32_t max_blocks_per_seq,
                                   const int32_t* context_lens, const int32_t* query_start, int32_t num_seqs,
                                   int32_t num_q_heads, int32_t num_query_tokens, int32_t max_context_len,
                                   float scale, void* out, int32_t out_dtype, void* workspace,
                                   size_t workspace_bytes, const pkv_cache_desc* cache, void* stream);

/*
 * paged_kv_gather -- the block-table lookup alone (testing the indexing bit-exactly):
 * k_out[s][h][j][:] = k_cache[block_tables[s][j / bs]][h][j % bs][:] for j < n_s,
 * same for v.  Rows j >= context_lens[s] are not written.
 * k_out, v_out: device [num_seqs][num_kv_heads][max_context_len][head_dim].
 */
pkv_status paged_kv_gather(const void* k_cache, const void* v_cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t num_seqs, int32_t max_context_len, void* k_out, void* v_out,
                           const pkv_cache_desc* cache, void* stream);

/* ----------------------------------------------------------------------------------
 * Position rotation and norms of new tokens' queries and keys.  The pages have no
 * counterpart: what a model with rotary positions does to q and k between its projection
 * and the cache.
 * ---------------------------------------------------------------------------------- */

/* Which dimensions of a head turn together, i < rotary_dim / 2. */
typedef enum {
  PKV_ROTARY_HALF = 0,        /* i and i + rotary_dim / 2 */
  PKV_ROTARY_INTERLEAVED = 1  /* 2i and 2i + 1 */
} pkv_rotary_layout;

typedef struct {
  const double* inv_freq;  /* device [rotary_dim / 2]: radians per position */
  int32_t rotary_dim;      /* the first rotary_dim dimensions of a head turn: a multiple of 16, 0 to head_dim */
  int32_t layout;          /* pkv_rotary_layout */
  float factor;            /* of cosines and sines (1 unless a scaling rule gives another) */
  float eps;               /* of the norms; read where a weight is given */
  const void* q_weight;    /* device [head_dim] in the tensors' dtype, 16-byte aligned: norm of each query head */
  const void* k_weight;    /* the same for keys; NULL: no norm */
} pkv_rotary;

/* Frequencies of rotations scaled for longer contexts than a model was trained on. */
typedef enum {
  PKV_ROTARY_UNSCALED = 0,
  PKV_ROTARY_LINEAR = 1,  /* positions interpolated: every frequency divided by `factor` */
  PKV_ROTARY_BASE = 2,    /* base * factor^(rotary_dim / (rotary_dim - 2)): the lowest frequency divided by `factor` */
  PKV_ROTARY_PARTS = 3    /* by turns within original_len: fast_turns or more are kept, slow_turns or fewer divided by
                             `factor`, linear in the turns in between; cosines and sines times 0.1 ln(factor) + 1 */
} pkv_rotary_rule;

/*
 * A checkpoint wants the rule that it was trained with, and rules by parts are not all alike:
 *  - many blend linearly in the dimension's index i, between the (rounded) indices at which
 *    fast_turns and slow_turns are reached, where PKV_ROTARY_PARTS blends linearly in the turns.  In
 *    between the two differ by up to a factor of 3 (rotary_dim 128, base 10,000, factor 16, 4,096
 *    original tokens, turns 32 and 1).  No rule here gives those frequencies.
 *  - some blend as PKV_ROTARY_PARTS does (customarily with turns 4 and 1) but leave cosines and sines
 *    alone: take the frequencies, and 1 for pkv_rotary.factor.
 * pkv_rotary.inv_freq and factor take any values: where none of the rules is the checkpoint's,
 * compute them by its own.
 */

typedef struct {
  int32_t rule;                   /* pkv_rotary_rule */
  double factor;                  /* >= 1 */
  double original_len;            /* PKV_ROTARY_PARTS only, as are the next two */
  double fast_turns, slow_turns;  /* customarily 32 and 1 */
} pkv_rotary_scaling;

/*
 * paged_rotary_frequencies -- host only: inv_freq[i] = base^(-2 i / rotary_dim), i <
 * rotary_dim / 2, scaled by the rule (NULL: unscaled); *factor is what pkv_rotary.factor
 * then wants.  inv_freq and factor are host memory.
 */
pkv_status paged_rotary_frequencies(double* inv_freq, int32_t rotary_dim, double base,
                                    const pkv_rotary_scaling* scaling, float* factor);

/*
 * paged_qk_rotary -- norm and rotate queries and keys by their positions.  For every token
 * t with positions[t] >= 0 and every head of q and k, with x its head_dim values:
 *   y = x * weight / sqrt(mean(x^2) + eps)  (y = x where the weight is NULL);
 *   each pair (y_a, y_b) of the layout becomes (y_a c - y_b s, y_b c + y_a s), with
 *   c = factor cos(positions[t] * inv_freq[i]), s = factor sin(positions[t] * inv_freq[i]);
 * the other dimensions stay y.  fp32 throughout, one rounding at the end (RNE).  The angle is
 * taken modulo whole turns in integers, good to 2^-31 turns at any position for frequencies up to
 * 1; what is left of it past the nearest quarter turn is then rounded to fp32, by 2^-28 turns at
 * most.
 * Negative positions are padding: nothing of the token is written.
 *
 * q, k, q_out, k_out: device, dtype f32, f16 or bf16; a token's heads lie one after the
 * other ([num_heads][head_dim]), tokens are *_stride elements apart (at least the token's
 * own, a multiple of 16 bytes): parts of a fused projection's rows are taken as they are.
 * q_out may be q and k_out may be k (same strides); other overlaps are refused.
 * num_q_heads or num_kv_heads 0: that tensor is not looked at.
 * For 4-bit pools: rotate k with this call, then paged_kv4_append.
 */
pkv_status paged_qk_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
                           int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                           const pkv_rotary* rotary, void* q_out, int64_t q_out_stride, void* k_out,
                           int64_t k_out_stride, void* stream);

/*
 * paged_kv_append_rotary -- paged_qk_rotary and paged_kv_append in one pass: q goes, normed
 * and rotated, to q_out, k normed and rotated into its slot of k_cache, v as it is into its
 * slot of v_cache (bit-exact).  Arguments as in those calls; q, k, v and q_out have the
 * cache's dtype (f32, f16 or bf16) and heads of its head_dim, k and v its KV heads.
 * Tokens with a negative slot or a negative position are padding: nothing of them is
 * written, to q_out neither, and their slot or position does not matter.  Any other token's slot
 * >= num_blocks * block_size sets the device index flag and the token is skipped as well.
 * Slots must be distinct (duplicates race).
 */
pkv_status paged_kv_append_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                                  int32_t num_tokens, int32_t num_q_heads, const pkv_rotary* rotary, void* q_out,
                                  int64_t q_out_stride, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                                  void* stream);

/* ----------------------------------------------------------------------------------
 * Sliding windows.  The pages have no counterpart: layers whose tokens attend to the last
 * `window` tokens, their own among them, and to the first `sinks` of the sequence.
 *
 * A token at position p attends to the positions j <= p with j > p - window or j < sinks;
 * window >= 1, sinks >= 0.  A window or sinks past the sequence's start or end change nothing
 * else: window >= context_lens[s] is attention over all tokens.  Table entries of blocks
 * that hold no token attended to are never read, so a server can release those blocks; what
 * lies in rows that no token of a call attends to (a NaN, too) does not matter.
 * ---------------------------------------------------------------------------------- */

/*
 * paged_attention_decode_window -- paged_attention_decode over a window.  One new token per
 * sequence, at position context_lens[s] - 1; the other arguments, types and errors as there,
 * groups up to 16 for every dtype, one kernel, no workspace.  16-bit caches run on tensor
 * cores, their weights in two 16-bit parts; f32 caches on CUDA cores, fp32 throughout.
 * max_context_len: host upper bound on context_lens, at most 2^30 (a longer sequence sets the
 * device index flag, and its rows of out are left as they are).  Cost goes by the tokens
 * attended to, not by context_lens.
 */
pkv_status paged_attention_decode_window(const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t max_context_len, int32_t window, int32_t sinks, float scale, void* out,
                                         int32_t out_dtype, const pkv_cache_desc* cache, void* stream);

/*
 * paged_attention_prefill_window -- paged_attention_prefill over windows, each new token's
 * its own (arguments, types, limits and errors as there; no workspace).  A NaN or an infinity
 * in a V row that one of a call's new tokens attends to may reach the outputs of the
 * sequence's other new tokens (they share its products); in a K row it reaches those that
 * attend to it.
 */
pkv_status paged_attention_prefill_window(const void* q, const void* k_cache, const void* v_cache,
                                          const int32_t* block_tables, int32_t max_blocks_per_seq,
                                          const int32_t* context_lens, const int32_t* query_start, int32_t num_seqs,
                                          int32_t num_q_heads, int32_t num_query_tokens, int32_t max_context_len,
                                          int32_t window, int32_t sinks, float scale, void* out, int32_t out_dtype,
                                          const pkv_cache_desc* cache, void* stream);

/* Kernels of a windowed prefill. */
typedef enum {
  PKV_WINDOW_ROWS = 0,         /* up to 16 query rows of a KV head, as in windowed decode: a few new tokens */
  PKV_WINDOW_SHARED_TILES = 1, /* tiles of up to 128 query rows, two halves of their tokens at once */
  PKV_WINDOW_TILE_PAIRS = 2    /* two such tiles over the same tokens: long chunks */
} pkv_window_kernel;

/* What paged_attention_prefill_window will do for these sizes. */
typedef struct {
  int32_t kernel;          /* pkv_window_kernel */
  int32_t tokens_per_item; /* new tokens of a sequence that one item covers at most, for one KV head */
  int32_t ctas_per_item;   /* CTAs that share an item's tokens (0: there is nothing to do) */
} pkv_window_plan;

/*
 * paged_attention_prefill_window_plan -- fill *out with the plan that
 * paged_attention_prefill_window follows for these sizes (host only, no device work): the kernel
 * with the shortest estimate for sequences that share the new tokens out evenly.  Errors as the
 * call's checks of its sizes.
 */
pkv_status paged_attention_prefill_window_plan(int32_t num_seqs, int32_t num_q_heads, int32_t num_query_tokens,
                                               int32_t max_context_len, int32_t window, int32_t sinks,
                                               const pkv_cache_desc* cache, pkv_window_plan* out);

/* ----------------------------------------------------------------------------------
 * 4-bit caches.  The pages have no counterpart: a smaller form of the same cache, for more
 * context in the same memory.
 *
 * A pool with dtype PKV_KV4 is [num_blocks][num_kv_heads][block_size][head_dim * 5 / 8]
 * bytes (5 bits per value; 3.2 times the tokens of a 16-bit pool).  A row holds its D
 * values as D / 2 bytes of codes -- byte i: value 2i in the low half, 2i + 1 in the high
 * half -- and then D / 32 pairs (step, lo) of fp16, one for each group of 32 values.
 * Code c of a group stands for fp16(lo + c * step), rounded once (to nearest even).
 * paged_block_copy and paged_block_swap_out / _in take these pools like any other (a swap
 * buffer's rows are then head_dim * 5 / 8 bytes).
 * ---------------------------------------------------------------------------------- */

/*
 * paged_kv4_append -- round new tokens' K and V to 4 bits and write them into their slots
 * of a 4-bit pool (paged_kv_append for PKV_KV4 pools; same slots, same padding).
 *
 * k, v: device [num_tokens][num_kv_heads][head_dim] of kv_dtype (f32, f16 or bf16).  For
 * each group x[0..31], all operations rounded to nearest even:
 *   lo = fp16(min x), step = fp16(fp32(fp32(max x - lo) / 15)) (0 if negative),
 *   code = fp32(x - lo) / step to the nearest integer (the quotient exact), held within
 *   0..15; step 0 gives code 0.
 * Values beyond +-65408 are stored as +-65408.  A group with a NaN or an infinity gets
 * step = lo = NaN: all its 32 values read as NaN.
 * Slots must be distinct (duplicates race); negative slots are skipped; a slot
 * >= num_blocks * block_size sets the device index flag and is skipped.
 */
pkv_status paged_kv4_append(const void* k, const void* v, int32_t kv_dtype, const int64_t* slot_mapping,
                            int32_t num_tokens, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                            void* stream);

/*
 * paged_kv4_expand -- widen 4-bit blocks: block dst of the out pools becomes the values of
 * block src of the 4-bit pools (all KV heads and rows), for each pair.  What
 * paged_attention_prefill reads when earlier chunks are held in 4 bits.
 *
 * src_dst_pairs: device int64 [num_pairs][2]; destinations distinct (duplicates race).
 * out_cache: the out pools' geometry; block_size, num_kv_heads and head_dim as cache's,
 * dtype f32, f16 or bf16 (f32 and f16 hold the values exactly, bf16 rounds them to nearest
 * even).  Out-of-range ids set the device index flag and are skipped.
 */
pkv_status paged_kv4_expand(const int64_t* src_dst_pairs, int32_t num_pairs, const void* k_cache,
                            const void* v_cache, const pkv_cache_desc* cache, void* k_out, void* v_out,
                            const pkv_cache_desc* out_cache, void* stream);

/*
 * paged_attention_decode_kv4 -- single-token decode attention over a 4-bit pool:
 * paged_attention_decode with K_j and V_j the values that the rows stand for.
 *
 * q: device [num_seqs][num_q_heads][head_dim] of q_dtype (f32, f16 or bf16); out: q's
 * dtype or f32; query-head groups up to 16.  Softmax, sums and products in fp32: q in fp16
 * (f32 q in two fp16 parts) after a power-of-two scaling of each head's row, weights in
 * two fp16 parts: each within 2^-22 of itself, or 2^-36 of the largest met where that is more
 * (a weight below 2^-36 of it counts in the softmax's sum, not in the output).  Sums of n
 * values add up to n / 16 roundings of 2^-23, f32 outputs' to nearest, f16 and bf16 outputs'
 * towards zero (over 128 Ki tokens 2.7e-6 of the result), before the output's own rounding.
 * n == 0 gives zeros.  A NaN or infinity in a query row, or a NaN in a row attended to,
 * gives NaN as the formula does.  A sequence longer than max_context_len sets the device
 * index flag and is skipped.  The batch's tokens are shared out evenly among the CTAs,
 * whatever the lengths; sequences that cross a CTA's share are joined by a second kernel.
 * workspace: at least paged_attention_decode_kv4_workspace_bytes(...) bytes (0 when
 * max_context_len <= 128, and for small batches up to 512), 256-byte aligned, one per call in
 * flight; its size does not grow with the batch or the lengths past a limit of some 20 MB.  The result does not depend on
 * which physical blocks hold a sequence; where a sequence is cut depends on the lengths of
 * the whole batch, which can change its last bits.  out must not alias any input.
 */
size_t paged_attention_decode_kv4_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t max_context_len,
                                                  int32_t q_dtype, const pkv_cache_desc* cache);
pkv_status paged_attention_decode_kv4(const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                      int32_t max_context_len, float scale, void* out, int32_t out_dtype,
                                      void* workspace, size_t workspace_bytes, const pkv_cache_desc* cache,
                                      void* stream);

/* ----------------------------------------------------------------------------------
 * Eviction by accumulated attention weight.  The pages have no counterpart (they evict
 * whole blocks of preempted sequences); this shortens a sequence in place of preempting it:
 * the tokens that attention has used least leave, per KV head.
 * ---------------------------------------------------------------------------------- */

/*
 * paged_attention_weights -- add a decode step's attention weights to per-token
 * accumulators.  For every sequence s, KV head g and token j < n = context_lens[s]:
 *   weights_out[s][g][j] = (j < tracked_lens[s] ? weights[s][g][j] : 0)
 *                          + sum over g's query heads h of softmax_j(scale * q[s][h] . K_j).
 * Rows j >= n are not written.  tracked_lens (device int32 [num_seqs], or NULL = every
 * row): how many of a sequence's rows have an accumulator yet; the newer ones start at 0.
 * weights, weights_out: device f32 [num_seqs][num_kv_heads][weights_width],
 * weights_width >= max_context_len; they may be the same buffer, but not overlap otherwise.
 * q: device [num_seqs][num_q_heads][head_dim] of q_dtype, which is the cache's dtype; a
 * PKV_KV4 pool takes f32, f16 or bf16.  Query-head groups up to 16.  fp32 throughout
 * (products of 16-bit operands are exact).  A sequence longer than max_context_len sets
 * the device index flag and is skipped (max_context_len 0: nothing is looked at).  workspace: at least
 * paged_attention_weights_workspace_bytes(...) bytes (0 when max_context_len <= 512; else a
 * float per sequence, query head and token of max_context_len and a little more, of the whole
 * batch up to 4 GiB, in turns of fewer sequences beyond), 256-byte aligned, one per call
 * in flight.
 */
size_t paged_attention_weights_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t max_context_len,
                                               const pkv_cache_desc* cache);
pkv_status paged_attention_weights(const void* q, int32_t q_dtype, const void* k_cache, const int32_t* block_tables,
                                   int32_t max_blocks_per_seq, const int32_t* context_lens,
                                   const int32_t* tracked_lens, int32_t num_seqs, int32_t num_q_heads,
                                   int32_t max_context_len, float scale, const float* weights, float* weights_out,
                                   int64_t weights_width, void* workspace, size_t workspace_bytes,
                                   const pkv_cache_desc* cache, void* stream);

/*
 * paged_kv_evict -- shorten sequences to the rows that matter.  For every sequence s and
 * KV head g, of n = context_lens[s] rows k = min(keep_lens[s], n) are kept: the last
 * r = min(recent, k), and of rows 0 .. n - r - 1 the k - r with the largest
 * weights[s][g][j] (NaN counts as -infinity; equal weights: the lowest j first).  Kept rows
 * keep their order: row i of the shortened sequence is row j = kept[s][g][i],
 *   K/V row i of new_tables[s] = K/V row j of block_tables[s]  (bit-exact),
 *   weights_out[s][g][i] = weights[s][g][j],   i < k;
 * rows past k of kept, weights_out and the new blocks are not written, and the old blocks
 * are left as they are (so shared blocks may be evicted from).  Attend to the result with
 * new_tables and lengths k.  Heads choose on their own: K rows must carry their position
 * (rotary embeddings applied before the append), since row numbers change.
 *
 * Pools of any dtype, PKV_KV4 too.  weights, weights_out: device f32
 * [num_seqs][num_kv_heads][weights_width], not overlapping; kept: device int32
 * [num_seqs][num_kv_heads][max_keep]; keep_lens: device int32 [num_seqs], k <= max_keep;
 * new_tables: device int32 [num_seqs][max_new_blocks] of blocks that no listed sequence
 * reads or shares (pkv_bm_compact gives them).  A sequence whose lengths break these bounds
 * sets the device index flag and is skipped, as are rows with a block id out of range
 * (max_context_len 0: nothing is looked at).
 */
pkv_status paged_kv_evict(const float* weights, float* weights_out, int64_t weights_width, const int32_t* block_tables,
                          int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* keep_lens,
                          int32_t recent, const int32_t* new_tables, int32_t max_new_blocks, int32_t num_seqs,
                          int32_t max_context_len, int32_t max_keep, int32_t* kept, void* k_cache, void* v_cache,
                          const pkv_cache_desc* cache, void* stream);

/* ----------------------------------------------------------------------------------
 * Host block manager: which physical block every token lives in.
 * Pages: note-023, Method (allocate on demand as a sequence grows, free when it
 * finishes, share blocks between sequences with identical prefixes, copy on write when
 * one diverges) and Concepts (internal fragmentation = unused tail of the last block);
 * "Paged Attention" glossary, paragraphs 1-3; "PagedAttention & Continuous Batching",
 * shared-system-prompt paragraph (blocks of a finished request go to the next one).
 *
 * Host memory only; not thread-safe (one manager per host thread, or a caller lock).
 * Policy: free blocks form a LIFO stack (first hands out 0, 1, 2, ...; freed blocks are
 * reused first).  Every call either succeeds as a whole or changes nothing.
 * ---------------------------------------------------------------------------------- */
typedef struct pkv_block_manager pkv_block_manager;

typedef struct {
  int32_t num_blocks, free_blocks, used_blocks, num_sequences;
  int32_t shared_blocks;   /* blocks referenced by more than one sequence */
  int64_t stored_tokens;   /* valid rows held in used blocks (shared rows counted once) */
  int64_t logical_tokens;  /* sum of sequence lengths (shared rows counted per sharer) */
  int64_t allocated_slots; /* used_blocks * block_size */
  int64_t max_len;         /* longest sequence */
  int64_t copies;          /* copy-on-write copies made so far */
  int64_t swapped;         /* sequences swapped out (holding no blocks) */
} pkv_block_stats;

/* A manager for a pool of num_blocks blocks of block_size tokens.  Free with destroy. */
pkv_status pkv_bm_create(int32_t num_blocks, int32_t block_size, pkv_block_manager** out);
void pkv_bm_destroy(pkv_block_manager* manager);

/* A new sequence with a prompt of num_tokens tokens: ceil(num_tokens / block_size)
 * fresh blocks.  PKV_ERR_OUT_OF_BLOCKS if the pool cannot hold them. */
pkv_status pkv_bm_add_sequence(pkv_block_manager* manager, int64_t seq_id, int64_t num_tokens);

/* child shares every block of parent by reference (parallel sampling, beam search). */
pkv_status pkv_bm_fork(pkv_block_manager* manager, int64_t parent, int64_t child);

/*
 * Reserve the slot of one new token for each of n distinct sequences, in order.  A
 * sequence at a block boundary takes a fresh block; one whose last block is shared
 * gets a fresh copy of it first (copy-on-write) and the pair (old, fresh) is appended
 * to cow_pairs ([n][2] capacity, *num_cow set).  slots[i] = block * block_size + row,
 * ready for paged_kv_append; apply the pairs with paged_block_copy before the append.
 */
pkv_status pkv_bm_append(pkv_block_manager* manager, const int64_t* seq_ids, int32_t n, int64_t* slots,
                         int64_t* cow_pairs, int32_t* num_cow);

/* The sequence finished: drop its references; blocks no longer referenced are freed. */
pkv_status pkv_bm_free_sequence(pkv_block_manager* manager, int64_t seq_id);

/*
 * Preemption: *num_out = the sequence's blocks in logical order, copied to blocks_out
 * (capacity entries), and the sequence drops its references (blocks nobody else
 * holds become free).  The sequence stays known, with its length, as swapped out:
 * copy those blocks out with paged_block_swap_out before anything reuses them.
 */
pkv_status pkv_bm_swap_out(pkv_block_manager* manager, int64_t seq_id, int32_t* blocks_out, int32_t capacity,
                           int32_t* num_out);

/* Restore a swapped-out sequence into fresh private blocks, listed in logical order;
 * copy its data back into them with paged_block_swap_in.  PKV_ERR_OUT_OF_BLOCKS if
 * the pool cannot hold it (nothing changes). */
pkv_status pkv_bm_swap_in(pkv_block_manager* manager, int64_t seq_id, int32_t* blocks_out, int32_t capacity,
                          int32_t* num_out);

/*
 * Eviction: each of n distinct sequences gets ceil(new_lens[i] / block_size) fresh private
 * blocks, in order of sequence and position in blocks_out (capacity entries, *num_out set),
 * and drops its references to the old ones (blocks nobody else holds become free).  No fresh
 * block is an old one of any of the n: sequences that one paged_kv_evict shortens are
 * compacted in one call (one by one, a sequence's fresh blocks may be those that the one
 * before has just left, which the eviction still reads).  Take the old tables first;
 * paged_kv_evict then moves the kept rows from there.  new_lens[i] at most the sequence's
 * length.  The old blocks may be handed out again at once: issue the eviction before
 * anything that writes to them on the same stream.  PKV_ERR_OUT_OF_BLOCKS if the pool
 * cannot hold the fresh blocks beside the old ones (nothing changes).
 */
pkv_status pkv_bm_compact(pkv_block_manager* manager, const int64_t* seq_ids, const int64_t* new_lens, int32_t n,
                          int32_t* blocks_out, int32_t capacity, int32_t* num_out);

/* Rows of block_tables ([n][max_blocks], -1 padded) and context_lens for n sequences. */
pkv_status pkv_bm_block_tables(const pkv_block_manager* manager, const int64_t* seq_ids, int32_t n,
                               int32_t max_blocks, int32_t* tables, int32_t* lens);

pkv_status pkv_bm_stats(const pkv_block_manager* manager, pkv_block_stats* out);

/* Message of the last failed call on this host thread ("" if none). */
const char* paged_kv_last_error(void);

/*
 * Synchronise `stream`, then read and clear the device error flag of the current
 * device: PKV_OK, PKV_ERR_DEVICE_INDEX or PKV_ERR_DEVICE_TIMEOUT (PKV_ERR_CUDA if
 * the synchronisation itself fails).
 */
pkv_status paged_kv_device_error(void* stream);

/*
 * Diagnostic (no counterpart on the pages): enqueue one kernel whose bounded wait can
 * never complete -- an mbarrier expecting an arrival nobody makes -- so that the wait
 * gives up after limit_ns (at most 5 s), records PKV_ERR_DEVICE_TIMEOUT in the device
 * flag and returns.  Shows that a stuck wait ends with a status the host reads and
 * leaves the context usable; every wait in the library's kernels ends the same way
 * (their limit is 2 s).
 */
pkv_status paged_kv_selftest_wait_timeout(uint64_t limit_ns, void* stream);

/*
 * Diagnostic (no counterpart on the pages): set the bound of the pipeline waits in
 * the decode and prefill kernels launched from now on, process-wide (0 restores the
 * default of 2 s; at most 5 s, else PKV_ERR_INVALID_ARG).  A bound far below a
 * healthy wait (say 1 us) makes a normal call give up part-way: its kernels then take
 * their abort path -- they wait (each up to 2 s) for the copies and MMAs they have in
 * flight, free their tensor memory, record PKV_ERR_DEVICE_TIMEOUT in the device flag
 * and return -- so that path can be exercised without any real fault.  The output of
 * such a call is undefined.  Not for production use.
 */
pkv_status paged_kv_set_wait_limit(uint64_t limit_ns);

/* Library version, e.g. "0.1.0". */
const char* paged_kv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H */
