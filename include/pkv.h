/*
 * pkv.h -- C ABI of libpkv: paged-KV decode attention for one GB300 (sm_103a).
 *
 * What the library computes
 * -------------------------
 * A paged KV cache keeps every sequence's keys and values in a pool of
 * fixed-size physical blocks; a per-sequence block table maps logical block i
 * (tokens [16i, 16i+16)) to a physical block, and the attention kernel gathers
 * K/V from those non-contiguous blocks itself, with no compaction copy
 * (Continuous-Batching-LLM-Inference-Engine README, feature list "Paged
 * KV-cache" and "PagedAttention kernel"). The model's forward writes new K/V
 * into the cache through slot mappings and reads them back in the paged decode
 * attention kernel (mini-inference-engine, Connections "Llama forward -> Paged
 * KV cache: writes and reads"; low-latency-distributed-llm-serving-
 * infrastructure, Connections "Paged attention -> KV cache manager: maps cache
 * slots"). The cache may be stored as INT8 (paged-inference-engine overview,
 * "paged INT8 KV storage").
 *
 * Layouts (all row-major, contiguous):
 *   k_cache, v_cache  [num_blocks, num_kv_heads, block_size, head_dim]
 *                     one (block, kv_head) tile is one contiguous run of
 *                     block_size*head_dim elements
 *   k_scales, v_scales [num_blocks, num_kv_heads] fp32 (INT8 caches only)
 *   block_tables      int32 [batch, max_blocks_per_seq]; entries past a
 *                     sequence's ceil(len/16) blocks are not read
 *   context_lens      int32 [batch], including the token appended this step
 *   q, out            [batch, num_q_heads, head_dim], q's dtype
 *   k_new, v_new      [num_tokens, num_kv_heads, head_dim]
 *   slot_mapping      int64 [num_tokens], slot = block*block_size + row,
 *                     negative = skip
 * Query head h reads KV head h / (num_q_heads / num_kv_heads).
 *
 * Ownership and synchronisation: every pointer argument is caller-owned
 * DEVICE memory, except the pkv_cache_desc pointer and pair_axis (host). The library
 * allocates nothing. Between calls it keeps only lookups, each made once:
 * two driver entry points (the tensor-map encoder of the multi-query calls and
 * the current-context query of pkv_decode_attn_noalloc), per CUDA context the
 * address of pkv_decode_attn_noalloc's built-in scratch array, and per device
 * the default worker counts of pkv_sparse_decode_attn, pkv_decode_attn_mass and
 * pkv_window_decode_attn and whether their kernels' shared memory, and that of
 * pkv_block_select and pkv_evict_tokens, was granted. Host threads may call at
 * once, on streams of their own and with workspaces of their own.
 * Every call only
 * enqueues kernels on `stream` and returns; inputs must stay valid until the
 * stream has executed them.
 *
 * Errors: arguments are checked on the host before anything is launched; a
 * bad argument returns PKV_ERR_* and launches nothing. Conditions only the GPU
 * can see (a block-table entry or slot outside the pool, a context length
 * outside the table, a bounded in-kernel wait that ran out) are OR-ed as
 * PKV_DEV_* bits into *dev_status when dev_status is non-NULL; the kernel
 * then skips the offending work instead of touching memory outside the
 * buffers. The library never clears *dev_status.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as the CUDA runtime's cudaStream_t; NULL = legacy default stream. */
typedef struct CUstream_st *cudaStream_t;

typedef enum {
    PKV_OK = 0,
    PKV_ERR_INVALID_ARG = 1,   /* NULL / misaligned pointer, bad size or shape */
    PKV_ERR_UNSUPPORTED = 2,   /* valid but not built: head_dim, group, dtype  */
    PKV_ERR_WORKSPACE = 3,     /* workspace NULL or smaller than required      */
    PKV_ERR_CUDA = 4           /* a CUDA runtime call or launch failed         */
} pkv_status;

/* Bits OR-ed into *dev_status by the kernels. */
#define PKV_DEV_BAD_BLOCK  1u  /* block-table entry outside [0, num_blocks)    */
#define PKV_DEV_BAD_LENGTH 2u  /* context_len < 0 or > max_blocks_per_seq*16   */
#define PKV_DEV_BAD_SLOT   4u  /* slot >= num_blocks*block_size                */
#define PKV_DEV_TIMEOUT    8u  /* a bounded wait on an in-kernel copy ran out  */
#define PKV_DEV_BAD_INDEX 16u  /* pkv_merge_states: a row's range of states
                                  lies outside [0, num_states]; a listed block
                                  or a position outside its range           */

typedef enum { PKV_F16 = 0, PKV_BF16 = 1, PKV_I8 = 2, PKV_U4 = 3 } pkv_dtype;

/* The physical KV block pool. block_size must be 16, head_dim 64 or 128. */
typedef struct {
    int32_t num_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t head_dim;
    pkv_dtype kv_dtype;       /* PKV_F16, PKV_BF16 or PKV_I8; PKV_U4 where a
                                 call says so ("A cache in 4 bits") */
} pkv_cache_desc;

/* Human-readable name of a status code (static string, never NULL). */
const char *pkv_status_string(pkv_status s);

/* ------------------------------------------------------------------------
 * KV append (cache write)
 *
 * Writes k_new[n], v_new[n] to slot slot_mapping[n] of k_cache / v_cache for
 * every n with slot >= 0 (the cache write that the forward pass performs each
 * step; see the file comment). Duplicate non-negative slots in one call are a
 * caller error.
 *
 * fp16 / bf16 caches: src_dtype must equal kv_dtype; the rows are stored bit
 * for bit. k_scales, v_scales, workspace may be NULL.
 *
 * INT8 caches (PKV_I8): src_dtype is PKV_F16 or PKV_BF16. Codes are symmetric
 * in [-127, 127] with one fp32 scale per (block, kv_head), K and V separately,
 * scale = absmax/127 and round-to-nearest-even. Per (block, kv_head) tile
 * touched by the call: a = max|x| over the call's new values in the tile,
 * s_c = a/127 (fp32, IEEE division); with s_o the stored scale (0 = never
 * written): s = s_c if s_o == 0; s = s_o if s_c <= s_o; otherwise s = s_c and
 * every stored code q of the tile becomes rne((float)q * s_o / s) (fp32, left
 * to right). New codes are clamp(rne(x / s), -127, 127), or 0 when s == 0.
 * k_scales / v_scales must start at 0 for never-written blocks. The call needs
 * a workspace of pkv_append_workspace_size(cache) bytes (80 bytes per
 * (block, kv_head) tile; 16-byte aligned), zero-filled before its first use:
 * each call leaves it zero-filled again, so one workspace serves every later
 * call on the same cache (calls that overlap on the GPU must not share it).
 * Inputs must be finite.
 *
 * Alignment: k_new, v_new, k_cache, v_cache 16-byte aligned.
 * ------------------------------------------------------------------------ */
size_t pkv_append_workspace_size(const pkv_cache_desc *cache);

pkv_status pkv_append(const void *k_new, const void *v_new, pkv_dtype src_dtype,
                      int32_t num_tokens, const int64_t *slot_mapping,
                      void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                      const pkv_cache_desc *cache, void *workspace, size_t workspace_bytes,
                      uint32_t *dev_status, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Decode attention (one query token per sequence)
 *
 * out[b, h] = sum_p softmax_p(softmax_scale * <q[b,h], k_p>) * v_p over the
 * context_lens[b] tokens of sequence b, token p read from physical block
 * block_tables[b, p/16], row p%16 (the paged decode attention kernel of the
 * pages; see the file comment). INT8 values dequantise as code*scale[block,
 * kv_head]. context_lens[b] == 0 gives a zero row. Accumulation is fp32; out
 * is rounded to q's dtype (nearest-even).
 *
 * Work split: the (sequence, kv_head, block) units of the whole batch are cut
 * into num_parts equal contiguous ranges, one per worker warp (0 = the
 * device default of pkv_decode_default_parts). A sequence whose blocks fall in one
 * range is finished by that worker; the others leave fp32 partial states in
 * the workspace that the combine step merges:
 *   out = sum_i exp(m_i - M) o_i / sum_i exp(m_i - M) l_i,  M = max_i m_i.
 * num_parts, batch, num_q_heads and the cache must be the same in
 * pkv_decode_workspace_size, pkv_decode_split and pkv_decode_combine.
 *
 * Supported: block_size 16, head_dim 64 or 128, num_q_heads/num_kv_heads in
 * {1, 2, 4, 8}, 1 <= batch <= 8192; q_dtype == kv_dtype for fp16/bf16 caches,
 * q_dtype PKV_F16 or PKV_BF16 for INT8 caches. q, out, caches 16-byte aligned;
 * workspace 256-byte aligned. Over an INT8 cache q enters the products in fp16
 * (here, in pkv_decode_step and in pkv_multiquery_attn): a bf16 q must be at most
 * 65504 in magnitude, and its values below 2^-14 round to multiples of 2^-24.
 * ------------------------------------------------------------------------ */

/* The default num_parts on `device`: the split kernel's resident worker
 * warps, capped at 2 CTAs (8 warps) per SM for fp16/bf16 caches at head_dim
 * 128, where fewer, longer workers read the cache faster; INT8 caches run
 * CTAs of 6 warps, two per SM at batch 256 (fewer CTAs fit for much larger
 * batches). 0 if the configuration is unsupported. */
int32_t pkv_decode_default_parts(int32_t device, int32_t batch, int32_t num_q_heads,
                                 const pkv_cache_desc *cache);

/* Workspace bytes for these sizes (num_parts 0 = the current device's
 * default). Returns 0 for an unsupported configuration. */
size_t pkv_decode_workspace_size(int32_t batch, int32_t num_q_heads,
                                 const pkv_cache_desc *cache, int32_t num_parts);

/* Split phase and combine phase back to back on `stream`. */
pkv_status pkv_decode_attn(const void *q, pkv_dtype q_dtype,
                           const void *k_cache, const void *v_cache,
                           const float *k_scales, const float *v_scales,
                           const pkv_cache_desc *cache,
                           const int32_t *block_tables, int32_t max_blocks_per_seq,
                           const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                           float softmax_scale, void *out,
                           void *workspace, size_t workspace_bytes, int32_t num_parts,
                           uint32_t *dev_status, cudaStream_t stream);

/* Split phase only: each worker streams its range of KV blocks (online
 * softmax in fp32), writes finished sequences to out and partial states
 * (m, l, unnormalised o) to the workspace. Same arguments as pkv_decode_attn. */
pkv_status pkv_decode_split(const void *q, pkv_dtype q_dtype,
                            const void *k_cache, const void *v_cache,
                            const float *k_scales, const float *v_scales,
                            const pkv_cache_desc *cache,
                            const int32_t *block_tables, int32_t max_blocks_per_seq,
                            const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                            float softmax_scale, void *out,
                            void *workspace, size_t workspace_bytes, int32_t num_parts,
                            uint32_t *dev_status, cudaStream_t stream);

/* The decode step's cache write and attention in one call: writes k_new[b],
 * v_new[b] ([batch, num_kv_heads, head_dim]; the cache dtype for fp16 / bf16
 * caches, q_dtype for INT8 caches) at position context_lens[b] - 1 of each
 * sequence, i.e. physical block block_tables[b, (L-1)/16], row (L-1)%16
 * (nothing for L == 0), then computes pkv_decode_attn over the caches
 * including that token. The same result, bit for bit in the cache (codes
 * and scales for INT8) and in out, as pkv_append with those slots followed
 * by pkv_decode_attn, in fewer launches: for fp16 / bf16 caches the split
 * kernel copies each new row into shared memory in place of the tile's row
 * (from k_new / v_new, beside the cache rows before it) and stores it into
 * the cache from there (split [+ combine]); for INT8 caches one append
 * kernel settles each touched tile's scales, requantises it if a scale
 * grows and encodes the row, one warp per (sequence, kv head), without
 * pkv_append's gather pass (append + split [+ combine]; k_scales, v_scales
 * as for pkv_append, NULL for 16-bit caches). The block receiving a
 * sequence's new token must not be shared with another sequence
 * (copy-on-write). Same workspace as pkv_decode_attn; k_new, v_new 16-byte
 * aligned. run_combine = 0 runs only the split phase (as pkv_decode_split;
 * pkv_decode_combine must follow), 1 both. */
pkv_status pkv_decode_step(const void *q, pkv_dtype q_dtype, const void *k_new,
                           const void *v_new, void *k_cache, void *v_cache,
                           float *k_scales, float *v_scales,
                           const pkv_cache_desc *cache, const int32_t *block_tables,
                           int32_t max_blocks_per_seq, const int32_t *context_lens,
                           int32_t batch, int32_t num_q_heads, float softmax_scale, void *out,
                           void *workspace, size_t workspace_bytes, int32_t num_parts,
                           int32_t run_combine, uint32_t *dev_status, cudaStream_t stream);

/* Combine phase (the split-K reduce): merges the partial states a preceding
 * pkv_decode_split left in `workspace` into out, and writes zero rows for
 * empty sequences. Must follow that split call on the same stream with the
 * same batch, num_q_heads, cache, num_parts and workspace. */
pkv_status pkv_decode_combine(const pkv_cache_desc *cache, int32_t batch,
                              int32_t num_q_heads, pkv_dtype out_dtype, void *out,
                              const void *workspace, size_t workspace_bytes,
                              int32_t num_parts, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Merge of partial attention states (the split-K reduce on its own)
 *
 * Attention over a set of tokens may be computed piece by piece: piece i
 * leaves the state (m_i, l_i, o_i), m_i its largest score, l_i = sum_t
 * exp(s_t - m_i) and o_i = sum_t exp(s_t - m_i) v_t (unnormalised, natural
 * exponent). The attention over the union of the pieces is
 *   out = sum_i exp(m_i - M) o_i / sum_i exp(m_i - M) l_i,   M = max_i m_i,
 * whatever the partition: the flash-decoding reduce that pkv_decode_combine
 * applies to the split kernel's own pieces. This call merges states the
 * caller brings, e.g. the pieces of one sequence computed on several GPUs and
 * gathered (the decode kernel's work split is described under "Decode
 * attention"; the pages name no reduce, so its form is the split identity
 * above).
 *
 * part_m, part_l  fp32 [num_states, num_heads]
 * part_o          fp32 [num_states, num_heads, head_dim], 16-byte aligned
 * row_ptr         int32 [num_rows + 1], non-decreasing: row r merges states
 *                 row_ptr[r] .. row_ptr[r+1] - 1 (a range outside
 *                 [0, num_states] is flagged PKV_DEV_BAD_INDEX, row zeroed)
 * out             [num_rows, num_heads, head_dim] in out_dtype (PKV_F16 or
 *                 PKV_BF16), fp32 arithmetic, rounded to nearest even;
 *                 8-byte aligned
 * out_m, out_l    optional fp32 [num_rows, num_heads]: the merged M and
 *                 sum_i exp(m_i - M) l_i, so that (out_m, out_l, out * out_l)
 *                 is itself a state of the union
 * A state with m = -inf (or NaN) or l <= 0 contributes nothing; a row with no
 * other state gets zeros (out_m = -inf, out_l = 0). head_dim: a multiple of
 * 4, at most 512. All arrays are device memory.
 * ------------------------------------------------------------------------ */
pkv_status pkv_merge_states(const float *part_m, const float *part_l, const float *part_o,
                            int64_t num_states, const int32_t *row_ptr, int32_t num_rows,
                            int32_t num_heads, int32_t head_dim, pkv_dtype out_dtype,
                            void *out, float *out_m, float *out_l, uint32_t *dev_status,
                            cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Multi-query attention: speculative verification and prefill chunks
 *
 * n_b = cu_q[b+1] - cu_q[b] new query tokens per sequence (already appended
 * to the cache), causal among themselves: query i of sequence b sits at
 * position L_b - n_b + i (L_b = context_lens[b]) and attends to positions
 * 0 .. L_b - n_b + i. This is the target model scoring a draft's K tokens
 * plus one in one batched pass (Continuous-Batching-LLM-Inference-Engine
 * README, feature list "Speculative decoding") and a prefill chunk mixed into
 * a continuous batch (mini-inference-engine overview). n_b = 1 everywhere is
 * decode attention.
 *
 * q, out: [cu_q[batch], num_q_heads, head_dim]. fp16 / bf16 caches: q in
 * the cache's dtype; INT8 caches: q PKV_F16 or PKV_BF16 (16-byte aligned),
 * k_scales / v_scales as for pkv_decode_attn (NULL for 16-bit caches), values
 * dequantised as code * scale. cu_q: device int32 [batch+1], non-decreasing.
 * max_q_len bounds every n_b; a sequence with n_b > max_q_len, n_b > L_b or
 * L_b beyond its table is flagged PKV_DEV_BAD_LENGTH and its rows are not
 * written. The g = num_q_heads / num_kv_heads query heads of each KV head
 * and the n_b queries form the rows of a tensor-core tile. Supported:
 * head_dim 64 or 128, g in {1, 2, 4, 8}, batch <= 4096. Workspace:
 * pkv_multiquery_workspace_size with the same batch, num_q_heads, max_q_len,
 * cache and num_parts (0 = one range per resident worker); 256-byte aligned.
 * Caches 16-byte aligned.
 * Three kernels serve the call, by rows = max_q_len * g:
 *  - fp16 / bf16 caches, rows >= 128 (a prefill chunk), q and out 16-byte
 *    aligned: a tcgen05 / tensor-memory kernel with one CTA per (sequence,
 *    kv head, 128-row tile) and no split (num_parts and the workspace are
 *    then not used, but are still checked);
 *  - rows <= 24 (speculative verification) over fp16 / bf16 caches, or over
 *    INT8 caches at head_dim 128: an mma.sync kernel with the rows on the
 *    MMA's N side, one warp per worker (num_parts counts warps);
 *  - otherwise: an mma.sync kernel with 16 rows per warp, one CTA per
 *    worker.
 * The split kernels cut their stream of units, (row tile, block) pairs of all
 * kv heads, into num_parts ranges and a combine kernel merges the pieces through
 * the workspace; a call of 2^31 - 1 units or more is flagged PKV_DEV_BAD_LENGTH and
 * writes nothing. max_blocks_per_seq: below 2^27. All compute the
 * same causal attention within the same tolerance (INT8: within 2e-2 of
 * attention over the dequantised cache).
 * ------------------------------------------------------------------------ */
size_t pkv_multiquery_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_q_len,
                                     const pkv_cache_desc *cache, int32_t num_parts);

pkv_status pkv_multiquery_attn(const void *q, pkv_dtype q_dtype, const int32_t *cu_q,
                               int32_t max_q_len, const void *k_cache, const void *v_cache,
                               const float *k_scales, const float *v_scales,
                               const pkv_cache_desc *cache, const int32_t *block_tables,
                               int32_t max_blocks_per_seq, const int32_t *context_lens,
                               int32_t batch, int32_t num_q_heads, float softmax_scale,
                               void *out, void *workspace, size_t workspace_bytes,
                               int32_t num_parts, uint32_t *dev_status, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Copy-on-write block copy (fork / rollback)
 *
 * Copies whole physical blocks src_blocks[i] -> dst_blocks[i] (all kv heads,
 * K and V, and for INT8 caches the K and V scales), i < num_pairs: the
 * private copy a copy-on-write block gets before a sequence writes into it,
 * and the rollback of a rejected speculative draft onto such copies
 * (Continuous-Batching-LLM-Inference-Engine README, feature list "Paged
 * KV-cache": copy-on-write reference counting; "Speculative decoding":
 * KV-cache rollback uses copy-on-write).
 *
 * src_blocks, dst_blocks: device int32 [num_pairs]. A pair with an id outside
 * [0, num_blocks) is skipped and flagged PKV_DEV_BAD_BLOCK; src == dst is a
 * no-op. A block that is a destination and also a source in the same call
 * gives an unspecified result (pairs run in parallel). k_scales, v_scales may
 * be NULL except for INT8 caches. Caches 16-byte aligned.
 * ------------------------------------------------------------------------ */
pkv_status pkv_copy_blocks(void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                           const pkv_cache_desc *cache, const int32_t *src_blocks,
                           const int32_t *dst_blocks, int32_t num_pairs, uint32_t *dev_status,
                           cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Decode attention without any allocation by anyone
 *
 * No counterpart on the source pages: this variant exists for callers that
 * cannot call cudaMalloc. Some runtimes plan all device memory ahead of time
 * and own the allocator, so a library may not take memory of its own; on a
 * latency-critical serving loop an allocation (and the device-wide
 * synchronisation a cudaFree brings) is not acceptable either; and such a
 * caller cannot size and keep a workspace for pkv_decode_attn.
 *
 * Same computation and arguments as pkv_decode_attn, without workspace and
 * workspace_bytes: the scratch is a fixed array of PKV_NOALLOC_SCRATCH_BYTES
 * compiled into the library, which every GPU that loads the library keeps
 * until the process exits. The function itself allocates nothing.
 *
 * - Calls that need more scratch than that (pkv_decode_workspace_size for
 *   the same batch, num_q_heads, cache and num_parts) return
 *   PKV_ERR_WORKSPACE and launch nothing.
 * - The array's device address belongs to a CUDA context: the first call in
 *   each context (e.g. the device's primary context, which the CUDA runtime
 *   uses) looks it up once, with that device current; later calls in the same
 *   context reuse it. Make that first call before any stream capture. Up to
 *   64 (device, context) pairs per process; more return PKV_ERR_UNSUPPORTED.
 * - All calls share the one array and it keeps the last call's contents;
 *   nothing in it needs to start at zero, since each call rewrites every part
 *   it later reads. Calls whose work overlaps on the GPU (other streams, other
 *   host threads) race on it: order them, e.g. on one stream.
 * ------------------------------------------------------------------------ */
#define PKV_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

pkv_status pkv_decode_attn_noalloc(const void *q, pkv_dtype q_dtype,
                                   const void *k_cache, const void *v_cache,
                                   const float *k_scales, const float *v_scales,
                                   const pkv_cache_desc *cache,
                                   const int32_t *block_tables, int32_t max_blocks_per_seq,
                                   const int32_t *context_lens, int32_t batch,
                                   int32_t num_q_heads, float softmax_scale, void *out,
                                   int32_t num_parts, uint32_t *dev_status,
                                   cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Norms of queries and keys, position rotation, cache write
 *
 * What a model does between its projection and the cache, in one pass: every
 * head row x of q and k (head_dim values) becomes y_d = x_d * w_d /
 * sqrt(mean(x^2) + eps) (w = q_weight or k_weight [head_dim] in `dtype`; NULL:
 * y = x), and the pairs of y's first rot_dim values turn by the token's
 * angles: (u, v) -> (u c - v s, u s + v c), c = cos_sin[pos, j], s =
 * cos_sin[pos, rot_dim/2 + j] for pair j. Pair j is (j, j + rot_dim/2), or
 * (2j, 2j + 1) if interleaved = 1. fp32 arithmetic, rounded once.
 *
 * Positions may have several axes (e.g. time, height, width): positions is
 * int32 [num_axes, num_tokens] and pair_axis, a HOST array of rot_dim/2 axis
 * numbers that is read during the call, says which axis turns which pair (NULL:
 * axis 0 for all). Squares are summed in fp32, so values beyond 1e18 overflow
 * the norm. cos_sin is fp32 [max_position, rot_dim], 16-byte aligned. A
 * token with a position (of any axis) outside [0, max_position) is flagged
 * PKV_DEV_BAD_INDEX and nothing of it is written.
 *
 * q, k, v: [num_tokens, heads, head_dim] with q_stride, k_stride, v_stride
 * elements between tokens (a multiple of 8, at least heads * head_dim), so
 * they may be parts of one projection's rows. q_out [num_tokens, num_q_heads,
 * head_dim] and k_out are contiguous; q_out == q and k_out == k are allowed
 * where the strides agree (other overlaps are a caller error).
 *
 * pkv_qk_norm_rope_append writes K, and V bit for bit, to slot
 * slot_mapping[n] of the cache instead (as pkv_append: negative = not written,
 * beyond the pool = flagged PKV_DEV_BAD_SLOT and not written; q_out is written
 * either way; duplicate non-negative slots are a caller error), for fp16 /
 * bf16 caches; for INT8 caches, call pkv_qk_norm_rope and pkv_append.
 *
 * Supported: dtype PKV_F16 / PKV_BF16, head_dim 64 or 128, rot_dim a multiple
 * of 16 (0: no rotation, cos_sin and positions may be NULL), num_axes 1 to 4.
 * q, k, v, outputs, weights 16-byte aligned.
 * ------------------------------------------------------------------------ */
pkv_status pkv_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                            pkv_dtype dtype, int32_t num_tokens, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, const void *q_weight,
                            const void *k_weight, float eps, const float *cos_sin,
                            int32_t max_position, int32_t rot_dim, int32_t interleaved,
                            const int32_t *positions, int32_t num_axes,
                            const int32_t *pair_axis, void *q_out, void *k_out,
                            uint32_t *dev_status, cudaStream_t stream);

pkv_status pkv_qk_norm_rope_append(const void *q, int64_t q_stride, const void *k,
                                   int64_t k_stride, const void *v, int64_t v_stride,
                                   pkv_dtype dtype, int32_t num_tokens, int32_t num_q_heads,
                                   const void *q_weight, const void *k_weight, float eps,
                                   const float *cos_sin, int32_t max_position, int32_t rot_dim,
                                   int32_t interleaved, const int32_t *positions,
                                   int32_t num_axes, const int32_t *pair_axis, void *q_out,
                                   const int64_t *slot_mapping, void *k_cache, void *v_cache,
                                   const pkv_cache_desc *cache, uint32_t *dev_status,
                                   cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Sparse decode attention: a cheap score chooses blocks
 *
 * For long contexts a decode step may attend to the blocks that matter most
 * instead of all of them. Four calls:
 *
 * pkv_block_bounds keeps, beside the cache, bounds [num_blocks, num_kv_heads,
 * 2, head_dim] in the cache's element type: the channel-wise minimum and
 * maximum of a block's keys (INT8: of its codes). After tokens were appended
 * it recomputes, from the cache, the blocks that hold positions L_b - n_b ..
 * L_b - 1 of each sequence (their rows below L_b): L_b = context_lens[b], n_b
 * = num_new[b] (NULL: 1 for every non-empty sequence; max_new is then 1).
 * max_new bounds every n_b; a sequence with n_b > max_new, n_b > L_b or L_b
 * beyond its table is flagged PKV_DEV_BAD_LENGTH and skipped. A block that gets
 * new tokens must not be shared with another sequence (copy-on-write). Bounds
 * follow no other change of the cache: whoever moves keys (pkv_evict_tokens,
 * pkv_copy_blocks) calls this for the blocks concerned, or their scores are no
 * upper bounds any more. A channel's NaN keys are passed over unless all are NaN.
 *
 * pkv_block_scores writes scores fp32 [batch, num_kv_heads,
 * max_blocks_per_seq]: for block j of sequence b the largest value that
 * <q_h, k> could take over keys within the block's bounds, maximised over the
 * KV head's query heads h: max_h sum_d max(q_hd lo_d, q_hd hi_d) (INT8: times
 * the block's scale), before any softmax scale; -inf at and past the end of
 * the sequence and for a block-table entry outside the pool (flagged). Bounds
 * may be infinite: zero times infinity counts as zero. A head whose sum is not
 * a number (NaN in q, infinities of both signs) does not count.
 *
 * pkv_block_select lists, for each (sequence, kv head), min(n, budget) of the
 * sequence's n = ceil(L_b / 16) blocks in ascending order: the first
 * keep_first, the last keep_last (keep_first + keep_last <= budget) and, of
 * the others, those with the largest scores. Exact: equal scores go to the
 * lowest block, NaN ranks lowest, -0 equals +0. block_lists int32 [batch,
 * num_kv_heads, budget] (-1 past the count), list_lens int32 [batch].
 *
 * pkv_sparse_decode_attn is pkv_decode_attn over the listed blocks: kv head h
 * of sequence b reads the first list_lens[b] entries of block_lists[b, h]
 * (int32 [batch, num_kv_heads, max_list]), block indices of the sequence in
 * any order (one listed twice counts twice). Tokens at and past context_lens[b] are
 * masked. An entry outside [0, ceil(L_b / 16)) is flagged PKV_DEV_BAD_INDEX
 * and skipped, a block-table entry outside the pool PKV_DEV_BAD_BLOCK, a list
 * length outside [0, max_list] PKV_DEV_BAD_LENGTH and clamped. No valid token
 * gives a zero row, a score that is NaN or +inf a row of NaN (and, in
 * pkv_decode_attn_mass, weights of NaN for the head's tokens). Types, heads, alignment and num_parts as for
 * pkv_decode_attn (0 also leaves short calls to a thread block or a cluster of
 * them per sequence and kv head); workspace: pkv_sparse_decode_workspace_size bytes, 256-byte
 * aligned, which calls that may overlap on the GPU must not share. A bf16 q over
 * an INT8 cache may have any size, here, in pkv_block_scores and in
 * pkv_decode_attn_mass: each head enters the products in fp16 times a power of
 * two, exact but for values below 2^-28 of the head's largest. The softmax
 * weights of such a call meet the codes of V in fp16 too (off by up to 2^-11 of a
 * weight, which the rounding of a bf16 output hides; all others keep 2^-16).
 * ------------------------------------------------------------------------ */
pkv_status pkv_block_bounds(const void *k_cache, const pkv_cache_desc *cache,
                            const int32_t *block_tables, int32_t max_blocks_per_seq,
                            const int32_t *context_lens, const int32_t *num_new, int32_t max_new,
                            int32_t batch, void *bounds, uint32_t *dev_status,
                            cudaStream_t stream);

pkv_status pkv_block_scores(const void *q, pkv_dtype q_dtype, const void *bounds,
                            const float *k_scales, const pkv_cache_desc *cache,
                            const int32_t *block_tables, int32_t max_blocks_per_seq,
                            const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                            float *scores, uint32_t *dev_status, cudaStream_t stream);

pkv_status pkv_block_select(const float *scores, int32_t batch, int32_t num_kv_heads,
                            int32_t max_blocks_per_seq, const int32_t *context_lens,
                            int32_t keep_first, int32_t keep_last, int32_t budget,
                            int32_t *block_lists, int32_t *list_lens, uint32_t *dev_status,
                            cudaStream_t stream);

size_t pkv_sparse_decode_workspace_size(int32_t batch, int32_t num_q_heads,
                                        const pkv_cache_desc *cache, int32_t num_parts);

pkv_status pkv_sparse_decode_attn(const void *q, pkv_dtype q_dtype,
                                  const void *k_cache, const void *v_cache,
                                  const float *k_scales, const float *v_scales,
                                  const pkv_cache_desc *cache,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *context_lens, const int32_t *block_lists,
                                  int32_t max_list, const int32_t *list_lens, int32_t batch,
                                  int32_t num_q_heads, float softmax_scale, void *out,
                                  void *workspace, size_t workspace_bytes, int32_t num_parts,
                                  uint32_t *dev_status, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Eviction from the cache by accumulated attention weight
 *
 * pkv_decode_attn_mass is pkv_decode_attn that also reports how much weight
 * every cached token got: with p_ht the softmax weight of token t for query
 * head h,
 *   mass_out[b, kvh, t] = (mass_in ? mass_in[b, kvh, t] : 0) + sum_h p_ht
 * over the KV head's query heads, for t < L_b (entries at and past L_b are
 * neither read nor written). mass_in, mass_out: fp32 [batch, num_kv_heads,
 * max_blocks_per_seq * 16]; the same array, or two that do not overlap. Tokens of a
 * block-table entry outside the pool get no weight. The workspace
 * (pkv_decode_mass_workspace_size, 256-byte aligned) also holds the scores, 4
 * bytes per query head and token of the table; calls that may overlap on the
 * GPU must not share it. Otherwise as pkv_decode_attn, num_parts as for
 * pkv_sparse_decode_attn.
 *
 * pkv_evict_tokens cuts every sequence to at most `budget` tokens, for each
 * (sequence, kv head) on its own: kept are the first keep_first, the last
 * keep_last (keep_first + keep_last <= budget) and, of the others, those with
 * the largest mass (exact, as pkv_block_select), min(L_b, budget) in all. The
 * kept rows of K and V become, in order, tokens 0, 1, ... of new_tables (int32
 * [batch, new_max_blocks], block ids of the same pool; budget <= 16 *
 * new_max_blocks). Written besides: kept int32 [batch, num_kv_heads, budget],
 * the old positions (-1 past the count); new_lens int32 [batch]; new_mass fp32
 * [batch, num_kv_heads, new_max_blocks * 16], the kept tokens' mass and zeros
 * behind it. INT8: a new tile's scale is the largest of its rows' old scales s,
 * and codes become rne((float)q * s_old / s), as in pkv_append; tiles whose
 * rows all stay where they are keep their codes and scale.
 * A row of new_tables that names old blocks of its sequence at their own places
 * compacts the sequence in place: new_tables may be block_tables (with
 * new_max_blocks == max_blocks_per_seq), a copy of it, or of its first columns.
 * Other new blocks must not be any sequence's old ones. No two sequences may
 * share a new block (copy-on-write). Rows move, so afterwards new_lens and
 * new_mass stand for context_lens and mass, and the bounds that pkv_block_scores
 * reads are stale for every new block: call pkv_block_bounds over new_tables and
 * new_lens with num_new = new_lens, max_new = budget. new_lens and
 * new_mass must not overlap context_lens and mass. INT8: blocks that became free
 * keep their scales; set them to 0 before they are written again. A length outside its table
 * is flagged PKV_DEV_BAD_LENGTH and keeps nothing; rows whose old block is
 * outside the pool become zeros, tiles whose new block is are not written
 * (PKV_DEV_BAD_BLOCK). head_dim 64 or 128; caches 16-byte aligned.
 * ------------------------------------------------------------------------ */
size_t pkv_decode_mass_workspace_size(int32_t batch, int32_t num_q_heads,
                                      int32_t max_blocks_per_seq, const pkv_cache_desc *cache,
                                      int32_t num_parts);

pkv_status pkv_decode_attn_mass(const void *q, pkv_dtype q_dtype,
                                const void *k_cache, const void *v_cache,
                                const float *k_scales, const float *v_scales,
                                const pkv_cache_desc *cache,
                                const int32_t *block_tables, int32_t max_blocks_per_seq,
                                const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                                float softmax_scale, void *out, const float *mass_in,
                                float *mass_out, void *workspace, size_t workspace_bytes,
                                int32_t num_parts, uint32_t *dev_status, cudaStream_t stream);

pkv_status pkv_evict_tokens(void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                            const pkv_cache_desc *cache, const int32_t *block_tables,
                            int32_t max_blocks_per_seq, const int32_t *context_lens,
                            const float *mass, int32_t batch, int32_t budget, int32_t keep_first,
                            int32_t keep_last, const int32_t *new_tables, int32_t new_max_blocks,
                            int32_t *new_lens, float *new_mass, int32_t *kept,
                            uint32_t *dev_status, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * A cache in 4 bits: quantised as it is written, read back, attended to
 *
 * A row is the head_dim values x of one token and kv head, K and V apart, of a
 * 16-bit type T (PKV_F16 or PKV_BF16, one for the whole cache). In fp32,
 *   lo = min x,  s = the smallest value of T not below (max x - lo) / 15, or the one
 *   below that where 15 s + lo would pass T's largest value,
 *   code = rne((x - lo) / s) in 0 .. 15 (0 where s = 0),  value = code * s + lo,
 * so that a value is off by at most s / 2, and finite in T. x - lo is rounded to fp32,
 * the quotient is decided exactly. A row's scale is its own: writing a token changes
 * nothing of another, in whatever order tokens come.
 *
 * k_cache, v_cache: bytes [num_blocks, num_kv_heads, 16, head_dim / 2], channel 2i
 * in the low half of byte i and 2i + 1 in the high one. k_params, v_params:
 * [num_blocks, num_kv_heads, 16, 2] of T, (s, lo) of every row. 4.25 bits per
 * value at head_dim 128, 4.5 at 64. In pkv_cache_desc kv_dtype is PKV_U4 and
 * head_dim counts values.
 *
 * pkv_u4_append writes k_new[n], v_new[n] ([num_tokens, num_kv_heads, head_dim] of
 * T = src_dtype, k_stride and v_stride values between tokens: a multiple of 8, at
 * least num_kv_heads * head_dim, so they may be parts of a projection's rows) to
 * slot slot_mapping[n]: negative = not written, beyond the pool = flagged
 * PKV_DEV_BAD_SLOT and not written, duplicate non-negative slots are a caller
 * error. Inputs must be finite, and max x - min x of a row too (fp32).
 *
 * pkv_u4_read_blocks writes the values, rounded to T = out_dtype, of whole blocks
 * src_blocks[i] -> dst_blocks[i] (int32 [num_pairs]) into a 16-bit cache k_out,
 * v_out [out_num_blocks, num_kv_heads, 16, head_dim], which pkv_multiquery_attn
 * and pkv_window_multiquery_attn read: a prompt chunk's attention over a prefix
 * held in 4 bits. A pair with an id outside its pool is flagged PKV_DEV_BAD_BLOCK
 * and skipped; a block may be read several times. A destination that occurs twice is
 * a caller error: each of its values comes from one of its sources, neighbours not
 * always from the same. Rows never written give what their bytes stand for.
 *
 * Attention for single tokens: pkv_window_decode_attn (window 0: full attention).
 * head_dim 64 or 128; all arrays 16-byte aligned (slot_mapping 8, block lists 4).
 * ------------------------------------------------------------------------ */
pkv_status pkv_u4_append(const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
                         pkv_dtype src_dtype, int32_t num_tokens, const int64_t *slot_mapping,
                         void *k_cache, void *v_cache, void *k_params, void *v_params,
                         const pkv_cache_desc *cache, uint32_t *dev_status, cudaStream_t stream);

pkv_status pkv_u4_read_blocks(const void *k_cache, const void *v_cache, const void *k_params,
                              const void *v_params, const pkv_cache_desc *cache,
                              const int32_t *src_blocks, pkv_dtype out_dtype, void *k_out,
                              void *v_out, int32_t out_num_blocks, const int32_t *dst_blocks,
                              int32_t num_pairs, uint32_t *dev_status, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Attention with a sliding window and sinks
 *
 * A query at position p sees token t <= p of its sequence if window == 0, or
 * t > p - window (the last `window` tokens, its own among them), or t < num_sinks
 * (the first tokens stay visible): layers with a sliding window, and serving
 * beyond the cache that one keeps. No other block is read: table entries of blocks
 * without a visible token may be anything, and their blocks may belong to other
 * sequences by now. What the rows of hidden tokens hold does not matter in
 * pkv_window_decode_attn.
 *
 * pkv_window_decode_attn is pkv_decode_attn (one query per sequence, at position
 * context_lens[b] - 1) over the visible tokens. Caches: fp16, bf16, INT8 with
 * float k_scales, v_scales, and PKV_U4 with the pairs of k_params, v_params as
 * k_scales, v_scales, of q_dtype's type and 16-byte aligned. A bf16 q over INT8 or
 * 4-bit codes may have any size, as for pkv_sparse_decode_attn; softmax weights
 * meet the codes of V in fp16 there (off by up to 2^-11 of a weight, which the
 * rounding of a bf16 output hides; with an fp16 q 2^-21). No visible token
 * (context_lens[b] == 0) gives a zero row, a visible score that is NaN or +inf a
 * row of NaN. num_parts as for pkv_sparse_decode_attn; workspace:
 * pkv_window_decode_workspace_size bytes, 256-byte aligned, which calls that may
 * overlap on the GPU must not share.
 *
 * pkv_window_multiquery_attn is pkv_multiquery_attn (runs of queries, causal among
 * themselves: prompt chunks, speculative verification) over the tokens that each
 * query sees; 16-bit and INT8 caches, its types, layouts, limits and alignment, and
 * pkv_window_multiquery_workspace_size. Rows that some query of the call sees must
 * be finite, also where others do not see them. The weights enter the products in two
 * parts over 16-bit caches (off by up to 2^-16 in bf16, 2^-21 in fp16) and over INT8 with
 * an fp16 q, in one fp16 part over INT8 with a bf16 q (2^-11, which the output's rounding
 * hides); INT8 V scales between 2^-113 and 2^100, those of a sequence within 2^120 of each
 * other. Runs of more than 32 rows (max_q_len times the group's heads) with q and out
 * 16-byte aligned may take, by their sizes, a kernel without pieces or combine. Such runs
 * of a bf16 q over INT8 always take it, and q may have any size there; in other runs over
 * INT8 a bf16 q must be at most 65504 in magnitude, as in pkv_multiquery_attn.
 * ------------------------------------------------------------------------ */
size_t pkv_window_decode_workspace_size(int32_t batch, int32_t num_q_heads,
                                        const pkv_cache_desc *cache, int32_t num_parts);

pkv_status pkv_window_decode_attn(const void *q, pkv_dtype q_dtype,
                                  const void *k_cache, const void *v_cache,
                                  const void *k_scales, const void *v_scales,
                                  const pkv_cache_desc *cache,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *context_lens, int32_t batch,
                                  int32_t num_q_heads, float softmax_scale, int32_t window,
                                  int32_t num_sinks, void *out, void *workspace,
                                  size_t workspace_bytes, int32_t num_parts,
                                  uint32_t *dev_status, cudaStream_t stream);

size_t pkv_window_multiquery_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_q_len,
                                            const pkv_cache_desc *cache, int32_t num_parts);

pkv_status pkv_window_multiquery_attn(const void *q, pkv_dtype q_dtype, const int32_t *cu_q,
                                      int32_t max_q_len, const void *k_cache, const void *v_cache,
                                      const float *k_scales, const float *v_scales,
                                      const pkv_cache_desc *cache, const int32_t *block_tables,
                                      int32_t max_blocks_per_seq, const int32_t *context_lens,
                                      int32_t batch, int32_t num_q_heads, float softmax_scale,
                                      int32_t window, int32_t num_sinks, void *out,
                                      void *workspace, size_t workspace_bytes, int32_t num_parts,
                                      uint32_t *dev_status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
