/*
 * pa.h -- C interface of the GB300 paged-KV decode library (libpa.so).
 *
 * The library implements the data-parallel hot path of paged KV caching:
 *   pa_reshape_and_cache  write new tokens' K/V into pool slots,
 *   pa_rope_and_cache     the same with queries and keys rotated by position,
 *   pa_gather_cache       read cached rows back as values,
 *   pa_copy_blocks        copy-on-write of shared blocks (one layer, or
 *                         all layers: pa_copy_blocks_layers),
 *   pa_swap_blocks        block copies between a device and a host pool,
 *   pa_decode             one decode step of attention over a paged pool,
 *   pa_decode_weights     the same, and the keys' weights added up,
 *   pa_decode_shared      the same for sequences that share prefixes, each attended
 *                         once,
 *   pa_attention          several causal query tokens per sequence,
 *   pa_prefill            causal attention of whole prompts, packed,
 *   pa_prefill_cached     the same over the paged pool (prompt chunks, prompts
 *                         behind a cached prefix),
 *   pa_evict              bring sequences down to a budget of tokens by their
 *                         accumulated attention weight.
 *
 * Layouts (row-major, innermost last):
 *   k_cache, v_cache   [num_blocks, block_size, num_kv_heads, head_dim]
 *                      one pool per layer, K and V separate
 *                      ("kv-cache-memory-core", section 2.2).
 *   block_tables       int32 [num_seqs, max_blocks_per_seq]; entry j of row i
 *                      is the physical block holding tokens
 *                      [j*block_size, (j+1)*block_size) of sequence i
 *                      ("vLLM intro part 2", section 3.2).  Entries at or past
 *                      cdiv(seq_lens[i], block_size) are never read.
 *   seq_lens           int32 [num_seqs], tokens attended per sequence.
 *   slot_mapping       int64 [num_tokens], absolute pool slot of each new
 *                      token, block*block_size + offset (same section).
 *   q, out             [num_seqs, num_q_heads, head_dim], one decode query
 *                      per sequence; out has the type of q.
 *   key, value         [num_tokens, num_kv_heads, head_dim].
 *   Query head h reads KV head h / (num_q_heads / num_kv_heads)
 *   ("kv-cache-memory-core", section 4.2, grouped-query attention).
 *
 * Ownership and execution: every pointer is a device pointer owned by the
 * caller, including the workspace.  Every call is asynchronous on `stream`,
 * allocates nothing and never synchronises the host.  Host-side argument
 * checks return a status before anything is launched.  Out-of-range indices
 * met on the device (a block id, a slot or a copy pair outside the pool, a
 * sequence longer than its table) skip the affected unit and OR a bit into
 * *err_flag (if err_flag is non-null); kernels never trap.  Identical inputs
 * give bit-identical outputs (no floating-point atomics).
 *
 * Supported shapes: head_dim 64 or 128; block_size 8, 16, 32, 64 or 128;
 * num_q_heads a multiple of num_kv_heads; num_kv_heads <= 256.
 * Element types: f32 caches need f32 q; f16/bf16 caches need q of the same
 * type; fp8 caches (e4m3 or e5m2) take f16 or bf16 q (head_dim 128 only).
 *
 * 4-bit caches (PA_INT4): a row -- one token's head_dim values of one KV head
 * -- is held as 4-bit codes c in 0..15 and two f16 numbers (step, low), with
 *   low = f16(min x),  step = f16((max x - low) / 15),
 *   c = (x - low) / step rounded to nearest even and limited to 0..15,
 *   and read as low + step * c;
 * x is limited to +-65504 first, a row of equal values has step 0, and a row
 * that holds a NaN reads as NaN throughout.  f16 outputs (values read back and
 * attention) are limited to +-65504: step may be rounded up, and the top of a row
 * that reaches 65504 then lies at up to 65536.  A block of a K (or V) pool is
 * block_size * num_kv_heads * (head_dim / 2 + 4) bytes: codes [num_kv_heads,
 * block_size, head_dim / 2], dimension 2b in the low nibble of byte b, then
 * (step, low) [num_kv_heads, block_size, 2].  k_scale and v_scale are ignored.
 */
#ifndef PA_H
#define PA_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,   /* null pointer, negative size, inconsistent shape */
    PA_ERR_UNSUPPORTED = 2,   /* valid but not supported (dtype combo, head_dim, ...) */
    PA_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
    PA_ERR_CUDA = 4           /* a CUDA runtime/driver call failed; see pa_last_error_detail */
} pa_status;

typedef enum {
    PA_F32 = 0,
    PA_F16 = 1,
    PA_BF16 = 2,
    PA_FP8_E4M3 = 3,          /* OCP E4M3 (finite-only, max 448), one byte */
    PA_FP8_E5M2 = 4,          /* OCP E5M2 (IEEE-like inf/NaN, max 57344), one byte */
    PA_INT4 = 5               /* 4-bit codes with a (step, low) pair per row; a cache type only */
} pa_dtype;

/* Bits OR-ed into *err_flag by device code. */
#define PA_ERRBIT_BAD_BLOCK     1u   /* block table entry outside [0, num_blocks) */
#define PA_ERRBIT_BAD_SLOT      2u   /* slot_mapping entry >= num_blocks*block_size */
#define PA_ERRBIT_BAD_PAIR      4u   /* copy pair id outside [0, num_blocks) */
#define PA_ERRBIT_SEQ_TOO_LONG  8u   /* seq_lens[i] < 0 or > max_blocks_per_seq*block_size */
#define PA_ERRBIT_WAIT_TIMEOUT 16u   /* an internal pipeline wait exceeded its time limit */
#define PA_ERRBIT_BAD_QUERY    32u   /* pa_attention, pa_prefill*: q_start (k_start) entries not
                                        increasing within [0, total_q], or a sequence with
                                        more than pa_attention's max_q_len query tokens; its
                                        rows are left unwritten.  pa_decode_shared: a group
                                        whose group_start entries do not fit */
#define PA_ERRBIT_BAD_POSITION 64u   /* pa_rope_and_cache: a position outside the table */

/* Human-readable name of a status. */
const char* pa_status_string(pa_status s);

/* Detail of the most recent failure on the calling host thread ("" if none). */
const char* pa_last_error_detail(void);

/*
 * pa_decode_workspace_size -- bytes of device workspace pa_decode needs on the
 * current device for these bounds.  max_seq_len bounds every seq_lens[i];
 * partition_tokens is the value that will be passed to pa_decode.
 * Returns 0 for invalid arguments.
 */
size_t pa_decode_workspace_size(int num_seqs, int num_q_heads, int max_seq_len,
                                int head_dim, int partition_tokens);

/*
 * pa_decode -- single-query decode attention over a paged KV pool
 * ("vLLM intro part 2", section 4 (kernel layer, the softmax and dot-product
 * formulas); PagedAttention note (vagrantpi PKM), kernel steps: look up the
 * block table, load block by block, merge across blocks with online softmax).
 *
 * For every sequence i and query head h, with g = h / (num_q_heads /
 * num_kv_heads) and L = seq_lens[i]:
 *   s_t   = scale * <q[i,h,:], K_t>            t in [0, L)
 *   out   = sum_t softmax(s)_t * V_t
 * where K_t, V_t are row (t % block_size, g) of physical block
 * block_tables[i][t / block_size].  fp8 caches are read as
 * K_t = e4m3(k) * k_scale, V_t = e4m3(v) * v_scale (scales ignored otherwise);
 * the scales are applied to the scores and the output, never per element.
 * 4-bit caches (f16 or bf16 q) are read as low + step * code.  L == 0 writes
 * zeros.
 *
 * The work is split into chunks of 16 tokens (32 for fp8 caches with
 * head_dim 128 and at most 8 query heads per KV head, 32 to 128 for 4-bit
 * caches), balanced over
 * persistent CTAs; sequences spanning several CTAs (or longer than
 * partition_tokens) are merged afterwards by a log-sum-exp reduction kernel
 * on the same stream.
 *   partition_tokens  0 lets the library choose split points; otherwise a
 *                     positive multiple of 16: sequences are additionally
 *                     split every partition_tokens tokens (4-bit caches: that
 *                     rounded up to a multiple of 32 to 128 tokens).
 * Precision: scores and sums accumulate in fp32.  The probabilities enter
 * P*V rounded to the MMA operand type: bf16 (8 significant bits) for bf16
 * caches, f16 (11 bits) for f16 caches and fp8 caches on 16-token chunks.  Outputs
 * of f16 caches are finite, within +-65504, where the values are.  With
 * a 4-bit cache it is the product of a probability and its value row's step that
 * is rounded, to f16: 11 bits down to 2^-20 of the largest such product of the
 * query row, fewer below.  There a bf16 query is scaled by a power of two into
 * f16; its elements below 2^-28 of the largest in a group of 8 or 16 rows are
 * rounded to a multiple of 2^-38 of that.
 * On the fp8 32-token path (e4m3 and e5m2 caches: the key and value bytes
 * are MMA operands as stored) the query and the probabilities are each carried
 * as two e4m3 terms, 8 significant bits (exact for bf16 queries, except
 * elements below 2^-9 of the largest in their GQA group); an infinite query
 * element saturates to +-448 there instead of propagating.  pa_decode_simt
 * keeps everything in fp32.  f32 caches (with f32 q) run on CUDA-core
 * FMAs in fp32 throughout: fp32 is no tensor-core operand type here, so that
 * kernel is the only one for them.
 *   workspace         device buffer of at least pa_decode_workspace_size(...)
 *                     bytes, 256-byte aligned; contents need no initialisation
 *                     and are scratch between calls.  Calls sharing one
 *                     workspace must not overlap on the GPU.
 *   err_flag          optional device int32 receiving PA_ERRBIT_* bits.
 * Alignment: q, out, k_cache, v_cache must be 16-byte aligned.
 */
pa_status pa_decode(void* out, const void* q, pa_dtype q_dtype,
                    const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                    const int32_t* block_tables, int max_blocks_per_seq,
                    const int32_t* seq_lens, int num_seqs, int num_q_heads,
                    int num_kv_heads, int head_dim, int block_size, int num_blocks,
                    float scale, float k_scale, float v_scale,
                    int partition_tokens, void* workspace, size_t workspace_bytes,
                    int32_t* err_flag, cudaStream_t stream);

/*
 * pa_decode_simt -- the same operation, arguments and results as pa_decode,
 * computed with CUDA-core FMAs instead of tensor-core MMAs, for every cache
 * type but 4-bit.  pa_decode runs this kernel for f32 caches; for the other types it
 * is a measured comparison point.
 */
pa_status pa_decode_simt(void* out, const void* q, pa_dtype q_dtype,
                         const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                         const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* seq_lens, int num_seqs, int num_q_heads,
                         int num_kv_heads, int head_dim, int block_size, int num_blocks,
                         float scale, float k_scale, float v_scale,
                         int partition_tokens, void* workspace, size_t workspace_bytes,
                         int32_t* err_flag, cudaStream_t stream);

/*
 * pa_decode_weights -- pa_decode that also adds up the attention that every
 * cached token receives, for pa_evict.  With p the softmax weights of
 * pa_decode, the entry of token t of sequence i and KV head g (pool slot
 * block * block_size + off) becomes
 *   weights[block][g][off] += sum over the heads h of group g of p[i, h, t]
 * except for the sequence's last fresh[i] tokens (null: 1, the token that this
 * step wrote), whose entries start from 0: slots carry what their former
 * owner left.  After a prompt of n tokens pass n once, then null.  weights is
 * f32 [num_blocks, num_kv_heads, block_size]; entries of other slots are left
 * as they were.  Sequences must not share blocks in one call (every holder
 * would add to the same entries); the sums are f32, one addition per call.  A
 * head whose scores are all -infinity (output 0) adds nothing.  Block copies and
 * swaps of K and V leave the weights behind: a copied or swapped block's go by
 * the same calls with the weights as K pool and V pool, f32 of head_dim 1.
 * Any cache type of pa_decode; fp8 caches run a kernel that converts K and V
 * to f16, so that the scores keep the query's full precision; the others give
 * pa_decode's output.
 *   fresh             int32 [num_seqs] on the device, or null
 *   workspace         at least pa_decode_weights_workspace_size(...) bytes: that of
 *                     pa_decode and 4 bytes per query head and place of the tables
 *                     (num_seqs * max_blocks_per_seq * block_size places)
 * Other arguments as for pa_decode; at most 65535 sequences.
 */
size_t pa_decode_weights_workspace_size(int num_seqs, int num_q_heads, int max_seq_len,
                                        int head_dim);
pa_status pa_decode_weights(void* out, float* weights, const void* q, pa_dtype q_dtype,
                            const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* seq_lens, const int32_t* fresh, int num_seqs,
                            int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, float scale, float k_scale, float v_scale,
                            void* workspace, size_t workspace_bytes,
                            int32_t* err_flag, cudaStream_t stream);

/*
 * pa_decode_shared -- pa_decode for sequences that share prefixes (forks of one
 * request, conversations about one document, a common system prompt): the keys of a
 * prefix are read once for all sequences of its group.
 * Group j holds the sequences group_start[j] .. group_start[j+1]-1, whose first
 * prefix_lens[j] tokens lie in the same blocks: all their tables name those blocks,
 * and the first one's is read for the group (each its own where there is too little to
 * share to pay for it: fewer than 2048 tokens' reads saved).  A prefix that ends inside a
 * block counts up to that block.  Lengths, tables and results are those of pa_decode;
 * groups of one, prefixes of 0 and sequences in no group are fine.
 *   group_start       int32 [num_groups + 1] on the device, non-decreasing within
 *                     [0, num_seqs].  A group whose entries do not fit is passed over
 *                     with PA_ERRBIT_BAD_QUERY: its sequences attend by themselves.
 *   prefix_lens       int32 [num_groups] on the device
 *   workspace         at least pa_decode_shared_workspace_size(...) bytes, 256-byte
 *                     aligned, no initialisation; calls sharing one must not overlap
 *                     on the GPU.
 *                     Beside pa_decode's it has one f32 row per (sequence, query head)
 *                     and, for prefixes cut into ranges, at most 512 rows per SM (40 MB
 *                     at head_dim 128); the number of groups adds nothing.
 * A sequence shorter than its group's prefix, or longer than its table, is left
 * unwritten with PA_ERRBIT_SEQ_TOO_LONG.  f16 and bf16 pools with q of the same type;
 * at most 128 query heads per KV head.  Precision: over the prefix as pa_prefill,
 * else as pa_decode; f16 outputs of finite values are finite, within +-65504.
 */
size_t pa_decode_shared_workspace_size(int num_seqs, int num_groups, int num_q_heads,
                                       int num_kv_heads, int max_seq_len, int head_dim);
pa_status pa_decode_shared(void* out, const void* q, pa_dtype q_dtype,
                           const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                           const int32_t* block_tables, int max_blocks_per_seq,
                           const int32_t* seq_lens, const int32_t* group_start,
                           const int32_t* prefix_lens, int num_seqs, int num_groups,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, float scale, void* workspace, size_t workspace_bytes,
                           int32_t* err_flag, cudaStream_t stream);

/*
 * pa_decode_noalloc -- pa_decode for callers that cannot supply a workspace.
 * The pages have no counterpart: this exists for callers that must not
 * allocate device memory on the call path, such as a serving loop whose
 * memory is fully pre-partitioned by its own allocator, or a plugin inside a
 * host framework that owns all device memory.  Arguments and results are
 * those of pa_decode without the workspace; the split-KV partials go to a
 * scratch array of PA_NOALLOC_SCRATCH_BYTES that the library keeps in device
 * memory on every GPU it is loaded on, until the process exits.
 *   - The first call on a device looks up the array's address on that device
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *   - A batch needing more scratch than PA_NOALLOC_SCRATCH_BYTES (see
 *     pa_decode_workspace_size) returns PA_ERR_WORKSPACE and launches nothing.
 *   - All calls on a device share the array and it keeps the previous call's
 *     contents; calls whose GPU work overlaps race on it.  No contents need
 *     to start at zero.
 *   - Nothing is allocated or freed.
 */
#define PA_NOALLOC_SCRATCH_BYTES (32u << 20)
pa_status pa_decode_noalloc(void* out, const void* q, pa_dtype q_dtype,
                            const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* seq_lens, int num_seqs, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size, int num_blocks,
                            float scale, float k_scale, float v_scale,
                            int partition_tokens, int32_t* err_flag, cudaStream_t stream);

/*
 * pa_reshape_and_cache -- write token t's K and V rows ([num_kv_heads,
 * head_dim] each) into pool slot slot_mapping[t] ("vLLM intro part 2",
 * section 3.2, slot_mapping; "kv-cache-memory-core", section 3, decode
 * appends one slot per step).
 *   slot < 0                          padding: skipped, no error.
 *   slot >= num_blocks*block_size     skipped, PA_ERRBIT_BAD_SLOT.
 * Same-type writes copy bits.  An fp8 cache quantises on write
 * ("kv-cache-memory-core", section 4.4): byte = e4m3_satfinite_rne(x / scale)
 * with x the source value widened to float, IEEE float division, round to
 * nearest even, saturation to +-448; NaN becomes the NaN code.  Sources for
 * an fp8 cache may be f32, f16 or bf16; other caches need src == kv dtype.
 * A 4-bit cache quantises each row on write (head of this file) from f32, f16
 * or bf16; it needs head_dim 64 or 128, a block_size of a multiple of 8, blocks
 * of less than 2 GB, and fewer than 2^31 rows (tokens x heads) and pool slots.
 * Duplicate slots within one call leave one of the writes (unspecified which);
 * in a 4-bit cache such a row may mix the codes of one with the (step, low) of
 * another.
 */
pa_status pa_reshape_and_cache(void* k_cache, void* v_cache, pa_dtype kv_dtype,
                               const void* key, const void* value, pa_dtype src_dtype,
                               const int64_t* slot_mapping, int num_tokens,
                               int num_kv_heads, int head_dim, int block_size,
                               int num_blocks, float k_scale, float v_scale,
                               int32_t* err_flag, cudaStream_t stream);

/*
 * pa_rope_and_cache -- rotate the queries and keys of new tokens by their
 * positions and write K and V into the pool, in one launch.
 *   q, q_out           [num_tokens, num_q_heads, head_dim]; q_out gets the rotated
 *                      queries and may be q.  num_q_heads 0 (q and q_out null): keys
 *                      and values alone.
 *   key, value         [num_tokens, num_kv_heads, head_dim]; the pool gets, at slot
 *                      slot_mapping[t], what pa_reshape_and_cache would write of the
 *                      rotated key and the value.
 *   key_out            the rotated keys, for a prompt's own attention (pa_prefill);
 *                      null or key itself are both fine.
 *   cos_sin            f32 [max_positions, rot_dim]: row p holds the rot_dim / 2
 *                      cosines, then sines, of position p's angles.
 *   positions          int64 [num_axes, num_tokens].  With one axis (sections
 *                      ignored) every pair of a token turns by its position.  With
 *                      2 to 4 (time, height, width, ...) the first sections[0] pairs
 *                      turn by the position on axis 0, the next sections[1] by that on
 *                      axis 1, and so on; sections is a HOST array of num_axes numbers
 *                      that add up to rot_dim / 2.
 * With a = x[i], b = x[i + rot_dim / 2] (interleaved != 0: a = x[2 i],
 * b = x[2 i + 1]), pair i < rot_dim / 2 becomes a cos - b sin and b cos + a sin, in
 * f32, rounded once to the type of q and key; elements from rot_dim on stay as they
 * are.  rot_dim is a multiple of 16, at most head_dim; head_dim 64 or 128.
 * Sources f32, f16 or bf16, q, key and value of one type: that of the pool, or any
 * for fp8 and 4-bit pools, which quantise the rounded key.
 *   slot < 0                          padding: nothing of the token is written.
 *   slot >= num_blocks*block_size     the same, and PA_ERRBIT_BAD_SLOT.
 *   a position outside the table      the same, and PA_ERRBIT_BAD_POSITION.
 * Other arguments, limits and duplicate slots as for pa_reshape_and_cache; fewer
 * than 2^31 rows (tokens x (query + 2 KV heads)) and pool slots.
 */
pa_status pa_rope_and_cache(void* k_cache, void* v_cache, pa_dtype kv_dtype, void* q_out,
                            void* key_out, const void* q, const void* key, const void* value,
                            pa_dtype src_dtype, const int64_t* positions, int num_axes,
                            const int* sections, const float* cos_sin, int max_positions,
                            int rot_dim, int interleaved, const int64_t* slot_mapping,
                            int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                            int block_size, int num_blocks, float k_scale, float v_scale,
                            int32_t* err_flag, cudaStream_t stream);

/*
 * pa_gather_cache -- the inverse of pa_reshape_and_cache: row t of key and
 * value ([num_kv_heads, head_dim] each) becomes the K and V row of pool slot
 * slot_mapping[t], as values of dst_dtype (a cached prefix handed to a kernel
 * that wants contiguous K and V).
 *   slot < 0                          the row is left as it was, no error.
 *   slot >= num_blocks*block_size     the same, and PA_ERRBIT_BAD_SLOT.
 * f32, f16 and bf16 caches need dst_dtype == kv_dtype and move bits; fp8
 * caches (code times k_scale or v_scale) and 4-bit caches (low + step * c)
 * give f32, f16 or bf16, computed in f32 and rounded to nearest even.  The
 * same slot may appear more than once.  head_dim 64 or 128; fewer than 2^31
 * rows (tokens x heads) and pool slots; 4-bit blocks of less than 2 GB.
 */
pa_status pa_gather_cache(void* key, void* value, pa_dtype dst_dtype,
                          const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                          const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                          int head_dim, int block_size, int num_blocks, float k_scale,
                          float v_scale, int32_t* err_flag, cudaStream_t stream);

/* Bytes of one K (or V) block of a pool, 0 for invalid arguments. */
size_t pa_block_bytes(pa_dtype kv_dtype, int num_kv_heads, int head_dim, int block_size);

/*
 * pa_copy_blocks -- copy-on-write block copies ("vLLM intro part 2",
 * section 5; aibook "显存与 KV 缓存", the copy-on-write steps: copy first,
 * repoint the table, then write).  For each pair p, the whole K block and V
 * block block_mapping[2p] are copied onto block block_mapping[2p+1].
 * num_pairs == 0 is a no-op.  A pair with an id outside [0, num_blocks) is
 * skipped with PA_ERRBIT_BAD_PAIR.  Destinations must be distinct and must
 * not be the source of another pair in the same call.
 */
pa_status pa_copy_blocks(void* k_cache, void* v_cache, pa_dtype kv_dtype,
                         const int64_t* block_mapping, int num_pairs,
                         int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, int32_t* err_flag, cudaStream_t stream);

/*
 * pa_attention -- causal attention of several new query tokens per sequence
 * over the paged pool, their K/V already written (speculative lookahead
 * tokens, or a chunk of a prompt: the "new" and "lookahead" spans one request
 * computes in one iteration, "分页省的不是 KV 字节", section 2, the
 * allocate_slots layout).  Sequence i owns query rows q_start[i] ..
 * q_start[i+1]-1 of q and out ([total_q, num_q_heads, head_dim]); they are the
 * last n_i = q_start[i+1] - q_start[i] of its L_i = seq_lens[i] tokens, and
 * query token j, at position p = L_i - n_i + j, attends keys 0..p:
 *   out[q_start[i] + j, h] = sum_{t<=p} softmax_t(scale * <q, K_t>) V_t.
 * A token with p < 0 (n_i > L_i) gets zeros.  One pass reads each K/V byte
 * once for all of a sequence's query tokens: the (token, head) rows of a GQA
 * group share the MMA tile.  q_start is a device int32 array of num_seqs + 1
 * entries, non-decreasing, q_start[0] = 0, q_start[num_seqs] = total_q; every
 * n_i <= max_q_len, and max_q_len * (num_q_heads / num_kv_heads) <= 128.
 * Tensor cores only (f16, bf16, fp8 and 4-bit caches); other arguments as for
 * pa_decode.  With every n_i = 1 the result equals pa_decode's.
 * Kernels: with at least 48 rows per KV head (max_q_len * G), a 16-bit cache
 * and partition_tokens a multiple of 32, the rows of up to four KV heads
 * (each padded to a multiple of 32) fill one 128-row tcgen05 tile whose S and
 * O accumulators live in tensor memory (32-token chunks, P rounded to the
 * cache's 16-bit type); otherwise 16-row mma.sync tiles as in pa_decode.
 */
size_t pa_attention_workspace_size(int num_seqs, int max_q_len, int num_q_heads, int max_seq_len,
                                   int head_dim, int partition_tokens);
pa_status pa_attention(void* out, const void* q, pa_dtype q_dtype,
                       const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                       const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* seq_lens, const int32_t* q_start, int num_seqs,
                       int total_q, int max_q_len, int num_q_heads, int num_kv_heads,
                       int head_dim, int block_size, int num_blocks, float scale,
                       float k_scale, float v_scale, int partition_tokens, void* workspace,
                       size_t workspace_bytes, int32_t* err_flag, cudaStream_t stream);

/*
 * pa_prefill -- causal attention of whole prompts, packed one behind the other,
 * with K and V contiguous (as a projection leaves them, or pa_gather_cache).
 * Sequence i owns query rows q_start[i] .. q_start[i+1]-1 of q and out
 * ([total_q, num_q_heads, head_dim]) and rows k_start[i] .. k_start[i+1]-1 of key
 * and value ([total_k, num_kv_heads, head_dim]; k_start null: q_start).  Its n_i
 * query tokens are the last n_i of its L_i tokens; query token j, at position
 * p = L_i - n_i + j, attends keys 0..p:
 *   out[q_start[i] + j, h] = sum_{t<=p} softmax_t(scale * <q, K_t>) V_t.
 * A token with p < 0 gets zeros, and so does one whose scores are all -infinity.
 * Keys and values that a token may not attend have no influence on it, whatever
 * they hold.  q_start and k_start: int32 [num_seqs + 1] on the device,
 * non-decreasing within [0, total_q] and [0, total_k]; rows of q and out that
 * belong to no sequence are left as they are.  A sequence whose entries do not
 * fit is skipped with PA_ERRBIT_BAD_QUERY.  Sequences may have any length,
 * 0 and 1 among them.
 * f16 or bf16, q, K, V and out of one type; head_dim 64 or 128; at most 128 query
 * heads per KV head; tensors 16-byte aligned.  Scores, sums and outputs are held
 * in f32; the weights enter P*V rounded to the type (f16: 11 bits down to 2^-21 of
 * the row's largest, fewer below; bf16: 8 bits).  f16 outputs of finite values are
 * finite, within +-65504.
 *   workspace         at least pa_prefill_workspace_size(...) bytes, 256-byte
 *                     aligned, no initialisation; calls sharing one must not
 *                     overlap on the GPU.  It holds the partial results of batches
 *                     too small to fill the GPU; others do not touch it.  The size
 *                     for some numbers of sequences and rows serves all smaller ones.
 */
size_t pa_prefill_workspace_size(int num_seqs, int total_q, int num_q_heads, int num_kv_heads,
                                 int head_dim);
pa_status pa_prefill(void* out, const void* q, const void* key, const void* value, pa_dtype dtype,
                     const int32_t* q_start, const int32_t* k_start, int num_seqs, int total_q,
                     int total_k, int num_q_heads, int num_kv_heads, int head_dim, float scale,
                     void* workspace, size_t workspace_bytes, int32_t* err_flag,
                     cudaStream_t stream);

/*
 * pa_prefill_cached -- pa_prefill with K and V in the paged pool (written by
 * pa_rope_and_cache or pa_reshape_and_cache): sequence i has L_i = seq_lens[i]
 * tokens there, the last n_i of them new.  For prompts whose first blocks were in
 * the prefix cache and for prompts that come in chunks; pa_attention does the same
 * for up to 128 (token, head) rows per KV head.  Keys of a block outside the pool
 * are left out (PA_ERRBIT_BAD_BLOCK); a sequence longer than its table is skipped
 * (PA_ERRBIT_SEQ_TOO_LONG).  f16 and bf16 pools; of others, pa_gather_cache makes
 * the contiguous K and V that pa_prefill takes.  Block sizes as for pa_decode;
 * fewer than 2^31 - 128 pool slots.
 */
pa_status pa_prefill_cached(void* out, const void* q, pa_dtype q_dtype,
                            const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* seq_lens, const int32_t* q_start, int num_seqs,
                            int total_q, int num_q_heads, int num_kv_heads, int head_dim,
                            int block_size, int num_blocks, float scale, void* workspace,
                            size_t workspace_bytes, int32_t* err_flag, cudaStream_t stream);

/*
 * pa_evict -- bring every sequence longer than `budget` down to it, per KV
 * head: of its L = seq_lens[i] tokens the first num_sink, the last num_recent
 * and, of those between, the budget - num_sink - num_recent of largest
 * accumulated weight stay (equal weights: the lower position; NaN counts as
 * the lowest).  weights is f32 [num_blocks, num_kv_heads, block_size], one
 * entry per pool slot and KV head, addressed through the same block tables as
 * the pools.
 * The kept rows of K, V and weights move to positions 0 .. budget-1: with
 * heavy = budget - num_recent, a kept row below heavy stays where it is; the
 * i-th position below heavy that is not kept takes the i-th kept row of
 * [heavy, L - num_recent); the recent rows take [heavy, budget) in their order.
 * (Attention does not depend on the order of the rows; keys carry their
 * position already.)  Different heads may keep different tokens, so all heads
 * of a sequence still share one table.
 *   new_block_tables  null: in place, the blocks of the tables must then be
 *                     this sequence's alone; rows from budget on are left as
 *                     they were and their blocks may be released.  Otherwise
 *                     int32 [num_seqs, new_max_blocks_per_seq]: all kept rows
 *                     (all L when L <= budget) are copied into these blocks,
 *                     which must be apart from the old ones; the old ones are
 *                     left as they were, and may be shared.
 *   new_seq_lens      int32 [num_seqs] out: min(L, budget).  May be seq_lens.
 *   kept              int32 [num_seqs, num_kv_heads, budget] out, may be null:
 *                     the former position of each position's row, -1 from the
 *                     new length on.
 * A sequence with L < 0 or longer than its table (PA_ERRBIT_SEQ_TOO_LONG), or
 * with a block outside the pool among the blocks it uses
 * (PA_ERRBIT_BAD_BLOCK), is skipped: kept is -1 throughout, its new length is
 * L in place and 0 otherwise.
 * The time grows with the width of the tables, not with the lengths alone: no
 * wider than the batch needs is best.
 * Any cache type; a head's row must be a multiple of 16 bytes, at most 1024, and
 * a block less than 2 GB; budget <= 2^30.
 *   workspace         at least pa_evict_workspace_size(...) bytes, 256-byte
 *                     aligned, no initialisation; calls sharing one must not
 *                     overlap on the GPU.
 */
size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int max_seq_len, int budget);
pa_status pa_evict(void* k_cache, void* v_cache, pa_dtype kv_dtype, float* weights,
                   const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                   const int32_t* new_block_tables, int new_max_blocks_per_seq,
                   int32_t* new_seq_lens, int32_t* kept, int num_seqs, int num_kv_heads,
                   int head_dim, int block_size, int num_blocks, int budget, int num_sink,
                   int num_recent, void* workspace, size_t workspace_bytes,
                   int32_t* err_flag, cudaStream_t stream);

/*
 * pa_copy_blocks_layers -- pa_copy_blocks for every layer of a model in one
 * launch: the same pairs are copied in each of the num_layers K and V pools.
 * k_caches and v_caches are HOST arrays of num_layers device pointers (pools
 * of identical shape, 16-byte aligned); num_layers <= 256.
 */
pa_status pa_copy_blocks_layers(void* const* k_caches, void* const* v_caches, int num_layers,
                                pa_dtype kv_dtype, const int64_t* block_mapping, int num_pairs,
                                int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                int32_t* err_flag, cudaStream_t stream);

/*
 * pa_swap_blocks -- block-granular swap between two pools of the same block
 * shape, typically a device pool and a host pool (preemption by swapping a
 * request's KV out to CPU memory and back in, "kv-cache-memory-core", the
 * preemption section: swap keeps the progress at the cost of CPU memory and
 * interconnect bandwidth).  For each pair p the K and V block
 * block_mapping[2p] of the source pool are copied to block
 * block_mapping[2p+1] of the destination pool.  Either pool may be host
 * memory the device can address (pinned with cudaHostAlloc / cudaMallocHost,
 * or cudaHostRegister-ed); block_mapping must be device-accessible.  Ids
 * outside their pool are skipped with PA_ERRBIT_BAD_PAIR.  The two pools must
 * not overlap.  A kernel performs the copy, so swaps of many scattered blocks
 * cost one launch, not one transfer per block.
 */
pa_status pa_swap_blocks(void* dst_k, void* dst_v, int dst_num_blocks, const void* src_k,
                         const void* src_v, int src_num_blocks, pa_dtype kv_dtype,
                         const int64_t* block_mapping, int num_pairs, int num_kv_heads,
                         int head_dim, int block_size, int32_t* err_flag, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_H */
