/*
 * pagedattn.h -- C ABI of libpagedattn.so: attention over a paged KV cache on
 * NVIDIA GB300 (sm_103a).
 *
 * The cache is a pool of fixed-size physical blocks; each request reaches its
 * tokens through a Block Table row that maps logical block b (tokens
 * b*block_size .. b*block_size + block_size - 1) to a physical block id
 * ("PagedAttention 显存分页与连续批处理(Continuous Batching)实战",
 * "PagedAttention 核心机理" part 1; "连续批处理：推理吞吐的范式革命",
 * section 2.2).
 *
 * Conventions for every call:
 *  - pa_bf16 is a raw bfloat16 bit pattern.  Every array pointer is a DEVICE
 *    pointer owned by the caller, C-contiguous, 16-byte aligned; the library
 *    never frees or keeps it.
 *  - KV cache layout: [num_blocks, block_size, num_kv_heads, head_dim].
 *  - Calls are asynchronous on `stream` (0 = legacy default stream).  The
 *    returned status covers argument checks and launch errors only.  Index
 *    errors found on the device (a slot, block id or length out of range)
 *    make the kernel skip that work item and set a device error word, which
 *    pa_check_device_errors() reads back.
 *  - The library allocates no device memory at run time.  pa_paged_attention
 *    takes a caller-provided workspace of pa_workspace_size() bytes (the
 *    allocation-free variant at the end of this header uses a fixed array
 *    built into the library instead).
 *  - Supported: block_size 16 or 32 for attention (the cache writes, block
 *    copies and swaps take any positive block_size); head_dim 64 or 128;
 *    num_q_heads a multiple of num_kv_heads with group size num_q_heads /
 *    num_kv_heads in {1, 2, 4, 8}; num_kv_heads in {1, 2, 4, 8}.  Anything
 *    else returns PA_ERR_UNSUPPORTED.
 *  - On error the call returns a non-zero status and pa_get_last_error()
 *    returns a message (per thread, valid until the next call on the thread).
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t pa_bf16;

enum pa_status {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,   /* bad size, null or misaligned pointer         */
  PA_ERR_UNSUPPORTED = 2,   /* valid but not implemented (shape, block size) */
  PA_ERR_CUDA = 3,          /* a CUDA runtime call or a launch failed       */
  PA_ERR_DEVICE_BOUNDS = 4, /* a kernel found an index out of range         */
  PA_ERR_TIMEOUT = 5,       /* a kernel gave up a bounded wait              */
  PA_ERR_WORKSPACE = 6      /* workspace missing, too small or misaligned   */
};

/* Library version, major * 10000 + minor * 100 + patch. */
int pa_version(void);

/* Message for the last non-zero status returned on this thread. */
const char *pa_get_last_error(void);

/*
 * Slot scatter.  For each new token t in [0, num_tokens) with
 * s = slot_mapping[t] >= 0, copy k[t, :, :] to k_cache[s / block_size,
 * s % block_size, :, :] and v[t] to v_cache likewise (a bit copy).  A negative
 * slot skips the token.  Slots must be distinct within one call.  This is how
 * a step's new tokens reach their on-demand allocated physical slots
 * ("PagedAttention 显存分页与连续批处理实战", comparison table: blocks are
 * allocated on demand as a block fills; TypeScript Block Manager appendToken).
 *
 *   k, v          [num_tokens, num_kv_heads, head_dim]  bf16, read
 *   k_cache, v_cache  [num_blocks, block_size, num_kv_heads, head_dim], written
 *   slot_mapping  [num_tokens] int32, read
 * A slot >= num_blocks * block_size is skipped and flags PA_ERR_DEVICE_BOUNDS.
 */
int pa_reshape_and_cache(const pa_bf16 *k, const pa_bf16 *v, int32_t num_tokens,
                         pa_bf16 *k_cache, pa_bf16 *v_cache, int32_t num_blocks,
                         int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                         const int32_t *slot_mapping, cudaStream_t stream);

/*
 * Workspace bytes for pa_paged_attention on the current device: enough for
 * every call whose num_seqs, num_tokens, max_q_len and max_seq_len are at
 * most these (so one buffer sized for a serving loop's largest step serves
 * all its steps).  The size depends only on the arguments and the device's SM
 * count.  A call needs at least its split-KV decode scratch; the prefill
 * kernel splits keys only as far as the rest of the workspace allows, so a
 * smaller workspace is never an error past that, only fewer key pieces.
 * Returns 0 if an argument is invalid.
 */
size_t pa_workspace_size(int32_t num_seqs, int32_t num_tokens, int32_t num_q_heads,
                         int32_t num_kv_heads, int32_t head_dim, int32_t max_q_len,
                         int32_t max_seq_len);

/*
 * Number of pieces the tensor-core prefill kernel splits each request's keys
 * into for a pa_paged_attention call with these sizes on the current device
 * (informational; 1 means no split).  With more than one piece, every prefill
 * row is written as per-piece partial results into the workspace and a second
 * kernel combines them with log-sum-exp weights, so the call launches one
 * kernel more.  Returns 0 if an argument is invalid.
 */
int pa_prefill_splits(int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                      int32_t head_dim, int32_t max_q_len, int32_t max_seq_len);

/*
 * Causal, GQA-aware, variable-length attention over the paged cache
 * ("连续批处理：推理吞吐的范式革命", section 4.1: walk the request's Block
 * Table, score q.k scaled, softmax, weighted sum of v, normalise; chunked
 * prefill mixes prompt slices and decode tokens in one batch:
 * "PagedAttention 显存分页与连续批处理实战", Chunked Prefill section).
 *
 * Request s owns query tokens query_start_loc[s] .. query_start_loc[s+1]-1
 * (q_len = their count, 0 allowed) and seq_lens[s] cached tokens, which
 * include those q_len tokens (write them with pa_reshape_and_cache first).
 * Query row i of request s is at position p = seq_lens[s] - q_len + i and
 * attends to positions 0..p; q head h reads kv head h / (num_q_heads /
 * num_kv_heads):
 *   out[t, h, :] = sum_j softmax_j(scale * q[t,h,:] . K[s,j,g,:]) V[s,j,g,:]
 * where K[s, j] = k_cache[block_tables[s, j / block_size], j % block_size].
 *
 *   q             [num_tokens, num_q_heads, head_dim] bf16, read
 *   k_cache, v_cache  [num_blocks, block_size, num_kv_heads, head_dim], read
 *   block_tables  [num_seqs, max_blocks] int32, read; only entries
 *                 0 .. ceil(seq_lens[s] / block_size) - 1 are read
 *   seq_lens      [num_seqs] int32, read
 *   query_start_loc [num_seqs + 1] int32, read, non-decreasing, last entry
 *                 <= num_tokens
 *   max_q_len, max_seq_len  host-side upper bounds of q_len and seq_lens
 *                 (size the launch; a request beyond them flags
 *                 PA_ERR_DEVICE_BOUNDS and its rows are not written)
 *   out           [num_tokens, num_q_heads, head_dim] bf16, written for every
 *                 token that belongs to a request; other rows are untouched
 *   workspace     device buffer of >= pa_workspace_size(...) bytes,
 *                 256-byte aligned; its contents on entry do not matter and
 *                 it must not be used by another call running concurrently
 * Accumulation is fp32; out is rounded to nearest even.  Rows with q_len == 1
 * run on the split-KV decode kernel, rows of requests with q_len >= 2 on the
 * tensor-core prefill kernel.  Where p . V runs on the tensor cores (prefill
 * rows, and decode rows when num_q_heads / num_kv_heads is 8) the softmax
 * weights enter it rounded to bf16, and the normalising sum adds the same
 * rounded weights, so every output row is an exact convex combination of V
 * rows with those weights.  A request with q_len > seq_len, seq_len >
 * max_blocks * block_size or a block id outside [0, num_blocks) flags
 * PA_ERR_DEVICE_BOUNDS.
 */
int pa_paged_attention(const pa_bf16 *q, const pa_bf16 *k_cache, const pa_bf16 *v_cache,
                       int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                       int32_t num_kv_heads, int32_t head_dim, const int32_t *block_tables,
                       int32_t max_blocks, const int32_t *seq_lens,
                       const int32_t *query_start_loc, int32_t num_seqs, int32_t num_tokens,
                       int32_t max_q_len, int32_t max_seq_len, float scale, pa_bf16 *out,
                       void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * pa_paged_attention with a host-side lower bound on the requests' query
 * rows as well: min_q_len <= q_len for every request with at least one row
 * (0 or 1: no bound).  With min_q_len >= 2 the call has no decode rows, so
 * only the prefill kernel runs (no empty decode launch after it); a request
 * with exactly one row then flags PA_ERR_DEVICE_BOUNDS and its row is not
 * written.  min_q_len > max_q_len is PA_ERR_INVALID_ARG.  Everything else is
 * pa_paged_attention.
 */
int pa_paged_attention_qrange(const pa_bf16 *q, const pa_bf16 *k_cache, const pa_bf16 *v_cache,
                              int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, const int32_t *block_tables,
                              int32_t max_blocks, const int32_t *seq_lens,
                              const int32_t *query_start_loc, int32_t num_seqs,
                              int32_t num_tokens, int32_t min_q_len, int32_t max_q_len,
                              int32_t max_seq_len, float scale, pa_bf16 *out, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/*
 * One decode step in one kernel: pa_reshape_and_cache followed by
 * pa_paged_attention, for a step whose requests all have q_len <= 1 (every
 * row a decode row; max_q_len is 1).  The decode kernel takes each request's
 * new key and value rows (token t = query_start_loc[s]) from k_new / v_new
 * straight into its copy of the request's last page, and stores them to
 * slot_mapping[t] from there, so no separate scatter runs and the new rows
 * are read from HBM once.  Precondition: slot_mapping[t] is the slot of the
 * request's position seq_lens[s] - 1 (its block table entry), or negative (the
 * row is not written and the cache's row is read, as with a separate
 * scatter); any other slot flags PA_ERR_DEVICE_BOUNDS.  Tokens outside every
 * request are not written.  bf16 cache only; arguments, workspace and errors
 * otherwise as pa_reshape_and_cache and pa_paged_attention.
 */
int pa_decode_step(const pa_bf16 *q, const pa_bf16 *k_new, const pa_bf16 *v_new,
                   pa_bf16 *k_cache, pa_bf16 *v_cache, int32_t num_blocks, int32_t block_size,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                   const int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens,
                   const int32_t *query_start_loc, int32_t num_seqs, int32_t num_tokens,
                   int32_t max_seq_len, const int32_t *slot_mapping, float scale, pa_bf16 *out,
                   void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * One serving step's slot scatter and attention, for any mix of decode rows
 * and chunked-prefill rows ("PagedAttention 显存分页与连续批处理(Continuous
 * Batching)实战", Chunked Prefill section: each iteration mixes prompt
 * slices with the running decodes), without a separate scatter kernel:
 * pa_reshape_and_cache followed by pa_paged_attention, in the attention
 * kernels themselves.  The tensor-core kernel takes a prefill request's new
 * key and value rows (tokens query_start_loc[s] ..) from k_new / v_new rather
 * than from the cache, and stores them to their slots while it runs; the
 * decode kernel does the same for decode rows (as pa_decode_step).  Outputs
 * and the cache afterwards are bit-identical to the two separate calls.
 * Precondition: slot_mapping[t] of query row i of request s is the slot of
 * its position seq_lens[s] - q_len + i (its block table entry).  A prefill
 * row with any other slot is not stored and flags PA_ERR_DEVICE_BOUNDS (its
 * attention still uses its k_new / v_new row); a decode row follows
 * pa_decode_step (a negative slot reads the cache's row, any other slot
 * flags).  Tokens outside every request are not written.  bf16 cache only;
 * arguments, workspace and errors otherwise as pa_reshape_and_cache and
 * pa_paged_attention.  Cost: every later query tile of a chunk reads the
 * chunk's new rows from k_new / v_new, and on a GB300 that measured slower
 * than one scatter launch (a 512-token chunk with 128 decode rows: 150 us
 * against 141 us for the two calls), so the step graph does not use it.
 */
int pa_paged_attention_step(const pa_bf16 *q, const pa_bf16 *k_new, const pa_bf16 *v_new,
                            pa_bf16 *k_cache, pa_bf16 *v_cache, int32_t num_blocks,
                            int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                            int32_t head_dim, const int32_t *block_tables, int32_t max_blocks,
                            const int32_t *seq_lens, const int32_t *query_start_loc,
                            int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
                            int32_t max_seq_len, const int32_t *slot_mapping, float scale,
                            pa_bf16 *out, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/*
 * Copy-on-write block copy: for each pair i, physical block
 * src_dst_pairs[2i+1] of both caches becomes a bit copy of block
 * src_dst_pairs[2i] ("PagedAttention 显存分页与连续批处理实战", comparison
 * table, Copy-on-Write sharing of prompt blocks; "连续批处理：推理吞吐的范式革命",
 * section 4.2, prefix sharing).  Destinations must be distinct and no
 * destination may be a source of the same call (pairs are then independent
 * and run in parallel).  A pair whose source is -1 is padding and is skipped
 * (a fixed-size pair list, as a captured step graph uses); any other id
 * outside [0, num_blocks) skips the pair and flags PA_ERR_DEVICE_BOUNDS.
 *
 *   src_dst_pairs [num_pairs, 2] int32 device array, read
 */
int pa_copy_blocks(pa_bf16 *k_cache, pa_bf16 *v_cache, int32_t num_blocks, int32_t block_size,
                   int32_t num_kv_heads, int32_t head_dim, const int32_t *src_dst_pairs,
                   int32_t num_pairs, cudaStream_t stream);

/*
 * Block swap for preemption by swapping instead of recomputing
 * ("连续批处理：推理吞吐的范式革命", section 3.3: a preempted request's KV
 * cache moves to CPU memory and comes back without recomputation;
 * "vLLM中的PagedAttention机制与显存优化实践", section 2.1: swap is
 * block-grained and runs asynchronously on its own CUDA streams, so pass a
 * side stream to overlap it with attention on another).
 *
 * pa_swap_out copies blocks block_ids[0..n) of both caches to the host:
 * host_k[i] and host_v[i] ([n, block_size, num_kv_heads, head_dim] bf16
 * each, in list order) become bit copies of block block_ids[i].  A kernel
 * first packs the blocks into `staging`, then two cudaMemcpyAsync calls copy
 * it to the host (use pinned host memory for the copies to be asynchronous).
 * pa_swap_in is the reverse: block block_ids[i] of both caches becomes a bit
 * copy of host_k[i] / host_v[i]; ids must then be distinct.
 *
 *   block_ids  [n] int32 device array, read; an id outside [0, num_blocks)
 *              skips that block and flags PA_ERR_DEVICE_BOUNDS
 *   staging    device buffer of pa_swap_staging_bytes(n, ...) bytes,
 *              16-byte aligned, owned by the caller, not used by another call
 *              meanwhile; its contents on entry do not matter
 *   host_k/v   host buffers of n * block_size * num_kv_heads * head_dim bf16
 * Asynchronous on `stream`: host_k / host_v hold the blocks after the stream
 * has synchronised (swap-out), and may be reused once it has (swap-in).
 */
size_t pa_swap_staging_bytes(int32_t n, int32_t block_size, int32_t num_kv_heads,
                             int32_t head_dim);
int pa_swap_out(const pa_bf16 *k_cache, const pa_bf16 *v_cache, int32_t num_blocks,
                int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                const int32_t *block_ids, int32_t n, pa_bf16 *staging, pa_bf16 *host_k,
                pa_bf16 *host_v, cudaStream_t stream);
int pa_swap_in(pa_bf16 *k_cache, pa_bf16 *v_cache, int32_t num_blocks, int32_t block_size,
               int32_t num_kv_heads, int32_t head_dim, const int32_t *block_ids, int32_t n,
               pa_bf16 *staging, const pa_bf16 *host_k, const pa_bf16 *host_v,
               cudaStream_t stream);

/*
 * 8-bit KV cache.  The pages have no counterpart: every cache they describe
 * holds the model's own precision.  This variant stores FP8 E4M3 codes (1
 * sign, 4 exponent bits of bias 7, 3 mantissa bits, no infinities, largest
 * magnitude 448) and one fp32 scale per cached (token, kv head) row, so
 * decode attention reads about half the bytes.  Each 16-token page of a
 * block holds its codes, then their scales, so one copy brings both:
 *
 *   page               [16, num_kv_heads, head_dim] uint8 codes, then
 *                      [16, num_kv_heads] fp32 scales:
 *                      pa_fp8_page_bytes(num_kv_heads, head_dim)
 *                      = 16 * num_kv_heads * (head_dim + 4) bytes
 *   k_cache, v_cache   [num_blocks, block_size / 16] pages
 *
 * The slot of token row r of page p of block b is b * block_size + 16 p + r.
 * block_size is a multiple of 16 (16 or 32 for attention).
 *
 * A row x (head_dim bf16 values) is stored as scale = max |x| / 448 (1 when
 * the row is all zero) and codes e4m3(x_c / scale), rounding to nearest with
 * ties to even and saturating; both divisions are fp32, round to nearest.
 * Attention uses code * scale in place of each cached value.  The decode
 * kernel (q_len 1) runs q . k and p . V on the tensor cores with
 * q * scale * log2(e) and p * value scale * 2^9 rounded to f16 (codes
 * convert to f16 exactly; the 2^9 is removed exactly).  The prefill kernel
 * (q_len >= 2, the chunked-prefill rows) turns each cached row into
 * f16(code * f16(scale)) in shared memory (codes exact in f16, one rounding
 * of the scale and one of the product), and runs
 * its tcgen05 products on f16 operands: q * scale * log2(e) and p rounded
 * to f16.  The row maxima this is good for: in the prefill kernel 1.1e-4 to
 * 65504 (values below 6.1e-5, f16's normal range, are right to 2^-23 whatever
 * their row; past 65504 they are infinite); in the decode kernel any for keys,
 * up to 5e4 for values (p * value scale * 2^9 is right to 2^-25 below f16's
 * normal range).  head_dim is 64 or 128; the same shapes as the bf16 cache.
 *
 * pa_fp8_page_bytes: the page size above (0 for a non-positive argument).
 *
 * pa_reshape_and_cache_fp8: pa_reshape_and_cache, quantising each new row
 * (codes and scale written to the new token's slot).  Alignment: k, v and
 * both caches 16 bytes, slot_mapping 4 bytes.
 */
size_t pa_fp8_page_bytes(int32_t num_kv_heads, int32_t head_dim);

int pa_reshape_and_cache_fp8(const pa_bf16 *k, const pa_bf16 *v, int32_t num_tokens,
                             uint8_t *k_cache, uint8_t *v_cache, int32_t num_blocks,
                             int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                             const int32_t *slot_mapping, cudaStream_t stream);

/*
 * pa_paged_attention over the 8-bit cache (same arguments, meaning, errors
 * and workspace as pa_paged_attention, with the caches in the page format
 * above).  Decode and prefill rows, mixed in one call, as
 * pa_paged_attention (see above for the arithmetic).
 */
int pa_paged_attention_fp8(const pa_bf16 *q, const uint8_t *k_cache, const uint8_t *v_cache,
                           int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim, const int32_t *block_tables,
                           int32_t max_blocks, const int32_t *seq_lens,
                           const int32_t *query_start_loc, int32_t num_seqs, int32_t num_tokens,
                           int32_t max_q_len, int32_t max_seq_len, float scale, pa_bf16 *out,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * pa_copy_blocks over the 8-bit cache: each pair copies the destination
 * block's pages (codes and scales) from the source block (same pair rules,
 * padding and errors).  Both caches 16-byte aligned.
 */
int pa_copy_blocks_fp8(uint8_t *k_cache, uint8_t *v_cache, int32_t num_blocks,
                       int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                       const int32_t *src_dst_pairs, int32_t num_pairs, cudaStream_t stream);

/*
 * A step's integer inputs built on the GPU from the requests' lengths: what
 * the pages' block manager does on the host when a step is scheduled ("blocks
 * are allocated on demand as a block fills": "PagedAttention 显存分页与连续批处理
 * 实战", comparison table and TypeScript Block Manager), so that a loop of
 * steps can run without the host between them.
 *
 * Request s has c = context_lens[s] tokens in the cache and gets n =
 * new_lens[s] more (0 allowed), which need ceil((c + n) / block_size) -
 * ceil(c / block_size) blocks.  Requests are served in order while the blocks
 * and the token rows last: the first request that does not fit in what is
 * left of the free list or of num_tokens ends the served ones, and it and all
 * after it get no block and no row.  Blocks are taken from the top of the free
 * list (its entry free_count - 1 first), as the host allocator hands them out.
 *   block_tables[s, j]    the new block's id, for j = ceil(c / block_size) ..
 *                         ceil((c + n) / block_size) - 1 (other entries are
 *                         left as they are)
 *   seq_lens[s]           c + n (c when the request was not served)
 *   query_start_loc[s]    new tokens of the served requests before s
 *   slot_mapping[t]       slot of the token in row t; -1 past the last token
 *   positions[a, t]       position of the token in row t, c + i for the i-th
 *                         new one, plus position_offsets[s], alike on every
 *                         axis; 0 past the last token.  (A caller with image
 *                         or video tokens overwrites their columns.)
 *   free_count_out        free_count minus the blocks handed out
 * These are pa_rotary_reshape_and_cache's, pa_reshape_and_cache's and
 * pa_paged_attention's inputs.  Copy-on-write stays with the caller: the block
 * that holds position c - 1 must be the request's own when c is not a
 * multiple of block_size (pa_copy_blocks).
 *
 *   context_lens, new_lens [num_seqs] int32, read
 *   position_offsets [num_seqs] int32, read, or NULL (0)
 *   block_tables  [num_seqs, max_blocks] int32, entries 0 .. ceil(c /
 *                 block_size) - 1 set; read and written
 *   free_blocks   [num_blocks] int32, read; the first free_count entries are
 *                 distinct free block ids
 *   free_count, free_count_out  [1] int32, read and written; may be the same
 *   seq_lens      [num_seqs] int32, written; may be context_lens itself (a
 *                 replayed step then goes on from the last one)
 *   query_start_loc [num_seqs + 1], slot_mapping [num_tokens] int32, written
 *   positions     [num_axes, num_tokens] int32, written (num_axes 0 .. 4; 0:
 *                 not written, may be NULL)
 * No two of the other arrays may overlap.  All 4-byte aligned.  num_seqs is at
 * most 16384.  Flags PA_ERR_DEVICE_BOUNDS: a request that was not served; a
 * negative length or c + n > max_blocks * block_size (that request gets no
 * block and no row, later ones are served); a free_count outside [0,
 * num_blocks] (taken as 0); a block id outside [0, num_blocks) (-1 goes into
 * the table and the slot).
 */
int pa_build_step(const int32_t *context_lens, const int32_t *new_lens,
                  const int32_t *position_offsets, int32_t num_seqs, int32_t num_tokens,
                  int32_t num_axes, int32_t *block_tables, int32_t max_blocks,
                  int32_t block_size, const int32_t *free_blocks, const int32_t *free_count,
                  int32_t *free_count_out, int32_t num_blocks, int32_t *seq_lens,
                  int32_t *query_start_loc, int32_t *slot_mapping, int32_t *positions,
                  cudaStream_t stream);

/*
 * Rotary positions with one or several axes on a step's queries and keys, and
 * the slot scatter of its keys and values (pa_reshape_and_cache) in the same
 * pass.  The pages have no counterpart: they take q, k and v as given.
 *
 * Pair i (i < rotary_dim / 2) of every q and k head of token t is turned by
 *   theta = positions[axes[i], t] * inv_freq[i]   (radians),
 *   (x1, x2) -> (x1 cos theta - x2 sin theta, x2 cos theta + x1 sin theta),
 * with (x1, x2) the elements (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when
 * interleaved is not 0.  Elements from rotary_dim on are passed through.  With
 * one axis these are ordinary rotary positions; with several (time, height,
 * width of image and video tokens) each frequency belongs to the axis axes[i]
 * names.  theta is taken modulo a turn in 64-bit integer arithmetic, so far
 * positions lose nothing; the rotation is fp32 and each result is rounded
 * once, to bf16 (nearest even) or, for keys in the 8-bit cache, to its code.
 *
 *   q             [num_tokens, num_q_heads, head_dim] bf16, read; token t at
 *                 q + t * q_stride elements, its heads contiguous (so q, k and
 *                 v may be slices of one projection's output)
 *   k, v          [num_tokens, num_kv_heads, head_dim] bf16, read, alike
 *   positions     num_axes rows of num_tokens int32 (any sign), row a at
 *                 positions + a * positions_stride
 *   inv_freq      [rotary_dim / 2] double, finite, |inv_freq| < 2^31
 *   axes          [rotary_dim / 2] int32 in [0, num_axes), or NULL (axis 0)
 *   q_out         [num_tokens, num_q_heads, head_dim] bf16, written, every
 *                 row; may be q itself when q_stride is the row's length
 *   k_cache, v_cache  as pa_reshape_and_cache (as pa_reshape_and_cache_fp8
 *                 for the _fp8 form), written at the tokens' slots
 *   slot_mapping  [num_tokens] int32, read; distinct; negative: the token's
 *                 key and value are not written (its q_out row is)
 * head_dim 64 or 128; rotary_dim a multiple of 16 up to head_dim (0: none);
 * num_axes 1 .. 4; strides multiples of 8 elements; q, k, v, q_out and the
 * caches 16-byte aligned.  A slot past the pool is skipped, an axis or a
 * frequency out of range is taken as 0; each flags PA_ERR_DEVICE_BOUNDS.
 */
int pa_rotary_reshape_and_cache(const pa_bf16 *q, int64_t q_stride, const pa_bf16 *k,
                                int64_t k_stride, const pa_bf16 *v, int64_t v_stride,
                                int32_t num_tokens, const int32_t *positions,
                                int64_t positions_stride, int32_t num_axes,
                                const double *inv_freq, const int32_t *axes, int32_t rotary_dim,
                                int32_t interleaved, pa_bf16 *q_out, pa_bf16 *k_cache,
                                pa_bf16 *v_cache, int32_t num_blocks, int32_t block_size,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                const int32_t *slot_mapping, cudaStream_t stream);
int pa_rotary_reshape_and_cache_fp8(const pa_bf16 *q, int64_t q_stride, const pa_bf16 *k,
                                    int64_t k_stride, const pa_bf16 *v, int64_t v_stride,
                                    int32_t num_tokens, const int32_t *positions,
                                    int64_t positions_stride, int32_t num_axes,
                                    const double *inv_freq, const int32_t *axes,
                                    int32_t rotary_dim, int32_t interleaved, pa_bf16 *q_out,
                                    uint8_t *k_cache, uint8_t *v_cache, int32_t num_blocks,
                                    int32_t block_size, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t head_dim,
                                    const int32_t *slot_mapping, cudaStream_t stream);

/*
 * pa_paged_attention with a sliding window and sink tokens: the query row at
 * position p attends to the positions j <= p with p - j < window or
 * j < num_sinks (the row's own position always among them).  The pages have
 * no counterpart: their attention is over the whole sequence.
 *
 * Only block-table entries of blocks that hold a key some row of the call
 * sees are read: with first = seq_lens[s] - q_len - window + 1 (the first
 * row's first position), entries whose blocks lie wholly between num_sinks
 * and first may hold anything, and their blocks may have been freed and
 * reused (a rolling cache).  Cached rows outside every row's view have no
 * effect, whatever they hold.  Among the rows of a prompt chunk a key that is
 * not finite reaches those that see it, and a value that is not finite may
 * also reach those computed with them (up to 256 / group consecutive tokens).
 *
 *   window        >= 1; a window of max_seq_len or more is
 *                 pa_paged_attention_qrange
 *   num_sinks     >= 0
 *   min_q_len     as pa_paged_attention_qrange (0 or 1: no bound)
 * Everything else (layouts, workspace of pa_workspace_size() bytes, errors,
 * precision) as pa_paged_attention, and as pa_paged_attention_fp8 for the
 * 8-bit cache's form.
 */
int pa_paged_attention_window(const pa_bf16 *q, const pa_bf16 *k_cache, const pa_bf16 *v_cache,
                              int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim,
                              const int32_t *block_tables, int32_t max_blocks,
                              const int32_t *seq_lens, const int32_t *query_start_loc,
                              int32_t num_seqs, int32_t num_tokens, int32_t min_q_len,
                              int32_t max_q_len, int32_t max_seq_len, int32_t window,
                              int32_t num_sinks, float scale, pa_bf16 *out, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);
int pa_paged_attention_window_fp8(const pa_bf16 *q, const uint8_t *k_cache,
                                  const uint8_t *v_cache, int32_t num_blocks,
                                  int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, const int32_t *block_tables,
                                  int32_t max_blocks, const int32_t *seq_lens,
                                  const int32_t *query_start_loc, int32_t num_seqs,
                                  int32_t num_tokens, int32_t min_q_len, int32_t max_q_len,
                                  int32_t max_seq_len, int32_t window, int32_t num_sinks,
                                  float scale, pa_bf16 *out, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/*
 * Long contexts: read less of the cache, or hold less of it.
 *
 * pa_summarize_blocks, pa_select_blocks and pa_paged_attention_blocks let each
 * query attend to a chosen part of its context: bounds of each block's keys
 * are kept up to date beside the cache, every query picks blocks by a score
 * from the bounds, and the attention reads those blocks alone.
 * pa_paged_attention_weights is attention that also adds up how much weight
 * each cached token gets, and pa_evict_tokens drops the tokens of least weight
 * and returns the blocks that this empties.  The pages have no counterpart for
 * either ("PagedAttention 核心机理" reads every block of a request).
 *
 * All take block_size 16 or 32, head_dim 64 or 128, num_kv_heads 1, 2, 4 or 8
 * and (where there are queries) group sizes 1, 2, 4 and 8; anything else is
 * PA_ERR_UNSUPPORTED.  They run on the GPU alone and may be captured.
 *
 * pa_summarize_blocks: for the blocks that the step's new tokens are in
 * (request s: positions seq_lens[s] - q_len .. seq_lens[s] - 1, q_len from
 * query_start_loc), and each kv head, the largest and the smallest value of
 * every channel over the block's keys below seq_lens[s]:
 *   bounds        int8 [num_blocks, num_kv_heads, 2, head_dim], the maxima's
 *                 codes, then the minima's; 16-byte aligned
 *   bound_scales  float [num_blocks, num_kv_heads]: p, the least power of two
 *                 with |x| <= 127 p for all of them (1 where all are 0; not
 *                 below 2^-126)
 *   codes         ceil(max / p) and floor(min / p): bounds after rounding too
 * A NaN in a key counts as 0 and an infinity as the largest finite float.
 * Call it after the step's keys are in the cache.  query_start_loc NULL: every
 * block of every request (after an eviction, a swap in or a block copy);
 * num_tokens is then not used.  Of blocks that several requests share, those
 * that are full come out alike whichever request writes them.
 */
int pa_summarize_blocks(const pa_bf16 *k_cache, int32_t num_blocks, int32_t block_size,
                        int32_t num_kv_heads, int32_t head_dim, const int32_t *block_tables,
                        int32_t max_blocks, const int32_t *seq_lens,
                        const int32_t *query_start_loc, int32_t num_seqs, int32_t num_tokens,
                        int8_t *bounds, float *bound_scales, cudaStream_t stream);
int pa_summarize_blocks_fp8(const uint8_t *k_cache, int32_t num_blocks, int32_t block_size,
                            int32_t num_kv_heads, int32_t head_dim, const int32_t *block_tables,
                            int32_t max_blocks, const int32_t *seq_lens,
                            const int32_t *query_start_loc, int32_t num_seqs, int32_t num_tokens,
                            int8_t *bounds, float *bound_scales, cudaStream_t stream);

/*
 * pa_select_blocks: for each new token (position p) and kv head, num_selected
 * of the blocks 0 .. p / block_size: the first num_sinks, the last num_recent
 * (at least 1, so the token's own block is among them), and of the others
 * those of the highest score, ties to the lowest index.
 *   selected      int32 [num_tokens, num_kv_heads, num_selected]: logical
 *                 block indices in increasing order, then -1 where there are
 *                 fewer; rows of no request are left as they were
 *   score         of a block for a kv head: the largest over the q heads of
 *                 its group of  p_q p sum_c x_c (x_c > 0 ? max_c : min_c),  with
 *                 q's codes x = rint(q / p_q) (nearest, ties to even), p_q by
 *                 the rule of bound_scales, and the block's codes and scale:
 *                 an upper bound of q k over the block's keys, but for the
 *                 rounding of q.  The sums are of integers and exact, and
 *                 scores are compared by them and the powers of two, whatever
 *                 their size, so the result depends on nothing but the inputs.
 *   max_seq_len   at most 49152 blocks
 * The product is with q as it is given (scale the scores and they keep their
 * order).
 */
int pa_select_blocks(const pa_bf16 *q, const int8_t *bounds, const float *bound_scales,
                     int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t head_dim, const int32_t *block_tables,
                     int32_t max_blocks, const int32_t *seq_lens, const int32_t *query_start_loc,
                     int32_t num_seqs, int32_t num_tokens, int32_t max_seq_len,
                     int32_t num_selected, int32_t num_sinks, int32_t num_recent,
                     int32_t *selected, cudaStream_t stream);

/*
 * pa_paged_attention_blocks: attention of each new token (position p, q_len
 * of any length) over the blocks listed for it and its kv head, and in them
 * over the positions up to p.
 *   selected      as pa_select_blocks writes it; in any order, negative
 *                 entries are passed over, an entry listed twice counts twice,
 *                 an entry past the token's own block is flagged and passed
 *                 over.  A token with nothing listed gets zeros.
 * No workspace.  Rows of out that belong to no request are left as they were.
 * Weights are rounded to 2^-16 (two bf16), sums are in fp32.  Every token
 * reads its own blocks: meant for decode rows and a few drafted tokens.
 */
int pa_paged_attention_blocks(const pa_bf16 *q, const pa_bf16 *k_cache, const pa_bf16 *v_cache,
                              int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim,
                              const int32_t *block_tables, int32_t max_blocks,
                              const int32_t *seq_lens, const int32_t *query_start_loc,
                              int32_t num_seqs, int32_t num_tokens, float scale,
                              const int32_t *selected, int32_t num_selected, pa_bf16 *out,
                              cudaStream_t stream);
int pa_paged_attention_blocks_fp8(const pa_bf16 *q, const uint8_t *k_cache,
                                  const uint8_t *v_cache, int32_t num_blocks, int32_t block_size,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  const int32_t *block_tables, int32_t max_blocks,
                                  const int32_t *seq_lens, const int32_t *query_start_loc,
                                  int32_t num_seqs, int32_t num_tokens, float scale,
                                  const int32_t *selected, int32_t num_selected, pa_bf16 *out,
                                  cudaStream_t stream);

/*
 * pa_paged_attention_weights: pa_paged_attention, and
 *   weights       float [num_seqs, num_kv_heads, weights_len], row s of the
 *                 request in row s of block_tables, entry j its cached token
 *                 j: for j < seq_lens[s] the sum, over the request's new rows
 *                 that see token j and over the q heads of the kv head, of the
 *                 softmax weight of j is added; the entries of the new tokens
 *                 (the last q_len) start from 0 in this call.  Entries from
 *                 seq_lens[s] on, and rows of requests without new tokens, are
 *                 left as they were.  weights_len >= max_seq_len.
 * The weights are fp32 sums in one order (no atomics); the scores behind them
 * are sums of exact products in fp32.  Prompt chunks' outputs are
 * pa_paged_attention's; decode rows' weights are rounded to 2^-16.
 * Workspace: pa_weights_workspace_size() bytes, 256-byte aligned; calls with
 * max_q_len <= 1 use none (NULL will do).
 */
size_t pa_weights_workspace_size(int32_t num_seqs, int32_t num_tokens, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t max_q_len,
                                 int32_t max_seq_len);
int pa_paged_attention_weights(const pa_bf16 *q, const pa_bf16 *k_cache, const pa_bf16 *v_cache,
                               int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim,
                               const int32_t *block_tables, int32_t max_blocks,
                               const int32_t *seq_lens, const int32_t *query_start_loc,
                               int32_t num_seqs, int32_t num_tokens, int32_t min_q_len,
                               int32_t max_q_len, int32_t max_seq_len, float scale,
                               float *weights, int32_t weights_len, pa_bf16 *out,
                               void *workspace, size_t workspace_bytes, cudaStream_t stream);
int pa_paged_attention_weights_fp8(const pa_bf16 *q, const uint8_t *k_cache,
                                   const uint8_t *v_cache, int32_t num_blocks,
                                   int32_t block_size, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim,
                                   const int32_t *block_tables, int32_t max_blocks,
                                   const int32_t *seq_lens, const int32_t *query_start_loc,
                                   int32_t num_seqs, int32_t num_tokens, int32_t min_q_len,
                                   int32_t max_q_len, int32_t max_seq_len, float scale,
                                   float *weights, int32_t weights_len, pa_bf16 *out,
                                   void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream);

/*
 * pa_evict_tokens: each request s with seq_lens[s] > budgets[s] keeps
 * budgets[s] tokens, for each kv head its own: the first num_sinks, the last
 * num_recent, and of those between the ones of the largest weights (ties: the
 * lowest index; NaN counts as the largest).  The kept tokens' K, V and weights
 * move together in order: kept token i becomes token i.  Rows and weights from
 * the new length on are left as they were, and so are the block tables: the
 * entries past the new length's blocks hold nothing any more (pa_build_step
 * writes them anew).
 *   seq_lens      [num_seqs], at most max_seq_len (itself at most 524288);
 *                 the tokens' rows must belong to the request alone (copy
 *                 shared blocks first; a budget of seq_lens[s] or more leaves
 *                 a request alone)
 *   budgets       [num_seqs], each at least num_sinks + num_recent
 *   seq_lens_out  [num_seqs] new lengths; may be seq_lens
 *   free_blocks   [num_blocks], free_count [1]: as pa_build_step takes them;
 *                 the blocks of the tables' columns from ceil(budget /
 *                 block_size) on are pushed in the order of requests and
 *                 columns, entries that name no block passed over (and
 *                 flagged).  free_count_out [1] may be free_count.
 *   position_offsets  [num_seqs] or NULL: the tokens that went are added, so
 *                 that pa_build_step gives later tokens their true positions
 * A model of several layers has caches and weights for each, and one set of
 * tables, lengths and offsets and one free list for all: one call a layer, all
 * with the same lengths and count.  Every call but the last writes its new
 * lengths and count elsewhere (seq_lens_out, free_count_out: scratch of their
 * own) and has position_offsets NULL; the blocks that each pushes are the same,
 * to the same places.  With lengths updated in place by the first layer's call
 * the others would find nothing to evict and move no row.
 * A length or budget out of range is flagged and its request left alone.  A
 * table entry that names no block is flagged: a row that would move from or to
 * it does not, and the row and weight in its place stay as they are.
 */
int pa_evict_tokens(pa_bf16 *k_cache, pa_bf16 *v_cache, float *weights, int32_t weights_len,
                    int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                    int32_t head_dim, const int32_t *block_tables, int32_t max_blocks,
                    const int32_t *seq_lens, const int32_t *budgets, int32_t num_seqs,
                    int32_t max_seq_len, int32_t num_sinks, int32_t num_recent,
                    int32_t *free_blocks, const int32_t *free_count, int32_t *seq_lens_out,
                    int32_t *free_count_out, int32_t *position_offsets, cudaStream_t stream);
int pa_evict_tokens_fp8(uint8_t *k_cache, uint8_t *v_cache, float *weights, int32_t weights_len,
                        int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                        int32_t head_dim, const int32_t *block_tables, int32_t max_blocks,
                        const int32_t *seq_lens, const int32_t *budgets, int32_t num_seqs,
                        int32_t max_seq_len, int32_t num_sinks, int32_t num_recent,
                        int32_t *free_blocks, const int32_t *free_count, int32_t *seq_lens_out,
                        int32_t *free_count_out, int32_t *position_offsets,
                        cudaStream_t stream);

/*
 * Synchronises `stream`, then reads and clears the device error word that
 * the kernels of this library set on the current device.  Returns PA_OK,
 * PA_ERR_DEVICE_BOUNDS, PA_ERR_TIMEOUT or PA_ERR_CUDA.
 */
int pa_check_device_errors(cudaStream_t stream);

/*
 * Failure-detection self-test.  Every wait inside the library's kernels (on
 * a copy landing, on a tensor-core product, on another warp's hand-off) is
 * bounded: past its limit (2 s) the kernel sets PA_ERR_TIMEOUT's bit in the
 * device error word, stops waiting, waits (with the limit again) for its own
 * copies in flight and returns, so the context stays usable.
 * This call runs that same wait, with limit_ns (at most 1 s), on a barrier
 * that nothing completes, and then the wait for copies in flight on one that
 * completes 0.2 s later; pa_check_device_errors afterwards returns
 * PA_ERR_TIMEOUT (device word 0x2; 0x3 if the second wait gave up too).  It
 * faults nothing and hangs nothing.  limit_ns of 0 or above 1 s is
 * PA_ERR_INVALID_ARG.
 */
int pa_selftest_wait_timeout(uint64_t limit_ns, cudaStream_t stream);

/*
 * Allocation-free form of pa_paged_attention.  The pages have no counterpart
 * for it; it exists for callers that cannot allocate device memory where they
 * run attention: code running while a stream is captured into a CUDA graph,
 * plugins whose host owns all device memory, serving loops that must not
 * allocate after start-up.
 *
 * Same arguments, layout and results as pa_paged_attention, minus the
 * workspace: scratch comes from an array built into the library
 * (pa_noalloc_scratch_bytes() bytes, 8 MiB, held on every device that loads
 * the library until the process exits).  A call needing more scratch than
 * that (see pa_workspace_size) returns PA_ERR_WORKSPACE.  Allocates nothing.
 * The first call on a device looks up the array's device address and keeps
 * it for the life of the process: make that first call before any stream
 * capture (a call with num_seqs = 0 and a valid cache geometry does only
 * this set-up and launches nothing), and do not use the library across a
 * cudaDeviceReset, after which the kept address is stale.  Calls share the
 * array, so calls whose executions overlap on the GPU race and must be
 * serialised by the caller.
 */
size_t pa_noalloc_scratch_bytes(void);

int pa_paged_attention_noalloc(const pa_bf16 *q, const pa_bf16 *k_cache,
                               const pa_bf16 *v_cache, int32_t num_blocks, int32_t block_size,
                               int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               const int32_t *block_tables, int32_t max_blocks,
                               const int32_t *seq_lens, const int32_t *query_start_loc,
                               int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
                               int32_t max_seq_len, float scale, pa_bf16 *out,
                               cudaStream_t stream);

/*
 * One serving step captured as a CUDA graph: block copies (pa_copy_blocks),
 * slot scatter (pa_reshape_and_cache) and attention (pa_paged_attention) of
 * the iteration-level schedule ("PagedAttention 显存分页与连续批处理
 * (Continuous Batching)实战", continuous batching and Chunked Prefill
 * sections: every step runs the same sequence of operations over whichever
 * requests the scheduler picked), launched with one call instead of three to
 * five kernel launches.  The pages have no counterpart for the graph itself.
 *
 * The graph is built once over fixed device buffers sized for the largest
 * step (the pa_step_buffers maxima); before each launch the caller writes the
 * step's inputs into those buffers, padded to the maxima:
 *   - tokens t >= the step's count: slot_mapping[t] = -1 (not written);
 *   - sequences s >= the step's count: query_start_loc[s + 1] =
 *     query_start_loc[s] (no rows) and seq_lens[s] = 0;
 *   - copy pairs i >= the step's count: copy_pairs[2i] = -1 (skipped).
 * A step's sizes must stay within the maxima (max_q_len and max_seq_len
 * included: a request beyond them flags PA_ERR_DEVICE_BOUNDS at run time).
 * The graph runs scatter + attention as pa_decode_step (max_q_len 1: one
 * kernel, whose slot precondition applies) or as pa_reshape_and_cache then
 * pa_paged_attention.
 * Rows of out that belong to no request are left as they were.
 *
 * If host_meta is not NULL, every launch first copies meta_bytes from
 * host_meta (pinned host memory) to dev_meta, so that the step's inputs (the
 * integer arrays, and q / k_new / v_new too if the caller places them there)
 * can live in one region of dev_meta and reach the GPU in one copy inside the
 * graph.  If host_out is not NULL, every launch ends by copying the first
 * out_copy_bytes of out to host_out (pinned host memory).  The copies read
 * and write host memory when the launch executes on the GPU, not when it is
 * issued: do not touch those buffers until then (for example, alternate two
 * graphs over two sets of host buffers).
 *
 * Buffers stay owned by the caller and must outlive the graph.  Launches of
 * one graph, and of graphs sharing buffers, must not overlap on the GPU.
 */
typedef struct pa_step_buffers {
  pa_bf16 *k_cache, *v_cache;   /* [num_blocks, block_size, num_kv_heads, head_dim] */
  int32_t num_blocks, block_size, num_q_heads, num_kv_heads, head_dim;
  int32_t max_tokens;           /* rows of q, k_new, v_new, out, slot_mapping */
  int32_t max_seqs;             /* rows of block_tables and seq_lens (+1: query_start_loc) */
  int32_t max_blocks;           /* columns of block_tables */
  int32_t max_pairs;            /* rows of copy_pairs; 0: the graph has no copy step */
  int32_t max_q_len, max_seq_len;
  float scale;
  const pa_bf16 *q;             /* [max_tokens, num_q_heads, head_dim] */
  const pa_bf16 *k_new, *v_new; /* [max_tokens, num_kv_heads, head_dim] */
  pa_bf16 *out;                 /* [max_tokens, num_q_heads, head_dim] */
  const int32_t *slot_mapping;  /* [max_tokens] */
  const int32_t *block_tables;  /* [max_seqs, max_blocks] */
  const int32_t *seq_lens;      /* [max_seqs] */
  const int32_t *query_start_loc; /* [max_seqs + 1] */
  const int32_t *copy_pairs;    /* [max_pairs, 2] or NULL when max_pairs == 0 */
  void *workspace;              /* >= pa_workspace_size(max_seqs, max_tokens, ...) bytes */
  size_t workspace_bytes;
  const void *host_meta;        /* optional pinned host source of a per-launch copy */
  void *dev_meta;
  size_t meta_bytes;
  void *host_out;               /* optional pinned host destination of out */
  size_t out_copy_bytes;        /* <= max_tokens * num_q_heads * head_dim * 2 */
} pa_step_buffers;

typedef struct pa_step_graph pa_step_graph;

/*
 * Validates the buffers (the same checks as the three calls), captures the
 * step on the current device and instantiates it.  On success *graph owns
 * the graph; destroy it with pa_step_graph_destroy.  Nothing runs on the GPU.
 */
int pa_step_graph_create(const pa_step_buffers *buffers, pa_step_graph **graph);

/* Launches the captured step on `stream` (asynchronous). */
int pa_step_graph_launch(pa_step_graph *graph, cudaStream_t stream);

/* Frees the graph (NULL is a no-op).  Launches in flight may finish first. */
int pa_step_graph_destroy(pa_step_graph *graph);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
