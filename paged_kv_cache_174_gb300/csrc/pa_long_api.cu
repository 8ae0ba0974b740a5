// pa_long_api.cu -- the C ABI of the operators for long contexts (declared in
// include/pagedattn.h): argument checks and dispatch.  No device memory is allocated.
#include <climits>

#include "pagedattn.h"
#include "pa_internal.h"

namespace {

using pa::api_fail;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_fail(cudaError_t e, const char* what) {
  return api_fail(PA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// What every call here checks of the cache and of the step's sizes.
int check_step(int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
               int32_t max_blocks, int32_t num_seqs, int32_t num_tokens) {
  if (num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return api_fail(PA_ERR_INVALID_ARG,
                    "cache geometry must be positive (num_blocks=%d block_size=%d "
                    "num_kv_heads=%d head_dim=%d)",
                    num_blocks, block_size, num_kv_heads, head_dim);
  if (num_seqs < 0 || num_tokens < 0 || max_blocks < 0)
    return api_fail(PA_ERR_INVALID_ARG, "negative size argument");
  if (block_size != 16 && block_size != 32)
    return api_fail(PA_ERR_UNSUPPORTED, "block_size %d (16 and 32 are implemented)", block_size);
  if (head_dim != 64 && head_dim != 128)
    return api_fail(PA_ERR_UNSUPPORTED, "head_dim %d (64 and 128 are implemented)", head_dim);
  if (num_kv_heads != 1 && num_kv_heads != 2 && num_kv_heads != 4 && num_kv_heads != 8)
    return api_fail(PA_ERR_UNSUPPORTED, "num_kv_heads %d (1, 2, 4 and 8 are implemented)",
                    num_kv_heads);
  if ((int64_t)num_blocks * block_size > INT32_MAX)
    return api_fail(PA_ERR_UNSUPPORTED, "num_blocks * block_size above 2^31 - 1 token slots");
  if ((int64_t)max_blocks * block_size > INT32_MAX)
    return api_fail(PA_ERR_UNSUPPORTED, "max_blocks * block_size above 2^31 - 1 positions");
  return PA_OK;
}

int check_heads(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (num_q_heads <= 0 || num_q_heads % num_kv_heads != 0)
    return api_fail(PA_ERR_INVALID_ARG,
                    "num_q_heads %d must be a positive multiple of num_kv_heads %d", num_q_heads,
                    num_kv_heads);
  const int group = num_q_heads / num_kv_heads;
  if (!pa::decode_supported(head_dim, group, num_kv_heads))
    return api_fail(PA_ERR_UNSUPPORTED, "shape head_dim=%d group=%d num_kv_heads=%d", head_dim,
                    group, num_kv_heads);
  return PA_OK;
}

// Units times the most CTAs that one gets has to fit a grid.
int check_units(int64_t units) {
  if (units > INT32_MAX / 16)
    return api_fail(PA_ERR_UNSUPPORTED, "%lld (row, kv head) pairs (at most 2^27 - 1)",
                    (long long)units);
  return PA_OK;
}

int log2_of(int block_size) { return block_size == 32 ? 5 : 4; }

constexpr float kLog2E = 1.4426950408889634f;

int summarize_impl(const void* k_cache, bool fp8, int32_t num_blocks, int32_t block_size,
                   int32_t num_kv_heads, int32_t head_dim, const int32_t* block_tables,
                   int32_t max_blocks, const int32_t* seq_lens, const int32_t* query_start_loc,
                   int32_t num_seqs, int32_t num_tokens, int8_t* bounds, float* bound_scales,
                   cudaStream_t stream) {
  int st = check_step(num_blocks, block_size, num_kv_heads, head_dim, max_blocks, num_seqs,
                      num_tokens);
  if (st) return st;
  const int64_t places = query_start_loc ? num_tokens / block_size + 2ll * num_seqs
                                         : (int64_t)num_seqs * max_blocks;
  st = check_units(places * num_kv_heads);
  if (st) return st;
  if (num_seqs == 0 || max_blocks == 0 || (query_start_loc && num_tokens == 0)) return PA_OK;
  if (!k_cache || !block_tables || !seq_lens || !bounds || !bound_scales)
    return api_fail(PA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(bound_scales, 4) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4))
    return api_fail(PA_ERR_INVALID_ARG,
                    "the cache and the bounds must be 16-byte aligned, other arrays 4-byte");
  pa::BoundsArgs a = {};
  a.k_cache = k_cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start_loc = query_start_loc;
  a.bounds = bounds;
  a.scales = bound_scales;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.n_kv = num_kv_heads;
  a.head_dim = head_dim;
  a.block_log2 = log2_of(block_size);
  a.fp8 = fp8;
  int sms = 0;
  st = pa::api_device_state(&a.err, &sms);
  if (st) return st;
  pa::NvtxRange range("bounds of the blocks' keys");
  const cudaError_t e = pa::launch_bounds(a, sms, stream);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "summarize_blocks launch");
}

int sparse_impl(const pa_bf16* q, const void* k_cache, const void* v_cache, bool fp8,
                int32_t num_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                int32_t head_dim, const int32_t* block_tables, int32_t max_blocks,
                const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_seqs,
                int32_t num_tokens, float scale, const int32_t* selected, int32_t num_selected,
                pa_bf16* out, cudaStream_t stream) {
  int st = check_step(num_blocks, block_size, num_kv_heads, head_dim, max_blocks, num_seqs,
                      num_tokens);
  if (st) return st;
  st = check_heads(num_q_heads, num_kv_heads, head_dim);
  if (st) return st;
  if (!(scale == scale)) return api_fail(PA_ERR_INVALID_ARG, "scale is NaN");
  if (num_selected < 1) return api_fail(PA_ERR_INVALID_ARG, "num_selected %d < 1", num_selected);
  if ((int64_t)num_selected * block_size > INT32_MAX / 64)
    return api_fail(PA_ERR_UNSUPPORTED, "num_selected %d", num_selected);
  st = check_units((int64_t)num_tokens * num_kv_heads);
  if (st) return st;
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start_loc || !selected ||
      !out)
    return api_fail(PA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
      !aligned(selected, 4))
    return api_fail(PA_ERR_INVALID_ARG,
                    "q, out and the caches must be 16-byte aligned, int32 arrays 4-byte");
  pa::SparseArgs a = {};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start_loc = query_start_loc;
  a.selected = selected;
  a.out = out;
  a.scale_log2 = scale * kLog2E;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.n_kv = num_kv_heads;
  a.group = num_q_heads / num_kv_heads;
  a.head_dim = head_dim;
  a.block_shift = log2_of(block_size) - 4;
  a.num_selected = num_selected;
  a.fp8 = fp8;
  int sms = 0;
  st = pa::api_device_state(&a.err, &sms);
  if (st) return st;
  pa::NvtxRange range("attention over chosen blocks");
  const cudaError_t e = pa::launch_sparse(a, sms, stream);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "paged_attention_blocks launch");
}

size_t round_up(size_t n) { return (n + 255) & ~size_t(255); }

int weights_impl(const pa_bf16* q, const void* k_cache, const void* v_cache, bool fp8,
                 int32_t num_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                 int32_t head_dim, const int32_t* block_tables, int32_t max_blocks,
                 const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_seqs,
                 int32_t num_tokens, int32_t min_q_len, int32_t max_q_len, int32_t max_seq_len,
                 float scale, float* weights, int32_t weights_len, pa_bf16* out, void* workspace,
                 size_t workspace_bytes, cudaStream_t stream) {
  int st = check_step(num_blocks, block_size, num_kv_heads, head_dim, max_blocks, num_seqs,
                      num_tokens);
  if (st) return st;
  st = check_heads(num_q_heads, num_kv_heads, head_dim);
  if (st) return st;
  if (max_q_len < 0 || max_seq_len < 0 || weights_len < 0)
    return api_fail(PA_ERR_INVALID_ARG, "negative size argument");
  if (max_q_len > max_seq_len)
    return api_fail(PA_ERR_INVALID_ARG, "max_q_len %d > max_seq_len %d", max_q_len, max_seq_len);
  if (min_q_len > max_q_len)
    return api_fail(PA_ERR_INVALID_ARG, "min_q_len %d > max_q_len %d", min_q_len, max_q_len);
  if (!(scale == scale)) return api_fail(PA_ERR_INVALID_ARG, "scale is NaN");
  if (weights_len < max_seq_len)
    return api_fail(PA_ERR_INVALID_ARG, "weights_len %d cannot hold max_seq_len %d", weights_len,
                    max_seq_len);
  if ((int64_t)max_blocks * block_size < max_seq_len && num_seqs > 0)
    return api_fail(PA_ERR_INVALID_ARG, "max_blocks %d * block_size cannot hold max_seq_len %d",
                    max_blocks, max_seq_len);
  st = check_units((int64_t)num_seqs * num_kv_heads);
  if (st) return st;
  if (num_seqs == 0 || num_tokens == 0 || max_seq_len == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start_loc || !weights ||
      !out)
    return api_fail(PA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
      !aligned(weights, 4))
    return api_fail(PA_ERR_INVALID_ARG,
                    "q, out and the caches must be 16-byte aligned, other arrays 4-byte");
  unsigned* err = nullptr;
  int sms = 0;
  st = pa::api_device_state(&err, &sms);
  if (st) return st;
  const int group = num_q_heads / num_kv_heads;
  const int shift = log2_of(block_size) - 4;
  if (max_q_len >= 2) {
    const size_t sums = round_up((size_t)num_tokens * num_q_heads * sizeof(float));
    if (!workspace || !aligned(workspace, 256))
      return api_fail(PA_ERR_WORKSPACE, "workspace must be a non-null 256-byte aligned pointer");
    if (workspace_bytes < sums)
      return api_fail(PA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes,
                      sums);
    // the prefill's key pieces take only what the workspace has left
    const pa::PrefillPlan plan =
        pa::prefill_plan(num_tokens, num_q_heads, num_kv_heads, head_dim, max_q_len, max_seq_len,
                         sms, workspace_bytes - sums);
    pa::AttnArgs a = {};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.fp8 = fp8;
    a.num_blocks = num_blocks;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.query_start_loc = query_start_loc;
    a.num_seqs = num_seqs;
    a.num_tokens = num_tokens;
    a.max_q_len = max_q_len;
    a.max_seq_len = max_seq_len;
    a.block_shift = shift;
    a.scale = scale;
    a.out = out;
    a.err = err;
    a.no_decode = min_q_len >= 2;
    a.min_q_len = min_q_len;
    pa::NvtxRange range("prefill (tcgen05) + accumulated weights of its rows");
    cudaError_t e =
        pa::launch_prefill(a, plan, static_cast<unsigned char*>(workspace) + sums, sms, stream);
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
    pa::ChunkArgs c = {};
    c.q = q;
    c.k_cache = k_cache;
    c.block_tables = block_tables;
    c.seq_lens = seq_lens;
    c.query_start_loc = query_start_loc;
    c.weights = weights;
    c.sums = static_cast<float*>(workspace);
    c.err = err;
    c.weights_stride = weights_len;
    c.scale_log2 = scale * kLog2E;
    c.num_blocks = num_blocks;
    c.max_blocks = max_blocks;
    c.num_seqs = num_seqs;
    c.num_tokens = num_tokens;
    c.n_q = num_q_heads;
    c.n_kv = num_kv_heads;
    c.group = group;
    c.head_dim = head_dim;
    c.block_shift = shift;
    c.max_seq_len = max_seq_len;
    c.fp8 = fp8;
    e = pa::launch_chunk_weights(c, max_q_len, sms, stream);
    if (e != cudaSuccess) return cuda_fail(e, "accumulated weights launch");
  }
  if (min_q_len >= 2) return PA_OK;  // no request has a single query row
  pa::WeighArgs w = {};
  w.q = q;
  w.k_cache = k_cache;
  w.v_cache = v_cache;
  w.block_tables = block_tables;
  w.seq_lens = seq_lens;
  w.query_start_loc = query_start_loc;
  w.weights = weights;
  w.out = out;
  w.err = err;
  w.weights_stride = weights_len;
  w.scale_log2 = scale * kLog2E;
  w.num_blocks = num_blocks;
  w.max_blocks = max_blocks;
  w.num_seqs = num_seqs;
  w.num_tokens = num_tokens;
  w.n_kv = num_kv_heads;
  w.group = group;
  w.head_dim = head_dim;
  w.block_shift = shift;
  w.max_seq_len = max_seq_len;
  w.chunks = max_q_len >= 2;
  w.fp8 = fp8;
  pa::NvtxRange range("weighing decode");
  const cudaError_t e = pa::launch_weigh(w, sms, stream);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "weighing decode launch");
}

int evict_impl(void* k_cache, void* v_cache, bool fp8, float* weights, int32_t weights_len,
               int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
               const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
               const int32_t* budgets, int32_t num_seqs, int32_t max_seq_len, int32_t num_sinks,
               int32_t num_recent, int32_t* free_blocks, const int32_t* free_count,
               int32_t* seq_lens_out, int32_t* free_count_out, int32_t* position_offsets,
               cudaStream_t stream) {
  int st = check_step(num_blocks, block_size, num_kv_heads, head_dim, max_blocks, num_seqs, 0);
  if (st) return st;
  if (weights_len < 0 || max_seq_len < 0)
    return api_fail(PA_ERR_INVALID_ARG, "negative size argument");
  if (num_sinks < 0 || num_recent < 0 || (int64_t)num_sinks + num_recent > INT32_MAX)
    return api_fail(PA_ERR_INVALID_ARG, "num_sinks %d, num_recent %d", num_sinks, num_recent);
  if (weights_len < max_seq_len)
    return api_fail(PA_ERR_INVALID_ARG, "weights_len %d cannot hold max_seq_len %d", weights_len,
                    max_seq_len);
  if (max_seq_len > pa::kEvictMaxLen)
    return api_fail(PA_ERR_UNSUPPORTED, "max_seq_len %d (at most %d)", max_seq_len,
                    pa::kEvictMaxLen);
  if ((int64_t)num_seqs * num_kv_heads > INT32_MAX / 8 - 1) return check_units(INT64_MAX);
  if (!free_blocks || !free_count || !free_count_out ||
      (num_seqs > 0 && (!k_cache || !v_cache || !weights || !block_tables || !seq_lens ||
                        !budgets || !seq_lens_out)))
    return api_fail(PA_ERR_INVALID_ARG, "null pointer argument");
  const void* words[] = {weights,    block_tables, seq_lens,       budgets,         free_blocks,
                         free_count, seq_lens_out, free_count_out, position_offsets};
  for (const void* x : words)
    if (!aligned(x, 4))
      return api_fail(PA_ERR_INVALID_ARG, "the weights and int32 arrays must be 4-byte aligned");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16))
    return api_fail(PA_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  pa::EvictArgs a = {};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.weights = weights;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.budgets = budgets;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.seq_lens_out = seq_lens_out;
  a.free_count_out = free_count_out;
  a.position_offsets = position_offsets;
  a.weights_stride = weights_len;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.num_seqs = num_seqs;
  a.n_kv = num_kv_heads;
  a.head_dim = head_dim;
  a.block_log2 = log2_of(block_size);
  a.num_sinks = num_sinks;
  a.num_recent = num_recent;
  a.max_seq_len = max_seq_len;
  a.fp8 = fp8;
  int sms = 0;
  st = pa::api_device_state(&a.err, &sms);
  if (st) return st;
  pa::NvtxRange range("eviction (choice, compaction, blocks returned)");
  const cudaError_t e = pa::launch_evict(a, sms, stream);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "evict_tokens launch");
}

}  // namespace

extern "C" {

int pa_summarize_blocks(const pa_bf16* k_cache, int32_t num_blocks, int32_t block_size,
                        int32_t num_kv_heads, int32_t head_dim, const int32_t* block_tables,
                        int32_t max_blocks, const int32_t* seq_lens,
                        const int32_t* query_start_loc, int32_t num_seqs, int32_t num_tokens,
                        int8_t* bounds, float* bound_scales, cudaStream_t stream) {
  return summarize_impl(k_cache, false, num_blocks, block_size, num_kv_heads, head_dim,
                        block_tables, max_blocks, seq_lens, query_start_loc, num_seqs, num_tokens,
                        bounds, bound_scales, stream);
}
int pa_summarize_blocks_fp8(const uint8_t* k_cache, int32_t num_blocks, int32_t block_size,
                            int32_t num_kv_heads, int32_t head_dim, const int32_t* block_tables,
                            int32_t max_blocks, const int32_t* seq_lens,
                            const int32_t* query_start_loc, int32_t num_seqs, int32_t num_tokens,
                            int8_t* bounds, float* bound_scales, cudaStream_t stream) {
  return summarize_impl(k_cache, true, num_blocks, block_size, num_kv_heads, head_dim,
                        block_tables, max_blocks, seq_lens, query_start_loc, num_seqs, num_tokens,
                        bounds, bound_scales, stream);
}

int pa_select_blocks(const pa_bf16* q, const int8_t* bounds, const float* bound_scales,
                     int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t head_dim, const int32_t* block_tables,
                     int32_t max_blocks, const int32_t* seq_lens, const int32_t* query_start_loc,
                     int32_t num_seqs, int32_t num_tokens, int32_t max_seq_len,
                     int32_t num_selected, int32_t num_sinks, int32_t num_recent,
                     int32_t* selected, cudaStream_t stream) {
  int st = check_step(num_blocks, block_size, num_kv_heads, head_dim, max_blocks, num_seqs,
                      num_tokens);
  if (st) return st;
  st = check_heads(num_q_heads, num_kv_heads, head_dim);
  if (st) return st;
  if (max_seq_len < 0) return api_fail(PA_ERR_INVALID_ARG, "negative size argument");
  if (num_sinks < 0 || num_recent < 1)
    return api_fail(PA_ERR_INVALID_ARG, "num_sinks %d (at least 0), num_recent %d (at least 1)",
                    num_sinks, num_recent);
  if ((int64_t)num_sinks + num_recent > num_selected)
    return api_fail(PA_ERR_INVALID_ARG, "num_selected %d holds no %d first and %d last blocks",
                    num_selected, num_sinks, num_recent);
  st = check_units((int64_t)num_tokens * num_kv_heads);
  if (st) return st;
  if ((int64_t)max_seq_len > (int64_t)pa::kSelectMaxBlocks * block_size)
    return api_fail(PA_ERR_UNSUPPORTED, "max_seq_len %d (at most %d blocks)", max_seq_len,
                    pa::kSelectMaxBlocks);
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!q || !bounds || !bound_scales || !block_tables || !seq_lens || !query_start_loc ||
      !selected)
    return api_fail(PA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(bound_scales, 4) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
      !aligned(selected, 4))
    return api_fail(PA_ERR_INVALID_ARG,
                    "q and the bounds must be 16-byte aligned, other arrays 4-byte");
  pa::SelectArgs a = {};
  a.q = q;
  a.bounds = bounds;
  a.scales = bound_scales;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start_loc = query_start_loc;
  a.selected = selected;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.n_kv = num_kv_heads;
  a.group = num_q_heads / num_kv_heads;
  a.head_dim = head_dim;
  a.block_log2 = log2_of(block_size);
  a.num_selected = num_selected;
  a.num_sinks = num_sinks;
  a.num_recent = num_recent;
  a.max_seq_len = max_seq_len;
  int sms = 0;
  st = pa::api_device_state(&a.err, &sms);
  if (st) return st;
  pa::NvtxRange range("choice of blocks");
  const cudaError_t e = pa::launch_select(a, sms, stream);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "select_blocks launch");
}

int pa_paged_attention_blocks(const pa_bf16* q, const pa_bf16* k_cache, const pa_bf16* v_cache,
                              int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, const int32_t* block_tables,
                              int32_t max_blocks, const int32_t* seq_lens,
                              const int32_t* query_start_loc, int32_t num_seqs,
                              int32_t num_tokens, float scale, const int32_t* selected,
                              int32_t num_selected, pa_bf16* out, cudaStream_t stream) {
  return sparse_impl(q, k_cache, v_cache, false, num_blocks, block_size, num_q_heads,
                     num_kv_heads, head_dim, block_tables, max_blocks, seq_lens, query_start_loc,
                     num_seqs, num_tokens, scale, selected, num_selected, out, stream);
}
int pa_paged_attention_blocks_fp8(const pa_bf16* q, const uint8_t* k_cache,
                                  const uint8_t* v_cache, int32_t num_blocks, int32_t block_size,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  const int32_t* block_tables, int32_t max_blocks,
                                  const int32_t* seq_lens, const int32_t* query_start_loc,
                                  int32_t num_seqs, int32_t num_tokens, float scale,
                                  const int32_t* selected, int32_t num_selected, pa_bf16* out,
                                  cudaStream_t stream) {
  return sparse_impl(q, k_cache, v_cache, true, num_blocks, block_size, num_q_heads, num_kv_heads,
                     head_dim, block_tables, max_blocks, seq_lens, query_start_loc, num_seqs,
                     num_tokens, scale, selected, num_selected, out, stream);
}

size_t pa_weights_workspace_size(int32_t num_seqs, int32_t num_tokens, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t max_q_len,
                                 int32_t max_seq_len) {
  if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_q_len < 0 || max_seq_len < 0 || num_q_heads % num_kv_heads != 0)
    return 0;
  if (!pa::decode_supported(head_dim, num_q_heads / num_kv_heads, num_kv_heads)) return 0;
  int sms = 0;
  if (pa::api_device_state(nullptr, &sms)) return 0;
  if (max_q_len < 2) return 256;
  const size_t sums = (size_t)num_tokens * num_q_heads * sizeof(float);
  return round_up(sums + 256) +
         round_up(pa::prefill_workspace_bound(num_tokens, num_q_heads, num_kv_heads, head_dim,
                                              max_q_len, max_seq_len, sms));
}

int pa_paged_attention_weights(const pa_bf16* q, const pa_bf16* k_cache, const pa_bf16* v_cache,
                               int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim,
                               const int32_t* block_tables, int32_t max_blocks,
                               const int32_t* seq_lens, const int32_t* query_start_loc,
                               int32_t num_seqs, int32_t num_tokens, int32_t min_q_len,
                               int32_t max_q_len, int32_t max_seq_len, float scale,
                               float* weights, int32_t weights_len, pa_bf16* out, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
  return weights_impl(q, k_cache, v_cache, false, num_blocks, block_size, num_q_heads,
                      num_kv_heads, head_dim, block_tables, max_blocks, seq_lens, query_start_loc,
                      num_seqs, num_tokens, min_q_len, max_q_len, max_seq_len, scale, weights,
                      weights_len, out, workspace, workspace_bytes, stream);
}
int pa_paged_attention_weights_fp8(const pa_bf16* q, const uint8_t* k_cache,
                                   const uint8_t* v_cache, int32_t num_blocks, int32_t block_size,
                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                   const int32_t* block_tables, int32_t max_blocks,
                                   const int32_t* seq_lens, const int32_t* query_start_loc,
                                   int32_t num_seqs, int32_t num_tokens, int32_t min_q_len,
                                   int32_t max_q_len, int32_t max_seq_len, float scale,
                                   float* weights, int32_t weights_len, pa_bf16* out,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return weights_impl(q, k_cache, v_cache, true, num_blocks, block_size, num_q_heads,
                      num_kv_heads, head_dim, block_tables, max_blocks, seq_lens, query_start_loc,
                      num_seqs, num_tokens, min_q_len, max_q_len, max_seq_len, scale, weights,
                      weights_len, out, workspace, workspace_bytes, stream);
}

int pa_evict_tokens(pa_bf16* k_cache, pa_bf16* v_cache, float* weights, int32_t weights_len,
                    int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                    int32_t head_dim, const int32_t* block_tables, int32_t max_blocks,
                    const int32_t* seq_lens, const int32_t* budgets, int32_t num_seqs,
                    int32_t max_seq_len, int32_t num_sinks, int32_t num_recent,
                    int32_t* free_blocks, const int32_t* free_count, int32_t* seq_lens_out,
                    int32_t* free_count_out, int32_t* position_offsets, cudaStream_t stream) {
  return evict_impl(k_cache, v_cache, false, weights, weights_len, num_blocks, block_size,
                    num_kv_heads, head_dim, block_tables, max_blocks, seq_lens, budgets, num_seqs,
                    max_seq_len, num_sinks, num_recent, free_blocks, free_count, seq_lens_out,
                    free_count_out, position_offsets, stream);
}
int pa_evict_tokens_fp8(uint8_t* k_cache, uint8_t* v_cache, float* weights, int32_t weights_len,
                        int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                        int32_t head_dim, const int32_t* block_tables, int32_t max_blocks,
                        const int32_t* seq_lens, const int32_t* budgets, int32_t num_seqs,
                        int32_t max_seq_len, int32_t num_sinks, int32_t num_recent,
                        int32_t* free_blocks, const int32_t* free_count, int32_t* seq_lens_out,
                        int32_t* free_count_out, int32_t* position_offsets,
                        cudaStream_t stream) {
  return evict_impl(k_cache, v_cache, true, weights, weights_len, num_blocks, block_size,
                    num_kv_heads, head_dim, block_tables, max_blocks, seq_lens, budgets, num_seqs,
                    max_seq_len, num_sinks, num_recent, free_blocks, free_count, seq_lens_out,
                    free_count_out, position_offsets, stream);
}

}  // extern "C"
