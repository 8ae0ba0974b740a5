// pa_internal.h -- host-side interfaces between the C-ABI layer (pa_api.cu)
// and the kernel translation units.  Not installed; not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

namespace pa {

// A named NVTX range over a scope of host code (the launches of one call), so
// that a profiler groups each kernel under the library call that issued it.
// NVTX is header-only: with no tool attached a push or pop is a test of a
// function pointer and nothing else.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Launches a kernel that may be scheduled while the one before it on the stream
// finishes (programmatic dependent launch); the kernel has to call
// after_prior_kernels() (pa_common.cuh) before it reads anything.  It saves most
// of the gap between two launches.
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, unsigned cluster, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Bits of the device error word (read back by pa_check_device_errors).
enum : unsigned {
  DEVERR_BOUNDS = 1u,   // an index / length was out of range; work skipped
  DEVERR_TIMEOUT = 2u,  // a bounded wait gave up
};

// 8-bit cache page: the codes of 16 token rows ([16, n_kv, head_dim] bytes),
// then their fp32 scales ([16, n_kv]); a block holds block_size / 16 pages.
constexpr int kFp8PageTokens = 16;
__host__ __device__ constexpr int64_t fp8_page_bytes(int n_kv, int head_dim) {
  return (int64_t)kFp8PageTokens * n_kv * (head_dim + 4);
}
__host__ __device__ constexpr int64_t fp8_scales_offset(int n_kv, int head_dim) {
  return (int64_t)kFp8PageTokens * n_kv * head_dim;
}

// Geometry and pointers of one paged-attention call, already validated.
struct AttnArgs {
  const uint16_t* q;
  const void* k_cache;     // bf16 values, or (fp8) pages of E4M3 codes and row scales
  const void* v_cache;
  bool fp8;
  // Fused scatter (decode-only steps over the bf16 cache): the decode kernel
  // takes each decode request's new row from these and stores it to its
  // slot; all null when the scatter ran as its own kernel.
  const uint16_t* fuse_k_new;
  const uint16_t* fuse_v_new;
  const int32_t* fuse_slot_mapping;
  int32_t num_blocks;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  const int32_t* block_tables;
  int32_t max_blocks;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t max_q_len;
  int32_t max_seq_len;
  // log2(block_size / 16): the kernels walk 16-token pages, and page j of a
  // request lives in block block_tables[j >> block_shift], 16-token half
  // (j & ((1 << block_shift) - 1)) of it
  int32_t block_shift;
  float scale;
  uint16_t* out;
  unsigned* err;  // device error word
  // The kernel launched just before on the stream is the prefill kernel
  // (which triggers its dependents at once and writes only prefill rows):
  // the decode kernel may then start on SMs it leaves free.
  bool after_prefill;
  int32_t min_q_len;  // the caller's promise (0 or 1: none)
  // Sliding window (0: none): position p attends to positions above p - window
  // and to the first num_sinks ones.
  int32_t window;
  int32_t num_sinks;
  // The caller promised that no request has exactly one query row: the
  // decode kernel is not launched, and the prefill kernel flags a request
  // with one row as a bounds error instead of leaving its row unwritten.
  bool no_decode;
};

// Workspace carve-up shared by the launchers (sizes in bytes, 256-aligned).
struct DecodeWorkspace {
  float* part_o;    // [ctas * 2, num_q_heads, head_dim]
  float* part_ml;   // [ctas * 2, num_q_heads, 2]  (running max in log2 units, sum)
  int4* seq_rec;    // [num_seqs]
};

size_t decode_workspace_bytes(int ctas, int num_seqs, int num_q_heads, int head_dim);
DecodeWorkspace decode_workspace(void* base, int ctas, int num_seqs, int num_q_heads,
                                 int head_dim);
int decode_ctas(int sm_count);

// Each launcher returns cudaSuccess or the launch error.  Unsupported shapes
// are rejected by the API layer before these are called.
bool decode_supported(int head_dim, int group, int num_kv_heads);
cudaError_t launch_decode(const AttnArgs& a, const DecodeWorkspace& ws, int ctas,
                          cudaStream_t stream);
cudaError_t launch_decode_fp8(const AttnArgs& a, const DecodeWorkspace& ws, int ctas,
                              cudaStream_t stream);
cudaError_t launch_decode_fused(const AttnArgs& a, const DecodeWorkspace& ws, int ctas,
                                cudaStream_t stream);

cudaError_t launch_decode_window(const AttnArgs& a, const DecodeWorkspace& ws, int ctas,
                                 cudaStream_t stream);
cudaError_t launch_decode_window_fp8(const AttnArgs& a, const DecodeWorkspace& ws, int ctas,
                                     cudaStream_t stream);

bool prefill_supported(int head_dim, int group, int num_kv_heads);
// How the prefill kernel splits the keys of each query-tile pair, and the
// workspace bytes the pieces take (0 when nsplit == 1).
struct PrefillPlan {
  int nsplit;
  size_t bytes;
};
PrefillPlan prefill_plan(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                         int max_q_len, int max_seq_len, int sm_count, size_t max_bytes);
// The most bytes any call with at most num_tokens tokens (and these bounds)
// would use for key pieces.
size_t prefill_workspace_bound(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                               int max_q_len, int max_seq_len, int sm_count);
cudaError_t launch_prefill(const AttnArgs& a, const PrefillPlan& plan, void* ws, int sm_count,
                           cudaStream_t stream);

cudaError_t launch_reshape_and_cache(const uint16_t* k, const uint16_t* v, int32_t num_tokens,
                                     uint16_t* k_cache, uint16_t* v_cache, int64_t num_slots,
                                     int32_t row_elems, const int32_t* slot_mapping,
                                     unsigned* err, cudaStream_t stream);

cudaError_t launch_reshape_and_cache_fp8(const uint16_t* k, const uint16_t* v,
                                         int32_t num_tokens, uint8_t* k_cache, uint8_t* v_cache,
                                         int64_t num_slots, int32_t num_kv_heads,
                                         int32_t head_dim, const int32_t* slot_mapping,
                                         unsigned* err, cudaStream_t stream);
cudaError_t launch_copy_blocks(uint16_t* k_cache, uint16_t* v_cache, int32_t num_blocks,
                               int64_t block_elems, const int32_t* pairs, int32_t num_pairs,
                               unsigned* err, cudaStream_t stream);

// Block swap through a device staging buffer of 2 * n * block_elems values:
// out = true packs the blocks and copies them to host_k / host_v; out = false
// copies host_k / host_v in and unpacks them into the cache.
cudaError_t launch_swap(uint16_t* k_cache, uint16_t* v_cache, int32_t num_blocks,
                        int64_t block_elems, const int32_t* ids, int32_t n, uint16_t* staging,
                        uint16_t* host_k, uint16_t* host_v, bool out, unsigned* err,
                        cudaStream_t stream);

// Whether units of two query tiles of tile_rows tokens each finish sooner than units
// of one, where one with two takes cost times as long: whether halving the number
// of units saves enough rounds over the SMs.  The host knows the call's rows, its
// requests and their fewest and most rows, and takes the rows past each request's
// fewest to be those of as few requests of max_q_len rows as hold them (requests of
// one row are decoded elsewhere).  Requests within one tile never have a second one
// to share a unit with.
inline bool pairs_finish_sooner(int num_tokens, int num_seqs, int min_q_len, int max_q_len,
                                int tile_rows, int num_kv_heads, int sm_count, double cost) {
  const long long fewest = min_q_len > 1 ? min_q_len : 1;
  const long long rows = num_tokens - num_seqs * fewest, span = max_q_len - fewest;
  if (max_q_len <= tile_rows || rows < 0 || span < 0) return false;
  const long long whole = span ? rows / span : 0, rest = span ? rows % span : 0;
  const long long others = num_seqs - whole - (rest ? 1 : 0);
  const auto rounds = [&](long long unit_rows) {
    const auto tiles = [&](long long n) { return n > 1 ? (n + unit_rows - 1) / unit_rows : 0; };
    const long long units = whole * tiles(max_q_len) + (rest ? tiles(rest + fewest) : 0) +
                            (others > 0 ? others * tiles(fewest) : 0);
    return (double)((units * num_kv_heads + sm_count - 1) / sm_count);
  };
  return rounds(2 * tile_rows) * cost < rounds(tile_rows);
}

// A step's integer inputs from the requests' lengths (pa_step.cu).
struct StepPlanArgs {
  const int32_t* context_lens;      // [num_seqs]
  const int32_t* new_lens;          // [num_seqs]
  const int32_t* position_offsets;  // [num_seqs] or null
  int32_t* block_tables;            // [num_seqs, max_blocks]
  const int32_t* free_blocks;       // [num_blocks], the last free_count on top
  const int32_t* free_count;        // [1]
  int32_t* free_count_out;          // [1]
  int32_t* seq_lens;                // [num_seqs]
  int32_t* query_start_loc;         // [num_seqs + 1]
  int32_t* slot_mapping;            // [num_tokens]
  int32_t* positions;               // [num_axes, num_tokens]
  unsigned* err;
  int32_t num_seqs, num_tokens, num_axes, max_blocks, block_size, num_blocks;
};
constexpr int kMaxPlanSeqs = 16384;  // three words of shared memory each
cudaError_t launch_build_step(const StepPlanArgs& p, cudaStream_t stream);

constexpr int kMaxRotaryAxes = 4;

// Rotary positions on q and k with the slot scatter of k and v (pa_rotary.cu).
struct RotaryArgs {
  const uint16_t* q;  // token rows at these strides (elements), heads contiguous
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* positions;  // [num_axes] rows at positions_stride
  int64_t positions_stride;
  const double* inv_freq;  // [rotary_dim / 2]
  const int32_t* axes;     // [rotary_dim / 2] or null (axis 0)
  const int32_t* slot_mapping;
  uint16_t* q_out;  // [num_tokens, n_q, head_dim]
  void* k_cache;    // bf16 values, or (fp8) pages of E4M3 codes and row scales
  void* v_cache;
  unsigned* err;
  int64_t num_slots;
  int32_t num_tokens, n_q, n_kv, head_dim, rotary_dim, num_axes;
  bool interleaved;
  bool fp8;
};
cudaError_t launch_rotary_cache(const RotaryArgs& p, cudaStream_t stream);

// Bounds of the blocks' keys (pa_blocks.cu).
struct BoundsArgs {
  const void* k_cache;  // bf16 values, or (fp8) pages of E4M3 codes and row scales
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;  // or null: every block of every request
  int8_t* bounds;                  // [num_blocks, n_kv, 2, head_dim]
  float* scales;                   // [num_blocks, n_kv]
  unsigned* err;
  long long slots;  // (set by the launcher) places for a (request, block)
  int32_t heads;    // (set by the launcher) kv heads that a warp takes in turn
  int32_t num_blocks, max_blocks, num_seqs, num_tokens, n_kv, head_dim, block_log2;
  bool fp8;
};
cudaError_t launch_bounds(BoundsArgs p, int sm_count, cudaStream_t stream);

// The blocks that each query attends to (pa_blocks.cu).
struct SelectArgs {
  const uint16_t* q;
  const int8_t* bounds;
  const float* scales;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  int32_t* selected;  // [num_tokens, n_kv, num_selected]
  unsigned* err;
  int32_t num_blocks, max_blocks, num_seqs, num_tokens, n_kv, group, head_dim, block_log2;
  int32_t num_selected, num_sinks, num_recent, max_seq_len;
  int32_t max_keys;  // (set by the launcher) blocks of max_seq_len
};
// Blocks of a request: a key each in shared memory, and an eighth of the table.
constexpr int kSelectMaxBlocks = 48 * 1024;
constexpr int kSelectSmem = kSelectMaxBlocks / 8 * 9 * 4;
cudaError_t launch_select(SelectArgs p, int sm_count, cudaStream_t stream);

// Attention over chosen blocks (pa_sparse.cu).
struct SparseArgs {
  const uint16_t* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  const int32_t* selected;  // [num_tokens, n_kv, num_selected]
  uint16_t* out;
  unsigned* err;
  float scale_log2;
  int32_t num_blocks, max_blocks, num_seqs, num_tokens, n_kv, group, head_dim;
  int32_t block_shift;  // log2(block_size / 16)
  int32_t num_selected;
  bool fp8;
};
cudaError_t launch_sparse(const SparseArgs& p, int sm_count, cudaStream_t stream);

// Decode attention that adds the weights up (pa_weights.cu).
struct WeighArgs {
  const uint16_t* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  float* weights;  // [num_seqs, n_kv, weights_stride]
  uint16_t* out;
  unsigned* err;
  int64_t weights_stride;
  float scale_log2;
  int32_t num_blocks, max_blocks, num_seqs, num_tokens, n_kv, group, head_dim;
  int32_t block_shift;  // log2(block_size / 16)
  int32_t max_seq_len;
  int32_t kept_pages;  // (set by the launcher) pages of a CTA whose scores are kept
  bool chunks;         // requests with more than one row are taken elsewhere
  bool fp8;
};
cudaError_t launch_weigh(const WeighArgs& p, int sm_count, cudaStream_t stream);

// Accumulated weights of chunks (pa_weights_chunk.cu).
struct ChunkArgs {
  const uint16_t* q;
  const void* k_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  float* weights;
  float* sums;  // [n_kv, num_tokens, group] log2 of each row's sum of exponentials
  unsigned* err;
  int64_t weights_stride;
  float scale_log2;
  int32_t num_blocks, max_blocks, num_seqs, num_tokens, n_q, n_kv, group, head_dim;
  int32_t block_shift, max_seq_len;
  int32_t skip;  // (set by the launcher) chunk requests of earlier launches
  bool fp8;
};
cudaError_t launch_chunk_weights(const ChunkArgs& p, int max_q_len, int sm_count,
                                 cudaStream_t stream);

// Eviction by accumulated weight (pa_evict.cu).
struct EvictArgs {
  void* k_cache;
  void* v_cache;
  float* weights;  // [num_seqs, n_kv, weights_stride]
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* budgets;
  int32_t* free_blocks;
  const int32_t* free_count;
  int32_t* seq_lens_out;
  int32_t* free_count_out;
  int32_t* position_offsets;  // or null
  unsigned* err;
  int64_t weights_stride;
  int32_t num_blocks, max_blocks, num_seqs, n_kv, head_dim, block_log2;
  int32_t num_sinks, num_recent, max_seq_len;
  bool fp8;
  bool staged;  // (set by the launcher) the weights' keys fit in shared memory
};
constexpr int kEvictMaxLen = 1 << 19;          // two bits a token in shared memory
cudaError_t launch_evict(EvictArgs p, int sm_count, cudaStream_t stream);

cudaError_t launch_wait_timeout_selftest(unsigned long long limit_ns, unsigned* err,
                                         cudaStream_t stream);

// Error reporting of the C ABI (sets the message pa_get_last_error returns)
// and the per-device state lookup, for the parts of the ABI outside pa_api.cu.
int api_fail(int status, const char* fmt, ...);
int api_warm_device();
// The current device's error word and SM count.
int api_device_state(unsigned** err, int* sms);

}  // namespace pa
