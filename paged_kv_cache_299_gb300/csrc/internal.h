// Host-side launchers shared between the C-ABI entry points (api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pagedkv.h"

namespace pkv {

constexpr int kMaxDevices = 64;  // devices whose kernel attributes are remembered as set

cudaError_t launch_slot_mapping(const int32_t* block_tables, int32_t max_blocks_per_seq,
                                const int32_t* context_lens, const int32_t* query_start_loc,
                                int32_t num_seqs, int32_t num_tokens, int32_t num_blocks,
                                int64_t* slot_mapping, int32_t* status, cudaStream_t stream);

cudaError_t launch_reshape_and_cache(const void* key, const void* value,
                                     const int64_t* slot_mapping, int32_t num_tokens,
                                     void* key_cache, void* value_cache, int32_t num_blocks,
                                     int32_t num_kv_heads, int32_t* status,
                                     cudaStream_t stream);

cudaError_t launch_wait_timeout_selftest(int32_t* status, int32_t limit_ms, cudaStream_t stream);
cudaError_t launch_stream_read(const void* buf, size_t bytes, uint32_t* x, cudaStream_t stream);

cudaError_t launch_copy_blocks(void* key_cache, void* value_cache, const int64_t* block_mapping,
                               int32_t num_pairs, int32_t num_blocks, int32_t num_kv_heads,
                               int32_t* status, cudaStream_t stream);

cudaError_t launch_copy_blocks_q8(void* key_cache, void* value_cache, float* key_scale,
                                  float* value_scale, const int64_t* block_mapping,
                                  int32_t num_pairs, int32_t num_blocks, int32_t num_kv_heads,
                                  int32_t* status, cudaStream_t stream);

// Rotating appends (pa_rope_append, pa_rope_append_q8).  Strides are elements from one
// token's rows to the next one's.
struct AppendArgs {
  const void* q;  // null with num_q_heads == 0
  void* q_out;
  const void* key;
  const void* value;
  int64_t q_stride, q_out_stride, key_stride, value_stride;
  const float* cos_sin;  // [max_positions][64]: 32 cosines, then 32 sines; null: no rotation
  int32_t max_positions;
  bool interleaved;
  const int32_t* positions;  // [num_axes][num_tokens] rows of cos_sin; null: the slots' positions
  int32_t num_axes;          // 1 .. 4
  uint64_t pair_axes;        // two bits per pair: its axis
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  const int32_t* query_start_loc;  // null: one token per sequence
  int32_t num_seqs, num_tokens, num_q_heads, num_kv_heads, num_blocks;
  void* key_cache;
  void* value_cache;
  float* key_scale;  // 8-bit pools only
  float* value_scale;
  int32_t* status;
};

cudaError_t launch_rope_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_rope_append_q8(const AppendArgs& a, cudaStream_t stream);

// Compaction of kept tokens (pa_compact_tokens, pa_compact_tokens_q8).
struct CompactArgs {
  const int32_t* kept;  // rising offsets from first[s]
  const int32_t* kept_start_loc;
  const int32_t* first;
  int32_t num_kept, max_kept, num_seqs;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  int32_t num_blocks, num_kv_heads;
  void* key_cache;
  void* value_cache;
  float* key_scale;  // 8-bit pools only
  float* value_scale;
  int32_t* status;
};

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream);
cudaError_t launch_compact_q8(const CompactArgs& a, cudaStream_t stream);

// Attention of drafted trees (pa_tree_attention, pa_tree_attention_q8).
struct TreeArgs {
  void* out;
  const void* q;
  const int32_t* tree_mask;  // [num_query_tokens][mask_words] bits
  int32_t mask_words;
  const int32_t* query_start_loc;
  int32_t num_query_tokens;
  int32_t max_query_len;
  const void* key_cache;
  const void* value_cache;
  const float* key_scale;  // 8-bit pools only
  const float* value_scale;
  int32_t num_blocks, num_kv_heads, num_q_heads;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  int32_t num_seqs;
  float scale;
  void* workspace;
  int32_t* status;
};

size_t tree_workspace_size();  // on the current device; 0 without one
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream);
cudaError_t launch_tree_q8(const TreeArgs& a, cudaStream_t stream);

// Attention over the 8-bit pools: rows of q are either one per sequence (query_start_loc
// null) or causal chunks.
struct AttendQ8Args {
  void* out;
  const void* q;
  const int32_t* query_start_loc;
  int32_t num_query_tokens;
  int32_t max_query_len;
  int32_t max_context_len;  // the decode's alone
  const void* key_cache;
  const void* value_cache;
  const float* key_scale;
  const float* value_scale;
  int32_t num_blocks, num_kv_heads, num_q_heads;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  int32_t num_seqs;
  float scale;
  int32_t* status;
  const int32_t* tree_mask = nullptr;  // few rows: those of drafted trees, [num_query_tokens][mask_words]
  int32_t mask_words = 0;
};

cudaError_t launch_prefill_q8(const AttendQ8Args& a, cudaStream_t stream);
// Its form for chunks of a few rows (at most 32 per K/V head), and whether a call is one.
bool rows_q8_takes(const AttendQ8Args& a);
int rows_q8_cluster(const AttendQ8Args& a, int sms);  // CTAs that share a (sequence, K/V head)
cudaError_t launch_rows_q8(const AttendQ8Args& a, cudaStream_t stream);

// Work decomposition of one pa_decode call (identical in the size query and the call).
struct DecodePlan {
  int group;          // q heads per kv head
  int grid;           // CTAs of the attention kernel (persistent, <= resident capacity)
  int runs;           // units of the tile decomposition; CTA c serves runs c, c + grid, ...
  int chunk;          // tiles per run (fixed mode), 0 = balanced split of the real total
  int64_t tile_bound; // > 0: host upper bound of the tile count, checked on the device
  size_t smem_bytes;  // dynamic shared memory of the attention kernel
  bool fused_merge;          // split segments merged inside the attention kernel
  bool merge_split_heads;    // otherwise: the merge kernel takes one CTA per query head
  bool prefetch_ok;          // warps may ask L2 for tiles past their ring before the wait
  size_t ws_count_offset;    // offset of the piece counters (must start zeroed)
  size_t ws_meta_bytes;      // offset of the partials inside the workspace
  size_t workspace_bytes;    // total workspace
};

// Returns cudaSuccess and fills `plan`, or an error (e.g. no device).
// max_sms > 0 confines the persistent grid to that many SMs (the rest stay free for a
// kernel launched beside it).
cudaError_t plan_decode(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads,
                        int32_t max_context_len, int32_t partition_tokens, DecodePlan* plan,
                        int32_t max_sms = 0);

// The same for pa_decode_q8.
cudaError_t plan_decode_q8(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads,
                           int32_t max_context_len, DecodePlan* plan, int32_t max_sms = 0);
cudaError_t launch_decode_q8(const AttendQ8Args& a, const DecodePlan& plan, void* workspace,
                             bool overlap_previous, cudaStream_t stream);

struct DecodeArgs {
  void* out;
  const void* q;
  const void* key_cache;
  const void* value_cache;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t num_blocks;
  float scale;
  void* workspace;
  int32_t* status;
  const void* k_new = nullptr;  // fused append (pa_decode_append), else null
  const void* v_new = nullptr;
  const int32_t* q_rows = nullptr;  // mixed batch: query/output row per sequence (prefix sums
                                    // of q_len); only q_len == 1 sequences are served
  int32_t num_query_tokens = 0;
  // Programmatic dependent launch: the kernel may start before the previous kernel in the
  // stream has finished; it reads block_tables, context_lens (and q_rows) and its first
  // K/V tiles before waiting for that kernel, everything else after.
  bool overlap_previous = false;
};

cudaError_t launch_decode(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);

// Tensor map of a [rows][64] bf16 array read in boxes of `box_rows` rows with the 128-byte
// swizzle (the K/V pools, rows = blocks x kv heads x 16); false if the driver call fails.
bool encode_pool_rows(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows);

// Tensor map of q [tokens][heads][64] in boxes of box_tokens x box_heads rows, 128-byte swizzle.
bool encode_query_tiles(CUtensorMap* map, const void* base, uint64_t tokens, uint64_t heads,
                        uint32_t box_heads, uint32_t box_tokens);

// Tensor map of an 8-bit pool as [tiles][1 KiB], for loads that gather four tiles.
bool encode_tile_rows(CUtensorMap* map, const void* base, uint64_t tiles);

struct PrefillArgs {
  void* out;
  const void* q;
  const int32_t* query_start_loc;
  int32_t num_query_tokens;
  int32_t max_query_len;
  const void* key_cache;
  const void* value_cache;
  int32_t num_blocks;
  int32_t num_kv_heads;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  int32_t num_seqs;
  int32_t num_q_heads;
  float scale;
  int32_t* status;
};

// overlap_previous: programmatic dependent launch behind the previous kernel in the stream
// (the kernel waits for it only at its end); max_sms > 0: at most two CTAs on each of that
// many SMs.
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream, bool overlap_previous = false,
                           int32_t max_sms = 0);

// Unified varlen launch: the decode kernel serves the one-row sequences in place (the
// workspace is its workspace), the chunk kernel the others.  Sizes on the current device:
// an upper bound for any head count and context (the size query), and the exact need of
// one call.
int decode_max_seqs();
size_t varlen_workspace_size(int32_t num_seqs, int32_t num_query_tokens);
size_t varlen_workspace_need(const PrefillArgs& a);
// decode_sms in 1 .. SMs-1: the decode rows on that many SMs and the chunks on the others,
// at the same time; 0: each kernel on every SM, one after the other.
cudaError_t launch_varlen(const PrefillArgs& a, void* workspace, cudaStream_t stream,
                          int32_t decode_sms = 0);

}  // namespace pkv
