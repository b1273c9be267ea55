// What the decode kernels share: the flattened (sequence, kv head, block) tile space and its
// balanced split into runs.
#pragma once

#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {

namespace {

constexpr float kRescaleThreshold = 8.0f;     // log2 units: rescale when max grows > 2^8
constexpr int kMaxSeqs = 4096;

struct KParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t num_blocks;
  float q_scale;  // scale * log2(e): scores come out in log2 units
  int32_t grid;      // runs of the decomposition (warp w of the grid serves runs
                     // w, w + warps, ...)
  int32_t chunk;     // tiles per run, 0 = balanced split into `grid` runs
  int64_t tile_bound;  // > 0: the host's upper bound of the tile count (partitioned runs)
  int64_t* ws_total;    // total tiles, written by CTA 0
  int32_t* ws_seq_base; // [num_seqs + 1] blocks-per-head prefix, written by CTA 0
  float* partials;      // [runs][2][GROUP][kPartialFloats]
  int32_t* seg_count;   // [num_seqs * Hkv] pieces published per split segment (fused merge);
                        // zero between calls: the merging warp resets its counter
                        // (8-bit decode: one per CTA, by a split segment's first)
  int32_t fused_merge;  // 1: the last warp to finish a split segment merges it in place
  int32_t prefetch_ok;  // 1: a warp may ask L2 for tiles past its ring before its wait
  const uint8_t* k_new;  // optional [num_seqs][Hkv][64] bf16: token at position L-1 to store
  const uint8_t* v_new;  //   (fused append: stored to its slot and used in attention)
  uint8_t* key_cache_w;    // writable views of the pools (fused append)
  uint8_t* value_cache_w;
  int32_t* status;
  // Mixed batches (the varlen launch): sequence s's query and output row is q_rows[s], and
  // only sequences with exactly one row (q_rows[s+1] - q_rows[s] == 1) are served here; the
  // others are left alone (no tiles, nothing written).  nullptr: row s, every sequence.
  const int32_t* q_rows;
  int32_t num_query_tokens;
};

// Run containing tile x (x < total).  Runs are [run_start(c), run_start(c+1)).
__device__ __forceinline__ int64_t run_of(int64_t x, int64_t total, int32_t grid,
                                          int32_t chunk) {
  if (chunk > 0) return x / chunk;
  return ((x + 1) * grid - 1) / total;
}

// Largest s in [0, num_seqs) with kv * base[s] <= y (y < kv * base[num_seqs]).
__device__ __forceinline__ int find_seq(const int32_t* base, int num_seqs, int64_t y, int kv) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(base[mid]) * kv <= y) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct Piece {
  int s, g, b0, b1, nb;
};

// bf16 pair {lo = x, hi = y}
__device__ __forceinline__ uint32_t pack_bf16x2(float x, float y) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Per-sequence block counts and their exclusive prefix (the tile index space), into
// seq_base[0 .. S] in shared memory; warp_sums is scratch.  Every thread of the CTA calls it.
template <int WARPS, bool kRows>
__device__ __forceinline__ void block_prefix(const KParams& p, int32_t* seq_base,
                                             int64_t* warp_sums) {
  constexpr int kThreads = WARPS * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.num_seqs, KV = p.num_kv_heads;
  for (int i = tid; i < S; i += kThreads) {
    const int32_t L = p.context_lens[i];
    int32_t nb = 0;
    bool serve = true;
    if (kRows) {  // mixed batch: decode rows only, the same checks as chunks
      const int32_t r0 = p.q_rows[i];
      const int32_t q_len = p.q_rows[i + 1] - r0;
      serve = q_len == 1;
      if (serve && (r0 < 0 || r0 >= p.num_query_tokens || L < 1)) {
        if (blockIdx.x == 0) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
        serve = false;
      }
    }
    if (!serve) {
    } else if (L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize) {
      if (blockIdx.x == 0) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
    } else {
      nb = (L + kBlockSize - 1) / kBlockSize;
    }
    seq_base[i] = nb;
  }
  __syncthreads();
  {
    const int per = (S + kThreads - 1) / kThreads;
    const int beg = min(tid * per, S);
    const int end = min(beg + per, S);
    int64_t local = 0;
    for (int i = beg; i < end; ++i) local += seq_base[i];
    int64_t incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int64_t run = incl - local;
    int64_t grand = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) run += warp_sums[w];
      grand += warp_sums[w];
    }
    const bool overflow = grand * KV > 0x7fffffffLL;
    for (int i = beg; i < end; ++i) {
      const int32_t v = seq_base[i];
      seq_base[i] = static_cast<int32_t>(overflow ? 0 : run);
      run += v;
    }
    if (tid == 0) seq_base[S] = static_cast<int32_t>(overflow ? 0 : grand);
    if (overflow && tid == 0 && blockIdx.x == 0) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
  }
  __syncthreads();
}

// Block-table window: lane j holds the tile (phys_block * Hkv + kv_head) of the j-th of
// `n` consecutive tiles of one run, or -1 for an invalid block id.
struct Window {
  int32_t tile;  // raw block id until resolved (see resolve_window), then the tile or -1
  int32_t g;
  int n;
};

}  // namespace

}  // namespace pkv
