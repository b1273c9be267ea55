// Compaction of kept tokens: of every sequence, the tokens at first + kept[0] < first + kept[1] < ...
// move to first, first + 1, ..., in place, keys and values of all heads (the accepted nodes of a
// drafted tree behind their prefix; a history thinned out).
//
// In place.  kept rises from kept[0] >= 0, so kept[i] >= i: a token moves to a slot at or before its
// own, and a slot below i is the source of no token from i on.  So the list is taken in rounds whose
// rows are all read before the first is written; the next round's rows lie behind all of them.
// Sequences, heads and pools share nothing.
//
// The 8-bit pools.  A round takes whole destination blocks, one per warp; their sources lie in the
// same block or behind it, so what a round writes, scales included, no later one reads.  A block's
// new rows are code * scale of where they were, and go into it as an append of these values would
// put them: a scale of their own where the block's first slot is among them, and one that only grows
// where earlier tokens stay.
//
// Memory-bound: every row is read and written once.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr int kRowLanes = 8;                 // lanes of a bf16 row, 16 bytes each
constexpr int kRowsAtOnce = 32 / kRowLanes;  // 4
constexpr int kUnroll = 4;                   // rows a lane has in flight
constexpr int kWarpRows = kRowsAtOnce * kUnroll;  // 16: a warp's share of a round
constexpr int kCtaWarps = 4;  // of a CTA whose warps serve an item each

// The list of sequence s; false where there is nothing to do, or it was reported.
__device__ __forceinline__ bool kept_list(const CompactArgs& a, int32_t s, bool report, int32_t* start, int32_t* n,
                                          int32_t* first) {
  *start = a.kept_start_loc[s];
  *n = a.kept_start_loc[s + 1] - *start;
  if (*n == 0) return false;
  *first = a.first[s];
  if (*n < 0 || *n > a.max_kept || *start < 0 || *n > a.num_kept - *start || *first < 0) {
    if (report) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return false;
  }
  return true;
}

// Source position of the list's entry i, or -1 (reported) where it does not rise or lies past the
// block-table row.
__device__ __forceinline__ int64_t source_of(const CompactArgs& a, const int32_t* kept, int32_t i, int32_t first,
                                             bool report) {
  const int32_t k = __ldg(kept + i);
  const int32_t before = i > 0 ? __ldg(kept + i - 1) : -1;
  const int64_t p = static_cast<int64_t>(first) + k;
  if (k <= before || k < i || p >= static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize) {
    if (report) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return -1;
  }
  return p;
}

// Physical block of position p of a sequence, or -1 (reported).
__device__ __forceinline__ int32_t block_of(const CompactArgs& a, const int32_t* table, int64_t p, bool report) {
  const int32_t b = __ldg(table + p / kBlockSize);
  if (b >= 0 && b < a.num_blocks) return b;
  if (report) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
  return -1;
}

// WARPS warps (of one CTA, if more than one) serve one (sequence, K/V head, pool).
template <int WARPS>
__global__ void __launch_bounds__((WARPS > 1 ? WARPS : kCtaWarps) * 32) compact_kernel(const CompactArgs a) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int64_t item = WARPS > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kCtaWarps + warp;
  const int64_t items = 2ll * a.num_seqs * a.num_kv_heads;
  if (item >= items) return;
  const bool is_k = (item & 1) == 0;
  const int h = static_cast<int>((item >> 1) % a.num_kv_heads);
  const int32_t s = static_cast<int32_t>((item >> 1) / a.num_kv_heads);
  const bool report = is_k && h == 0 && lane % kRowLanes == 0;
  int32_t start, n, first;
  if (!kept_list(a, s, report, &start, &n, &first)) return;
  const int32_t* const kept = a.kept + start;
  const int32_t* const table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  uint4* const pool = static_cast<uint4*>(is_k ? a.key_cache : a.value_cache);
  // 16-byte chunk of this lane in the row of position p
  auto place = [&](int32_t block, int64_t p) -> int64_t {
    return ((static_cast<int64_t>(block) * a.num_kv_heads + h) * kBlockSize + p % kBlockSize) * kRowLanes +
           lane % kRowLanes;
  };
  const int mine = (WARPS > 1 ? warp : 0) * kWarpRows + lane / kRowLanes;
  for (int32_t i0 = 0; i0 < n; i0 += WARPS * kWarpRows) {
    uint4 x[kUnroll];
    int64_t to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t i = i0 + mine + u * kRowsAtOnce;
      to[u] = -1;
      if (i >= n) continue;
      const int64_t src = source_of(a, kept, i, first, report);
      const int64_t dst = static_cast<int64_t>(first) + i;
      if (src < 0 || src == dst) continue;
      const int32_t from = block_of(a, table, src, report), at = block_of(a, table, dst, report);
      if (from < 0 || at < 0) continue;
      x[u] = pool[place(from, src)];
      to[u] = place(at, dst);
    }
    if (WARPS > 1) __syncthreads(); else __syncwarp();  // a round is read before it is written
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (to[u] >= 0) pool[to[u]] = x[u];
  }
}

// ---- 8-bit pools ---------------------------------------------------------------------------
__device__ __forceinline__ void codes16_to_floats(const uint4& c, float scale, float (&y)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    codes4_to_half2x2(w[i], lo, hi);
    const float2 p = half2_to_float2(lo), q = half2_to_float2(hi);
    y[4 * i] = p.x * scale;
    y[4 * i + 1] = p.y * scale;
    y[4 * i + 2] = q.x * scale;
    y[4 * i + 3] = q.y * scale;
  }
}

__device__ __forceinline__ uint4 floats16_to_codes(const float (&y)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = floats_to_codes2(y[4 * i] * inv, y[4 * i + 1] * inv) |
           (static_cast<uint32_t>(floats_to_codes2(y[4 * i + 2] * inv, y[4 * i + 3] * inv)) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int WARPS>
__global__ void __launch_bounds__((WARPS > 1 ? WARPS : kCtaWarps) * 32) compact_q8_kernel(const CompactArgs a) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int64_t item = WARPS > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kCtaWarps + warp;
  const int64_t items = 2ll * a.num_seqs * a.num_kv_heads;
  if (item >= items) return;
  const bool is_k = (item & 1) == 0;
  const int h = static_cast<int>((item >> 1) % a.num_kv_heads);
  const int32_t s = static_cast<int32_t>((item >> 1) / a.num_kv_heads);
  const bool report = is_k && h == 0;
  int32_t start, n, first;
  if (!kept_list(a, s, report && lane == 0, &start, &n, &first)) return;
  const int32_t* const kept = a.kept + start;
  const int32_t* const table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  uint8_t* const pool = static_cast<uint8_t*>(is_k ? a.key_cache : a.value_cache);
  float* const scales = is_k ? a.key_scale : a.value_scale;
  const int row0 = lane / kQ8RowLanes, l = lane % kQ8RowLanes;
  const int64_t b_lo = first / kBlockSize, b_hi = (static_cast<int64_t>(first) + n - 1) / kBlockSize;
  for (int64_t b0 = b_lo; b0 <= b_hi; b0 += WARPS) {
    const int64_t b = b0 + (WARPS > 1 ? warp : 0);
    bool live = b <= b_hi;
    // rows o0 .. o1 - 1 of the block are written; row o is the list's entry b * 16 + o - first
    const int o0 = b == b_lo ? first % kBlockSize : 0;
    const int o1 = live ? static_cast<int>(min(static_cast<int64_t>(kBlockSize), first + n - b * kBlockSize)) : 0;
    const int32_t at = live ? block_of(a, table, b * kBlockSize, report && lane == 0) : -1;
    live = at >= 0;
    const int64_t tile = (static_cast<int64_t>(at < 0 ? 0 : at) * a.num_kv_heads + h);
    float y[kQ8RowSteps][16];
    float amax = 0.f, old = 0.f;
    if (live) {
      bool bad_index = false, bad_scale = false;
      uint4 c[kQ8RowSteps];
      float from_scale[kQ8RowSteps];
      old = scales[tile];
#pragma unroll
      for (int k = 0; k < kQ8RowSteps; ++k) {
        const int o = row0 + k * kQ8WarpRows;
        c[k] = make_uint4(0u, 0u, 0u, 0u);
        from_scale[k] = 1.f;
        if (o < o0 || o >= o1) continue;
        const int64_t src = source_of(a, kept, static_cast<int32_t>(b * kBlockSize + o - first), first, report && l == 0);
        const int32_t from = src < 0 ? -1 : block_of(a, table, src, report && l == 0);
        if (from < 0) {
          bad_index = true;
          continue;
        }
        const int64_t t = static_cast<int64_t>(from) * a.num_kv_heads + h;
        from_scale[k] = scales[t];
        c[k] = reinterpret_cast<const uint4*>(pool + t * kQ8TileBytes + src % kBlockSize * kQ8RowBytes)[l];
      }
#pragma unroll
      for (int k = 0; k < kQ8RowSteps; ++k) {
        bad_scale |= !(from_scale[k] >= 0.f && from_scale[k] < INFINITY);
        codes16_to_floats(c[k], from_scale[k], y[k]);
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[k][i]));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      bad_scale |= o0 > 0 && !scale_ok(old);
      if (__any_sync(0xffffffffu, bad_index)) live = false;
      if (__any_sync(0xffffffffu, bad_scale) || !(amax < INFINITY)) {
        if (lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_SCALE);
        live = false;
      }
    }
    if (WARPS > 1) __syncthreads(); else __syncwarp();  // a round is read before it is written
    if (!live) continue;
    uint8_t* const codes = pool + tile * kQ8TileBytes;
    float now = scale_for(amax);
    if (o0 > 0) {
      if (now > old)
        rescale_rows(codes, old / now, o0, lane);
      else
        now = old;
    }
    const float inv = 1.f / now;
#pragma unroll
    for (int k = 0; k < kQ8RowSteps; ++k) {
      const int o = row0 + k * kQ8WarpRows;
      if (o >= o0 && o < o1) reinterpret_cast<uint4*>(codes + o * kQ8RowBytes)[l] = floats16_to_codes(y[k], inv);
    }
    if (lane == 0) scales[tile] = now;
  }
}

template <typename One, typename Four, typename Sixteen>
cudaError_t launch(const CompactArgs& a, cudaStream_t stream, One one, Four four, Sixteen sixteen) {
  const int64_t items = 2ll * a.num_seqs * a.num_kv_heads;
  if (a.max_kept <= 2 * kWarpRows)
    one<<<static_cast<unsigned>((items + kCtaWarps - 1) / kCtaWarps), kCtaWarps * 32, 0, stream>>>(a);
  else if (a.max_kept <= 8 * kWarpRows)
    four<<<static_cast<unsigned>(items), 4 * 32, 0, stream>>>(a);
  else
    sixteen<<<static_cast<unsigned>(items), 16 * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
  return launch(a, stream, compact_kernel<1>, compact_kernel<4>, compact_kernel<16>);
}

cudaError_t launch_compact_q8(const CompactArgs& a, cudaStream_t stream) {
  return launch(a, stream, compact_q8_kernel<1>, compact_q8_kernel<4>, compact_q8_kernel<16>);
}

}  // namespace pkv
