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
// Every row is read and written once.  Measured (8 K/V heads): 64 histories of 300 to 500 kept tokens (106.9 MB) 13.2
// us where a replay finds what the last one wrote in L2; 21.4 where eleven such batches take turns, so that every row
// comes from DRAM and goes back there within the time (5.0 TB/s, 0.74 of the copy rate: a CTA either reads a
// round or writes one, and between the two nothing is in flight); 256 of 100 to 250 34.2 (5.2 TB/s).  In the 8-bit
// pools the same 64 (53.7 MB) 20.2 and 28.4 us (1.9 TB/s): list, tables and scales are waited for block by
// block.  32 paths of up to 5 tokens 2.6 us, 256 of up to 8 in the 8-bit pools 5.8: the launch and the chain of
// dependent loads.
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
constexpr int64_t kManyItems = 2 * 152;   // more items than CTAs of 16 warps run side by side
constexpr int64_t kManyShort = 8 * 152;  // (8 bits, up to 8 tokens: 512 items 3.2 us with two warps each, 3.9 with one;
                                         // 4096 items 7.4 and 6.2)

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

// Source positions of N entries i[u] of a list (below 0: none wanted), or -1; an entry that does not rise
// or lies past the block-table row is reported.  Loads of one kind come side by side, here and below: a
// round is a chain of list, tables and rows.
template <int N>
__device__ __forceinline__ bool sources_of(const CompactArgs& a, const int32_t* kept, const int32_t (&i)[N],
                                           int32_t first, int32_t (&src)[N]) {
  int32_t k[N], before[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    k[u] = i[u] >= 0 ? __ldg(kept + i[u]) : 0;
    before[u] = i[u] > 0 ? __ldg(kept + i[u] - 1) : -1;
  }
  bool fine = true;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int64_t p = static_cast<int64_t>(first) + k[u];
    const bool bad = k[u] <= before[u] || k[u] < i[u] || p > INT32_MAX ||
                     p >= static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize;
    if (i[u] >= 0 && bad) fine = false;
    src[u] = i[u] < 0 || bad ? -1 : static_cast<int32_t>(p);
  }
  return fine;
}

// Physical blocks of N positions (below 0: none wanted), or -1; false where one is bad.
template <int N>
__device__ __forceinline__ bool blocks_of(const CompactArgs& a, const int32_t* table, const int32_t (&p)[N],
                                          int32_t (&block)[N]) {
#pragma unroll
  for (int u = 0; u < N; ++u) block[u] = p[u] >= 0 ? __ldg(table + p[u] / kBlockSize) : 0;
  bool fine = true;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const bool bad = block[u] < 0 || block[u] >= a.num_blocks;
    if (bad) fine = false;
    if (bad || p[u] < 0) block[u] = -1;
  }
  return fine;
}

// Where N entries of a list (below 0: none wanted) move: positions and blocks; one block of a move is below 0
// where nothing is to do, or something was reported.
template <int N>
__device__ __forceinline__ void moves_of(const CompactArgs& a, const int32_t* kept, const int32_t* table,
                                         const int32_t (&i)[N], int32_t first, bool report, int32_t (&src)[N],
                                         int32_t (&dst)[N], int32_t (&from)[N], int32_t (&at)[N]) {
  const bool fine = sources_of(a, kept, i, first, src);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    dst[u] = src[u] >= 0 ? first + i[u] : -1;
    if (src[u] == dst[u]) src[u] = dst[u] = -1;  // it stays
  }
  const bool blocks = blocks_of(a, table, src, from) & blocks_of(a, table, dst, at);
  if (report && !fine) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
  if (report && !blocks) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
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
  const bool report = is_k && h == 0;
  int32_t start, n, first;
  if (!kept_list(a, s, report && lane == 0, &start, &n, &first)) return;
  const int32_t* const kept = a.kept + start;
  const int32_t* const table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  uint4* const pool = static_cast<uint4*>(is_k ? a.key_cache : a.value_cache);
  const int mine = (WARPS > 1 ? warp : 0) * kWarpRows + lane / kRowLanes;
  auto place = [&](int32_t block, int32_t p) -> uint4* {  // 16-byte chunk of this lane in the row of position p
    return pool + ((static_cast<int64_t>(block) * a.num_kv_heads + h) * kBlockSize + p % kBlockSize) * kRowLanes +
           lane % kRowLanes;
  };
  if (WARPS == 1) {
    for (int32_t i0 = 0; i0 < n; i0 += kWarpRows) {
      int32_t i[kUnroll], src[kUnroll], dst[kUnroll], from[kUnroll], at[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int32_t x = i0 + mine + u * kRowsAtOnce;
        i[u] = x < n ? x : -1;
      }
      moves_of(a, kept, table, i, first, report, src, dst, from, at);
      uint4 x[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (from[u] >= 0 && at[u] >= 0) x[u] = *place(from[u], src[u]);
      __syncwarp();  // a round is read before it is written
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (from[u] >= 0 && at[u] >= 0) *place(at[u], dst[u]) = x[u];
    }
    return;
  }
  // A CTA looks kRounds rounds' moves up at once, a thread kMoves of them, and keeps them in shared memory, so that
  // the list and the tables are waited for once.
  constexpr int kRounds = 4, kRoundRows = WARPS * kWarpRows, kMoves = kRounds * kRoundRows / (WARPS * 32);
  __shared__ int2 blocks[kRounds * kRoundRows];      // of source and destination; below 0: nothing moves
  __shared__ uint8_t offset[kRounds * kRoundRows];   // the source's in its block
  for (int32_t i0 = 0; i0 < n; i0 += kRounds * kRoundRows) {
    int32_t i[kMoves], src[kMoves], dst[kMoves], from[kMoves], at[kMoves];
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const int32_t x = i0 + static_cast<int>(threadIdx.x) + u * WARPS * 32;
      i[u] = x < n ? x : -1;
    }
    moves_of(a, kept, table, i, first, report, src, dst, from, at);
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const int e = threadIdx.x + u * WARPS * 32;
      blocks[e] = at[u] >= 0 ? make_int2(from[u], at[u]) : make_int2(-1, -1);
      offset[e] = static_cast<uint8_t>(src[u] & (kBlockSize - 1));
    }
    __syncthreads();
#pragma unroll 1
    for (int e0 = 0; e0 < kRounds * kRoundRows && i0 + e0 < n; e0 += kRoundRows) {
      uint4 x[kUnroll];
      int2 b[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int e = e0 + mine + u * kRowsAtOnce;
        b[u] = blocks[e];
        if (b[u].x >= 0) x[u] = *place(b[u].x, offset[e]);
      }
      __syncthreads();  // a round is read before it is written
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (b[u].x >= 0) *place(b[u].y, first + i0 + e0 + mine + u * kRowsAtOnce) = x[u];
    }
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
  const int warp = WARPS > 1 ? threadIdx.x >> 5 : 0;
  const int64_t item = WARPS > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kCtaWarps + (threadIdx.x >> 5);
  if (item >= 2ll * a.num_seqs * a.num_kv_heads) return;
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
  // A round: a destination block per warp.
  struct Round {
    uint4 c[kQ8RowSteps];
    float scale[kQ8RowSteps], old;  // of the rows' blocks, and the destination's
    int32_t block;                  // or -1: nothing to write
  };
  // rows o0 .. o1 - 1 of block b are written; row o is the list's entry b * 16 + o - first
  auto first_row = [&](int64_t b) { return b == b_lo ? first % kBlockSize : 0; };
  auto last_row = [&](int64_t b) {
    // (in 64 bits: a wrong `first` may lie near the end of the ints)
    return b <= b_hi ? static_cast<int>(min(static_cast<int64_t>(kBlockSize), static_cast<int64_t>(first) + n - b * kBlockSize)) : 0;
  };
  auto read = [&](int64_t b, Round& r) {
    const int o0 = first_row(b), o1 = last_row(b);
    int32_t i[kQ8RowSteps], from[kQ8RowSteps], at[1];
    int32_t src[kQ8RowSteps];
#pragma unroll
    for (int k = 0; k < kQ8RowSteps; ++k) {
      const int o = row0 + k * kQ8WarpRows;
      i[k] = o >= o0 && o < o1 ? static_cast<int32_t>(b * kBlockSize + o - first) : -1;
    }
    const bool all_fine = __all_sync(0xffffffffu, sources_of(a, kept, i, first, src));
    // (a destination is known to lie in the table by its sources, at or behind it)
    const int32_t dst[1] = {all_fine && b <= b_hi ? static_cast<int32_t>(b * kBlockSize) : -1};
    const bool blocks = blocks_of(a, table, src, from) & blocks_of(a, table, dst, at);
    const bool all_blocks = __all_sync(0xffffffffu, blocks);
    if (report && lane == 0 && !all_fine) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    if (report && lane == 0 && !all_blocks) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
    r.block = all_fine && all_blocks ? at[0] : -1;
    r.old = r.block >= 0 ? scales[static_cast<int64_t>(r.block) * a.num_kv_heads + h] : 1.f;
#pragma unroll
    for (int k = 0; k < kQ8RowSteps; ++k) {
      r.c[k] = make_uint4(0u, 0u, 0u, 0u);
      r.scale[k] = 1.f;
      if (from[k] < 0) continue;
      const int64_t t = static_cast<int64_t>(from[k]) * a.num_kv_heads + h;
      r.scale[k] = scales[t];
      r.c[k] = reinterpret_cast<const uint4*>(pool + t * kQ8TileBytes + src[k] % kBlockSize * kQ8RowBytes)[l];
    }
  };
  auto write = [&](int64_t b, const Round& r) {
    const int o0 = first_row(b), o1 = last_row(b);
    float y[kQ8RowSteps][16];
    float amax = 0.f;
    bool bad = o0 > 0 && !scale_ok(r.old);
#pragma unroll
    for (int k = 0; k < kQ8RowSteps; ++k) {
      bad |= !(r.scale[k] >= 0.f && r.scale[k] < INFINITY);
      codes16_to_floats(r.c[k], r.scale[k], y[k]);
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[k][i]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    bad = __any_sync(0xffffffffu, bad) || !(amax < INFINITY);
    if (WARPS > 1) __syncthreads(); else __syncwarp();  // a round is read before it is written
    if (r.block < 0) return;
    if (bad) {
      if (lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_SCALE);
      return;
    }
    const int64_t tile = static_cast<int64_t>(r.block) * a.num_kv_heads + h;
    uint8_t* const codes = pool + tile * kQ8TileBytes;
    float now = scale_for(amax);
    if (o0 > 0) {
      if (now > r.old)
        rescale_rows(codes, r.old / now, o0, lane);
      else
        now = r.old;
    }
    const float inv = 1.f / now;
#pragma unroll
    for (int k = 0; k < kQ8RowSteps; ++k) {
      const int o = row0 + k * kQ8WarpRows;
      if (o >= o0 && o < o1) reinterpret_cast<uint4*>(codes + o * kQ8RowBytes)[l] = floats16_to_codes(y[k], inv);
    }
    if (lane == 0) scales[tile] = now;
  };
  for (int64_t b0 = b_lo; b0 <= b_hi; b0 += WARPS) {
    Round r;
    read(b0 + warp, r);
    write(b0 + warp, r);
  }
}

}  // namespace

// Warps of an item (sequence, head, pool), by the longest list: of a few tokens a warp, four items a CTA;
// otherwise a CTA, of sixteen warps as long as the CTAs run side by side, of four beyond (bf16, 4, 8 and 16
// warps: 8 sequences of 300 to 500 tokens, 8 heads 6.3, 4.3, 4.2 us, 64 of them 13.5, 14.5, 17.1, 256 of 100 to 250
// 33.0, 39.3, 50.5, 2 of 4000 to 6000 40.2, 23.1, 18.5).
cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
  const int64_t items = 2ll * a.num_seqs * a.num_kv_heads;
  const unsigned grid = static_cast<unsigned>(items);
  if (a.max_kept <= 2 * kWarpRows)
    compact_kernel<1><<<static_cast<unsigned>((items + kCtaWarps - 1) / kCtaWarps), kCtaWarps * 32, 0, stream>>>(a);
  else if (a.max_kept <= 8 * kWarpRows || items > kManyItems)
    compact_kernel<4><<<grid, 4 * 32, 0, stream>>>(a);
  else
    compact_kernel<16><<<grid, 16 * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_compact_q8(const CompactArgs& a, cudaStream_t stream) {
  const int64_t items = 2ll * a.num_seqs * a.num_kv_heads;
  const unsigned grid = static_cast<unsigned>(items);
  if (a.max_kept <= 2 * kBlockSize + 1 && items > kManyShort)
    compact_q8_kernel<1><<<static_cast<unsigned>((items + kCtaWarps - 1) / kCtaWarps), kCtaWarps * 32, 0, stream>>>(a);
  else if (a.max_kept <= kBlockSize + 1)  // two blocks at most
    compact_q8_kernel<2><<<grid, 2 * 32, 0, stream>>>(a);
  else if (a.max_kept <= 8 * kBlockSize)
    compact_q8_kernel<4><<<grid, 4 * 32, 0, stream>>>(a);
  else if (items > kManyItems)
    compact_q8_kernel<8><<<grid, 8 * 32, 0, stream>>>(a);
  else
    compact_q8_kernel<16><<<grid, 16 * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
