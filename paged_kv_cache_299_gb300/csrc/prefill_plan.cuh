// The in-kernel plan of the chunk-attention kernels: the work units (query tile, K/V head) of
// a batch, ordered heaviest first and dealt to the CTAs of a persistent grid.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace pkv {

namespace {

constexpr int kMaxUnitsPerCta = 256;   // work units one CTA can hold in its list
constexpr int kMaxSortPairs = 2048;    // (sequence, query tile) pairs sorted in-kernel
constexpr int kSortBuckets = 64;

constexpr int sort_scratch_bytes(int threads) {
  return 4 * kMaxSortPairs * 4 + (1 + threads / 32) * kSortBuckets * 4;
}

struct PParams {
  __nv_bfloat16* out;
  const int32_t* query_start_loc;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  int32_t num_blocks;
  int32_t num_kv_heads;
  int32_t num_q_heads;
  float qk_scale;  // scale * log2(e)
  int32_t* status;
  int32_t num_query_tokens;
  int32_t max_query_len;  // 8-bit kernel: longer chunks are reported and skipped
  int32_t num_seqs;
  int32_t q_tiles;  // query tiles of the longest chunk: ceil(max_query_len / 32)
  int32_t skip_single;  // 1: sequences with exactly one query row are served elsewhere
};

// One work unit: query tile `tile` (TOKENS tokens) of sequence s against K/V head g, with everything the roles derive from it.
struct Unit {
  int s, g, tile;
  int q0, q_len, L;
  int tok0, ntok, keys, n_kv, blocks_needed;
};

// Whether sequence s has query rows to serve, and its rows / context.  Sequences with no rows
// are skipped silently; rows outside q / out, more of them than max_query_len (BOUNDED), or a context
// shorter than the chunk or longer than its block-table row are reported (when `report`) and skipped.
template <bool BOUNDED>
__device__ __forceinline__ bool sequence_ok(const PParams& p, int s, int* q0, int* q_len, int* L,
                                            bool report) {
  *q0 = p.query_start_loc[s];
  *q_len = p.query_start_loc[s + 1] - *q0;
  if (*q_len <= 0) return false;
  *L = p.context_lens[s];
  if (*q0 < 0 || *q0 + *q_len > p.num_query_tokens || (BOUNDED && *q_len > p.max_query_len) || *L < *q_len ||
      static_cast<int64_t>(*L) > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize) {
    if (report) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
    return false;
  }
  return true;
}

template <int TOKENS, int KEYS>
__device__ __forceinline__ int tile_work(int L, int q_len, int tile) {
  const int ntok = min(TOKENS, q_len - tile * TOKENS);
  return (L - q_len + tile * TOKENS + ntok + KEYS - 1) / KEYS;
}

template <int TOKENS, int KEYS>
__device__ __forceinline__ void fill_unit(Unit& u) {
  u.tok0 = u.tile * TOKENS;
  u.ntok = min(TOKENS, u.q_len - u.tok0);
  u.keys = u.L - u.q_len + u.tok0 + u.ntok;  // this tile needs keys 0 .. keys-1
  u.n_kv = (u.keys + KEYS - 1) / KEYS;
  u.blocks_needed = (u.keys + kBlockSize - 1) / kBlockSize;
}

// The CTA's sequence of work units.  Sorted mode: the units (every existing (sequence, query
// tile) pair x K/V head) were ordered heaviest first by the in-kernel plan, and this CTA's
// share (a snake over the order: round r takes position r*G + c, or r*G + G-1-c on odd
// rounds) sits in shared memory.  Otherwise (very large batches) units are taken in grid
// order, the query-tile index slowest and reversed, CTA c serving c, c + G, c + 2G, ...
struct Schedule {
  const int32_t* unit_s;   // shared memory (sorted mode)
  const int32_t* unit_tg;  // tile * 64 + g
  int n_units;             // sorted mode: this CTA's unit count; -1: grid order
  // sorted mode, where the plan kept them: first row, rows and context of each unit's sequence
  const int32_t* unit_q0 = nullptr;
  const int32_t* unit_len = nullptr;
  const int32_t* unit_L = nullptr;
};

// KEPT: the 8-bit kernel's form, from what the plan kept of the sequences, chunks bounded by
// max_query_len (which the plan has reported by then).
template <int TOKENS, int KEYS, bool KEPT = false>
__device__ __forceinline__ bool next_unit(const PParams& p, const Schedule& sc, int& k, Unit& u) {
  if (sc.n_units >= 0) {
    if (k >= sc.n_units) return false;
    u.s = sc.unit_s[k];
    const int tg = sc.unit_tg[k];
    u.tile = tg >> 6;
    u.g = tg & 63;
    if (KEPT) {
      u.q0 = sc.unit_q0[k];
      u.q_len = sc.unit_len[k];
      u.L = sc.unit_L[k];
    } else {
      sequence_ok<KEPT>(p, u.s, &u.q0, &u.q_len, &u.L, false);
    }
    ++k;
    fill_unit<TOKENS, KEYS>(u);
    return true;
  }
  using Index = std::conditional_t<KEPT, uint32_t, int64_t>;  // (KEPT: the caller keeps the units below 2^31; with
  // 64-bit divisions inlined in every role, 3 chunks of some 4000 rows took 662 us against 645)
  const Index per_tile = static_cast<Index>(p.num_seqs) * p.num_kv_heads;
  const Index total = per_tile * p.q_tiles;
  for (;;) {
    const Index x = blockIdx.x + static_cast<Index>(k) * gridDim.x;
    if (x >= total) return false;
    ++k;
    const Index rem = x % per_tile;
    u.tile = p.q_tiles - 1 - static_cast<int>(x / per_tile);
    u.g = static_cast<int>(rem / p.num_seqs);
    u.s = static_cast<int>(rem % p.num_seqs);
    if (!sequence_ok<false>(p, u.s, &u.q0, &u.q_len, &u.L, u.tile == 0 && u.g == 0)) continue;
    if (u.tile * TOKENS >= u.q_len || (KEPT && u.q_len > p.max_query_len) || (p.skip_single && u.q_len == 1)) continue;
    fill_unit<TOKENS, KEYS>(u);
    return true;
  }
}

// Exclusive block-wide prefix sum over THREADS values; *total gets the sum.
template <int THREADS>
__device__ __forceinline__ int block_exclusive_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int x = scratch[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

// In-kernel plan, run by every CTA on the same inputs (so every CTA derives the same order):
// list the (sequence, query tile) pairs, sort them by their number of KEYS-key tiles, heaviest
// first (a stable counting sort on 64 buckets: ranks within a bucket come from warp matches
// in pair order, THREADS pairs per round), and take this CTA's units.  Returns the unit count, or
// -1 when the batch has more pairs than the sort handles (grid order then).
// RANK_PAIRS > 0: up to that many pairs are ranked directly, each thread counting the pairs that
// come before its own (fewer barriers than the counting sort: 8 chunks of 512 rows 70.9 us against
// 72.7), and unit_q0 / unit_len / unit_L
// keep each unit's sequence for next_unit<.., true>.
template <int TOKENS, int KEYS, int THREADS, int RANK_PAIRS = 0>
__device__ int plan_units(const PParams& p, uint8_t* scratch, int* red, int32_t* unit_s,
                          int32_t* unit_tg, int32_t* unit_q0 = nullptr, int32_t* unit_len = nullptr,
                          int32_t* unit_L = nullptr) {
  const int tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  constexpr int kWarpsP = THREADS / 32;
  static_assert(kWarpsP <= 24, "red holds 32 ints, the warps' from the ninth on");
  int* pair_s = reinterpret_cast<int*>(scratch);  // [kMaxSortPairs]
  int* pair_t = pair_s + kMaxSortPairs;
  int* pair_w = pair_t + kMaxSortPairs;
  int* sorted = pair_w + kMaxSortPairs;
  int* base = sorted + kMaxSortPairs;              // [kSortBuckets] next position per bucket
  int* wcnt = base + kSortBuckets;                 // [kWarpsP][kSortBuckets] per-round counts
  // 1. enumerate the pairs, THREADS sequences at a time
  int n = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += THREADS) {
    const int s = s0 + tid;
    int q0 = 0, q_len = 0, L = 0, tiles = 0;
    if (s < p.num_seqs && sequence_ok<(RANK_PAIRS > 0)>(p, s, &q0, &q_len, &L, blockIdx.x == 0) &&
        !(p.skip_single && q_len == 1))
      tiles = (q_len + TOKENS - 1) / TOKENS;
    int total;
    const int excl = block_exclusive_scan<THREADS>(tiles, red, &total);
    if (n + total <= kMaxSortPairs) {
      for (int t = 0; t < tiles; ++t) {
        pair_s[n + excl + t] = s;
        pair_t[n + excl + t] = t;
        pair_w[n + excl + t] = tile_work<TOKENS, KEYS>(L, q_len, t);
      }
    }
    n += total;
  }
  const int units = n * p.num_kv_heads;
  const int G = gridDim.x;
  if (n > kMaxSortPairs || (units + G - 1) / G > kMaxUnitsPerCta) return -1;
  const bool rank = n <= RANK_PAIRS;  // uniform
  if (rank) {
    __syncthreads();
    for (int i = tid; i < n; i += THREADS) {
      const int w = pair_w[i];
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const int x = pair_w[j];
        before += x > w || (x == w && j < i);
      }
      sorted[before] = i;
    }
    __syncthreads();
  } else {
    for (int i = tid; i < kSortBuckets * (kWarpsP + 1); i += THREADS) base[i] = 0;  // + wcnt
    __syncthreads();  // the pairs written above are read by other threads below
    // 2. largest work, then bucket = work scaled to 0..63 (heavier = higher)
    int wmax = 0;
    for (int i = tid; i < n; i += THREADS) wmax = max(wmax, pair_w[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) wmax = max(wmax, __shfl_xor_sync(0xffffffffu, wmax, d));
    if (lane == 0) red[8 + warp] = wmax;
    __syncthreads();
    wmax = 0;
    for (int w = 0; w < kWarpsP; ++w) wmax = max(wmax, red[8 + w]);
    auto bucket = [&](int i) {
      const int b = static_cast<int>((static_cast<int64_t>(pair_w[i]) * kSortBuckets) / (wmax + 1));
      return min(max(b, 0), kSortBuckets - 1);
    };
    for (int i = tid; i < n; i += THREADS) atomicAdd(&base[bucket(i)], 1);
    __syncthreads();
    // 3. bucket starts, heaviest bucket first (one warp, two buckets per lane)
    if (warp == 0) {
      const int hi = base[kSortBuckets - 1 - 2 * lane], lo = base[kSortBuckets - 2 - 2 * lane];
      int incl = hi + lo;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += x;
      }
      const int start = incl - hi - lo;
      base[kSortBuckets - 1 - 2 * lane] = start;
      base[kSortBuckets - 2 - 2 * lane] = start + hi;
    }
    __syncthreads();
    // 4. stable placement, pair i = round * THREADS + tid: its rank in its bucket counts the pairs of
    // earlier rounds (base), of earlier warps in this round (wcnt) and of lower lanes (match)
    for (int r0 = 0; r0 < n; r0 += THREADS) {
      const int i = r0 + tid;
      const int b = i < n ? bucket(i) : kSortBuckets;  // kSortBuckets: no pair
      const unsigned same = __match_any_sync(0xffffffffu, b);
      const int rank = __popc(same & ((1u << lane) - 1u));
      if (b < kSortBuckets && rank == 0) wcnt[warp * kSortBuckets + b] = __popc(same);
      __syncthreads();
      if (b < kSortBuckets) {
        int before = base[b] + rank;
        for (int w = 0; w < warp; ++w) before += wcnt[w * kSortBuckets + b];
        sorted[before] = i;
      }
      __syncthreads();
      if (tid < kSortBuckets) {
        int add = 0;
        for (int w = 0; w < kWarpsP; ++w) {
          add += wcnt[w * kSortBuckets + tid];
          wcnt[w * kSortBuckets + tid] = 0;
        }
        base[tid] += add;
      }
      __syncthreads();
    }
  }
  // 5. this CTA's units: a snake over the sorted order, K/V head fastest
  const int c = blockIdx.x;
  const int rounds = (units + G - 1) / G;
  int mine = 0;
  for (int r = 0; r < rounds; ++r) {
    const int pos = r * G + ((r & 1) ? G - 1 - c : c);
    if (pos < units) ++mine;
  }
  for (int k = tid; k < mine; k += THREADS) {
    const int pos = k * G + ((k & 1) ? G - 1 - c : c);
    const int pr = sorted[pos / p.num_kv_heads];
    unit_s[k] = pair_s[pr];
    unit_tg[k] = pair_t[pr] * 64 + pos % p.num_kv_heads;
    if (unit_q0 != nullptr) sequence_ok<(RANK_PAIRS > 0)>(p, pair_s[pr], &unit_q0[k], &unit_len[k], &unit_L[k], false);
  }
  return mine;
}

}  // namespace

}  // namespace pkv
