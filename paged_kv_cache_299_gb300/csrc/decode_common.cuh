// What the decode kernels share: the flattened (sequence, kv head, block) tile space, its
// balanced split into runs, and the log-sum-exp merge of segments that were split.
#pragma once

#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {

namespace {

constexpr int kPartialFloats = kHeadDim + 2;  // o[64], max (log2 units), sum
constexpr float kRescaleThreshold = 8.0f;     // log2 units: rescale when max grows > 2^8
constexpr int kMaxSeqs = 4096;
constexpr int kMergeThreads = 512;
constexpr int kMergeUnroll = 4;  // partials whose loads one warp has in flight at once
constexpr int kMergeSplitPieces = 16;  // segments with this many pieces merge per query head

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

// Query / output row of sequence s (kRows: the mixed-batch form, a separate instantiation
// so that the plain decode path compiles without it).
template <bool kRows>
__device__ __forceinline__ int64_t row_of(const KParams& p, int s) {
  if (kRows) return p.q_rows[s];
  return s;
}

__device__ __forceinline__ int64_t run_start(int64_t c, int64_t total, int32_t grid,
                                             int32_t chunk) {
  if (chunk > 0) return c * chunk < total ? c * chunk : total;
  return c * total / grid;
}

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

__device__ __forceinline__ Piece piece_at(const int32_t* base, int num_seqs, int kv, int64_t y,
                                          int64_t run_end) {
  Piece pc;
  pc.s = find_seq(base, num_seqs, y, kv);
  pc.nb = base[pc.s + 1] - base[pc.s];
  const int64_t off = y - static_cast<int64_t>(base[pc.s]) * kv;
  pc.g = static_cast<int>(off / pc.nb);
  pc.b0 = static_cast<int>(off % pc.nb);
  const int64_t left = run_end - y;
  pc.b1 = (pc.nb - pc.b0 <= left) ? pc.nb : pc.b0 + static_cast<int>(left);
  return pc;
}

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

// Pieces of segment [x0, x1) (one (sequence, kv head)): the non-empty runs it touches.  The
// first piece sits in slot 0 of its run when the segment starts the run, else in slot 1;
// every later piece starts its run (slot 0).
struct SegmentPieces {
  int64_t c_first, c_last;
  int first_slot;
};

__device__ __forceinline__ SegmentPieces segment_pieces(int64_t x0, int64_t x1, int64_t total,
                                                        int32_t runs, int32_t chunk) {
  SegmentPieces sp;
  sp.c_first = run_of(x0, total, runs, chunk);
  sp.c_last = run_of(x1 - 1, total, runs, chunk);
  sp.first_slot = x0 == run_start(sp.c_first, total, runs, chunk) ? 0 : 1;
  return sp;
}

// Number of pieces of a segment, and the run holding piece k (balanced splits only, which
// is the only mode that merges inside the attention kernel).  With at least one tile per
// run (total >= runs) every run is non-empty and piece k lies in run c_first + k; otherwise
// every non-empty run holds exactly one tile and piece k is the run of tile x0 + k.
__device__ __forceinline__ int segment_piece_count(const SegmentPieces& sp, int64_t x0, int64_t x1,
                                                   int64_t total, int32_t runs) {
  return total >= runs ? static_cast<int>(sp.c_last - sp.c_first + 1) : static_cast<int>(x1 - x0);
}
__device__ __forceinline__ int64_t segment_piece_run(const SegmentPieces& sp, int64_t x0, int k,
                                                     int64_t total, int32_t runs, int32_t chunk) {
  return total >= runs ? sp.c_first + k : run_of(x0 + k, total, runs, chunk);
}

// One warp combines all pieces of a split segment (log-sum-exp weights) and writes the bf16
// rows of its GROUP query heads.  Lane k reads piece k's (max, sum), so the pieces' loads
// overlap; chunks of 32 pieces are combined with a running maximum.  Partials were written
// by other warps in this launch, so they are read through L2 (__ldcg), after the caller's
// acquire fence.
constexpr int kFewPieces = 4;  // segments of up to this many pieces merge in one load round

// Partials written by warps of this CTA (published with CTA-scope ordering) are read with
// plain loads; partials from other SMs through L2.
template <bool kLocal>
__device__ __forceinline__ float ld_partial(const float* a) {
  return kLocal ? *a : __ldcg(a);
}
template <bool kLocal>
__device__ __forceinline__ float2 ld_partial2(const float2* a) {
  return kLocal ? *a : __ldcg(a);
}

template <int GROUP, bool kLocal, bool kRows, int UNROLL = 4>
__device__ void merge_segment_in_warp(const KParams& p, const SegmentPieces& sp, int64_t x0,
                                      int64_t x1, int64_t total, int s, int g, int lane) {
  const int n = segment_piece_count(sp, x0, x1, total, p.grid);
  if (n <= kFewPieces) {
    // Few pieces (the usual case): every lane loads the (max, sum) of all pieces and its
    // own output slice of each, all in one round of loads, and combines them in registers.
    float mk[kFewPieces][GROUP], lk[kFewPieces][GROUP];
    float2 vk[kFewPieces][GROUP];
#pragma unroll
    for (int k = 0; k < kFewPieces; ++k) {
      if (k < n) {
        const int64_t c = segment_piece_run(sp, x0, k, total, p.grid, p.chunk);
        const int slot = k == 0 ? sp.first_slot : 0;
        const float* rec = p.partials + (c * 2 + slot) * GROUP * kPartialFloats;
#pragma unroll
        for (int h = 0; h < GROUP; ++h) {
          mk[k][h] = ld_partial<kLocal>(rec + h * kPartialFloats + kHeadDim);
          lk[k][h] = ld_partial<kLocal>(rec + h * kPartialFloats + kHeadDim + 1);
          vk[k][h] = ld_partial2<kLocal>(reinterpret_cast<const float2*>(rec + h * kPartialFloats) + lane);
        }
      } else {
#pragma unroll
        for (int h = 0; h < GROUP; ++h) {
          mk[k][h] = -INFINITY;
          lk[k][h] = 0.f;
          vk[k][h] = make_float2(0.f, 0.f);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < GROUP; ++h) {
      float mh = mk[0][h];
#pragma unroll
      for (int k = 1; k < kFewPieces; ++k) mh = fmaxf(mh, mk[k][h]);
      float lh = 0.f;
      float2 ah = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kFewPieces; ++k) {
        const float wgt = k < n ? fast_exp2(mk[k][h] - mh) : 0.f;
        lh += wgt * lk[k][h];
        ah.x += wgt * vk[k][h].x;
        ah.y += wgt * vk[k][h].y;
      }
      const float inv = 1.f / lh;
      __nv_bfloat16* out =
          p.out + (row_of<kRows>(p, s) * p.num_q_heads + g * GROUP + h) * kHeadDim;
      reinterpret_cast<__nv_bfloat162*>(out)[lane] = __floats2bfloat162_rn(ah.x * inv, ah.y * inv);
    }
    return;
  }
  float M[GROUP], L[GROUP];
  float2 acc[GROUP];
#pragma unroll
  for (int h = 0; h < GROUP; ++h) {
    M[h] = -INFINITY;
    L[h] = 0.f;
    acc[h] = make_float2(0.f, 0.f);
  }
  for (int base = 0; base < n; base += 32) {
    const int k = base + lane;
    const bool valid = k < n;
    const float* rec = p.partials;
    if (valid) {
      const int64_t c = segment_piece_run(sp, x0, k, total, p.grid, p.chunk);
      const int slot = k == 0 ? sp.first_slot : 0;
      rec = p.partials + (c * 2 + slot) * GROUP * kPartialFloats;
    }
    // every head's (max, sum) of piece k, all loads in flight together
    float mk[GROUP], lk[GROUP], wk[GROUP];
#pragma unroll
    for (int h = 0; h < GROUP; ++h) {
      mk[h] = valid ? ld_partial<kLocal>(rec + h * kPartialFloats + kHeadDim) : -INFINITY;
      lk[h] = valid ? ld_partial<kLocal>(rec + h * kPartialFloats + kHeadDim + 1) : 0.f;
    }
#pragma unroll
    for (int h = 0; h < GROUP; ++h) {
      float cm = mk[h];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, off));
      const float nm = fmaxf(M[h], cm);
      const float keep = M[h] == -INFINITY ? 0.f : fast_exp2(M[h] - nm);
      wk[h] = valid ? fast_exp2(mk[h] - nm) : 0.f;
      float lw = wk[h] * lk[h];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
      L[h] = L[h] * keep + lw;
      acc[h].x *= keep;
      acc[h].y *= keep;
      M[h] = nm;
    }
    // output slices: UNROLL pieces x GROUP heads of loads in flight per round
    const int cnt = min(32, n - base);
    for (int j0 = 0; j0 < cnt; j0 += UNROLL) {
      float2 v[UNROLL][GROUP];
      float w[UNROLL][GROUP];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int j = j0 + u < cnt ? j0 + u : j0;  // clamp; weight zeroed below
        const float* rj = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(rec), j));
#pragma unroll
        for (int h = 0; h < GROUP; ++h) {
          w[u][h] = __shfl_sync(0xffffffffu, wk[h], j);
          if (j0 + u >= cnt) w[u][h] = 0.f;
          v[u][h] = ld_partial2<kLocal>(reinterpret_cast<const float2*>(rj + h * kPartialFloats) + lane);
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
#pragma unroll
        for (int h = 0; h < GROUP; ++h) {
          acc[h].x += w[u][h] * v[u][h].x;
          acc[h].y += w[u][h] * v[u][h].y;
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < GROUP; ++h) {
    const float inv = 1.f / L[h];
    __nv_bfloat16* out =
        p.out + (row_of<kRows>(p, s) * p.num_q_heads + g * GROUP + h) * kHeadDim;
    reinterpret_cast<__nv_bfloat162*>(out)[lane] =
        __floats2bfloat162_rn(acc[h].x * inv, acc[h].y * inv);
  }
}

// Splits weighted by segment: every (sequence, kv head) segment counts EXTRA units on top of its
// tiles (what starting and publishing a piece costs, in tiles), EXTRA also where it has none,
// and the runs divide the units evenly.  Units of sequence s start at unit_base(s), those of its
// segment g at + g (nb + EXTRA), its tiles' at + EXTRA.
template <int EXTRA>
__device__ __forceinline__ int64_t unit_base(const int32_t* base, int s, int kv) {
  return static_cast<int64_t>(kv) * (static_cast<int64_t>(base[s]) + static_cast<int64_t>(EXTRA) * s);
}

// Combines the partials of every (sequence, kv head) whose tiles were split across CTAs,
// and writes zero rows for empty contexts.  One CTA per (sequence, kv head, HPC of the
// head's GROUP query heads): HPC = GROUP when segments have few pieces, 1 when they have
// many (long contexts), so that GROUP times as many CTAs share the loads.  Each warp folds
// its partials into a running (maximum, sum, o) per query head, rescaling by the
// log-sum-exp weights as the maximum grows, with U partials' loads in flight per round;
// the warps' states are then combined the same way.
template <int GROUP, int HPC, bool kRows, int EXTRA>
__global__ void __launch_bounds__(kMergeThreads)
merge_partials_kernel(const KParams p) {
  constexpr int kWarps = kMergeThreads / 32;
  constexpr int kSplit = GROUP / HPC;
  constexpr int U = HPC == 1 ? 2 * kMergeUnroll : kMergeUnroll;
  __shared__ float red_m[kWarps][HPC];
  __shared__ float red_l[kWarps][HPC];
  __shared__ float red_o[kWarps][HPC][kHeadDim];
  const int g = blockIdx.x / kSplit;
  const int h0 = (blockIdx.x % kSplit) * HPC;
  const int s = blockIdx.y;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int KV = p.num_kv_heads;
  __nv_bfloat16* out =
      p.out + (row_of<kRows>(p, s) * p.num_q_heads + g * GROUP + h0) * kHeadDim;
  const int32_t base = p.ws_seq_base[s];
  const int nb = p.ws_seq_base[s + 1] - base;
  if (nb == 0) {
    // an empty context gives a zero row; in a mixed batch nb == 0 means the sequence is not
    // a decode row (or was flagged), and its row is left alone
    if (!kRows)
      for (int e = tid; e < HPC * kHeadDim; e += kMergeThreads) out[e] = __float2bfloat16_rn(0.f);
    return;
  }
  const int64_t total = *p.ws_total;
  const int64_t x0 = static_cast<int64_t>(KV) * (base + static_cast<int64_t>(EXTRA) * s) +
                     static_cast<int64_t>(g) * (nb + EXTRA) + EXTRA;
  const int64_t x1 = x0 + nb;
  const int64_t c_first = run_of(x0, total, p.grid, p.chunk);
  const int64_t c_last = run_of(x1 - 1, total, p.grid, p.chunk);
  if (c_last >= p.grid) {  // tiles beyond the grid (contexts above max_context_len)
    if (tid == 0) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
    return;
  }
  if (c_first == c_last) return;  // written directly by the attention kernel
  const int n = static_cast<int>(c_last - c_first + 1);
  int first_slot = x0 == run_start(c_first, total, p.grid, p.chunk) ? 0 : 1;
  if (EXTRA > 0) first_slot = 1;  // the weighted kernel's rule

  auto record = [&](int k, int h) -> const float* {
    const int64_t c = c_first + k;
    const int slot = k == 0 ? first_slot : 0;
    return p.partials + ((c * 2 + slot) * GROUP + h0 + h) * kPartialFloats;
  };
  // With at least one tile per run (the usual case) no run is empty and the test is skipped.
  const bool maybe_empty = total < p.grid;
  auto empty_run = [&](int k) -> bool {
    if (!maybe_empty) return false;
    const int64_t c = c_first + k;
    return run_start(c, total, p.grid, p.chunk) == run_start(c + 1, total, p.grid, p.chunk);
  };

  float M[HPC], L[HPC];
  float2 A[HPC];
#pragma unroll
  for (int h = 0; h < HPC; ++h) {
    M[h] = -INFINITY;
    L[h] = 0.f;
    A[h] = make_float2(0.f, 0.f);
  }
  // Each warp takes U partials per round and issues all their loads before combining them,
  // so a round costs one memory latency.
  for (int k0 = warp * U; k0 < n; k0 += kWarps * U) {
    float mk[U][HPC], lk[U][HPC];
    float2 vk[U][HPC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u;
      const bool use = k < n && !empty_run(k);
#pragma unroll
      for (int h = 0; h < HPC; ++h) {
        if (use) {
          const float* r = record(k, h);
          mk[u][h] = r[kHeadDim];
          lk[u][h] = r[kHeadDim + 1];
          vk[u][h] = *reinterpret_cast<const float2*>(r + 2 * lane);
        } else {
          mk[u][h] = -INFINITY;
          lk[u][h] = 0.f;
          vk[u][h] = make_float2(0.f, 0.f);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < HPC; ++h) {
      float mu = mk[0][h];
#pragma unroll
      for (int u = 1; u < U; ++u) mu = fmaxf(mu, mk[u][h]);
      const float nm = fmaxf(M[h], mu);
      if (nm == -INFINITY) continue;  // nothing of this head loaded yet
      const float keep = M[h] == -INFINITY ? 0.f : fast_exp2(M[h] - nm);
      L[h] *= keep;
      A[h].x *= keep;
      A[h].y *= keep;
      M[h] = nm;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float wgt = mk[u][h] == -INFINITY ? 0.f : fast_exp2(mk[u][h] - nm);
        L[h] += wgt * lk[u][h];
        A[h].x += wgt * vk[u][h].x;
        A[h].y += wgt * vk[u][h].y;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < HPC; ++h) {
    red_o[warp][h][2 * lane] = A[h].x;
    red_o[warp][h][2 * lane + 1] = A[h].y;
    if (lane == 0) {
      red_m[warp][h] = M[h];
      red_l[warp][h] = L[h];
    }
  }
  __syncthreads();
  for (int e = tid; e < HPC * kHeadDim; e += kMergeThreads) {
    const int h = e / kHeadDim;
    const int d = e % kHeadDim;
    float gm = -INFINITY;
    for (int w = 0; w < kWarps; ++w) gm = fmaxf(gm, red_m[w][h]);
    float o = 0.f, lsum = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      if (red_m[w][h] == -INFINITY) continue;  // a warp without partials
      const float wgt = fast_exp2(red_m[w][h] - gm);
      o += wgt * red_o[w][h][d];
      lsum += wgt * red_l[w][h];
    }
    out[e] = __float2bfloat16_rn(o / lsum);
  }
}

// The merge kernel behind an attention launch that left its split segments' partials.
template <int GROUP, int EXTRA = 0>
cudaError_t launch_merge(const KParams& p, const DecodePlan& plan, bool rows, cudaStream_t stream) {
  if (plan.merge_split_heads && GROUP > 1) {  // one CTA per query head
    const dim3 mgrid(p.num_kv_heads * GROUP, p.num_seqs);
    if (rows)
      merge_partials_kernel<GROUP, 1, true, EXTRA><<<mgrid, kMergeThreads, 0, stream>>>(p);
    else
      merge_partials_kernel<GROUP, 1, false, EXTRA><<<mgrid, kMergeThreads, 0, stream>>>(p);
  } else {  // one CTA per kv head
    const dim3 mgrid(p.num_kv_heads, p.num_seqs);
    if (rows)
      merge_partials_kernel<GROUP, GROUP, true, EXTRA><<<mgrid, kMergeThreads, 0, stream>>>(p);
    else
      merge_partials_kernel<GROUP, GROUP, false, EXTRA><<<mgrid, kMergeThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

}  // namespace pkv
