// Paged decode attention over the 8-bit pools.
//
// For every sequence s and query head h, out = softmax(scale * q K^T) V over the
// context_lens[s] cached tokens, K = code * key_scale and V = code * value_scale with one
// scale per (block, K/V head).  A tile, the 16 tokens of one (block, head), therefore has one
// scale for its scores and one for its share of the output:
//   s_j = (scale * key_scale) q . code_j        O += value_scale * sum_j p_j code_j
// so codes enter the tensor cores as they are and the scales cost one multiplication per
// score and one per output element and tile.
//
// GB300 design.  HBM-bound: a tile is 1 KiB of K and 1 KiB of V, half the bf16 cache's.  The
// frame is the bf16 decode kernel's: the flattened (sequence, K/V head, block) tiles are cut
// into equal contiguous runs, one per warp of a persistent grid, and each warp streams its run
// through a private ring in shared memory.  Measured, one launch: 4 x 131072 tokens (539 MB)
// 91.2 us, 5.9 TB/s, 0.87 of the measured copy rate; 256 contexts of 1 to 8192 tokens (208 MB)
// 42.6 us, 4.9 TB/s; one of 300 tokens 6.9 us.  What bounds it: the stream of tiles for the
// first; start-up (tables, then tiles), uneven ends of the warps and publishing for the second;
// three dependent memory latencies and the launch for the third.  What differs from the bf16
// kernel:
//   * one plain bulk copy per pool (a tile is contiguous), 4 stages of 2 KiB per warp: 15 MB in
//     flight over the device.  Measured with 3 / 4 / 5 / 6 stages: 4 x 131072 tokens 105.9 /
//     91.3 / 95.1 / 92.6 us, 256 mixed contexts 47.8 / 42.5 / 43.8 / 43.8 (fewer leave the memory
//     idle; with more, the tables, scales and queries read on the way wait behind the tiles);
//   * the split counts a segment as two tiles more than it has, for what a piece costs besides
//     its tiles; pieces meet on their CTA first, then one record per CTA (publish_piece);
//   * a few short contexts get a CTA per segment instead (cta_per_segment);
//   * the two scales of each of the next 32 tiles sit in the lanes' registers, loaded when
//     the first of them is issued, a ring's length before it is consumed;
//   * codes become f16 (cvt.rn.f16x2.e4m3x2, exact: about 43 pairs per clock and SM measured,
//     against 14 for the bit form of bf16), straight into mma.sync m16n8k16 fragments: the
//     order of the dims along K and of the tokens along P V is free, so every lane reads 16
//     (K) or 8 (V) consecutive bytes of a token;
//   * q enters as f16 scaled by a power of two per row so that its largest element lies in
//     [2^13, 2^14): a bf16 significand fits, and elements down to 2^-27 of the largest keep
//     all their bits;
//   * p enters as f16 times 2^7 (at most 2^15 under the lazy maximum), so weights down to
//     2^-31 of the largest survive; half a step of f16, 2^-12, is their rounding.  The value
//     scales carry 2^-15 (a power of two, so exact), which keeps the sums of p V at the size of
//     the values: they would pass fp32's range 2^15 earlier otherwise.
#include <math.h>

#include "common.cuh"
#include "decode_common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 12;   // streaming warps per CTA, one CTA per SM
constexpr int kStages = 4;   // ring depth per warp: 8 KiB in flight (figures above)
constexpr int kStageBytes = 2 * kQ8TileBytes;
constexpr int kWindow = 32;  // tiles whose block ids and scales are held in the lanes
// Units (tiles, and kSegmentUnits per segment) a run has at least: 2, against 4, 3000 tokens of
// one sequence 10.3 and 11.6 us, 16 sequences of 200 without a CTA per segment 9.9 and 11.3.
constexpr int kMinUnitsPerRun = 2;
// What a piece costs besides its tiles, in tiles: with 1 / 2 / 3, 256 mixed contexts take 44.6 /
// 42.5 / 43.0 us, 200 of up to 64000 tokens 126.8 / 124.6 / 125.0.
constexpr int kSegmentUnits = 2;
// Tiles that a CTA per segment may cost the longest one's warps (cta_per_segment).  With such
// CTAs, and without: one sequence of 300 tokens 6.9 and 9.6 us, 16 of 200 7.3 and 10.2, 16 of
// 1500 11.6 and 15.0; 7 tiles of slack instead of 5 lose on 4 x 1500 tokens (11.0 us against
// 10.4), 4 lose on 8 x 1500 (11.9 against 11.1).
constexpr int kOwnCtaSlack = 5;
constexpr float kPShift = 7.f;                // log2 of the factor on p
constexpr float kVFactor = 1.f / 32768.f;     // 2^-(kPShift + 8): on the value scales, and on l
static_assert(kStages <= kWindow, "a window's scales are loaded a ring's length ahead");

struct Q8Params {
  const float* key_scale;
  const float* value_scale;
  int32_t max_context_len;  // contexts above it are reported
};

// D (+)= A B for A with rows 8-15 zero, f16 in, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0,
                                             uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1), "f"(0.f));
}

// Two consecutive tiles a and b of a segment (32 tokens).  Lane (r = lane / 4, q = lane % 4):
// MMA row r is query head r of the group (rows past it are zero).  Along the dims, MMA step j
// takes dims 16q + 4j .. + 3 of lane q, for K and Q alike; output n-tile j holds dims 16q + j
// and 16q + 8 + j of head r.  m is the running reference maximum (log2 units, raised only when
// a score exceeds it by more than 2^8), l this lane's share of the sum of p; p, l and o all
// carry 2^kPShift.  MASK: only the first `valid` tokens count; the rest may hold anything.
template <bool MASK>
__device__ __forceinline__ void attend_pair(const uint8_t* ta, const uint8_t* tb, int r, int q,
                                            int valid, const float (&xs)[2], const float (&vs)[2],
                                            const uint32_t (&qa0)[4], const uint32_t (&qa2)[4],
                                            float& m, float& l, float2 (&o)[8]) {
  const int t0 = q8_token_of(2 * q);
  const int k_off = q8_token_of(r) * kQ8RowBytes + 16 * q;
  const int v_off = kQ8TileBytes + t0 * kQ8RowBytes + 8 * r;
  uint2 v[2][4];  // tokens t0, t0 + 2, t0 + 8, t0 + 10 of each tile, codes of dims 8r .. 8r + 7
  float x[2][4];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const uint8_t* tile = t ? tb : ta;
    const uint4 k0 = lds128(tile + k_off);
    const uint4 k1 = lds128(tile + k_off + 8 * kQ8RowBytes);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[t][i] = *reinterpret_cast<const uint2*>(tile + v_off + (2 * (i & 1) + 8 * (i >> 1)) * kQ8RowBytes);
    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
    float s0[4], s1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t a, b, c, d;
      codes4_to_half2x2(w0[j], a, b);
      codes4_to_half2x2(w1[j], c, d);
      if (j == 0) {
        mma_f16_zero(s0, qa0[j], qa2[j], a, b);
        mma_f16_zero(s1, qa0[j], qa2[j], c, d);
      } else {
        mma_f16(s0, qa0[j], qa2[j], a, b);
        mma_f16(s1, qa0[j], qa2[j], c, d);
      }
    }
    x[t][0] = s0[0] * xs[t];
    x[t][1] = s0[1] * xs[t];
    x[t][2] = s1[0] * xs[t];
    x[t][3] = s1[1] * xs[t];
    if (MASK) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (16 * t + t0 + 2 * (i & 1) + 8 * (i >> 1) >= valid) {
          x[t][i] = -INFINITY;
          v[t][i] = make_uint2(0u, 0u);
        }
      }
    }
  }
  float mt = fmaxf(max3f(x[0][0], x[0][1], x[0][2]), max3f(x[0][3], x[1][0], x[1][1]));
  mt = max3f(mt, x[1][2], x[1][3]);
  mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
  mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
  const bool grow = mt - m > kRescaleThreshold;  // first pair: m = -inf
  if (__any_sync(0xffffffffu, grow)) {
    const float alpha = grow ? fast_exp2(m - mt) : 1.f;
    if (grow) m = mt;
    l *= alpha;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[j].x *= alpha;
      o[j].y *= alpha;
    }
  }
  const float ref = m - kPShift;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float p0 = fast_exp2(x[t][0] - ref), p1 = fast_exp2(x[t][1] - ref);
    const float p2 = fast_exp2(x[t][2] - ref), p3 = fast_exp2(x[t][3] - ref);
    l += (p0 + p1) + (p2 + p3);
    const uint32_t pa0 = pack_half2_rn(p0, p1), pa2 = pack_half2_rn(p2, p3);
    const float2 vs2 = make_float2(MASK && t == 1 && valid <= kBlockSize ? 0.f : vs[t],
                                   MASK && t == 1 && valid <= kBlockSize ? 0.f : vs[t]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = h ? v[t][0].y : v[t][0].x, b = h ? v[t][1].y : v[t][1].x;
      const uint32_t c = h ? v[t][2].y : v[t][2].x, d = h ? v[t][3].y : v[t][3].x;
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // bytes 2u, 2u + 1 of both tokens, interleaved
        uint32_t b00, b01, b10, b11;
        codes4_to_half2x2(__byte_perm(a, b, u ? 0x7362 : 0x5140), b00, b01);
        codes4_to_half2x2(__byte_perm(c, d, u ? 0x7362 : 0x5140), b10, b11);
        float acc[4];
        const int j = 4 * h + 2 * u;
        mma_f16_zero(acc, pa0, pa2, b00, b10);
        o[j] = __ffma2_rn(make_float2(acc[0], acc[1]), vs2, o[j]);
        mma_f16_zero(acc, pa0, pa2, b01, b11);
        o[j + 1] = __ffma2_rn(make_float2(acc[0], acc[1]), vs2, o[j + 1]);
      }
    }
  }
}

// Splits weighted by segment: every (sequence, kv head) segment counts kSegmentUnits units on top of its
// tiles (what starting and publishing a piece costs, in tiles), kSegmentUnits also where it has none,
// and the runs divide the units evenly.  Units of sequence s start at unit_base(s), those of its
// segment g at + g (nb + kSegmentUnits), its tiles' at + kSegmentUnits.
__device__ __forceinline__ int64_t unit_base(const int32_t* base, int s, int kv) {
  return static_cast<int64_t>(kv) * (static_cast<int64_t>(base[s]) + static_cast<int64_t>(kSegmentUnits) * s);
}

// A piece's partial: per query head 64 floats of o, the maximum (log2 units) and the sum,
// padded to 16 bytes.
constexpr int kRecordFloats = kHeadDim + 4;

// Folds n records of GROUP heads into (M, L) per head and acc, of dims 4 (lane % 16) .. + 3:
// record k (k > 0) is at rec0 + k * step, record 0 at rec0 + off0.  Half warps take every other
// record's rows, eight records a round.
template <int GROUP>
__device__ __forceinline__ void fold_records(const float* rec0, int64_t off0, int64_t step, int n,
                                             int lane, float (&M)[GROUP], float (&L)[GROUP],
                                             float4 (&acc)[GROUP]) {
  const int hw = lane >> 4;
  auto record = [&](int k) { return rec0 + (k == 0 ? off0 : k * step); };
  float4 v[4][GROUP];
  auto load_rows = [&](int k0, int last) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* r = record(min(k0 + 2 * u + hw, last));
#pragma unroll
      for (int h = 0; h < GROUP; ++h)
        v[u][h] = *reinterpret_cast<const float4*>(r + h * kRecordFloats + 4 * (lane & 15));
    }
  };
#pragma unroll
  for (int h = 0; h < GROUP; ++h) {
    M[h] = -INFINITY;
    L[h] = 0.f;
    acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += 32) {  // lane k weighs record k0 + k
    const int cnt = min(32, n - k0);
    load_rows(k0, n - 1);
    const float* mine = record(k0 + min(lane, cnt - 1));
    float2 ml[GROUP];
    float wk[GROUP];
#pragma unroll
    for (int h = 0; h < GROUP; ++h)
      ml[h] = *reinterpret_cast<const float2*>(mine + h * kRecordFloats + kHeadDim);
#pragma unroll
    for (int h = 0; h < GROUP; ++h) {
      float nm = ml[h].x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
      nm = fmaxf(nm, M[h]);
      const float keep = k0 == 0 ? 0.f : fast_exp2(M[h] - nm);
      wk[h] = lane < cnt ? fast_exp2(ml[h].x - nm) : 0.f;
      float lw = wk[h] * ml[h].y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, d);
      L[h] = L[h] * keep + lw;
      acc[h].x *= keep;
      acc[h].y *= keep;
      acc[h].z *= keep;
      acc[h].w *= keep;
      M[h] = nm;
    }
#pragma unroll 1
    for (int j0 = 0; j0 < cnt; j0 += 8) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + 2 * u + hw;
#pragma unroll
        for (int h = 0; h < GROUP; ++h) {
          float w = __shfl_sync(0xffffffffu, wk[h], j & 31);
          if (j >= cnt) w = 0.f;
          acc[h].x += w * v[u][h].x;
          acc[h].y += w * v[u][h].y;
          acc[h].z += w * v[u][h].z;
          acc[h].w += w * v[u][h].w;
        }
      }
      if (j0 + 8 < cnt) load_rows(k0 + j0 + 8, n - 1);
    }
  }
#pragma unroll
  for (int h = 0; h < GROUP; ++h) {  // the two half warps' shares
    acc[h].x += __shfl_xor_sync(0xffffffffu, acc[h].x, 16);
    acc[h].y += __shfl_xor_sync(0xffffffffu, acc[h].y, 16);
    acc[h].z += __shfl_xor_sync(0xffffffffu, acc[h].z, 16);
    acc[h].w += __shfl_xor_sync(0xffffffffu, acc[h].w, 16);
  }
}

// Where the partial of a split segment's piece goes, and how its pieces meet: those of one CTA
// (its runs are consecutive) in shared memory, the CTAs' records in the workspace.
struct Meeting {
  int c_first;  // the segment's first run
  int n_cta;    // CTAs it spans
  int lo;       // this CTA's first run of it, and how many there are
  int n_here;
};

__device__ __forceinline__ Meeting meeting_of(const int32_t* seq_base, int KV, const Piece& pc,
                                              int64_t units, int runs, bool own) {
  const int here = static_cast<int>(blockIdx.x) * kWarps;
  if (own) return {here, 1, here, min(pc.nb, kWarps)};
  const int64_t x0 = unit_base(seq_base, pc.s, KV) +
                     static_cast<int64_t>(pc.g) * (pc.nb + kSegmentUnits) + kSegmentUnits;
  Meeting m;
  m.c_first = static_cast<int>(run_of(x0, units, runs, 0));
  const int c_last = static_cast<int>(run_of(x0 + pc.nb - 1, units, runs, 0));
  m.n_cta = c_last / kWarps - m.c_first / kWarps + 1;
  m.lo = max(m.c_first, here);
  m.n_here = min(c_last, here + kWarps - 1) - m.lo + 1;
  return m;
}

// Record of run c: a run writes at most two partials, of the segment that it begins inside
// (slot 0) and of the one that begins in it and goes on in the next run (slot 1).
template <int GROUP>
__device__ __forceinline__ int64_t record_of(int64_t c, bool begins) {
  return (c * 2 + (begins ? 1 : 0)) * GROUP * kRecordFloats;
}

// Publishes a piece whose partial this warp has written.  (One meeting of all pieces by the last
// warp cost 0.15 us per piece: one sequence of 8000 tokens, 228 pieces per segment, 44 us against
// 12; a merge kernel behind the attention cost 200 sequences of up to 16000 tokens 105 us against
// 86.)  The last of a CTA's pieces folds them
// into one record; the last CTA folds the CTAs' records and writes the rows.  A segment within
// one CTA is done after the first meeting.  Serial work per segment is thus a dozen records in
// shared memory and one per CTA, however long the context, and no second kernel is needed.  The
// order of the sums is that of the runs, whoever comes last.
template <int GROUP>
__device__ __forceinline__ void publish_piece(const KParams& p, const Meeting& m, const float* local,
                                              int* cta_seg_count, int s, int g, int lane) {
  const int here = static_cast<int>(blockIdx.x) * kWarps;
#pragma unroll 1
  for (int level = m.n_here > 1 ? 0 : 1; level < 2; ++level) {
    int last = 0;
    if (level == 0) {
      // two segments with two runs each on this CTA never share the first of them
      int* count = &cta_seg_count[m.lo - here];
      __threadfence_block();
      __syncwarp();
      if (lane == 0) {
        last = atomicAdd(count, 1) == m.n_here - 1;
        if (last) *count = 0;
      }
    } else {
      // by the segment's first CTA: only one segment goes on past a CTA's last run
      int32_t* count = &p.seg_count[m.c_first / kWarps];
      __threadfence();
      __syncwarp();
      if (lane == 0) {
        last = atomicAdd(count, 1) == m.n_cta - 1;
        if (last) *count = 0;  // ready for the next call
      }
    }
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    if (level == 0) __threadfence_block(); else __threadfence();
    // (plain loads: the fence orders them after the counts of the records' writers)
    float M[GROUP], L[GROUP];
    float4 acc[GROUP];
    const int64_t run_step = record_of<GROUP>(1, false);
    if (level == 0)
      fold_records<GROUP>(local + (m.lo - here) * run_step, m.lo == m.c_first ? run_step / 2 : 0, run_step,
                          m.n_here, lane, M, L, acc);
    else
      fold_records<GROUP>(p.partials + m.c_first / kWarps * kWarps * run_step,
                          m.c_first % kWarps * run_step + run_step / 2, kWarps * run_step, m.n_cta, lane, M,
                          L, acc);
    if (level == 1 || m.n_cta == 1) {
      if (lane < 16) {
#pragma unroll
        for (int h = 0; h < GROUP; ++h) {
          const float inv = 1.f / L[h];
          __nv_bfloat16* out = p.out + (static_cast<int64_t>(s) * p.num_q_heads + g * GROUP + h) * kHeadDim;
          *reinterpret_cast<uint2*>(out + 4 * lane) =
              make_uint2(pack_bf16x2(acc[h].x * inv, acc[h].y * inv), pack_bf16x2(acc[h].z * inv, acc[h].w * inv));
        }
      }
      return;
    }
    float* rec = p.partials + record_of<GROUP>(m.lo, m.lo == m.c_first);
#pragma unroll
    for (int h = 0; h < GROUP; ++h) {
      if (lane < 16) *reinterpret_cast<float4*>(rec + h * kRecordFloats + 4 * lane) = acc[h];
      if (lane == 16) *reinterpret_cast<float2*>(rec + h * kRecordFloats + kHeadDim) = make_float2(M[h], L[h]);
    }
  }
}

// Whether every segment gets a CTA of its own, whose warps share its tiles: all pieces then meet
// in shared memory.  For batches of no more segments than CTAs in which that costs the longest
// segment's warps at most kOwnCtaSlack tiles more than the even split would give them.
__device__ __forceinline__ bool cta_per_segment(const KParams& p, const int32_t* seq_base, int64_t units,
                                                int lane) {
  if (static_cast<int64_t>(p.num_seqs) * p.num_kv_heads * kWarps > p.grid) return false;
  int most = 0;
  for (int s = lane; s < p.num_seqs; s += 32) most = max(most, seq_base[s + 1] - seq_base[s]);
  most = __reduce_max_sync(0xffffffffu, most);
  return static_cast<int64_t>(most) * p.grid <= (units + static_cast<int64_t>(kOwnCtaSlack) * p.grid) * kWarps;
}

template <int GROUP>
__global__ void __launch_bounds__(kWarps * 32, 1)
paged_decode_q8_kernel(const __grid_constant__ KParams p, const Q8Params sp8) {
  constexpr int kThreads = kWarps * 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x;
  // (through a shuffle, so that what depends on it stays in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int lane = tid & 31;
  const int S = p.num_seqs;
  const int KV = p.num_kv_heads;

  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * kStages * kStageBytes);
  uint64_t* full_bar = bars + warp * kStages;
  float* local = reinterpret_cast<float*>(bars + kWarps * kStages);  // [warp][2][GROUP] records
  int32_t* seq_base = reinterpret_cast<int32_t*>(local + record_of<GROUP>(kWarps, false));
  __shared__ int64_t warp_sums[kWarps];
  // piece counters of split segments whose pieces all run on this CTA, by the segment's
  // first run modulo kWarps (two such segments never share a first run)
  __shared__ int cta_seg_count[kWarps];
  if (tid < kWarps) cta_seg_count[tid] = 0;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full_bar[i], 1);
    fence_barrier_init();
  }
  // query rows are read in the middle of a stream: into L2 now
  {
    const int64_t q_rows = static_cast<int64_t>(S) * p.num_q_heads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + tid; i < q_rows;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      prefetch_l2(reinterpret_cast<const uint8_t*>(p.q) + i * kRowBytes);
  }
  block_prefix<kWarps, false>(p, seq_base, warp_sums);

  // From here on every warp works alone, on one run: the plan never makes more runs than
  // the grid has warps.
  const int gw = blockIdx.x * kWarps + warp;
  const int64_t units = unit_base(seq_base, S, KV);
  const bool own = cta_per_segment(p, seq_base, units, lane);
  const int runs = own ? S * KV * kWarps
                       : static_cast<int>(max(int64_t{1}, min(static_cast<int64_t>(p.grid), units / kMinUnitsPerRun)));
  if (gw >= runs) return;
  const uint64_t policy = l2_evict_first_policy();
  const int r = lane >> 2;
  const int q = lane & 3;
  // The run's tiles: lane 0 locates its first unit, lane 1 the next run's, in one search.
  // (block_prefix keeps the tile count below 2^31, so units fit 32 unsigned bits.)
  int start, stop;
  int wc_s, wc_off;  // sequence of tile wc_y and its place among the sequence's KV x nb tiles
  if (own) {
    wc_s = static_cast<int>(blockIdx.x) / KV;
    const int nb = seq_base[wc_s + 1] - seq_base[wc_s];
    const int d = max(1, min(nb, kWarps));  // warps with tiles
    wc_off = (static_cast<int>(blockIdx.x) % KV) * nb;
    start = seq_base[wc_s] * KV + wc_off;
    stop = start + min(warp + 1, d) * nb / d;
    start += min(warp, d) * nb / d;
    wc_off += min(warp, d) * nb / d;
  } else {
    const uint32_t u32 = static_cast<uint32_t>(units), n = static_cast<uint32_t>(runs);
    const uint32_t c = static_cast<uint32_t>(gw + (lane & 1));
    const uint32_t each = u32 / n;
    // c * units / n without 64 bits (n stays below 2^16)
    const uint32_t y = c * each + c * (u32 - each * n) / n;
    auto units_before = [&](int s) {  // of sequence s
      return static_cast<uint32_t>(KV) * static_cast<uint32_t>(seq_base[s] + kSegmentUnits * s);
    };
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (units_before(mid) <= y) lo = mid; else hi = mid - 1;
    }
    const int nb = seq_base[lo + 1] - seq_base[lo];
    const int off = static_cast<int>(y - units_before(lo));
    int g = off / (nb + kSegmentUnits);
    int place = g * nb + max(0, off - g * (nb + kSegmentUnits) - kSegmentUnits);
    if (g >= KV) place = KV * nb;  // past the last unit
    const int t = seq_base[lo] * KV + place;
    start = __shfl_sync(0xffffffffu, t, 0);
    stop = __shfl_sync(0xffffffffu, t, 1);
    wc_s = __shfl_sync(0xffffffffu, lo, 0);
    wc_off = __shfl_sync(0xffffffffu, place, 0);
  }
  // past the end of its sequence, a place moves to the next one that has tiles
  auto settle = [&](int& s, int& off) {
    while (s + 1 < S && off >= (seq_base[s + 1] - seq_base[s]) * KV) {
      off = 0;
      ++s;
    }
  };
  settle(wc_s, wc_off);
  Piece nx;  // the first piece
  nx.s = wc_s;
  nx.nb = max(1, seq_base[wc_s + 1] - seq_base[wc_s]);
  nx.g = wc_off / nx.nb;
  nx.b0 = wc_off - nx.g * nx.nb;
  nx.b1 = min(nx.nb, nx.b0 + stop - start);

  // ---- issue side: windows of 32 tiles of the run ----
  int wc_y = start;
  auto next_window = [&]() -> Window {
    Window w;
    w.tile = 0;
    w.g = 0;
    w.n = min(stop - wc_y, kWindow);
    int s = wc_s, off = wc_off + lane;
    if (lane < w.n) {
      if (off >= (seq_base[s + 1] - seq_base[s]) * KV) {
        s = find_seq(seq_base, S, wc_y + lane, KV);
        off = wc_y + lane - seq_base[s] * KV;
      }
      const int nb = seq_base[s + 1] - seq_base[s];
      w.g = off / nb;
      w.tile = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + off - w.g * nb);
    }
    if (w.n > 0) {
      wc_y += w.n;
      wc_s = __shfl_sync(0xffffffffu, s, w.n - 1);
      wc_off = __shfl_sync(0xffffffffu, off, w.n - 1) + 1;
      settle(wc_s, wc_off);
    }
    return w;
  };
  // Scales of the window whose tiles are consumed (cur_*) and of the one being issued (nxt_*).
  // A run's windows are 32 tiles each but its last, so tile i of the run is entry i % 32 of
  // window i / 32 on both sides; the issue side is at most one window ahead.
  float cur_ks = 0.f, cur_vs = 0.f, nxt_ks = 0.f, nxt_vs = 0.f;
  auto resolve_window = [&](Window& w) {
    const bool bad = lane < w.n && (w.tile < 0 || w.tile >= p.num_blocks);
    const bool live = lane < w.n && !bad;
    w.tile = live ? w.tile * KV + w.g : -1;
    nxt_ks = live ? __ldg(sp8.key_scale + w.tile) : 0.f;
    nxt_vs = live ? __ldg(sp8.value_scale + w.tile) * kVFactor : 0.f;
    if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(p.status, PA_DEVFLAG_BAD_BLOCK);
  };
  Window cur = next_window();
  Window nxt = next_window();
  resolve_window(cur);
  int cur_i = 0;
  int issued = 0;
  // Lane `slot` (0 or 1) requests tile t into the ring's stage issued + slot.
  auto request = [&](int32_t t, int slot) {
    const int st = (issued + slot) % kStages;
    if (t >= 0) {
      mbar_arrive_expect_tx(&full_bar[st], kStageBytes);
      uint8_t* dst = ring + st * kStageBytes;
      const int64_t off = static_cast<int64_t>(t) * kQ8TileBytes;
      bulk_load(dst, p.key_cache + off, kQ8TileBytes, &full_bar[st], policy);
      bulk_load(dst + kQ8TileBytes, p.value_cache + off, kQ8TileBytes, &full_bar[st], policy);
    } else {
      mbar_arrive(&full_bar[st]);  // invalid block: release the stage with stale data
    }
  };
  // Requests the next n (1 or 2) tiles of the run, as far as there are any.
  auto issue = [&](int n) {
    if (cur_i + n <= cur.n) {
      const int32_t t = __shfl_sync(0xffffffffu, cur.tile, cur_i + (n - 1 & lane));
      if (lane < n) request(t, lane);
      issued += n;
      cur_i += n;
      return;
    }
#pragma unroll 1
    for (; n > 0; --n) {
      if (cur_i >= cur.n) {
        cur = nxt;
        cur_i = 0;
        if (cur.n == 0) return;  // nothing left
        resolve_window(cur);
        nxt = next_window();
      }
      const int32_t t = __shfl_sync(0xffffffffu, cur.tile, cur_i);
      if (lane == 0) request(t, 0);
      ++issued;
      ++cur_i;
    }
  };
  {  // the ring's first fill, one lane per stage (a first window below 32 tiles is the only one)
    const int n0 = cur.n < kStages ? cur.n : kStages;
    if (lane < n0) request(cur.tile, lane);
    issued = cur_i = n0;
  }
  // Everything above reads only block tables, contexts, scales and codes; queries are read and
  // anything written only after the previous kernel in the stream has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  {
    // empty contexts: zero rows (no tile writes them); others against the caller's bound; a sequence
    // per warp of the grid (the bound tested piece by piece: 256 mixed contexts 42.6 us against 42.4)
    const int row_elems = p.num_q_heads * kHeadDim;
    for (int s0 = gw; s0 < S; s0 += runs) {
      if (seq_base[s0 + 1] != seq_base[s0]) {
        if (lane == 0 && p.context_lens[s0] > sp8.max_context_len) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
        continue;
      }
      __nv_bfloat16* out = p.out + static_cast<int64_t>(s0) * row_elems;
      for (int e = lane; e < row_elems; e += 32) out[e] = __float2bfloat16_rn(0.f);
    }
  }

  // ---- consume side: piece by piece ----
  // This lane's 16 dims of query head r of a piece (lanes past the group take the last head's
  // and drop them).
  auto query_of = [&](int s, int g) {
    return reinterpret_cast<const uint4*>(
        p.q + (static_cast<int64_t>(s) * p.num_q_heads + g * GROUP + min(r, GROUP - 1)) * kHeadDim) + 2 * q;
  };
  int waited = 0;  // tiles whose data this warp has waited for
  bool ok = true;
  for (int y = start; y < stop;) {
    const Piece pc = nx;
    const int32_t L = __ldg(p.context_lens + pc.s);
    const uint4 qx = __ldg(query_of(pc.s, pc.g)), qy = __ldg(query_of(pc.s, pc.g) + 1);
    const bool whole = pc.b0 == 0 && pc.b1 == pc.nb;
    const int ntiles = pc.b1 - pc.b0;
    const int left = stop - y - ntiles;
    if (left > 0) {  // the next head of this sequence, or the next sequence that has tokens
      if (++nx.g == KV) {
        nx.g = 0;
        do {
          ++nx.s;
          nx.nb = seq_base[nx.s + 1] - seq_base[nx.s];
        } while (nx.nb == 0);
      }
      nx.b0 = 0;
      nx.b1 = min(nx.nb, left);
    }

    // The query, to f16 under the row's power of two.
    uint32_t qa0[4], qa2[4];
    float row_scale = p.q_scale;
    {
      const uint32_t w[8] = {qx.x, qx.y, qx.z, qx.w, qy.x, qy.y, qy.z, qy.w};
      const bool real = r < GROUP;
      uint32_t big = 0u;  // largest magnitude as bits (a NaN's bits exceed infinity's)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        big = max(big, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const int shift = query_shift(big);
      const float up = power_of_two(shift);
      row_scale *= power_of_two(-shift);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = bf16x2_to_float2(w[2 * j]), b = bf16x2_to_float2(w[2 * j + 1]);
        qa0[j] = real ? pack_half2_rn(a.x * up, a.y * up) : 0u;
        qa2[j] = real ? pack_half2_rn(b.x * up, b.y * up) : 0u;
      }
    }
    float m = -INFINITY, l = 0.f;
    float2 o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = make_float2(0.f, 0.f);

    const int full = min(ntiles, L / kBlockSize - pc.b0);  // tiles without a masked token
#pragma unroll 1
    for (int k = ok ? 0 : ntiles; k < ntiles;) {
      if ((waited & (kWindow - 1)) == 0) {
        cur_ks = nxt_ks;
        cur_vs = nxt_vs;
      }
      // Pairs of full tiles whose scales and refills come from the windows at hand: the tight
      // loop, without a test but for the data.
      const int before = waited;
      int pairs = min(min(full - k, kWindow - (waited & (kWindow - 1))), cur.n - cur_i) >> 1;
#pragma unroll 1
      for (; pairs > 0; --pairs) {
        const int sa = waited % kStages, sb = (waited + 1) % kStages;
        const int w = waited & (kWindow - 1);
        const float xs[2] = {row_scale * __shfl_sync(0xffffffffu, cur_ks, w),
                             row_scale * __shfl_sync(0xffffffffu, cur_ks, w + 1)};
        const float vs[2] = {__shfl_sync(0xffffffffu, cur_vs, w), __shfl_sync(0xffffffffu, cur_vs, w + 1)};
        const int32_t t = __shfl_sync(0xffffffffu, cur.tile, cur_i + (lane & 1));
        bool here = mbar_wait(&full_bar[sa], static_cast<uint32_t>((waited / kStages) & 1));
        here &= mbar_wait(&full_bar[sb], static_cast<uint32_t>(((waited + 1) / kStages) & 1));
        if (!__all_sync(0xffffffffu, here)) {
          ok = false;  // (the pieces left are published without their tiles)
          break;
        }
        attend_pair<false>(ring + sa * kStageBytes, ring + sb * kStageBytes, r, q, 2 * kBlockSize, xs, vs,
                           qa0, qa2, m, l, o);
        // Every lane's reads of these stages have completed (their values fed the arithmetic
        // above); the warp barrier orders them before the refills.
        __syncwarp();
        if (lane < 2) request(t, lane);
        issued += 2;
        cur_i += 2;
        waited += 2;
        k += 2;
      }
      if (!ok || k >= ntiles) break;
      if (waited != before && (waited & (kWindow - 1)) == 0) continue;  // the next window's scales first
      // One pair, or a single tile, with everything that can happen at an edge.
      const bool two = k + 1 < ntiles;
      const int sa = waited % kStages, sb = (waited + 1) % kStages;
      float xs[2], vs[2];
      xs[0] = row_scale * __shfl_sync(0xffffffffu, cur_ks, waited & (kWindow - 1));
      vs[0] = __shfl_sync(0xffffffffu, cur_vs, waited & (kWindow - 1));
      if (two && ((waited + 1) & (kWindow - 1)) == 0) {
        cur_ks = nxt_ks;
        cur_vs = nxt_vs;
      }
      xs[1] = row_scale * __shfl_sync(0xffffffffu, cur_ks, (waited + 1) & (kWindow - 1));
      vs[1] = __shfl_sync(0xffffffffu, cur_vs, (waited + 1) & (kWindow - 1));
      bool here = mbar_wait(&full_bar[sa], static_cast<uint32_t>((waited / kStages) & 1));
      if (two)
        here &= mbar_wait(&full_bar[sb], static_cast<uint32_t>(((waited + 1) / kStages) & 1));
      if (!__all_sync(0xffffffffu, here)) {
        ok = false;
        break;
      }
      const uint8_t* ta = ring + sa * kStageBytes;
      const int valid = L - (pc.b0 + k) * kBlockSize;
      attend_pair<true>(ta, two ? ring + sb * kStageBytes : ta, r, q, two ? valid : min(valid, kBlockSize),
                        xs, vs, qa0, qa2, m, l, o);
      __syncwarp();
      const int n = two ? 2 : 1;
      waited += n;
      k += n;
      issue(n);
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    l *= kVFactor;  // as o, through the value scales
    Meeting meet = {};
    if (!whole) meet = meeting_of(seq_base, KV, pc, units, runs, own);
    if (r < GROUP) {
      if (whole) {
        const float inv = 1.f / l;
        const int64_t row = static_cast<int64_t>(pc.s) * p.num_q_heads + pc.g * GROUP + r;
        uint4* dst = reinterpret_cast<uint4*>(p.out + row * kHeadDim + 16 * q);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = pack_bf16x2(o[2 * j].x * inv, o[2 * j + 1].x * inv);
          w[4 + j] = pack_bf16x2(o[2 * j].y * inv, o[2 * j + 1].y * inv);
        }
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        const bool begins = pc.b0 == 0;
        float* dst = (meet.n_here > 1 ? local + record_of<GROUP>(warp, begins)
                                      : p.partials + record_of<GROUP>(gw, begins)) + r * kRecordFloats;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          *reinterpret_cast<float2*>(dst + 16 * q + 2 * j) = make_float2(o[2 * j].x, o[2 * j + 1].x);
          *reinterpret_cast<float2*>(dst + 16 * q + 8 + 2 * j) = make_float2(o[2 * j].y, o[2 * j + 1].y);
        }
        if (q == 0) *reinterpret_cast<float2*>(dst + kHeadDim) = make_float2(m, l);
      }
    }
    if (!whole) publish_piece<GROUP>(p, meet, local, cta_seg_count, pc.s, pc.g, lane);
    y += ntiles;
  }
  // After a timeout, leave no copy in flight into this warp's ring (bounded waits).
  if (!ok && lane == 0) {
    flag_error(p.status, PA_DEVFLAG_TIMEOUT);
    for (int t = waited; t < issued; ++t) {
      if (!mbar_wait(&full_bar[t % kStages], static_cast<uint32_t>((t / kStages) & 1))) break;
    }
  }
}

size_t smem_bytes(int num_seqs, int group) {
  return static_cast<size_t>(kWarps) * kStages * (kStageBytes + sizeof(uint64_t)) +
         static_cast<size_t>(kWarps) * 2 * group * kRecordFloats * sizeof(float) +
         sizeof(int32_t) * (num_seqs + 1);
}

template <int GROUP>
cudaError_t prepare_kernel() {
  static bool done[kMaxDevices] = {};  // benign race: the attribute calls are idempotent
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(paged_decode_q8_kernel<GROUP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem_bytes(kMaxSeqs, GROUP)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_decode_q8_kernel<GROUP>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
  return e;
}

template <int GROUP>
cudaError_t launch(const AttendQ8Args& a, const DecodePlan& plan, void* workspace,
                   bool overlap_previous, cudaStream_t stream) {
  cudaError_t e = prepare_kernel<GROUP>();
  if (e != cudaSuccess) return e;
  KParams p = {};
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.key_cache = static_cast<const uint8_t*>(a.key_cache);
  p.value_cache = static_cast<const uint8_t*>(a.value_cache);
  p.block_tables = a.block_tables;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.context_lens = a.context_lens;
  p.num_seqs = a.num_seqs;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.q_scale = a.scale * 1.4426950408889634f;
  p.grid = plan.runs;
  p.chunk = 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.seg_count = reinterpret_cast<int32_t*>(ws + plan.ws_count_offset);  // [CTAs]
  p.partials = reinterpret_cast<float*>(ws + plan.ws_meta_bytes);
  p.status = a.status;
  const Q8Params s = {a.key_scale, a.value_scale, a.max_context_len};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = plan.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = overlap_previous ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_decode_q8_kernel<GROUP>, p, s);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t plan_decode_q8(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads,
                           int32_t max_context_len, DecodePlan* plan, int32_t max_sms) {
  const int group = num_q_heads / num_kv_heads;
  plan->group = group;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t blocks_max = (static_cast<int64_t>(max_context_len) + kBlockSize - 1) / kBlockSize;
  const int64_t tiles_upper = static_cast<int64_t>(num_seqs) * num_kv_heads * blocks_max;
  // one CTA per SM (the ring takes most of its shared memory)
  const int64_t resident = max_sms > 0 && max_sms < sms ? max_sms : sms;
  int64_t runs = resident * kWarps;
  const int64_t segments = static_cast<int64_t>(num_seqs) * num_kv_heads;
  int64_t by_size = (tiles_upper + segments * kSegmentUnits) / kMinUnitsPerRun;
  if (segments <= resident && by_size < segments * kWarps) by_size = segments * kWarps;  // a CTA each
  if (by_size < runs) runs = by_size;
  if (runs < 1) runs = 1;
  plan->runs = static_cast<int>(runs);
  plan->chunk = 0;
  plan->tile_bound = 0;
  plan->grid = static_cast<int>((runs + kWarps - 1) / kWarps);
  plan->smem_bytes = smem_bytes(num_seqs, group);
  plan->fused_merge = true;
  plan->merge_split_heads = false;
  plan->prefetch_ok = false;
  // A counter per CTA, then the records: neither place nor size depends on the call's sizes, so the
  // counters that every call leaves at zero are the next one's, whatever batch that serves.
  plan->ws_count_offset = 0;
  plan->ws_meta_bytes = (sizeof(int32_t) * sms + 255) / 256 * 256;
  // sized for the whole device, so that any SM budget fits
  const int64_t runs_full = runs > static_cast<int64_t>(sms) * kWarps
                                ? runs : static_cast<int64_t>(sms) * kWarps;
  plan->workspace_bytes = plan->ws_meta_bytes +
                          static_cast<size_t>(runs_full) * 2 * group * kRecordFloats * sizeof(float);
  return cudaSuccess;
}

cudaError_t launch_decode_q8(const AttendQ8Args& a, const DecodePlan& plan, void* workspace,
                             bool overlap_previous, cudaStream_t stream) {
  switch (plan.group) {
    case 1: return launch<1>(a, plan, workspace, overlap_previous, stream);
    case 2: return launch<2>(a, plan, workspace, overlap_previous, stream);
    case 4: return launch<4>(a, plan, workspace, overlap_previous, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
