// Causal chunk attention over the 8-bit pools, on tcgen05 tensor cores.
//
// A sequence appends a chunk of q_len tokens to a context of L tokens (the chunk's own K/V
// stored already); chunk row i sits at position L - q_len + i and attends keys 0 .. L - q_len
// + i, K = code * key_scale and V = code * value_scale with one scale per (block, K/V head).
// For key j of block b, with the value scale written as 2^e f, 1 <= f < 2:
//   x_j = (scale key_scale_b) q . code_j
//   p'_j = 2^(log2e x_j + log2 f_b - m)           (m the running maximum of log2e x)
//   O += sum_j p'_j (2^e_b code_j),   l += sum_b (1 / f_b) sum_{j in b} p'_j,   out = O / l
// so a block's scales cost no work per element: the score factor replaces the constant one,
// f rides in the exponent, and 2^e is exact in the bf16 that V becomes on its way anyway.
// K stays unscaled and becomes f16 (exact, one instruction per two codes); q becomes f16 too,
// each row under a power of two that brings its largest element to [2^13, 2^14).
//
// GB300 design.  The bf16 chunk kernel is held by the chain of issuing and awaiting small MMAs
// (a 64-key tile of 128 rows at a time), so this one makes the tiles four times as large:
//   * A work unit is a pair of query tiles, 2 x 128 MMA rows (256 / GROUP tokens x GROUP heads
//     that share a K/V head), of one sequence; every 128-key K/V tile, converted once, feeds
//     both.  One CTA per SM, persistent, units dealt heaviest first as in the bf16 kernel.
//   * Tensor memory (all 512 columns): scores S of each half 128 columns, P of each half 64,
//     O of each half 64.  P has columns of its own, so the next tile's scores are issued as
//     soon as the row warps have read this tile's into registers.
//   * Warps 0-7 and 8-15: the row warps of the two halves, two threads per row (64 keys each):
//     read S, mask the diagonal tiles, maximum (exchanged between the two), exponentials, P as
//     bf16, row sums in fp32; O is rescaled in place only when a row's maximum grows by more
//     than 2^8.  At a unit's last tile they turn the next unit's Q into f16 in shared memory.
//   * Warps 16-19 (V, to bf16) and 22-23 (K, to f16): converters.  They read a landed tile of
//     codes and write it in the 128-byte-swizzled layout that the MMAs read, into rings of
//     three each.
//   * Warp 20: one elected lane issues S = Q K^T (M128 N128 K64) and O += P V (M128 N64 K128).
//   * Warp 21: four gathering TMA copies per tile (four blocks of one pool each) into a ring of
//     three raw tiles, the blocks' scales beside them by 4-byte asynchronous copies on the same
//     mbarrier; Q by TMA.  (One bulk copy per block and pool took some 1,600 cycles a tile to
//     issue.)
// Measured: 3 chunks of some 4000 rows over 8000 tokens 645 us, 840 TFLOP/s or 0.44 of the measured
// bf16 product rate; 8 chunks of 512 rows 65.7 us (602 TFLOP/s).  Bound: a 128-key tile of both
// halves takes some 2,600 cycles, in which the tensor core works about 1,600 (24 small MMAs, 60
// to 80 cycles each whatever their N) and the row warps about 2,200 (scores from tensor memory
// 190, maximum and its exchange 350 to 500, 64 exponentials a thread with P 1,100, P's store 270);
// the rest is what each waits for the other.  Eight row warps instead of sixteen took 909 us (of
// 831 then).  The heaviest CTA has 5 % more tiles than the average.
// Every mbarrier wait is bounded; on timeout the CTA records PA_DEVFLAG_TIMEOUT, drains its
// own copies and MMAs, frees its tensor memory and returns.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "prefill_plan.cuh"
#include "q8.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kTileM = 128;                       // MMA rows of one half
constexpr int kTileN = 128;                       // keys per K/V tile
constexpr int kBlocksPerTile = kTileN / kBlockSize;
constexpr int kThreads = 768;
constexpr int kRowWarps = 8;                      // per half: four for each half of a tile's keys
constexpr int kRowThreads = 2 * kRowWarps * 32;
constexpr int kVWarps = 4, kKWarps = 2;           // converters
constexpr int kVWarp0 = 16, kMmaWarp = 20, kProducerWarp = 21, kKWarp0 = 22;
constexpr int kRing = 3;                          // stages of each of the three rings
constexpr int kConstRing = 8;                     // tiles whose score constants are kept
constexpr int kConsts = 3 * kBlocksPerTile;       // key scale, log2 f, 1 / f of every block
constexpr int kQBytes = kTileM * kRowBytes;       // one half's Q: 16 KiB
constexpr int kOpBytes = kTileN * kRowBytes;      // one converted K or V tile: 16 KiB
constexpr int kRawBytes = 2 * kTileN * kQ8RowBytes;  // codes of K, then of V: 16 KiB
constexpr int kQOff = 0;                          // [2 halves][2 buffers]
constexpr int kKOff = kQOff + 4 * kQBytes;
constexpr int kVOff = kKOff + kRing * kOpBytes;
constexpr int kRawOff = kVOff + kRing * kOpBytes;
constexpr int kRawScaleOff = kRawOff + kRing * kRawBytes;  // [kRing][2][8] floats
constexpr int kConstOff = kRawScaleOff + kRing * 2 * kBlocksPerTile * 4;
constexpr int kXchOff = kConstOff + kConstRing * kConsts * 4;  // [half][3][2][128] floats
constexpr int kBarOff = kXchOff + 2 * 3 * 2 * kTileM * 4;
constexpr int kNumBars = 4 + 4 + 2 + 6 * kRing + 5 * 2 + 1;
constexpr int kMiscOff = kBarOff + (kNumBars + 1) / 2 * 16;
constexpr int kUnitOff = kMiscOff + 160;
constexpr int kSmemBytes = kUnitOff + 5 * kMaxUnitsPerCta * 4;
constexpr int kRankPairs = 256;  // up to this many (sequence, tile) pairs are ranked by counting
static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");
static_assert(sort_scratch_bytes(kThreads) <= kRawOff, "sort scratch fits below the raw ring");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0;    // + 128 per half: fp32 scores
constexpr uint32_t kPCol = 256;  // + 64 per half: bf16 pairs
constexpr uint32_t kOCol = 384;  // + 64 per half: fp32
// The exponent reference m is set this much (log2) above the largest score so far and raised
// when a score passes it: weights stay below 2, so the sums of p V keep the size of the values,
// and a row rescales only when its maximum grows by more than 2^8.
constexpr float kHeadroom = 8.0f;
// Register split (setmaxnreg): the row warps' threads and the others' share what the CTA was
// launched with; the launcher checks that it suffices.
constexpr int kRowRegs = 96;
constexpr int kOtherRegs = 48;

struct Pools {
  const float* key_scale;
  const float* value_scale;
};

// wait_or_abort whose usual case, a phase that has completed, is one try_wait.
__device__ __forceinline__ bool wait_ready(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           int32_t* status) {
  return mbar_try_wait(bar, parity) || wait_or_abort(bar, parity, abort_flag, status);
}

// Four 1 KiB tiles of a pool, rows[0..3] of its [tiles][1 KiB] view, by one copy.
__device__ __forceinline__ void gather4(void* dst, const CUtensorMap* map, const int32_t* rows,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(rows[0]), "r"(rows[1]), "r"(rows[2]),
      "r"(rows[3]), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void async_copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// One arrival on `bar` (counted in its initial count) when this thread's asynchronous copies
// so far have landed.
__device__ __forceinline__ void async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// True in one lane of a converged warp (the same one on every call of the kernel).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// A shared-memory float, read where it is used (not held in a register from before).
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ void lds_f32x4(uint32_t addr, float (&v)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr));
}

// Instruction descriptor, kind::f16 with f16 A/B (both K-major) and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The tiles of K/V each half of a unit needs (the second half may have no tokens).
template <int HALF_TOKENS>
__device__ __forceinline__ int half_tiles(const Unit& u, int half) {
  const int n = min(HALF_TOKENS, u.ntok - half * HALF_TOKENS);
  if (n <= 0) return 0;
  return (u.L - u.q_len + u.tok0 + half * HALF_TOKENS + n + kTileN - 1) / kTileN;
}

__device__ __forceinline__ uint32_t pack_bf2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four codes of a word as bf16 pairs times 2^-120 (exact): the code's exponent and
// significand bits, three places down from the bf16's, under its sign.
__device__ __forceinline__ void codes4_to_bf2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);
  lo = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u);
  hi = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
}

// f of a scale 2^e f, 1 <= f < 2, below the normal floats too; 1 for a scale of 0.
__device__ __forceinline__ float significand(float s) {
  const uint32_t b = __float_as_uint(s);
  const int down = max(__clz(b) - 8, 0);  // places that a subnormal's first bit lies below the others'
  return __uint_as_float(((b << down) & 0x7fffffu) | 0x3f800000u);
}

// 2^e as a bf16 pair, -126 <= e <= 127.
__device__ __forceinline__ uint32_t bf2_power(int e) {
  return static_cast<uint32_t>(e + 127) * 0x00800080u;
}

// Chunk c (16 bytes) of row r in the 128-byte-swizzled layout of 128-byte rows.
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r * kRowBytes + ((c ^ (r & 7)) << 4));
}

// Lanes whose numbers differ in bit `d` exchange: the lower's b for the upper's a.
__device__ __forceinline__ void swap_chunks(uint4& a, uint4& b, bool upper, int d) {
  uint4 give = upper ? a : b;
  give.x = __shfl_xor_sync(0xffffffffu, give.x, d);
  give.y = __shfl_xor_sync(0xffffffffu, give.y, d);
  give.z = __shfl_xor_sync(0xffffffffu, give.z, d);
  give.w = __shfl_xor_sync(0xffffffffu, give.w, d);
  if (upper) a = give; else b = give;
}

template <int GROUP>
__global__ void __launch_bounds__(kThreads, 1)
paged_chunk_q8_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const PParams p, const Pools pools) {
  constexpr int kHalfTokens = kTileM / GROUP;
  constexpr int kUnitTokens = 2 * kHalfTokens;
  const int tid = threadIdx.x;
  // (through a shuffle, so that what depends on it stays in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int lane = tid & 31;
  extern __shared__ __align__(1024) uint8_t smem[];  // 128-byte swizzle atoms need 1 KiB
  if ((smem_addr(smem) & 1023u) != 0) {
    if (tid == 0) flag_error(p.status, PA_DEVFLAG_LAYOUT);
    return;
  }
  uint8_t* sq = smem + kQOff;
  uint8_t* sk = smem + kKOff;
  uint8_t* sv = smem + kVOff;
  uint8_t* sraw = smem + kRawOff;
  float* raw_scale = reinterpret_cast<float*>(smem + kRawScaleOff);
  float* consts = reinterpret_cast<float*>(smem + kConstOff);
  float* xch = reinterpret_cast<float*>(smem + kXchOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  // A half that has no rows in a unit takes no part in it: Q buffers and phases count the units
  // of each half by themselves.
  uint64_t* q_full = bars;                   // [half][2] Q (bf16) landed in a buffer
  uint64_t* q_empty = q_full + 4;            // [half][2] the last scores that read it are done
  uint64_t* q_ready = q_empty + 4;           // [half] the half's next Q is f16
  uint64_t* raw_full = q_ready + 2;          // [kRing] codes and scales landed
  uint64_t* raw_empty = raw_full + kRing;    // [kRing] and were read
  uint64_t* k_full = raw_empty + kRing;      // [kRing] K converted
  uint64_t* k_empty = k_full + kRing;        // [kRing] scores that read it done
  uint64_t* v_full = k_empty + kRing;
  uint64_t* v_empty = v_full + kRing;
  // [half] scores in tensor memory: the MMAs' commit, and an arrival of the issuing warp, which
  // has seen K's arrivals and so passes on what the converters wrote before them (the constants)
  uint64_t* s_full = v_empty + kRing;
  uint64_t* s_free = s_full + 2;             // [half] scores read into registers
  uint64_t* p_full = s_free + 2;             // [half] P in tensor memory
  uint64_t* pv_done = p_full + 2;            // [half] P V done: P free, O up to date
  uint64_t* o_free = pv_done + 2;            // [half] O of a finished unit read out
  uint64_t* drain = o_free + 2;
  int* misc = reinterpret_cast<int*>(smem + kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int& abort_flag = *reinterpret_cast<volatile int*>(misc + 1);
  int* n_units_s = misc + 2;
  int* red = misc + 4;  // 32 ints of scan scratch
  int32_t* unit_s = reinterpret_cast<int32_t*>(smem + kUnitOff);
  int32_t* unit_tg = unit_s + kMaxUnitsPerCta;
  int32_t* unit_q0 = unit_tg + kMaxUnitsPerCta;
  int32_t* unit_len = unit_q0 + kMaxUnitsPerCta;
  int32_t* unit_L = unit_len + kMaxUnitsPerCta;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_ready[b], kRowWarps);
      mbar_init(&s_full[b], 2);
      mbar_init(&s_free[b], kRowWarps);
      mbar_init(&p_full[b], kRowWarps);
      mbar_init(&pv_done[b], 1);
      mbar_init(&o_free[b], kRowWarps);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&raw_full[i], 1 + kBlocksPerTile);
      mbar_init(&raw_empty[i], kVWarps + kKWarps);
      mbar_init(&k_full[i], kKWarps);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], kVWarps);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    abort_flag = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tensormap(&tmap_q);
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
  }
  const int n_units = plan_units<kUnitTokens, kTileN, kThreads, kRankPairs>(
      p, smem, red, unit_s, unit_tg, unit_q0, unit_len, unit_L);
  if (tid == 0) *n_units_s = n_units;
  fence_proxy_async_smem();  // the plan's scratch before copies and MMAs touch the buffers
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Schedule sc;
  sc.unit_s = unit_s;
  sc.unit_tg = unit_tg;
  sc.n_units = *n_units_s;
  sc.unit_q0 = unit_q0;
  sc.unit_len = unit_len;
  sc.unit_L = unit_L;

  if (warp < 2 * kRowWarps) {
    // ============================ row warps ============================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const int half = warp >> 3;
    const int part = (warp >> 2) & 1;  // keys 64 part .. 64 part + 63 of every tile
    const int r = (warp & 3) * 32 + lane;  // row of the half == TMEM lane
    const int tt = r / GROUP;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + kSCol + half * kTileN + part * (kTileN / 2);
    const uint32_t p_addr = lane_addr + kPCol + half * (kTileN / 2) + part * (kTileN / 4);
    const uint32_t o_addr = lane_addr + kOCol + half * kHeadDim + part * (kHeadDim / 2);
    // The two warps of the same rows exchange a float per row (slot 0 or 1: a tile's maximum;
    // 2: the sum at the end) and go on together.  A warp that gives up (for a
    // timeout somewhere) arrives once more, so that its partner is not left waiting, and the
    // partner then sees the flag.
    float* const my_xch = xch + (half * 3 * 2 + part) * kTileM + r;
    const int pair_bar = 1 + half * 4 + (warp & 3);
    auto exchange = [&](int slot, float mine, int& gone) -> float {
      my_xch[slot * 2 * kTileM] = mine;
      named_barrier_sync(pair_bar, 64);
      gone = abort_flag;  // tested before the next barrier of the pair
      return my_xch[slot * 2 * kTileM + (part ? -kTileM : kTileM)];
    };
    auto wait_row = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_ready(bar, parity, &abort_flag, p.status));
    };
    int k = 0;
    int qc = 0;          // Qs this half has turned into f16
    bool have_q = false;  // the coming unit's among them
    float q_factor = 0.f, q_factor_next = 0.f;  // score factor of this row
    // Turn this row of the half's next Q into f16, in place, under the row's power of two: both
    // warps look at the whole row, each writes half of it.
    auto convert_q = [&]() -> bool {
      const int b = 2 * half + (qc & 1);
      if (!wait_row(&q_full[b], static_cast<uint32_t>((qc >> 1) & 1))) return false;
      uint8_t* q = sq + b * kQBytes;
      uint4 w[4];
      uint32_t big = 0u;  // largest magnitude as bits
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 x = lds128(q + swz(r, c ^ (4 * part)));  // its own half first
        if (c < 4) w[c] = x;
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          big = max(big, max((y[i] << 16) & 0x7fff0000u, y[i] & 0x7fff0000u));
      }
      const int shift = query_shift(big);
      const float up = power_of_two(shift);
      q_factor_next = p.qk_scale * power_of_two(-shift);
      named_barrier_sync(pair_bar, 64);  // both have read
      if (!__all_sync(0xffffffffu, abort_flag == 0)) return false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_float2(x[i]);
          y[i] = pack_half2_rn(f.x * up, f.y * up);
        }
        *reinterpret_cast<uint4*>(q + swz(r, c ^ (4 * part))) = make_uint4(y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready[half]);
      ++qc;
      have_q = true;
      return true;
    };
    bool ok = true;
    int jt = 0;  // K/V tiles of the CTA before this unit
    int c = 0;   // tiles of this half so far
    while (ok) {
      // of a unit, only what a row needs stays in registers
      int n_mine, n_kv, pos, pos_lo;
      int out_token, out_left, out_head;  // the half's first output row, its rows left, the K/V head
      bool next_mine;
      {
        Unit u;
        if (!next_unit<kUnitTokens, kTileN, true>(p, sc, k, u)) break;
        n_mine = half_tiles<kHalfTokens>(u, half);
        n_kv = u.n_kv;
        const int token = u.tok0 + half * kHalfTokens + tt;
        pos = u.L - u.q_len + min(token, u.q_len - 1);
        pos_lo = u.L - u.q_len + u.tok0 + half * kHalfTokens;
        out_token = u.q0 + u.tok0 + half * kHalfTokens;
        out_left = u.q_len - u.tok0 - half * kHalfTokens;
        out_head = u.g;
        int peek = k;
        next_mine = next_unit<kUnitTokens, kTileN, true>(p, sc, peek, u) && half_tiles<kHalfTokens>(u, half) > 0;
      }
      if (n_mine > 0) {
        if (!have_q && !(ok = convert_q())) break;
        have_q = false;
        q_factor = q_factor_next;
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < n_mine; ++j, ++c) {
          if (!(ok = wait_row(&s_full[half], static_cast<uint32_t>(c & 1)))) break;
          tc_fence_after_sync();
          // The next unit's Q, before its first scores are wanted.  Only now: these scores
          // show that the issuing thread has seen this unit's Q, so q_ready can complete a
          // phase again.
          if (j == n_mine - 1 && next_mine && !(ok = convert_q())) break;
          uint32_t v[2][32];
          float bm[kBlocksPerTile / 2];  // largest raw score of each block
#pragma unroll
          for (int b = 0; b < kBlocksPerTile / 2; ++b)
            tmem_ld16_max(s_addr + 16 * b, &v[b >> 1][16 * (b & 1)], bm[b]);
          tmem_wait_ld();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[half]);
          const int kb = j * kTileN + part * (kTileN / 2);
          if (kb + kTileN / 2 - 1 > pos_lo) {
            // a tile on the causal diagonal: hide keys past each row's position
#pragma unroll
            for (int b = 0; b < kBlocksPerTile / 2; ++b) {
              bm[b] = -INFINITY;
#pragma unroll
              for (int i = 16 * b; i < 16 * b + 16; ++i) {
                if (kb + i > pos) v[i >> 5][i & 31] = __float_as_uint(-INFINITY);
                bm[b] = fmaxf(bm[b], __uint_as_float(v[i >> 5][i & 31]));
              }
            }
          }
          const int slot = (jt + j) % kConstRing;
          const uint32_t cs = smem_addr(consts + slot * kConsts + part * (kBlocksPerTile / 2));
          float f[kBlocksPerTile / 2];  // score factors of this warp's blocks
          lds_f32x4(cs, f);
#pragma unroll
          for (int b = 0; b < kBlocksPerTile / 2; ++b)
            f[b] = fmaxf(f[b] * q_factor, 1.17549435e-38f);  // (a hidden key's -inf * 0 is a NaN)
          const float mt = fmaxf(max3f(bm[0] * f[0], bm[1] * f[1], bm[2] * f[2]), bm[3] * f[3]);
          int gone;
          const float theirs = exchange(c & 1, mt, gone);
          const float m_new = max3f(m, mt, theirs);
          const bool grow = m_new > m;  // true on the first tile
          float alpha = 1.f;
          if (grow) {
            alpha = fast_exp2(m - (m_new + kHeadroom));
            m = m_new + kHeadroom;
          }
          l *= alpha;
          // p' two at a time, packed to bf16 over the scores
          float lf[kBlocksPerTile / 2];
          lds_f32x4(cs + 4 * kBlocksPerTile, lf);
#pragma unroll
          for (int b = 0; b < kBlocksPerTile / 2; ++b) {
            const float nb = lf[b] - m;
            const float2 fb = make_float2(f[b], f[b]);
            const float2 nb2 = make_float2(nb, nb);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kBlockSize / 2; ++i) {
              const int e = b * kBlockSize + 2 * i;
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[e >> 5][e & 31]),
                                                      __uint_as_float(v[e >> 5][(e & 31) + 1])),
                                          fb, nb2);
              const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              sum = __fadd2_rn(sum, y);
              v[0][e >> 1] = pack_bf2(y.x, y.y);
            }
            l += (sum.x + sum.y) * lds_f32(cs + 4 * (2 * kBlocksPerTile + b));
          }
          if (!(ok = __all_sync(0xffffffffu, gone == 0))) break;
          if (c > 0) {  // the previous P V: P's columns are free and O is up to date
            if (!(ok = wait_row(&pv_done[half], static_cast<uint32_t>((c - 1) & 1)))) break;
            tc_fence_after_sync();
          }
          tmem_st32(p_addr, v[0]);
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            const float2 a2 = make_float2(alpha, alpha);
            uint32_t(&o)[32] = v[1];  // this warp's 32 columns of O
            tmem_ld32(o_addr, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = __fmul2_rn(
                  make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), a2);
              o[2 * i] = __float_as_uint(x.x);
              o[2 * i + 1] = __float_as_uint(x.y);
            }
            tmem_st32(o_addr, o);
          }
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[half]);
        }
        if (!ok) break;
        // ---- epilogue: this warp's 32 dims ----
        int gone;
        const float theirs = exchange(2, l, gone);
        if (!(ok = __all_sync(0xffffffffu, gone == 0))) break;
        if (!(ok = wait_row(&pv_done[half], static_cast<uint32_t>((c - 1) & 1)))) break;
        tc_fence_after_sync();
        uint32_t o[32];
        tmem_ld32(o_addr, o);
        tmem_wait_ld();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[half]);
        const float inv = 1.f / (l + theirs);
        // Four lanes exchange what they hold (four rows by four 16-byte chunks), so that each store
        // covers 64 bytes of eight rows: a lane's own row at a time touched 32 lines a store (8 x
        // 512 rows 70.0 us against 68.4).
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c] = make_uint4(pack_bf2(__uint_as_float(o[8 * c]) * inv, __uint_as_float(o[8 * c + 1]) * inv),
                            pack_bf2(__uint_as_float(o[8 * c + 2]) * inv, __uint_as_float(o[8 * c + 3]) * inv),
                            pack_bf2(__uint_as_float(o[8 * c + 4]) * inv, __uint_as_float(o[8 * c + 5]) * inv),
                            pack_bf2(__uint_as_float(o[8 * c + 6]) * inv, __uint_as_float(o[8 * c + 7]) * inv));
        swap_chunks(w[0], w[1], lane & 1, 1);
        swap_chunks(w[2], w[3], lane & 1, 1);
        swap_chunks(w[0], w[2], lane & 2, 2);
        swap_chunks(w[1], w[3], lane & 2, 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = (r & ~3) + i;
          if (rr / GROUP < out_left)
            *reinterpret_cast<uint4*>(
                p.out + (static_cast<int64_t>(out_token + rr / GROUP) * p.num_q_heads + out_head * GROUP + rr % GROUP) *
                            kHeadDim + part * (kHeadDim / 2) + 8 * (lane & 3)) = w[i];
        }
      }
      jt += n_kv;
    }
    if (!ok) asm volatile("bar.arrive %0, 64;" ::"r"(pair_bar) : "memory");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kMmaWarp) {
      // ============================ V converters ============================
      constexpr int kMyBlocks = kBlocksPerTile / kVWarps;
      const int cw = warp - kVWarp0;  // blocks kMyBlocks cw .. of every tile
      const int row0 = cw * kMyBlocks * kBlockSize + (lane >> 2);
      const int c0 = 2 * (lane & 3);  // 16 codes of a row: two 16-byte chunks
      int k = 0, st = 0;
      uint32_t ph = 0;
      Unit cur;
      bool ok = true;
      while (ok && next_unit<kUnitTokens, kTileN, true>(p, sc, k, cur)) {
        for (int j = 0; j < cur.n_kv; ++j) {
          ok = wait_ready(&raw_full[st], ph, &abort_flag, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          const uint8_t* raw = sraw + st * kRawBytes + kTileN * kQ8RowBytes + cw * kMyBlocks * kQ8TileBytes + 16 * lane;
          uint4 in[2 * kMyBlocks];
#pragma unroll
          for (int i = 0; i < 2 * kMyBlocks; ++i) in[i] = lds128(raw + i * 512);
          uint32_t my_m = 0u;  // lane b: 2^(120 + e) of block b's value scale, a bf16 pair
          int my_high = 0;     // e where 120 + e is beyond bf16: then my_m is 2^120
          if (lane < kMyBlocks) {
            const uint32_t bits = __float_as_uint(
                raw_scale[st * 2 * kBlocksPerTile + kBlocksPerTile + kMyBlocks * cw + lane]) & 0x7fffffffu;
            const int e = static_cast<int>(bits >> 23) - 127;
            if (e > -127) {
              my_high = e > 7 ? min(e, 127) : 0;
              my_m = bf2_power(e > 7 ? 120 : 120 + e);
            } else if (bits != 0u) {  // below the normal floats: e = -118 - clz
              my_m = bf2_power(2 - __clz(bits));
            }
          }
          const bool any_high = __any_sync(0xffffffffu, my_high != 0);
          ok = wait_ready(&v_empty[st], ph ^ 1u, &abort_flag, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          uint8_t* dst = sv + st * kOpBytes;
          const int keys_left = cur.keys - j * kTileN - row0;
#pragma unroll
          for (int i = 0; i < 2 * kMyBlocks; ++i) {
            uint4 w = in[i];
            // keys past the last needed one weigh nothing, but may hold anything
            if (8 * i >= keys_left) w = make_uint4(0u, 0u, 0u, 0u);
            uint4 a, b;
            codes4_to_bf2x2(w.x, a.x, a.y);
            codes4_to_bf2x2(w.y, a.z, a.w);
            codes4_to_bf2x2(w.z, b.x, b.y);
            codes4_to_bf2x2(w.w, b.z, b.w);
            const uint32_t m0 = __shfl_sync(0xffffffffu, my_m, i >> 1);
            a.x = mul_bf2(a.x, m0); a.y = mul_bf2(a.y, m0); a.z = mul_bf2(a.z, m0); a.w = mul_bf2(a.w, m0);
            b.x = mul_bf2(b.x, m0); b.y = mul_bf2(b.y, m0); b.z = mul_bf2(b.z, m0); b.w = mul_bf2(b.w, m0);
            if (any_high) {  // a scale above 2^7: the rest of it
              const uint32_t m1 = bf2_power(__shfl_sync(0xffffffffu, my_high, i >> 1));
              a.x = mul_bf2(a.x, m1); a.y = mul_bf2(a.y, m1); a.z = mul_bf2(a.z, m1); a.w = mul_bf2(a.w, m1);
              b.x = mul_bf2(b.x, m1); b.y = mul_bf2(b.y, m1); b.z = mul_bf2(b.z, m1); b.w = mul_bf2(b.w, m1);
            }
            *reinterpret_cast<uint4*>(dst + swz(row0 + 8 * i, c0)) = a;
            *reinterpret_cast<uint4*>(dst + swz(row0 + 8 * i, c0 + 1)) = b;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v_full[st]);
            mbar_arrive(&raw_empty[st]);
          }
          if (++st == kRing) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
    } else if (warp >= kKWarp0) {
      // ============================ K converters ============================
      constexpr int kMyBlocks = kBlocksPerTile / kKWarps;
      const int cw = warp - kKWarp0;  // blocks kMyBlocks cw .. of every tile
      const int row0 = cw * kMyBlocks * kBlockSize + (lane >> 2);
      const int c0 = 2 * (lane & 3);
      int k = 0, st = 0, slot = 0;
      uint32_t ph = 0;
      Unit cur;
      bool ok = true;
      while (ok && next_unit<kUnitTokens, kTileN, true>(p, sc, k, cur)) {
        for (int j = 0; j < cur.n_kv; ++j) {
          ok = wait_ready(&raw_full[st], ph, &abort_flag, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          // the row warps' constants of this warp's blocks
          if (lane < kMyBlocks) {
            const int blk = kMyBlocks * cw + lane;
            const float* rs = raw_scale + st * 2 * kBlocksPerTile + blk;
            const bool needed = j * kBlocksPerTile + blk < cur.blocks_needed;
            const float f = significand(needed ? rs[kBlocksPerTile] : 1.f);  // of the value scale
            float* cs = consts + slot * kConsts + blk;
            cs[0] = needed ? rs[0] : 1.f;
            float lf = 0.f, fi = 1.f;
            if (f != 1.f) {
              lf = __log2f(f);
              fi = 1.f / f;
            }
            cs[kBlocksPerTile] = lf;
            cs[2 * kBlocksPerTile] = fi;
          }
          ok = wait_ready(&k_empty[st], ph ^ 1u, &abort_flag, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;  // (and the constants precede the arrival)
          const uint8_t* raw = sraw + st * kRawBytes + cw * kMyBlocks * kQ8TileBytes + 16 * lane;
          uint8_t* dst = sk + st * kOpBytes;
#pragma unroll
          for (int i = 0; i < 2 * kMyBlocks; ++i) {
            const uint4 w = lds128(raw + i * 512);
            uint4 a, b;
            codes4_to_half2x2(w.x, a.x, a.y);
            codes4_to_half2x2(w.y, a.z, a.w);
            codes4_to_half2x2(w.z, b.x, b.y);
            codes4_to_half2x2(w.w, b.z, b.w);
            *reinterpret_cast<uint4*>(dst + swz(row0 + 8 * i, c0)) = a;
            *reinterpret_cast<uint4*>(dst + swz(row0 + 8 * i, c0 + 1)) = b;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&k_full[st]);
            mbar_arrive(&raw_empty[st]);
          }
          if (++st == kRing) {
            st = 0;
            ph ^= 1u;
          }
          slot = (slot + 1) % kConstRing;
        }
      }
    } else if (warp == kMmaWarp) {
      // ============================ MMA issuer ============================
      // The whole warp walks the tiles, so that barriers, counters and descriptors stay
      // warp-uniform (uniform registers feed the MMAs); one elected lane issues.
      constexpr uint32_t kIdescS = idesc_f16_f32(kTileM, kTileN);
      constexpr uint32_t kIdescO = idesc_bf16_f32(kTileM, kHeadDim, true);
      const bool leader = elect_one();
      const uint64_t q_desc0 = sw128_desc(smem_addr(sq), 16, 1024);
      const uint64_t k_desc0 = sw128_desc(smem_addr(sk), 16, 1024);
      const uint64_t v_desc0 = sw128_desc(smem_addr(sv), 16, 1024);
      constexpr uint64_t kStageStep = kOpBytes >> 4;  // of a descriptor's start address
      constexpr uint64_t kQStep = kQBytes >> 4;
      int s_issued[2] = {0, 0}, pv_issued[2] = {0, 0}, q_used[2] = {0, 0}, o_used[2] = {0, 0};
      int ks = 0, vs = 0;            // ring stages of the next K and V tile
      uint32_t kph = 0, vph = 0;     // and their phases
      // scores of a unit's tile j, for the halves that need it
      auto issue_s = [&](int n0, int n1, int j) -> bool {
        if (!wait_ready(&k_full[ks], kph, &abort_flag, p.status)) return false;
        const uint64_t k_desc = k_desc0 + kStageStep * ks;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = h ? n1 : n0;
          if (j >= n) continue;
          if (j == 0) {
            if (!wait_ready(&q_ready[h], static_cast<uint32_t>(q_used[h] & 1), &abort_flag, p.status))
              return false;
            ++q_used[h];
          }
          if (s_issued[h] > 0 &&
              !wait_ready(&s_free[h], static_cast<uint32_t>((s_issued[h] - 1) & 1), &abort_flag,
                             p.status))
            return false;
          tc_fence_after_sync();
          const int qb = 2 * h + ((q_used[h] - 1) & 1);
          const uint64_t q_desc = q_desc0 + kQStep * qb;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kHeadDim / 16; ++kk)
              umma_bf16(tmem + kSCol + h * kTileN, q_desc + 2 * kk, k_desc + 2 * kk, kIdescS,
                        kk > 0 ? 1u : 0u);
            umma_commit(&s_full[h]);
            mbar_arrive(&s_full[h]);
            if (j == n - 1) umma_commit(&q_empty[qb]);
          }
          ++s_issued[h];
        }
        if (leader) umma_commit(&k_empty[ks]);
        if (++ks == kRing) {
          ks = 0;
          kph ^= 1u;
        }
        return true;
      };
      auto issue_pv = [&](int n0, int n1, int j) -> bool {
        if (!wait_ready(&v_full[vs], vph, &abort_flag, p.status)) return false;
        const uint64_t v_desc = v_desc0 + kStageStep * vs;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (j >= (h ? n1 : n0)) continue;
          if (!wait_ready(&p_full[h], static_cast<uint32_t>(pv_issued[h] & 1), &abort_flag, p.status))
            return false;
          if (j == 0) {  // O starts anew: the half's previous unit has been read out
            if (o_used[h] > 0 &&
                !wait_ready(&o_free[h], static_cast<uint32_t>((o_used[h] - 1) & 1), &abort_flag,
                               p.status))
              return false;
            ++o_used[h];
          }
          tc_fence_after_sync();
          if (leader) {
            umma_bf16_ts(tmem + kOCol + h * kHeadDim, tmem + kPCol + h * (kTileN / 2), v_desc, kIdescO,
                         j > 0 ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < kTileN / 16; ++kk)  // 16 keys: 2 KiB of V, 8 columns of P
              umma_bf16_ts(tmem + kOCol + h * kHeadDim, tmem + kPCol + h * (kTileN / 2) + kk * 8,
                           v_desc + 128 * kk, kIdescO, 1u);
            umma_commit(&pv_done[h]);
          }
          ++pv_issued[h];
        }
        if (leader) umma_commit(&v_empty[vs]);
        if (++vs == kRing) {
          vs = 0;
          vph ^= 1u;
        }
        return true;
      };
      int k = 0;
      Unit cur, nxt;
      bool have = next_unit<kUnitTokens, kTileN, true>(p, sc, k, cur);
      bool have_next = have && next_unit<kUnitTokens, kTileN, true>(p, sc, k, nxt);
      int n0 = 0, n1 = 0;
      bool ok = have;
      if (have) {
        n0 = half_tiles<kHalfTokens>(cur, 0);
        n1 = half_tiles<kHalfTokens>(cur, 1);
        ok = issue_s(n0, n1, 0);
      }
      while (ok && have) {
        int m0 = 0, m1 = 0;
        if (have_next) {
          m0 = half_tiles<kHalfTokens>(nxt, 0);
          m1 = half_tiles<kHalfTokens>(nxt, 1);
        }
        const int n_kv = cur.n_kv;
        for (int j = 0; ok && j < n_kv; ++j) {
          const bool last = j + 1 == n_kv;
          if (!last || have_next) ok = issue_s(last ? m0 : n0, last ? m1 : n1, last ? 0 : j + 1);
          if (ok) ok = issue_pv(n0, n1, j);
        }
        cur = nxt;
        n0 = m0;
        n1 = m1;
        have = have_next;
        if (have) have_next = next_unit<kUnitTokens, kTileN, true>(p, sc, k, nxt);
      }
      // wait (bounded) until every MMA issued above has completed
      if (leader) {
        umma_commit(drain);
        if (!mbar_wait(drain, 0)) flag_error(p.status, PA_DEVFLAG_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == kProducerWarp) {
      // ============================ producer ============================
      const bool leader = elect_one();
      int k = 0;
      Unit cur, nxt;
      bool have = next_unit<kUnitTokens, kTileN, true>(p, sc, k, cur);
      bool have_next = have && next_unit<kUnitTokens, kTileN, true>(p, sc, k, nxt);
      int nq[2] = {0, 0};  // Qs requested for each half
      auto load_q = [&](const Unit& u) {
        bool ok = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (half_tiles<kHalfTokens>(u, h) == 0) continue;
          const int b = 2 * h + (nq[h] & 1);
          if (lane == 0 && ok) {
            if (nq[h] >= 2)
              ok = wait_ready(&q_empty[b], static_cast<uint32_t>(((nq[h] - 2) >> 1) & 1),
                                 &abort_flag, p.status);
            if (ok) {
              mbar_arrive_expect_tx(&q_full[b], kQBytes);
              tma_load_3d(sq + b * kQBytes, &tmap_q, 0, u.g * GROUP, u.q0 + u.tok0 + h * kHalfTokens,
                          &q_full[b]);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (ok) ++nq[h];
        }
        return ok;
      };
      bool ok = !have || load_q(cur);
      int jt = 0;
      while (ok && have) {
        const int32_t* row = p.block_tables + static_cast<int64_t>(cur.s) * p.max_blocks_per_seq;
        // 32 table entries (four tiles) at a time, one per lane, the next window in flight
        auto fetch = [&](int base) -> int32_t {
          return base + lane < cur.blocks_needed ? __ldg(row + base + lane) : 0;
        };
        int win_base = 0;
        int32_t win = fetch(0);
        int32_t win_next = fetch(32);
        for (int j = 0; j < cur.n_kv; ++j, ++jt) {
          // the next unit's Q, once this unit's pipeline is under way
          if (have_next && j == min(1, cur.n_kv - 1) && !(ok = load_q(nxt))) break;
          const int st = jt % kRing;
          const int lb0 = j * kBlocksPerTile;
          if (lb0 >= win_base + 32) {
            win_base += 32;
            win = win_next;
            win_next = fetch(win_base + 32);
          }
          const int lb = lb0 + lane;
          const bool need = lane < kBlocksPerTile && lb < cur.blocks_needed;
          const int32_t entry =
              __shfl_sync(0xffffffffu, win, (lb0 - win_base) + (lane & (kBlocksPerTile - 1)));
          const bool bad = need && (entry < 0 || entry >= p.num_blocks);
          if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(p.status, PA_DEVFLAG_BAD_BLOCK);
          // tile (row) of each block; one that is not needed, or bad, brings the pool's first
          const int32_t tile = need && !bad ? entry * p.num_kv_heads + cur.g : 0;
          int32_t rows[kBlocksPerTile];
#pragma unroll
          for (int b = 0; b < kBlocksPerTile; ++b) rows[b] = __shfl_sync(0xffffffffu, tile, b);
          ok = wait_ready(&raw_empty[st], static_cast<uint32_t>((jt / kRing) & 1) ^ 1u, &abort_flag, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (leader) {
            mbar_arrive_expect_tx(&raw_full[st], kRawBytes);
            uint8_t* dst = sraw + st * kRawBytes;
#pragma unroll
            for (int b = 0; b < kBlocksPerTile; b += 4) {
              gather4(dst + b * kQ8TileBytes, &tmap_k, &rows[b], &raw_full[st]);
              gather4(dst + (kBlocksPerTile + b) * kQ8TileBytes, &tmap_v, &rows[b], &raw_full[st]);
            }
          }
          if (lane < kBlocksPerTile) {
            float* s = raw_scale + st * 2 * kBlocksPerTile + lane;
            async_copy4(s, pools.key_scale + tile);
            async_copy4(s + kBlocksPerTile, pools.value_scale + tile);
            async_arrive(&raw_full[st]);
          }
        }
        cur = nxt;
        have = have_next;
        if (have) have_next = next_unit<kUnitTokens, kTileN, true>(p, sc, k, nxt);
      }
      // leave no copy in flight: wait (bounded) for the last Q of each buffer and the last
      // fill of each stage
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) {
        for (int h = 0; h < 2; ++h) {
          for (int b = 0; b < 2 && b < nq[h]; ++b) {
            const int last = b + ((nq[h] - 1 - b) / 2) * 2;
            if (!mbar_wait(&q_full[2 * h + b], static_cast<uint32_t>((last >> 1) & 1)))
              flag_error(p.status, PA_DEVFLAG_TIMEOUT);
          }
        }
        for (int st = 0; st < kRing && st < jt; ++st) {
          const int last = st + ((jt - 1 - st) / kRing) * kRing;
          if (!mbar_wait(&raw_full[st], static_cast<uint32_t>((last / kRing) & 1)))
            flag_error(p.status, PA_DEVFLAG_TIMEOUT);
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int GROUP>
cudaError_t launch(const AttendQ8Args& a, cudaStream_t stream) {
  static bool ready[kMaxDevices] = {};  // benign race: the calls are idempotent
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev]) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, paged_chunk_q8_kernel<GROUP>);
    if (e != cudaSuccess) return e;
    // setmaxnreg waits for registers the launch never had: refuse instead
    if (attr.numRegs * kThreads < kRowThreads * kRowRegs + (kThreads - kRowThreads) * kOtherRegs)
      return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(paged_chunk_q8_kernel<GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  CUtensorMap tq;
  if (!encode_query_tiles(&tq, a.q, static_cast<uint64_t>(a.num_query_tokens), a.num_q_heads, GROUP,
                          kTileM / GROUP))
    return cudaErrorInvalidValue;
  CUtensorMap tk, tv;
  const uint64_t tiles = static_cast<uint64_t>(a.num_blocks) * a.num_kv_heads;
  if (!encode_tile_rows(&tk, a.key_cache, tiles) || !encode_tile_rows(&tv, a.value_cache, tiles))
    return cudaErrorInvalidValue;
  PParams p = {};
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.query_start_loc = a.query_start_loc;
  p.block_tables = a.block_tables;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.context_lens = a.context_lens;
  p.num_blocks = a.num_blocks;
  p.num_kv_heads = a.num_kv_heads;
  p.num_q_heads = a.num_q_heads;
  p.qk_scale = a.scale * 1.4426950408889634f;
  p.status = a.status;
  p.num_query_tokens = a.num_query_tokens;
  p.max_query_len = a.max_query_len;
  p.num_seqs = a.num_seqs;
  constexpr int kUnitTokens = 2 * kTileM / GROUP;
  p.q_tiles = (a.max_query_len + kUnitTokens - 1) / kUnitTokens;
  p.skip_single = 0;
  const Pools pools = {a.key_scale, a.value_scale};
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * p.q_tiles;
  const int64_t grid = units < sms ? units : sms;
  if (grid < 1) return cudaSuccess;
  paged_chunk_q8_kernel<GROUP><<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(tq, tk, tv, p, pools);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_q8(const AttendQ8Args& a, cudaStream_t stream) {
  if (rows_q8_takes(a)) return launch_rows_q8(a, stream);
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch<1>(a, stream);
    case 2: return launch<2>(a, stream);
    case 4: return launch<4>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
