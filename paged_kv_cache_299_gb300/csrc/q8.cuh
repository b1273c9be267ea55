// The 8-bit cache's number format: a cached value is an e4m3 code times the scale of its
// (block, K/V head), a power of two when this library chose it.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace pkv {

constexpr int kQ8RowBytes = kHeadDim;                // one token of one head: 64 codes
constexpr int kQ8TileBytes = kHeadDim * kBlockSize;  // one (block, kv head) tile: 1 KiB
constexpr float kCodeMax = 448.f;                    // largest e4m3 magnitude
constexpr int kMinScaleExp = -126;                   // scales stay normal floats

// The four codes of a word -> two half2 (bytes 0, 1 and bytes 2, 3), exact (every e4m3 value is an
// f16 value).
__device__ __forceinline__ void codes4_to_half2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two floats -> two codes (a in the low byte), round to nearest even, saturating at +-448.
__device__ __forceinline__ uint16_t floats_to_codes2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}

// 2^e of the smallest e >= kMinScaleExp with amax <= 448 * 2^e, for finite amax >= 0.
// 448 = 1.75 * 2^8, so with amax = 1.m * 2^x the exponent is x - 8, one more where the
// significand exceeds 1.75.  Zeros and subnormals take the smallest scale.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < kMinScaleExp) e = kMinScaleExp;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A word's codes with the largest of its sign in place of one that is no number (0x7f, 0xff).
__device__ __forceinline__ uint32_t number_codes(uint32_t w) {
  return w & ~((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7);
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

// A warp over a tile's rows: four lanes a row, 16 codes each.
constexpr int kQ8RowLanes = 4;
constexpr int kQ8WarpRows = 32 / kQ8RowLanes;            // rows side by side
constexpr int kQ8RowSteps = kBlockSize / kQ8WarpRows;  // rows of a tile per lane

// Multiplies the codes of a tile's rows 0 .. o0-1 by `ratio` (below 1), rounding once.  Powers
// of two keep them exact down to the subnormal codes.  By a whole warp.
__device__ __forceinline__ void rescale_rows(uint8_t* tile, float ratio, int o0, int lane) {
#pragma unroll
  for (int k = 0; k < kQ8RowSteps; ++k) {
    const int row = k * kQ8WarpRows + lane / kQ8RowLanes;
    if (row >= o0) continue;
    uint4* p = reinterpret_cast<uint4*>(tile + row * kQ8RowBytes) + lane % kQ8RowLanes;
    const uint4 c = *p;
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t out[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      uint32_t lo, hi;
      codes4_to_half2x2(in[h], lo, hi);
      const float2 a = half2_to_float2(lo), b = half2_to_float2(hi);
      out[h] = floats_to_codes2(a.x * ratio, a.y * ratio) |
               (static_cast<uint32_t>(floats_to_codes2(b.x * ratio, b.y * ratio)) << 16);
    }
    *p = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// One tile of a pool into shared memory, by one asynchronous copy.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_half2_rn(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A query row enters the products as f16 under a power of two, q 2^shift, that brings its largest
// element to [2^13, 2^14): a bf16 significand fits, and elements down to 2^-27 of the largest keep
// all their bits.  big: the largest magnitude's float bits (a row of zeros, or one with an infinity or
// a NaN, stays as it is).
__device__ __forceinline__ int query_shift(uint32_t big) {
  return big != 0u && big < 0x7f800000u ? min(126, 13 + 127 - static_cast<int>(max(big >> 23, 1u))) : 0;
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// Token of column n (0..7) of the first score n-tile; the second's are eight further.  Lane q of a
// quad owns columns 2q and 2q + 1, so its tokens are t, t + 2, t + 8 and t + 10 with t = (q & 1) +
// 4 (q >> 1): their 64-byte rows fall on both halves of the shared-memory banks, which leaves two
// wavefronts per 128 bytes for the 8-byte V reads and the 16-byte K reads alike (the natural order
// leaves four and one).
__device__ __forceinline__ int q8_token_of(int n) {
  return ((n >> 1) & 1) + 2 * (n & 1) + 4 * (n >> 2);
}

__device__ __forceinline__ bool scale_ok(float s) { return s > 0.f && s < INFINITY; }

}  // namespace pkv
