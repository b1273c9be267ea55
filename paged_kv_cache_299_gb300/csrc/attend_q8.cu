// Attention over the 8-bit pools, in its simplest form: one warp per (query row, query head)
// walks the row's keys with a running maximum and sum.
//   s_j = scale * q . (code_j * key_scale),  out = sum_j p_j (code_j * value_scale) / sum_j p_j
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {

namespace {

// Row of q -> sequence and number of keys it sees; false: nothing to serve.
__device__ __forceinline__ bool row_keys(const AttendQ8Args& a, int32_t row, bool report, int32_t* seq,
                                         int32_t* keys) {
  int32_t s = row, first = row, q_len = 1;
  if (a.query_start_loc != nullptr) {
    if (row >= a.query_start_loc[a.num_seqs]) return false;
    int32_t lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (a.query_start_loc[mid] <= row) lo = mid; else hi = mid - 1;
    }
    s = lo;
    first = a.query_start_loc[s];
    q_len = a.query_start_loc[s + 1] - first;
  }
  const int32_t L = a.context_lens[s];
  if (L < 0 || (a.query_start_loc != nullptr && L < q_len) || row < first || row - first >= q_len ||
      static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize) {
    if (report) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return false;
  }
  *seq = s;
  *keys = L - q_len + (row - first) + 1;
  if (a.query_start_loc == nullptr) *keys = L;
  return true;
}

__global__ void __launch_bounds__(128) attend_q8_rows_kernel(const AttendQ8Args a, int64_t rows) {
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= rows * a.num_q_heads) return;
  const int32_t row = static_cast<int32_t>(w / a.num_q_heads);
  const int h = static_cast<int>(w % a.num_q_heads);
  const int g = h / (a.num_q_heads / a.num_kv_heads);
  int32_t s, keys;
  if (!row_keys(a, row, h == 0 && lane == 0, &s, &keys)) return;
  const uint32_t* q32 = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                          w * kHeadDim);
  const float2 q = bf16x2_to_float2(q32[lane]);
  const float qs = a.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  for (int32_t j0 = 0; j0 < keys; j0 += kBlockSize) {
    const int32_t phys = table[j0 / kBlockSize];
    if (phys < 0 || phys >= a.num_blocks) {
      if (lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
      return;
    }
    const int64_t tile = static_cast<int64_t>(phys) * a.num_kv_heads + g;
    const uint16_t* kt = reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(a.key_cache) + tile * kQ8TileBytes);
    const uint16_t* vt = reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(a.value_cache) + tile * kQ8TileBytes);
    const float ks = a.key_scale[tile], vs = a.value_scale[tile];
    const int n = min(kBlockSize, keys - j0);
    for (int j = 0; j < n; ++j) {
      const float2 k = half2_to_float2(codes2_to_half2(kt[j * 32 + lane]));
      const float2 v = half2_to_float2(codes2_to_half2(vt[j * 32 + lane]));
      float x = q.x * k.x + q.y * k.y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= qs * ks;
      const float mn = fmaxf(m, x);
      const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float p = exp2f(x - mn);
      l = l * keep + p;
      o.x = o.x * keep + p * v.x * vs;
      o.y = o.y * keep + p * v.y * vs;
      m = mn;
    }
  }
  const float inv = keys > 0 ? 1.f / l : 0.f;  // no keys: a zero row
  reinterpret_cast<__nv_bfloat162*>(a.out)[w * (kHeadDim / 2) + lane] =
      __floats2bfloat162_rn(o.x * inv, o.y * inv);
}

}  // namespace

cudaError_t launch_attend_q8_rows(const AttendQ8Args& a, cudaStream_t stream) {
  const int64_t rows = a.query_start_loc == nullptr ? a.num_seqs : a.num_query_tokens;
  const int64_t warps = rows * a.num_q_heads;
  attend_q8_rows_kernel<<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(a, rows);
  return cudaGetLastError();
}

}  // namespace pkv
