// Attention of drafted trees over a paged cache, bf16 and 8-bit pools.
//
// A sequence's last q_len tokens are the nodes of a tree (their keys and values stored already) behind
// a prefix of P = L - q_len tokens.  Row i sees every key of the prefix and drafted key j where bit j of
// its mask row is set:
//   out_i = sum_j softmax_j(scale q_i . K_j) V_j over the keys it sees, 0 where it sees none.
//
// One warp per (row, query head), a key per lane.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;

template <bool Q8>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const TreeArgs a) {
  __shared__ float sq[kWarps][kHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int32_t row = static_cast<int32_t>(w / a.num_q_heads);
  const int head = static_cast<int>(w % a.num_q_heads);
  if (row >= a.num_query_tokens) return;
  int32_t s = 0;
  while (s < a.num_seqs && a.query_start_loc[s + 1] <= row) ++s;
  if (s >= a.num_seqs) return;
  const int32_t q0 = a.query_start_loc[s], q_len = a.query_start_loc[s + 1] - q0, L = a.context_lens[s];
  if (q0 < 0 || row < q0 || q_len > a.num_query_tokens - q0 || q_len > a.max_query_len || L < q_len ||
      static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize) {
    if (lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return;
  }
  const int g = head / (a.num_q_heads / a.num_kv_heads);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + w * kHeadDim;
  sq[warp][lane] = __bfloat162float(q[lane]);
  sq[warp][lane + 32] = __bfloat162float(q[lane + 32]);
  __syncwarp();
  const int P = L - q_len;
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int32_t* bits = a.tree_mask + static_cast<int64_t>(row) * a.mask_words;
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int k0 = 0; k0 < L; k0 += 32) {
    const int k = k0 + lane;
    bool seen = k < L && (k < P || ((bits[(k - P) >> 5] >> ((k - P) & 31)) & 1) != 0);
    int64_t at = 0;  // row of the pool
    if (seen) {
      const int32_t b = table[k / kBlockSize];
      if (b < 0 || b >= a.num_blocks) {
        flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
        seen = false;
      } else {
        at = (static_cast<int64_t>(b) * a.num_kv_heads + g) * kBlockSize + k % kBlockSize;
      }
    }
    float x = -INFINITY;
    if (seen) {
      x = 0.f;
      for (int d = 0; d < kHeadDim; d += 4) {
        float4 f;
        if (Q8) {
          uint32_t lo, hi;
          codes4_to_half2x2(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.key_cache) + at * kHeadDim + d), lo, hi);
          const float2 y = half2_to_float2(lo), z = half2_to_float2(hi);
          f = make_float4(y.x, y.y, z.x, z.y);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.key_cache) + at * kHeadDim + d);
          const float2 y = bf16x2_to_float2(u.x), z = bf16x2_to_float2(u.y);
          f = make_float4(y.x, y.y, z.x, z.y);
        }
        x += sq[warp][d] * f.x + sq[warp][d + 1] * f.y + sq[warp][d + 2] * f.z + sq[warp][d + 3] * f.w;
      }
      x *= a.scale * 1.4426950408889634f;
      if (Q8) x *= a.key_scale[at / kBlockSize];
    }
    float top = x;
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float m_new = fmaxf(m, top);
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = fast_exp2(m - ref);
    m = m_new;
    const float p = seen ? fast_exp2(x - ref) : 0.f;
    l = l * alpha + p;
    o0 *= alpha;
    o1 *= alpha;
    for (int j = 0; j < 32; ++j) {
      if (!__shfl_sync(0xffffffffu, seen, j)) continue;
      const float pj = __shfl_sync(0xffffffffu, p, j);
      const int64_t aj = __shfl_sync(0xffffffffu, at, j);
      if (Q8) {
        uint32_t lo, hi;
        codes4_to_half2x2(*reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(a.value_cache) + aj * kHeadDim + 2 * lane), lo, hi);
        const float2 v = half2_to_float2(lo);
        const float sc = a.value_scale[aj / kBlockSize];
        o0 += pj * (v.x * sc);
        o1 += pj * (v.y * sc);
      } else {
        const float2 v = bf16x2_to_float2(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.value_cache) + aj * kHeadDim)[lane]);
        o0 += pj * v.x;
        o1 += pj * v.y;
      }
    }
  }
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
  reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + w * kHeadDim)[lane] =
      __floats2bfloat162_rn(o0 * inv, o1 * inv);
}

}  // namespace

size_t tree_workspace_size() { return 16; }

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(a.num_query_tokens) * a.num_q_heads;
  tree_kernel<false><<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_q8(const TreeArgs& a, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(a.num_query_tokens) * a.num_q_heads;
  tree_kernel<true><<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
