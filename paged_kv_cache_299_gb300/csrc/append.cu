// Appends with the position rotation on the way: queries and keys of the new tokens are
// rotated by their positions and keys and values stored into the paged pools, in one launch
// (slot mapping, rotation and store each cost a pass over the rows otherwise).
//
// Rotation: the 64 dims of a head row form 32 pairs (a, b), either dims (i, i + 32) or the
// neighbours (2i, 2i + 1); the pair i of a token at position p becomes
//   (a cos - b sin, b cos + a sin),   cos = table[p][i], sin = table[p][32 + i],
// evaluated in fp32 and rounded once to what is stored (bf16, or a code of the 8-bit pools).
//
// Memory-bound: every row is read once and written once.  Eight lanes carry one head row (16
// bytes each); the partner dims of the (i, i + 32) form sit four lanes away.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kChunkDims = 8;                       // dims per lane (16 bytes of bf16)
constexpr int kLanesPerRow = kHeadDim / kChunkDims;  // 8
constexpr int kRowsPerWarp = 32 / kLanesPerRow;     // 4 head rows side by side
constexpr int kPairs = kHeadDim / 2;

// Sequence of token t (the last s with query_start_loc[s] <= t; without query_start_loc,
// sequence t) and its logical position.  false: the token is padding (at or past
// query_start_loc[num_seqs], or a context of 0 in the one-token form) or was flagged.
__device__ __forceinline__ bool locate(const AppendArgs& a, int32_t t, bool report, int32_t* seq,
                                       int64_t* pos) {
  int32_t s, first, q_len;
  if (a.query_start_loc == nullptr) {
    s = t;
    first = t;
    q_len = 1;
    if (a.context_lens[s] == 0) return false;
  } else {
    if (t >= a.query_start_loc[a.num_seqs]) return false;
    int32_t lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (a.query_start_loc[mid] <= t) lo = mid; else hi = mid - 1;
    }
    s = lo;
    first = a.query_start_loc[s];
    q_len = a.query_start_loc[s + 1] - first;
  }
  const int64_t p = static_cast<int64_t>(a.context_lens[s]) - q_len + (t - first);
  if (p < 0 || t < first || t - first >= q_len ||
      p >= static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize ||
      (a.cos_sin != nullptr && p >= a.max_positions) || a.context_lens[s] < q_len) {
    if (report) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return false;
  }
  *seq = s;
  *pos = p;
  return true;
}

// The cosines and (signed) sines a lane applies to its eight dims, y = own * c + other * s:
// kInterleaved: four pairs, c[i] / s[i] of pair 4 * lane + i.  Otherwise eight, those of dims
// 8 * (lane & 3) .. + 7, the sines negated in the first half of the row.
struct Angles {
  float c[kChunkDims], s[kChunkDims];
};

template <bool kInterleaved>
__device__ __forceinline__ void load_angles(const float* __restrict__ row, int chunk, Angles& g) {
  if (kInterleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * chunk));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + kPairs + 4 * chunk));
    g.c[0] = c.x; g.c[1] = c.y; g.c[2] = c.z; g.c[3] = c.w;
    g.s[0] = s.x; g.s[1] = s.y; g.s[2] = s.z; g.s[3] = s.w;
  } else {
    const int i0 = kChunkDims * (chunk & 3);
    const float sign = chunk < 4 ? -1.f : 1.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + i0 + 4 * h));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + kPairs + i0 + 4 * h));
      g.c[4 * h] = c.x; g.c[4 * h + 1] = c.y; g.c[4 * h + 2] = c.z; g.c[4 * h + 3] = c.w;
      g.s[4 * h] = sign * s.x; g.s[4 * h + 1] = sign * s.y;
      g.s[4 * h + 2] = sign * s.z; g.s[4 * h + 3] = sign * s.w;
    }
  }
}

// Eight dims of a row, rotated, in fp32.  All 32 lanes take part (the partner dims travel by
// shuffles); x is this lane's 16 bytes.
template <bool kInterleaved>
__device__ __forceinline__ void rotate8(const uint4 x, const Angles& g, float (&y)[kChunkDims]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = bf16x2_to_float2(w[i]);
    if (kInterleaved) {
      y[2 * i] = v.x * g.c[i] - v.y * g.s[i];
      y[2 * i + 1] = v.y * g.c[i] + v.x * g.s[i];
    } else {
      const float2 o = bf16x2_to_float2(__shfl_xor_sync(0xffffffffu, w[i], 4));
      y[2 * i] = v.x * g.c[2 * i] + o.x * g.s[2 * i];
      y[2 * i + 1] = v.y * g.c[2 * i + 1] + o.y * g.s[2 * i + 1];
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float (&y)[kChunkDims]) {
  return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

// One warp serves rows part, part + parts, ... (four at a time) of token t: its query rows,
// then, with kStore, its key and its value rows.
template <bool kInterleaved, bool kStore>
__device__ void token_rows(const AppendArgs& a, int32_t t, int part, int parts, int lane) {
  int32_t seq;
  int64_t pos;
  if (!locate(a, t, part == 0 && lane == 0, &seq, &pos)) return;
  const int chunk = lane % kLanesPerRow;
  int64_t tile0 = 0;  // first (block, head) tile of the token's block
  if (kStore) {
    const int32_t phys =
        a.block_tables[static_cast<int64_t>(seq) * a.max_blocks_per_seq + pos / kBlockSize];
    if (phys < 0 || phys >= a.num_blocks) {
      if (part == 0 && lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
      return;
    }
    tile0 = static_cast<int64_t>(phys) * a.num_kv_heads;
  }
  Angles g;
  load_angles<kInterleaved>(a.cos_sin + pos * kHeadDim, chunk, g);
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int rows = kStore ? hq + 2 * hkv : hq;
  for (int r0 = part * kRowsPerWarp; r0 < rows; r0 += parts * kRowsPerWarp) {
    const int r = r0 + lane / kLanesPerRow;
    const bool valid = r < rows;
    const __nv_bfloat16* src = nullptr;
    __nv_bfloat16* dst = nullptr;
    bool turn = true;
    if (valid) {
      if (r < hq) {
        src = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride + r * kHeadDim;
        dst = static_cast<__nv_bfloat16*>(a.q_out) + t * a.q_out_stride + r * kHeadDim;
      } else {
        const bool is_k = r < hq + hkv;
        const int h = r - hq - (is_k ? 0 : hkv);
        src = is_k ? static_cast<const __nv_bfloat16*>(a.key) + t * a.key_stride
                   : static_cast<const __nv_bfloat16*>(a.value) + t * a.value_stride;
        src += h * kHeadDim;
        dst = static_cast<__nv_bfloat16*>(is_k ? a.key_cache : a.value_cache) +
              ((tile0 + h) * kBlockSize + pos % kBlockSize) * kHeadDim;
        turn = is_k;
      }
    }
    // plain loads: q_out may be q itself
    uint4 x = valid ? reinterpret_cast<const uint4*>(src)[chunk] : make_uint4(0, 0, 0, 0);
    float y[kChunkDims];
    rotate8<kInterleaved>(x, g, y);
    if (turn) x = pack8(y);
    if (valid) reinterpret_cast<uint4*>(dst)[chunk] = x;
  }
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const AppendArgs a, int parts) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  const int64_t t = w / parts;
  if (t >= a.num_tokens) return;
  token_rows<kInterleaved, true>(a, static_cast<int32_t>(t), static_cast<int>(w % parts), parts,
                                 threadIdx.x & 31);
}

// ---- 8-bit pools ---------------------------------------------------------------------------
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// Largest finite magnitude of eight values; *bad is set where one is not finite.
__device__ __forceinline__ float amax8(const float (&y)[kChunkDims], bool* bad) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kChunkDims; ++i) {
    const float v = fabsf(y[i]);
    if (v < INFINITY) m = fmaxf(m, v); else *bad = true;
  }
  return m;
}

// Eight values -> eight codes of y * inv; NaN becomes 0, infinities saturate.
__device__ __forceinline__ uint2 codes8(const float (&y)[kChunkDims], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = y[4 * h + i] * inv;
      if (v[i] != v[i]) v[i] = 0.f;
    }
    w[h] = floats_to_codes2(v[0], v[1]) |
           (static_cast<uint32_t>(floats_to_codes2(v[2], v[3])) << 16);
  }
  return make_uint2(w[0], w[1]);
}

constexpr int kRowSteps = kBlockSize / kRowsPerWarp;  // 4 rows of the block per lane

// Scale of a block that receives new values of largest magnitude amax, and the rescaling of
// the codes it holds already (rows 0 .. o0-1).  A block whose first token is written now
// starts with a scale of its own; otherwise the scale only grows from `old`.  Powers of two
// keep the rescaled codes exact down to the subnormal codes.
__device__ __forceinline__ float settle_scale(float old, uint8_t* tile, float amax, int o0,
                                              int lane) {
  float s = scale_for(amax);
  if (o0 > 0) {
    if (s > old) {
      const float ratio = old / s;
#pragma unroll
      for (int k = 0; k < kRowSteps; ++k) {
        const int row = k * kRowsPerWarp + lane / kLanesPerRow;
        if (row >= o0) continue;
        uint2* p = reinterpret_cast<uint2*>(tile + row * kQ8RowBytes) + lane % kLanesPerRow;
        const uint2 c = *p;
        const uint32_t in[2] = {c.x, c.y};
        uint32_t out[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t lo, hi;
          codes4_to_half2x2(in[h], lo, hi);
          const float2 a = half2_to_float2(lo), b = half2_to_float2(hi);
          out[h] = floats_to_codes2(a.x * ratio, a.y * ratio) |
                   (static_cast<uint32_t>(floats_to_codes2(b.x * ratio, b.y * ratio)) << 16);
        }
        *p = make_uint2(out[0], out[1]);
      }
    } else {
      s = old;
    }
  }
  return s;
}

// One warp serves one (sequence, block it appends to, K/V head): it holds the block's new
// rows of K and V (at most 16 each) in registers, finds their largest magnitudes, settles
// the two scales and writes codes.  The tokens of a block are all this warp's, so nothing is
// shared between warps and results do not depend on any order.
template <bool kRotate, bool kInterleaved>
__device__ void block_rows(const AppendArgs& a, int64_t item, int lane) {
  const int head = static_cast<int>(item % a.num_kv_heads);
  const int64_t v = item / a.num_kv_heads;
  int32_t s;
  int64_t index;  // of the block among those the sequence appends to
  int32_t first, q_len;
  if (a.query_start_loc == nullptr) {
    s = static_cast<int32_t>(v);
    index = 0;
    first = s;
    q_len = 1;
    if (a.context_lens[s] == 0) return;  // padding
  } else {
    // sequence s owns indices base(s) .. base(s+1)-1 with base(s) = start(s) / 16 + 2 s, at
    // least as many as the blocks its tokens can touch
    int32_t lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if ((a.query_start_loc[mid] >> 4) + 2ll * mid <= v) lo = mid; else hi = mid - 1;
    }
    s = lo;
    first = a.query_start_loc[s];
    q_len = a.query_start_loc[s + 1] - first;
    index = v - ((first >> 4) + 2ll * s);
    if (q_len <= 0) return;
  }
  const int64_t ctx = a.context_lens[s];
  const int64_t p0 = ctx - q_len;  // position of the first new token
  const bool tell = lane == 0 && head == 0 && index == 0;
  if (first < 0 || static_cast<int64_t>(first) + q_len > a.num_tokens || p0 < 0 ||
      ctx > static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize ||
      (kRotate && ctx > a.max_positions)) {
    if (tell) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return;
  }
  const int64_t b = p0 / kBlockSize + index;
  if (index < 0 || b * kBlockSize >= ctx) return;  // no such block
  const int o0 = index == 0 ? static_cast<int>(p0 % kBlockSize) : 0;
  const int o1 = static_cast<int>(ctx - b * kBlockSize < kBlockSize ? ctx - b * kBlockSize : kBlockSize);
  const int32_t phys = a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + b];
  if (phys < 0 || phys >= a.num_blocks) {
    if (lane == 0 && head == 0) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
    return;
  }
  const int64_t tile = static_cast<int64_t>(phys) * a.num_kv_heads + head;
  const int chunk = lane % kLanesPerRow;
  const int64_t t0 = first + (b * kBlockSize - p0);  // token of row 0 (may precede the chunk)
  const float k_old = a.key_scale[tile], v_old = a.value_scale[tile];
  uint4 kx[kRowSteps], vx[kRowSteps];
#pragma unroll
  for (int k = 0; k < kRowSteps; ++k) {
    const int row = k * kRowsPerWarp + lane / kLanesPerRow;
    const bool valid = row >= o0 && row < o1;
    kx[k] = vx[k] = make_uint4(0, 0, 0, 0);
    if (valid) {
      kx[k] = ldg_nc128(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.key) +
                                                       (t0 + row) * a.key_stride + head * kHeadDim) + chunk);
      vx[k] = ldg_nc128(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.value) +
                                                       (t0 + row) * a.value_stride + head * kHeadDim) + chunk);
    }
  }
  float ky[kRowSteps][kChunkDims];
  float kmax = 0.f, vmax = 0.f;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kRowSteps; ++k) {
    const int row = k * kRowsPerWarp + lane / kLanesPerRow;
    if (kRotate) {
      const bool valid = row >= o0 && row < o1;
      Angles g = {};
      if (valid) load_angles<kInterleaved>(a.cos_sin + (b * kBlockSize + row) * kHeadDim, chunk, g);
      rotate8<kInterleaved>(kx[k], g, ky[k]);
    } else {
      const uint32_t w[4] = {kx[k].x, kx[k].y, kx[k].z, kx[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_float2(w[i]);
        ky[k][2 * i] = f.x;
        ky[k][2 * i + 1] = f.y;
      }
    }
    kmax = fmaxf(kmax, amax8(ky[k], &bad));
    float vy[kChunkDims];
    const uint32_t w[4] = {vx[k].x, vx[k].y, vx[k].z, vx[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(w[i]);
      vy[2 * i] = f.x;
      vy[2 * i + 1] = f.y;
    }
    vmax = fmaxf(vmax, amax8(vy, &bad));
  }
  kmax = warp_max(kmax);
  vmax = warp_max(vmax);
  if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(a.status, PA_DEVFLAG_NONFINITE);
  uint8_t* kt = static_cast<uint8_t*>(a.key_cache) + tile * kQ8TileBytes;
  uint8_t* vt = static_cast<uint8_t*>(a.value_cache) + tile * kQ8TileBytes;
  if (o0 > 0 && !(scale_ok(k_old) && scale_ok(v_old))) {
    if (lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_SCALE);
    return;
  }
  const float ks = settle_scale(k_old, kt, kmax, o0, lane);
  const float vs = settle_scale(v_old, vt, vmax, o0, lane);
  const float ki = 1.f / ks, vi = 1.f / vs;
#pragma unroll
  for (int k = 0; k < kRowSteps; ++k) {
    const int row = k * kRowsPerWarp + lane / kLanesPerRow;
    if (row < o0 || row >= o1) continue;
    float vy[kChunkDims];
    const uint32_t w[4] = {vx[k].x, vx[k].y, vx[k].z, vx[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(w[i]);
      vy[2 * i] = f.x;
      vy[2 * i + 1] = f.y;
    }
    reinterpret_cast<uint2*>(kt + row * kQ8RowBytes)[chunk] = codes8(ky[k], ki);
    reinterpret_cast<uint2*>(vt + row * kQ8RowBytes)[chunk] = codes8(vy, vi);
  }
  __syncwarp();  // every lane has read the old scales
  if (lane == 0) {
    a.key_scale[tile] = ks;
    a.value_scale[tile] = vs;
  }
}

// Warps 0 .. items-1 serve the blocks, the rest the query rows.
template <bool kRotate, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
rope_append_q8_kernel(const AppendArgs a, int64_t items, int64_t item_ctas, int parts) {
  const int lane = threadIdx.x & 31;
  if (blockIdx.x < item_ctas) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
    if (w < items) block_rows<kRotate, kInterleaved>(a, w, lane);
    return;
  }
  if (kRotate) {
    const int64_t w = (blockIdx.x - item_ctas) * kWarpsPerCta + (threadIdx.x >> 5);
    const int64_t t = w / parts;
    if (t < a.num_tokens)
      token_rows<kInterleaved, false>(a, static_cast<int32_t>(t), static_cast<int>(w % parts),
                                      parts, lane);
  }
}

// Warps a token's rows are spread over: enough that a small batch still occupies the device.
int parts_for(int64_t tokens, int rows) {
  constexpr int64_t kWarpsWanted = 152 * 16;
  const int most = (rows + kRowsPerWarp - 1) / kRowsPerWarp;
  const int64_t parts = tokens > 0 ? kWarpsWanted / tokens : 1;
  return static_cast<int>(parts < 1 ? 1 : parts > most ? most : parts);
}

}  // namespace

cudaError_t launch_rope_append(const AppendArgs& a, cudaStream_t stream) {
  const int parts = parts_for(a.num_tokens, a.num_q_heads + 2 * a.num_kv_heads);
  const int64_t ctas = (static_cast<int64_t>(a.num_tokens) * parts + kWarpsPerCta - 1) / kWarpsPerCta;
  if (a.interleaved)
    rope_append_kernel<true><<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(a, parts);
  else
    rope_append_kernel<false><<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(a, parts);
  return cudaGetLastError();
}

cudaError_t launch_rope_append_q8(const AppendArgs& a, cudaStream_t stream) {
  const int64_t blocks = a.query_start_loc == nullptr
                             ? a.num_seqs
                             : (static_cast<int64_t>(a.num_tokens) >> 4) + 2ll * a.num_seqs;
  const int64_t items = blocks * a.num_kv_heads;
  const int64_t item_ctas = (items + kWarpsPerCta - 1) / kWarpsPerCta;
  int parts = 1;
  int64_t q_ctas = 0;
  if (a.num_q_heads > 0) {
    parts = parts_for(a.num_tokens, a.num_q_heads);
    q_ctas = (static_cast<int64_t>(a.num_tokens) * parts + kWarpsPerCta - 1) / kWarpsPerCta;
  }
  const unsigned grid = static_cast<unsigned>(item_ctas + q_ctas);
  if (a.cos_sin == nullptr)
    rope_append_q8_kernel<false, false><<<grid, kThreads, 0, stream>>>(a, items, item_ctas, parts);
  else if (a.interleaved)
    rope_append_q8_kernel<true, true><<<grid, kThreads, 0, stream>>>(a, items, item_ctas, parts);
  else
    rope_append_q8_kernel<true, false><<<grid, kThreads, 0, stream>>>(a, items, item_ctas, parts);
  return cudaGetLastError();
}

}  // namespace pkv
