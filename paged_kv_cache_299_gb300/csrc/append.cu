// Appends with the position rotation on the way: queries and keys of the new tokens are
// rotated by their positions and keys and values stored into the paged pools, in one launch
// (slot mapping, rotation and store each cost a pass over the rows otherwise).
//
// Rotation: the 64 dims of a head row form 32 pairs (a, b), either dims (i, i + 32) or the
// neighbours (2i, 2i + 1); the pair i of a token at position p becomes
//   (a cos - b sin, b cos + a sin),   cos = table[p][i], sin = table[p][32 + i],
// evaluated in fp32 and rounded once to what is stored (bf16, or a code of the 8-bit pools).
//
// Memory-bound: every row is read once and written once.  Four lanes carry one head row, each
// both members of eight pairs, so a row's rotation needs no exchange and a lane's cosines and
// sines serve all the heads of its token.  Measured (32 query and 8 K/V heads): 16,000 prompt
// tokens 32.7 us into the bf16 pools, 6.2 TB/s or 0.91 of the measured copy rate, 32.2 us into the
// 8-bit ones, 5.6 TB/s (0.82; the block's maximum stands between its loads and its stores); a
// decode step of 64 tokens 2.0 us and of 256 into the 8-bit pools 2.3, three dependent loads
// (context, block table, scale) and the launch.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;  // (256: 36.3 us against 35.1 for 16k prompt tokens into the 8-bit pools)
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kPairs = kHeadDim / 2;
constexpr int kLanePairs = 8;                     // rotation pairs per lane: 16 dims, 32 bytes
constexpr int kLanesPerRow = kPairs / kLanePairs;  // 4
constexpr int kRowsPerWarp = 32 / kLanesPerRow;   // 8 head rows side by side
constexpr int kUnroll = 3;  // rows a lane has in flight: 48 rows (32 + 2 x 8 heads) in two rounds

// The last i in [0, n) with value(i) <= key, for value rising and value(0) <= key (0 otherwise).  A
// warp probes 32 places a step, so a batch of up to 32 sequences costs one load's latency.
template <typename Value>
__device__ __forceinline__ int32_t last_at_most(int32_t n, int64_t key, int lane, const Value& value) {
  int32_t lo = 0;
  while (n > 1) {
    const int32_t step = (n + 31) / 32;
    const int32_t i = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < n && value(lo + i) <= key);
    const int32_t skip = max(__popc(le) - 1, 0) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

// Sequence of token t (the last s with query_start_loc[s] <= t; without query_start_loc,
// sequence t) and its logical position.  false: the token is padding (at or past
// query_start_loc[num_seqs], or a context of 0 in the one-token form) or was flagged.  (Rows past
// num_tokens are flagged through token 0, as their own have no warp.)
__device__ __forceinline__ bool locate(const AppendArgs& a, int32_t t, int lane, bool report, int32_t* seq,
                                       int64_t* pos) {
  int32_t s, first, q_len;
  if (a.query_start_loc == nullptr) {
    s = t;
    first = t;
    q_len = 1;
    if (a.context_lens[s] == 0) return false;
  } else {
    const int32_t end = a.query_start_loc[a.num_seqs];
    if (t == 0 && report && end > a.num_tokens) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    if (t >= end) return false;
    s = last_at_most(a.num_seqs, t, lane, [&](int32_t i) { return a.query_start_loc[i]; });
    first = a.query_start_loc[s];
    q_len = a.query_start_loc[s + 1] - first;
  }
  const int64_t p = static_cast<int64_t>(a.context_lens[s]) - q_len + (t - first);
  if (p < 0 || t < first || t - first >= q_len || q_len > a.num_tokens - first ||
      p >= static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize ||
      (a.cos_sin != nullptr && p >= a.max_positions) || a.context_lens[s] < q_len) {
    if (report) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return false;
  }
  *seq = s;
  *pos = p;
  return true;
}

// A lane's 16 dims of a head row: both members of pairs 8 l .. 8 l + 7 (l = lane % 4), so no
// value has to travel between lanes.  kInterleaved: dims 16 l .. 16 l + 15; otherwise dims 8 l
// .. 8 l + 7 and 32 + 8 l .. 32 + 8 l + 7.  first / second: byte offsets / 16 of its two chunks.
template <bool kInterleaved>
__device__ __forceinline__ int first_chunk(int l) { return kInterleaved ? 2 * l : l; }
template <bool kInterleaved>
__device__ __forceinline__ int second_chunk(int l) { return kInterleaved ? 2 * l + 1 : 4 + l; }

struct Angles {
  float c[kLanePairs], s[kLanePairs];
};

__device__ __forceinline__ void load_angles(const float* __restrict__ row, int l, Angles& g) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + kLanePairs * l + 4 * h));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + kPairs + kLanePairs * l + 4 * h));
    g.c[4 * h] = c.x; g.c[4 * h + 1] = c.y; g.c[4 * h + 2] = c.z; g.c[4 * h + 3] = c.w;
    g.s[4 * h] = s.x; g.s[4 * h + 1] = s.y; g.s[4 * h + 2] = s.z; g.s[4 * h + 3] = s.w;
  }
}

// The lane's 16 dims in fp32: y[0..7] its first chunk, y[8..15] its second.
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&y)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = bf16x2_to_float2(w[i]);
    y[2 * i] = v.x;
    y[2 * i + 1] = v.y;
  }
}

template <bool kInterleaved>
__device__ __forceinline__ void rotate16(const Angles& g, float (&y)[16]) {
#pragma unroll
  for (int i = 0; i < kLanePairs; ++i) {
    float& a = y[kInterleaved ? 2 * i : i];
    float& b = y[kInterleaved ? 2 * i + 1 : 8 + i];
    const float x = a;
    a = x * g.c[i] - b * g.s[i];
    b = b * g.c[i] + x * g.s[i];
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float* y) {
  return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

// One warp serves rows part, part + parts, ... (eight at a time) of token t: its query rows,
// then, with kStore, its key and its value rows.  kUnroll rows a lane are loaded before the
// first is written.
template <bool kInterleaved, bool kStore>
__device__ void token_rows(const AppendArgs& a, int32_t t, int part, int parts, int lane) {
  int32_t seq;
  int64_t pos;
  if (!locate(a, t, lane, part == 0 && lane == 0, &seq, &pos)) return;
  const int l = lane % kLanesPerRow;
  const int c0 = first_chunk<kInterleaved>(l), c1 = second_chunk<kInterleaved>(l);
  Angles g;
  load_angles(a.cos_sin + pos * kHeadDim, l, g);
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
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;
  const int rows = kStore ? hq + 2 * hkv : hq;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride;
  const __nv_bfloat16* key = static_cast<const __nv_bfloat16*>(a.key) + t * a.key_stride;
  const __nv_bfloat16* value = static_cast<const __nv_bfloat16*>(a.value) + t * a.value_stride;
  const int step = parts * kRowsPerWarp;
  for (int r0 = part * kRowsPerWarp + lane / kLanesPerRow; r0 < rows; r0 += kUnroll * step) {
    uint4 x[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) continue;
      const __nv_bfloat16* src = q + r * kHeadDim;
      if (kStore && r >= hq) src = r < hq + hkv ? key + (r - hq) * kHeadDim : value + (r - hq - hkv) * kHeadDim;
      // plain loads: q_out may be q itself
      x[u][0] = reinterpret_cast<const uint4*>(src)[c0];
      x[u][1] = reinterpret_cast<const uint4*>(src)[c1];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * step;
      if (r >= rows) continue;
      __nv_bfloat16* dst;
      if (!kStore || r < hq) {
        dst = static_cast<__nv_bfloat16*>(a.q_out) + t * a.q_out_stride + r * kHeadDim;
      } else {
        const bool is_k = r < hq + hkv;
        const int h = r - hq - (is_k ? 0 : hkv);
        dst = static_cast<__nv_bfloat16*>(is_k ? a.key_cache : a.value_cache) +
              ((tile0 + h) * kBlockSize + pos % kBlockSize) * kHeadDim;
      }
      if (!kStore || r < hq + hkv) {
        float y[16];
        unpack16(x[u][0], x[u][1], y);
        rotate16<kInterleaved>(g, y);
        x[u][0] = pack8(y);
        x[u][1] = pack8(y + 8);
      }
      reinterpret_cast<uint4*>(dst)[c0] = x[u][0];
      reinterpret_cast<uint4*>(dst)[c1] = x[u][1];
    }
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

// Largest finite magnitude of sixteen values; *bad is set where one is not finite.
__device__ __forceinline__ float amax16(const float (&y)[16], bool* bad) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = fabsf(y[i]);
    if (v < INFINITY) m = fmaxf(m, v); else *bad = true;
  }
  return m;
}

// Eight values -> eight codes of y * inv; NaN becomes 0, infinities saturate.
__device__ __forceinline__ uint2 codes8(const float* y, float inv) {
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

constexpr int kRowSteps = kBlockSize / kRowsPerWarp;  // 2 rows of the block per lane

// Multiplies the codes of a tile's rows 0 .. o0-1 by `ratio` (below 1), rounding once.  Powers
// of two keep them exact down to the subnormal codes.  By a whole warp.
__device__ __forceinline__ void rescale_rows(uint8_t* tile, float ratio, int o0, int lane) {
#pragma unroll
  for (int k = 0; k < kRowSteps; ++k) {
    const int row = k * kRowsPerWarp + lane / kLanesPerRow;
    if (row >= o0) continue;
    uint4* p = reinterpret_cast<uint4*>(tile + row * kQ8RowBytes) + lane % kLanesPerRow;
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

// A lane's sixteen values as codes, into its places of a row of a tile.
template <bool kInterleaved>
__device__ __forceinline__ void store_codes(uint8_t* row, const float* y, float inv, int l) {
  const uint2 w0 = codes8(y, inv), w1 = codes8(y + 8, inv);
  if (kInterleaved) {
    reinterpret_cast<uint4*>(row)[l] = make_uint4(w0.x, w0.y, w1.x, w1.y);
  } else {
    reinterpret_cast<uint2*>(row)[first_chunk<false>(l)] = w0;
    reinterpret_cast<uint2*>(row)[second_chunk<false>(l)] = w1;
  }
}

// Decode steps (one token per sequence): one warp serves a token's rows of eight heads in one
// pool, four lanes each.  A block with earlier tokens whose scale has to grow is rescaled by
// the whole warp.  (A warp per head and pool, as chunks have it, took 4.5 us for 256
// sequences and 12.1 for 1024, this 2.5 and 3.2.)
template <bool kRotate, bool kInterleaved>
__device__ void step_rows(const AppendArgs& a, int64_t item, int lane) {
  const bool is_k = (item & 1) == 0;
  item >>= 1;
  const int groups = (a.num_kv_heads + kRowsPerWarp - 1) / kRowsPerWarp;
  const int h0 = static_cast<int>(item % groups) * kRowsPerWarp;
  const int64_t t = item / groups;
  const bool tell = lane == 0 && h0 == 0 && is_k;
  const int32_t ctx = a.context_lens[t];
  if (ctx == 0) return;  // padding
  if (ctx < 0 || static_cast<int64_t>(ctx) > static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize ||
      (kRotate && ctx > a.max_positions)) {
    if (tell) flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    return;
  }
  const int32_t pos = ctx - 1;
  const int o = pos % kBlockSize;
  const int head = min(h0 + lane / kLanesPerRow, a.num_kv_heads - 1);
  const bool active = h0 + lane / kLanesPerRow < a.num_kv_heads;
  const int l = lane % kLanesPerRow;
  const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(is_k ? a.key : a.value) +
                                   t * (is_k ? a.key_stride : a.value_stride) + head * kHeadDim;
  const uint4 x0 = ldg_nc128(reinterpret_cast<const uint4*>(src) + first_chunk<kInterleaved>(l));
  const uint4 x1 = ldg_nc128(reinterpret_cast<const uint4*>(src) + second_chunk<kInterleaved>(l));
  const bool turn = kRotate && is_k;
  Angles g = {};
  if (turn) load_angles(a.cos_sin + static_cast<int64_t>(pos) * kHeadDim, l, g);
  const int32_t phys = a.block_tables[t * a.max_blocks_per_seq + pos / kBlockSize];
  if (phys < 0 || phys >= a.num_blocks) {
    if (tell) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
    return;
  }
  const int64_t tile = static_cast<int64_t>(phys) * a.num_kv_heads + head;
  float* const scale = (is_k ? a.key_scale : a.value_scale) + tile;
  uint8_t* const pool = static_cast<uint8_t*>(is_k ? a.key_cache : a.value_cache);
  const float old = *scale;
  float y[16];
  bool bad = false;
  unpack16(x0, x1, y);
  if (turn) rotate16<kInterleaved>(g, y);
  float amax = amax16(y, &bad);
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(a.status, PA_DEVFLAG_NONFINITE);
  const bool held = o > 0;  // the block has earlier tokens
  const bool usable = !held || scale_ok(old);
  if (__any_sync(0xffffffffu, !usable) && lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_SCALE);
  const float need = scale_for(amax);
  const float now = held && !(need > old) ? old : need;
  unsigned grow = __ballot_sync(0xffffffffu, active && usable && held && need > old && l == 0);
  const float ratio = old / now;
  while (grow != 0u) {
    const int from = __ffs(grow) - 1;
    grow &= grow - 1u;
    rescale_rows(pool + __shfl_sync(0xffffffffu, tile, from) * kQ8TileBytes,
                 __shfl_sync(0xffffffffu, ratio, from), o, lane);
  }
  if (active && usable) {
    store_codes<kInterleaved>(pool + tile * kQ8TileBytes + o * kQ8RowBytes, y, 1.f / now, l);
    if (l == 0) *scale = now;  // (its four lanes have read the old one)
  }
}

// One warp serves one (sequence, block it appends to, K/V head, pool): it holds the block's
// new rows (at most 16) in registers, finds their largest magnitude, settles the scale and
// writes codes.  The tokens of a block are all this warp's, so nothing is shared between warps
// and results do not depend on any order.
template <bool kRotate, bool kInterleaved>
__device__ void block_rows(const AppendArgs& a, int64_t item, int lane) {
  const bool is_k = (item & 1) == 0;
  item >>= 1;
  const int head = static_cast<int>(item % a.num_kv_heads);
  const int64_t v = item / a.num_kv_heads;
  int32_t s;
  int64_t index;  // of the block among those the sequence appends to
  int32_t first, q_len;
  {
    // sequence s owns indices base(s) .. base(s+1)-1 with base(s) = start(s) / 16 + 2 s, at
    // least as many as the blocks its tokens can touch
    s = last_at_most(a.num_seqs, v, lane, [&](int32_t i) { return (a.query_start_loc[i] >> 4) + 2ll * i; });
    first = a.query_start_loc[s];
    q_len = a.query_start_loc[s + 1] - first;
    index = v - ((first >> 4) + 2ll * s);
    if (item == 0 && is_k && lane == 0 && a.query_start_loc[a.num_seqs] > a.num_tokens)
      flag_error(a.status, PA_DEVFLAG_BAD_CONTEXT);
    if (q_len <= 0) return;
  }
  const int64_t ctx = a.context_lens[s];
  const int64_t p0 = ctx - q_len;  // position of the first new token
  const bool tell = lane == 0 && head == 0 && index == 0 && is_k;
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
    if (lane == 0 && head == 0 && is_k) flag_error(a.status, PA_DEVFLAG_BAD_BLOCK);
    return;
  }
  const int64_t tile = static_cast<int64_t>(phys) * a.num_kv_heads + head;
  const int l = lane % kLanesPerRow;
  const int c0 = first_chunk<kInterleaved>(l), c1 = second_chunk<kInterleaved>(l);
  const int64_t t0 = first + (b * kBlockSize - p0);  // token of row 0 (may precede the chunk)
  float* const scale = (is_k ? a.key_scale : a.value_scale) + tile;
  uint8_t* const codes = static_cast<uint8_t*>(is_k ? a.key_cache : a.value_cache) + tile * kQ8TileBytes;
  const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(is_k ? a.key : a.value) + head * kHeadDim;
  const int64_t stride = is_k ? a.key_stride : a.value_stride;
  const float old = *scale;
  uint4 x[kRowSteps][2];
#pragma unroll
  for (int k = 0; k < kRowSteps; ++k) {
    const int row = k * kRowsPerWarp + lane / kLanesPerRow;
    x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
    if (row >= o0 && row < o1) {
      const uint4* p = reinterpret_cast<const uint4*>(src + (t0 + row) * stride);
      x[k][0] = ldg_nc128(p + c0);
      x[k][1] = ldg_nc128(p + c1);
    }
  }
  float y[kRowSteps][16];
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kRowSteps; ++k) {
    const int row = k * kRowsPerWarp + lane / kLanesPerRow;
    Angles g = {};
    const bool turn = kRotate && is_k && row >= o0 && row < o1;
    if (turn) load_angles(a.cos_sin + (b * kBlockSize + row) * kHeadDim, l, g);
    unpack16(x[k][0], x[k][1], y[k]);
    if (turn) rotate16<kInterleaved>(g, y[k]);
    amax = fmaxf(amax, amax16(y[k], &bad));
  }
  amax = warp_max(amax);
  if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(a.status, PA_DEVFLAG_NONFINITE);
  if (o0 > 0 && !scale_ok(old)) {
    if (lane == 0) flag_error(a.status, PA_DEVFLAG_BAD_SCALE);
    return;
  }
  // A block whose first token is written now starts with a scale of its own; otherwise it grows.
  float now = scale_for(amax);
  if (o0 > 0) {
    if (now > old)
      rescale_rows(codes, old / now, o0, lane);
    else
      now = old;
  }
  const float inv = 1.f / now;
#pragma unroll
  for (int k = 0; k < kRowSteps; ++k) {
    const int row = k * kRowsPerWarp + lane / kLanesPerRow;
    if (row >= o0 && row < o1) store_codes<kInterleaved>(codes + row * kQ8RowBytes, y[k], inv, l);
  }
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *scale = now;
}

// Item CTAs serve the blocks (or a step's tokens), the rest the query rows: the item CTAs first,
// or, with share > 0, both kinds alternating in proportion (share: item CTAs per CTA, times 2^31).
template <bool kRotate, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
rope_append_q8_kernel(const AppendArgs a, int64_t items, uint32_t item_ctas, uint32_t share, int parts) {
  const int lane = threadIdx.x & 31;
  uint32_t before = min(blockIdx.x, item_ctas);  // item CTAs before this one
  bool item = blockIdx.x < item_ctas;
  if (share > 0) {
    const uint64_t mark = static_cast<uint64_t>(blockIdx.x) * share;
    before = static_cast<uint32_t>(mark >> 31);
    item = static_cast<uint32_t>((mark + share) >> 31) > before;
  }
  if (item) {
    const int64_t w = static_cast<int64_t>(before) * kWarpsPerCta + (threadIdx.x >> 5);
    if (w >= items) return;
    if (a.query_start_loc == nullptr)
      step_rows<kRotate, kInterleaved>(a, w, lane);
    else
      block_rows<kRotate, kInterleaved>(a, w, lane);
    return;
  }
  if (kRotate) {
    const int64_t w = static_cast<int64_t>(blockIdx.x - before) * kWarpsPerCta + (threadIdx.x >> 5);
    const int64_t t = w / parts;
    if (t < a.num_tokens)
      token_rows<kInterleaved, false>(a, static_cast<int32_t>(t), static_cast<int>(w % parts),
                                      parts, lane);
  }
}

// Warps a token's rows are spread over: enough that a small batch still occupies the device
// (64 tokens 2.2 us, 3.3 with one warp each; 1024 tokens 3.4 us, 3.9 with four times the warps).
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
  const int64_t items =  // K and V
      2 * (a.query_start_loc == nullptr
               ? static_cast<int64_t>(a.num_seqs) * ((a.num_kv_heads + kRowsPerWarp - 1) / kRowsPerWarp)
               : ((static_cast<int64_t>(a.num_tokens) >> 4) + 2ll * a.num_seqs) * a.num_kv_heads);
  const int64_t item_ctas = (items + kWarpsPerCta - 1) / kWarpsPerCta;
  int parts = 1;
  int64_t q_ctas = 0;
  if (a.num_q_heads > 0) {
    parts = parts_for(a.num_tokens, a.num_q_heads);
    q_ctas = (static_cast<int64_t>(a.num_tokens) * parts + kWarpsPerCta - 1) / kWarpsPerCta;
  }
  const int64_t ctas = item_ctas + q_ctas;
  // In a batch of several waves the blocks' chains of loads run beside the queries' stream: 16,000
  // prompt tokens 32.2 us against 34.4 with the item CTAs first.  Those start a small one earlier:
  // 3000 tokens 9.8 us against 10.1, steps of 1024 tokens 3.3 against 3.6.
  constexpr int64_t kAlternateCtas = 152 * 24;
  // (rounded up: with fewer than 2^31 CTAs that adds no item CTA)
  const uint32_t share =
      ctas > kAlternateCtas && q_ctas > 0 ? static_cast<uint32_t>(((item_ctas << 31) + ctas - 1) / ctas) : 0;
  const unsigned grid = static_cast<unsigned>(ctas);
  const uint32_t first = static_cast<uint32_t>(item_ctas);
  if (a.cos_sin == nullptr)
    rope_append_q8_kernel<false, false><<<grid, kThreads, 0, stream>>>(a, items, first, share, parts);
  else if (a.interleaved)
    rope_append_q8_kernel<true, true><<<grid, kThreads, 0, stream>>>(a, items, first, share, parts);
  else
    rope_append_q8_kernel<true, false><<<grid, kThreads, 0, stream>>>(a, items, first, share, parts);
  return cudaGetLastError();
}

}  // namespace pkv
