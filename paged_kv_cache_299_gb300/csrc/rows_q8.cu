// Causal attention of short chunks over the 8-bit pools: a few query rows per sequence (a
// verify step's K + 1 tokens), up to 32 rows per K/V head.
//
// Chunk row i of a sequence sits at position L - q_len + i and attends keys 0 .. L - q_len + i.
// The mathematics of a tile is the 8-bit decode's: one scale per tile for the scores, one for
// its share of the output; codes, queries and weights enter the tensor cores as f16.
//
// GB300 design.  With so few rows a K/V tile's bytes, not its products, are the work, and a
// 128-row tensor-memory tile would be mostly padding: the warp-level tensor-core instruction
// takes rows by eights (NT = 1 to 4 groups).  A segment (sequence, K/V head) belongs to a cluster
// of 1 to 8 CTAs; its tiles are cut into equal runs, one per warp, each streamed through a ring
// of its own as in the decode, and the warps' partial outputs meet in shared memory, the CTAs'
// in the cluster's.  So nothing is kept outside the launch: the call needs no workspace.
//
// Measured, against the tensor-memory kernel on the same calls: a verify step of 32 x 5 rows,
// contexts 487-1022, 16.6 us against 22.4; 32 x 5 rows at 800 tokens 12.8 against 24.9, 256 x 5 at
// 1000 92 against 152, 4 x 5 at 131072 160 (3.4 TB/s) against 946; 128 x 8 at 4000 181 against
// 242.  Bound: by the latency of the chain score, exponential, product per tile, of which an SM
// holds twelve (44 % of the issue slots and 41 % of DRAM busy at 4 x 131072 tokens); small batches
// by start-up.  12 warps on one CTA, or 15 on three (the registers spill), were slower: 256 x 5 at
// 1000 124 and 107 us.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 6;    // streaming warps per CTA, two CTAs per SM
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;   // ring depth per warp
constexpr int kStageBytes = 2 * kQ8TileBytes;
constexpr int kWindow = 32;  // tiles whose block ids and scales are held in the lanes
constexpr int kMaxCluster = 8;
// Up to this many groups of eight rows, tiles are taken in pairs (more work side by side; beyond,
// the registers spill).  Pairs and single tiles: 32 x 2 rows at 800 tokens (one group) 8.6 and 9.1
// us, 256 x 3 at 1000 (two) 71.8 and 73.5, 256 x 5 (three) 97.3 and 92.1, 32 x 8 (four) 16.5, 15.2.
constexpr int kPairGroups = 2;
constexpr int kRecordFloats = kHeadDim + 4;  // o, maximum (log2 units), sum, padded to 16 bytes
constexpr float kRescaleThreshold = 8.f;     // as in the decode, like the factors below
constexpr float kPShift = 7.f;
constexpr float kVFactor = 1.f / 32768.f;

struct RowsParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const int32_t* query_start_loc;
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const float* key_scale;
  const float* value_scale;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  int32_t num_blocks, num_kv_heads, num_q_heads, group;
  int32_t num_query_tokens, max_query_len;
  float q_scale;  // scale * log2(e)
  int32_t* status;
};

__device__ __forceinline__ void mma_rows(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_rows_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this CTA's shared-memory address `a` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t a, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
  return d;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Running state of a lane (r = lane / 4, q = lane % 4) for NT groups of eight rows: maximum and
// sum of row 8 nt + r (the sum over the lane's own tokens), output dims 8 r .. 8 r + 7 of rows
// 8 nt + 2 q and 8 nt + 2 q + 1 (o[nt][j]: dims 8 r + 2 j, + 1, both rows each).
template <int NT>
struct Rows {
  uint32_t q[(NT + 1) / 2][4][4];  // f16 query fragments, 16 rows each
  float factor[NT];                // score factor of row 8 nt + r
  int pos[NT];                     // last key that row sees
  float m[NT], l[NT];
  float2 o[NT][4][2];
};

// T tiles (16 tokens each) at a time.  Scores are Q K^T with 16 rows a fragment, so P arrives
// with a row's neighbouring tokens in one register, which is what the second factor of O^T = V^T
// P^T wants: 16 dims by 8 rows, no padding beyond the eighth row.  Fragments and the order of
// dims and tokens as in the 8-bit decode.  MASK: row x sees tokens up to pos[x], tile t holds
// tokens from first[t] on, and tokens past `end` may hold anything.
template <int NT, int T, bool MASK>
__device__ __forceinline__ void attend_tiles(const uint8_t* const (&tiles)[T], int r, int q,
                                             const float (&ks)[T], const float (&vs)[T],
                                             const int (&first)[T], int end, Rows<NT>& w) {
  constexpr int MT = (NT + 1) / 2;
  const int t0 = q8_token_of(2 * q);
  uint2 v[T][4];  // tokens t0, t0 + 2, t0 + 8, t0 + 10
  float x[T][NT][4];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const uint8_t* kp = tiles[t] + q8_token_of(r) * kQ8RowBytes + 16 * q;
    const uint8_t* vp = tiles[t] + kQ8TileBytes + t0 * kQ8RowBytes + 8 * r;
    const uint4 k0 = lds128(kp), k1 = lds128(kp + 8 * kQ8RowBytes);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[t][i] = *reinterpret_cast<const uint2*>(vp + (2 * (i & 1) + 8 * (i >> 1)) * kQ8RowBytes);
    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
    float s0[MT][4], s1[MT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t a, b, c, d;
      codes4_to_half2x2(w0[j], a, b);
      codes4_to_half2x2(w1[j], c, d);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (j == 0) {
          mma_rows_zero(s0[mt], w.q[mt][j], a, b);
          mma_rows_zero(s1[mt], w.q[mt][j], c, d);
        } else {
          mma_rows(s0[mt], w.q[mt][j], a, b);
          mma_rows(s1[mt], w.q[mt][j], c, d);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float f = w.factor[nt] * ks[t];
      x[t][nt][0] = s0[nt >> 1][2 * (nt & 1)] * f;
      x[t][nt][1] = s0[nt >> 1][2 * (nt & 1) + 1] * f;
      x[t][nt][2] = s1[nt >> 1][2 * (nt & 1)] * f;
      x[t][nt][3] = s1[nt >> 1][2 * (nt & 1) + 1] * f;
    }
    if (MASK) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = first[t] + t0 + 2 * (i & 1) + 8 * (i >> 1);
        if (token > end) v[t][i] = make_uint2(0u, 0u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (token > w.pos[nt]) x[t][nt][i] = -INFINITY;
      }
    }
  }
  float top[NT];
  bool any = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float y = fmaxf(max3f(x[0][nt][0], x[0][nt][1], x[0][nt][2]), x[0][nt][3]);
    if (T == 2) y = max3f(max3f(y, x[T - 1][nt][0], x[T - 1][nt][1]), x[T - 1][nt][2], x[T - 1][nt][3]);
    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
    top[nt] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
    any |= top[nt] - w.m[nt] > kRescaleThreshold;  // (-inf - -inf is not)
  }
  if (__any_sync(0xffffffffu, any)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool grow = top[nt] - w.m[nt] > kRescaleThreshold;
      const float alpha = grow ? fast_exp2(w.m[nt] - top[nt]) : 1.f;
      if (grow) w.m[nt] = top[nt];
      w.l[nt] *= alpha;
      const float2 a2 = make_float2(__shfl_sync(0xffffffffu, alpha, 8 * q),  // rows 2 q and 2 q + 1
                                    __shfl_sync(0xffffffffu, alpha, 8 * q + 4));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w.o[nt][j][0] = __fmul2_rn(w.o[nt][j][0], a2);
        w.o[nt][j][1] = __fmul2_rn(w.o[nt][j][1], a2);
      }
    }
  }
  uint32_t p[T][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    // a row that has seen no token yet has only weights of 0
    const float ref = (MASK && w.m[nt] == -INFINITY ? 0.f : w.m[nt]) - kPShift;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float p0 = fast_exp2(x[t][nt][0] - ref), p1 = fast_exp2(x[t][nt][1] - ref);
      const float p2 = fast_exp2(x[t][nt][2] - ref), p3 = fast_exp2(x[t][nt][3] - ref);
      w.l[nt] += (p0 + p1) + (p2 + p3);
      p[t][nt][0] = pack_half2_rn(p0, p1);
      p[t][nt][1] = pack_half2_rn(p2, p3);
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const float2 vs2 = make_float2(vs[t], vs[t]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = h ? v[t][0].y : v[t][0].x, b = h ? v[t][1].y : v[t][1].x;
      const uint32_t c = h ? v[t][2].y : v[t][2].x, d = h ? v[t][3].y : v[t][3].x;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t f[4];  // dims 8 r + 4 h + 2 u (and + 1) by the lane's four tokens
        codes4_to_half2x2(__byte_perm(a, b, u ? 0x7362 : 0x5140), f[0], f[1]);
        codes4_to_half2x2(__byte_perm(c, d, u ? 0x7362 : 0x5140), f[2], f[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4];
          mma_rows_zero(acc, f, p[t][nt][0], p[t][nt][1]);
          float2(&o)[2] = w.o[nt][2 * h + u];
          o[0] = __ffma2_rn(make_float2(acc[0], acc[1]), vs2, o[0]);
          o[1] = __ffma2_rn(make_float2(acc[2], acc[3]), vs2, o[1]);
        }
      }
    }
  }
}

// Weighs records of one row: folds (m, l) and four dims of n records.  ml(k) and row(k) read them.
template <int N, typename ML, typename Row>
__device__ __forceinline__ void fold(int n, const ML& ml, const Row& row, float& M, float& L, float4& acc) {
  float2 x[N];
  M = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    x[k] = k < n ? ml(k) : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, x[k].x);
  }
  const float ref = M == -INFINITY ? 0.f : M;  // no token seen: weights of 0
  L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k < n) {
      const float w = fast_exp2(x[k].x - ref);
      const float4 v = row(k);
      L += w * x[k].y;
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    }
  }
}

template <int NT>
constexpr int smem_bytes() {
  return kWarps * kStages * (kStageBytes + 8) + (kWarps + 1) * 8 * NT * kRecordFloats * 4;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 2)
paged_rows_q8_kernel(const __grid_constant__ RowsParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int lane = tid & 31;
  const int r = lane >> 2, q = lane & 3;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kWarps * kStages * kStageBytes) + warp * kStages;
  float* records = reinterpret_cast<float*>(smem + kWarps * kStages * (kStageBytes + 8));  // [warp][row]
  float* folded = records + kWarps * 8 * NT * kRecordFloats;                             // [row]
  const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_size());
  const int seg = static_cast<int>(blockIdx.x) / ctas;
  const int KV = p.num_kv_heads;
  const int s = seg / KV, g = seg % KV;

  // (the same for every CTA of a cluster, so all of them leave here or none)
  const int q0 = p.query_start_loc[s];
  const int q_len = p.query_start_loc[s + 1] - q0;
  const int L = p.context_lens[s];
  if (q_len <= 0) return;
  if (q0 < 0 || q_len > p.num_query_tokens - q0 || q_len > p.max_query_len || L < q_len ||
      static_cast<int64_t>(L) > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize) {
    if (g == 0 && rank == 0 && tid == 0) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
    return;
  }
  const int rows = q_len * p.group;  // <= 8 NT
  // this warp's blocks of the segment
  const int nb = (L + kBlockSize - 1) / kBlockSize;
  const int parts = ctas * kWarps, part = rank * kWarps + warp;
  const int b_lo = static_cast<int>(static_cast<int64_t>(part) * nb / parts);
  const int n = static_cast<int>(static_cast<int64_t>(part + 1) * nb / parts) - b_lo;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full_bar[i], 1);
    fence_barrier_init();
  }
  __syncwarp();

  // Tiles (or -1: none, or a bad block) and scales of 32 blocks, one per lane.
  struct Window {
    int32_t tile;
    float ks, vs;
  };
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + b_lo;
  auto window = [&](int base) -> Window {
    Window w = {-1, 0.f, 0.f};
    bool bad = false;
    if (base + lane < n) {
      const int32_t e = __ldg(table + base + lane);
      bad = e < 0 || e >= p.num_blocks;
      if (!bad) {
        w.tile = e * KV + g;
        w.ks = __ldg(p.key_scale + w.tile);
        w.vs = __ldg(p.value_scale + w.tile) * kVFactor;
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(p.status, PA_DEVFLAG_BAD_BLOCK);
    return w;
  };
  constexpr int T = NT <= kPairGroups ? 2 : 1;  // tiles per step
  const uint64_t policy = l2_evict_first_policy();
  auto request = [&](int32_t tile, int st) {
    if (tile >= 0) {
      mbar_arrive_expect_tx(&full_bar[st], kStageBytes);
      uint8_t* dst = ring + st * kStageBytes;
      const int64_t off = static_cast<int64_t>(tile) * kQ8TileBytes;
      bulk_load(dst, p.key_cache + off, kQ8TileBytes, &full_bar[st], policy);
      bulk_load(dst + kQ8TileBytes, p.value_cache + off, kQ8TileBytes, &full_bar[st], policy);
    } else {
      mbar_arrive(&full_bar[st]);  // a bad block: release the stage with stale data
    }
  };
  Window cur = window(0);
  int issued = min(n, kStages);
  if (lane < issued) request(cur.tile, lane);
  Window nxt = window(kWindow);

  Rows<NT> w;
  // The queries, to f16 under each row's power of two (rows past the last repeat it).
#pragma unroll
  for (int nt = 0; nt < (NT + 1) / 2 * 2; ++nt) {
    const int mt = nt >> 1, y = nt & 1;
    const int row = min(8 * nt + r, rows - 1);
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + (static_cast<int64_t>(q0 + row / p.group) * p.num_q_heads + g * p.group + row % p.group) * kHeadDim) + 2 * q;
    const uint4 a = __ldg(src), b = __ldg(src + 1);
    const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t big = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, max((x[i] << 16) & 0x7fff0000u, x[i] & 0x7fff0000u));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const int shift = query_shift(big);
    const float up = power_of_two(shift);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 c = bf16x2_to_float2(x[2 * j]), d = bf16x2_to_float2(x[2 * j + 1]);
      w.q[mt][j][y] = nt < NT ? pack_half2_rn(c.x * up, c.y * up) : 0u;
      w.q[mt][j][2 + y] = nt < NT ? pack_half2_rn(d.x * up, d.y * up) : 0u;
    }
    if (nt < NT) {
      w.factor[nt] = p.q_scale * power_of_two(-shift);
      w.pos[nt] = L - q_len + row / p.group;
      w.m[nt] = -INFINITY;
      w.l[nt] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) w.o[nt][j][0] = w.o[nt][j][1] = make_float2(0.f, 0.f);
    }
  }

  // blocks below this one are seen whole by every row
  const int whole = (L - q_len + 1) / kBlockSize - b_lo;
  bool ok = true;
  int k = 0;
#pragma unroll 1
  while (k < n) {
    if (k > 0 && (k & (kWindow - 1)) == 0) {
      cur = nxt;
      nxt = window(k + kWindow);
    }
    // (windows and rings hold an even number of tiles and the steps but the last are of T, so a
    // step's tiles lie in one window)
    const int left = n - k;
    const uint8_t* tiles[T];
    float ks[T], vs[T];
    int first[T];
    bool here = true;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int at = t < left ? k + t : k;  // a step short of tiles repeats the first, unseen
      here &= mbar_wait(&full_bar[at % kStages], static_cast<uint32_t>((at / kStages) & 1));
      tiles[t] = ring + at % kStages * kStageBytes;
      ks[t] = __shfl_sync(0xffffffffu, cur.ks, at & (kWindow - 1));
      vs[t] = __shfl_sync(0xffffffffu, cur.vs, at & (kWindow - 1));
      first[t] = t < left ? (b_lo + at) * kBlockSize : 0x7fffff00;
    }
    if (!(ok = __all_sync(0xffffffffu, here))) break;
    if (k + T <= min(whole, n)) {
      attend_tiles<NT, T, false>(tiles, r, q, ks, vs, first, 0, w);
    } else {
#pragma unroll
      for (int t = 1; t < T; ++t)
        if (t >= left) vs[t] = 0.f;
      attend_tiles<NT, T, true>(tiles, r, q, ks, vs, first, L - 1, w);
    }
    __syncwarp();  // every lane has read the stages
    k += T;
    const int more = min(T, n - issued);
    if (more > 0) {
      const int i = issued + min(lane, more - 1);
      const int32_t a = __shfl_sync(0xffffffffu, cur.tile, i & (kWindow - 1));
      const int32_t b = __shfl_sync(0xffffffffu, nxt.tile, i & (kWindow - 1));
      if (lane < more) request(((issued ^ (k - T)) & ~(kWindow - 1)) != 0 ? b : a, i % kStages);
      issued += more;
    }
  }
  if (!ok && lane == 0) {  // leave no copy in flight (bounded waits)
    flag_error(p.status, PA_DEVFLAG_TIMEOUT);
    for (int t = k; t < issued; ++t)  // (the step's own first)
      if (!mbar_wait(&full_bar[t % kStages], static_cast<uint32_t>((t / kStages) & 1))) break;
  }

  // ---- the warps' shares meet ----
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float l = w.l[nt];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    float* rec = records + (warp * 8 * NT + 8 * nt) * kRecordFloats;
    if (q == 0) *reinterpret_cast<float2*>(rec + r * kRecordFloats + kHeadDim) = make_float2(w.m[nt], l * kVFactor);
    const auto& o = w.o[nt];
    float4* dst = reinterpret_cast<float4*>(rec + 2 * q * kRecordFloats + 8 * r);
    dst[0] = make_float4(o[0][0].x, o[0][1].x, o[1][0].x, o[1][1].x);
    dst[1] = make_float4(o[2][0].x, o[2][1].x, o[3][0].x, o[3][1].x);
    dst += kRecordFloats / 4;
    dst[0] = make_float4(o[0][0].y, o[0][1].y, o[1][0].y, o[1][1].y);
    dst[1] = make_float4(o[2][0].y, o[2][1].y, o[3][0].y, o[3][1].y);
  }
  __syncthreads();
  auto finish = [&](int row, int c, float Lsum, const float4& acc) {
    const float inv = 1.f / Lsum;
    __nv_bfloat16* out = p.out + (static_cast<int64_t>(q0 + row / p.group) * p.num_q_heads + g * p.group +
                                  row % p.group) * kHeadDim;
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(out + 4 * c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  };
  float M, Ls;
  float4 acc;
  for (int i = tid; i < rows * 16; i += kThreads) {  // a row's four dims
    const int row = i >> 4, c = i & 15;
    const float* rec = records + row * kRecordFloats;
    fold<kWarps>(
        kWarps, [&](int x) { return *reinterpret_cast<const float2*>(rec + x * 8 * NT * kRecordFloats + kHeadDim); },
        [&](int x) { return *reinterpret_cast<const float4*>(rec + x * 8 * NT * kRecordFloats + 4 * c); }, M, Ls, acc);
    if (ctas == 1) {
      finish(row, c, Ls, acc);
    } else {
      *reinterpret_cast<float4*>(folded + row * kRecordFloats + 4 * c) = acc;
      if (c == 0) *reinterpret_cast<float2*>(folded + row * kRecordFloats + kHeadDim) = make_float2(M, Ls);
    }
  }
  if (ctas == 1) return;
  cluster_sync();
  const uint32_t base = smem_addr(folded);
  for (int i = rank * kThreads + tid; i < rows * 16; i += ctas * kThreads) {
    const int row = i >> 4, c = i & 15;
    const uint32_t a = base + row * kRecordFloats * 4;
    fold<kMaxCluster>(
        ctas, [&](int x) { return ld_cluster2(map_rank(a + kHeadDim * 4, x)); },
        [&](int x) { return ld_cluster4(map_rank(a + 16 * c, x)); }, M, Ls, acc);
    finish(row, c, Ls, acc);
  }
  cluster_sync();  // this CTA's shared memory outlives the others' reads
}

template <int NT>
cudaError_t launch(const RowsParams& p, int64_t segments, int cluster, cudaStream_t stream) {
  static bool done[kMaxDevices] = {};  // benign race: the attribute calls are idempotent
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !done[dev]) {
    e = cudaFuncSetAttribute(paged_rows_q8_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NT>());
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(paged_rows_q8_kernel<NT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(segments * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<NT>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_rows_q8_kernel<NT>, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

bool rows_q8_takes(const AttendQ8Args& a) {
  const int group = a.num_q_heads / a.num_kv_heads;
  return static_cast<int64_t>(a.max_query_len) * group <= 32 &&
         static_cast<int64_t>(a.num_seqs) * a.num_kv_heads < (1 << 27);
}

cudaError_t launch_rows_q8(const AttendQ8Args& a, cudaStream_t stream) {
  RowsParams p;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.query_start_loc = a.query_start_loc;
  p.key_cache = static_cast<const uint8_t*>(a.key_cache);
  p.value_cache = static_cast<const uint8_t*>(a.value_cache);
  p.key_scale = a.key_scale;
  p.value_scale = a.value_scale;
  p.block_tables = a.block_tables;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.context_lens = a.context_lens;
  p.num_blocks = a.num_blocks;
  p.num_kv_heads = a.num_kv_heads;
  p.num_q_heads = a.num_q_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.num_query_tokens = a.num_query_tokens;
  p.max_query_len = a.max_query_len;
  p.q_scale = a.scale * 1.4426950408889634f;
  p.status = a.status;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs per segment: as many as run side by side, two per SM, and may have a tile per warp each
  // (5 rows at 1000 tokens 6.7 us with clusters up to that, 9.0 where it takes four tiles).
  const int64_t segments = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  int cluster = 1;
  while (cluster < kMaxCluster && segments * cluster * 2 <= 2 * sms &&
         a.max_blocks_per_seq >= 2 * cluster * kWarps)
    cluster *= 2;
  switch ((p.max_query_len * p.group + 7) / 8) {  // groups of eight rows
    case 1: return launch<1>(p, segments, cluster, stream);
    case 2: return launch<2>(p, segments, cluster, stream);
    case 3: return launch<3>(p, segments, cluster, stream);
    default: return launch<4>(p, segments, cluster, stream);
  }
}

}  // namespace pkv
