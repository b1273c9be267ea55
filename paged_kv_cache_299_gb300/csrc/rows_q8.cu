// Causal attention of short chunks over the 8-bit pools: a few query rows per sequence (a
// verify step's K + 1 tokens), up to 32 rows per K/V head.
//
// Chunk row i of a sequence sits at position L - q_len + i and attends keys 0 .. L - q_len + i.
// The mathematics of a tile is the 8-bit decode's: one scale per tile for the scores, one for
// its share of the output; codes, queries and weights enter the tensor cores as f16.
//
// GB300 design.  With so few rows a K/V tile's bytes, not its products, are the work, and a
// 128-row tensor-memory tile would be mostly padding: the warp-level tensor-core instruction
// takes 16 rows, MT = 1 or 2 of them per K/V head.  A segment (sequence, K/V head) belongs to a
// cluster of 1 to 8 CTAs; its tiles are cut into equal runs, one per warp, each streamed through
// a ring of its own as in the decode, and the warps' partial outputs meet in shared memory, the
// CTAs' in the cluster's.  So nothing is kept outside the launch: the call needs no workspace.
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
constexpr int kRecordFloats = kHeadDim + 4;  // o, maximum (log2 units), sum, padded to 16 bytes
constexpr float kRescaleThreshold = 8.f;     // as in the decode, like the factors below
constexpr float kPShift = 7.f;
constexpr float kVFactor = 1.f / 32768.f;
constexpr int kQExp = 13;

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

// Running state of a lane's rows: row 16 mt + r (index 0) and + 8 (index 1), r = lane / 4.
template <int MT>
struct Rows {
  uint32_t q[MT][4][4];   // f16 query fragments
  float factor[MT][2];    // score factor of the row
  float m[MT][2], l[MT][2];
  float2 o[MT][2][8];
};

// One tile (16 tokens).  Fragments and dims as in the 8-bit decode; MASK: row x of the lane sees
// tokens 0 .. last[x] of the tile (none if negative), and tokens past `held` may hold anything.
template <int MT, bool MASK>
__device__ __forceinline__ void attend_tile(const uint8_t* tile, int r, int q, float ks, float vs,
                                            const int (&last)[MT][2], int held, Rows<MT>& w) {
  const int t0 = q8_token_of(2 * q, 0);
  const uint8_t* kp = tile + q8_token_of(r, 0) * kQ8RowBytes + 16 * q;
  const uint8_t* vp = tile + kQ8TileBytes + t0 * kQ8RowBytes + 8 * r;
  const uint4 k0 = lds128(kp), k1 = lds128(kp + 8 * kQ8RowBytes);
  uint2 v[4];  // tokens t0, t0 + 2, t0 + 8, t0 + 10
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = *reinterpret_cast<const uint2*>(vp + (2 * (i & 1) + 8 * (i >> 1)) * kQ8RowBytes);
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
  if (MASK) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + 2 * (i & 1) + 8 * (i >> 1) > held) v[i] = make_uint2(0u, 0u);
  }
  uint32_t p[MT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const float f = w.factor[mt][y] * ks;
      float x[4] = {s0[mt][2 * y] * f, s0[mt][2 * y + 1] * f, s1[mt][2 * y] * f, s1[mt][2 * y + 1] * f};
      if (MASK) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t0 + 2 * (i & 1) + 8 * (i >> 1) > last[mt][y]) x[i] = -INFINITY;
      }
      float t = fmaxf(max3f(x[0], x[1], x[2]), x[3]);
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
      const bool grow = t - w.m[mt][y] > kRescaleThreshold;  // (-inf - -inf is not)
      if (__any_sync(0xffffffffu, grow)) {
        const float alpha = grow ? fast_exp2(w.m[mt][y] - t) : 1.f;
        if (grow) w.m[mt][y] = t;
        w.l[mt][y] *= alpha;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w.o[mt][y][j].x *= alpha;
          w.o[mt][y][j].y *= alpha;
        }
      }
      // a row that has seen no token yet has only weights of 0
      const float ref = (MASK && w.m[mt][y] == -INFINITY ? 0.f : w.m[mt][y]) - kPShift;
      const float p0 = fast_exp2(x[0] - ref), p1 = fast_exp2(x[1] - ref);
      const float p2 = fast_exp2(x[2] - ref), p3 = fast_exp2(x[3] - ref);
      w.l[mt][y] += (p0 + p1) + (p2 + p3);
      p[mt][y] = pack_half2_rn(p0, p1);
      p[mt][2 + y] = pack_half2_rn(p2, p3);
    }
  }
  const float2 vs2 = make_float2(vs, vs);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = h ? v[0].y : v[0].x, b = h ? v[1].y : v[1].x;
    const uint32_t c = h ? v[2].y : v[2].x, d = h ? v[3].y : v[3].x;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t b00, b01, b10, b11;
      codes4_to_half2x2(__byte_perm(a, b, u ? 0x7362 : 0x5140), b00, b01);
      codes4_to_half2x2(__byte_perm(c, d, u ? 0x7362 : 0x5140), b10, b11);
      const int j = 4 * h + 2 * u;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float acc[4];
        mma_rows_zero(acc, p[mt], b00, b10);
        w.o[mt][0][j] = __ffma2_rn(make_float2(acc[0], acc[1]), vs2, w.o[mt][0][j]);
        w.o[mt][1][j] = __ffma2_rn(make_float2(acc[2], acc[3]), vs2, w.o[mt][1][j]);
        mma_rows_zero(acc, p[mt], b01, b11);
        w.o[mt][0][j + 1] = __ffma2_rn(make_float2(acc[0], acc[1]), vs2, w.o[mt][0][j + 1]);
        w.o[mt][1][j + 1] = __ffma2_rn(make_float2(acc[2], acc[3]), vs2, w.o[mt][1][j + 1]);
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

template <int MT>
constexpr int smem_bytes() {
  return kWarps * kStages * (kStageBytes + 8) + (kWarps + 1) * 16 * MT * kRecordFloats * 4;
}

template <int MT>
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
  float* folded = records + kWarps * 16 * MT * kRecordFloats;                             // [row]
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
  const int rows = q_len * p.group;  // <= 16 MT
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

  Rows<MT> w;
  // The queries, to f16 under each row's power of two (rows past the last repeat it).
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int row = min(16 * mt + 8 * y + r, rows - 1);
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(q0 + row / p.group) * p.num_q_heads + g * p.group + row % p.group) * kHeadDim) + 2 * q;
      const uint4 a = __ldg(src), b = __ldg(src + 1);
      const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t big = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) big = max(big, max((x[i] << 16) & 0x7fff0000u, x[i] & 0x7fff0000u));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      int shift = 0;
      if (big != 0u && big < 0x7f800000u)
        shift = min(126, kQExp + 127 - static_cast<int>(max(big >> 23, 1u)));
      const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
      w.factor[mt][y] = p.q_scale * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = bf16x2_to_float2(x[2 * j]), d = bf16x2_to_float2(x[2 * j + 1]);
        w.q[mt][j][y] = pack_half2_rn(c.x * up, c.y * up);
        w.q[mt][j][2 + y] = pack_half2_rn(d.x * up, d.y * up);
      }
      w.m[mt][y] = -INFINITY;
      w.l[mt][y] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) w.o[mt][y][j] = make_float2(0.f, 0.f);
    }
  }

  // blocks below this one are seen whole by every row
  const int whole = (L - q_len + 1) / kBlockSize;
  bool ok = true;
  int k = 0;
#pragma unroll 1
  for (; k < n; ++k) {
    if (k > 0 && (k & (kWindow - 1)) == 0) {
      cur = nxt;
      nxt = window(k + kWindow);
    }
    const int st = k % kStages;
    const bool here = mbar_wait(&full_bar[st], static_cast<uint32_t>((k / kStages) & 1));
    if (!(ok = __all_sync(0xffffffffu, here))) break;
    const float ks = __shfl_sync(0xffffffffu, cur.ks, k & (kWindow - 1));
    const float vs = __shfl_sync(0xffffffffu, cur.vs, k & (kWindow - 1));
    const uint8_t* tile = ring + st * kStageBytes;
    int last[MT][2] = {};
    const int first = (b_lo + k) * kBlockSize;  // token 0 of the tile
    if (b_lo + k < whole) {
      attend_tile<MT, false>(tile, r, q, ks, vs, last, kBlockSize - 1, w);
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          last[mt][y] = L - q_len + min(16 * mt + 8 * y + r, rows - 1) / p.group - first;
      attend_tile<MT, true>(tile, r, q, ks, vs, last, L - 1 - first, w);
    }
    __syncwarp();  // every lane has read the stage
    if (issued < n) {
      const int32_t a = __shfl_sync(0xffffffffu, cur.tile, issued & (kWindow - 1));
      const int32_t b = __shfl_sync(0xffffffffu, nxt.tile, issued & (kWindow - 1));
      if (lane == 0) request((issued ^ k) & ~(kWindow - 1) ? b : a, st);
      ++issued;
    }
  }
  if (!ok && lane == 0) {  // leave no copy in flight (bounded waits)
    flag_error(p.status, PA_DEVFLAG_TIMEOUT);
    for (int t = k; t < issued; ++t)
      if (!mbar_wait(&full_bar[t % kStages], static_cast<uint32_t>((t / kStages) & 1))) break;
  }

  // ---- the warps' shares meet ----
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float l = w.l[mt][y];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      float* dst = records + (warp * 16 * MT + 16 * mt + 8 * y + r) * kRecordFloats;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<float2*>(dst + 16 * q + 2 * j) = make_float2(w.o[mt][y][2 * j].x, w.o[mt][y][2 * j + 1].x);
        *reinterpret_cast<float2*>(dst + 16 * q + 8 + 2 * j) = make_float2(w.o[mt][y][2 * j].y, w.o[mt][y][2 * j + 1].y);
      }
      if (q == 0) *reinterpret_cast<float2*>(dst + kHeadDim) = make_float2(w.m[mt][y], l * kVFactor);
    }
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
        kWarps, [&](int x) { return *reinterpret_cast<const float2*>(rec + x * 16 * MT * kRecordFloats + kHeadDim); },
        [&](int x) { return *reinterpret_cast<const float4*>(rec + x * 16 * MT * kRecordFloats + 4 * c); }, M, Ls, acc);
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

template <int MT>
cudaError_t launch(const RowsParams& p, int64_t segments, int cluster, cudaStream_t stream) {
  static bool done[kMaxDevices] = {};  // benign race: the attribute calls are idempotent
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !done[dev]) {
    e = cudaFuncSetAttribute(paged_rows_q8_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<MT>());
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(paged_rows_q8_kernel<MT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(segments * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<MT>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_rows_q8_kernel<MT>, p);
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
  // CTAs per segment: as many as run side by side and have a few tiles per warp each.
  const int64_t segments = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  int cluster = 1;
  while (cluster < kMaxCluster && segments * cluster * 2 <= 2 * sms &&
         a.max_blocks_per_seq >= 2 * cluster * kWarps * kStages)
    cluster *= 2;
  return p.max_query_len * p.group <= 16 ? launch<1>(p, segments, cluster, stream)
                                         : launch<2>(p, segments, cluster, stream);
}

}  // namespace pkv
