// Attention of drafted trees over a paged cache, bf16 and 8-bit pools, on tcgen05 tensor cores.
//
// A sequence's last q_len tokens are the nodes of a tree (their keys and values stored already) behind
// a prefix of P = L - q_len tokens.  Row i sees every key of the prefix and drafted key j where bit j of
// its mask row is set:
//   out_i = sum_j softmax_j(scale q_i . K_j) V_j over the keys it sees, 0 where it sees none.
//
// GB300 design.  The rows are few and the keys many: what counts is to stream K and V past 128 MMA rows
// (128 / GROUP tokens x GROUP heads that share a K/V head) on every SM, whatever the batch looks like.
//   * The work is a row of 128-key tiles: all tiles of all (sequence, K/V head, query tile) segments, one
//     after the other, for a persistent grid that fills every SM.  Where there are CTAs enough, every
//     segment gets CTAs of its own, as many as bring the longest piece down; otherwise, or where lengths are
//     so uneven that equal shares win, the row is cut into equal runs, one per CTA, that begin and end
//     inside segments.  A segment that one CTA serves whole goes straight to the output; pieces of a split
//     one are kept in fp32 (sum, maximum, weight) in the workspace, and the warp that finishes last for its
//     rows weighs them together, in the pieces' order (many pieces in groups, then the groups): the result
//     does not depend on who that is.
//   * Trees of at most 128 rows (64 over 8 bits): two CTAs per SM of one half (128 MMA rows) each, because a tile's chain
//     (scores, softmax, product) is latency: 128 keys a tile amortise it, two chains fill in for each other.
//     Larger ones: one CTA per SM with two halves that share every K and V tile, which is fetched, and
//     converted, once for 256 rows (8-bit 2 x 131072 x 60: 324 us with 128 rows a CTA, 197 with halves, when they came;
//     bf16 4 x 131072 x 26, 104 rows: 180 us with 128, 205 with halves; 32 ragged trees, of up to 128: 19.6 and 29.0).
//   * Tensor memory (256 columns a half): scores S 128, P 64 (bf16 pairs), O 64.  P has columns of its own,
//     so the next tile's scores are issued as soon as the row warps have read this tile's.
//   * Row warps, eight a half: two threads per row, 64 keys each.  Each also reads its partner's scores,
//     for their maximum alone (a reduction that comes with the load), so both follow the same running
//     maximum without meeting.  Exponentials and row sums in fp32, P as bf16 (what the
//     product takes; up to 2^-8 of each weight, of both signs, so that sums lose far less); O is rescaled
//     in place when a row's maximum grows past the headroom left above it.
//   * One warp issues the MMAs: S = Q K^T (M128 N128 K64) and O += P V (M128 N64 K128); one the copies.
//   * Masks are looked at only in tiles that hold drafted keys.  There the row warps also clear V rows
//     past the context, and elements of drafted values that are no numbers (0 x NaN would reach rows
//     that do not see them); the rows that do see them get them back in the epilogue.
//   * 8-bit pools: six more warps (two for K, four for V; four and four beside two halves) turn codes into bf16 (exact) in shared memory.  With the value scale of
//     a block written as 2^e f, 1 <= f < 2: V becomes 2^e code, f rides in the exponent of the weights and
//     leaves the row sum again by 1 / f; the key scale multiplies the block's scores.
// Measured (GB300, 32 query and 8 K/V heads, us in a graph; floor: K and V read once at the copy rate):
// 26 nodes over four contexts of 131,072 179 (floor 159: 6.0 TB/s, 0.89 of the copy rate; DRAM), over one of
// 131,072 67, of 16,000 26; 12 over one of 300 10.3 and 32 ragged trees over 100-1500 18.7 (the start: plan,
// table, first tile, some 5 us; the masked last tile; the meeting of pieces, some 2.5 us); 60 nodes over
// four of 131,072 266 (256 rows: a tile's chain, 2,350 cycles).  8-bit: 60 over two of 131,072 181 (floor 68)
// and 48 mixed trees 50 (floor 7.4): instructions (7,900 a tile of 256 rows, 2,200 of them the converters', at 66 %
// of the issue slots: 3,000 cycles) and 3 to 5 us from one piece to the next.
// Every mbarrier wait is bounded; on timeout the CTA records PA_DEVFLAG_TIMEOUT, drains its own copies
// and MMAs, frees its tensor memory, counts its pieces as delivered and returns.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kTileM = 128;  // MMA rows of one half
constexpr int kTileN = 128;  // keys per tile
constexpr int kBlocksPerTile = kTileN / kBlockSize;
constexpr int kHalfWarps = 8;                 // row warps of one half
constexpr int kQBytes = kTileM * kRowBytes;   // 16 KiB
constexpr int kOpBytes = kTileN * kRowBytes;  // one K or V tile of bf16: 16 KiB
constexpr int kRawBytes = 2 * kTileN * kQ8RowBytes;  // codes of K, then of V
constexpr int kConsts = 3 * kBlocksPerTile;   // score factor, log2 f, 1 / f of every block
constexpr int kMaxMaskWords = 32;
constexpr float kHeadroom = 8.0f;  // the reference of the exponents lies this far (log2) above the maximum
constexpr float kLargeScore = 131072.f;  // 2^17: a rounding of the score (log2 units) is then 2^-7
constexpr int kPartChunks = kHeadDim / 8 + 1;  // float4s of a row for each half of the dims: sum; maximum, weight
constexpr int kRecordFloat4s = 2 * kPartChunks * kTileM;  // of one half
constexpr int kMinPiece = 6;      // tiles of a piece of a split segment, at least (4, 6 and 8: 32 ragged trees 20.1, 19.6, 19.8 us)
// What meeting costs, in tiles: equal runs begin to pay beyond it (bf16, 3, 5 and 8: 16 x 8000 x 32 61.5, 60.1,
// 59.8 us, 20 x 2000 x 32 31.3, 31.3, 28.3; 8 bits, 3 and 5: 16 x 8000 x 32 83.3 and 91.8, 4 x 16000 x 26 48.0, 54.0).
constexpr int kSplitTilesBf16 = 8, kSplitTilesQ8 = 3;
constexpr int kFlatPieces = 10;   // so many pieces are weighed at once, more by groups first: one warp's loads
constexpr int kGroupPieces = 8;   // of a record take 0.4 us, a meeting of a group 2
constexpr int kTogether = 3;      // records whose loads are in flight at a time
// What a piece costs beside its tiles, in tiles (bf16, 1, 3, 4 and 5: 64 x 1-8192 x 4-64 87.2, 77.9, 75.5, 77.0 us,
// 40 x 1-32000 x 8-60 131.9, 121.9, 116.2, 117.3; 8 bits: 48 x 1-8192 x 4-64 53.2, 50.5, 51.8, 53.3, 40 x 1-32000 x 8-60
// 149.5, 135.5, 137.9, 140.6).
constexpr int kPieceTilesBf16 = 4, kPieceTilesQ8 = 3;
constexpr int kRowsBlocks = 128;  // 8-bit blocks per CTA of the few-rows kernel, at most: some 20 us
constexpr int kMaxDealtSeqs = 1024;  // sequences whose segments may get CTAs of their own
constexpr int kPieceRing = 4;
constexpr int kWalkBytes = 56;

struct TreeParams {
  __nv_bfloat16* out;
  const int32_t* tree_mask;
  const int32_t* query_start_loc;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const __nv_bfloat16* value_cache;  // bf16 pools
  const float* key_scale;            // 8-bit pools
  const float* value_scale;
  int32_t* counters;  // [grid][row warps] pieces delivered by each of the segment that starts in a CTA and goes on
  // [grid][2][row warps] the same of groups of pieces, by the CTA of a group's first piece: a later group of the
  // segment that comes from the CTAs before, or the first of the one that starts there (a CTA can hold both).
  int32_t* group_counters;
  float4* records;    // [grid][2][halves][half of the dims][kPartChunks][128]
  int32_t* status;
  int32_t mask_words, max_blocks_per_seq, num_blocks, num_kv_heads, num_q_heads;
  int32_t num_query_tokens, max_query_len, num_seqs;
  float qk_scale;  // scale * log2(e)
};

// a / b, a >= 0 and b > 0: a division of 64 bits takes several hundred cycles, one of 32 a quarter of that.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The sequence whose tiles a run is in.
struct Seq {
  int s, q0, q_len, L;
  int tiles;    // of a segment
  int q_tiles;  // segments of a K/V head; 0: none to serve
};

// Sequences without rows have no work; ones that cannot be served are reported (when `report`).
template <int TOKENS>
__device__ __forceinline__ void load_seq(const TreeParams& p, int s, bool report, Seq& q) {
  q.s = s;
  q.q0 = __ldg(p.query_start_loc + s);
  q.q_len = __ldg(p.query_start_loc + s + 1) - q.q0;
  q.L = __ldg(p.context_lens + s);
  q.q_tiles = 0;
  q.tiles = 1;
  if (q.q_len == 0) return;
  if (q.q_len < 0 || q.q0 < 0 || q.q_len > p.num_query_tokens - q.q0 || q.q_len > p.max_query_len || q.L < q.q_len ||
      q.L > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize ||
      q.L > static_cast<int64_t>(p.num_blocks) * kBlockSize) {
    if (report) flag_error(p.status, PA_DEVFLAG_BAD_CONTEXT);
    return;
  }
  q.tiles = (q.L + kTileN - 1) / kTileN;
  q.q_tiles = (q.q_len + TOKENS - 1) / TOKENS;
}

// A segment's length in the row of all tiles: what it costs beside its tiles comes first.
template <int COST>
__device__ __forceinline__ int span(const Seq& q) { return q.tiles + COST; }

// A piece of a segment: key tiles j0 .. j0 + n - 1 of the query tile that begins at tok0, against K/V head g.
struct Piece {
  int s, g, q0, q_len, L, tok0;
  int j0, n;     // n == 0: none
  int from, to;  // the CTAs that the segment is split over: one, if the piece is all of it
};

// Walks a run: the query tiles of a K/V head, then the next head's, then the next sequence's.
struct Walk {
  int64_t at, end;  // the next tile and the run's end among all
  Seq q;
  int g, q_tile, v;  // the segment, and its tile
};

// w.q is set; the walk begins at place `off` of its sequence's `length`-long segments.
__device__ __forceinline__ int enter_seq(Walk& w, int64_t off, int length) {
  const int64_t seg = quotient(off, length);
  w.g = static_cast<int>(quotient(seg, w.q.q_tiles));
  w.q_tile = static_cast<int>(seg - static_cast<int64_t>(w.g) * w.q.q_tiles);
  return static_cast<int>(off - seg * length);
}

static_assert(sizeof(Walk) == kWalkBytes, "room for a walk");

// Where all CTAs' runs lie: run r holds tiles total r / runs .. total (r + 1) / runs - 1.
struct Runs {
  int64_t total;
  int runs;
  int own_first, own_last;  // the CTAs of the one segment this CTA has a piece of; -1: it has a run of all tiles
};
__device__ __forceinline__ int64_t run_start(const Runs& x, int64_t r) { return quotient(x.total * r, x.runs); }
// The run that holds a tile (none is empty).
__device__ __forceinline__ int run_of(const Runs& x, int64_t tile) {
  return static_cast<int>(quotient((tile + 1) * x.runs + x.total - 1, x.total) - 1);
}

template <int TOKENS, int COST>
__device__ __forceinline__ bool next_piece(const TreeParams& p, const Runs& runs, Walk& w, Piece& u) {
  while (w.at < w.end) {
    while (w.q.q_tiles == 0 || w.g == p.num_kv_heads) {
      load_seq<TOKENS>(p, w.q.s + 1, false, w.q);
      w.g = w.q_tile = w.v = 0;
    }
    const int n = static_cast<int>(min(static_cast<int64_t>(span<COST>(w.q) - w.v), w.end - w.at));
    const int64_t first = w.at - w.v;  // where the segment begins
    u.s = w.q.s;
    u.q0 = w.q.q0;
    u.q_len = w.q.q_len;
    u.L = w.q.L;
    u.g = w.g;
    u.tok0 = w.q_tile * TOKENS;
    u.j0 = max(w.v - COST, 0);
    u.n = w.v + n - COST - u.j0;
    w.at += n;
    w.v += n;
    if (w.v == span<COST>(w.q)) {
      w.v = 0;
      if (++w.q_tile == w.q.q_tiles) {
        w.q_tile = 0;
        ++w.g;
      }
    }
    if (u.n <= 0) continue;  // (nothing but what comes before the tiles)
    u.from = runs.own_first;
    u.to = runs.own_last;
    if (runs.own_first < 0) {
      u.from = u.to = static_cast<int>(blockIdx.x);
      if (u.j0 > 0) u.from = run_of(runs, first + COST);
      if (u.j0 + u.n < w.q.tiles) u.to = run_of(runs, first + span<COST>(w.q) - 1);
    }
    return true;
  }
  return false;
}

// HALVES 1: 128 rows a CTA, two CTAs per SM; 2: 256 rows that share every K and V tile, one CTA per SM.
template <bool Q8, int HALVES>
struct Layout {
  static constexpr int kRowWarps = HALVES * kHalfWarps;
  static constexpr int kMmaWarp = kRowWarps, kProducerWarp = kRowWarps + 1, kConvWarp0 = kRowWarps + 2;
  static constexpr int kKWarps = Q8 ? (HALVES == 1 ? 2 : 4) : 0, kVWarps = Q8 ? 4 : 0;
  static constexpr int kThreads = Q8 ? (HALVES == 1 ? 512 : 896) : (kRowWarps + 2) * 32;
  static constexpr int kCtasPerSm = HALVES == 1 ? 2 : 1;
  // Register split of the 8-bit kernels (setmaxnreg): what the CTA was launched with.
  static constexpr int kRowRegs = HALVES == 1 ? 88 : 96, kOtherRegs = 40;
  static constexpr uint32_t kTmemCols = 256 * HALVES;
  static constexpr uint32_t kSCol = 0, kPCol = 128 * HALVES, kOCol = 192 * HALVES;  // + 128, 64, 64 per half
  static constexpr int kRing = Q8 ? (HALVES == 1 ? 2 : 3) : (HALVES == 1 ? 3 : 6);  // stages of K and V operands
  static constexpr int kRawRing = HALVES == 1 ? 2 : 4;                               // stages of codes
  static constexpr int kConstRing = HALVES == 1 ? 4 : 8;  // tiles whose score constants are kept (kRing + 2, at least)
  static constexpr int kKOff = HALVES * kQBytes;
  static constexpr int kVOff = kKOff + kRing * kOpBytes;
  static constexpr int kRawOff = kVOff + kRing * kOpBytes;
  static constexpr int kConstOff = kRawOff + (Q8 ? kRawRing * kRawBytes : 0);
  static constexpr int kRawScaleOff = kConstOff + (Q8 ? kConstRing * kConsts * 4 : 0);
  static constexpr int kBarOff = kRawScaleOff + (Q8 ? kRawRing * 2 * kBlocksPerTile * 4 : 0);
  static constexpr int kNumBars = 6 * HALVES + 2 + 2 * kRing + (Q8 ? 2 * kRawRing + 2 * kRing : 0);
  static constexpr int kMiscOff = kBarOff + (kNumBars + 1) / 2 * 16;
  static constexpr int kPieceOff = kMiscOff + 16 + 4 * kRowWarps;  // the row warps' pieces and the walks
  static constexpr int kOddOff = kPieceOff + kPieceRing * static_cast<int>(sizeof(Piece)) + 2 * kWalkBytes + static_cast<int>(sizeof(Runs));
  static constexpr int kKeysOff = kOddOff;  // 8-bit pools: [kRawRing]
  // drafted tokens whose values are no numbers: [3][any; 32 words of bits]
  static constexpr int kBytes = kOddOff + (Q8 ? 4 * kRawRing : 3 * (1 + kMaxMaskWords) * 4);
  static_assert(kCtasPerSm * (kBytes + 1024) <= 228 * 1024, "CTAs of an SM fit in its shared memory");
};

// Bits o .. o + 31 of what a row sees, counted from the first drafted key: below 0 the prefix, from q_len
// on nothing.
__device__ __forceinline__ uint32_t mask_word(const int32_t* bits, int q_len, int i) {
  if (i < 0) return 0xffffffffu;
  const int left = q_len - 32 * i;
  if (left <= 0) return 0u;
  const uint32_t w = static_cast<uint32_t>(__ldg(bits + i));
  return left >= 32 ? w : w & ((1u << left) - 1u);
}
__device__ __forceinline__ uint32_t seen_bits(const int32_t* bits, int q_len, int o) {
  return __funnelshift_r(mask_word(bits, q_len, o >> 5), mask_word(bits, q_len, (o >> 5) + 1), o & 31);
}

// A bf16 pair's elements that are no numbers (infinities and NaNs): ones in their halves.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// wait_ready, its unusual case out of line where OUT: the loops of the roles share the instruction caches.  The
// issuing and loading warps over bf16 pools: 100 trees of 5-16 nodes over 50-3000 tokens 62.9 us against 65.6; over 8
// bits a call costs them registers (2 x 131072 x 60 195 us against 183).  The converters: 180.5 us against 183.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return wait_or_abort(bar, parity, abort_flag, status);
}
template <bool OUT>
__device__ __forceinline__ bool wait_role(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if (!OUT) return wait_ready(bar, parity, abort_flag, status);
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, status);
}

template <int GROUP, bool Q8, int HALVES>
__global__ void __launch_bounds__(Layout<Q8, HALVES>::kThreads, Layout<Q8, HALVES>::kCtasPerSm)
tree_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
            const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ TreeParams p) {
  using Lay = Layout<Q8, HALVES>;
  constexpr int kThreads = Lay::kThreads, kRing = Lay::kRing, kRawRing = Lay::kRawRing;
  constexpr int kConstRing = Lay::kConstRing;
  constexpr int kRowWarps = Lay::kRowWarps, kConvWarp0 = Lay::kConvWarp0;
  constexpr int kKWarps = Lay::kKWarps, kVWarps = Lay::kVWarps;
  constexpr int kMmaWarp = Lay::kMmaWarp, kProducerWarp = Lay::kProducerWarp;
  constexpr int kHalfTokens = kTileM / GROUP;      // query tokens of a half
  constexpr int kTokens = HALVES * kHalfTokens;    // and of a segment
  constexpr int kSplitTiles = Q8 ? kSplitTilesQ8 : kSplitTilesBf16;
  constexpr int kPieceTiles = Q8 ? kPieceTilesQ8 : kPieceTilesBf16;
  static_assert(kSplitTiles < kThreads / 32, "a warp for every length tried");
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (so that what depends on it stays uniform)
  const int lane = tid & 31;
  extern __shared__ __align__(1024) uint8_t smem[];  // 128-byte swizzle atoms need 1 KiB
  if ((smem_addr(smem) & 1023u) != 0) {
    if (tid == 0) flag_error(p.status, PA_DEVFLAG_LAYOUT);
    return;
  }
  uint8_t* sq = smem;
  uint8_t* sk = smem + Lay::kKOff;
  uint8_t* sv = smem + Lay::kVOff;
  uint8_t* sraw = smem + Lay::kRawOff;
  float* consts = reinterpret_cast<float*>(smem + Lay::kConstOff);
  float* raw_scale = reinterpret_cast<float*>(smem + Lay::kRawScaleOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBarOff);
  // [HALVES] each.  A half without rows in a piece takes no part in it; phases count what it took part in.
  uint64_t* q_full = bars;             // a piece's Q landed
  uint64_t* s_full = q_full + HALVES;  // scores in tensor memory
  uint64_t* s_free = s_full + HALVES;  // and read into registers
  uint64_t* p_full = s_free + HALVES;  // P in tensor memory
  uint64_t* o_free = p_full + HALVES;  // O of a finished piece read out
  uint64_t* pv_done = o_free + HALVES;  // P V of a tile done: P free, O up to date
  uint64_t* l_bar = pv_done + HALVES;   // all row warps: the sums of a row exchanged
  uint64_t* drain = l_bar + 1;
  uint64_t* kv_full = drain + 1;          // [kRing] K (and V, from bf16 pools) of a tile there
  uint64_t* tile_done = kv_full + kRing;  // [kRing] P V of a tile done: its stage is free
  uint64_t* v_full = tile_done + kRing;   // 8-bit pools: [kRing] V converted
  uint64_t* k_empty = v_full + kRing;     // [kRing] scores that read K done
  uint64_t* raw_full = k_empty + kRing;   // [kRawRing] codes and scales landed
  uint64_t* raw_empty = raw_full + kRawRing;
  int* misc = reinterpret_cast<int*>(smem + Lay::kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int& abort_flag = *reinterpret_cast<volatile int*>(misc + 1);
  int* own_first = misc + 2;  // CTAs of the one segment this CTA has a piece of; -1: a run of the row of tiles
  int* own_last = misc + 3;
  int* raw_keys = reinterpret_cast<int*>(smem + Lay::kKeysOff);  // keys of the context from a stage's first on; 0: the end
  uint32_t* odd = reinterpret_cast<uint32_t*>(smem + Lay::kOddOff);
  auto piece_slot = [&](int u) -> Piece* {
    return reinterpret_cast<Piece*>(smem + Lay::kPieceOff + (u & (kPieceRing - 1)) * sizeof(Piece));
  };
  Walk* const row_walk = reinterpret_cast<Walk*>(smem + Lay::kPieceOff + kPieceRing * static_cast<int>(sizeof(Piece)));
  Walk* const start_walk = row_walk + 1;
  Runs* const shared_runs = reinterpret_cast<Runs*>(start_walk + 1);
  int* delivered = misc + 4;  // [row warps] pieces of split segments that each row warp has delivered

  if (tid == 0) {
    for (int h = 0; h < HALVES; ++h) {
      mbar_init(&q_full[h], 1);
      mbar_init(&s_full[h], Q8 ? 2 : 1);
      mbar_init(&s_free[h], kHalfWarps);
      mbar_init(&p_full[h], kHalfWarps);
      mbar_init(&o_free[h], kHalfWarps);
      mbar_init(&pv_done[h], 1);
    }
    mbar_init(l_bar, kRowWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&kv_full[i], Q8 ? kKWarps : 1);
      mbar_init(&tile_done[i], 1);
      if (Q8) {
        mbar_init(&v_full[i], kVWarps);
        mbar_init(&k_empty[i], 1);
      }
    }
    if (Q8) {
      for (int i = 0; i < kRawRing; ++i) {
        mbar_init(&raw_full[i], 1 + kBlocksPerTile);
        mbar_init(&raw_empty[i], kKWarps + kVWarps);
      }
    }
    fence_barrier_init();
    abort_flag = 0;
    piece_slot(0)->n = 0;
    start_walk->at = start_walk->end = 0;
    *own_first = *own_last = -1;
    for (int i = 0; i < kRowWarps; ++i) delivered[i] = 0;
  }
  if (!Q8 && tid < 3 * (1 + kMaxMaskWords)) odd[tid] = 0u;
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, Lay::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tensormap(&tmap_q);
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
  }
  // ---- the plan: what this CTA serves ----
  Runs runs;
  runs.own_first = runs.own_last = -1;
  {
    const int ctas = static_cast<int>(gridDim.x);
    // CTAs of their own are dealt under the shortest piece length for which the pieces are no more than the
    // CTAs; no shorter one fits, and one longer by kSplitTiles is no better than equal runs.
    auto shortest = [&](int segments) {
      return max(static_cast<int>(quotient(runs.total - kPieceTiles * segments + ctas - 1, ctas)), kMinPiece);
    };
    auto inclusive = [&](auto x) {
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const auto y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      return x;
    };
    // This CTA's run begins at place `off` of sequence q, or its piece is number `off` of q's: by one thread.
    auto settle = [&](const Seq& q, int64_t off, int length) {
      Walk w;
      w.q = q;
      if (length > 0) {
        const int pieces = (q.tiles + length - 1) / length;
        const int k = enter_seq(w, off, pieces);
        const int j0 = static_cast<int>(quotient(static_cast<int64_t>(q.tiles) * k, pieces));
        const int j1 = static_cast<int>(quotient(static_cast<int64_t>(q.tiles) * (k + 1), pieces));
        w.v = kPieceTiles + j0;
        w.at = 0;  // the walk ends with the piece
        w.end = j1 - j0;
        runs.own_first = static_cast<int>(blockIdx.x) - k;
        runs.own_last = runs.own_first + pieces - 1;
      } else {
        w.v = enter_seq(w, off, span<kPieceTiles>(q));
        w.at = run_start(runs, blockIdx.x);
        w.end = run_start(runs, blockIdx.x + 1);
      }
      *start_walk = w;
      *own_first = runs.own_first;
      *own_last = runs.own_last;
      // the row warps' first two pieces
      Piece x;
      if (!next_piece<kTokens, kPieceTiles>(p, runs, w, x)) x.n = 0;
      *piece_slot(0) = x;
      if (length > 0 || !next_piece<kTokens, kPieceTiles>(p, runs, w, x)) x.n = 0;
      *piece_slot(1) = x;
      *row_walk = w;
    };
    if (p.num_seqs <= 32) {
      // one warp, a sequence per lane: the CTA need not meet
      if (warp == 0) {
        Seq q;
        q.q_tiles = 0;
        q.tiles = 1;
        if (lane < p.num_seqs) load_seq<kTokens>(p, lane, blockIdx.x == 0, q);
        const int segments = q.q_tiles * p.num_kv_heads;
        const int64_t tiles = static_cast<int64_t>(span<kPieceTiles>(q)) * segments;
        int64_t upto = inclusive(tiles);
        runs.total = __shfl_sync(0xffffffffu, upto, 31);
        runs.runs = static_cast<int>(min(static_cast<int64_t>(ctas), max(runs.total, int64_t{1})));
        const int all = __reduce_add_sync(0xffffffffu, segments);
        int length = 0, pieces = 0;
        if (all <= ctas && runs.total > 0) {
          const int low = shortest(all);
          for (int t = 0; t <= kSplitTiles && length == 0; ++t) {
            pieces = segments * ((q.tiles + low + t - 1) / (low + t));
            if (__reduce_add_sync(0xffffffffu, pieces) <= ctas) length = low + t;
          }
        }
        const int64_t mine = length > 0 ? pieces : tiles;
        if (length > 0) upto = inclusive(pieces);
        const int64_t want = length > 0 ? blockIdx.x
                             : static_cast<int>(blockIdx.x) < runs.runs ? run_start(runs, blockIdx.x) : -1;
        if (lane == 0) *shared_runs = runs;
        if (want >= upto - mine && want < upto) settle(q, want - (upto - mine), length);
      }
    } else {
      int64_t* warp_sum = reinterpret_cast<int64_t*>(smem);  // (before any copy lands there)
      int* seq_tiles = reinterpret_cast<int*>(smem + 1024);  // of every sequence, and its segments
      int* seq_segments = seq_tiles + kMaxDealtSeqs;
      int* tried = seq_segments + kMaxDealtSeqs;  // CTAs wanted by each warp's piece length
      const int per = (p.num_seqs + kThreads - 1) / kThreads;
      const int s0 = min(tid * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
      int64_t mine = 0, segments = 0;  // tiles, then CTAs wanted
      Seq q;
      for (int s = s0; s < s1; ++s) {
        load_seq<kTokens>(p, s, blockIdx.x == 0, q);
        const int n = q.q_tiles * p.num_kv_heads;
        mine += static_cast<int64_t>(span<kPieceTiles>(q)) * n;
        segments += n;
        if (p.num_seqs <= kMaxDealtSeqs) {
          seq_tiles[s] = q.tiles;
          seq_segments[s] = n;
        }
      }
      // the sum of what the threads before this one have, and of all
      auto scan = [&](int64_t x, int64_t* sums, int64_t* total) -> int64_t {
        const int64_t upto = inclusive(x);
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int64_t first = upto - x;
        *total = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
          if (i < warp) first += sums[i];
          *total += sums[i];
        }
        return first;
      };
      // (a number of segments beyond the CTAs' matters no further)
      const int some = static_cast<int>(min(segments, int64_t{ctas} + 1));
      const int most = __reduce_max_sync(0xffffffffu, some), sum = __reduce_add_sync(0xffffffffu, some);
      if (lane == 0) tried[warp] = most > ctas ? most : sum;
      int64_t before = scan(mine, warp_sum, &runs.total);
      int64_t all = 0;
      for (int i = 0; i < kThreads / 32; ++i) all += tried[i];
      runs.runs = static_cast<int>(min(static_cast<int64_t>(ctas), max(runs.total, int64_t{1})));
      int length = 0;
      if (p.num_seqs <= kMaxDealtSeqs && all <= ctas && runs.total > 0) {
        __syncthreads();  // (`tried` has been read)
        const int t = shortest(static_cast<int>(all)) + min(warp, kSplitTiles);  // every warp tries a length
        int wanted = 0;
        for (int s = lane; s < p.num_seqs; s += 32) wanted += seq_segments[s] * ((seq_tiles[s] + t - 1) / t);
        wanted = __reduce_add_sync(0xffffffffu, wanted);
        if (lane == 0) tried[warp] = wanted <= ctas ? t : 0;
        __syncthreads();
        for (int i = kSplitTiles; i >= 0; --i)
          if (tried[i] > 0) length = tried[i];
      }
      int64_t want = static_cast<int>(blockIdx.x) < runs.runs ? run_start(runs, blockIdx.x) : -1;
      if (length > 0) {
        mine = 0;
        for (int s = s0; s < s1; ++s) mine += seq_segments[s] * ((seq_tiles[s] + length - 1) / length);
        int64_t total;
        before = scan(mine, warp_sum + kThreads / 32, &total);
        want = blockIdx.x;
      }
      if (tid == 0) *shared_runs = runs;
      if (want >= before && want < before + mine) {
        int64_t off = want - before;
        for (int s = s0; s < s1; ++s) {
          load_seq<kTokens>(p, s, false, q);
          const int64_t n = static_cast<int64_t>(length > 0 ? (q.tiles + length - 1) / length : span<kPieceTiles>(q)) *
                            (q.q_tiles * p.num_kv_heads);
          if (off < n) {
            settle(q, off, length);
            break;
          }
          off -= n;
        }
      }
    }
  }
  fence_proxy_async_smem();  // the plan's scratch before copies touch the buffers
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  runs = *shared_runs;
  runs.own_first = *own_first;
  runs.own_last = *own_last;
  // Whether a half holds any token of a piece, and any of the 32 MMA rows of row warp w.
  auto half_active = [&](const Piece& u, int h) { return u.tok0 + h * kHalfTokens < u.q_len; };
  auto warp_active = [&](const Piece& u, int w) {
    return u.tok0 + (w / kHalfWarps) * kHalfTokens + (w & 3) * 32 / GROUP < u.q_len;
  };
  // Where row warps w deliver the group of a segment's pieces (from CTA `from` on) whose first is CTA `first`'s.
  auto group_counter = [&](int first, int from, int w) -> int32_t* {
    return p.group_counters + (2 * first + (first == from ? 1 : 0)) * kRowWarps + w;
  };

  if (warp < kRowWarps) {
    // ============================ row warps ============================
    if (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Lay::kRowRegs));
    const int half = warp / kHalfWarps;
    const int part = (warp >> 2) & 1;      // keys 64 part .. 64 part + 63 of every tile
    const int r = (warp & 3) * 32 + lane;  // MMA row == TMEM lane; also a key of the tile, for V
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_mine = lane_addr + Lay::kSCol + half * kTileN + part * (kTileN / 2);
    const uint32_t s_theirs = s_mine ^ (kTileN / 2);
    const uint32_t p_addr = lane_addr + Lay::kPCol + half * (kTileN / 2) + part * (kTileN / 4);
    const uint32_t o_addr = p_addr + (Lay::kOCol - Lay::kPCol);
    const uint32_t o_theirs = o_addr ^ (kHeadDim / 2);
    auto wait_row = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_ready(bar, parity, &abort_flag, p.status));
    };
    // this row's mask, and how far into its tile the first drafted key lies
    auto mask_row = [&](const Piece* u) -> const int32_t* {
      return p.tree_mask + static_cast<int64_t>(u->q0 + min(u->tok0 + half * kHalfTokens + r / GROUP, u->q_len - 1)) * p.mask_words;
    };
    auto cur_lead = [&](const Piece* u) -> int { return (u->L - u->q_len) % kTileN; };
    // This thread's share of a CTA's record: of its piece of the segment that begins there, or else.
    auto record_of = [&](int cta, bool begins) -> float4* {
      return p.records + ((2ll * cta + (begins ? 1 : 0)) * HALVES + half) * kRecordFloat4s + part * kPartChunks * kTileM + r;
    };
    const bool q_loader = (warp & (kHalfWarps - 1)) == 0 && lane == 0;
    auto load_q = [&](const Piece& x) {
      mbar_arrive_expect_tx(&q_full[half], kQBytes);
      tma_load_3d(sq + half * kQBytes, &tmap_q, 0, x.g * GROUP, x.q0 + x.tok0 + half * kHalfTokens, &q_full[half]);
    };
    auto wanted = [&](int u) { return piece_slot(u)->n > 0 && half_active(*piece_slot(u), half); };
    if (q_loader && wanted(0)) load_q(*piece_slot(0));
    bool ok = true;
    int c = 0;       // tiles that this half took part in
    int skipped = 0;  // and ones of pieces without rows for it (half 1)
    int units = 0;   // pieces so far
    int took = 0;    // and those this half took part in
    // until the half's last P V is done
    auto wait_pv = [&]() -> bool { return wait_row(&pv_done[half], static_cast<uint32_t>((c - 1) & 1)); };
    // V rows past the context weigh nothing but may hold anything, and so may drafted values that some row
    // does not see: in a tile that starts at drafted key `base`, this thread clears half of row r of what
    // lies past the last one, and elements that are no numbers, whose tokens it notes down.
    auto clear_values = [&](const Piece* cur, int base) -> bool {
      const int ring = c % kRing;  // (half 0 takes part in every tile)
      if (!wait_row(&kv_full[ring], static_cast<uint32_t>(c / kRing & 1))) return false;
      const int key = base + r;
      if (key >= 0) {
        uint32_t any = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4* x = reinterpret_cast<uint4*>(sv + ring * kOpBytes + swz(r, 4 * part + i));
          if (key >= cur->q_len) {
            *x = make_uint4(0u, 0u, 0u, 0u);
          } else {
            const uint4 y = *x;
            const uint4 z = make_uint4(odd_halves(y.x), odd_halves(y.y), odd_halves(y.z), odd_halves(y.w));
            if ((z.x | z.y | z.z | z.w) != 0u) {
              any = 1u;
              *x = make_uint4(y.x & ~z.x, y.y & ~z.y, y.z & ~z.z, y.w & ~z.w);
            }
          }
        }
        if (any != 0u) {
          uint32_t* const my_odd = odd + units % 3 * (1 + kMaxMaskWords);
          atomicOr(my_odd + 1 + (key >> 5), 1u << (key & 31));
          atomicOr(my_odd, 1u);
        }
      }
      fence_proxy_async_smem();
      return true;
    };
    // Pieces come through shared memory, written two ahead by one thread, so that the tiles' loop keeps its
    // registers (and the MMA warp has them too).  Piece u + 2 is written in piece u, when all row warps have left
    // piece u - 2, whose slot it takes; they look it up after they met in the epilogue of u or u + 1.
    for (; ok && piece_slot(units)->n > 0; ++units) {
      const Piece* const cur = piece_slot(units);
      const int n = cur->n;
      const int tail_j = (cur->L - cur->q_len) / kTileN - cur->j0;  // from here on tiles hold drafted keys
      if (HALVES > 1 && !half_active(*cur, half)) {  // (half 1)
        // (the next piece's Q is wanted before half 0 can finish this one)
        if (q_loader && wanted(units + 1)) load_q(*piece_slot(units + 1));
        if (lane == 0) mbar_arrive(l_bar);
        ok = wait_row(l_bar, static_cast<uint32_t>(units & 1));
        skipped += n;
        continue;
      }
      ++took;
      if (!warp_active(*cur, warp)) {
        // a warp without rows keeps the others' pace (its rows of P and O may hold anything)
        for (int j = 0; ok && j < n; ++j, ++c) {
          if (!(ok = wait_row(&s_full[half], static_cast<uint32_t>(c & 1)))) break;
          if (lane == 0) mbar_arrive(&s_free[half]);
          if (!Q8 && half == 0 && j >= tail_j && !(ok = clear_values(cur, (j - tail_j) * kTileN - cur_lead(cur)))) break;
          // (the next scores may be there before the others' P: an arrival now would count for theirs)
          if (c > 0 && !(ok = wait_pv())) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[half]);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(l_bar);
        if (!(ok = wait_row(l_bar, static_cast<uint32_t>(units & 1)))) break;
        if (lane == 0) mbar_arrive(&o_free[half]);
        continue;
      }
      prefetch_l1(mask_row(cur));
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++c) {
        if (!(ok = wait_row(&s_full[half], static_cast<uint32_t>(c & 1)))) break;
        tc_fence_after_sync();
        // the piece's last scores are done with Q: the next piece's may land there
        if (j == n - 1 && q_loader && wanted(units + 1)) load_q(*piece_slot(units + 1));
        uint32_t v[2][32];
        float top[kBlocksPerTile / 2];  // largest raw score of each block
#pragma unroll
        for (int b = 0; b < kBlocksPerTile / 2; ++b)
          tmem_ld16_max(s_theirs + 16 * b, &v[b >> 1][16 * (b & 1)], top[b]);
        tmem_wait_ld();
        const bool tail = j >= tail_j;  // (uniform)
        if (tail) {
          const int base = (j - tail_j) * kTileN - cur_lead(cur) + (part ^ 1) * (kTileN / 2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (base + 32 * h + 32 <= 0) continue;  // keys of the prefix (uniform)
            const uint32_t seen = seen_bits(mask_row(cur), cur->q_len, base + 32 * h);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float x = -INFINITY;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if ((seen >> (16 * b + i)) & 1u) x = fmaxf(x, __uint_as_float(v[h][16 * b + i]));
              top[2 * h + b] = x;
            }
          }
        }
        const uint32_t cs = smem_addr(consts + (c + skipped) % kConstRing * kConsts);
        // score factor of a part's block; read where it is used
        auto factor = [&](int of_part, int b) -> float {
          return Q8 ? lds_f32(cs + 4 * (of_part * (kBlocksPerTile / 2) + b)) : p.qk_scale;
        };
        auto largest = [&](int of_part) -> float {
          if (!Q8) return fmaxf(max3f(top[0], top[1], top[2]), top[3]) * p.qk_scale;
          float f[kBlocksPerTile / 2];
          lds_f32x4(cs + 4 * of_part * (kBlocksPerTile / 2), f);
          return fmaxf(max3f(top[0] * f[0], top[1] * f[1], top[2] * f[2]), top[3] * f[3]);
        };
        float mt = largest(part ^ 1);
#pragma unroll
        for (int b = 0; b < kBlocksPerTile / 2; ++b)
          tmem_ld16_max(s_mine + 16 * b, &v[b >> 1][16 * (b & 1)], top[b]);
        tmem_wait_ld();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[half]);
        if (tail) {
          const int base = (j - tail_j) * kTileN - cur_lead(cur) + part * (kTileN / 2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (base + 32 * h + 32 <= 0) continue;
            const uint32_t seen = seen_bits(mask_row(cur), cur->q_len, base + 32 * h);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float x = -INFINITY;
#pragma unroll
              for (int i = 16 * b; i < 16 * b + 16; ++i) {
                if (!((seen >> i) & 1u)) v[h][i] = __float_as_uint(-INFINITY);
                x = fmaxf(x, __uint_as_float(v[h][i]));
              }
              top[2 * h + b] = x;
            }
          }
          if (!Q8 && half == 0 && !(ok = clear_values(cur, (j - tail_j) * kTileN - cur_lead(cur)))) break;
        }
        mt = fmaxf(mt, largest(part));
        const bool grow = mt > m;  // true on the first tile in which the row sees a key
        float alpha = 1.f;
        if (grow) {
          alpha = fast_exp2(m - (mt + kHeadroom));
          m = mt + kHeadroom;
        }
        l *= alpha;
        const float ref = m == -INFINITY ? 0.f : m;  // a row that has seen no key yet: weights of 0
        const bool large = __any_sync(0xffffffffu, fabsf(ref) > kLargeScore);
        if (large) {
          // score x factor has to be rounded as it was for the maximum, or the fused form below would leave
          // the rounding of a large product, whole powers of two, in the exponent
#pragma unroll
          for (int b = 0; b < kBlocksPerTile / 2; ++b) {
            const float fb = factor(part, b);
#pragma unroll
            for (int i = kBlockSize * b; i < kBlockSize * (b + 1); ++i)
              v[i >> 5][i & 31] = __float_as_uint(__fmul_rn(__uint_as_float(v[i >> 5][i & 31]), fb));
          }
        }
        const float2 ref2 = make_float2(-ref, -ref);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int b = 0; b < kBlocksPerTile / 2; ++b) {
          const float fb = large ? 1.f : factor(part, b);
          const float2 fb2 = make_float2(fb, fb);
          float2 nb2 = ref2;
          if (Q8) {
            const float nb = lds_f32(cs + 4 * (kBlocksPerTile + part * (kBlocksPerTile / 2) + b)) - ref;
            nb2 = make_float2(nb, nb);
            sum = make_float2(0.f, 0.f);
          }
#pragma unroll
          for (int i = 0; i < kBlockSize / 2; ++i) {
            const int e = b * kBlockSize + 2 * i;
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[e >> 5][e & 31]),
                                                    __uint_as_float(v[e >> 5][(e & 31) + 1])), fb2, nb2);
            const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            sum = __fadd2_rn(sum, y);
            v[0][e >> 1] = pack_bf2(y.x, y.y);
          }
          if (Q8) l += (sum.x + sum.y) * lds_f32(cs + 4 * (2 * kBlocksPerTile + part * (kBlocksPerTile / 2) + b));
        }
        if (!Q8) l += sum.x + sum.y;
        if (c > 0) {  // the previous P V: P's columns are free and O is up to date
          if (!(ok = wait_pv())) break;
          tc_fence_after_sync();
        }
        tmem_st32(p_addr, v[0]);
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          const float2 a2 = make_float2(alpha, alpha);
          uint32_t(&o)[32] = v[1];  // this thread's 32 columns of O
          tmem_ld32(o_addr, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), a2);
            o[2 * i] = __float_as_uint(x.x);
            o[2 * i + 1] = __float_as_uint(x.y);
          }
          tmem_st32(o_addr, o);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[half]);
        if (j == 0 && warp == 0 && lane == 0) {
          Walk w = *row_walk;
          Piece x;
          if (!next_piece<kTokens, kPieceTiles>(p, runs, w, x)) x.n = 0;
          *piece_slot(units + 2) = x;
          *row_walk = w;
        }
      }
      if (!ok) break;
      // ---- epilogue: this thread's 32 dims ----
      if (!(ok = wait_pv())) break;
      tc_fence_after_sync();
      uint32_t o[32];
      tmem_ld32(o_addr, o);
      tmem_wait_ld();
      // the two sums of a row meet over O's columns, which nothing writes before o_free
      tmem_st1(o_addr, __float_as_uint(l));
      tmem_wait_st();
      tc_fence_before_sync();
      // (the next piece's odd tokens: the buffer was last read two pieces ago, before the row warps last met)
      if (!Q8 && tid == 0) {
        uint32_t* next_odd = odd + (units + 1) % 3 * (1 + kMaxMaskWords);
        if (next_odd[0] != 0u)
          for (int i = 0; i <= kMaxMaskWords; ++i) next_odd[i] = 0u;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(l_bar);
      if (!(ok = wait_row(l_bar, static_cast<uint32_t>(units & 1)))) break;
      tc_fence_after_sync();
      const float l_theirs = __uint_as_float(tmem_ld1(o_theirs));
      tmem_wait_ld();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[half]);
      l = part ? l_theirs + l : l + l_theirs;
      const uint32_t* const my_odd = odd + units % 3 * (1 + kMaxMaskWords);
      if (!Q8 && *const_cast<const volatile uint32_t*>(my_odd) != 0u) {
        // drafted values that are no numbers go to the rows that see them, and to no other
        const int32_t* table = p.block_tables + static_cast<int64_t>(cur->s) * p.max_blocks_per_seq;
        const int32_t* bits = mask_row(cur);
        for (int i = 0; 32 * i < cur->q_len; ++i) {
          uint32_t w = my_odd[1 + i] & mask_word(bits, cur->q_len, i);
          while (w != 0u) {
            const int pos = cur->L - cur->q_len + 32 * i + __ffs(w) - 1;
            w &= w - 1u;
            const int32_t b = __ldg(table + pos / kBlockSize);
            if (b < 0 || b >= p.num_blocks) continue;
            const uint4* x = reinterpret_cast<const uint4*>(
                p.value_cache + ((static_cast<int64_t>(b) * p.num_kv_heads + cur->g) * kBlockSize + pos % kBlockSize) *
                                    kHeadDim + part * (kHeadDim / 2));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 y = __ldg(x + k);
              const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 g = bf16x2_to_float2(z[e] & odd_halves(z[e]));
                o[8 * k + 2 * e] = __float_as_uint(__uint_as_float(o[8 * k + 2 * e]) + g.x);
                o[8 * k + 2 * e + 1] = __float_as_uint(__uint_as_float(o[8 * k + 2 * e + 1]) + g.y);
              }
            }
          }
        }
      }
      const int tok0 = cur->tok0 + half * kHalfTokens;
      const bool row_ok = tok0 + r / GROUP < cur->q_len;
      const int from = cur->from, to = cur->to;
      bool write = from == to;
      if (!write) {
        // ---- a piece of a split segment: its record, and the warp that comes last weighs them all ----
        // whether this warp is the last of `count` to arrive at a counter; then it sees what the others wrote
        auto arrive = [&](int32_t* counter, int count) -> bool {
          __threadfence();
          __syncwarp();
          int last = 0;
          if (lane == 0) {
            last = atomicAdd(counter, 1) == count - 1;
            if (last) *counter = 0;
          }
          last = __shfl_sync(0xffffffffu, last, 0);
          if (last) __threadfence();
          return last != 0;
        };
        // weighs the records of `count` CTAs, every `step`-th from `cta` on, into m, l and o
        auto weigh = [&](int cta, int step, int count) {
#pragma unroll
          for (int d = 0; d < 2; ++d) {  // 16 of the thread's dims at a time, kTogether records' loads in flight
            float acc[16] = {};
            l = 0.f;
            m = -INFINITY;
            for (int k0 = 0; k0 < count; k0 += kTogether) {
              float4 x[kTogether][4], ml[kTogether];
#pragma unroll
              for (int u = 0; u < kTogether; ++u) {
                const int c = cta + min(k0 + u, count - 1) * step;
                const float4* rec = record_of(c, c == from);
                ml[u] = __ldcg(rec + 8 * kTileM);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = __ldcg(rec + (4 * d + i) * kTileM);
              }
              float top = m;
#pragma unroll
              for (int u = 0; u < kTogether; ++u) top = fmaxf(top, ml[u].x);
              const float at = top == -INFINITY ? 0.f : top;  // a row that has seen no key yet
              const float alpha = fast_exp2(m - at);
              m = top;
              l *= alpha;
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[i] *= alpha;
#pragma unroll
              for (int u = 0; u < kTogether; ++u) {
                if (k0 + u >= count) continue;
                const float w = fast_exp2(ml[u].x - at);
                l += w * ml[u].y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  acc[4 * i] += w * x[u][i].x;
                  acc[4 * i + 1] += w * x[u][i].y;
                  acc[4 * i + 2] += w * x[u][i].z;
                  acc[4 * i + 3] += w * x[u][i].w;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) o[16 * d + i] = __float_as_uint(acc[i]);
          }
        };
        auto keep = [&](float4* rec) {
          if (!row_ok) return;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            rec[i * kTileM] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                          __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          rec[8 * kTileM] = make_float4(m, l, 0.f, 0.f);
        };
        const int pieces = to - from + 1;
        keep(record_of(blockIdx.x, cur->j0 == 0));
        int32_t* const counter = p.counters + from * kRowWarps + warp;
        if (pieces <= kFlatPieces) {
          write = arrive(counter, pieces);
          if (write && row_ok) weigh(from, 1, pieces);
        } else {
          // groups first, whose sums take the place of their first records; then the groups
          const int first = from + (static_cast<int>(blockIdx.x) - from) / kGroupPieces * kGroupPieces;
          const int count = min(kGroupPieces, to + 1 - first);
          if (arrive(group_counter(first, from, warp), count)) {
            if (row_ok) weigh(first, 1, count);
            keep(record_of(first, first == from));
            const int groups = (pieces + kGroupPieces - 1) / kGroupPieces;
            write = arrive(counter, groups);
            if (write && row_ok) weigh(from, kGroupPieces, groups);
          }
        }
        if (lane == 0) ++delivered[warp];
      }
      if (write) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        // Four lanes exchange what they hold (four rows by four 16-byte chunks), so that each store covers
        // 64 bytes of eight rows.
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = make_uint4(pack_bf2(__uint_as_float(o[8 * i]) * inv, __uint_as_float(o[8 * i + 1]) * inv),
                            pack_bf2(__uint_as_float(o[8 * i + 2]) * inv, __uint_as_float(o[8 * i + 3]) * inv),
                            pack_bf2(__uint_as_float(o[8 * i + 4]) * inv, __uint_as_float(o[8 * i + 5]) * inv),
                            pack_bf2(__uint_as_float(o[8 * i + 6]) * inv, __uint_as_float(o[8 * i + 7]) * inv));
        swap_chunks(w[0], w[1], lane & 1, 1);
        swap_chunks(w[2], w[3], lane & 1, 1);
        swap_chunks(w[0], w[2], lane & 2, 2);
        swap_chunks(w[1], w[3], lane & 2, 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = (r & ~3) + i;
          if (tok0 + rr / GROUP < cur->q_len)
            *reinterpret_cast<uint4*>(
                p.out + (static_cast<int64_t>(cur->q0 + tok0 + rr / GROUP) * p.num_q_heads + cur->g * GROUP +
                         rr % GROUP) * kHeadDim + part * (kHeadDim / 2) + 8 * (lane & 3)) = w[i];
        }
      }
    }
    if (!ok && q_loader) {  // leave no copy in flight (bounded waits)
      flag_error(p.status, PA_DEVFLAG_TIMEOUT);
      // (the Q of the piece given up on, or the next one's too)
      if (took > 0) mbar_wait(&q_full[half], static_cast<uint32_t>((took - 1) & 1));
      mbar_wait(&q_full[half], static_cast<uint32_t>(took & 1));
    }
  } else {
    if (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Lay::kOtherRegs));
    if (warp == kMmaWarp) {
      // ============================ MMA issuer ============================
      // The whole warp walks the tiles, so that barriers, counters and descriptors stay uniform; one
      // elected lane issues.  Order: S(0), S(1), PV(0), S(2), PV(1), ... over the tiles of all pieces.
      constexpr uint32_t kIdescS = idesc_bf16_f32(kTileM, kTileN, false);
      constexpr uint32_t kIdescO = idesc_bf16_f32(kTileM, kHeadDim, true);
      const bool leader = elect_one();
      const uint64_t q_desc = sw128_desc(smem_addr(sq), 16, 1024);
      const uint64_t k_desc0 = sw128_desc(smem_addr(sk), 16, 1024);
      const uint64_t v_desc0 = sw128_desc(smem_addr(sv), 16, 1024);
      constexpr uint64_t kStageStep = kOpBytes >> 4;  // of a descriptor's start address
      constexpr uint64_t kQStep = kQBytes >> 4;
      int s_issued[HALVES] = {}, pv_issued[HALVES] = {}, q_used[HALVES] = {}, o_used[HALVES] = {};
      int ks = 0, vs = 0;
      uint32_t kph = 0, vph = 0;
      // a tile's scores, for the first `halves` of them
      auto issue_s = [&](bool first, int halves) -> bool {
        if (!wait_role<!Q8>(&kv_full[ks], kph, &abort_flag, p.status)) return false;
        const uint64_t k_desc = k_desc0 + kStageStep * ks;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          if (h >= halves) continue;
          if (first && !wait_role<!Q8>(&q_full[h], static_cast<uint32_t>(q_used[h]++ & 1), &abort_flag, p.status))
            return false;
          if (s_issued[h] > 0 &&
              !wait_role<!Q8>(&s_free[h], static_cast<uint32_t>((s_issued[h] - 1) & 1), &abort_flag, p.status))
            return false;
          tc_fence_after_sync();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kHeadDim / 16; ++kk)
              umma_bf16(tmem + Lay::kSCol + h * kTileN, q_desc + kQStep * h + 2 * kk, k_desc + 2 * kk, kIdescS,
                        kk > 0 ? 1u : 0u);
            umma_commit(&s_full[h]);
            if (Q8) mbar_arrive(&s_full[h]);  // passes on what the converters wrote before their arrivals (the constants)
          }
          ++s_issued[h];
        }
        if (Q8 && leader) umma_commit(&k_empty[ks]);
        if (++ks == kRing) {
          ks = 0;
          kph ^= 1u;
        }
        return true;
      };
      // and its P V: half 0 first, whose row warps clear V for both
      auto issue_pv = [&](bool first, int halves) -> bool {
        if (Q8 && !wait_role<!Q8>(&v_full[vs], vph, &abort_flag, p.status)) return false;
        const uint64_t v_desc = v_desc0 + kStageStep * vs;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          if (h >= halves) continue;
          if (!wait_role<!Q8>(&p_full[h], static_cast<uint32_t>(pv_issued[h] & 1), &abort_flag, p.status)) return false;
          if (first) {  // O starts anew: the half's previous piece has been read out
            if (o_used[h] > 0 &&
                !wait_role<!Q8>(&o_free[h], static_cast<uint32_t>((o_used[h] - 1) & 1), &abort_flag, p.status))
              return false;
            ++o_used[h];
          }
          tc_fence_after_sync();
          if (leader) {
            const uint32_t o_tmem = tmem + Lay::kOCol + h * kHeadDim, p_tmem = tmem + Lay::kPCol + h * (kTileN / 2);
            umma_bf16_ts(o_tmem, p_tmem, v_desc, kIdescO, first ? 0u : 1u);
#pragma unroll
            for (int kk = 1; kk < kTileN / 16; ++kk)  // 16 keys: 2 KiB of V, 8 columns of P
              umma_bf16_ts(o_tmem, p_tmem + kk * 8, v_desc + 128 * kk, kIdescO, 1u);
            umma_commit(&pv_done[h]);
          }
          ++pv_issued[h];
        }
        if (leader) umma_commit(&tile_done[vs]);
        if (++vs == kRing) {
          vs = 0;
          vph ^= 1u;
        }
        return true;
      };
      // Pieces as the row warps have them: piece u + 1 was written before warp 0 read piece u's last scores.
      auto halves_of = [&](const Piece& u) { return HALVES > 1 && half_active(u, 1) ? 2 : 1; };
      int units = 0;
      int n = piece_slot(0)->n, halves = n > 0 ? halves_of(*piece_slot(0)) : 0;
      bool ok = n > 0 && issue_s(true, halves);
      while (ok && n > 0) {
        int after = 0, halves_after = 0;
        for (int j = 0; ok && j < n; ++j) {
          const bool last = j + 1 == n;
          if (last) {
            if (!(ok = wait_role<!Q8>(s_free, static_cast<uint32_t>((s_issued[0] - 1) & 1), &abort_flag, p.status))) break;
            const Piece& next = *piece_slot(units + 1);
            after = next.n;
            halves_after = halves_of(next);
          }
          if (!last || after > 0) ok = issue_s(last, last ? halves_after : halves);
          if (ok) ok = issue_pv(j == 0, halves);
        }
        n = after;
        halves = halves_after;
        ++units;
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
      Walk walk = *start_walk;
      Piece cur;
      bool ok = true;
      int jt = 0;
      constexpr int kStages = Q8 ? kRawRing : kRing;
      uint64_t* const full = Q8 ? raw_full : kv_full;
      uint64_t* const empty = Q8 ? raw_empty : tile_done;
      while (ok && next_piece<kTokens, kPieceTiles>(p, runs, walk, cur)) {
        const int32_t* row = p.block_tables + static_cast<int64_t>(cur.s) * p.max_blocks_per_seq;
        const int blocks = (cur.L + kBlockSize - 1) / kBlockSize;
        // 32 table entries (four tiles) at a time, one per lane, the next window in flight
        int win_base = cur.j0 * kBlocksPerTile;
        auto fetch = [&](int base) -> int32_t { return base + lane < blocks ? __ldg(row + base + lane) : 0; };
        int32_t win = fetch(win_base);
        int32_t win_next = fetch(win_base + 32);
        for (int j = 0; j < cur.n; ++j, ++jt) {
          const int st = jt % kStages;
          const int lb0 = (cur.j0 + j) * kBlocksPerTile;
          if (lb0 >= win_base + 32) {
            win_base += 32;
            win = win_next;
            win_next = fetch(win_base + 32);
          }
          const bool need = lane < kBlocksPerTile && lb0 + lane < blocks;
          const int32_t entry = __shfl_sync(0xffffffffu, win, (lb0 - win_base) + (lane & (kBlocksPerTile - 1)));
          const bool bad = need && (entry < 0 || entry >= p.num_blocks);
          if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(p.status, PA_DEVFLAG_BAD_BLOCK);
          ok = wait_role<!Q8>(&empty[st], static_cast<uint32_t>((jt / kStages) & 1) ^ 1u, &abort_flag, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (Q8) {
            // tile (row) of each block; one that is not needed, or bad, brings the pool's first
            const int32_t tile = need && !bad ? entry * p.num_kv_heads + cur.g : 0;
            int32_t rows[kBlocksPerTile];
#pragma unroll
            for (int b = 0; b < kBlocksPerTile; ++b) rows[b] = __shfl_sync(0xffffffffu, tile, b);
            if (leader) {
              raw_keys[st] = cur.L - (cur.j0 + j) * kTileN;
              mbar_arrive_expect_tx(&full[st], kRawBytes);
              uint8_t* dst = sraw + st * kRawBytes;
#pragma unroll
              for (int b = 0; b < kBlocksPerTile; b += 4) {
                gather4(dst + b * kQ8TileBytes, &tmap_k, &rows[b], &full[st]);
                gather4(dst + (kBlocksPerTile + b) * kQ8TileBytes, &tmap_v, &rows[b], &full[st]);
              }
            }
            if (lane < kBlocksPerTile) {
              float* s = raw_scale + st * 2 * kBlocksPerTile + lane;
              async_copy4(s, p.key_scale + tile);
              async_copy4(s + kBlocksPerTile, p.value_scale + tile);
              async_arrive(&full[st]);
            }
          } else {
            const bool load = need && !bad;
            const unsigned mask = __ballot_sync(0xffffffffu, load);
            if (lane == 0) mbar_arrive_expect_tx(&full[st], __popc(mask) * 2u * kTileBytes);
            __syncwarp();
            if (load) {
              const int y = (entry * p.num_kv_heads + cur.g) * kBlockSize;
              tma_load_2d(sk + st * kOpBytes + lane * kTileBytes, &tmap_k, 0, y, &full[st]);
              tma_load_2d(sv + st * kOpBytes + lane * kTileBytes, &tmap_v, 0, y, &full[st]);
            }
          }
        }
      }
      int ended = -1;
      if (Q8 && ok) {  // the converters' end: a stage without keys
        const int st = jt % kStages;
        ok = wait_role<!Q8>(&empty[st], static_cast<uint32_t>((jt / kStages) & 1) ^ 1u, &abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && leader) {
          raw_keys[st] = 0;
          mbar_arrive(&full[st]);
        }
        if (ok && lane < kBlocksPerTile) mbar_arrive(&full[st]);
        if (ok) ended = st;  // (its last fill has been read)
      }
      // leave no copy in flight: wait (bounded) for the last fill of each stage
      if (Q8) asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) {
        for (int st = 0; st < kStages && st < jt; ++st) {
          if (st == ended) continue;
          const int last = st + ((jt - 1 - st) / kStages) * kStages;
          if (!mbar_wait(&full[st], static_cast<uint32_t>((last / kStages) & 1)))
            flag_error(p.status, PA_DEVFLAG_TIMEOUT);
        }
      }
      __syncwarp();
    } else if (warp < kConvWarp0 + kKWarps + kVWarps) {
      // ============================ converters (8-bit pools) ============================
      // kKWarps warps for K and kVWarps for V, each with its share of a tile's blocks, so that K runs ahead of
      // the products that V waits for.
      constexpr int kBatch = kQ8RowSteps;  // a block's rows of a lane, loaded first (the stores may alias the loads)
      const bool is_k = warp < kConvWarp0 + kKWarps;
      const int cw = warp - kConvWarp0 - (is_k ? 0 : kKWarps);
      const int blocks = kBlocksPerTile / (is_k ? kKWarps : kVWarps);  // blocks cw * blocks .. of every tile
      const int row0 = cw * blocks * kBlockSize + (lane >> 2);
      const int c0 = 2 * (lane & 3);  // 16 codes of a row: two 16-byte chunks
      uint64_t* const full = is_k ? kv_full : v_full;
      uint64_t* const empty = is_k ? k_empty : tile_done;
      int st = 0, rs = 0, slot = 0;   // operand stage, stage of codes
      uint32_t ph = 0, rph = 0;
      for (;;) {
        bool ok = wait_role<true>(&raw_full[rs], rph, &abort_flag, p.status);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int keys = raw_keys[rs];
        if (keys == 0) break;
        ok = wait_role<true>(&empty[st], ph ^ 1u, &abort_flag, p.status);
        if (!__all_sync(0xffffffffu, ok)) break;
        // lane b: what block b's codes, as bf16 pairs times 2^-120, are multiplied by: 2^120 for K, and
        // 2^(120 + e) for V, e where 120 + e is beyond bf16 apart
        uint32_t up = bf2_power(120);
        int high = 0;
        if (lane < blocks) {
          const int blk = cw * blocks + lane;
          const bool needed = blk * kBlockSize < keys;
          const float* scales = raw_scale + rs * 2 * kBlocksPerTile + blk;
          const float value = needed ? scales[kBlocksPerTile] : 1.f;
          if (is_k) {  // the row warps' constants
            const float f = significand(value);
            float lf = 0.f, fi = 1.f;
            if (f != 1.f) {
              lf = __log2f(f);
              fi = __fdividef(1.f, f);
            }
            float* cs = consts + slot * kConsts + blk;
            // (a hidden key's score is minus infinity: times 0 it would be a NaN)
            cs[0] = fmaxf((needed ? scales[0] : 1.f) * p.qk_scale, 1.17549435e-38f);
            cs[kBlocksPerTile] = lf;
            cs[2 * kBlocksPerTile] = fi;
          } else {
            const uint32_t bits = __float_as_uint(value) & 0x7fffffffu;
            const int e = static_cast<int>(bits >> 23) - 127;
            if (e > -127) {
              high = e > 7 ? min(e, 127) : 0;
              up = bf2_power(e > 7 ? 120 : 120 + e);
            } else {  // below the normal floats: e = -118 - clz; zero
              up = bits != 0u ? bf2_power(2 - __clz(bits)) : 0u;
            }
          }
        }
        const bool any_high = __any_sync(0xffffffffu, high != 0);
        const uint8_t* raw = sraw + rs * kRawBytes + (is_k ? 0 : kTileN * kQ8RowBytes) + cw * blocks * kQ8TileBytes + 16 * lane;
        uint8_t* dst = (is_k ? sk : sv) + st * kOpBytes;
        const int keys_left = keys - row0;
#pragma unroll 1  // (and the rest of a large scale beside the loop: 185 us against 183, 16 x 8000 x 32 83 against 78)
        for (int i0 = 0; i0 < 2 * blocks; i0 += kBatch) {
          uint4 in[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) in[i] = lds128(raw + (i0 + i) * 512);
          if (!is_k && keys < kTileN) {  // V past the context weighs nothing, but may hold anything
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (8 * (i0 + i) >= keys_left) in[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          const uint32_t m0 = __shfl_sync(0xffffffffu, up, i0 / kBatch);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const uint4 w = in[i];
            uint4 a, b;
            codes4_to_bf2x2(w.x, a.x, a.y);
            codes4_to_bf2x2(w.y, a.z, a.w);
            codes4_to_bf2x2(w.z, b.x, b.y);
            codes4_to_bf2x2(w.w, b.z, b.w);
            a.x = mul_bf2(a.x, m0); a.y = mul_bf2(a.y, m0); a.z = mul_bf2(a.z, m0); a.w = mul_bf2(a.w, m0);
            b.x = mul_bf2(b.x, m0); b.y = mul_bf2(b.y, m0); b.z = mul_bf2(b.z, m0); b.w = mul_bf2(b.w, m0);
            *reinterpret_cast<uint4*>(dst + swz(row0 + 8 * (i0 + i), c0)) = a;
            *reinterpret_cast<uint4*>(dst + swz(row0 + 8 * (i0 + i), c0 + 1)) = b;
          }
        }
        if (any_high) {  // a scale above 2^7: the rest of it (each lane what it wrote)
#pragma unroll 1
          for (int i = 0; i < 2 * blocks; ++i) {
            const uint32_t m1 = bf2_power(__shfl_sync(0xffffffffu, high, i / kBatch));
#pragma unroll 1
            for (int c = c0; c < c0 + 2; ++c) {
              uint4* const at = reinterpret_cast<uint4*>(dst + swz(row0 + 8 * i, c));
              const uint4 a = *at;
              *at = make_uint4(mul_bf2(a.x, m1), mul_bf2(a.y, m1), mul_bf2(a.z, m1), mul_bf2(a.w, m1));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[st]);
          mbar_arrive(&raw_empty[rs]);
        }
        if (++st == kRing) {
          st = 0;
          ph ^= 1u;
        }
        if (++rs == kRawRing) {
          rs = 0;
          rph ^= 1u;
        }
        slot = (slot + 1) % kConstRing;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, Lay::kTmemCols);
  }
  if (abort_flag != 0 && tid < kRowWarps) {
    // the counters come back to zero all the same: pieces that were not delivered count as if
    Walk w = *start_walk;
    Piece u;
    int n = 0;
    while (next_piece<kTokens, kPieceTiles>(p, runs, w, u)) {
      if (u.from == u.to || !warp_active(u, tid) || n++ < delivered[tid]) continue;
      const int pieces = u.to - u.from + 1;
      int32_t* counter = p.counters + u.from * kRowWarps + tid;
      int count = pieces;
      if (pieces > kFlatPieces) {
        const int first = u.from + (static_cast<int>(blockIdx.x) - u.from) / kGroupPieces * kGroupPieces;
        int32_t* group = group_counter(first, u.from, tid);
        if (atomicAdd(group, 1) != min(kGroupPieces, u.to + 1 - first) - 1) continue;
        *group = 0;
        count = (pieces + kGroupPieces - 1) / kGroupPieces;
      }
      if (atomicAdd(counter, 1) == count - 1) *counter = 0;
    }
  }
}

// Both forms have 16 row warps and 256 rows per SM, so their counters and records take the same room, and
// the counters the same place.
constexpr size_t counter_bytes(int sms) { return (static_cast<size_t>(sms) * 2 * kHalfWarps * 4 + 255) / 256 * 256; }
constexpr size_t record_bytes(int sms) { return static_cast<size_t>(sms) * 2 * 2 * kRecordFloat4s * 16; }

cudaError_t device_sms(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
}

template <int GROUP, bool Q8, int HALVES>
cudaError_t launch(const TreeArgs& a, cudaStream_t stream) {
  using Lay = Layout<Q8, HALVES>;
  static bool ready[kMaxDevices] = {};  // benign race: the calls are idempotent
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  auto kernel = tree_kernel<GROUP, Q8, HALVES>;
  if (dev >= kMaxDevices || !ready[dev]) {
    if (Q8) {
      cudaFuncAttributes attr;
      if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
      // setmaxnreg waits for registers the launch never had: refuse instead
      if (attr.numRegs * Lay::kThreads < Lay::kRowWarps * 32 * Lay::kRowRegs + (Lay::kThreads - Lay::kRowWarps * 32) * Lay::kOtherRegs)
        return cudaErrorInvalidConfiguration;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  CUtensorMap tq, tk, tv;
  if (!encode_query_tiles(&tq, a.q, static_cast<uint64_t>(a.num_query_tokens), a.num_q_heads, GROUP, kTileM / GROUP))
    return cudaErrorInvalidValue;
  const uint64_t tiles = static_cast<uint64_t>(a.num_blocks) * a.num_kv_heads;
  const bool maps = Q8 ? encode_tile_rows(&tk, a.key_cache, tiles) && encode_tile_rows(&tv, a.value_cache, tiles)
                       : encode_pool_rows(&tk, a.key_cache, tiles * kBlockSize, kBlockSize) &&
                             encode_pool_rows(&tv, a.value_cache, tiles * kBlockSize, kBlockSize);
  if (!maps) return cudaErrorInvalidValue;
  TreeParams p;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.tree_mask = a.tree_mask;
  p.query_start_loc = a.query_start_loc;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.value_cache = static_cast<const __nv_bfloat16*>(a.value_cache);
  p.key_scale = a.key_scale;
  p.value_scale = a.value_scale;
  p.counters = static_cast<int32_t*>(a.workspace);
  p.group_counters = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) + counter_bytes(sms));
  p.records = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.workspace) + 3 * counter_bytes(sms));
  p.status = a.status;
  p.mask_words = a.mask_words;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_blocks = a.num_blocks;
  p.num_kv_heads = a.num_kv_heads;
  p.num_q_heads = a.num_q_heads;
  p.num_query_tokens = a.num_query_tokens;
  p.max_query_len = a.max_query_len;
  p.num_seqs = a.num_seqs;
  p.qk_scale = a.scale * 1.4426950408889634f;
  // no more CTAs than there can be tiles
  constexpr int kTokens = HALVES * kTileM / GROUP;
  const int64_t segments = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * ((a.max_query_len + kTokens - 1) / kTokens);
  const int64_t longest = (static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize + kTileN - 1) / kTileN;
  const int64_t most = Lay::kCtasPerSm * sms;
  const int64_t grid = segments >= most || longest >= most || segments * longest >= most ? most : segments * longest;
  kernel<<<static_cast<unsigned>(grid), Lay::kThreads, Lay::kBytes, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

// More rows than one half holds: both halves, so that a tile is fetched (and converted) once for them.  Over 8
// bits from half of that on, although the second half idles: the converters serve one CTA an SM instead of two
// (one and two CTAs: 1 x 16000 x 26 26.1 and 35.7 us, 1 x 131072 x 26 78.1, 90.5, 20 x 2000 x 32 33.9, 37.8, but
// 64 x 2000 x 16, 64 rows, 90.7 and 73.6).  Eight converter warps beside two halves, four for K (six: 16 x 8000 x 32
// 78.3 us against 75.0, 1 x 131072 x 26 83.0 and 78.9, 2 x 131072 x 60 183.2 and 180.7, 48 mixed 52.7 and 53.5).  bf16 figures in this file's header.
template <int GROUP, bool Q8>
cudaError_t launch_halves(const TreeArgs& a, cudaStream_t stream) {
  return a.max_query_len * GROUP > (Q8 ? kTileM / 2 : kTileM) ? launch<GROUP, Q8, 2>(a, stream) : launch<GROUP, Q8, 1>(a, stream);
}

template <bool Q8>
cudaError_t launch_group(const TreeArgs& a, cudaStream_t stream) {
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_halves<1, Q8>(a, stream);
    case 2: return launch_halves<2, Q8>(a, stream);
    case 4: return launch_halves<4, Q8>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

size_t tree_workspace_size() {
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return 0;
  return 3 * counter_bytes(sms) + record_bytes(sms);
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) { return launch_group<false>(a, stream); }
cudaError_t launch_tree_q8(const TreeArgs& a, cudaStream_t stream) {
  AttendQ8Args r;
  r.out = a.out;
  r.q = a.q;
  r.query_start_loc = a.query_start_loc;
  r.num_query_tokens = a.num_query_tokens;
  r.max_query_len = a.max_query_len;
  r.max_context_len = 0;
  r.key_cache = a.key_cache;
  r.value_cache = a.value_cache;
  r.key_scale = a.key_scale;
  r.value_scale = a.value_scale;
  r.num_blocks = a.num_blocks;
  r.num_kv_heads = a.num_kv_heads;
  r.num_q_heads = a.num_q_heads;
  r.block_tables = a.block_tables;
  r.max_blocks_per_seq = a.max_blocks_per_seq;
  r.context_lens = a.context_lens;
  r.num_seqs = a.num_seqs;
  r.scale = a.scale;
  r.status = a.status;
  r.tree_mask = a.tree_mask;
  r.mask_words = a.mask_words;
  int dev = 0, sms = 0;
  const cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (rows_q8_takes(r)) {
    // Few rows run best on the few-rows kernel (8 nodes, 8 K/V heads: one context of 700 9.1 us against 14.0, of
    // 4000 11.9 and 19.5, 32 of 1000 18.9 and 21.6, 100 of 2000 82 and 94), but its clusters take equal parts of a
    // segment, so the longest context there may be is what it waits for (64 of 1-8192 90 us against 47, 64 of 1-32000
    // 321 and 100, one of 131072 160 and 65, 20 of 16000 182 and 124): where that is long, even batches do
    // without it as well (64 of 4000 101 and 110, 40 of 4000 75.5 and 74.8).
    if (r.max_blocks_per_seq <= kRowsBlocks * rows_q8_cluster(r, sms)) return launch_rows_q8(r, stream);
  }
  return launch_group<true>(a, stream);
}

}  // namespace pkv
