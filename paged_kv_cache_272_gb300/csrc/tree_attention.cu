// Attention of a tree of drafted tokens over the paged cache, on tcgen05 tensor cores.
//
// Sequence s has L drafted tokens, the last L of its context_lens[s] cached tokens.  Token i
// sees every cached token before the tree and the tree tokens its mask row names:
//   x_t = scale q . K_t,   out = sum_t exp(x_t - max x) V_t / sum_t exp(x_t - max x)
// over those t; a token that sees nothing gives zeros.  A masked K or V row takes no part
// whatever it holds.
//
// Rows.  The (token, query head) pairs that share one KV head are the rows of a product:
// row r is token r / G and head r % G of the group, 128 rows to a tile.  Keys come in tiles
// of 64.  One CTA runs a list of (sequence, KV head, row tile, key range) segments:
//  * warps 0-3 ("softmax"): thread t owns row t (TMEM lane t).  They stage Q (the first 64
//    head-dim columns in TMEM, the others in shared memory), read each score tile, mask it,
//    keep the running maximum and sum in fp32, write the weights to TMEM, rescale the output
//    accumulator when the maximum grows by more than 2^8, and finish a segment.  A warp whose
//    rows are all past the tree only keeps the barriers going.
//  * warp 4 issues S = Q K^T, warp 7 O += P V (one lane each; issuing takes longer than the
//    product runs, so neither waits behind the other).
//  * warps 5 and 6 fill the K and the V ring with TMA copies of the blocks the table names.
//    E4M3 cache: K's codes are an operand as they are (q as the sum of two E4M3 terms); V's
//    go through warps 8-11, which widen them to f16, exactly, because the weights need f16's
//    range.
//
// Split.  With few rows the work is reading the cache, and a batch may be one long sequence
// or many short ones.  So the key tiles of all (sequence, KV head) pairs of a row tile are
// laid end to end, a few units for each pair's start before its tiles, and cut into runs of
// equal length, one per resident CTA.  Long pairs so give every CTA about as many tiles; where a
// pair has about as many tiles as start units, a run can fall within the latter and have none.
// A pair cut by a run's end leaves normalised fp32 partial results (at most two per CTA, so the
// workspace does not grow with the batch) that tree_merge_kernel joins by their log-sum-exp in
// the order of the keys; nothing is summed in an order that depends on timing.  Each CTA finds
// its run from context_lens by itself: one launch for the attention, one for the join.  The row
// tiles of a pair are run by neighbouring CTAs, which start together and stay near enough for the
// cache to come from DRAM
// once and from L2 for the others (eight sequences of 65536 tokens, three row tiles: 676-701 us;
// with one row tile's CTAs after the other's, which drift apart by more than L2 holds, 776 beside
// 705).
//
// Masked values.  A weight of zero times a V element that is not finite would spoil a row
// that does not see it.  Tiles that overlap the tree (every row sees the others) are checked:
// elements that are not finite are taken out of the product, and the rows that do see them
// get them added at the end.
#include <cuda.h>
#include <math.h>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <climits>

#include "tcgen05.cuh"

namespace pkv {
namespace {

using namespace t5;

constexpr unsigned kFullMask = 0xffffffffu;
constexpr int kTileRows = 128;
constexpr int kTileKeys = 64;
constexpr int kTileBlocks = kTileKeys / kBlockSize;
// Threads per CTA: warps 0-3 softmax, 4-7 products and copies, 8-11 (E4M3) widening.
__host__ __device__ constexpr int tree_threads(bool f8) { return f8 ? 384 : 256; }
// E4M3: 384 threads of 80 registers, twice per SM; the softmax warps take 160 and the others
// leave 40 (128 x 160 + 256 x 40 = 384 x 80).  Batch of 64: 170.7 us with 128 / 56, 166.7 with
// 144 / 48, 166.1 with 160 / 40.  24 bytes are spilled and 36 read back.
constexpr int kLaunchRegs = 80, kSoftmaxRegs = 160, kOtherRegs = 40;
static_assert(128 * kSoftmaxRegs + 256 * kOtherRegs <= 384 * kLaunchRegs, "register split");
constexpr uint32_t kTmemColumns = 256;
constexpr int kMaxRowTiles = 64;  // row tiles of one launch
// A segment's start and finish, in key tiles.  Measured, 3 / 4 / 5 / 6: 32 ragged sequences 77.5 /
// 76.6 / 76.1 / 76.0 us, short MHA contexts 23.8 / 23.6 / 23.4 / 24.2; E4M3, 64 ragged sequences,
// 4 / 6 / 8 / 10 / 12: 170.1 / 168.0 / 167.2 / 167.3 / 166.1 (q's two terms take longer to make),
// while pairs of 12 tiles (38 sequences, 4 KV heads), whose runs are short, take 31-33 with any.
constexpr int kStart = 5, kStartF8 = 12;
// Least units of a run: one sequence of 700 tokens takes 14.3 us with runs of 3, 12.9 with 4
// (fewer parts to join), 13.7 with 5, 14.4 with 6.
constexpr int kMinRun = 4;
// E4M3: a weight enters its product as f16 of 2^kLift times itself, so that one of 2^-21 of the
// row's largest still has all of f16's bits and none above 2^-32 is lost (the sum keeps them all:
// unlifted, the part of a run's keys below 2^-25 each vanished from the result, a percent of it
// at half a million keys).  The lagging reference lets weights grow by 2^8: at most 2^15.
constexpr float kLiftF8 = 7.f;

struct TreeArgs {
  uint16_t *out;                // [T][Hq][D] bf16
  const uint16_t *q;            // [T][Hq][D] bf16
  const void *k_cache, *v_cache;
  const int32_t *block_tables;  // [S][MB]
  const int32_t *context_lens;  // [S]
  const int32_t *query_start;   // [S+1]
  const uint64_t *masks;        // [T][W]
  int num_seqs, num_tokens, max_blocks, q_heads, kv_heads, group, num_blocks, words;
  int max_query_len;
  float scale_log2;             // scale * log2(e) (* k_scale of an E4M3 cache)
  float v_scale;
  const float *k_scales, *v_scales;  // [Hkv] or null
  int runs;                     // CTAs that share the key tiles
  int start;                    // what a segment costs besides its tiles, in tiles
  int m0, row_tiles;            // this launch's row tiles m0 .. m0 + row_tiles - 1
  struct TreeJoin *join;        // [CTAs] what starts and does not end in a CTA
  float *part_lse;              // [CTAs][2][128] log2-sum-exp2
  float4 *part_o;               // [CTAs][2][D / 4][128 rows] normalised: a warp's rows store
                                // and load side by side
  int32_t *err;
};

struct __align__(16) TreeJoin {
  int q0, rows, g, m;  // first token, rows of the sequence, KV head, row tile
  int parts, pad[3];   // 0: nothing to join
};

struct SeqInfo {
  int q0, L, ctx, tiles, row_tiles;  // tiles 0: nothing to do
};

__device__ __forceinline__ SeqInfo seq_info(const TreeArgs &a, int s, bool flag) {
  SeqInfo i;
  const int q1 = a.query_start[s + 1];
  i.q0 = a.query_start[s];
  i.ctx = a.context_lens[s];
  const int64_t L = (int64_t)q1 - i.q0;
  if (i.q0 < 0 || L < 0 || q1 > a.num_tokens || L > a.max_query_len || L > i.ctx ||
      (int64_t)i.ctx > (int64_t)a.max_blocks * kBlockSize || i.ctx > INT_MAX - kTileKeys) {
    if (flag) flag_error(a.err, PKV_DEV_BAD_CONTEXT);
    i.L = i.tiles = i.row_tiles = 0;
    return i;
  }
  i.L = (int)L;
  i.tiles = i.L > 0 ? (int)(((int64_t)i.ctx + kTileKeys - 1) / kTileKeys) : 0;
  i.row_tiles = (int)((L * a.group + kTileRows - 1) / kTileRows);
  return i;
}

// A CTA's run, filled by plan_run.  Runs are cut in units: a (sequence, KV head) pair is as
// many as it has key tiles and a.start more at its beginning, which stand for the time that
// any segment takes to start and finish (Q, first scores, last product, output).  A run that
// meets many short pairs so gets fewer tiles.
struct Plan {
  unsigned long long tiles[kMaxRowTiles];  // units of row tile m (all KV heads), its CTAs in
                                           // the top 16 bits (2^48 units are years of work);
                                           // later the ring of segments and the walk
  unsigned long long warp_sum[tree_threads(true) / 32];
  unsigned long long first;  // unit of the row tile
  long long left;          // units of the run
  long long cta_tiles, extra;  // run length of this row tile's CTAs: cta_tiles, one more for
  int cta, slot;               // the first `extra`; this CTA's number there, and its place in
  int m;                       // the workspace (the numbers of all row tiles end to end)
};

// The segments of a run.  The K warp walks them in order, ahead of everyone, and hands them on
// through a small ring in shared memory; one with no tiles ends the run.  It is at most eight
// segments ahead of the slowest reader: K of tile t is copied once S of tile t - KS is done,
// which the softmax warps' work on tile t - KS - 1 precedes, and the ring is written one tile
// before that copy.
struct __align__(16) Segment {
  int s, g, q0, L, ctx, tiles, j0, j1;
};
constexpr int kSegRing = 8;
static_assert(kSegRing * sizeof(Segment) <= kMaxRowTiles * sizeof(unsigned long long), "ring");

// Where a run stands.  In shared memory (one lane of the K warp moves it on): the copying warps
// have few registers to spare.
struct Walk {
  long long left;  // units
  int s, g, unit;  // sequence, KV head, unit of the pair
  SeqInfo i;
  // The run's first unit is unit `off` of sequence s (KV heads end to end).
  __device__ __forceinline__ void begin(const TreeArgs &a, int seq, const SeqInfo &info,
                                        unsigned long long off, long long units) {
    const unsigned n = (unsigned)(info.tiles + a.start);
    left = units, s = seq, i = info;
    if (off >> 32) {
      g = (int)(off / n), unit = (int)(off % n);
    } else {
      g = (int)((unsigned)off / n), unit = (int)((unsigned)off % n);
    }
  }
  __device__ __forceinline__ void next(const TreeArgs &a, int m, Segment &o) {
    while (left > 0) {
      if (g == a.kv_heads) {
        g = 0;
        do {
          if (++s >= a.num_seqs) left = 0;  // not reached: the run's units are counted
          else i = seq_info(a, s, false);
        } while (left > 0 && (i.tiles == 0 || i.row_tiles <= m));
        if (left == 0) break;
      }
      const int end = (int)min((long long)(i.tiles + a.start), unit + left);
      left -= end - unit;
      o.s = s, o.g = g, o.q0 = i.q0, o.L = i.L, o.ctx = i.ctx, o.tiles = i.tiles;
      o.j0 = max(unit - a.start, 0), o.j1 = max(end - a.start, 0);
      unit = 0;
      ++g;
      if (o.j1 > o.j0) return;
    }
    o.j0 = o.j1 = 0;
  }
};
constexpr int kWalkAt = kSegRing * (int)sizeof(Segment);  // bytes into Plan::tiles
static_assert(kWalkAt + sizeof(Walk) <= sizeof(Plan::tiles), "room behind the ring");
__device__ __forceinline__ Walk *walk_of(Plan *p) {
  return reinterpret_cast<Walk *>(reinterpret_cast<char *>(p->tiles) + kWalkAt);
}

// floor(a b / c), b <= c, without a 128-bit product: b and c lose low bits they do not need.
__device__ __forceinline__ int share(int a, unsigned long long b, unsigned long long c) {
  while (c >> 48) b >>= 1, c >>= 1;
  return (int)((unsigned long long)a * b / c);
}

// CTAs for that many units.
__device__ __forceinline__ int most_ctas(unsigned long long units, int ctas) {
  const unsigned long long few = (units + kMinRun - 1) / kMinRun;
  return few < (unsigned long long)ctas ? (int)few : ctas;
}

// Several row tiles, one thread: this CTA's row tile (p->m), its number c there, its place in
// the workspace, the row tile's CTAs n and units.  Not inlined: inlined, it took registers from
// the loops (E4M3 batch 176 -> 200 us).
struct RowTileShare {
  unsigned long long units;
  int c, n, m, slot;
};
__device__ __noinline__ RowTileShare row_tile_share(unsigned long long *tiles, int row_tiles,
                                                     int kv_heads, int runs) {
  RowTileShare o = {0, (int)blockIdx.x, 0, 0, (int)blockIdx.x};
  unsigned long long total = 0;
#pragma unroll 1
  for (int m = row_tiles - 1; m >= 0; --m) {
    o.units += tiles[m] * (unsigned)kv_heads;
    tiles[m] = o.units;
    total += o.units;
  }
  int k = 0;
#pragma unroll 1
  for (; k < row_tiles && tiles[k]; ++k)
    tiles[k] |= (unsigned long long)most_ctas(tiles[k], max(share(runs, tiles[k], total), 1)) << 48;
  // The row tiles' CTAs of one number are neighbours (a row tile has no more than the one
  // before it): while k row tiles have CTAs left, k at a time.
  int from = 0;
#pragma unroll 1
  for (; k > 0; --k) {
    const int upto = (int)(tiles[k - 1] >> 48), level = (upto - from) * k;
    if (o.c < level) {
      o.m = o.c % k, o.c = from + o.c / k;
      o.units = tiles[o.m] & ((1ull << 48) - 1);
      o.n = (int)(tiles[o.m] >> 48);
      o.slot = o.c;
#pragma unroll 1
      for (int i = 0; i < o.m; ++i) o.slot += (int)(tiles[i] >> 48);
      break;
    }
    o.c -= level;
    from = upto;
  }
  return o;
}

// One thread: run c of the n that share `units`.
__device__ __forceinline__ void cut_run(Plan *p, unsigned long long units, int n, int c, int m,
                                        int slot) {
  p->slot = slot;  // its own even with nothing to do
  p->left = 0;
  if (c >= n) return;
  unsigned long long q, r;
  if (units >> 32)
    q = units / (unsigned)n, r = units % (unsigned)n;
  else
    q = (unsigned)units / (unsigned)n, r = (unsigned)units % (unsigned)n;
  p->m = m;
  p->cta = c;
  p->cta_tiles = (long long)q;
  p->extra = (long long)r;
  p->left = (long long)q + (c < (long long)r ? 1 : 0);
  p->first = (unsigned)c * q + min((long long)c, (long long)r);
}

// Which key tiles this CTA runs (all threads; the result in *p and its walk after the last
// barrier).  Short on purpose: code that runs once is bound by the instruction fetch, ~20 cycles
// each.
template <int kThreads>
__device__ __forceinline__ void plan_run(const TreeArgs &a, Plan *p) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool one = a.row_tiles == 1;
  // One row tile and a thread for every sequence: the units of a KV head are summed once, and
  // the thread whose sequence the run begins in has what it needs.
  const bool once = one && a.num_seqs <= kThreads;
  SeqInfo i;
  i.tiles = 0;
  if (!once) {
    if (!one && tid < kMaxRowTiles) p->tiles[tid] = 0;
    if (!one) __syncthreads();
    unsigned long long mine = 0;
#pragma unroll 1
    for (int s = tid; s < a.num_seqs; s += kThreads) {
      i = seq_info(a, s, blockIdx.x == 0);
      const int last = min(i.row_tiles - a.m0, a.row_tiles);
      if (i.tiles == 0 || last <= 0) continue;
      mine += i.tiles + a.start;
      if (!one) atomicAdd(&p->tiles[last - 1], (unsigned long long)(i.tiles + a.start));
    }
    if (one) {
#pragma unroll 1
      for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(kFullMask, mine, off);
      if (lane == 0) p->warp_sum[warp] = mine;
    }
    __syncthreads();
    if (tid == 0) {
      RowTileShare o = {0, (int)blockIdx.x, 0, 0, (int)blockIdx.x};
      if (one) {
#pragma unroll 1
        for (int w = 0; w < kThreads / 32; ++w) o.units += p->warp_sum[w];
        o.units *= (unsigned)a.kv_heads;
        o.n = most_ctas(o.units, a.runs);
      } else {
        o = row_tile_share(p->tiles, a.row_tiles, a.kv_heads, a.runs);
      }
      cut_run(p, o.units, o.n, o.c, a.m0 + o.m, o.slot);
    }
    __syncthreads();
    if (p->left == 0) return;
  }
  const int m = once ? a.m0 : p->m;
  unsigned long long base = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < a.num_seqs; s0 += kThreads) {
    const int s = s0 + tid;
    unsigned long long n = 0;
    if (s < a.num_seqs) {
      i = seq_info(a, s, once && blockIdx.x == 0);
      if (i.tiles > 0 && i.row_tiles > m) n = (unsigned long long)(i.tiles + a.start);
    }
    unsigned long long incl = n;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long v = __shfl_up_sync(kFullMask, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) p->warp_sum[warp] = incl;
    __syncthreads();
    unsigned long long first = base + incl - n;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32 && s0 + 32 * w < a.num_seqs; ++w) {
      const unsigned long long v = p->warp_sum[w];
      if (w < warp) first += v;
      base += v;
    }
    if (once) {
      if (tid == 0) {
        const unsigned long long units = base * (unsigned)a.kv_heads;
        cut_run(p, units, most_ctas(units, a.runs), blockIdx.x, m, blockIdx.x);
      }
      __syncthreads();
    }
    first *= (unsigned)a.kv_heads;
    const unsigned long long u0 = p->first;
    if (p->left && u0 >= first && u0 - first < n * (unsigned)a.kv_heads)
      walk_of(p)->begin(a, s, i, u0 - first, p->left);
    if (once || u0 < base * (unsigned)a.kv_heads) break;
    __syncthreads();
  }
  __syncthreads();
}

// Shared memory of one CTA (two per SM).  D: head dim; F8: E4M3 cache.
template <int D, bool F8>
struct TreeLayout {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kTileKeys * 128;           // 64 keys x 64 columns of 2 bytes
  static constexpr int kRaw = kTileKeys * D;              // a tile of codes
  static constexpr int KS = F8 ? 4 : 3;                   // K ring
  static constexpr int kKSlot = F8 ? kRaw : kHalves * kHalf;
  static constexpr int VS = F8 && D == 128 ? 2 : 3;       // V ring (f16 values of an E4M3 cache)
  static constexpr int kVSlot = kHalves * kHalf;
  static constexpr int RS = F8 ? 4 : 0;                   // V codes on their way to the V ring
  // What of Q is not in TMEM (bf16 its columns 64..127, E4M3 at D 128 its second term), and
  // the finished rows on their way out.
  static constexpr int kQ = 0;
  static constexpr int kK = kTileRows * 128;
  static constexpr int kV = kK + KS * kKSlot;
  static constexpr int kRawV = kV + VS * kVSlot;
  static constexpr int kBars = kRawV + RS * kRaw;
  static constexpr int kNumBars = 2 * KS + 2 * VS + 7 + 2 * RS + kSegRing;
  static constexpr int kMisc = kBars + kNumBars * 8;  // TMEM address, abort flag, V marks
  static constexpr int kPlan = (kMisc + 80 + 15) / 16 * 16;  // holds the segments: 16-byte loads
  static constexpr int kSmem = kPlan + (int)sizeof(Plan);
  // at least 78 KB, so that no more than two CTAs share an SM (256 TMEM columns each)
  static constexpr int kSmemLaunch = kSmem > 78 * 1024 ? kSmem : 78 * 1024;
  static_assert(2 * (kSmemLaunch + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(kPlan % alignof(Segment) == 0 && kBars % 8 == 0, "alignment");
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}
// Two f16 values -> their E4M3 codes (low 16 bits), and exactly what is left of the values.
__device__ __forceinline__ uint32_t e4m3_split(__half2 &x) {
  const uint32_t c = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
  x = __hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
  return c & 0xffffu;
}
// Two E4M3 codes (low 16 bits) -> two f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {  // bit 7 of each NaN code's byte
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// The bits of a row's mask for keys t0 .. t0 + 63 (bit c: key t0 + c is visible): cached
// tokens before the tree, and the tree tokens the row names.
__device__ __forceinline__ uint64_t visible_bits(const uint64_t *mask, int t0, int first, int L) {
  const int o = t0 - first;  // tree index of key t0
  if (o <= -kTileKeys) return ~0ull;
  const int words = (L + 63) >> 6;
  uint64_t b;
  if (o < 0) {
    b = ((1ull << -o) - 1) | (mask[0] << -o);
  } else {
    const int w = o >> 6, sh = o & 63;
    b = w < words ? mask[w] >> sh : 0ull;
    if (sh && w + 1 < words) b |= mask[w + 1] << (64 - sh);
  }
  const int end = L - o;  // keys past the tree's end
  return end >= 64 ? b : b & ((1ull << end) - 1);
}

// The values that were taken out of a row's products because they are not finite, added to
// the row's stored result (a bf16 row, or a part's) where the row sees them.
template <int D, bool F8>
__device__ __noinline__ void add_odd_values(const TreeArgs &a, const Segment &seg,
                                            const uint64_t *mask, uint32_t tiles, uint16_t *out,
                                            float *part) {
  const int first = seg.ctx - seg.L;
#pragma unroll 1
  for (; tiles; tiles &= tiles - 1) {
    const int t0 = (first / kTileKeys + __ffs(tiles) - 1) * kTileKeys;
    uint64_t see = visible_bits(mask, t0, first, seg.L);
    if (t0 < first) see &= ~((1ull << (first - t0)) - 1);
#pragma unroll 1
    for (; see; see &= see - 1) {
      const int key = t0 + __ffsll((long long)see) - 1, at = key % kBlockSize;
      const int blk = a.block_tables[(size_t)seg.s * a.max_blocks + key / kBlockSize];
      if ((unsigned)blk >= (unsigned)a.num_blocks) continue;
      const size_t tile = ((size_t)blk * a.kv_heads + seg.g) * (kBlockSize * D);
#pragma unroll 1
      for (int d = 0; d < D; ++d) {
        const float v =
            F8 ? e4m3_to_f32(static_cast<const uint8_t *>(a.v_cache)[tile + d * kBlockSize + at])
               : bf16_to_f32(static_cast<const uint16_t *>(a.v_cache)[tile + at * D + d]);
        if (fabsf(v) < INFINITY) continue;
        if (out)
          out[d] = f32_to_bf16(bf16_to_f32(out[d]) + v);
        else
          part[(d >> 2) * (4 * kTileRows) + (d & 3)] += v;
      }
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(tree_threads(F8), 2)
    tree_attention_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv) {
  using Lay = TreeLayout<D, F8>;
  constexpr int H = Lay::kHalves, KS = Lay::KS, VS = Lay::VS, RS = Lay::RS;
  constexpr float kLift = F8 ? kLiftF8 : 0.f;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {  // the swizzled tiles need a 1024-byte aligned window
    // Every CTA of the launch comes here or none does, so each slot of the workspace gets its
    // word for the join: nothing to do.
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x == 0) {
      flag_error(a.err, PKV_DEV_LAYOUT);
      a.join[blockIdx.x].parts = 0;
    }
    return;
  }
  const uint32_t sQ = base + Lay::kQ, sK = base + Lay::kK, sV = base + Lay::kV;
  const uint32_t k_full = base + Lay::kBars, k_empty = k_full + 8 * KS;
  const uint32_t v_full = k_empty + 8 * KS, v_empty = v_full + 8 * VS;
  const uint32_t s_full = v_empty + 8 * VS, s_free = s_full + 8, p_full = s_free + 8;
  const uint32_t o_done = p_full + 8, fin_s = o_done + 8, fin_o = fin_s + 8;
  const uint32_t q_full = fin_o + 8, raw_full = q_full + 8, raw_empty = raw_full + 8 * RS;
  const uint32_t seg_full = raw_empty + 8 * RS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  // Marks of V tiles that held a value not finite.  E4M3: [ring slot], 1 + the number of the
  // CTA's tile that had one.  bf16: [tile of the tree], the number of the segment that did.
  volatile int *v_bad = abort_flag + 1;
  constexpr int kMarks = F8 ? VS : PKV_TREE_MAX_TOKENS / kTileKeys + 1;
  static_assert(8 + 4 * kMarks <= 80, "marks");
  Plan *plan = reinterpret_cast<Plan *>(smem + Lay::kPlan);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(k_full + 8 * i, kTileBlocks);
      mbar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(v_full + 8 * i, kTileBlocks);  // E4M3: one per widening warp
      mbar_init(v_empty + 8 * i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 4);
    mbar_init(p_full, 4);
    mbar_init(o_done, 1);
    mbar_init(fin_s, 1);
    mbar_init(fin_o, 1);
    mbar_init(q_full, 4);
    for (int i = 0; i < kSegRing; ++i) mbar_init(seg_full + 8 * i, 1);
    for (int i = 0; i < RS; ++i) {
      mbar_init(raw_full + 8 * i, kTileBlocks);
      mbar_init(raw_empty + 8 * i, 4);
    }
    *abort_flag = 0;
    for (int i = 0; i < kMarks; ++i) v_bad[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();
  // After the wait: a kernel before this one may still have to allocate its own.
  if (warp == 4) {
    alloc(smem_u32(tmem_slot), kTmemColumns);
    fence_before();
  }
  plan_run<tree_threads(F8)>(a, plan);
  fence_after();
  if (plan->left == 0) {
    if (threadIdx.x == 0) a.join[plan->slot].parts = 0;
    if (warp == 4) dealloc(*tmem_slot, kTmemColumns);
    return;
  }
  const int G = a.group;
  // Columns of TMEM: S, P, the part of Q kept there, O.  A role reads what it needs of these for
  // itself; held across the split into roles, they were spilled in all of them.
  const volatile uint32_t *tmem_at = tmem_slot;
  const volatile int *row_tile = &plan->m;
  Segment *ring_seg = reinterpret_cast<Segment *>(plan->tiles);
  Segment seg;
  // The run's segment n; false: the run is over (or a wait gave up).
  auto segment = [&](int n) {
    if (!mbar_wait(seg_full + 8 * (n % kSegRing), (uint32_t)(n / kSegRing) & 1u, abort_flag, a.err))
      return false;
    seg = ring_seg[n % kSegRing];
    return seg.j1 > seg.j0;
  };

  if (warp < 4) {
    if constexpr (F8) set_regs_up<kSoftmaxRegs>();
    // ---------------- softmax warps: thread t owns row t ----------------
    const uint32_t tmem = *tmem_at;
    const uint32_t tS = tmem, tP = tmem + 64, tQ = tmem + 96, tO = tmem + 128;
    const int r0 = *row_tile * kTileRows;
    const int t = threadIdx.x;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const int r = r0 + t;
    int jt = 0;   // tiles done (the barriers' phases)
    int nseg = 0; // segments begun
    bool ok = true;
    if (t == 0) a.join[plan->slot].parts = 0;
    while (ok && segment(nseg)) {
      ++nseg;
      const int rows = seg.L * G;
      const bool valid = r < rows, live = r0 + warp * 32 < rows;
      const int i = (valid ? r : rows - 1) / G, first = seg.ctx - seg.L;
      const size_t row = ((size_t)(seg.q0 + i) * a.q_heads + seg.g * G + r % G) * D;
      const uint64_t *mask = a.masks + (size_t)(seg.q0 + i) * a.words;
      float sl = a.scale_log2;
      float vs = a.v_scale;
      if (F8 && a.k_scales != nullptr) {
        const float ks = a.k_scales[seg.g];
        vs = a.v_scales[seg.g];
        if (t == 0 && !(ks > 0.f && vs > 0.f)) flag_error(a.err, PKV_DEV_BAD_SCALE);
        sl *= ks;
      }
      const uint4 *qrow = reinterpret_cast<const uint4 *>(a.q + row);
      if constexpr (!F8) {
        // columns 0..63 to TMEM (two 16-bit elements per column), 64..127 to shared memory
        uint4 v[8 * H];
#pragma unroll
        for (int c = 0; c < 8 * H; ++c) v[c] = valid ? qrow[c] : make_uint4(0u, 0u, 0u, 0u);
        tmem_st32(tQ + lane_base, reinterpret_cast<uint32_t (&)[32]>(v));
#pragma unroll
        for (int c = 8; c < 8 * H; ++c)
          st_shared_v4(sQ + t * 128 + (((c & 7) ^ (t & 7)) << 4), v[c]);
      } else {
        // The score product is one of E4M3 with E4M3, so that K's codes enter it as they lie
        // in the cache.  q is the sum of two E4M3 terms, q 2^e = q1 + q2, e putting the row's
        // largest element in [128, 256): q1 takes 4 significant bits and q2 the other 4 of
        // bf16's 8, exactly for elements down to 2^-9 of the largest, and to 2^-10 absolute
        // below.  q1 goes to TMEM (four codes per column), q2 to shared memory (D 64: TMEM).
        uint4 v[8 * H];  // every load before the first use
#pragma unroll
        for (int c = 0; c < 8 * H; ++c) v[c] = valid ? qrow[c] : make_uint4(0u, 0u, 0u, 0u);
        __nv_bfloat162 big = __float2bfloat162_rn(0.f);  // largest magnitudes (a NaN stays)
        auto grow = [&](uint32_t w) {
          big = __hmax2_nan(big, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)));
        };
#pragma unroll
        for (int c = 0; c < 8 * H; ++c) grow(v[c].x), grow(v[c].y), grow(v[c].z), grow(v[c].w);
        const uint32_t bb = *reinterpret_cast<const uint32_t *>(&big) & 0x7fff7fffu;
        const int bits = max(bb & 0xffffu, bb >> 16);
        const bool odd = bits >= 0x7f80;  // an infinity or NaN: no finite score in this row
        const int e = odd || bits == 0 ? 0 : min(134 - (bits >> 7), 120);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        // not to zero, which times a masked score's -inf is NaN; the scores that 2^-126 stands
        // in for are below 2^-100 either way
        sl = fmaxf(sl * __uint_as_float((uint32_t)(127 - e) << 23), 1.17549435e-38f);
#pragma unroll 1
        for (int c = 0; c < 2 * H; ++c) {  // 32 elements; the row moves down by as many
          uint32_t q1[8], q2[8];
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const uint4 &x4 = v[h >> 1];
            const uint32_t w0 = h & 1 ? x4.z : x4.x, w1 = h & 1 ? x4.w : x4.y;
            // f16 holds q 2^e exactly where q1 + q2 can (down to 2^-17)
            __half2 x0 = __floats2half2_rn(bf16_lo(w0) * up, bf16_hi(w0) * up);
            __half2 x1 = __floats2half2_rn(bf16_lo(w1) * up, bf16_hi(w1) * up);
            q1[h] = e4m3_split(x0), q1[h] |= e4m3_split(x1) << 16;
            q2[h] = e4m3_split(x0), q2[h] |= e4m3_split(x1) << 16;
            if (odd) q1[h] = ~0u;
          }
#pragma unroll
          for (int i2 = 0; i2 + 4 < 8 * H; ++i2) v[i2] = v[i2 + 4];
          tmem_st8(tQ + 8 * c + lane_base, q1);
          if (H == 1) {
            tmem_st8(tQ + 16 + 8 * c + lane_base, q2);
          } else {
            st_shared_v4(sQ + t * 128 + (((2 * c) ^ (t & 7)) << 4),
                         make_uint4(q2[0], q2[1], q2[2], q2[3]));
            st_shared_v4(sQ + t * 128 + (((2 * c + 1) ^ (t & 7)) << 4),
                         make_uint4(q2[4], q2[5], q2[6], q2[7]));
          }
        }
      }
      wait_st();
      fence_proxy_async();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      float m = -INFINITY, l = 0.f;
      uint32_t bad = 0;  // tree tiles whose V held a value not finite
      const int tree_tile = first / kTileKeys;
      for (int j = seg.j0; j < seg.j1; ++j, ++jt) {
        const int t0 = j * kTileKeys;
        const bool in_tree = t0 + kTileKeys > first;
        const uint64_t bits = in_tree && valid ? visible_bits(mask, t0, first, seg.L) : ~0ull;
        if (!mbar_wait(s_full, (uint32_t)jt & 1u, abort_flag, a.err)) {
          ok = false;
          break;
        }
        fence_after();
        bool p_free = j == seg.j0;  // P's columns: free once the P V before has completed
        uint32_t pk[32];
        if (live) {
          uint32_t x[64];
          {
            uint32_t (&x0)[32] = *reinterpret_cast<uint32_t (*)[32]>(&x[0]);
            uint32_t (&x1)[32] = *reinterpret_cast<uint32_t (*)[32]>(&x[32]);
            tmem_ld32(tS + lane_base, x0);
            tmem_ld32(tS + 32 + lane_base, x1);
            wait_ld();
          }
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);  // the next score product may overwrite S
          if (__builtin_expect(in_tree, 0)) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!((bits >> c) & 1)) x[c] = __float_as_uint(-INFINITY);
          }
          float mxv[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mxv[c] = -INFINITY;
#pragma unroll
          for (int c = 0; c < 64; c += 2)
            mxv[(c >> 1) & 7] =
                max3(mxv[(c >> 1) & 7], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
          const float mx = sl * max3(max3(mxv[0], mxv[1], mxv[2]), max3(mxv[3], mxv[4], mxv[5]),
                                     fmaxf(mxv[6], mxv[7]));
          if (j == seg.j0) {
            m = mx;
          } else {
            // The reference may lag the maximum by 2^8: weights stay below 2^8 and share one
            // reference with the sum and the output, so only a larger jump rescales those.
            const bool need = mx > m + 8.f;
            if (__builtin_expect(__any_sync(kFullMask, need), 0)) {
              if (!mbar_wait(o_done, (uint32_t)(jt - 1) & 1u, abort_flag, a.err)) {
                ok = false;
                break;
              }
              p_free = true;
              fence_after();
              const float mn = need ? mx : m;
              const float corr = need ? ex2(m - mn) : 1.f;
              m = mn;
              l *= corr;
#pragma unroll 1
              for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(tO + 32 * cc + lane_base, o);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st32(tO + 32 * cc + lane_base, o);
              }
              wait_st();
            }
          }
          // a row that has seen nothing yet: every weight 2^-inf = 0
          const float ref = (m == -INFINITY ? 0.f : m) - kLift;
          uint64_t ps2[4];
          const uint64_t sl2 = f32x2(sl, sl), nm2 = f32x2(-ref, -ref);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float e0, e1;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])),
                                  sl2, nm2),
                        e0, e1);
            const float p0 = ex2(e0), p1 = ex2(e1);
            const uint64_t pp = f32x2(p0, p1);
            ps2[c & 3] = c < 4 ? pp : add_f32x2(ps2[c & 3], pp);
            // The product takes 16-bit weights (the sum keeps them in fp32): bf16 beside bf16
            // V, off by 2^-8 of each at most, as the output's own rounding; f16 beside E4M3 codes,
            // 2^-11 of each down to kLift's floor.
            pk[c] = F8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
          }
          float s0, s1;
          f32x2_split(add_f32x2(add_f32x2(ps2[0], ps2[1]), add_f32x2(ps2[2], ps2[3])), s0, s1);
          l += s0 + s1;
        } else {
          if (lane == 0) mbar_arrive(s_free);
        }
        if (__builtin_expect(in_tree, 0)) {
          // keys past the context weigh nothing: their V (whatever it is) becomes zero, and
          // so do values of tree tokens that are not finite (E4M3: done by the V warp)
          const int slot = jt % VS;
          if (!mbar_wait(v_full + 8 * slot, (uint32_t)(jt / VS) & 1u, abort_flag, a.err)) {
            ok = false;
            break;
          }
          if (!F8) {
            const uint32_t vst = sV + slot * Lay::kVSlot;
            for (int e = t; e < kTileKeys * 8 * H; e += 128) {
              const int key = e / (8 * H), rem = e % (8 * H);
              const uint32_t at = vst + (rem >> 3) * Lay::kHalf + key * 128 + (rem & 7) * 16;
              if (t0 + key >= seg.ctx) {
                st_shared_v4(at, make_uint4(0u, 0u, 0u, 0u));
              } else if (t0 + key >= first) {
                uint4 v = ld_shared_v4(at);
                uint32_t *w = &v.x;
                bool hit = false;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if ((w[q] & 0x7f80u) == 0x7f80u) w[q] &= 0xffff0000u, hit = true;
                  if ((w[q] & 0x7f800000u) == 0x7f800000u) w[q] &= 0x0000ffffu, hit = true;
                }
                if (hit) {
                  st_shared_v4(at, v);
                  v_bad[j - tree_tile] = nseg;
                }
              }
            }
            fence_proxy_async();
          } else if (v_bad[slot] == jt + 1) {
            bad |= 1u << (j - tree_tile);
          }
        }
        if (!p_free) {
          if (!mbar_wait(o_done, (uint32_t)(jt - 1) & 1u, abort_flag, a.err)) {
            ok = false;
            break;
          }
          fence_after();
        }
        if (live) {
          tmem_st32(tP + lane_base, pk);
          wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (!ok || !mbar_wait(o_done, (uint32_t)(jt - 1) & 1u, abort_flag, a.err)) {
        ok = false;
        break;
      }
      fence_after();
      if (!live) continue;
      if (!F8)
        // every warp's marks precede its last arrival on p_full, and so this product's end;
        // the next segment's follow this warp's arrival on q_full
        for (int j = max(seg.j0, tree_tile); j < seg.j1; ++j)
          if (v_bad[j - tree_tile] == nseg) bad |= 1u << (j - tree_tile);
      const bool whole = seg.j0 == 0 && seg.j1 == seg.tiles;
      const float inv = l == 0.f ? 0.f : vs / l;
      const size_t part = ((size_t)plan->slot * 2 + (seg.j0 > 0 ? 0 : 1)) * kTileRows + t;
      if (whole) {
        // through this warp's rows of the staging region, so that a row's 128 bytes leave by
        // adjacent lanes
        const uint32_t stage = sQ + t * 128;
#pragma unroll 1
        for (int half = 0; half < H; ++half) {
#pragma unroll 1
          for (int cc = 0; cc < 2; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + 64 * half + 32 * cc + lane_base, o);
            wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int i2 = 0; i2 < 4; ++i2)
                w[i2] = pack_bf16(__uint_as_float(o[8 * c + 2 * i2]) * inv,
                                  __uint_as_float(o[8 * c + 2 * i2 + 1]) * inv);
              st_shared_v4(stage + (((4 * cc + c) ^ (t & 7)) << 4),
                           make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          __syncwarp();
          int rr = warp * 32 + (lane >> 3), tok = (r0 + rr) / G, head = (r0 + rr) - tok * G;
#pragma unroll 1
          for (; rr < warp * 32 + 32 && r0 + rr < rows; rr += 4) {
            *reinterpret_cast<uint4 *>(
                a.out + ((size_t)(seg.q0 + tok) * a.q_heads + seg.g * G + head) * D + 64 * half +
                8 * (lane & 7)) = ld_shared_v4(sQ + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            for (head += 4; head >= G; head -= G) ++tok;
          }
          __syncwarp();
        }
      } else {
        if (valid) a.part_lse[part] = l == 0.f ? -INFINITY : m + log2f(l);
        float4 *dst = a.part_o + (part - t) * (D / 4) + t;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * cc + lane_base, o);
          wait_ld();
          if (valid)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(8 * cc + e) * kTileRows] =
                  make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                              __uint_as_float(o[4 * e + 2]) * inv,
                              __uint_as_float(o[4 * e + 3]) * inv);
        }
      }
      if (__builtin_expect(bad != 0 && valid, 0))
        add_odd_values<D, F8>(
            a, seg, mask, bad, whole ? a.out + row : nullptr,
            whole ? nullptr : reinterpret_cast<float *>(a.part_o + (part - t) * (D / 4) + t));
      if (t == 0 && seg.j0 == 0 && !whole) {
        // the CTAs that run the rest of this pair's key tiles
        int parts = 1;
        for (long long rest = seg.tiles - seg.j1; rest > 0; ++parts)
          rest -= plan->cta_tiles + (plan->cta + parts < plan->extra ? 1 : 0);
        a.join[plan->slot] = TreeJoin{seg.q0, rows, seg.g, plan->m, parts, {0, 0, 0}};
      }
    }
    fence_before();
  } else {
  if constexpr (F8) set_regs_down<kOtherRegs>();
  if (warp == 4) {
    // ---------------- S warp: lane 0 issues S = Q K^T ----------------
    const uint32_t tmem = *tmem_at, tS = tmem, tQ = tmem + 96;
    constexpr uint32_t id = F8 ? idesc_e4m3(kTileRows, kTileKeys) : idesc(kTileRows, kTileKeys, false, false);
    int jt = 0, ok = 1;
    for (int nseg = 0; ok && segment(nseg); ++nseg) {
      if (lane == 0) ok = mbar_spin_wait(q_full, (uint32_t)nseg & 1u, abort_flag, a.err);
      ok = __shfl_sync(kFullMask, ok, 0);  // Q is staged
      if (!ok) break;
      fence_after();
      for (int j = seg.j0; j < seg.j1; ++j, ++jt) {
        const int sb = jt % KS;
        if (lane == 0)
          ok = mbar_spin_wait(k_full + 8 * sb, (uint32_t)(jt / KS) & 1u, abort_flag, a.err) &&
               (jt < 1 || mbar_spin_wait(s_free, (uint32_t)(jt - 1) & 1u, abort_flag, a.err));
        ok = __shfl_sync(kFullMask, ok, 0);
        if (!ok) break;
        fence_after();
        const uint32_t kst = sK + sb * Lay::kKSlot;
        if (lane == 0) {
          if constexpr (!F8) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t b = desc_sw128(kst + (kk >> 2) * Lay::kHalf + (kk & 3) * 32, 16, 1024);
              if (kk < 4)
                mma_ts(tS, tQ + 8 * kk, b, id, kk > 0 ? 1u : 0u);
              else
                mma_ss(tS, desc_sw128(sQ + (kk & 3) * 32, 16, 1024), b, id, 1u);
            }
          } else {
            // rows of 128 codes (128-byte swizzle) or 64 (64-byte), 32 columns a product
#pragma unroll
            for (int kk = 0; kk < 2 * D / 32; ++kk) {
              const int c = kk % (D / 32);
              const uint64_t b = H == 2 ? desc_sw128(kst + c * 32, 16, 1024)
                                        : desc_sw64(kst + c * 32, 16, 512);
              if (H == 1 || kk < D / 32)
                mma_ts_f8(tS, tQ + 8 * kk, b, id, kk > 0 ? 1u : 0u);
              else
                mma_ss_f8(tS, desc_sw128(sQ + c * 32, 16, 1024), b, id, 1u);
            }
          }
          commit(s_full);
          commit(k_empty + 8 * sb);
        }
        __syncwarp();
      }
    }
    if (lane == 0) commit(fin_s);
    __syncwarp();
    mbar_drain(fin_s, 0);
    fence_before();
  } else if (warp == 7) {
    // ---------------- P V warp: lane 0 issues O += P V ----------------
    const uint32_t tmem = *tmem_at, tP = tmem + 64, tO = tmem + 128;
    fence_after();
    // bf16: V [keys][D] (MN-major); E4M3: V widened to [D][keys] (K-major)
    constexpr uint32_t id = idesc(kTileRows, D, F8, !F8);
    int jt = 0, ok = 1;
    for (int nseg = 0; ok && segment(nseg); ++nseg) {
      for (int j = seg.j0; j < seg.j1; ++j, ++jt) {
        const int sb = jt % VS;
        if (lane == 0)
          ok = mbar_spin_wait(p_full, (uint32_t)jt & 1u, abort_flag, a.err) &&
               mbar_spin_wait(v_full + 8 * sb, (uint32_t)(jt / VS) & 1u, abort_flag, a.err);
        ok = __shfl_sync(kFullMask, ok, 0);
        if (!ok) break;
        fence_after();
        const uint32_t vst = sV + sb * Lay::kVSlot;
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            mma_ts(tO, tP + 8 * k,
                   F8 ? desc_sw128(vst + 32 * k, 16, 1024)
                      : desc_sw128(vst + 2048 * k, Lay::kHalf, 1024),
                   id, (j > seg.j0 || k > 0) ? 1u : 0u);
          commit(o_done);
          commit(v_empty + 8 * sb);
        }
        __syncwarp();
      }
    }
    if (lane == 0) commit(fin_o);
    __syncwarp();
    mbar_drain(fin_o, 0);
    fence_before();
  } else if (warp < 7) {
    // ---------------- copying warps: warp 5 K, warp 6 V ----------------
    const bool is_v = warp == 6;
    // one row tile: the cache is read once, its L2 lines go first; several: the row tiles of
    // a pair share them
    uint64_t pol;
    if (a.row_tiles == 1)
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    else
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    // What this warp copies: tiles into a ring of `slots`, lane b the tile's block b.
    const int slots = F8 && is_v ? RS : is_v ? VS : KS;
    const uint32_t full = F8 && is_v ? raw_full : is_v ? v_full : k_full;
    const uint32_t empty = F8 && is_v ? raw_empty : is_v ? v_empty : k_empty;
    const uint32_t ring = F8 && is_v ? base + Lay::kRawV : is_v ? sV : sK;
    int nseg = 0;
    int aj = 0;
    // The table's entry of key tile j for this lane's block (`held`: not past the context).
    // Read one tile before it is looked at, so that nothing waits for the load.
    bool held = false;
    int next_blk = -1;
    auto read_block = [&](int j) {
      const int tok = j * kTileKeys + lane * kBlockSize;
      held = lane < kTileBlocks && tok < seg.ctx;
      if (held) next_blk = a.block_tables[(size_t)seg.s * a.max_blocks + tok / kBlockSize];
    };
    // The next segment: the K warp finds and publishes it, both take it from the ring.
    auto advance = [&]() {
      if (!is_v && lane == 0) {
        walk_of(plan)->next(a, plan->m, ring_seg[nseg % kSegRing]);
        mbar_arrive(seg_full + 8 * (nseg % kSegRing));
      }
      __syncwarp();
      if (!__all_sync(kFullMask, segment(nseg++))) return false;
      aj = seg.j0;
      read_block(aj);
      return true;
    };
    bool more = advance();
    int issued = 0, slot_in = 0;
    uint32_t empty_parity = 1;  // of the ring's previous round
    // Queues the run's next tile once its slot is free; false: gave up.
    auto issue = [&]() {
      int blk = held ? next_blk : -1;
      const int g = seg.g;
      if (held && (unsigned)blk >= (unsigned)a.num_blocks) {
        flag_error(a.err, PKV_DEV_BAD_BLOCK);
        blk = -1;
      }
      if (++aj < seg.j1)
        read_block(aj);  // one tile ahead
      else
        more = advance();
      if (issued >= slots && !mbar_wait(empty + 8 * slot_in, empty_parity, abort_flag, a.err))
        return false;
      if (lane < kTileBlocks) {
        const uint32_t bar = full + 8 * slot_in;
        mbar_arrive_expect_tx(bar, blk >= 0 ? (uint32_t)(kBlockSize * D * (F8 ? 1 : 2)) : 0u);
        if (blk >= 0) {
          const int row = (blk * a.kv_heads + g) * kBlockSize;
          if constexpr (!F8) {
            const uint32_t dst = ring + slot_in * Lay::kVSlot + lane * 2048;
#pragma unroll
            for (int h = 0; h < H; ++h)
              tma_load_2d_hint(dst + h * Lay::kHalf, is_v ? &tv : &tk, 64 * h, row, bar, pol);
          } else if (is_v) {  // [D][16] codes, contiguous
            bulk_load_hint(ring + slot_in * Lay::kRaw + lane * (kBlockSize * D),
                           static_cast<const uint8_t *>(a.v_cache) + (size_t)row * D,
                           kBlockSize * D, bar, pol);
          } else {
            tma_load_2d_hint(ring + slot_in * Lay::kRaw + lane * (kBlockSize * D), &tk, 0, row, bar,
                             pol);
          }
        }
      }
      ++issued;
      if (++slot_in == slots) slot_in = 0, empty_parity ^= 1;
      return true;
    };
    while (more && __all_sync(kFullMask, issue())) {
    }
    if (lane == 0 && *abort_flag)
      for (int j = max(0, issued - slots); j < issued; ++j)
        mbar_drain(full + 8 * (j % slots), (uint32_t)(j / slots) & 1u);
  } else if constexpr (F8) {
    // ---------------- widening warps ----------------
    // The V codes [D][16 keys] of each tile to f16, exactly, as a K-major operand [D][64 keys]
    // (128-byte swizzle), a quarter of the 16-code rows each.
    {
      bool ok = true;
      int jt = 0;
      for (int nseg = 0; ok && segment(nseg); ++nseg) {
        const int first = seg.ctx - seg.L;
        for (int j = seg.j0; j < seg.j1; ++j, ++jt) {
          const int slot = jt % VS, rs = jt % RS, t0 = j * kTileKeys;
          ok = mbar_wait(raw_full + 8 * rs, (uint32_t)(jt / RS) & 1u, abort_flag, a.err) &&
               (jt < VS || mbar_wait(v_empty + 8 * slot, (uint32_t)((jt - VS) / VS) & 1u,
                                     abort_flag, a.err));
          ok = __all_sync(kFullMask, ok);
          if (!ok) break;
          // A step: 16 codes a lane, row d of block blk, to two chunks of the operand's row.
          // The loop stays short: a longer body and the softmax's code do not fit the
          // instruction cache together (batch of 64: 166 us, unrolled twice 170, four times 179).
          constexpr int kSteps = kTileKeys * D / (16 * 128);
          const int e0 = (warp - 8) * 32 + lane;
          const uint32_t src = base + Lay::kRawV + rs * Lay::kRaw + e0 * 16;
          const uint32_t dst = sV + slot * Lay::kVSlot;
          bool hit = false;
          if (__builtin_expect(t0 + kTileKeys > first, 0)) {
            // a tile of the tree: keys past the context, and values that are not finite,
            // become zero
            auto bytes_below = [](int n) {  // a mask of a word's first n bytes
              return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
            };
#pragma unroll 1
            for (int it = 0; it < kSteps; ++it) {
              uint4 v = ld_shared_v4(src + it * 2048);
              int key = t0 + (it * 128 + e0) / D * kBlockSize;
              uint32_t *w = &v.x;
#pragma unroll
              for (int q = 0; q < 4; ++q, key += 4) {
                const uint32_t held = bytes_below(seg.ctx - key);
                const uint32_t nan = nan_codes(w[q]) & held & ~bytes_below(first - key);
                hit |= nan != 0;
                w[q] &= held & ~((nan >> 7) * 0xffu);
              }
              st_shared_v4(src + it * 2048, v);
            }
          }
#pragma unroll 1
          for (int it = 0; it < kSteps; ++it) {
            const uint4 v = ld_shared_v4(src + it * 2048);
            const int e = it * 128 + e0, blk = e / D, d = e % D;
            const uint32_t row = dst + d * 128;
            st_shared_v4(row + (((blk * 2) ^ (d & 7)) << 4),
                         make_uint4(e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16),
                                    e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.y >> 16)));
            st_shared_v4(row + (((blk * 2 + 1) ^ (d & 7)) << 4),
                         make_uint4(e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.z >> 16),
                                    e4m3x2_to_f16x2(v.w), e4m3x2_to_f16x2(v.w >> 16)));
          }
          if (hit) v_bad[slot] = jt + 1;  // read by the softmax warps after v_full
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(raw_empty + 8 * rs);
            mbar_arrive(v_full + 8 * slot);
          }
        }
      }
    }
  }
  }

  __syncthreads();
  if (warp == 4) {
    fence_after();
    dealloc(*tmem_slot, kTmemColumns);
  }
}

// Joins the parts of a (sequence, KV head, row tile) whose key tiles several CTAs ran: part 0
// is the last segment of CTA b, part k > 0 the first segment of CTA b + k.
//   M = max lse_k,  out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M)   over lse_k > -inf
// A thread has one row and four head-dim columns at a time, a warp 32 adjacent rows: its loads
// are whole lines, just written and still in L2.  What costs is the round trips (the record,
// then the weights, then the values), so the first two parts' are asked for with the record:
// where they lie does not depend on it, and most pairs have two or three.
constexpr int kMergeThreads = 256, kMergeSplit = 4;
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, t = threadIdx.x & (kTileRows - 1);
  constexpr int kStep = kMergeSplit * (kMergeThreads / kTileRows);
  constexpr int kCols = D / 4 / kStep;  // of a thread
  const int c0 = blockIdx.y * (kMergeThreads / kTileRows) + threadIdx.x / kTileRows;
  // part 0 is CTA b's second slot, part k > 0 the first of CTA b + k
  const float *lse = a.part_lse + (size_t)(2 * b) * kTileRows + t;
  const float4 *val = a.part_o + ((size_t)(2 * b) * (D / 4) + c0) * kTileRows + t;
  auto slot = [&](int k) { return 2 * k + (k == 0 ? 1 : 0); };
  auto value = [&](int k, int c) {
    return __ldcg(val + ((size_t)slot(k) * (D / 4) + c * kStep) * kTileRows);
  };
  const float x0 = __ldcg(lse + slot(0) * kTileRows);
  float x1 = -INFINITY;
  float4 v0[kCols], v1[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) v0[c] = value(0, c);
  if (b + 1 < gridDim.x) {
    x1 = __ldcg(lse + slot(1) * kTileRows);
#pragma unroll
    for (int c = 0; c < kCols; ++c) v1[c] = value(1, c);
  }
  const TreeJoin it = a.join[b];
  if (it.parts == 0) return;
  const int G = a.group, r = it.m * kTileRows + t;
  if (r >= it.rows) return;
  float M = fmaxf(x0, x1);
#pragma unroll 4
  for (int k = 2; k < it.parts; ++k) M = fmaxf(M, __ldcg(lse + slot(k) * kTileRows));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 o[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float x, const float4(&v)[kCols]) {
    const float w = exp2f(x - ref);
    L += w;
    if (w != 0.f) {
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        o[c] = make_float4(fmaf(w, v[c].x, o[c].x), fmaf(w, v[c].y, o[c].y),
                           fmaf(w, v[c].z, o[c].z), fmaf(w, v[c].w, o[c].w));
    } else if (x != -INFINITY) {
      // a weight that vanishes in fp32 but is above zero: of its values those that are not
      // finite count (a part that saw nothing, lse -inf, adds nothing)
      auto odd = [](float e) { return fabsf(e) < INFINITY ? 0.f : e; };
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        o[c] = make_float4(o[c].x + odd(v[c].x), o[c].y + odd(v[c].y), o[c].z + odd(v[c].z),
                           o[c].w + odd(v[c].w));
    }
  };
  add(x0, v0);
  add(x1, v1);
#pragma unroll 4
  for (int k = 2; k < it.parts; ++k) {
    float4 v[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) v[c] = value(k, c);
    add(__ldcg(lse + slot(k) * kTileRows), v);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint16_t *out = a.out + ((size_t)(it.q0 + r / G) * a.q_heads + it.g * G + r % G) * D + 4 * c0;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    *reinterpret_cast<uint2 *>(out + 4 * kStep * c) =
        make_uint2(pack_bf16(o[c].x * inv, o[c].y * inv), pack_bf16(o[c].z * inv, o[c].w * inv));
}

// Workspace: join records, then the parts' log-sum-exps and outputs.
struct TreeWorkspace {
  int64_t ctas;
  size_t lse_off, o_off, total;
};
TreeWorkspace tree_workspace(int group, int head_dim, int max_query_len) {
  TreeWorkspace w;
  const int64_t tiles = ((int64_t)max_query_len * group + kTileRows - 1) / kTileRows;
  w.ctas = 2 * device_sm_count() + (tiles < kMaxRowTiles ? tiles : kMaxRowTiles);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  w.lse_off = up(w.ctas * sizeof(TreeJoin));
  w.o_off = up(w.lse_off + w.ctas * 2 * kTileRows * sizeof(float));
  w.total = up(w.o_off + w.ctas * 2 * kTileRows * (size_t)head_dim * sizeof(float));
  return w;
}

template <int D, bool F8>
int launch_tree(TreeArgs a, int64_t tiles, int64_t ctas, const CUtensorMap &tk,
                const CUtensorMap &tv, cudaStream_t st) {
  using Lay = TreeLayout<D, F8>;
  static std::atomic<int> ready[kMaxDevices];  // shared-memory opt-in and carve-out, per device
  const int r = per_device_setup(ready, [] {
    cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<D, F8>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Lay::kSmemLaunch);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(tree_attention_kernel<D, F8>,
                               cudaFuncAttributePreferredSharedMemoryCarveout,
                               (int)cudaSharedmemCarveoutMaxShared);
    // the register split above draws on what the kernel was compiled for
    cudaFuncAttributes at;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, tree_attention_kernel<D, F8>);
    return e == cudaSuccess && (!F8 || at.numRegs >= kLaunchRegs) ? 1 : -1;
  });
  if (r <= 0) return PKV_ERR_CUDA;
  a.runs = 2 * device_sm_count();
  a.start = F8 ? kStartF8 : kStart;
  for (int64_t m0 = 0; m0 < tiles; m0 += kMaxRowTiles) {
    a.m0 = (int)m0;
    a.row_tiles = (int)(tiles - m0 < kMaxRowTiles ? tiles - m0 : kMaxRowTiles);
    const unsigned grid = (unsigned)(a.runs + a.row_tiles - 1);
    if ((int64_t)grid > ctas) return PKV_ERR_WORKSPACE;
    if (launch_pdl(tree_attention_kernel<D, F8>, dim3(grid), dim3(tree_threads(F8)),
                   (size_t)Lay::kSmemLaunch, st, a, tk, tv) != cudaSuccess ||
        launch_pdl(tree_merge_kernel<D>, dim3(grid, kMergeSplit), dim3(kMergeThreads), 0, st, a) != cudaSuccess)
      return PKV_ERR_CUDA;
  }
  return PKV_OK;
}

int tree_impl(uint16_t *out, const uint16_t *q, const void *k_cache, const void *v_cache,
              const int32_t *block_tables, const int32_t *context_lens,
              const int32_t *query_start, const uint64_t *masks, int mask_words, int num_seqs,
              int num_tokens, int max_blocks_per_seq, int num_q_heads, int num_kv_heads,
              int head_dim, int block_size, int num_blocks, float scale, bool f8, float k_scale,
              float v_scale, const float *k_scales, const float *v_scales, int max_query_len,
              void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
  if (block_size != kBlockSize) return PKV_ERR_BLOCK_SIZE;
  if (num_seqs < 0 || num_seqs > 65535 || num_tokens < 0 || max_blocks_per_seq <= 0 ||
      num_q_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535 || num_blocks <= 0 ||
      num_q_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128) || mask_words <= 0 ||
      mask_words > PKV_TREE_MAX_TOKENS / 64 || max_query_len < 0 ||
      max_query_len > 64 * mask_words || !(scale > 0.f) || !(k_scale > 0.f) || !(v_scale > 0.f))
    return PKV_ERR_SHAPE;
  if ((uint64_t)num_blocks * num_kv_heads * kBlockSize >= (1ull << 31) ||
      (int64_t)max_query_len * num_q_heads > INT_MAX)
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start ||
      !masks || !workspace)
    return PKV_ERR_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_ALIGN;
  const int group = num_q_heads / num_kv_heads;
  const TreeWorkspace ws = tree_workspace(group, head_dim, max_query_len);
  if (workspace_bytes < ws.total) return PKV_ERR_WORKSPACE;
  TreeArgs a = {};
  a.out = out, a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
  a.block_tables = block_tables, a.context_lens = context_lens, a.query_start = query_start;
  a.masks = masks;
  a.num_seqs = num_seqs, a.num_tokens = num_tokens, a.max_blocks = max_blocks_per_seq;
  a.q_heads = num_q_heads, a.kv_heads = num_kv_heads, a.group = group;
  a.num_blocks = num_blocks, a.words = mask_words, a.max_query_len = max_query_len;
  a.scale_log2 = (float)((double)scale * (double)k_scale * 1.4426950408889634);
  a.v_scale = v_scale;
  a.k_scales = k_scales, a.v_scales = v_scales;
  char *wb = static_cast<char *>(workspace);
  a.join = reinterpret_cast<TreeJoin *>(wb);
  a.part_lse = reinterpret_cast<float *>(wb + ws.lse_off);
  a.part_o = reinterpret_cast<float4 *>(wb + ws.o_off);
  a.err = err_flag;
  CUtensorMap tk = {}, tv = {};
  const uint64_t rows = (uint64_t)num_blocks * num_kv_heads * kBlockSize;
  if (!kv_tensor_map(&tk, k_cache, rows, head_dim, f8 ? 1 : 2) ||
      (!f8 && !kv_tensor_map(&tv, v_cache, rows, head_dim, 2)))
    return PKV_ERR_CUDA;
  const int64_t tiles = ((int64_t)max_query_len * group + kTileRows - 1) / kTileRows;
  const cudaStream_t st = (cudaStream_t)stream;
  if (head_dim == 128)
    return f8 ? launch_tree<128, true>(a, tiles, ws.ctas, tk, tv, st)
              : launch_tree<128, false>(a, tiles, ws.ctas, tk, tv, st);
  return f8 ? launch_tree<64, true>(a, tiles, ws.ctas, tk, tv, st)
            : launch_tree<64, false>(a, tiles, ws.ctas, tk, tv, st);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t paged_attention_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim,
                                           int max_query_len) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128) || max_query_len < 0 ||
      max_query_len > PKV_TREE_MAX_TOKENS)
    return 0;
  return tree_workspace(num_q_heads / num_kv_heads, head_dim, max_query_len).total;
}

int paged_attention_tree(uint16_t *out, const uint16_t *q, const uint16_t *k_cache,
                         const uint16_t *v_cache, const int32_t *block_tables,
                         const int32_t *context_lens, const int32_t *query_start,
                         const uint64_t *tree_masks, int mask_words, int num_seqs,
                         int num_tokens, int max_blocks_per_seq, int num_q_heads,
                         int num_kv_heads, int head_dim, int block_size, int num_blocks,
                         float scale, int max_query_len, void *workspace,
                         size_t workspace_bytes, int32_t *err_flag, void *stream) {
  return tree_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start, tree_masks,
                   mask_words, num_seqs, num_tokens, max_blocks_per_seq, num_q_heads,
                   num_kv_heads, head_dim, block_size, num_blocks, scale, false, 1.f, 1.f, nullptr,
                   nullptr, max_query_len, workspace, workspace_bytes, err_flag, stream);
}

int paged_attention_tree_fp8(uint16_t *out, const uint16_t *q, const uint8_t *k_cache,
                             const uint8_t *v_cache, const int32_t *block_tables,
                             const int32_t *context_lens, const int32_t *query_start,
                             const uint64_t *tree_masks, int mask_words, int num_seqs,
                             int num_tokens, int max_blocks_per_seq, int num_q_heads,
                             int num_kv_heads, int head_dim, int block_size, int num_blocks,
                             float scale, float k_scale, float v_scale, const float *k_scales,
                             const float *v_scales, int max_query_len, void *workspace,
                             size_t workspace_bytes, int32_t *err_flag, void *stream) {
  if ((k_scales == nullptr) != (v_scales == nullptr)) return PKV_ERR_NULL;
  if (k_scales != nullptr) k_scale = v_scale = 1.f;
  return tree_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start, tree_masks,
                   mask_words, num_seqs, num_tokens, max_blocks_per_seq, num_q_heads,
                   num_kv_heads, head_dim, block_size, num_blocks, scale, true, k_scale, v_scale,
                   k_scales, v_scales, max_query_len, workspace, workspace_bytes, err_flag,
                   stream);
}

}  // extern "C"
