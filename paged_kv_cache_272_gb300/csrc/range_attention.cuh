// Attention of row tiles over ranges of keys of the paged cache, on tcgen05 tensor cores: the
// kernel behind shared-prefix decode and behind scored attention.
//
// A row tile is 128 rows: the (token, query head) pairs of one KV head's group, of tokens whose
// keys come through one block table.  Row r is token r / G and head r % G of the group.  For
// shared-prefix decode the tokens are one of each sequence of a group, the keys the prefix.  For
// scored attention they are a sequence's new tokens, each with a range of keys of its own.  A plan
// (one CTA, a launch of its own) lists the row tiles and the keys [kb, ke) each needs, and cuts the
// keys of (row tile, KV head) pairs, in tiles of 64, into runs of equal length, one per resident
// CTA, or has the CTAs claim whole pairs:
//  * all pairs' tiles laid end to end, a few units for each pair's start before them; or
//  * (shared-prefix decode) each row tile of a group in a lane of its own, cut alike, so that the
//    row tiles of one key range run side by side and the keys come from DRAM once; or
//  * (scored attention, many even pairs) pairs claimed in the order of sequence, KV head, row tile,
//    so that what runs at any time are the row tiles of a few key ranges, which L2 keeps (chunks of
//    512 over 4096 keys, eight sequences: 0.19 GB from DRAM, in runs 1.8), the last pairs in halves,
//    so that the CTAs end together.
// A pair that was cut leaves normalised fp32 parts that another launch joins by their log-sum-exp
// in the order of the keys; no result depends on timing.
//
// One CTA, warps by role:
//  * 0-3 softmax: thread t owns row t (TMEM lane t).  Q staged (64 head-dim columns in TMEM,
//    the others in shared memory), scores read, changed (cap, distance), masked; running maximum
//    and sum in fp32; weights to TMEM; the output accumulator rescaled when the maximum grows by
//    more than 2^8; a segment finished.
//  * 4 issues S = Q K^T, 7 O += P V (one lane each).
//  * 5 and 6 copy K and V blocks by TMA, through the block table.
//  * E4M3 cache: K's codes are an operand as they are (q as the sum of two E4M3 terms), V's are
//    widened to f16, exactly, by warps 8-11.
//
// Masked values.  Keys outside [kb, ke) are other sequences' or nobody's, and where rows differ
// in what they see a weight of zero times a V element that is not finite would spoil a row that
// does not see it.  So in the tiles on such borders V rows outside [kb, ke) become zero, and
// elements that are not finite of keys that not every row sees are taken out of the product and
// added at the end to the rows that do.
//
// What bounds it (GB300): a decode of 24 sequences of up to 8192 keys, 32 heads, reads its 2.16 GB at
// 6.6 TB/s, the copy's rate.  Chunks of 512 (eight, window 4096, 32 heads on 8) are bound by the
// softmax warps, two a scheduler: 259 us, 1060 TFLOP/s; 357 with a cap (no pipe above 36%, 2.1 issues
// a cycle and SM).  Short ranges (packed documents, 7 key tiles a segment: 55 us)
// by a segment's start and finish, the plan and the join.
#pragma once

#include <cuda.h>
#include <math.h>

#include <atomic>
#include <climits>

#include "e4m3.cuh"
#include "run_join.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace ra {

using namespace t5;

constexpr unsigned kFullMask = 0xffffffffu;
constexpr int kTileKeys = 64;
constexpr int kTileBlocks = kTileKeys / kBlockSize;
__host__ __device__ constexpr int threads(bool f8) { return f8 ? 384 : 256; }
// Registers per thread, 64 K for the two CTAs of an SM: what the kernel is compiled and launched
// with, and what the softmax warps take of the others' share.
template <bool F8>
struct Regs {
  static constexpr int launch = F8 ? 80 : 128, softmax = F8 ? 160 : 168, other = F8 ? 40 : 88;
  static_assert(128 * softmax + (threads(F8) - 128) * other <= threads(F8) * launch, "split");
};
constexpr uint32_t kTmemColumns = 256;
// A segment's start and finish, in key tiles, and the least units of a run: as measured for the
// attention of drafted trees, whose segments do the same.
constexpr int kStart = 5, kStartF8 = 12;
constexpr int kMinRun = 4;
// E4M3: weights enter their product as f16 of 2^kLift times themselves, so that none above 2^-32
// of the largest is lost.
constexpr float kLiftF8 = 7.f;
// tanh(y) / y for |y| <= near, in powers of y^2 (least largest error of y times it).  To a cap of 64:
// off by 2^-19.7 of the cap, 2^-13.7 at most in the exponent, far below a weight's rounding, and most
// tiles of usual scores take it.  Above, where that is up to 0.005: the first power is 1, so that
// scores far below the cap stay what they are, and it is off by 2^-23.6 of the cap.
struct TanhFit {
  float near, c[4];
};
constexpr float kFineCap = 64.f;
inline TanhFit tanh_fit(float cap) {
  return cap <= kFineCap ? TanhFit{0.65f, {0.9999839067459106f, -0.33280691504478455f,
                                           0.1286155879497528f, -0.037672240287065506f}}
                         : TanhFit{0.45f, {1.f, -0.3332953155040741f, 0.1323312669992447f,
                                           -0.04587532579898834f}};
}

// What a score goes through: nothing (every row of a tile sees the same keys), a key range per
// row, or that and a cap, a distance bias or both (instances of their own: what the others need
// costs registers and instruction fetch; in one instance a cap takes 405 us instead of 354, a bias
// 310 instead of 292).
enum Mode { kPlain, kRanges, kCapped, kBiased, kCappedBiased };
__host__ __device__ constexpr bool has_cap(Mode m) { return m == kCapped || m == kCappedBiased; }
__host__ __device__ constexpr bool has_bias(Mode m) { return m == kBiased || m == kCappedBiased; }

struct __align__(16) RowTile {
  int seq;          // block table row
  int q0, L;        // first token and tokens of the owner of the rows (L G rows)
  int ctx;          // scored: cached tokens of the sequence (token i stands at ctx - L + i)
  int m;            // row tile of the owner
  int kb, ke;       // keys some row sees lie in [kb, ke)
  int ib, ie;       // keys in [ib, ie) are seen by every row
  int tiles;        // key tiles from kb rounded down to a block on; 0: nothing to do
  int first, count; // row tiles that share this one's keys
  int extra, run0, step, pad0;
  unsigned long long unit0, stride;  // unit of (this, head g) = unit0 + g stride
  unsigned long long quot, pad;      // units of a run: quot, one more for the first `extra` runs;
                                     // these are the runs run0, run0 + step, ..
  __device__ __forceinline__ int run_of(unsigned long long unit) const {
    const unsigned long long longer = (unsigned long long)extra * (quot + 1);
    const unsigned long long a = unit < longer ? unit : unit - longer;
    const unsigned long long b = unit < longer ? quot + 1 : quot;
    const int i = (unit < longer ? 0 : extra) +
                  (int)(((a | b) >> 32) == 0 ? (unsigned)a / (unsigned)b : a / b);
    return run0 + i * step;
  }
};

struct __align__(16) Run {
  int tile, g, unit;  // where it begins: row tile, KV head, unit of that pair
  int lane;           // it goes on with the same row tile's next head (else with the next pair)
  long long units, pad;
};
struct PlanHead {
  int runs;    // -1: pairs are claimed
  int claims;  // what there is to claim: whole pairs, then two halves each of the others
  int next, whole;
};
// Pairs of row tile and KV head in the order of claims: pair p is of the row tiles that share keys
// with tile p / H.
struct Pair {
  int tile, g;
};
__device__ __forceinline__ Pair pair_of(int p, int first, int count, int H) {
  const int in = p - first * H;
  return Pair{first + in % count, in / count};
}
// Whether a pair of the last ones is done in halves.
__device__ __forceinline__ bool halved(int tiles) { return tiles >= 2 * kMinRun; }

// First unit of run i of those that share units evenly.
__device__ __forceinline__ unsigned long long run_begin(unsigned long long quot, int extra, int i) {
  return (unsigned long long)i * quot + (unsigned long long)min(i, extra);
}

// Shared-prefix decode: what the join needs of a sequence.
struct __align__(16) SeqParts {
  int own, parts;     // its own keys' partial results (own -1: it is in no group)
  int index, prefix;  // its number within the group, the first row tile of the prefix (-1: none)
};

struct Args {
  uint16_t *out;                // [T][Hq][D] bf16
  const uint16_t *q;            // [T][Hq][D] bf16
  const void *k_cache, *v_cache;
  const int32_t *block_tables;  // [S][MB]
  const int32_t *context_lens;  // [S]
  const int32_t *starts;        // query_start [S+1], or group_start [groups + 1]
  const int32_t *prefix_lens;   // shared: [groups]
  const int32_t *key_begin, *key_end;  // scored: [T] or null
  const float *slopes;          // scored: [Hq] or null
  int num_groups;
  int num_seqs, num_tokens, max_blocks, q_heads, kv_heads, group, num_blocks;
  float scale;                  // (* k_scale of an E4M3 cache)
  float cap;                    // 0: none
  TanhFit fit;                  // of the cap
  float v_scale;
  const float *k_scales, *v_scales;  // [Hkv] or null
  int ctas;                     // most runs
  int start;                    // what a segment costs besides its tiles, in tiles
  int max_tiles;                // row tiles the workspace holds
  PlanHead *head;
  Run *run;                     // [ctas]
  RowTile *tile;                // [max_tiles]
  unsigned long long *before;   // [max_tiles + 1] units of the row tiles before, one KV head
  int32_t *tile0;               // [owners + 1] first row tile of each owner
  SeqParts *parts;              // shared: [S]
  int variant, least_tiles;     // shared: PKV_SHARED_*, key tiles of a head to save in all
  int lane_tiles;               // shared: key tiles (all heads) from which on row tiles run in lanes
  int32_t *groups;              // shared: [2][3][groups + 1] the plan's lists
  TreeJoin *join;               // [ctas]
  float *part_lse;              // [ctas][2][128] log2-sum-exp2
  float4 *part_o;               // [ctas][2][D / 4][128] normalised; shared: [..][128][D / 4]
  // shared: [S][Hq] and [S][Hq][D / 4], first parts of the prefix.  The runs' parts follow, then
  // the own keys': one numbering of rows for all of them.
  float *row_lse;
  float4 *row_o;
  int32_t *err;
};

// ---- plan ---------------------------------------------------------------------------
// Threads of a plan: as many as there are things to list, of a few sizes (a barrier of 32 warps and
// what is read again from memory are what its phases cost: a microsecond each).
constexpr int kPlanThreads = 1024;
inline unsigned plan_threads(int64_t things) {
  return things <= 128 ? 128u : things <= 256 ? 256u : things <= 512 ? 512u : (unsigned)kPlanThreads;
}
// What the runs are cut by, of the first kPlanThreads row tiles, in shared memory.
struct FewTiles {
  int tiles[kPlanThreads], first[kPlanThreads], count[kPlanThreads];
};

// Exclusive sums of N values over the CTA's threads, in place; `total` for all.  scratch: 33 N
// words.
template <int N>
__device__ __forceinline__ void cta_scan(unsigned long long (&v)[N], unsigned long long (&total)[N],
                                         unsigned long long *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  unsigned long long incl[N];
#pragma unroll
  for (int i = 0; i < N; ++i) incl[i] = v[i];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned long long t = __shfl_up_sync(kFullMask, incl[i], off);
      if (lane >= off) incl[i] += t;
    }
  }
  __syncthreads();  // scratch of the scan before
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 31) scratch[33 * i + warp] = incl[i];
  __syncthreads();
  if (warp < N) {
    const unsigned long long mine = lane < warps ? scratch[33 * warp + lane] : 0;
    unsigned long long s = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long t = __shfl_up_sync(kFullMask, s, off);
      if (lane >= off) s += t;
    }
    if (lane < warps) scratch[33 * warp + lane] = s - mine;
    if (lane == 31) scratch[33 * warp + 32] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = scratch[33 * i + 32];
    v[i] = scratch[33 * i + warp] + incl[i] - v[i];
  }
}
__device__ __forceinline__ unsigned long long cta_scan(unsigned long long v,
                                                       unsigned long long *scratch,
                                                       unsigned long long &total) {
  unsigned long long x[1] = {v}, t[1];
  cta_scan(x, t, scratch);
  total = t[0];
  return x[0];
}

// Last i in [0, n) with a[i] <= x (a[0] <= x).
template <typename T, typename X>
__device__ __forceinline__ int last_not_above(const T *a, int n, X x) {
  int lo = 0, hi = n;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((X)a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// a / b, mostly of numbers that 32 bits hold.
__device__ __forceinline__ unsigned long long quotient(unsigned long long a, unsigned long long b) {
  return ((a | b) >> 32) == 0 ? (unsigned)a / (unsigned)b : a / b;
}

__device__ __forceinline__ int key_tiles(int kb, int ke) {
  const int origin = kb & ~(kBlockSize - 1);
  return (int)(((int64_t)ke - origin + kTileKeys - 1) / kTileKeys);
}

// The row tiles are listed (tile[0 .. n), all but unit0 to quot; the first kPlanThreads of them in
// `few` too): cuts them into runs.  All threads of the plan's CTA.
__device__ __forceinline__ void plan_runs(const Args &a, int n, const FewTiles &few,
                                          unsigned long long *scratch) {
  const int tid = threadIdx.x, threads = blockDim.x;
  // units of the row tiles before, one KV head (looked up by bisection: in shared memory where
  // they are few)
  __shared__ unsigned long long few_before[kPlanThreads + 1];
  const bool is_few = n <= kPlanThreads;
  unsigned long long *const before = is_few ? few_before : a.before;
  auto first_of = [&](int i) { return is_few ? few.first[i] : a.tile[i].first; };
  auto count_of = [&](int i) { return is_few ? few.count[i] : a.tile[i].count; };
  unsigned long long base = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += threads) {
    const int i = i0 + tid;
    const int t = i < n ? (is_few ? few.tiles[i] : a.tile[i].tiles) : 0;
    unsigned long long total;
    const unsigned long long ex =
        cta_scan(t > 0 ? (unsigned long long)(t + a.start) : 0, scratch, total);
    if (i < n) before[i] = base + ex;
    base += total;
  }
  if (tid == 0) before[n] = base;
  __syncthreads();
  const unsigned H = (unsigned)a.kv_heads;
  const unsigned long long units = base * H;
  const unsigned long long some = (units + kMinRun - 1) / kMinRun;
  const int runs = some < (unsigned long long)a.ctas ? (int)some : a.ctas;
  const unsigned long long quot = runs ? quotient(units, (unsigned)runs) : 0;
  const int extra = (int)(units - quot * (unsigned)runs);
  if (tid == 0) a.head->runs = runs;
#pragma unroll 1
  for (int i = tid; i < n; i += threads) {
    RowTile &t = a.tile[i];
    const int first = first_of(i);
    const unsigned long long b0 = before[first];
    t.unit0 = b0 * H + (before[i] - b0);
    t.stride = before[first + count_of(i)] - b0;
    t.quot = quot, t.extra = extra, t.run0 = 0, t.step = 1;
  }
#pragma unroll 1
  for (int r = tid; r < runs; r += threads) {
    const unsigned long long x = run_begin(quot, extra, r);
    // the row tile at that share of one head's units is of the block of tiles looked for
    const int i = last_not_above(before, n, quotient(x, H));
    const int first = first_of(i), count = count_of(i);
    const unsigned long long b0 = before[first], per = before[first + count] - b0;
    const unsigned long long rest = x - b0 * H, head = quotient(rest, per), in = rest - head * per;
    const int k = first + last_not_above(before + first, count, b0 + in);
    Run o;
    o.g = (int)head, o.tile = k, o.unit = (int)(in - (before[k] - b0));
    o.lane = 0, o.units = (long long)quot + (r < extra ? 1 : 0), o.pad = 0;
    a.run[r] = o;
  }
}

// ---- the attention kernel -----------------------------------------------------------
// Segments of a run.  The K warp walks them in order, ahead of everyone, and hands them on
// through a small ring; one with no tiles ends the run.  It is at most eight segments ahead of the
// slowest reader: K of tile t is copied once S of tile t - KS is done, which the softmax warps'
// work on tile t - KS - 1 precedes, and the ring is written one tile before that copy.
struct __align__(16) Segment {
  int seq, q0, L, ctx, m, kb, ke, ib, ie, tiles, count;  // of its row tile
  int g, j0, j1;  // KV head, key tiles
  int slot;       // of its partial result, where it is not all of its pair
  int last;       // a pair's first segment that does not finish it: the run that does (-1: none)
};
constexpr int kSegRing = 8;

// The key tile that a segment takes as its j-th, j0 <= j < j1: with biases the last, whose scores are
// the largest, comes first (in the order of the keys a steep slope raises the maximum by 2^8 with
// every tile, and the output is rescaled each time: chunks of 512 over 4096 keys 374 us so, 310
// from the last).
template <Mode MODE>
__device__ __forceinline__ int tile_at(const Segment &seg, int j) {
  return has_bias(MODE) ? seg.j0 + seg.j1 - 1 - j : j;
}

__device__ __forceinline__ void fill(Segment &o, const RowTile &t) {
  o.seq = t.seq, o.q0 = t.q0, o.L = t.L, o.ctx = t.ctx, o.m = t.m;
  o.kb = t.kb, o.ke = t.ke, o.ib = t.ib, o.ie = t.ie;
  o.tiles = t.tiles, o.count = t.count;
}

// The next claim, if there is one (three dependent reads, while tiles are on their way).
__device__ __forceinline__ void claim(const Args &a, const PlanHead &h, Segment &o) {
  o.j0 = o.j1 = 0, o.last = -1;
  for (;;) {
    const int r = atomicAdd(&a.head->next, 1);
    if (r >= h.claims) return;
    const int late = r - h.whole, p = late < 0 ? r : h.whole + late / 2;
    const RowTile &any = a.tile[p / a.kv_heads];
    const Pair pair = pair_of(p, any.first, any.count, a.kv_heads);
    const RowTile t = a.tile[pair.tile];
    const bool two = late >= 0 && halved(t.tiles), second = late >= 0 && (late & 1);
    if (second && !two) continue;
    fill(o, t);
    const int half = (t.tiles + 1) / 2;
    o.g = pair.g, o.j0 = second ? half : 0, o.j1 = two && !second ? half : t.tiles;
    o.slot = late + 1;  // halves of pair q of the late ones: 2 q + 1, 2 q + 2
    return;
  }
}

struct Walk {
  long long left;  // units of the run
  int tile, g, unit, lane;
  RowTile t;
  __device__ __forceinline__ void begin(const Args &a, const Run &r) {
    left = r.units, tile = r.tile, g = r.g, unit = r.unit, lane = r.lane;
    t = a.tile[tile];
  }
  __device__ __forceinline__ void next(const Args &a, Segment &o) {
    while (left > 0) {
      const int n = t.tiles > 0 ? t.tiles + a.start : 0;
      const int end = (int)min((long long)n, unit + left);
      left -= end - unit;
      fill(o, t);
      o.g = g, o.j0 = max(unit - a.start, 0), o.j1 = max(end - a.start, 0), o.last = -1;
      // of a run: its first segment goes on with a pair, its last begins one
      o.slot = 2 * (int)blockIdx.x + (o.j0 > 0 ? 0 : 1);
      if (o.j0 == 0 && o.j1 < t.tiles) o.last = t.run_of(t.unit0 + g * t.stride + (n - 1));
      unit = 0;
      if (left > 0) {
        const int was = tile;
        if (lane) {
          ++g;
        } else if (tile + 1 < t.first + t.count) {
          ++tile;
        } else if (g + 1 < a.kv_heads) {
          tile = t.first, ++g;
        } else {
          tile = t.first + t.count, g = 0;
        }
        // not reached: the run's units are counted
        if (tile >= a.max_tiles || g >= a.kv_heads) left = 0;
        else if (tile != was) t = a.tile[tile];
      }
      if (o.j1 > o.j0) return;
    }
    o.j0 = o.j1 = 0;
  }
};

struct Shared {  // beside the tiles
  Segment ring[kSegRing];
  Walk walk;
  PlanHead head;
};

// Shared memory of one CTA (two per SM).
template <int D, bool F8>
struct Layout {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kTileKeys * 128;           // 64 keys x 64 columns of 2 bytes
  static constexpr int kRaw = kTileKeys * D;              // a tile of codes
  static constexpr int KS = F8 ? 4 : 3;                   // K ring
  static constexpr int kKSlot = F8 ? kRaw : kHalves * kHalf;
  static constexpr int VS = F8 && D == 128 ? 2 : 3;       // V ring (f16 values of an E4M3 cache)
  static constexpr int kVSlot = kHalves * kHalf;
  static constexpr int RS = F8 ? 4 : 0;                   // V codes on their way to the V ring
  static constexpr int kQ = 0;
  static constexpr int kK = kTileRows * 128;
  static constexpr int kV = kK + KS * kKSlot;
  static constexpr int kRawV = kV + VS * kVSlot;
  static constexpr int kBars = kRawV + RS * kRaw;
  static constexpr int kNumBars = 2 * KS + 2 * VS + 7 + 2 * RS + kSegRing;
  static constexpr int kMisc = kBars + kNumBars * 8;  // TMEM address, abort flag, V marks
  static constexpr int kShared = (kMisc + 32 + 15) / 16 * 16;
  static constexpr int kSmem = kShared + (int)sizeof(Shared);
  // at least 78 KB, so that no more than two CTAs share an SM (256 TMEM columns each)
  static constexpr int kSmemLaunch = kSmem > 78 * 1024 ? kSmem : 78 * 1024;
  static_assert(2 * (kSmemLaunch + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(kShared % alignof(Segment) == 0 && kBars % 8 == 0, "alignment");
  static_assert(8 + 4 * (VS > 1 ? VS : 1) <= 32, "marks");
};

// The first n bits.
__device__ __forceinline__ uint64_t bits_below(int n) {
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}
// The first n bytes of a word.
__device__ __forceinline__ uint32_t bytes_below(int n) {
  return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

// The values that were taken out of a row's products because they are not finite, added to the
// row's stored result (a bf16 row, or fp32 columns in groups of four `step` floats apart) where
// the row sees them.
template <int D, bool F8>
__device__ __noinline__ void add_odd_values(const Args &a, const Segment &seg, int lo, int hi,
                                            uint16_t *out, float *part) {
  const int origin = seg.kb & ~(kBlockSize - 1);
#pragma unroll 1
  for (int j = seg.j0; j < seg.j1; ++j) {
    const int t0 = origin + j * kTileKeys;
    if (t0 >= seg.ib && t0 + kTileKeys <= seg.ie) continue;  // these stayed
#pragma unroll 1
    for (int key = max(t0, lo); key < min(t0 + kTileKeys, hi); ++key) {
      if (key >= seg.ib && key < seg.ie) continue;
      const int at = key % kBlockSize;
      const int blk = a.block_tables[(size_t)seg.seq * a.max_blocks + key / kBlockSize];
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

template <int D, bool F8, Mode MODE>
__global__ void __launch_bounds__(threads(F8), 2)
    range_attention_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv) {
  using Lay = Layout<D, F8>;
  constexpr int H = Lay::kHalves, KS = Lay::KS, VS = Lay::VS, RS = Lay::RS;
  constexpr bool kShared = MODE == kPlain;  // shared-prefix decode
  constexpr bool kCap = has_cap(MODE), kBias = has_bias(MODE), kChanged = kCap || kBias;
  constexpr float kLift = F8 ? kLiftF8 : 0.f;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {  // the swizzled tiles need a 1024-byte aligned window
    // every CTA of the launch comes here or none does
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) {
      flag_error(a.err, PKV_DEV_LAYOUT);
      if (!kShared) a.join[blockIdx.x].parts = 0;
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
  // Marks of V values that are not finite.  E4M3: [ring slot], 1 + the number of the CTA's tile
  // that had one.  bf16: the number of the last segment that had one.
  volatile int *v_bad = abort_flag + 1;
  constexpr int kMarks = F8 ? VS : 1;
  Shared *sh = reinterpret_cast<Shared *>(smem + Lay::kShared);

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
  // Shared prefixes: the launch behind is the own keys' kernel, which reads the plan (complete before
  // this launch) and may run beside this one.
  if (!kShared) pdl_trigger();
  pdl_wait();
  if (kShared) pdl_trigger();
  // After the wait: a kernel before this one may still have to allocate its own.
  if (warp == 4) {
    alloc(smem_u32(tmem_slot), kTmemColumns);
    fence_before();
  }
  if (threadIdx.x == 0) {
    const int r = blockIdx.x;
    const PlanHead h = *a.head;
    sh->head = h;
    sh->walk.left = h.runs < 0 ? 1 : 0;
    if (r < h.runs) sh->walk.begin(a, a.run[r]);
    if (!kShared && h.runs >= 0) a.join[r].parts = 0;
  }
  __syncthreads();
  fence_after();
  if (sh->walk.left == 0) {
    __syncthreads();
    if (warp == 4) dealloc(*tmem_slot, kTmemColumns);
    return;
  }
  __syncthreads();  // everyone has seen the run's length before the K warp moves on
  const int G = a.group;
  // Columns of TMEM: S, P, the part of Q kept there, O.  A role reads what it needs of these for
  // itself: held across the split into roles, they would be spilled in all of them.
  const volatile uint32_t *tmem_at = tmem_slot;
  Segment seg;
  // The run's segment n; false: the run is over (or a wait gave up).
  auto segment = [&](int n) {
    if (!mbar_wait(seg_full + 8 * (n % kSegRing), (uint32_t)(n / kSegRing) & 1u, abort_flag, a.err))
      return false;
    seg = sh->ring[n % kSegRing];
    return seg.j1 > seg.j0;
  };

  if (warp < 4) {
    set_regs_up<Regs<F8>::softmax>();
    // ---------------- softmax warps: thread t owns row t ----------------
    const uint32_t tmem = *tmem_at;
    const uint32_t tS = tmem, tP = tmem + 64, tQ = tmem + 96, tO = tmem + 128;
    const int t = threadIdx.x;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    int jt = 0;    // tiles done (the barriers' phases)
    int nseg = 0;  // segments begun
    bool ok = true;
    while (ok && segment(nseg)) {
      ++nseg;
      const int r0 = seg.m * kTileRows, r = r0 + t, rows = seg.L * G;
      const bool valid = r < rows, live = r0 + warp * 32 < rows;
      const int i = (valid ? r : rows - 1) / G, head = seg.g * G + r % G;
      const size_t row = (size_t)(seg.q0 + i) * a.q_heads + head;
      // keys this row sees
      int lo = seg.kb, hi = seg.ke;
      const int pos = seg.ctx - seg.L + i;
      if constexpr (MODE != kPlain) {
        lo = a.key_begin ? max(a.key_begin[seg.q0 + i], 0) : 0;
        hi = a.key_end ? max(min(a.key_end[seg.q0 + i], seg.ctx), 0) : pos + 1;
      }
      float sn = a.scale, vs = a.v_scale;
      if (F8 && a.k_scales != nullptr) {
        const float ks = a.k_scales[seg.g];
        vs = a.v_scales[seg.g];
        if (t == 0 && !(ks > 0.f && vs > 0.f)) flag_error(a.err, PKV_DEV_BAD_SCALE);
        sn *= ks;
      }
      float sl = sn * 1.4426950408889634f;
      const uint4 *qrow = reinterpret_cast<const uint4 *>(a.q + row * D);
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
        // q 2^e = q1 + q2 with E4M3 terms, e putting the row's largest element in [128, 256):
        // exact for elements down to 2^-9 of the largest, to 2^-10 absolute below.  q1 goes to
        // TMEM (four codes per column), q2 to shared memory (D 64: TMEM).
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

      // Scores in base 2: with a cap c, x -> c log2(e) tanh(x / c); the bias is taken relative
      // to the row's nearest key, so that it is exact where weights are (the softmax does not
      // change): -slope (|p - t| - nearest).
      float in = sl, amp = 0.f, slope = 0.f, near = 0.f, curve = 0.f;
      float w0 = 0.f, w1 = 0.f, w2 = 0.f, w3 = 0.f;
      if constexpr (kChanged) {
        if constexpr (kCap) {
          in = fminf(sl * 0.6931471805599453f / a.cap, 1e30f);
          amp = a.cap * 1.4426950408889634f;
          // amp y P(y^2) of y = in x, by powers of x (E4M3, whose x may be large: of y)
          const float by = F8 ? 1.f : in, by2 = by * by;
          w0 = amp * by, w1 = w0 * by2, w2 = w1 * by2, w3 = w2 * by2;
          // powers that fp32 does not hold, or only as infinity, which times a score of zero is NaN:
          // the other form
          curve = w3 >= 0x1p-100f && w3 <= 0x1p100f ? a.fit.near : -1.f;
          w0 *= a.fit.c[0], w1 *= a.fit.c[1], w2 *= a.fit.c[2], w3 *= a.fit.c[3];
        }
        if constexpr (kBias) {
          slope = a.slopes[head] * 1.4426950408889634f;
          near = (float)(pos < lo ? lo - pos : pos >= hi ? pos - (hi - 1) : 0);
        }
        sl = 1.f;
      }
      float m = -INFINITY, l = 0.f;
      bool bad = false;  // a tile's V held a value not finite (E4M3)
      const int origin = seg.kb & ~(kBlockSize - 1);
      for (int j = seg.j0; j < seg.j1; ++j, ++jt) {
        const int t0 = origin + tile_at<MODE>(seg, j) * kTileKeys;
        const bool edge = t0 < seg.ib || t0 + kTileKeys > seg.ie;
        const uint64_t bits = edge ? bits_below(hi - t0) & ~bits_below(lo - t0) : ~0ull;
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
          if constexpr (kChanged) {
            auto pair = [&](int c) {
              return f32x2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
            };
            auto keep = [&](int c, uint64_t v) {
              float lo2, hi2;
              f32x2_split(v, lo2, hi2);
              x[2 * c] = __float_as_uint(lo2), x[2 * c + 1] = __float_as_uint(hi2);
            };
            // Where no key of the tile is behind the token, the distance falls by one a key: the
            // bias is added with the scores' last step (else behind it).
            const bool linear = kBias && __all_sync(kFullMask, t0 + kTileKeys - 1 <= pos);
            const float first = linear ? slope * ((float)(t0 - pos) + near) : 0.f;
            const float per = linear ? slope : 0.f;
            uint64_t off[4];  // of a pair, from the first of its eight keys on
            if constexpr (kBias)
#pragma unroll
              for (int i2 = 0; i2 < 4; ++i2) off[i2] = f32x2(per * (2 * i2), per * (2 * i2 + 1));
            auto base = [&](int c) {
              const float b = fmaf(8.f * per, (float)(c / 4), first);
              return f32x2(b, b);
            };
            if constexpr (kCap) {
              if (__builtin_expect(edge, 0)) {  // keys not seen choose nothing
#pragma unroll
                for (int c = 0; c < 64; ++c)
                  if (!((bits >> c) & 1)) x[c] = 0u;
              }
              float f0 = 0.f, f1 = 0.f;  // largest |x| of the row in this tile
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                f0 = max3(f0, fabsf(__uint_as_float(x[c])), fabsf(__uint_as_float(x[c + 1])));
                f1 = max3(f1, fabsf(__uint_as_float(x[c + 2])), fabsf(__uint_as_float(x[c + 3])));
              }
              if (!__any_sync(kFullMask, fmaxf(f0, f1) * in > curve)) {
                // y P(y^2), P of degree 3 fitted to tanh(y) / y.
                // Five multiply-adds of two scores each, two cycles each, where the other form
                // takes twelve a score for its special functions
                const uint64_t q0 = f32x2(w0, w0), q1 = f32x2(w1, w1), q2 = f32x2(w2, w2);
                const uint64_t q3 = f32x2(w3, w3);
#pragma unroll
                for (int c = 0; c < 32; c += 4) {  // four chains side by side
                  uint64_t u[4], p[4];
                  if (F8)
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2) keep(c + i2, mul_f32x2(pair(c + i2), f32x2(in, in)));
#pragma unroll
                  for (int i2 = 0; i2 < 4; ++i2) u[i2] = mul_f32x2(pair(c + i2), pair(c + i2));
#pragma unroll
                  for (int i2 = 0; i2 < 4; ++i2) p[i2] = fma_f32x2(q3, u[i2], q2);
#pragma unroll
                  for (int i2 = 0; i2 < 4; ++i2) p[i2] = fma_f32x2(p[i2], u[i2], q1);
#pragma unroll
                  for (int i2 = 0; i2 < 4; ++i2) p[i2] = fma_f32x2(p[i2], u[i2], q0);
#pragma unroll
                  for (int i2 = 0; i2 < 4; ++i2)
                    keep(c + i2, kBias ? fma_f32x2(p[i2], pair(c + i2), add_f32x2(off[i2], base(c)))
                                       : mul_f32x2(p[i2], pair(c + i2)));
                }
              } else {
                // tanh y = 1 - 2 / (1 + e^2y), off by 2^-22
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                  float d;
                  asm("rcp.approx.ftz.f32 %0, %1;"
                      : "=f"(d)
                      : "f"(1.f + ex2(__uint_as_float(x[c]) * (in * 2.885390081777927f))));
                  x[c] = __float_as_uint(fmaf(-2.f * amp, d, amp + fmaf(per, (float)c, first)));
                }
              }
            } else {
#pragma unroll
              for (int c = 0; c < 32; ++c) keep(c, fma_f32x2(pair(c), f32x2(in, in), base(c)));
            }
            if constexpr (kBias) {
              if (linear) {  // (without a cap a pass of its own is faster: 292 us, 302 in one)
                if constexpr (!kCap)
#pragma unroll
                  for (int c = 0; c < 32; ++c) keep(c, add_f32x2(off[c & 3], pair(c)));
              } else {
                const float rel = (float)(t0 - pos);
#pragma unroll
                for (int c = 0; c < 64; ++c)
                  x[c] = __float_as_uint(
                      fmaf(-slope, fabsf(rel + (float)c) - near, __uint_as_float(x[c])));
              }
            }
          }
          if (__builtin_expect(edge, 0)) {
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
            const uint64_t x2 = f32x2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
            f32x2_split(kChanged ? add_f32x2(x2, nm2) : fma_f32x2(x2, sl2, nm2), e0, e1);
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
        if (__builtin_expect(edge, 0)) {
          // V rows of keys that no row sees become zero, whatever they hold, and elements that
          // are not finite of keys that not every row sees too (E4M3: done by the V warps)
          const int slot = jt % VS;
          if (!mbar_wait(v_full + 8 * slot, (uint32_t)(jt / VS) & 1u, abort_flag, a.err)) {
            ok = false;
            break;
          }
          if (!F8) {
            const uint32_t vst = sV + slot * Lay::kVSlot;
            for (int e = t; e < kTileKeys * 8 * H; e += 128) {
              const int key = e / (8 * H), rem = e % (8 * H), at_key = t0 + key;
              const uint32_t at = vst + (rem >> 3) * Lay::kHalf + key * 128 + (rem & 7) * 16;
              if (at_key < seg.kb || at_key >= seg.ke) {
                st_shared_v4(at, make_uint4(0u, 0u, 0u, 0u));
              } else if (MODE != kPlain && (at_key < seg.ib || at_key >= seg.ie)) {
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
                  v_bad[0] = nseg;
                }
              }
            }
            fence_proxy_async();
          } else if (v_bad[slot] == jt + 1) {
            bad = true;
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
      // every warp's marks precede its last arrival on p_full, and so this product's end; the
      // next segment's follow this warp's arrival on q_full
      if (!F8) bad = v_bad[0] == nseg;
      const bool whole = seg.j0 == 0 && seg.j1 == seg.tiles;
      const float inv = l == 0.f ? 0.f : vs / l;
      float *part = nullptr;  // this row's fp32 result, where it has one
      if (whole && !kShared) {
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
          int rr = warp * 32 + (lane >> 3), tok = (r0 + rr) / G, hd = (r0 + rr) - tok * G;
#pragma unroll 1
          for (; rr < warp * 32 + 32 && r0 + rr < rows; rr += 4) {
            *reinterpret_cast<uint4 *>(
                a.out + ((size_t)(seg.q0 + tok) * a.q_heads + seg.g * G + hd) * D + 64 * half +
                8 * (lane & 7)) = ld_shared_v4(sQ + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            for (hd += 4; hd >= G; hd -= G) ++tok;
          }
          __syncwarp();
        }
      } else {
        const float lse = l == 0.f ? -INFINITY : m - kLift + log2f(l);
        const size_t slot = (size_t)seg.slot;
        if constexpr (kShared) {
          // to rows of D floats, through this warp's rows of the staging region as above; a
          // pair's first part to the rows' own storage
          const bool own = seg.j0 == 0;
          if (valid) {
            if (own)
              a.row_lse[row] = lse;
            else
              a.part_lse[slot * kTileRows + t] = lse;
          }
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * cc + lane_base, o);
            wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int i2 = 0; i2 < 4; ++i2)
                w[i2] = __float_as_uint(__uint_as_float(o[4 * c + i2]) * inv);
              st_shared_v4(sQ + t * 128 + ((c ^ (t & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
            }
            __syncwarp();
            int rr = warp * 32 + (lane >> 3), tok = (r0 + rr) / G, hd = (r0 + rr) - tok * G;
#pragma unroll 1
            for (; rr < warp * 32 + 32 && r0 + rr < rows; rr += 4) {
              float4 *to = own ? a.row_o + ((size_t)(seg.q0 + tok) * a.q_heads + seg.g * G + hd) *
                                               (D / 4)
                               : a.part_o + (slot * kTileRows + rr) * (D / 4);
              *reinterpret_cast<uint4 *>(to + 8 * cc + (lane & 7)) =
                  ld_shared_v4(sQ + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
              for (hd += 4; hd >= G; hd -= G) ++tok;
            }
            __syncwarp();
          }
        } else {
          const size_t at = slot * kTileRows;
          if (valid) a.part_lse[at + t] = lse;
          float4 *dst = a.part_o + at * (D / 4) + t;
          part = reinterpret_cast<float *>(dst);
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * cc + lane_base, o);
            wait_ld();
            if (valid)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                dst[(8 * cc + e) * kTileRows] = make_float4(
                    __uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                    __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
          }
        }
      }
      if (MODE != kPlain && __builtin_expect(bad && valid, 0))
        add_odd_values<D, F8>(a, seg, lo, hi, part ? nullptr : a.out + row * D, part);
      if (!kShared && t == 0 && seg.last >= 0) {
        // the pair goes on in the runs that follow
        a.join[blockIdx.x] = TreeJoin{seg.q0, rows, seg.g, seg.m,
                                      seg.last - (int)blockIdx.x + 1, {0, 0, 0}};
      }
    }
    fence_before();
  } else {
  set_regs_down<Regs<F8>::other>();
  if (warp == 4) {
    // ---------------- S warp: lane 0 issues S = Q K^T ----------------
    const uint32_t tmem = *tmem_at, tS = tmem, tQ = tmem + 96;
    constexpr uint32_t id = F8 ? idesc_e4m3(kTileRows, kTileKeys) : idesc(kTileRows, kTileKeys, false, false);
    int jt = 0, ok = 1;
    for (int nseg = 0; ok && segment(nseg); ++nseg) {
      if (lane == 0) ok = mbar_wait(q_full, (uint32_t)nseg & 1u, abort_flag, a.err);
      ok = __shfl_sync(kFullMask, ok, 0);  // Q is staged
      if (!ok) break;
      fence_after();
      for (int j = seg.j0; j < seg.j1; ++j, ++jt) {
        const int sb = jt % KS;
        if (lane == 0)
          ok = mbar_wait(k_full + 8 * sb, (uint32_t)(jt / KS) & 1u, abort_flag, a.err) &&
               (jt < 1 || mbar_wait(s_free, (uint32_t)(jt - 1) & 1u, abort_flag, a.err));
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
          ok = mbar_wait(p_full, (uint32_t)jt & 1u, abort_flag, a.err) &&
               mbar_wait(v_full + 8 * sb, (uint32_t)(jt / VS) & 1u, abort_flag, a.err);
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
    // Keys that one row tile reads go first from L2; those that several read stay as long as
    // any other line.
    uint64_t once, again;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
    // What this warp copies: tiles into a ring of `slots`, lane b the tile's block b.
    const int slots = F8 && is_v ? RS : is_v ? VS : KS;
    const uint32_t full = F8 && is_v ? raw_full : is_v ? v_full : k_full;
    const uint32_t empty = F8 && is_v ? raw_empty : is_v ? v_empty : k_empty;
    const uint32_t ring = F8 && is_v ? base + Lay::kRawV : is_v ? sV : sK;
    int nseg = 0;
    int aj = 0;
    // The table's entry of key tile j for this lane's block (`held`: not past the keys).  Read
    // one tile before it is looked at, so that nothing waits for the load.
    bool held = false;
    int next_blk = -1;
    auto read_block = [&](int j) {
      const int tok = (seg.kb & ~(kBlockSize - 1)) + tile_at<MODE>(seg, j) * kTileKeys +
                      lane * kBlockSize;
      held = lane < kTileBlocks && tok < seg.ke;
      if (held) next_blk = a.block_tables[(size_t)seg.seq * a.max_blocks + tok / kBlockSize];
    };
    // The next segment: the K warp finds and publishes it, both take it from the ring.
    auto advance = [&]() {
      if (!is_v && lane == 0) {
        Segment &o = sh->ring[nseg % kSegRing];
        if (!kShared && sh->head.runs < 0)
          claim(a, sh->head, o);
        else
          sh->walk.next(a, o);
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
      const uint64_t pol = seg.count > 1 ? again : once;
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
    bool ok = true;
    int jt = 0;
    for (int nseg = 0; ok && segment(nseg); ++nseg) {
      const int origin = seg.kb & ~(kBlockSize - 1);
      for (int j = seg.j0; j < seg.j1; ++j, ++jt) {
        const int slot = jt % VS, rs = jt % RS;
        const int t0 = origin + tile_at<MODE>(seg, j) * kTileKeys;
        ok = mbar_wait(raw_full + 8 * rs, (uint32_t)(jt / RS) & 1u, abort_flag, a.err) &&
             (jt < VS || mbar_wait(v_empty + 8 * slot, (uint32_t)((jt - VS) / VS) & 1u,
                                   abort_flag, a.err));
        ok = __all_sync(kFullMask, ok);
        if (!ok) break;
        // A step: 16 codes a lane, row d of block blk, to two chunks of the operand's row.  The
        // loop stays short, for the instruction cache's sake.
        constexpr int kSteps = kTileKeys * D / (16 * 128);
        const int e0 = (warp - 8) * 32 + lane;
        const uint32_t src = base + Lay::kRawV + rs * Lay::kRaw + e0 * 16;
        const uint32_t dst = sV + slot * Lay::kVSlot;
        bool hit = false;
        if (__builtin_expect(t0 < seg.ib || t0 + kTileKeys > seg.ie, 0)) {
          // codes of keys that no row sees, and NaN codes of keys that not every row sees,
          // become zero
#pragma unroll 1
          for (int it = 0; it < kSteps; ++it) {
            uint4 v = ld_shared_v4(src + it * 2048);
            int key = t0 + (it * 128 + e0) / D * kBlockSize;
            uint32_t *w = &v.x;
#pragma unroll
            for (int q = 0; q < 4; ++q, key += 4) {
              const uint32_t held = bytes_below(seg.ke - key) & ~bytes_below(seg.kb - key);
              const uint32_t all = bytes_below(seg.ie - key) & ~bytes_below(seg.ib - key);
              const uint32_t nan = MODE == kPlain ? 0u : nan_codes(w[q]) & held & ~all;
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

  __syncthreads();
  if (warp == 4) {
    fence_after();
    dealloc(*tmem_slot, kTmemColumns);
  }
}

// ---- host ---------------------------------------------------------------------------
// Workspace of a call: the plan, the runs' parts, and (shared) the rows' first parts.
struct Workspace {
  int ctas;
  int64_t max_tiles;
  size_t run_off, tile_off, before_off, tile0_off, parts_off, groups_off, join_off, lse_off,
      o_off, total;
  int64_t first_slot, first_own;  // rows of partial results before those
};
inline Workspace workspace(int head_dim, int64_t max_tiles, int64_t owners, int64_t shared_seqs,
                           int64_t shared_rows, int64_t own_rows) {
  Workspace w = {};
  w.ctas = 2 * device_sm_count();
  w.max_tiles = max_tiles;
  size_t at = 256;  // the plan's head
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return here;
  };
  w.run_off = take((size_t)w.ctas * sizeof(Run));
  w.tile_off = take((size_t)max_tiles * sizeof(RowTile));
  w.before_off = take(((size_t)max_tiles + 1) * 8);
  w.tile0_off = take(((size_t)owners + 1) * 4);
  w.parts_off = take((size_t)shared_seqs * sizeof(SeqParts));
  w.groups_off = take(shared_seqs > 0 ? ((size_t)owners + 1) * 6 * 4 : 0);
  w.join_off = take((size_t)w.ctas * sizeof(TreeJoin));
  // Partial results: (shared) the rows' first parts, the runs' slots, (shared) the own keys'.
  w.first_slot = shared_rows;
  w.first_own = shared_rows + (int64_t)w.ctas * 2 * kTileRows;
  w.lse_off = take((size_t)(w.first_own + own_rows) * 4);
  w.o_off = take((size_t)(w.first_own + own_rows) * (size_t)head_dim * 4);
  w.total = at;
  return w;
}
inline void carve(Args &a, const Workspace &w, void *workspace, int head_dim) {
  char *b = static_cast<char *>(workspace);
  a.ctas = w.ctas;
  a.max_tiles = (int)w.max_tiles;
  a.head = reinterpret_cast<PlanHead *>(b);
  a.run = reinterpret_cast<Run *>(b + w.run_off);
  a.tile = reinterpret_cast<RowTile *>(b + w.tile_off);
  a.before = reinterpret_cast<unsigned long long *>(b + w.before_off);
  a.tile0 = reinterpret_cast<int32_t *>(b + w.tile0_off);
  a.parts = reinterpret_cast<SeqParts *>(b + w.parts_off);
  a.groups = reinterpret_cast<int32_t *>(b + w.groups_off);
  a.join = reinterpret_cast<TreeJoin *>(b + w.join_off);
  a.row_lse = reinterpret_cast<float *>(b + w.lse_off);
  a.row_o = reinterpret_cast<float4 *>(b + w.o_off);
  a.part_lse = a.row_lse + w.first_slot;
  a.part_o = a.row_o + w.first_slot * (head_dim / 4);
}

// Queues the attention kernel (the plan must be queued before it).
template <int D, bool F8, Mode MODE>
int launch(Args a, cudaStream_t st) {
  using Lay = Layout<D, F8>;
  static std::atomic<int> ready[kMaxDevices];  // shared-memory opt-in and carve-out, per device
  const int r = per_device_setup(ready, [] {
    const auto kernel = range_attention_kernel<D, F8, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Lay::kSmemLaunch);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               (int)cudaSharedmemCarveoutMaxShared);
    // the register split above draws on what the kernel was compiled for
    cudaFuncAttributes at;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, kernel);
    return e == cudaSuccess && at.numRegs >= Regs<F8>::launch ? 1 : -1;
  });
  if (r <= 0) return PKV_ERR_CUDA;
  CUtensorMap tk = {}, tv = {};
  const uint64_t rows = (uint64_t)a.num_blocks * a.kv_heads * kBlockSize;
  if (!kv_tensor_map(&tk, a.k_cache, rows, D, F8 ? 1 : 2) ||
      (!F8 && !kv_tensor_map(&tv, a.v_cache, rows, D, 2)))
    return PKV_ERR_CUDA;
  // Shared prefixes: the two launches behind read the plan without waiting for this one, so the
  // plan is complete before this one starts.  (In a graph as fast as a dependent launch, calls one
  // by one 1 to 4 us slower; with both launches waiting chats take 9 us more, documents 18.)
  const auto kernel = range_attention_kernel<D, F8, MODE>;
  const dim3 grid((unsigned)a.ctas), block(threads(F8));
  const size_t smem = Lay::kSmemLaunch;
  const cudaError_t e = MODE == kPlain ? launch_behind(kernel, grid, block, smem, st, a, tk, tv)
                                       : launch_pdl(kernel, grid, block, smem, st, a, tk, tv);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace ra
}  // namespace pkv
