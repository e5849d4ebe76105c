// Decode attention of a batch in groups that share a prefix (forked samples, a common system
// prompt or document): the prefix's keys are read once for the rows of all of a group's
// sequences, each sequence's own keys by itself, and the parts joined.
//
// One token a sequence.  The rows of a group's tokens that share a KV head are the row tiles of
// the prefix: 16 sequences of 8 heads fill one, and the score and value products of
// range_attention.cuh's kernel have all their rows.  A sequence alone has 8 of 128; its own keys
// go through the decode kernel's mma.sync tiles of 8 rows (attention_mma.cu), which read short key
// ranges at memory speed where a row tile's start and finish would take as long as their keys
// (long documents: 189 us, 263 with row tiles for all keys; E4M3, head_dim 64: 63, 149; for chats under
// one prompt row tiles for all were faster: 68, 62).
#include "attention.cuh"
#include "range_attention.cuh"

namespace pkv {
namespace ra {
namespace {

// What sharing must save to be worth it: of a group, key tiles (below, the row tiles' starts take as
// long; 64 groups of 4 with 256 tokens: 85 us shared, 75 not; 8 of 16: 46, 50), and of a call, bytes
// (below, the prefixes' kernel takes longer than what it saves; 59 MB 35 us shared, 32 not; 94 MB
// in groups of 4 42, 36; 114 MB 34, 34; E4M3 57 MB 38, 32; 114 MB 40, 38; 195 MB 56, 60).
constexpr int kLeastTiles = 16, kLeastBytes = 100 << 20;
// Own keys are cut into records of half of a CTA's share, of at least 256 tokens.
constexpr int kOwnPerCta = 2, kLeastOwn = 256, kMostOwn = INT_MAX & ~31;

// The prefixes' K and V from which on a group's row tiles run side by side, in lanes: their keys
// come from DRAM once, where L2 does not hold them all; with few keys lanes cut the pairs into more
// segments than runs laid end to end do.  (bf16, us in lanes and not, one group of 4 row tiles, two of
// 2, four of 2: 8 MB 43.0 and 42.6, 35.4 and 29.1, 48.7 and 45.9; 16 MB 44.9 and 46.8, 43.2 and 42.9,
// 52.0 and 53.1; 24 MB 50.1 and 51.0, 44.4 and 45.7, 54.4 and 55.9; 96 MB 74.5 and 76.3, 61.3 and 62.4,
// 71.5 and 72.5; 0.7 GB 194 and 251; 4 row tiles of 490 MB 175 and 267.  E4M3 from 8 to 96 MB
// within 4% of each other.)
constexpr int kLaneBytes = 24 << 20;
// Rows up to which the join takes a CTA for each (512 rows of 20 parts: 34 us so, 36 with a warp a
// row; 2048: 40 and 34).
constexpr int kFewRows = 1024;

struct OwnArgs {      // the plan's lists for the own keys' kernel (attention.cuh)
  int32_t *num_items, *part_eff, *work_next;
  int4 *items;
  int capacity;       // records
  int per_token;      // work items of a record: KV heads x query sub-groups
  int slots;          // about the kernel's resident CTAs
  int first_slot, first_own;  // rows of partial results before the runs' and before these
};

// The plan's view of the groups: in shared memory where there are few.
struct Groups {
  const int32_t *starts;  // [N + 1]
  int32_t *len;           // [N] tokens of the prefix that are shared, whole blocks
  int32_t *tile0, *run0;  // [N + 1] first row tile, first run
  int N;
};

// 0 where sharing does not pay, or the group's first sequence does not hold its prefix (every
// sequence then reads all of its keys through its own table).
__device__ __forceinline__ int shared_prefix(const Args &a, const Groups &gr, int g) {
  const int s0 = gr.starts[g], n = gr.starts[g + 1] - s0, p = a.prefix_lens[g];
  const int least = a.variant == PKV_SHARED_ALWAYS ? 0 : kLeastTiles;
  if (n < 2 || p <= 0 || a.variant == PKV_SHARED_NEVER ||
      (int64_t)(n - 1) * (p / kTileKeys) < least)
    return 0;
  const int ctx = a.context_lens[s0];
  return p <= ctx && (int64_t)ctx <= (int64_t)a.max_blocks * kBlockSize ? p & ~(kBlockSize - 1) : 0;
}

// A sequence's own keys [from, to), none where its lengths are wrong.
struct OwnKeys {
  int from, to, group;
};
__device__ __forceinline__ OwnKeys own_keys(const Args &a, const Groups &gr, int s, int ctx,
                                            bool flag) {
  OwnKeys k;
  k.group = last_not_above(gr.starts, gr.N, s);
  const int given = a.prefix_lens[k.group];
  k.from = k.to = 0;
  if (ctx < 0 || given < 0 || given > ctx ||
      (int64_t)ctx > (int64_t)a.max_blocks * kBlockSize || ctx > INT_MAX - kTileKeys) {
    if (flag) flag_error(a.err, PKV_DEV_BAD_CONTEXT);
    k.group = -1;
    return k;
  }
  k.from = gr.len[k.group], k.to = ctx;
  return k;
}

// The plan: CTA 0 lists the prefixes' row tiles and runs, CTA 1 the own keys' records and what
// the join needs.  Bound by dependent reads, barriers and instructions met for the first time:
// what groups need is read once, into shared memory, and the first thousand groups and
// sequences stay in their thread's registers.
struct Prefix {
  int keys, rows;  // key tiles, row tiles (0: not shared)
};

__device__ __forceinline__ void plan_prefixes(const Args &a, const Groups &gr,
                                              unsigned long long *scratch, int *fit,
                                              FewTiles &few) {
  const int tid = threadIdx.x, N = gr.N, threads = blockDim.x;
  const unsigned H = (unsigned)a.kv_heads;
  auto prefix_of = [&](int g) {
    Prefix p = {0, 0};
    if (g < N && gr.len[g] > 0) {
      p.keys = key_tiles(0, gr.len[g]);
      p.rows = (int)(((unsigned)(gr.starts[g + 1] - gr.starts[g]) * (unsigned)a.group +
                      kTileRows - 1) / kTileRows);
    }
    return p;
  };
  auto lane_of = [&](const Prefix &p) {  // units of a row tile, all heads
    return p.rows ? (unsigned long long)H * (unsigned)(p.keys + a.start) : 0ull;
  };
  const Prefix mine = prefix_of(tid);  // of the first `threads` groups
  int n = 0;
  unsigned long long keys = 0, units = 0;
#pragma unroll 1
  for (int b = 0; b < N; b += threads) {
    const int g = b + tid;
    const Prefix p = b == 0 ? mine : prefix_of(g);
    unsigned long long v[3] = {(unsigned)p.rows, p.rows ? (unsigned)p.keys : 0u,
                               p.rows * lane_of(p)};
    unsigned long long total[3];
    cta_scan(v, total, scratch);
    if (g < N) {
      const int first = n + (int)v[0];
      gr.tile0[g] = first;
#pragma unroll 1
      for (int m = 0; m < p.rows; ++m) {
        RowTile t;
        t.seq = t.q0 = gr.starts[g], t.L = gr.starts[g + 1] - t.q0, t.ctx = 0, t.m = m;
        t.kb = t.ib = 0, t.ke = t.ie = gr.len[g], t.tiles = p.keys;
        t.first = first, t.count = p.rows;
        a.tile[first + m] = t;
        if (first + m < kPlanThreads)
          few.tiles[first + m] = p.keys, few.first[first + m] = first, few.count[first + m] = p.rows;
      }
    }
    n += (int)total[0], keys += total[1], units += total[2];
  }
  if (tid == 0) gr.tile0[N] = n;
  // Lanes, where the keys are more than L2 keeps between two row tiles' reads: run lengths from
  // the even share up are tried, by a warp each, for one with which all groups' runs fit.
  constexpr int kTried = 32;
  if (tid == 0) *fit = kTried;
  __syncthreads();
  const unsigned long long even = quotient(units, (unsigned)a.ctas) + 1;
  auto longest = [&](int i) { return even + even * i / 128; };  // up to a quarter more
  if (keys * H > (unsigned long long)a.lane_tiles) {
#pragma unroll 1
    for (int i = tid >> 5; i < kTried; i += threads >> 5) {
      unsigned long long ctas = 0;
#pragma unroll 1
      for (int g = tid & 31; g < N; g += 32) {
        const Prefix p = prefix_of(g);
        ctas += p.rows * quotient(lane_of(p) + longest(i) - 1, longest(i));
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ctas += __shfl_xor_sync(kFullMask, ctas, off);
      if (ctas <= (unsigned)a.ctas) {
        if ((tid & 31) == 0) atomicMin(fit, i);
        break;
      }
    }
  }
  __syncthreads();
  if (*fit == kTried) {
    plan_runs(a, n, few, scratch);
    return;
  }
  const unsigned long long most = longest(*fit);
  int runs = 0;
#pragma unroll 1
  for (int b = 0; b < N; b += threads) {
    const int g = b + tid;
    const Prefix p = b == 0 ? mine : prefix_of(g);
    const int cuts = (int)quotient(lane_of(p) + most - 1, most);
    unsigned long long total;
    const unsigned long long ex = cta_scan((unsigned)(p.rows * cuts), scratch, total);
    if (g < N) {
      gr.run0[g] = runs + (int)ex;
#pragma unroll 1
      for (int m = 0; m < p.rows; ++m) {
        RowTile &t = a.tile[gr.tile0[g] + m];
        t.unit0 = 0, t.stride = (unsigned)(p.keys + a.start);
        t.quot = quotient(lane_of(p), (unsigned)cuts);
        t.extra = (int)(lane_of(p) - t.quot * (unsigned)cuts);
        t.run0 = runs + (int)ex + m, t.step = p.rows;
      }
    }
    runs += (int)total;
  }
  if (tid == 0) gr.run0[N] = runs, a.head->runs = runs;
  __syncthreads();
#pragma unroll 1
  for (int r = tid; r < runs; r += threads) {  // a group's lanes side by side
    const int g = last_not_above(gr.run0, N, r);
    const Prefix p = prefix_of(g);
    const int cuts = (gr.run0[g + 1] - gr.run0[g]) / p.rows, in = r - gr.run0[g];
    const int m = in % p.rows, i = in / p.rows;
    const unsigned long long lane = lane_of(p), quot = quotient(lane, (unsigned)cuts);
    const int extra = (int)(lane - quot * (unsigned)cuts);
    const unsigned long long x = run_begin(quot, extra, i);
    const unsigned pair = (unsigned)(p.keys + a.start);
    const int head = (int)quotient(x, pair);
    a.run[r] = Run{gr.tile0[g] + m, head, (int)(x - (unsigned long long)head * pair), 1,
                   (long long)quot + (i < extra ? 1 : 0), 0};
  }
}

__device__ __forceinline__ void plan_own(const Args &a, const OwnArgs &own, const Groups &gr,
                                         unsigned long long *scratch, int *at_bin) {
  constexpr int kBins = 32;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int N = gr.N, s0 = gr.starts[0], s1 = gr.starts[N];
  // First row tile of each group, and all own keys.
  OwnKeys first_keys = {0, 0, -1};  // of the first `threads` sequences
  unsigned long long tokens = 0;
  int n = 0;
  if (tid < kBins) at_bin[tid] = 0;
#pragma unroll 1
  for (int b = 0; b < N || b < s1 - s0; b += threads) {
    const int g = b + tid, s = s0 + b + tid;
    OwnKeys k = {0, 0, -1};
    if (s < s1) k = own_keys(a, gr, s, a.context_lens[s], true);
    if (b == 0) first_keys = k;
    unsigned rows = 0;
    if (g < N && gr.len[g] > 0)
      rows = ((unsigned)(gr.starts[g + 1] - gr.starts[g]) * (unsigned)a.group + kTileRows - 1) /
             kTileRows;
    unsigned long long v[2] = {rows, (unsigned)(k.to - k.from)}, total[2];
    cta_scan(v, total, scratch);
    if (g < N) gr.tile0[g] = n + (int)v[0];
    n += (int)total[0], tokens += total[1];
  }
  // The size of a record, then the records, longest first (by 32nds of that size).
  const unsigned long long share =
      quotient(tokens * (unsigned)own.per_token, (unsigned)kOwnPerCta * (unsigned)own.slots);
  // (the most that an int holds: above, no sequence has more than one record)
  const int P = (int)(share < kLeastOwn ? (unsigned long long)kLeastOwn
                                        : min((share + 32) & ~31ull, (unsigned long long)kMostOwn));
  auto bin_of = [&](int len) {  // of a record that is not whole
    return kBins - (int)quotient((unsigned long long)len * kBins + P - 1, (unsigned)P);
  };
#pragma unroll 1
  for (int s = s0 + tid; s < s1; s += threads) {
    const OwnKeys k =
        s == s0 + tid ? first_keys : own_keys(a, gr, s, a.context_lens[s], false);
    const int len = k.to - k.from, whole = len / P, rest = len % P;
    if (whole) atomicAdd(&at_bin[0], whole);  // the first bin: as long as a record gets
    if (rest) atomicAdd(&at_bin[bin_of(rest)], 1);
  }
  __syncthreads();
  if (tid < 32) {
    const int v = at_bin[tid];
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(kFullMask, incl, off);
      if (tid >= off) incl += t;
    }
    at_bin[tid] = incl - v;
    if (tid == 31) *own.num_items = incl, *own.work_next = 0, *own.part_eff = P;
  }
#pragma unroll 1
  for (int s = tid; s < a.num_seqs; s += threads)
    if (s < s0 || s >= s1) a.parts[s].own = -1;
  unsigned long long more = 0;  // records besides the first of each sequence before
#pragma unroll 1
  for (int b = s0; b < s1; b += threads) {  // (the scan's barriers: at_bin is complete)
    const int s = b + tid;
    OwnKeys k = first_keys;
    if (b > s0 && s < s1) k = own_keys(a, gr, s, a.context_lens[s], false);
    const int len = k.to - k.from, whole = len / P, rest = len % P;
    const int parts = whole + (rest ? 1 : 0);
    unsigned long long total;
    const unsigned long long ex = cta_scan(parts > 1 ? parts - 1 : 0, scratch, total);
    if (s < s1) {
      SeqParts o = {s + (int)(more + ex), parts, 0, -1};
      if (k.from > 0) o.index = s - gr.starts[k.group], o.prefix = gr.tile0[k.group];
      // P keeps this so: there are at most tokens / P records besides a sequence's first, for which
      // the capacity has 2 slots / per_token (and none where P is kMostOwn)
      const bool fits = (int64_t)o.own + parts <= own.capacity;
      if (!fits) {
        flag_error(a.err, PKV_DEV_BAD_CONTEXT);
        o = SeqParts{0, 0, 0, -1};
      }
      a.parts[s] = o;
      // alone: straight to `out`; else result o.own + i, told by its distance from s
      auto put = [&](int at, int i) {
        const int t0 = k.from + i * P;
        if (fits && at < own.capacity)
          own.items[at] = make_int4(s, t0, t0 + min(k.to - t0, P),
                                    o.prefix < 0 && parts == 1 ? 1 : ~(o.own + i - s));
      };
      if (whole) {
        const int at = atomicAdd(&at_bin[0], whole);
#pragma unroll 1
        for (int i = 0; i < whole; ++i) put(at + i, i);
      }
      if (rest) put(atomicAdd(&at_bin[bin_of(rest)], 1), whole);
    }
    more += total;
  }
}

__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(const __grid_constant__ Args a, const __grid_constant__ OwnArgs own) {
  __shared__ unsigned long long scratch[3 * 33];
  __shared__ int fit, at_bin[32];
  __shared__ unsigned long long saved;
  __shared__ int32_t few[4][kPlanThreads + 1];
  __shared__ FewTiles few_tiles;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, threads = blockDim.x, N = a.num_groups, cta = blockIdx.x;
  // (many groups: the two CTAs' lists in the workspace, a copy each)
  const int per = N + 1;
  Groups gr = {a.starts, a.groups + (cta * 3) * per, a.groups + (cta * 3 + 1) * per,
               a.groups + (cta * 3 + 2) * per, N};
  if (N <= kPlanThreads) gr = Groups{few[0], few[1], few[2], few[3], N};
  bool bad = false;
#pragma unroll 1
  for (int g = tid; g <= N; g += threads) {
    const int x = a.starts[g];
    bad |= x < 0 || x > a.num_seqs || (g > 0 && x < a.starts[g - 1]);
    if (N <= kPlanThreads) few[0][g] = x;
  }
  if (__syncthreads_or(bad)) {  // no groups then
    if (cta == 0) {
      if (tid == 0) a.head->runs = 0;
      return;
    }
    if (tid == 0) {
      flag_error(a.err, PKV_DEV_BAD_CONTEXT);
      *own.num_items = *own.work_next = 0, *own.part_eff = kLeastOwn;
    }
#pragma unroll 1
    for (int s = tid; s < a.num_seqs; s += threads) a.parts[s].own = -1;
    return;
  }
  if (tid == 0) saved = 0;
  __syncthreads();
  unsigned long long mine = 0;
#pragma unroll 1
  for (int g = tid; g < N; g += threads) {
    const int len = shared_prefix(a, gr, g);
    gr.len[g] = len;
    mine += (unsigned long long)(gr.starts[g + 1] - gr.starts[g] - 1) * (unsigned)(len / kTileKeys);
  }
  if (mine) atomicAdd(&saved, mine);
  __syncthreads();
  if (a.variant != PKV_SHARED_ALWAYS && saved < (unsigned long long)a.least_tiles) {
#pragma unroll 1
    for (int g = tid; g < N; g += threads) gr.len[g] = 0;
  }
  __syncthreads();
  if (cta == 0)
    plan_prefixes(a, gr, scratch, &fit, few_tiles);
  else
    plan_own(a, own, gr, scratch, at_bin);
}

// Joins the parts of a row: the prefix's (the first in the rows' own storage, the others in the
// first slots of the runs that went on with it), then the own keys'.  WPR warps share a row, where
// rows are few and their parts many.  What costs is the round trips: the sequence's record, the
// row tile's, then log-sum-exps and first values at once, the values in batches.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinBatch = 4;
template <int D, int WPR>
__global__ void __launch_bounds__(kJoinThreads, 6)
    shared_join_kernel(const __grid_constant__ Args a, const __grid_constant__ OwnArgs own) {
  __shared__ float sums[kJoinWarps][2];
  __shared__ float4 outs[kJoinWarps][D / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * (kJoinWarps / WPR) + warp / WPR;
  const int s = (int)(row / a.q_heads), head = (int)(row % a.q_heads), G = a.group, g = head / G;
  // (the plan is complete before the prefixes' launch starts, and so before this one: read before
  // waiting for the launch before, past what this SM kept of a plan before)
  __threadfence();
  SeqParts sp = {-1, 0, 0, -1};
  if (row < (int64_t)a.num_seqs * a.q_heads) sp = a.parts[s];
  // in no group; written already by its one part
  const bool on = sp.own >= 0 && (sp.prefix >= 0 || sp.parts != 1);
  int np = 0, pt = 0, slot0 = 0, step = 0;
  if (on && sp.prefix >= 0) {
    const int r = sp.index * G + head % G;
    const RowTile &t = a.tile[sp.prefix + r / kTileRows];
    const unsigned long long u = t.unit0 + g * t.stride + (unsigned)a.start;
    const int from = t.run_of(u), to = t.run_of(u + (unsigned)t.tiles - 1);
    pt = r % kTileRows, step = t.step, slot0 = 2 * from;
    np = (to - from) / step + 1;
  }
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = D / 4, kSide = 32 / kLanes;  // rows' lanes; parts side by side
  const int side = lane / kLanes;
  const float4 *const values = a.row_o + lane % kLanes;
  // this warp's share of the parts
  const int all = on ? np + sp.parts : 0, each = (all + WPR - 1) / WPR;
  const int begin = min(all, warp % WPR * each), parts = min(all, begin + each);
  float m = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // what is not finite stays where its weight vanishes
  auto odd = [](float e) { return fabsf(e) < INFINITY ? 0.f : e; };
  auto add = [&](float w, const float4 &v) {
    if (w != 0.f)
      o = make_float4(fmaf(w, v.x, o.x), fmaf(w, v.y, o.y), fmaf(w, v.z, o.z), fmaf(w, v.w, o.w));
    else
      o = make_float4(o.x + odd(v.x), o.y + odd(v.y), o.z + odd(v.z), o.w + odd(v.w));
  };
  auto rescale = [&](float top) {  // to the reference 2^top
    const float ref = top == -INFINITY ? 0.f : top, shrink = exp2f(m - ref);
    const float4 was = o;
    m = top;
    L *= shrink;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    add(shrink, was);
    return ref;
  };
  for (int k0 = begin; k0 < parts; k0 += 32) {
    const int n = min(32, parts - k0), k = k0 + lane;
    // lane i: the row of part k0 + i, its log-sum-exp, then its weight
    int at = 0;
    float x = -INFINITY;
    if (lane < n) {
      at = k >= np ? own.first_own + (sp.own + k - np) * a.q_heads + head
           : k == 0 ? (int)row : own.first_slot + (slot0 + 2 * step * k) * kTileRows + pt;
      x = __ldcg(a.row_lse + at);
    }
    float4 v[kJoinBatch];
    auto load = [&](int i) {
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        const int p = i + u * kSide + side, r = __shfl_sync(kFullMask, at, p & 31);
        if (p < n) v[u] = __ldcg(values + (size_t)r * kLanes);
      }
    };
    load(0);
    float top = x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
    const float ref = rescale(fmaxf(m, top));
    const float w = exp2f(x - ref);
    float sum = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
    L += sum;
    for (int i = 0; i < n; i += kJoinBatch * kSide) {
      if (i > 0) load(i);
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        const int p = i + u * kSide + side;
        const float wp = __shfl_sync(kFullMask, w, p & 31), xp = __shfl_sync(kFullMask, x, p & 31);
        if (p < n && xp != -INFINITY) add(wp, v[u]);
      }
    }
  }
  if (kSide == 2) {
    o.x += __shfl_xor_sync(kFullMask, o.x, 16);
    o.y += __shfl_xor_sync(kFullMask, o.y, 16);
    o.z += __shfl_xor_sync(kFullMask, o.z, 16);
    o.w += __shfl_xor_sync(kFullMask, o.w, 16);
  }
  if constexpr (WPR > 1) {
    if (lane < kLanes) outs[warp][lane] = o;
    if (lane == 0) sums[warp][0] = m, sums[warp][1] = L;
    __syncthreads();
    if (warp % WPR != 0) return;
    float top = m;
#pragma unroll
    for (int w = 1; w < WPR; ++w) top = fmaxf(top, sums[warp + w][0]);
    const float ref = rescale(top);
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      const float x = sums[warp + w][0], f = exp2f(x - ref);
      L = fmaf(sums[warp + w][1], f, L);
      if (x != -INFINITY) add(f, outs[warp + w][lane % kLanes]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  if (on && lane < kLanes)
    *reinterpret_cast<uint2 *>(a.out + (size_t)row * D + 4 * lane) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

// The workspace: range_attention.cuh's, then the own keys' lists and partial results.
struct SharedWorkspace {
  Workspace w;
  int per_token, slots, capacity;
  size_t counts_off, items_off, total;
};
SharedWorkspace shared_workspace(int num_seqs, int num_groups, int num_q_heads, int group,
                                 int head_dim) {
  SharedWorkspace s;
  const int64_t tiles = (int64_t)num_seqs * group / kTileRows + num_groups + 1;
  s.per_token = num_q_heads / group * ((group + 7) / 8);
  s.slots = 4 * device_sm_count();
  // a record's size keeps those besides each sequence's first within this
  s.capacity = num_seqs + kOwnPerCta * s.slots / s.per_token + 1;
  s.w = workspace(head_dim, tiles, num_groups, num_seqs, (int64_t)num_seqs * num_q_heads,
                  (int64_t)s.capacity * num_q_heads);
  size_t at = s.w.total;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return here;
  };
  s.counts_off = take(256 * 2);
  s.items_off = take((size_t)s.capacity * sizeof(int4));
  s.total = at;
  return s;
}

template <int D, bool F8>
int launch_shared(const Args &a, const OwnArgs &own, const AttnArgs &d, cudaStream_t st) {
  const unsigned threads = plan_threads(a.num_seqs > a.num_groups ? a.num_seqs : a.num_groups);
  if (launch_pdl(shared_plan_kernel, dim3(2), dim3(threads), 0, st, a, own) != cudaSuccess)
    return PKV_ERR_CUDA;
  const int r = launch<D, F8, kPlain>(a, st);
  if (r != PKV_OK) return r;
  if (launch_attn_mma(d, D, st) != cudaSuccess) return PKV_ERR_CUDA;
  const int64_t rows = (int64_t)a.num_seqs * a.q_heads;
  const int wpr = rows <= kFewRows ? kJoinWarps : 1;
  const unsigned grid = (unsigned)((rows * wpr + kJoinWarps - 1) / kJoinWarps);
  const auto join = wpr > 1 ? shared_join_kernel<D, kJoinWarps> : shared_join_kernel<D, 1>;
  return launch_pdl(join, dim3(grid), dim3(kJoinThreads), 0, st, a, own) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

std::atomic<int> g_variant{PKV_SHARED_AUTO};

bool sizes_ok(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim) {
  return num_seqs >= 0 && num_seqs <= 65535 && num_groups >= 0 && num_groups <= 65535 &&
         num_q_heads > 0 && num_kv_heads > 0 && num_kv_heads <= 65535 &&
         num_q_heads % num_kv_heads == 0 && (head_dim == 64 || head_dim == 128) &&
         (int64_t)num_seqs * num_q_heads <= INT_MAX / 8 &&  // (rows of partial results, twice and more)
         // row tiles x KV heads
         ((int64_t)num_seqs * (num_q_heads / num_kv_heads) / kTileRows + num_groups + 1) *
                 num_kv_heads <= INT_MAX / 2;
}

int shared_impl(uint16_t *out, const uint16_t *q, const void *k_cache, const void *v_cache,
                const int32_t *block_tables, const int32_t *context_lens,
                const int32_t *group_start, const int32_t *prefix_lens, int num_groups,
                int num_seqs, int max_blocks_per_seq, int num_q_heads, int num_kv_heads,
                int head_dim, int block_size, int num_blocks, float scale, bool f8, float k_scale,
                float v_scale, const float *k_scales, const float *v_scales, void *workspace,
                size_t workspace_bytes, int32_t *err_flag, void *stream) {
  if (block_size != kBlockSize) return PKV_ERR_BLOCK_SIZE;
  if (!sizes_ok(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim) ||
      max_blocks_per_seq <= 0 || num_blocks <= 0 || !(scale > 0.f) || !(k_scale > 0.f) ||
      !(v_scale > 0.f) || (uint64_t)num_blocks * num_kv_heads * kBlockSize >= (1ull << 31))
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || num_groups == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !group_start ||
      !prefix_lens || !workspace)
    return PKV_ERR_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_ALIGN;
  Args a = {};
  a.group = num_q_heads / num_kv_heads;
  const SharedWorkspace ws =
      shared_workspace(num_seqs, num_groups, num_q_heads, a.group, head_dim);
  if (workspace_bytes < ws.total) return PKV_ERR_WORKSPACE;
  carve(a, ws.w, workspace, head_dim);
  a.out = out, a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
  a.block_tables = block_tables, a.context_lens = context_lens, a.starts = group_start;
  a.prefix_lens = prefix_lens, a.num_groups = num_groups;
  a.num_seqs = a.num_tokens = num_seqs, a.max_blocks = max_blocks_per_seq;
  a.q_heads = num_q_heads, a.kv_heads = num_kv_heads, a.num_blocks = num_blocks;
  a.scale = (float)((double)scale * (double)k_scale);
  a.v_scale = v_scale, a.k_scales = k_scales, a.v_scales = v_scales;
  a.start = f8 ? kStartF8 : kStart;
  const int tile_bytes = 2 * kTileKeys * head_dim * (f8 ? 1 : 2);
  a.lane_tiles = kLaneBytes / tile_bytes;
  a.least_tiles = kLeastBytes / tile_bytes / num_kv_heads;
  a.variant = g_variant.load(std::memory_order_relaxed);
  a.err = err_flag;
  char *b = static_cast<char *>(workspace);
  OwnArgs own;
  own.num_items = reinterpret_cast<int32_t *>(b + ws.counts_off);
  own.part_eff = own.num_items + 1;
  own.work_next = own.num_items + 64;  // a line of its own: every CTA claims from it
  own.items = reinterpret_cast<int4 *>(b + ws.items_off);
  own.capacity = ws.capacity, own.per_token = ws.per_token, own.slots = ws.slots;
  own.first_slot = (int)ws.w.first_slot, own.first_own = (int)ws.w.first_own;
  AttnArgs d = {};
  d.beside = 1;
  d.out = out, d.q = q, d.k_cache = k_cache, d.v_cache = v_cache;
  d.block_tables = block_tables, d.context_lens = context_lens;
  d.num_seqs = ws.capacity, d.max_parts = 1;  // (sizes the launch; one result per record)
  d.max_blocks = max_blocks_per_seq;
  d.num_q_heads = num_q_heads, d.num_kv_heads = num_kv_heads, d.group = a.group;
  d.num_blocks = num_blocks, d.sub_groups = (a.group + 7) / 8;
  d.scale_log2 = (float)((double)scale * (double)k_scale * 1.4426950408889634);
  d.v_scale = v_scale, d.kv8 = f8 ? 1 : 0, d.k_scales = k_scales, d.v_scales = v_scales;
  d.num_items = own.num_items, d.part_eff = own.part_eff, d.work_next = own.work_next;
  d.items = own.items, d.part_lse = a.row_lse + ws.w.first_own;
  d.part_o = reinterpret_cast<float *>(a.row_o + ws.w.first_own * (head_dim / 4));
  d.err = err_flag;
  const cudaStream_t st = (cudaStream_t)stream;
  if (head_dim == 128)
    return f8 ? launch_shared<128, true>(a, own, d, st) : launch_shared<128, false>(a, own, d, st);
  return f8 ? launch_shared<64, true>(a, own, d, st) : launch_shared<64, false>(a, own, d, st);
}

}  // namespace
}  // namespace ra
}  // namespace pkv

using namespace pkv;

extern "C" {

int paged_attention_shared_set_variant(int variant) {
  if (variant != PKV_SHARED_AUTO && variant != PKV_SHARED_ALWAYS && variant != PKV_SHARED_NEVER)
    return PKV_ERR_ARG;
  return ra::g_variant.exchange(variant);
}

size_t paged_attention_shared_workspace_size(int num_seqs, int num_groups, int num_q_heads,
                                             int num_kv_heads, int head_dim) {
  if (!ra::sizes_ok(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim)) return 0;
  return ra::shared_workspace(num_seqs, num_groups, num_q_heads, num_q_heads / num_kv_heads,
                              head_dim).total;
}

int paged_attention_shared(uint16_t *out, const uint16_t *q, const uint16_t *k_cache,
                           const uint16_t *v_cache, const int32_t *block_tables,
                           const int32_t *context_lens, const int32_t *group_start,
                           const int32_t *prefix_lens, int num_groups, int num_seqs,
                           int max_blocks_per_seq, int num_q_heads, int num_kv_heads,
                           int head_dim, int block_size, int num_blocks, float scale,
                           void *workspace, size_t workspace_bytes, int32_t *err_flag,
                           void *stream) {
  return ra::shared_impl(out, q, k_cache, v_cache, block_tables, context_lens, group_start,
                         prefix_lens, num_groups, num_seqs, max_blocks_per_seq, num_q_heads,
                         num_kv_heads, head_dim, block_size, num_blocks, scale, false, 1.f, 1.f,
                         nullptr, nullptr, workspace, workspace_bytes, err_flag, stream);
}

int paged_attention_shared_fp8(uint16_t *out, const uint16_t *q, const uint8_t *k_cache,
                               const uint8_t *v_cache, const int32_t *block_tables,
                               const int32_t *context_lens, const int32_t *group_start,
                               const int32_t *prefix_lens, int num_groups, int num_seqs,
                               int max_blocks_per_seq, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, float scale,
                               float k_scale, float v_scale, const float *k_scales,
                               const float *v_scales, void *workspace, size_t workspace_bytes,
                               int32_t *err_flag, void *stream) {
  if ((k_scales == nullptr) != (v_scales == nullptr)) return PKV_ERR_NULL;
  if (k_scales != nullptr) k_scale = v_scale = 1.f;
  return ra::shared_impl(out, q, k_cache, v_cache, block_tables, context_lens, group_start,
                         prefix_lens, num_groups, num_seqs, max_blocks_per_seq, num_q_heads,
                         num_kv_heads, head_dim, block_size, num_blocks, scale, true, k_scale,
                         v_scale, k_scales, v_scales, workspace, workspace_bytes, err_flag, stream);
}

}  // extern "C"
