// Attention of new tokens (decode rows and prompt chunks) whose scores are capped, biased by
// distance, and limited to a range of keys per token, over the paged cache:
//   x_t = scale q . K_t;   x_t = cap tanh(x_t / cap);   x_t -= slope_h |p - t|
//   out = sum_t exp(x_t - max x) V_t / sum_t exp(x_t - max x),   key_begin <= t < key_end
// A range per token covers a sliding window, documents packed into one prompt, and a part of the
// prompt that every token sees.  A tile of 128 rows reads the keys that some row of it sees.  The
// kernel is range_attention.cuh's; here is its plan.
#include "range_attention.cuh"

namespace pkv {
namespace ra {
namespace {

__global__ void __launch_bounds__(kPlanThreads) scored_plan_kernel(const __grid_constant__ Args a) {
  __shared__ unsigned long long scratch[33];
  __shared__ int32_t few_seqs[kPlanThreads + 1];
  __shared__ FewTiles few;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, G = a.group, threads = blockDim.x;
  // first row tile of each sequence (looked up by bisection: in shared memory where they are few)
  int32_t *const first_tile = a.num_seqs <= kPlanThreads ? few_seqs : a.tile0;
  // Row tiles of each sequence.
  int n = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < a.num_seqs; s0 += threads) {
    const int s = s0 + tid;
    unsigned long long tiles = 0;
    if (s < a.num_seqs) {
      const int q0 = a.starts[s], q1 = a.starts[s + 1], ctx = a.context_lens[s];
      const int64_t L = (int64_t)q1 - q0;
      if (q0 < 0 || L < 0 || q1 > a.num_tokens || L > ctx ||
          (int64_t)ctx > (int64_t)a.max_blocks * kBlockSize || ctx > INT_MAX - kTileKeys)
        flag_error(a.err, PKV_DEV_BAD_CONTEXT);
      else
        tiles = (unsigned long long)((L * G + kTileRows - 1) / kTileRows);
    }
    unsigned long long total;
    const unsigned long long ex = cta_scan(tiles, scratch, total);
    if (s < a.num_seqs)
      first_tile[s] = (int)min((unsigned long long)n + ex, (unsigned long long)a.max_tiles);
    // more than the tokens can give (sequences that share rows): the rest is left out
    if (n + total > (unsigned long long)a.max_tiles) {
      if (tid == 0) flag_error(a.err, PKV_DEV_BAD_CONTEXT);
      total = (unsigned long long)(a.max_tiles - n);
    }
    n += (int)total;
  }
  if (tid == 0) first_tile[a.num_seqs] = n;
  __syncthreads();
  // The keys of each row tile, eight lanes each (a tile has 128 / G tokens).
  unsigned long long sum[1] = {0}, all[1];
  int longest = 0;
  constexpr int kLanes = 8;
  const int sub = lane % kLanes;
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += threads / kLanes) {
    const int k = k0 + tid / kLanes;
    RowTile t;
    int kb = INT_MAX, ke = 0, ib = 0, ie = INT_MAX;
    if (k < n) {
      const int s = last_not_above(first_tile, a.num_seqs, k);
      t.seq = s, t.q0 = a.starts[s], t.L = a.starts[s + 1] - t.q0, t.ctx = a.context_lens[s];
      t.first = first_tile[s], t.count = first_tile[s + 1] - t.first, t.m = k - t.first;
      const int i0 = (int)((int64_t)t.m * kTileRows / G);
      const int i1 = (int)min((int64_t)t.L, ((int64_t)(t.m + 1) * kTileRows - 1) / G + 1);
#pragma unroll 4
      for (int i = i0 + sub; i < i1; i += kLanes) {
        const int lo = a.key_begin ? max(a.key_begin[t.q0 + i], 0) : 0;
        const int hi = a.key_end ? max(min(a.key_end[t.q0 + i], t.ctx), 0) : t.ctx - t.L + i + 1;
        if (lo < hi) kb = min(kb, lo), ke = max(ke, hi);
        ib = max(ib, lo), ie = min(ie, hi);
      }
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) {
      kb = min(kb, __shfl_xor_sync(kFullMask, kb, off));
      ke = max(ke, __shfl_xor_sync(kFullMask, ke, off));
      ib = max(ib, __shfl_xor_sync(kFullMask, ib, off));
      ie = min(ie, __shfl_xor_sync(kFullMask, ie, off));
    }
    if (kb >= ke) kb = ke = 0;  // no key at all: one empty tile, whose rows become zero
    t.kb = kb, t.ke = ke, t.ib = ib, t.ie = ie;
    t.tiles = max(key_tiles(kb, ke), 1);
    if (k < n && sub == 0) {
      sum[0] += t.tiles, longest = max(longest, t.tiles);
      a.tile[k] = t;
      if (k < kPlanThreads) few.tiles[k] = t.tiles, few.first[k] = t.first, few.count[k] = t.count;
    }
  }
  __syncthreads();
  // Pairs are claimed where there are two per CTA and none is longer than two thirds of a CTA's
  // share, so that they come out even.  Measured, claimed and in runs, us: chunks of 512 over 4096
  // keys, eight sequences 259 and 298, sixteen ragged ones 335 and 473; decode of 24 sequences of
  // up to 8192 keys, 32 heads 349 and 377; where a few long sequences come last (longest pair 1.2
  // shares) 420 and 387, (0.7 shares) 316 and 298.
  const int64_t pairs = (int64_t)n * a.kv_heads;
  bool claims = pairs >= 2 * (int64_t)a.ctas && pairs <= INT_MAX / 2;
  if (claims) {
    cta_scan(sum, all, scratch);
    claims = __syncthreads_and(3 * (unsigned long long)longest * (unsigned)a.ctas <=
                               2 * all[0] * (unsigned)a.kv_heads);
  }
  if (!claims) {
    plan_runs(a, n, few, scratch);
    return;
  }
  // The join's records of the last ones, which are done in halves, are known here.
  const int late = a.ctas - 1, whole = (int)pairs - late;
#pragma unroll 1
  for (int q = tid; q < a.ctas; q += threads) {
    TreeJoin j = {0, 0, 0, 0, 0, {0, 0, 0}};
    if (q < late) {
      const int p = whole + q, any = p / a.kv_heads;
      const bool is_few = n <= kPlanThreads;
      const Pair pair = pair_of(p, is_few ? few.first[any] : a.tile[any].first,
                                is_few ? few.count[any] : a.tile[any].count, a.kv_heads);
      const RowTile &t = a.tile[pair.tile];
      if (halved(t.tiles)) j = TreeJoin{t.q0, t.L * G, pair.g, t.m, 2, {0, 0, 0}};
    }
    a.join[q] = j;
  }
  if (tid == 0) *a.head = PlanHead{-1, whole + 2 * late, 0, whole};
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads) scored_join_kernel(const __grid_constant__ Args a) {
  pdl_trigger();
  pdl_wait();
  join_runs<D>(a);
}

// Row tiles that T tokens of S sequences can have.
int64_t most_tiles(int num_seqs, int num_tokens, int group) {
  const int64_t rows = (int64_t)num_tokens * group;
  return rows / kTileRows + (num_seqs < num_tokens ? num_seqs : num_tokens) + 1;
}
Workspace scored_workspace(int num_seqs, int num_tokens, int group, int head_dim) {
  return workspace(head_dim, most_tiles(num_seqs, num_tokens, group), num_seqs, 0, 0, 0);
}

template <int D, bool F8>
int launch_scored(const Args &a, cudaStream_t st) {
  const int64_t lanes = 8 * (int64_t)a.max_tiles;
  if (launch_pdl(scored_plan_kernel, dim3(1),
                 dim3(plan_threads(lanes > a.num_seqs ? lanes : a.num_seqs)), 0, st, a) != cudaSuccess)
    return PKV_ERR_CUDA;
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  const int r = cap && bias ? launch<D, F8, kCappedBiased>(a, st)
                : cap       ? launch<D, F8, kCapped>(a, st)
                : bias      ? launch<D, F8, kBiased>(a, st)
                            : launch<D, F8, kRanges>(a, st);
  if (r != PKV_OK) return r;
  return launch_pdl(scored_join_kernel<D>, dim3((unsigned)a.ctas, kMergeSplit),
                    dim3(kMergeThreads), 0, st, a) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

bool sizes_ok(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim) {
  return num_seqs >= 0 && num_seqs <= 65535 && num_tokens >= 0 && num_q_heads > 0 &&
         num_kv_heads > 0 && num_kv_heads <= 65535 && num_q_heads % num_kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128) && (int64_t)num_tokens * num_q_heads <= INT_MAX;
}

int scored_impl(uint16_t *out, const uint16_t *q, const void *k_cache, const void *v_cache,
                const int32_t *block_tables, const int32_t *context_lens,
                const int32_t *query_start, const int32_t *key_begin, const int32_t *key_end,
                const float *slopes, float cap, int num_seqs, int num_tokens,
                int max_blocks_per_seq, int num_q_heads, int num_kv_heads, int head_dim,
                int block_size, int num_blocks, float scale, bool f8, float k_scale, float v_scale,
                const float *k_scales, const float *v_scales, void *workspace,
                size_t workspace_bytes, int32_t *err_flag, void *stream) {
  if (block_size != kBlockSize) return PKV_ERR_BLOCK_SIZE;
  if (!sizes_ok(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim) ||
      max_blocks_per_seq <= 0 || num_blocks <= 0 || !(scale > 0.f) ||
      !(cap >= 0.f && cap <= PKV_SCORED_MAX_CAP) ||
      !(k_scale > 0.f) || !(v_scale > 0.f) ||
      (uint64_t)num_blocks * num_kv_heads * kBlockSize >= (1ull << 31))
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start ||
      !workspace)
    return PKV_ERR_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_ALIGN;
  Args a = {};
  a.group = num_q_heads / num_kv_heads;
  const Workspace ws = scored_workspace(num_seqs, num_tokens, a.group, head_dim);
  if (workspace_bytes < ws.total) return PKV_ERR_WORKSPACE;
  carve(a, ws, workspace, head_dim);
  a.out = out, a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
  a.block_tables = block_tables, a.context_lens = context_lens, a.starts = query_start;
  a.key_begin = key_begin, a.key_end = key_end, a.slopes = slopes;
  a.cap = cap, a.fit = tanh_fit(cap);
  a.num_seqs = num_seqs, a.num_tokens = num_tokens, a.max_blocks = max_blocks_per_seq;
  a.q_heads = num_q_heads, a.kv_heads = num_kv_heads, a.num_blocks = num_blocks;
  a.scale = (float)((double)scale * (double)k_scale);
  a.v_scale = v_scale, a.k_scales = k_scales, a.v_scales = v_scales;
  a.start = f8 ? kStartF8 : kStart;
  // no more CTAs than the longest contexts that the block table holds have runs for
  const double runs = (double)ws.max_tiles * num_kv_heads *
                      (((double)max_blocks_per_seq + kTileBlocks - 1) / kTileBlocks + a.start) / kMinRun;
  if (runs + 1. < (double)a.ctas) a.ctas = (int)runs + 1;
  a.err = err_flag;
  const cudaStream_t st = (cudaStream_t)stream;
  if (head_dim == 128) return f8 ? launch_scored<128, true>(a, st) : launch_scored<128, false>(a, st);
  return f8 ? launch_scored<64, true>(a, st) : launch_scored<64, false>(a, st);
}

}  // namespace
}  // namespace ra
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t paged_attention_scored_workspace_size(int num_seqs, int num_tokens, int num_q_heads,
                                             int num_kv_heads, int head_dim) {
  if (!ra::sizes_ok(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim)) return 0;
  return ra::scored_workspace(num_seqs, num_tokens, num_q_heads / num_kv_heads, head_dim).total;
}

int paged_attention_scored(uint16_t *out, const uint16_t *q, const uint16_t *k_cache,
                           const uint16_t *v_cache, const int32_t *block_tables,
                           const int32_t *context_lens, const int32_t *query_start,
                           const int32_t *key_begin, const int32_t *key_end, const float *slopes,
                           float cap, int num_seqs, int num_tokens, int max_blocks_per_seq,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, float scale, void *workspace, size_t workspace_bytes,
                           int32_t *err_flag, void *stream) {
  return ra::scored_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                         key_begin, key_end, slopes, cap, num_seqs, num_tokens, max_blocks_per_seq,
                         num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, false,
                         1.f, 1.f, nullptr, nullptr, workspace, workspace_bytes, err_flag, stream);
}

int paged_attention_scored_fp8(uint16_t *out, const uint16_t *q, const uint8_t *k_cache,
                               const uint8_t *v_cache, const int32_t *block_tables,
                               const int32_t *context_lens, const int32_t *query_start,
                               const int32_t *key_begin, const int32_t *key_end,
                               const float *slopes, float cap, int num_seqs, int num_tokens,
                               int max_blocks_per_seq, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, float scale,
                               float k_scale, float v_scale, const float *k_scales,
                               const float *v_scales, void *workspace, size_t workspace_bytes,
                               int32_t *err_flag, void *stream) {
  if ((k_scales == nullptr) != (v_scales == nullptr)) return PKV_ERR_NULL;
  if (k_scales != nullptr) k_scale = v_scale = 1.f;
  return ra::scored_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                         key_begin, key_end, slopes, cap, num_seqs, num_tokens, max_blocks_per_seq,
                         num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, true,
                         k_scale, v_scale, k_scales, v_scales, workspace, workspace_bytes,
                         err_flag, stream);
}

}  // extern "C"
