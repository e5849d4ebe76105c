// Attention of a tree of drafted tokens over the paged cache.
//
// Sequence s has L drafted tokens, the last L of its context_lens[s] cached tokens.  Token i
// sees every cached token before the tree and the tree tokens its mask row names:
//   x_t = scale q . K_t,   out = sum_t exp(x_t - max x) V_t / sum_t exp(x_t - max x)
// over those t; a token that sees nothing gives zeros.  A masked K or V row takes no part
// whatever it holds.
//
// One warp per (drafted token, query head) walks the keys with a running maximum and sum.
#include <math.h>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>

#include "pkv_common.cuh"

namespace pkv {
namespace {

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
  float scale;
  float k_scale, v_scale;
  const float *k_scales, *v_scales;  // [Hkv] or null
  int32_t *err;
};

__device__ __forceinline__ float e4m3(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

template <int D, bool F8>
__global__ void __launch_bounds__(256) tree_simple_kernel(const TreeArgs a) {
  constexpr int PER = D / 32;
  pdl_trigger();
  pdl_wait();
  const int s = blockIdx.z, lane = threadIdx.x & 31;
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int q0 = a.query_start[s], q1 = a.query_start[s + 1], ctx = a.context_lens[s];
  const int64_t L = (int64_t)q1 - q0;
  if (q0 < 0 || L < 0 || q1 > a.num_tokens || L > a.max_query_len || L > ctx ||
      (int64_t)ctx > (int64_t)a.max_blocks * kBlockSize) {
    if (threadIdx.x == 0) flag_error(a.err, PKV_DEV_BAD_CONTEXT);
    return;
  }
  const int i = w / a.q_heads, h = w - i * a.q_heads, g = h / a.group;
  if (i >= L) return;
  float ks = a.k_scale, vs = a.v_scale;
  if (F8 && a.k_scales) {
    ks = a.k_scales[g], vs = a.v_scales[g];
    if (!(ks > 0.f) || !(vs > 0.f)) flag_error(a.err, PKV_DEV_BAD_SCALE);
  }
  const size_t row = ((size_t)(q0 + i) * a.q_heads + h) * D;
  float q[PER], acc[PER];
  for (int e = 0; e < PER; ++e) {
    q[e] = bf16_to_f32(a.q[row + lane + 32 * e]);
    acc[e] = 0.f;
  }
  const uint64_t *mask = a.masks + (size_t)(q0 + i) * a.words;
  const int32_t *bt = a.block_tables + (size_t)s * a.max_blocks;
  const int first = ctx - (int)L;
  float m = -INFINITY, l = 0.f;
  bool any = false;
  for (int t = 0; t < ctx; ++t) {
    const int j = t - first;
    if (j >= 0 && !((mask[j >> 6] >> (j & 63)) & 1)) continue;
    const int blk = bt[t >> 4];
    if ((unsigned)blk >= (unsigned)a.num_blocks) {
      if (lane == 0) flag_error(a.err, PKV_DEV_BAD_BLOCK);
      continue;
    }
    const size_t base = ((size_t)blk * a.kv_heads + g) * (kBlockSize * D);
    float k[PER], v[PER], x = 0.f;
    for (int e = 0; e < PER; ++e) {
      const int d = lane + 32 * e;
      if (F8) {
        k[e] = e4m3(static_cast<const uint8_t *>(a.k_cache)[base + (t & 15) * D + d]) * ks;
        v[e] = e4m3(static_cast<const uint8_t *>(a.v_cache)[base + d * kBlockSize + (t & 15)]) * vs;
      } else {
        k[e] = bf16_to_f32(static_cast<const uint16_t *>(a.k_cache)[base + (t & 15) * D + d]);
        v[e] = bf16_to_f32(static_cast<const uint16_t *>(a.v_cache)[base + (t & 15) * D + d]);
      }
      x = fmaf(q[e], k[e], x);
    }
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x *= a.scale;
    any = true;
    const float mn = fmaxf(m, x);
    const float c = m == -INFINITY ? 0.f : expf(m - mn), p = expf(x - mn);
    m = mn;
    l = fmaf(l, c, p);
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(acc[e], c, p * v[e]);
  }
  for (int e = 0; e < PER; ++e)
    a.out[row + lane + 32 * e] = f32_to_bf16(any ? acc[e] / l : 0.f);
}

size_t tree_workspace(int q_heads, int kv_heads, int head_dim, int max_query_len) {
  const int64_t rows = (int64_t)max_query_len * (q_heads / kv_heads);
  const int64_t ctas = 2 * device_sm_count() + (rows + 127) / 128;
  return (size_t)(ctas * 2 * 128 * (head_dim + 2) * 4 + 256);
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
  if (workspace_bytes < tree_workspace(num_q_heads, num_kv_heads, head_dim, max_query_len))
    return PKV_ERR_WORKSPACE;
  TreeArgs a;
  a.out = out, a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
  a.block_tables = block_tables, a.context_lens = context_lens, a.query_start = query_start;
  a.masks = masks;
  a.num_seqs = num_seqs, a.num_tokens = num_tokens, a.max_blocks = max_blocks_per_seq;
  a.q_heads = num_q_heads, a.kv_heads = num_kv_heads, a.group = num_q_heads / num_kv_heads;
  a.num_blocks = num_blocks, a.words = mask_words, a.max_query_len = max_query_len;
  a.scale = scale, a.k_scale = k_scale, a.v_scale = v_scale;
  a.k_scales = k_scales, a.v_scales = v_scales;
  a.err = err_flag;
  const dim3 grid((unsigned)(((int64_t)max_query_len * num_q_heads + 7) / 8), 1,
                  (unsigned)num_seqs);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (head_dim == 128)
    e = f8 ? launch_pdl(tree_simple_kernel<128, true>, grid, dim3(256), 0, st, a)
           : launch_pdl(tree_simple_kernel<128, false>, grid, dim3(256), 0, st, a);
  else
    e = f8 ? launch_pdl(tree_simple_kernel<64, true>, grid, dim3(256), 0, st, a)
           : launch_pdl(tree_simple_kernel<64, false>, grid, dim3(256), 0, st, a);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t paged_attention_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim,
                                           int max_query_len) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      head_dim <= 0 || max_query_len < 0)
    return 0;
  return tree_workspace(num_q_heads, num_kv_heads, head_dim, max_query_len);
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
