// The two ends of a drafted-tree step: ancestor masks and positions of the drafted tokens
// before attention, and the move of the accepted path's K/V rows after it.
//
// Masks.  Token i of a sequence's tree has parent p(i) < i (-1: the cached context).  It
// attends to itself and its ancestors, mask(i) = bit i | mask(p(i)), and stands at position
// base + depth, depth = |mask(i)| - 1.  One CTA per sequence, one thread per token, pointer
// jumping: after round k a row holds its nearest 2^k ancestors and jump(i) the next one, so
// ceil(log2(depth + 1)) rounds of  row(i) |= row(jump(i)), jump(i) = jump(jump(i))  finish
// any tree.  The bytes are a few per token; the time is the launch and two dependent reads.
//
// Commit.  A unit is one (KV head, cache, 128-byte slice of the rows) of a sequence.  A CTA
// reads the accepted rows of up to eight units, a warp each, into shared memory, waits, and
// writes them out, so a path may overlap the slots it moves to.  Latency-bound: lengths, path,
// slots and rows are dependent reads, so the rows of a warp are read in batches and the CTAs
// fit in one wave (one unit each, 200 sequences x 16 heads of an E4M3 cache were 6400 CTAs).
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kMaxWords = PKV_TREE_MAX_TOKENS / 64;

__global__ void __launch_bounds__(PKV_TREE_MAX_TOKENS)
    tree_masks_kernel(uint64_t *masks, int32_t *positions, const int32_t *parents,
                      const int32_t *query_start, const int32_t *context_lens,
                      const int32_t *position_base, int num_tokens, int W, int32_t *err) {
  extern __shared__ uint64_t rows[];  // [64 W][W], then int jump[64 W]
  int *jump = reinterpret_cast<int *>(rows + (size_t)64 * W * W);
  pdl_trigger();
  pdl_wait();
  const int s = blockIdx.x, i = threadIdx.x;
  const int q0 = query_start[s], q1 = query_start[s + 1], ctx = context_lens[s];
  const int64_t L64 = (int64_t)q1 - q0;
  if (q0 < 0 || q1 > num_tokens || L64 < 0 || L64 > 64 * W || L64 > ctx) {
    if (i == 0) flag_error(err, PKV_DEV_BAD_CONTEXT);
    return;
  }
  const int L = (int)L64;
  if (L == 0) return;
  int j = -1;
  if (i < L) {
    j = parents[q0 + i];
    if (j < -1 || j >= i) {
      flag_error(err, PKV_DEV_BAD_TREE);
      j = -1;
    }
    for (int w = 0; w < W; ++w) rows[(size_t)i * W + w] = w == (i >> 6) ? 1ull << (i & 63) : 0ull;
    jump[i] = j;
  }
  while (__syncthreads_or(j >= 0)) {
    uint64_t r[kMaxWords];
    int nj = -1;
    if (j >= 0) {
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w)
        if (w <= (j >> 6)) r[w] = rows[(size_t)j * W + w];
      nj = jump[j];
    }
    __syncthreads();
    if (j >= 0) {
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w)
        if (w <= (j >> 6)) rows[(size_t)i * W + w] |= r[w];
      jump[i] = nj;
    }
    j = nj;
  }
  for (int e = i; e < L * W; e += blockDim.x) masks[(size_t)q0 * W + e] = rows[e];
  if (positions != nullptr && i < L) {
    int depth = -1;
    for (int w = 0; w < W; ++w) depth += __popcll(rows[(size_t)i * W + w]);
    positions[q0 + i] = (position_base ? position_base[s] : ctx - L) + depth;
  }
}

struct CommitArgs {
  uint8_t *k_cache, *v_cache;
  const int64_t *slots;     // [T] slots of the drafted tokens
  const int64_t *dst_slots; // [S][A] or null (the sequence's own first slots)
  const int32_t *query_start, *accepted, *accepted_lens;
  int num_tokens, max_accept, heads, head_dim, elem;
  int slices, units;        // slices of a row; units of a sequence (2 * heads * slices)
  int per_cta;              // units of a CTA: 8, 4, 2 or 1
  int64_t num_slots;
  int v_transposed;         // E4M3 V: [D][16] within a block
  int32_t *err;
};

constexpr int kSlice = 128;         // bytes of a row in one unit
constexpr int kCommitWarps = 8, kCommitThreads = 32 * kCommitWarps;
constexpr int kCommitSmem = 64 * 1024;  // most a CTA stages when it has several units

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitArgs a) {
  extern __shared__ __align__(16) uint8_t stage[];  // [per_cta][max_accept][kSlice], slot pairs
  pdl_trigger();
  pdl_wait();
  const int s = blockIdx.x, u0 = blockIdx.y * a.per_cta;
  const int q0 = a.query_start[s], q1 = a.query_start[s + 1], n = a.accepted_lens[s];
  if (n == 0) return;
  const int64_t L = (int64_t)q1 - q0;
  if (q0 < 0 || L < 0 || q1 > a.num_tokens || n < 0 || n > a.max_accept ||
      (a.dst_slots == nullptr && n > L)) {
    if (threadIdx.x == 0) flag_error(a.err, PKV_DEV_BAD_CONTEXT);
    return;
  }
  // Source and destination slots of the accepted rows, once per CTA (-1: not moved).
  int64_t *const ss =
      reinterpret_cast<int64_t *>(stage + (size_t)a.per_cta * a.max_accept * kSlice);
  for (int r = threadIdx.x; r < n; r += kCommitThreads) {
    const int idx = a.accepted[(size_t)s * a.max_accept + r];
    int64_t src = -1, dst = -1;
    if (idx < 0 || idx >= L) {
      flag_error(a.err, PKV_DEV_BAD_ROW);
    } else {
      src = a.slots[q0 + idx];
      dst = a.dst_slots ? a.dst_slots[(size_t)s * a.max_accept + r] : a.slots[q0 + r];
      if (src >= a.num_slots || dst >= a.num_slots) {
        flag_error(a.err, PKV_DEV_BAD_SLOT);
        src = -1;
      }
    }
    ss[2 * r] = dst < 0 ? -1 : src;
    ss[2 * r + 1] = dst;
  }
  __syncthreads();
  // Warps of one unit share its rows.
  const int wpu = kCommitWarps / a.per_cta, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = warp / wpu, sub = warp % wpu, u = u0 + k;
  const bool on = u < a.units;
  const int slice = u % a.slices, hc = u / a.slices, h = hc >> 1;
  const bool is_v = (hc & 1) != 0;
  uint8_t *const cache = is_v ? a.v_cache : a.k_cache;
  uint8_t *const st = stage + (size_t)k * a.max_accept * kSlice;
  constexpr int kBatch = 4;  // rows in flight
  const bool bytes = is_v && a.v_transposed;
  // Transposed V: lane d owns head-dim rows d, d + 32, ... of the block, one byte per token.
  constexpr int kMost = 128 / 32;
  auto byte_at = [&](int64_t slot) {
    return cache + (((slot >> 4) * a.heads + h) * a.head_dim + lane) * kBlockSize + (slot & 15);
  };
  // The others: 16-byte vectors, several rows side by side.
  const int64_t row_bytes = (int64_t)a.head_dim * a.elem;
  const int lanes = row_bytes < kSlice ? (int)(row_bytes / 16) : kSlice / 16;
  const int e = lane % lanes, per = 32 / lanes, first = sub * per + lane / lanes;
  const int step = wpu * per;
  auto vec_at = [&](int64_t slot) {
    return reinterpret_cast<uint4 *>(
        cache + (((slot >> 4) * a.heads + h) * kBlockSize + (slot & 15)) * row_bytes +
        slice * kSlice + e * 16);
  };
  uint4 *const sv = reinterpret_cast<uint4 *>(st) + e;
  if (on && bytes) {
    for (int r0 = sub * kBatch; r0 < n; r0 += wpu * kBatch) {
      uint8_t v[kBatch][kMost];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (r0 + b < n && ss[2 * (r0 + b)] >= 0)
#pragma unroll
          for (int j = 0; j < kMost; ++j)
            if (32 * j < a.head_dim) v[b][j] = byte_at(ss[2 * (r0 + b)])[32 * j * kBlockSize];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (r0 + b < n && ss[2 * (r0 + b)] >= 0)
#pragma unroll
          for (int j = 0; j < kMost; ++j)
            if (32 * j < a.head_dim) st[(r0 + b) * kSlice + lane + 32 * j] = v[b][j];
    }
  } else if (on) {
    for (int r0 = first; r0 < n; r0 += step * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = r0 + b * step;
        if (r < n && ss[2 * r] >= 0) v[b] = *vec_at(ss[2 * r]);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = r0 + b * step;
        if (r < n && ss[2 * r] >= 0) sv[r * (kSlice / 16)] = v[b];
      }
    }
  }
  __syncthreads();
  if (on && bytes) {
    // four rows that fill an aligned word of the block leave as one
    auto word_at = [&](int r) {
      if (r + 3 >= n) return false;
      const int64_t dst = ss[2 * r + 1];
      bool ok = (dst & 3) == 0;
      for (int i = 0; i < 4; ++i) ok = ok && ss[2 * (r + i)] >= 0 && ss[2 * (r + i) + 1] == dst + i;
      return ok;
    };
    const int share = (n + wpu - 1) / wpu, end = min(n, (sub + 1) * share);
    for (int r = sub * share; r < end;) {
      const bool word = r + 3 < end && word_at(r);
      if (ss[2 * r] >= 0) {
        uint8_t *dst = byte_at(ss[2 * r + 1]);
        const uint8_t *src = st + r * kSlice + lane;
#pragma unroll
        for (int j = 0; j < kMost; ++j)
          if (32 * j < a.head_dim) {
            if (word)
              *reinterpret_cast<uint32_t *>(dst + 32 * j * kBlockSize) =
                  src[32 * j] | (uint32_t)src[32 * j + kSlice] << 8 |
                  (uint32_t)src[32 * j + 2 * kSlice] << 16 | (uint32_t)src[32 * j + 3 * kSlice] << 24;
            else
              dst[32 * j * kBlockSize] = src[32 * j];
          }
      }
      r += word ? 4 : 1;
    }
  } else if (on) {
    for (int r = first; r < n; r += step)
      if (ss[2 * r] >= 0) *vec_at(ss[2 * r + 1]) = sv[r * (kSlice / 16)];
  }
}

int commit_impl(void *k_cache, void *v_cache, const int64_t *slot_mapping,
                const int32_t *query_start, const int32_t *accepted, const int32_t *accepted_lens,
                const int64_t *dst_slots, int num_seqs, int num_tokens, int max_accept,
                int num_blocks, int num_kv_heads, int head_dim, int block_size, int elem,
                int32_t *err_flag, void *stream) {
  if (block_size != kBlockSize) return PKV_ERR_BLOCK_SIZE;
  if (num_seqs < 0 || num_tokens < 0 || max_accept < 0 || max_accept > PKV_TREE_MAX_TOKENS ||
      num_blocks <= 0 || num_kv_heads <= 0 || num_kv_heads > 16383 ||
      (head_dim != 64 && head_dim != 128))
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || num_tokens == 0 || max_accept == 0) return PKV_OK;
  if (!k_cache || !v_cache || !slot_mapping || !query_start || !accepted || !accepted_lens)
    return PKV_ERR_NULL;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
  CommitArgs a;
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.slots = slot_mapping;
  a.dst_slots = dst_slots;
  a.query_start = query_start;
  a.accepted = accepted;
  a.accepted_lens = accepted_lens;
  a.num_tokens = num_tokens;
  a.max_accept = max_accept;
  a.heads = num_kv_heads;
  a.head_dim = head_dim;
  a.elem = elem;
  a.num_slots = (int64_t)num_blocks * kBlockSize;
  a.v_transposed = elem == 1;
  a.err = err_flag;
  static std::atomic<int> ready[kMaxDevices];
  const int r = per_device_setup(ready, [] {
    return cudaFuncSetAttribute(tree_commit_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                PKV_TREE_MAX_TOKENS * (kSlice + 16) + kCommitSmem) == cudaSuccess
               ? 1
               : -1;
  });
  if (r <= 0) return PKV_ERR_CUDA;
  a.slices = (head_dim * elem + kSlice - 1) / kSlice;
  a.units = 2 * num_kv_heads * a.slices;
  a.per_cta = kCommitWarps;
  while (a.per_cta > 1 && (int64_t)a.per_cta * max_accept * kSlice > kCommitSmem) a.per_cta /= 2;
  const unsigned ny = (unsigned)((a.units + a.per_cta - 1) / a.per_cta);
  if (ny > 65535) return PKV_ERR_SHAPE;
  const cudaError_t e = launch_pdl(
      tree_commit_kernel, dim3((unsigned)num_seqs, ny), dim3(kCommitThreads),
      (size_t)max_accept * ((size_t)a.per_cta * kSlice + 16), (cudaStream_t)stream, a);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int paged_tree_masks(uint64_t *masks, int32_t *positions, const int32_t *parents,
                     const int32_t *query_start, const int32_t *context_lens,
                     const int32_t *position_base, int num_seqs, int num_tokens, int mask_words,
                     int32_t *err_flag, void *stream) {
  if (num_seqs < 0 || num_tokens < 0 || mask_words <= 0 || mask_words > kMaxWords)
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!masks || !parents || !query_start || !context_lens) return PKV_ERR_NULL;
  static std::atomic<int> ready[kMaxDevices];
  constexpr int kMost = 64 * kMaxWords * (kMaxWords * 8 + 4);
  const int r = per_device_setup(ready, [] {
    return cudaFuncSetAttribute(tree_masks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMost) == cudaSuccess
               ? 1
               : -1;
  });
  if (r <= 0) return PKV_ERR_CUDA;
  const cudaError_t e =
      launch_pdl(tree_masks_kernel, dim3((unsigned)num_seqs), dim3(64 * mask_words),
                 (size_t)64 * mask_words * (mask_words * 8 + 4), (cudaStream_t)stream, masks,
                 positions, parents, query_start, context_lens, position_base, num_tokens,
                 mask_words, err_flag);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int paged_tree_commit(uint16_t *k_cache, uint16_t *v_cache, const int64_t *slot_mapping,
                      const int32_t *query_start, const int32_t *accepted,
                      const int32_t *accepted_lens, const int64_t *dst_slots, int num_seqs,
                      int num_tokens, int max_accept, int num_blocks, int num_kv_heads,
                      int head_dim, int block_size, int32_t *err_flag, void *stream) {
  return commit_impl(k_cache, v_cache, slot_mapping, query_start, accepted, accepted_lens,
                     dst_slots, num_seqs, num_tokens, max_accept, num_blocks, num_kv_heads,
                     head_dim, block_size, 2, err_flag, stream);
}

int paged_tree_commit_fp8(uint8_t *k_cache, uint8_t *v_cache, const int64_t *slot_mapping,
                          const int32_t *query_start, const int32_t *accepted,
                          const int32_t *accepted_lens, const int64_t *dst_slots, int num_seqs,
                          int num_tokens, int max_accept, int num_blocks, int num_kv_heads,
                          int head_dim, int block_size, int32_t *err_flag, void *stream) {
  return commit_impl(k_cache, v_cache, slot_mapping, query_start, accepted, accepted_lens,
                     dst_slots, num_seqs, num_tokens, max_accept, num_blocks, num_kv_heads,
                     head_dim, block_size, 1, err_flag, stream);
}

}  // extern "C"
