// Verification of drafted tokens: which of a tree's tokens the target model keeps, and the
// token that follows, from the target's probabilities and given random numbers.
//
// At a node with target row p and draft row d (the distribution its children were drawn from)
// the children are tested in index order against what is left of p:
//   r_0 = p, m_0 = 1;   child with token x accepted when  u m_j d(x) < r_j(x);
//   after a rejection   r_{j+1} = max(r_j - m_j d, 0),  m_{j+1} = sum r_{j+1}
// and the token that follows the last accepted one is drawn from r_J by its running sum.  Since
// d >= 0 the residual needs no storage: r_j = max(p - M_j d, 0) with M_j = m_0 + .. + m_{j-1}.
// Without draft rows a child is a point mass: accepted when u m_j < r_j(x), else taken out of r.
//
// A path reads p and d at the drafted tokens, and two whole rows where it ends: S V values of p
// and of d are the floor.  One cluster of CTAs runs a sequence.  CTA 0 gathers what all tests
// need at once, walks the tree, and asks the cluster for a pass over the vocabulary where a
// residual's sum is needed; every CTA follows what CTA 0 wrote, so that the barriers match
// whatever the inputs hold.
//
// Sums.  The sampled token is an integer, looked up where the running sum passes a threshold, so
// the sums must be good to far less than a token's share and must not depend on how the row is
// cut: values enter as whole numbers of 2^-43 (p - M d formed as a pair of fp32 numbers, to 2^-47
// of its terms; verify_sum.cuh), and integer sums are the same in any order.  An fp32 number becomes two such
// integers by adding a constant whose last place is the unit: seven additions a value, where
// conversions to 64-bit integers took twice the time of everything else (64 trees: 151 us).  No
// result depends on the cluster's size or on timing.
//
// What bounds it (GB300): one chain of 6, 32000 words 9.6 us, which is the host's call; 64 trees of 20,
// 131072 words, fp32 47-51 us (67 MB needed, 96 read, 23% of DRAM's rate): passes that depend on one
// another, between cluster barriers.
#include <cooperative_groups.h>

#include "pkv_common.cuh"
#include "verify_sum.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 24;
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kTwo = 0x40000000u;  // 2.f

struct VerifyArgs {
  int32_t *accepted, *accepted_lens, *next;
  const int32_t *tokens, *parents, *query_start;
  const void *p, *d;
  int64_t p_stride, d_stride;
  const float *u, *w;
  int num_tokens, max_accept, vocab;
  int32_t *err;
};

struct Command {  // from CTA 0: sum the residual of a row
  int node;       // row; -1: the sequence has nothing to do
  int last;       // 1: then draw from it
  int gone;       // rejected tokens to leave out (no draft rows)
  float mh, ml;   // M as the sum of two fp32 numbers
  float w;
};

// An entry that is not a number in [0, 2) counts as zero.
__device__ __forceinline__ float probability(float v, bool &bad) {
  if (v >= 0.f && v < 2.f) return v;
  bad = true;
  return 0.f;
}
template <typename T>
struct Row {
  static constexpr int W = 16 / (int)sizeof(T);
  const T *at;
  int vocab, skew;  // elements from the 16-byte boundary below the row's start
  __device__ __forceinline__ Row(const void *base, int64_t row, int64_t stride, int V)
      : at(static_cast<const T *>(base) + row * stride), vocab(V),
        skew((int)((reinterpret_cast<uintptr_t>(at) & 15) / sizeof(T))) {}
  static __device__ __forceinline__ float one(const T *x) {
    if constexpr (sizeof(T) == 4)
      return __ldg(reinterpret_cast<const float *>(x));
    else
      return bf16_to_f32(__ldg(reinterpret_cast<const uint16_t *>(x)));
  }
  // Vector j counts from the boundary below the row's start; it is whole.
  __device__ __forceinline__ uint4 vector(int j) const { return ld_stream_v4(at + (j * W - skew)); }
  static __device__ __forceinline__ void widen(const uint4 &x, float (&v)[W]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
  // Elements first .. first + W - 1; whole: none is outside and `first` is on a boundary.
  __device__ __forceinline__ void load(int first, bool whole, float (&v)[W]) const {
    if (whole) {
      widen(ld_stream_v4(at + first), v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        v[i] = first + i >= 0 && first + i < vocab ? one(at + first + i) : 0.f;
    }
  }
};

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads, 4) tree_verify_kernel(const VerifyArgs a) {
  constexpr int W = Row<T>::W;
  __shared__ Command cmd;                              // written by CTA 0's thread 0 in all CTAs
  __shared__ unsigned long long cta_sum[2][kMaxCluster];
  __shared__ unsigned long long warp_sum[kVerifyWarps];
  __shared__ unsigned long long scan[kVerifyWarps];
  __shared__ int s_tok[PKV_TREE_MAX_TOKENS], s_par[PKV_TREE_MAX_TOKENS];
  __shared__ float s_p[PKV_TREE_MAX_TOKENS], s_d[PKV_TREE_MAX_TOKENS], s_u[PKV_TREE_MAX_TOKENS];
  __shared__ int s_gone[PKV_TREE_MAX_TOKENS];
  __shared__ int s_path[PKV_TREE_MAX_TOKENS];
  __shared__ bool s_first[PKV_TREE_MAX_TOKENS];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int s = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cluster.barrier_arrive();  // every CTA of the cluster runs before anything is written to it
  pdl_trigger();
  pdl_wait();
  bool bad = false;
  int q0 = 0, L = 0, rounds = 0;
  // Walk of CTA 0's first warp (all lanes alike): node, next child to look at, tokens kept.
  int node = 0, child = 1, kept = 1, gone = 0;
  double mass = 1.0, M = 0.0;
  bool fresh = true;
  if (rank == 0) {
    q0 = a.query_start[s];
    const int q1 = a.query_start[s + 1];
    const int64_t n = (int64_t)q1 - q0;
    const bool ok = q0 >= 0 && n >= 0 && q1 <= a.num_tokens && n <= PKV_TREE_MAX_TOKENS;
    if (!ok && tid == 0) flag_error(a.err, PKV_DEV_BAD_CONTEXT);
    L = ok ? (int)n : 0;
    for (int i = tid; i < L; i += kVerifyThreads) {
      const int par = a.parents[q0 + i], tok = a.tokens[q0 + i];
      const float u = a.u[q0 + i];
      float pv = 0.f, dv = 1.f;
      int up = -1;
      if (i == 0) {
        if (par != -1) flag_error(a.err, PKV_DEV_BAD_TREE);
      } else if (par < 0 || par >= i) {
        flag_error(a.err, PKV_DEV_BAD_TREE);
      } else if ((unsigned)tok >= (unsigned)a.vocab) {
        flag_error(a.err, PKV_DEV_BAD_ROW);
      } else {
        up = par;
        const int64_t row = (int64_t)q0 + par;
        pv = probability(Row<T>::one(static_cast<const T *>(a.p) + row * a.p_stride + tok), bad);
        if (DRAFT)
          dv = probability(Row<T>::one(static_cast<const T *>(a.d) + row * a.d_stride + tok), bad);
      }
      s_tok[i] = tok, s_par[i] = up, s_p[i] = pv, s_d[i] = dv, s_u[i] = u;
      s_first[i] = (double)u * (double)dv < (double)pv;  // as a node's first child
    }
    if (tid == 0) s_path[0] = 0;
  }
  __syncthreads();
  cluster.barrier_wait();
  for (;;) {
    if (rank == 0 && warp == 0) {
      int last = 1;
      if (L > 0) {
        // Next child of `node` at or behind `child`, L if there is none.
        auto next_child = [&]() {
          for (int i0 = child & ~31; i0 < L; i0 += 32) {
            const int i = i0 + lane;
            const unsigned hit = __ballot_sync(kAll, i >= child && i < L && s_par[i] == node);
            if (hit) return i0 + __ffs((int)hit) - 1;
          }
          return L;
        };
        while (kept < a.max_accept) {
          const int c = next_child();
          if (c >= L) break;
          child = c + 1;
          double r = (double)s_p[c];
          bool yes;
          if (fresh) {  // nothing rejected at this node yet
            yes = s_first[c];
          } else {
            if (DRAFT) {
              r -= M * (double)s_d[c];
            } else {
              for (int k = lane; k < gone; k += 32)
                if (s_gone[k] == s_tok[c]) r = 0.0;
              r = __any_sync(kAll, r == 0.0) ? 0.0 : r;
            }
            yes = (double)s_u[c] * mass * (double)s_d[c] < r;
          }
          fresh = yes;
          if (yes) {
            if (lane == 0) s_path[kept] = c;
            ++kept;
            node = c, gone = 0, mass = 1.0, M = 0.0;
            continue;
          }
          if (DRAFT) {
            M += mass;
            last = next_child() >= L;  // else its sum decides the next test
            break;
          }
          if (r > 0.0) {
            if (lane == 0) s_gone[gone] = s_tok[c];
            ++gone;
            mass = fmax(mass - r, 0.0);
            __syncwarp();
          }
        }
      }
      __syncwarp();
      if (lane < ctas) {
        Command *to = cluster.map_shared_rank(&cmd, lane);
        const float mh = (float)M;
        to->node = L > 0 ? q0 + node : -1;
        to->last = last;
        to->gone = gone;
        to->mh = mh, to->ml = (float)(M - (double)mh);
        to->w = L > 0 ? a.w[s] : 0.f;
      }
    }
    cluster.sync();
    const Command c = cmd;
    if (c.node < 0) break;
    float mh = c.mh, ml = c.ml;
    int ngone = DRAFT ? 0 : c.gone;
    if (!DRAFT && rank != 0) {
      const int *from = cluster.map_shared_rank(s_gone, 0);
      for (int i = tid; i < ngone; i += kVerifyThreads) s_gone[i] = from[i];
    }
    __syncthreads();
    const Row<T> p(a.p, c.node, a.p_stride, a.vocab);
    const Row<T> d(DRAFT ? a.d : a.p, c.node, DRAFT ? a.d_stride : a.p_stride, a.vocab);
    const bool same = !DRAFT || d.skew == p.skew;
    // The row's 16-byte vectors (from the boundary below its start): [from, to) are this CTA's.
    const int vecs = (a.vocab + p.skew + W - 1) / W;
    const int per_cta = (vecs + ctas - 1) / ctas;
    int from = min(vecs, rank * per_cta), to = min(vecs, from + per_cta);
    auto values = [&](int j, float (&x)[W], float (&y)[W]) {
      const int first = j * W - p.skew;
      const bool whole = first >= 0 && first + W <= a.vocab;
      p.load(first, whole, x);
      if (DRAFT) d.load(first, whole && same, y);
    };
    // A vector's values, sane (nearly always: one comparison for all of them).
    auto sane = [&](float (&x)[W], float (&y)[W]) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        top = max(top, __float_as_uint(x[i]));
        if (DRAFT) top = max(top, __float_as_uint(y[i]));
      }
      if (__builtin_expect(top >= kTwo, 0)) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          x[i] = probability(x[i], bad);
          if (DRAFT) y[i] = probability(y[i], bad);
        }
      }
    };
    auto add = [&](Sum &sum, float x, float y) {
      float s = x, t = 0.f;
      if (DRAFT) residual(x, y, mh, ml, s, t);
      sum.add(s, t);
    };
    // Sums of an eighth of them a warp; then, in the CTA where the drawn token is, of an eighth of
    // the eighth that holds it, until a vector a thread is left (the same instructions again:
    // others would come from memory).
    unsigned long long total = 0, rest = 0;
    bool narrow = false, drawn = false;
    for (;;) {
      const int per_warp = (to - from + kVerifyWarps - 1) / kVerifyWarps;
      const int w0 = min(to, from + warp * per_warp), w1 = min(to, w0 + per_warp);
      unsigned long long sum = 0;
      // Vectors [f0, f1) are whole ones: read in batches.  The row's ends one at a time (so all
      // of it where d's rows lie otherwise than p's).
      const int f0 = min(w1, max(w0, p.skew ? 1 : 0));
      const int f1 = same ? max(f0, min(w1, (a.vocab + p.skew) / W)) : f0;
      int j = f0 + lane;
      constexpr int kBatch = (DRAFT ? 16 : 32) / W;  // as the registers allow
      for (; j + (kBatch - 1) * 32 < f1; j += kBatch * 32) {
        uint4 x[kBatch], y[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          x[b] = p.vector(j + 32 * b);
          if (DRAFT) y[b] = d.vector(j + 32 * b);
        }
        Sum part;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          float xs[W], ys[W];
          Row<T>::widen(x[b], xs);
          if (DRAFT) Row<T>::widen(y[b], ys);
          sane(xs, ys);
#pragma unroll
          for (int i = 0; i < W; ++i) add(part, xs[i], ys[i]);
        }
        sum += part.value();
      }
      int k0 = w0 + lane, k1 = f0;
#pragma unroll 1
      for (int r = 0; r < 3; ++r) {
#pragma unroll 1
        for (int k = k0; k < k1; k += 32) {
          float x[W], y[W];
          values(k, x, y);
          sane(x, y);
          Sum part;
#pragma unroll
          for (int i = 0; i < W; ++i) add(part, x[i], y[i]);
          sum += part.value();
        }
        k0 = r == 0 ? j : f1 + lane, k1 = r == 0 ? f1 : w1;
      }
      for (int k = lane; k < ngone; k += 32) {  // distinct: the walk drops repetitions
        const int v = (s_gone[k] + p.skew) / W;
        if (v >= w0 && v < w1) {
          Sum part;
          part.add(probability(Row<T>::one(p.at + s_gone[k]), bad), 0.f);
          sum -= part.value();
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
      if (lane == 0) warp_sum[warp] = sum;
      __syncthreads();
      if (!narrow) {
        if (tid < ctas) {
          unsigned long long t = 0;
          for (int w = 0; w < kVerifyWarps; ++w) t += warp_sum[w];
          *cluster.map_shared_rank(&cta_sum[rounds & 1][rank], tid) = t;
        }
        cluster.sync();
        const unsigned long long *sums = cta_sum[rounds & 1];
        total = 0;
        for (int k = 0; k < ctas; ++k) total += sums[k];
        ++rounds;
        if (c.last && total == 0 && (mh != 0.f || ngone != 0)) {
          mh = ml = 0.f, ngone = 0;  // nothing is left: drawn from p itself
          continue;
        }
        if (!c.last || total == 0) break;
        // The token whose running sum first passes floor(w total), w in [0, 1) to 64 bits.
        const float wf = c.w >= 0.f ? c.w : 0.f;  // also a NaN
        const unsigned long long w64 =
            wf < 1.f ? (unsigned long long)(wf * 18446744073709551616.f) : ~0ull;
        rest = __umul64hi(w64, total);
        int who = 0;
        for (; who < ctas - 1 && rest >= sums[who]; ++who) rest -= sums[who];
        drawn = who == rank;
        if (!drawn) break;
        narrow = true;
      }
      int run = 0;
      for (; run < kVerifyWarps - 1 && rest >= warp_sum[run]; ++run) rest -= warp_sum[run];
      from = min(to, from + run * per_warp), to = min(to, from + per_warp);
      if (to - from <= kVerifyThreads) break;
      __syncthreads();  // warp_sum has been read
    }
    if (!c.last) {
      mass = (double)total / (double)(1ull << kUnitBits);
      continue;
    }
    if (total == 0 && rank == 0 && tid == 0) {
      a.next[s] = -1;
      flag_error(a.err, PKV_DEV_BAD_PROB);
    }
    if (!drawn) break;
    // A vector a thread.
    const int j = from + tid;
    float x[W], y[W];
    if (j < to) {
      values(j, x, y);
      sane(x, y);
    }
    unsigned long long mine = 0, each[W];
#pragma unroll 1
    for (int i = 0; i < W; ++i) {
      const int e = j * W - p.skew + i;
      Sum one;
      bool counts = j < to && (unsigned)e < (unsigned)a.vocab;
      for (int k = 0; k < ngone; ++k) counts = counts && s_gone[k] != e;
      if (counts) add(one, x[i], y[i]);
      each[i] = one.value();
      mine += each[i];
    }
    unsigned long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long t = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += t;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    unsigned long long before = incl - mine;
    for (int w = 0; w < warp; ++w) before += scan[w];
    const bool here = rest >= before && rest - before < mine;
    // no thread's: the row sums to more than 64 bits hold
    if (!__syncthreads_or(here) && tid == 0) a.next[s] = a.vocab - 1;
    if (here) {
      rest -= before;
      int i = 0;
#pragma unroll 1
      for (; i < W - 1 && rest >= each[i]; ++i) rest -= each[i];
      a.next[s] = j * W - p.skew + i;
    }
    break;
  }
  if (bad) flag_error(a.err, PKV_DEV_BAD_PROB);
  if (rank == 0) {
    __syncthreads();
    if (L == 0) kept = 0;
    if (tid == 0) {
      a.accepted_lens[s] = kept;
      if (L == 0) a.next[s] = -1;
      scan[0] = (unsigned long long)kept;
    }
    __syncthreads();
    const int n = (int)scan[0];
    for (int i = tid; i < a.max_accept; i += kVerifyThreads)
      a.accepted[(size_t)s * a.max_accept + i] = i < n ? s_path[i] : -1;
  }
}

template <typename T, bool DRAFT>
int launch_verify(const VerifyArgs &a, int num_seqs, cudaStream_t st) {
  // as many CTAs a sequence as the GPU holds at once (four per SM)
  int ctas = kMaxCluster;
  while (ctas > 1 && (int64_t)num_seqs * ctas > 4 * device_sm_count()) ctas /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_seqs * ctas));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<T, DRAFT>, a) == cudaSuccess ? PKV_OK
                                                                                  : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int paged_tree_verify(int32_t *accepted, int32_t *accepted_lens, int32_t *next_tokens,
                                 const int32_t *tokens, const int32_t *parents,
                                 const int32_t *query_start, const void *target_probs,
                                 int64_t target_stride, const void *draft_probs,
                                 int64_t draft_stride, int prob_bytes, const float *uniforms,
                                 const float *sample_uniforms, int num_seqs, int num_tokens,
                                 int max_accept, int vocab, int32_t *err_flag, void *stream) {
  if (num_seqs < 0 || num_seqs > (1 << 24) || num_tokens < 0 || max_accept <= 0 ||
      max_accept > PKV_TREE_MAX_TOKENS || vocab <= 0 || vocab > kMaxVocab ||
      (prob_bytes != 2 && prob_bytes != 4))
    return PKV_ERR_SHAPE;
  if (num_tokens > 1 && (target_stride < vocab || (draft_probs && draft_stride < vocab)))
    return PKV_ERR_SHAPE;
  if (num_seqs == 0) return PKV_OK;
  if (!accepted || !accepted_lens || !next_tokens || !query_start || !sample_uniforms ||
      (num_tokens > 0 && (!tokens || !parents || !target_probs || !uniforms)))
    return PKV_ERR_NULL;
  const uintptr_t low = (uintptr_t)(prob_bytes - 1);
  if ((reinterpret_cast<uintptr_t>(target_probs) & low) ||
      (reinterpret_cast<uintptr_t>(draft_probs) & low))
    return PKV_ERR_ALIGN;
  VerifyArgs a;
  a.accepted = accepted, a.accepted_lens = accepted_lens, a.next = next_tokens;
  a.tokens = tokens, a.parents = parents, a.query_start = query_start;
  a.p = target_probs, a.d = draft_probs;
  a.p_stride = target_stride, a.d_stride = draft_stride;
  a.u = uniforms, a.w = sample_uniforms;
  a.num_tokens = num_tokens, a.max_accept = max_accept, a.vocab = vocab;
  a.err = err_flag;
  const cudaStream_t st = (cudaStream_t)stream;
  if (prob_bytes == 4)
    return draft_probs ? launch_verify<float, true>(a, num_seqs, st)
                       : launch_verify<float, false>(a, num_seqs, st);
  return draft_probs ? launch_verify<uint16_t, true>(a, num_seqs, st)
                     : launch_verify<uint16_t, false>(a, num_seqs, st);
}
