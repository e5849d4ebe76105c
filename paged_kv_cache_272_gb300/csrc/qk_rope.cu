// Head-wise RMS norm of q and k, rotary positions, and the paged write of k and v, in one
// pass over a step's projections.
//
//   y = x / sqrt(mean(x^2) + eps) * w                    (per head; only with weights)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = pos[axis(i)] * inv_freq[i]
// for rotary pair i of the first rotary_dim elements: (y[i], y[i + rotary_dim / 2]), or
// (y[2 i], y[2 i + 1]) when interleaved.  All of it in fp32 with one rounding at the store
// (bf16, or the E4M3 code of value / scale).  v is stored as it is.
//
// Angles: a turn count t / 2 pi needs its fraction only, so a frequency w is held as a 64-bit
// fixed-point fraction of a turn per position and multiplied by the 32-bit position modulo
// 2^64.  The fraction is within 2^-64 (its truncation) + w 2^-72 (that of the 64 bits of 2 / pi)
// of a turn, the product of any position within 2^-33 + w 2^-41 -- where an fp32 product would
// be 0.06 rad off at a million.  Its top 32 bits, rounded to a float (2^-26 of a turn at most),
// go to sincospi.
//
// Layout: D / 8 lanes own a (token, head) row.  A rotating lane holds four elements of each
// half (half-split pairs) or four adjacent pairs, so both elements of a pair meet in one lane
// and nothing is exchanged but the norm's sum; its four sines stay in registers for all the
// heads it serves.  Two rows are in flight behind the one being worked on.
//
// Bound: for prompts latency at this occupancy (16384 tokens of head_dim 64: DRAM 49% busy, 2.3 of
// 4 instructions issued a cycle, 45% of the warps resident), 1.36 times the bytes' time; hence the
// rows in flight, the packed arithmetic and the division below.  E4M3 (16384 tokens, 64/8 heads of
// 128: 149 us for 94 of bytes) has V's codes besides, stored a byte at a time into the transposed
// blocks.
#include <math.h>

#include <cstring>

#include "kv_rows.cuh"
#include "pkv_common.cuh"
#include "tc_common.cuh"  // packed f32x2 arithmetic

namespace pkv {
namespace {

constexpr int kMaxAxes = 4;
constexpr int kMaxPairs = 64;
// 128 threads, eight CTAs per SM, two tokens each: a prompt of 16384 tokens (head_dim 64) takes
// 40.7 us; with four tokens 43.2, with 256 threads and four CTAs 43.5 (four tokens) or 47.8
// (two), and 53 when CTAs stay and take tile after tile.
constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 8;
constexpr int kMaxTile = 2;

// w / 2 pi of a turn per position, modulo one turn, as a fraction of 2^64.  w = m 2^(E - 1075);
// m times 2^66 / 2 pi (an integer to 2^-64 of itself) is shifted into place.  In integers,
// since the fp64 units are few.
__device__ __forceinline__ uint64_t turns_per_position(double w) {
  const uint64_t bits = (uint64_t)__double_as_longlong(w);
  const int E = (int)(bits >> 52) & 0x7ff, s = 1077 - E;
  const uint64_t m = E ? (bits & 0xfffffffffffffull) | 0x10000000000000ull : 0;
  const uint64_t k = 0xa2f9836e4e44152aull;
  const uint64_t hi = __umul64hi(m, k), lo = m * k;
  uint64_t f = s >= 128 ? 0 : s >= 64 ? hi >> (s - 64) : s > 0 ? (hi << (64 - s)) | (lo >> s) : lo;
  return bits >> 63 ? 0 - f : f;
}

struct RopeArgs {
  uint16_t *q_out;
  const uint16_t *q, *k, *v;
  int64_t q_out_stride, q_stride, k_stride, v_stride;  // elements between tokens
  const uint16_t *q_weight, *k_weight;                 // [D] or null
  float eps;
  const int32_t *positions;
  int64_t axis_stride;
  const double *inv_freq;
  int pairs;                 // rotary_dim / 2
  int interleaved;
  float rope_scale;
  const int64_t *slots;
  int num_tokens, q_heads, kv_heads;
  int64_t num_slots;
  void *k_cache, *v_cache;
  float k_scale, v_scale;
  const float *k_scales, *v_scales;
  int tile;                  // tokens per CTA (1 or 2)
  int chunk;                 // rows (q, k and v heads) per CTA
  int32_t *err;
  uint8_t pair_axis[kMaxPairs];
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ uint64_t bf16x2_to_f32x2(uint32_t w) { return f32x2(bf16_lo(w), bf16_hi(w)); }

// x / s rounded to nearest for a whole row by one reciprocal: with y = RN(1 / s), q = RN(x y)
// and the exact remainder r = x - q s, RN(q + r y) is the rounded quotient (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34, 1990), as long as nothing over- or underflows on the way: a scale within 2^+-60
// here, and quotients beyond 2^20 keep q (their code is that of the largest value either
// way); quotients that underflow have code 0.  Other scales divide.
struct RowDivide {
  float s, y;
  bool exact;
  __device__ explicit RowDivide(float scale) : s(scale), y(1.0f / scale) {
    exact = scale > 8.7e-19f && scale < 1.1e18f;
  }
  __device__ float2 operator()(float a, float b) const {
    if (!exact) return make_float2(__fdiv_rn(a, s), __fdiv_rn(b, s));
    const uint64_t x = f32x2(a, b), y2 = f32x2(y, y);
    const uint64_t q = mul_f32x2(x, y2);
    const uint64_t r = fma_f32x2(q, f32x2(-s, -s), x);
    const uint64_t z = fma_f32x2(r, y2, q);
    float q0, q1, z0, z1;
    f32x2_split(q, q0, q1);
    f32x2_split(z, z0, z1);
    auto pick = [](float big, float quot) {
      // a zero keeps the sign of the product (the correction's is always +0)
      const uint32_t z = __float_as_uint(quot) | (__float_as_uint(big) & 0x80000000u);
      return fabsf(big) > 1048576.f ? big : __uint_as_float(z);
    };
    return make_float2(pick(q0, z0), pick(q1, z1));
  }
  // Codes of four values, lowest byte first.
  __device__ uint32_t codes(float a, float b, float c, float d) const {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2((*this)(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2((*this)(c, d), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xffffu) | (hi << 16);
  }
};

template <int D, bool F8, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    qk_norm_rope_write_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8;
  constexpr int GROUPS = kRopeThreads / LPR;
  __shared__ __align__(16) float s_cos[kMaxTile][kMaxPairs], s_sin[kMaxTile][kMaxPairs];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, tile = a.tile;
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int e = tid % LPR, grp = tid / LPR;
  const int tt = grp % tile;
  const int64_t t = t0 + tt;
  const bool on = t < a.num_tokens;
  // This lane's elements of a q or k row: four from oa, four from ob.
  const int rot_lanes = a.pairs / 4;  // lanes whose elements rotate
  const bool rotates = e < rot_lanes;
  const int oa = INTER || !rotates ? 8 * e : 4 * e;
  const int ob = INTER || !rotates ? 8 * e + 4 : a.pairs + 4 * e;
  const int rows = a.q_heads + 2 * a.kv_heads, v_rows = a.q_heads + a.kv_heads;
  const int r_end = on ? min(rows, ((int)blockIdx.y + 1) * a.chunk) : 0, step = GROUPS / tile;
  const int r_begin = blockIdx.y * a.chunk + grp / tile;
  const uint16_t *const q_row = a.q + t * a.q_stride;
  const uint16_t *const k_row = a.k + t * a.k_stride - (int64_t)a.q_heads * D;
  const uint16_t *const v_row = a.v + t * a.v_stride - (int64_t)v_rows * D;
  auto load = [&](int r) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r >= r_end) return v;
    const uint16_t *p = (r < a.q_heads ? q_row : r < v_rows ? k_row : v_row) + r * D;
    if constexpr (INTER) return *reinterpret_cast<const uint4 *>(p + 8 * e);
    const bool is_v = r >= v_rows;
    const uint2 lo = *reinterpret_cast<const uint2 *>(p + (is_v ? 8 * e : oa));
    const uint2 hi = *reinterpret_cast<const uint2 *>(p + (is_v ? 8 * e + 4 : ob));
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  };
  uint4 next = load(r_begin), after = load(r_begin + step);
  const int64_t slot = on ? a.slots[t] : -1;
  auto weights = [&](const uint16_t *w) {  // this lane's, two packed words from oa, two from ob
    if (w == nullptr) return make_uint4(0u, 0u, 0u, 0u);
    const uint2 lo = *reinterpret_cast<const uint2 *>(w + oa);
    const uint2 hi = *reinterpret_cast<const uint2 *>(w + ob);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  };
  const uint4 qw = weights(a.q_weight), kw = weights(a.k_weight);
  for (int i = tid; i < tile * a.pairs; i += kRopeThreads) {
    const int tok = i / a.pairs, p = i - tok * a.pairs;
    if (t0 + tok < a.num_tokens) {
      const uint64_t frac = turns_per_position(a.inv_freq[p]);
      const int pos = a.positions[a.pair_axis[p] * a.axis_stride + t0 + tok];
      const int64_t turn = (int64_t)((uint64_t)(int64_t)pos * frac);  // modulo one turn
      float sn, cs;
      sincospif((float)((int32_t)(turn >> 32)) * (1.0f / 2147483648.0f), &sn, &cs);
      s_cos[tok][p] = cs * a.rope_scale;
      s_sin[tok][p] = sn * a.rope_scale;
    }
  }
  __syncthreads();
  if (!on) return;
  const unsigned gmask = (LPR == 16 ? 0xffffu : 0xffu) << ((tid & 31) & ~(LPR - 1));
  const int gbase = (tid & 31) & ~(LPR - 1);
  // pairs 4 e .. 4 e + 3, two at a time
  uint64_t cs[2] = {f32x2(1.f, 1.f), f32x2(1.f, 1.f)}, sn[2] = {0, 0}, ms[2] = {0, 0};
  if (rotates) {
    const float4 c = *reinterpret_cast<const float4 *>(&s_cos[tt][4 * e]);
    const float4 s = *reinterpret_cast<const float4 *>(&s_sin[tt][4 * e]);
    cs[0] = f32x2(c.x, c.y), cs[1] = f32x2(c.z, c.w);
    sn[0] = f32x2(s.x, s.y), sn[1] = f32x2(s.z, s.w);
    ms[0] = f32x2(-s.x, -s.y), ms[1] = f32x2(-s.z, -s.w);
  }
  bool write = slot >= 0;
  if (slot >= a.num_slots) {
    if (e == 0) flag_error(a.err, PKV_DEV_BAD_SLOT);
    write = false;
  }
  const int64_t block_row = (slot >> 4) * a.kv_heads;  // of KV head 0
  const int off = (int)(slot & 15);
  uint16_t *const q_out = a.q_out + t * a.q_out_stride;
#pragma unroll 1
  for (int r = r_begin; r < r_end; r += step) {
    const uint4 raw = next;
    next = after;
    after = load(r + 2 * step);
    const bool is_q = r < a.q_heads;
    if (!is_q && !write) continue;
    if (r >= v_rows) {
      const int64_t blk = (block_row + (r - v_rows)) * (kBlockSize * D);
      if constexpr (!F8) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.v_cache) + blk + off * D + 8 * e) = raw;
      } else {
        const float vs = a.v_scales ? a.v_scales[r - v_rows] : a.v_scale;
        if (!(vs > 0.f) || (a.k_scales && !(a.k_scales[r - v_rows] > 0.f))) {
          if (e == 0) flag_error(a.err, PKV_DEV_BAD_SCALE);
          continue;
        }
        // transposed block [D][16]: lanes trade codes so that a round covers consecutive rows
        const RowDivide div(vs);
        const uint32_t c0 = div.codes(bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y));
        const uint32_t c1 = div.codes(bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w));
        uint8_t *dst = static_cast<uint8_t *>(a.v_cache) + blk + e * kBlockSize + off;
        const uint32_t sh = 8 * (e & 3);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int from = gbase + (LPR * k + e) / 8;  // row LPR k + e is code (e & 7) there
          const uint32_t w0 = __shfl_sync(gmask, c0, from), w1 = __shfl_sync(gmask, c1, from);
          dst[LPR * kBlockSize * k] = (uint8_t)((e & 4 ? w1 : w0) >> sh);
        }
      }
      continue;
    }
    // A[i], B[i]: the elements of pair i, two pairs to a word
    uint64_t A[2], B[2];
    auto split = [](const uint4 &v, uint64_t(&x)[2], uint64_t(&z)[2]) {
      if constexpr (INTER) {
        x[0] = f32x2(bf16_lo(v.x), bf16_lo(v.y)), z[0] = f32x2(bf16_hi(v.x), bf16_hi(v.y));
        x[1] = f32x2(bf16_lo(v.z), bf16_lo(v.w)), z[1] = f32x2(bf16_hi(v.z), bf16_hi(v.w));
      } else {
        x[0] = bf16x2_to_f32x2(v.x), x[1] = bf16x2_to_f32x2(v.y);
        z[0] = bf16x2_to_f32x2(v.z), z[1] = bf16x2_to_f32x2(v.w);
      }
    };
    split(raw, A, B);
    if ((is_q ? a.q_weight : a.k_weight) != nullptr) {
      const uint64_t sq = fma_f32x2(
          A[0], A[0], fma_f32x2(A[1], A[1], fma_f32x2(B[0], B[0], mul_f32x2(B[1], B[1]))));
      float s0, s1;
      f32x2_split(sq, s0, s1);
      float ss = s0 + s1;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
      const float inv = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
      const uint64_t inv2 = f32x2(inv, inv);
      uint64_t wa[2], wb[2];
      split(is_q ? qw : kw, wa, wb);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        A[i] = mul_f32x2(mul_f32x2(A[i], inv2), wa[i]);
        B[i] = mul_f32x2(mul_f32x2(B[i], inv2), wb[i]);
      }
    }
    if (rotates) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t x = A[i];
        A[i] = fma_f32x2(x, cs[i], mul_f32x2(B[i], ms[i]));
        B[i] = fma_f32x2(B[i], cs[i], mul_f32x2(x, sn[i]));
      }
    }
    float x[4], z[4];
    f32x2_split(A[0], x[0], x[1]), f32x2_split(A[1], x[2], x[3]);
    f32x2_split(B[0], z[0], z[1]), f32x2_split(B[1], z[2], z[3]);
    if (!F8 || is_q) {
      uint2 lo, hi;
      if constexpr (INTER)
        lo = make_uint2(pack2(x[0], z[0]), pack2(x[1], z[1])),
        hi = make_uint2(pack2(x[2], z[2]), pack2(x[3], z[3]));
      else
        lo = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3])),
        hi = make_uint2(pack2(z[0], z[1]), pack2(z[2], z[3]));
      uint16_t *dst = is_q ? q_out + r * D
                           : static_cast<uint16_t *>(a.k_cache) +
                                 (block_row + (r - a.q_heads)) * (kBlockSize * D) + off * D;
      if constexpr (INTER) {
        *reinterpret_cast<uint4 *>(dst + 8 * e) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        *reinterpret_cast<uint2 *>(dst + oa) = lo;
        *reinterpret_cast<uint2 *>(dst + ob) = hi;
      }
    } else {
      const int h = r - a.q_heads;
      const float ks = a.k_scales ? a.k_scales[h] : a.k_scale;
      if (!(ks > 0.f) || (a.v_scales && !(a.v_scales[h] > 0.f))) {
        if (e == 0) flag_error(a.err, PKV_DEV_BAD_SCALE);
        continue;
      }
      const RowDivide div(ks);
      uint8_t *dst = static_cast<uint8_t *>(a.k_cache) + (block_row + h) * (kBlockSize * D) + off * D;
      if constexpr (INTER) {
        *reinterpret_cast<uint2 *>(dst + 8 * e) =
            make_uint2(div.codes(x[0], z[0], x[1], z[1]), div.codes(x[2], z[2], x[3], z[3]));
      } else {
        *reinterpret_cast<uint32_t *>(dst + oa) = div.codes(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint32_t *>(dst + ob) = div.codes(z[0], z[1], z[2], z[3]);
      }
    }
  }
}

template <int D, bool F8>
cudaError_t launch_rope(const RopeArgs &a, dim3 grid, cudaStream_t st) {
  return a.interleaved
             ? launch_pdl(qk_norm_rope_write_kernel<D, F8, true>, grid, dim3(kRopeThreads), 0, st, a)
             : launch_pdl(qk_norm_rope_write_kernel<D, F8, false>, grid, dim3(kRopeThreads), 0, st,
                          a);
}

int rope_impl(RopeArgs &a, const uint8_t *pair_axis, int num_axes, int rotary_dim, int num_blocks,
              int head_dim, int block_size, bool f8, void *stream) {
  if (block_size != kBlockSize) return PKV_ERR_BLOCK_SIZE;
  const int64_t q_row = (int64_t)a.q_heads * head_dim, kv_row = (int64_t)a.kv_heads * head_dim;
  if (a.num_tokens < 0 || num_blocks <= 0 || a.q_heads <= 0 || a.kv_heads <= 0 ||
      a.q_heads % a.kv_heads != 0 || a.q_heads > (1 << 20) || (head_dim != 64 && head_dim != 128) ||
      rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16 != 0 || num_axes < 1 ||
      num_axes > kMaxAxes || !(a.eps >= 0.f) || !(a.k_scale > 0.f) || !(a.v_scale > 0.f))
    return PKV_ERR_SHAPE;
  if (a.num_tokens == 0) return PKV_OK;
  if (!a.q_out || !a.q || !a.k || !a.v || !a.slots || !a.k_cache || !a.v_cache ||
      (rotary_dim > 0 && (!a.positions || !a.inv_freq)) || (num_axes > 1 && !pair_axis))
    return PKV_ERR_NULL;
  if (a.q_out_stride < q_row || a.q_stride < q_row || a.k_stride < kv_row || a.v_stride < kv_row)
    return PKV_ERR_SHAPE;
  if (!aligned16(a.q_out) || !aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) ||
      !aligned16(a.k_cache) || !aligned16(a.v_cache) || !aligned16(a.q_weight) ||
      !aligned16(a.k_weight) || a.q_out_stride % 8 || a.q_stride % 8 || a.k_stride % 8 ||
      a.v_stride % 8)
    return PKV_ERR_ALIGN;
  // q may be rotated in place (same rows), not otherwise overlapped by q_out
  a.pairs = rotary_dim / 2;
  std::memset(a.pair_axis, 0, sizeof(a.pair_axis));
  if (pair_axis)
    for (int i = 0; i < a.pairs; ++i) {
      if (pair_axis[i] >= num_axes) return PKV_ERR_ARG;
      a.pair_axis[i] = pair_axis[i];
    }
  a.num_slots = (int64_t)num_blocks * kBlockSize;
  const int rows = a.q_heads + 2 * a.kv_heads;
  const int groups = kRopeThreads * 8 / head_dim;
  // Many tokens: kMaxTile per CTA, every head (a token's sines are made once; one / two a CTA:
  // head_dim 64, 32/8 heads, 2432 tokens 7.9 / 6.9 us, 16384 tokens 45 / 40; head_dim 128, 64/8
  // heads, E4M3, 1021 tokens 15 / 25 and 2500 tokens 31 / 35, where two leave a short last wave,
  // 3648 tokens 40 / 40, 16384 155 / 149).  Fewer: one token per CTA, its rows split over CTAs
  // until there are as many as fit at once or a lane group has one row (400 tokens, 64/8 heads,
  // E4M3: 11.2 us with four CTAs per SM, 6.5 with eight, 8.5 with sixteen).
  const int sms = device_sm_count();
  a.tile = a.num_tokens >= (head_dim == 64 ? 8 : 24) * sms ? kMaxTile : 1;
  int parts = 1;
  if (a.tile == 1) {
    parts = kRopeCtas * sms / a.num_tokens;
    const int most = (rows + groups - 1) / groups;
    parts = parts < 1 ? 1 : parts > most ? most : parts;
  }
  a.chunk = ((rows + parts - 1) / parts + groups - 1) / groups * groups;
  const unsigned ny = (unsigned)((rows + a.chunk - 1) / a.chunk);
  if (ny > 65535) return PKV_ERR_SHAPE;
  const dim3 grid((unsigned)((a.num_tokens + a.tile - 1) / a.tile), ny);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (head_dim == 128)
    e = f8 ? launch_rope<128, true>(a, grid, st) : launch_rope<128, false>(a, grid, st);
  else
    e = f8 ? launch_rope<64, true>(a, grid, st) : launch_rope<64, false>(a, grid, st);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

RopeArgs rope_args(uint16_t *q_out, int64_t q_out_stride, const uint16_t *q, int64_t q_stride,
                   const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                   const uint16_t *q_weight, const uint16_t *k_weight, float eps,
                   const int32_t *positions, int64_t axis_stride, const double *inv_freq,
                   int interleaved, float rope_scale, const int64_t *slot_mapping, int num_tokens,
                   void *k_cache, void *v_cache, int num_q_heads, int num_kv_heads,
                   int32_t *err_flag) {
  RopeArgs a = {};
  a.q_out = q_out, a.q = q, a.k = k, a.v = v;
  a.q_out_stride = q_out_stride, a.q_stride = q_stride;
  a.k_stride = k_stride, a.v_stride = v_stride;
  a.q_weight = q_weight, a.k_weight = k_weight, a.eps = eps;
  a.positions = positions, a.axis_stride = axis_stride, a.inv_freq = inv_freq;
  a.interleaved = interleaved ? 1 : 0, a.rope_scale = rope_scale;
  a.slots = slot_mapping, a.num_tokens = num_tokens;
  a.q_heads = num_q_heads, a.kv_heads = num_kv_heads;
  a.k_cache = k_cache, a.v_cache = v_cache;
  a.k_scale = a.v_scale = 1.f;
  a.err = err_flag;
  return a;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int paged_qk_norm_rope_write(uint16_t *q_out, int64_t q_out_stride, const uint16_t *q,
                             int64_t q_stride, const uint16_t *k, int64_t k_stride,
                             const uint16_t *v, int64_t v_stride, const uint16_t *q_weight,
                             const uint16_t *k_weight, float eps, const int32_t *positions,
                             int64_t axis_stride, int num_axes, const uint8_t *pair_axis,
                             const double *inv_freq, int rotary_dim, int interleaved,
                             float rope_scale, const int64_t *slot_mapping, int num_tokens,
                             uint16_t *k_cache, uint16_t *v_cache, int num_blocks,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int32_t *err_flag, void *stream) {
  RopeArgs a = rope_args(q_out, q_out_stride, q, q_stride, k, k_stride, v, v_stride, q_weight,
                         k_weight, eps, positions, axis_stride, inv_freq, interleaved, rope_scale,
                         slot_mapping, num_tokens, k_cache, v_cache, num_q_heads, num_kv_heads,
                         err_flag);
  return rope_impl(a, pair_axis, num_axes, rotary_dim, num_blocks, head_dim, block_size, false,
                   stream);
}

int paged_qk_norm_rope_write_fp8(uint16_t *q_out, int64_t q_out_stride, const uint16_t *q,
                                 int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                 const uint16_t *v, int64_t v_stride, const uint16_t *q_weight,
                                 const uint16_t *k_weight, float eps, const int32_t *positions,
                                 int64_t axis_stride, int num_axes, const uint8_t *pair_axis,
                                 const double *inv_freq, int rotary_dim, int interleaved,
                                 float rope_scale, const int64_t *slot_mapping, int num_tokens,
                                 uint8_t *k_cache, uint8_t *v_cache, int num_blocks,
                                 int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, float k_scale, float v_scale,
                                 const float *k_scales, const float *v_scales,
                                 int32_t *err_flag, void *stream) {
  if ((k_scales == nullptr) != (v_scales == nullptr)) return PKV_ERR_NULL;
  RopeArgs a = rope_args(q_out, q_out_stride, q, q_stride, k, k_stride, v, v_stride, q_weight,
                         k_weight, eps, positions, axis_stride, inv_freq, interleaved, rope_scale,
                         slot_mapping, num_tokens, k_cache, v_cache, num_q_heads, num_kv_heads,
                         err_flag);
  if (k_scales == nullptr) a.k_scale = k_scale, a.v_scale = v_scale;
  a.k_scales = k_scales, a.v_scales = v_scales;
  return rope_impl(a, pair_axis, num_axes, rotary_dim, num_blocks, head_dim, block_size, true,
                   stream);
}

}  // extern "C"
