// Head-wise RMS norm of q and k, rotary positions, and the paged write of k and v, in one
// pass over a step's projections.
//
//   y = x / sqrt(mean(x^2) + eps) * w                    (per head; only with weights)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = pos[axis(i)] * inv_freq[i]
// for rotary pair i of the first rotary_dim elements: (y[i], y[i + rotary_dim / 2]), or
// (y[2 i], y[2 i + 1]) when interleaved.  All of it in fp32 with one rounding at the store
// (bf16, or the E4M3 code of value / scale).  v is stored as it is.
//
// Angles: a turn count t / 2 pi needs its fraction only, so a frequency is held as a 64-bit
// fixed-point fraction of a turn per position and multiplied by the 32-bit position modulo
// 2^64: the angle's error is that of the frequency's own rounding (2^-53) times the
// position, however far the position -- where an fp32 product would be 0.06 rad off at a
// million.  sincospi then takes the top bits.
//
// Bound: bytes.  Every row is read once and written once; a token's sines are made once per
// CTA (kTile tokens share it) and held in registers across the heads a lane serves.
#include <math.h>

#include <cstring>

#include "kv_rows.cuh"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kMaxAxes = 4;
constexpr int kMaxPairs = 64;
constexpr int kRopeThreads = 256;
constexpr int kMaxTile = 4;  // tokens per CTA
constexpr int kBatch = 4;    // rows a lane group has in flight

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
  int tile;                  // tokens per CTA (1, 2 or 4)
  int chunk;                 // rows (q, k and v heads) per CTA
  int32_t *err;
  uint8_t pair_axis[kMaxPairs];
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ uint4 ld_row(const uint16_t *p) {
  return *reinterpret_cast<const uint4 *>(p);
}

// One group of D / 8 lanes owns a (token, head) row, 8 elements a lane.
template <int D, bool F8>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_write_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8;
  constexpr int GROUPS = kRopeThreads / LPR;
  __shared__ __align__(16) float s_cos[kMaxTile][kMaxPairs], s_sin[kMaxTile][kMaxPairs];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, tile = a.tile;
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  for (int i = tid; i < tile * a.pairs; i += kRopeThreads) {
    const int tt = i / a.pairs, p = i - tt * a.pairs;
    if (t0 + tt < a.num_tokens) {
      const double turns = a.inv_freq[p] * 0.15915494309189533577;  // per position
      const uint64_t frac = (uint64_t)__double2ull_rd((turns - floor(turns)) * 18446744073709551616.0);
      const int pos = a.positions[a.pair_axis[p] * a.axis_stride + t0 + tt];
      const int64_t turn = (int64_t)((uint64_t)(int64_t)pos * frac);  // modulo one turn
      float sn, cs;
      sincospif((float)((int32_t)(turn >> 32)) * (1.0f / 2147483648.0f), &sn, &cs);
      s_cos[tt][p] = cs * a.rope_scale;
      s_sin[tt][p] = sn * a.rope_scale;
    }
  }
  __syncthreads();
  const int e = tid % LPR, grp = tid / LPR;
  const int tt = grp % tile;
  const int64_t t = t0 + tt;
  if (t >= a.num_tokens) return;
  const unsigned gmask = (LPR == 16 ? 0xffffu : 0xffu) << ((tid & 31) & ~(LPR - 1));
  const int gbase = (tid & 31) & ~(LPR - 1);
  // this lane's sines: 8 half-split elements share 8 pairs, 8 interleaved ones hold 4
  const int half_lanes = a.pairs / 8;  // lanes of one half (half-split)
  const bool rotates = e < 2 * half_lanes;
  const bool second = e >= half_lanes;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int p = a.interleaved ? 4 * e + (j >> 1) : (second ? e - half_lanes : e) * 8 + j;
    cs[j] = rotates ? s_cos[tt][p] : 1.f;
    sn[j] = rotates ? s_sin[tt][p] : 0.f;
  }
  const int partner = gbase + (!rotates ? e : second ? e - half_lanes : e + half_lanes);
  const int64_t slot = a.slots[t];
  bool write = slot >= 0;
  if (slot >= a.num_slots) {
    if (e == 0) flag_error(a.err, PKV_DEV_BAD_SLOT);
    write = false;
  }
  const int rows = a.q_heads + 2 * a.kv_heads;
  const int r_end = min(rows, ((int)blockIdx.y + 1) * a.chunk), step = GROUPS / tile;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 qw = a.q_weight ? *reinterpret_cast<const uint4 *>(a.q_weight + e * 8) : zero;
  const uint4 kw = a.k_weight ? *reinterpret_cast<const uint4 *>(a.k_weight + e * 8) : zero;
  for (int r0 = blockIdx.y * a.chunk + grp / tile; r0 < r_end; r0 += kBatch * step) {
    uint4 raw[kBatch];  // every load of the batch before the first use
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = r0 + u * step;
      raw[u] = zero;
      if (r < a.q_heads)
        raw[u] = ld_row(a.q + t * a.q_stride + (int64_t)r * D + e * 8);
      else if (r < r_end && write)
        raw[u] = r < a.q_heads + a.kv_heads
                     ? ld_row(a.k + t * a.k_stride + (int64_t)(r - a.q_heads) * D + e * 8)
                     : ld_row(a.v + t * a.v_stride +
                              (int64_t)(r - a.q_heads - a.kv_heads) * D + e * 8);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = r0 + u * step;
      const bool is_q = r < a.q_heads, is_v = r >= a.q_heads + a.kv_heads;
      if (r >= r_end || (!is_q && !write)) continue;
      const int h = is_q ? r : is_v ? r - a.q_heads - a.kv_heads : r - a.q_heads;
      const int64_t row16 = ((slot >> 4) * a.kv_heads + h) * kBlockSize + (slot & 15);
      float ks = a.k_scale, vs = a.v_scale;
      if (F8 && !is_q && a.k_scales != nullptr) {
        ks = a.k_scales[h], vs = a.v_scales[h];
        if (!(ks > 0.f) || !(vs > 0.f)) {
          if (e == 0) flag_error(a.err, PKV_DEV_BAD_SCALE);
          continue;
        }
      }
      if (is_v) {
        if constexpr (!F8) {
          reinterpret_cast<uint4 *>(a.v_cache)[row16 * LPR + e] = raw[u];
        } else {
          // transposed block [D][16]: lanes trade codes so a round covers consecutive rows
          const uint32_t c0 = quant4(raw[u].x, raw[u].y, vs), c1 = quant4(raw[u].z, raw[u].w, vs);
          uint8_t *blk = static_cast<uint8_t *>(a.v_cache) +
                         ((slot >> 4) * a.kv_heads + h) * (int64_t)(D * kBlockSize) + (slot & 15);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int d = LPR * k + e;
            const uint32_t w0 = __shfl_sync(gmask, c0, gbase + (d >> 3));
            const uint32_t w1 = __shfl_sync(gmask, c1, gbase + (d >> 3));
            blk[d * kBlockSize] = (uint8_t)(((d & 4) ? w1 : w0) >> (8 * (d & 3)));
          }
        }
        continue;
      }
      float x[8];
      unpack8(raw[u], x);
      if ((is_q ? a.q_weight : a.k_weight) != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(gmask, ss, off);
        const float inv = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
        float w[8];
        unpack8(is_q ? qw : kw, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * w[j];
      }
      float y[8];
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          y[j] = x[j] * cs[j] - x[j + 1] * sn[j];
          y[j + 1] = x[j + 1] * cs[j] + x[j] * sn[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float o = __shfl_sync(gmask, x[j], partner);
          y[j] = x[j] * cs[j] + (second ? o : -o) * sn[j];
        }
      }
      if (!rotates) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
      }
      if (!F8 || is_q) {
        const uint4 o = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]),
                                   pack2(y[6], y[7]));
        if (is_q)
          *reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride + (int64_t)h * D + e * 8) = o;
        else
          reinterpret_cast<uint4 *>(a.k_cache)[row16 * LPR + e] = o;
      } else {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[j] = __nv_cvt_float2_to_fp8x2(
              make_float2(__fdiv_rn(y[2 * j], ks), __fdiv_rn(y[2 * j + 1], ks)), __NV_SATFINITE,
              __NV_E4M3);
        reinterpret_cast<uint2 *>(a.k_cache)[row16 * LPR + e] =
            make_uint2((c[0] & 0xffffu) | (c[1] << 16), (c[2] & 0xffffu) | (c[3] << 16));
      }
    }
  }
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
  // Many tokens: 4 per CTA, every head (a token's sines are made once).  Fewer: one token per
  // CTA, its rows split over CTAs until there are four per SM or a lane group has one row.
  const int sms = device_sm_count();
  a.tile = a.num_tokens >= 16 * sms ? kMaxTile : 1;
  int parts = 1;
  if (a.tile == 1) {
    parts = 4 * sms / a.num_tokens;
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
    e = f8 ? launch_pdl(qk_norm_rope_write_kernel<128, true>, grid, dim3(kRopeThreads), 0, st, a)
           : launch_pdl(qk_norm_rope_write_kernel<128, false>, grid, dim3(kRopeThreads), 0, st, a);
  else
    e = f8 ? launch_pdl(qk_norm_rope_write_kernel<64, true>, grid, dim3(kRopeThreads), 0, st, a)
           : launch_pdl(qk_norm_rope_write_kernel<64, false>, grid, dim3(kRopeThreads), 0, st, a);
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
