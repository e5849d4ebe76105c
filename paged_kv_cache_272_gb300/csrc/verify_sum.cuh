// Residuals max(p - M d, 0) and their sums as whole numbers, for the verification of drafted tokens.
// Every step is rounded as it is written: where a product and an addition became one rounding, the
// error terms would count twice.  (Plain C++ too, for a compiler that contracts nothing.)
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define PKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PKV_HOST_DEVICE inline
#endif

namespace pkv {

#ifdef __CUDA_ARCH__
__device__ __forceinline__ float mul_rn(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add_rn(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float sub_rn(float a, float b) { return __fsub_rn(a, b); }
__device__ __forceinline__ uint32_t float_bits(float x) { return __float_as_uint(x); }
#else
PKV_HOST_DEVICE float mul_rn(float a, float b) { return a * b; }
PKV_HOST_DEVICE float add_rn(float a, float b) { return a + b; }
PKV_HOST_DEVICE float sub_rn(float a, float b) { return a - b; }
PKV_HOST_DEVICE uint32_t float_bits(float x) {
  uint32_t u;
  memcpy(&u, &x, 4);
  return u;
}
#endif

// A row's sums, in units of 2^-43: high 2^22 + low, both of 32 bits while the values summed are
// fewer than 2^9 and sum to less than 2^10.  An fp32 number s in [0, 2) loses a multiple of 2^-21 to
// the high part by the addition of a constant whose last place is that; what is left, 2^-22 at most, and
// the low number t, below 2^-22, go to the low part in the same way.  Together they are below 2^-21, 2^22
// units: the constant of 1.5 2^23 units keeps them in one binade, where the bits count units.  (A unit
// of 2^-44 leaves no place for t beside a remainder of half a high unit, whose bits then count twice
// or half: off by up to 2^-25 where one token dominates.)
constexpr int kUnitBits = 43, kHighBits = 21;
constexpr float kHighMagic = 12582912.f / (1 << kHighBits);  // 1.5 2^23 units of 2^-21
constexpr float kLowMagic = 12582912.f / (float)(1ull << kUnitBits);

struct Sum {
  uint32_t high = 0, low = 0;  // of the magic numbers' bits, modulo 2^32
  // s + t to half a unit (t rounded once more: 2^-46), s in [0, 2), |t| < 2^-22
  PKV_HOST_DEVICE void add(float s, float t) {
    const float a = add_rn(s, kHighMagic);
    const float b = add_rn(add_rn(sub_rn(s, sub_rn(a, kHighMagic)), t), kLowMagic);
    high += float_bits(a) - float_bits(kHighMagic);
    low += float_bits(b) - float_bits(kLowMagic);
  }
  PKV_HOST_DEVICE unsigned long long value() const {
    return ((unsigned long long)(long long)(int)high << (kUnitBits - kHighBits)) +
           (unsigned long long)(long long)(int)low;
  }
};

// max(p - M d, 0) as the sum of two numbers, M = mh + ml: the rounding errors of the product (and
// ml d) and of the difference are carried along, each 2^-24 of p or M d at most (what counts has
// M d <= p < 2, so |t| < 2^-22), and the low number is rounded at 2^-47 of p.
PKV_HOST_DEVICE void residual(float p, float d, float mh, float ml, float &s, float &t) {
  const float h = mul_rn(mh, d), e = fmaf(ml, d, fmaf(mh, d, -h));
  s = sub_rn(p, h);
  const float b = sub_rn(s, p);
  t = sub_rn(sub_rn(sub_rn(p, sub_rn(s, b)), add_rn(h, b)), e);
  if (!(add_rn(s, t) > 0.f)) s = t = 0.f;
}

}  // namespace pkv
