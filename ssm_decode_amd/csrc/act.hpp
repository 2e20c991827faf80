// SiLU and its derivative in fp32 for the memory-bound kernels, from the hardware's 2^x and 1/x (one ulp each).
#pragma once

#include "element.hpp"

namespace rs {

// 1 / (1 + e^-z). The product z log2(e) is rounded, which 2^x turns into a relative error of |z| 2^-24: below the
// rounding of 16-bit results for every z that they hold. For fp32 results (EXACT) the product's remainder goes in to first order.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) {
  constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = 1.9259629911e-8f, kLn2 = 0.69314718055994531f;
  // below -88 the result is under 2^-126 and taken as 0, above 88 it is 1
  const float c = fminf(fmaxf(z, -88.f), 88.f);
  const float t = -c * kLog2e;
  float e = __builtin_amdgcn_exp2f(t);
  if (EXACT) {
    const float low = __builtin_fmaf(-c, kLog2e, -t) - c * kLog2eLow;
    e = __builtin_fmaf(e, low * kLn2, e);
  }
  const float r = __builtin_amdgcn_rcpf(1.f + e);
  return z < -88.f ? 0.f : (z == z ? r : z);  // (max drops a NaN)
}

struct Silu {
  float value, slope;
};

// z sigmoid(z) and its derivative sigmoid(z) (1 + z (1 - sigmoid(z))).
template <bool EXACT>
__device__ __forceinline__ Silu silu(float z) {
  const float s = sigmoid<EXACT>(z);
  const float v = z * s;
  return Silu{v, __builtin_fmaf(v, 1.f - s, s)};
}

// Eight consecutive elements of any type as they come from memory, 16-byte aligned.
template <typename T>
struct Eight;
template <>
struct Eight<__bf16> {
  bf16x8 x;
};
template <>
struct Eight<_Float16> {
  f16x8 x;
};
template <>
struct Eight<float> {
  f32x8 x;
};
template <typename T>
__device__ __forceinline__ Eight<T> raw8(const T* p) {
  return Eight<T>{*reinterpret_cast<const decltype(Eight<T>::x)*>(p)};
}
template <>
__device__ __forceinline__ Eight<float> raw8<float>(const float* p) {
  return Eight<float>{load8(p)};
}
template <typename T>
__device__ __forceinline__ f32x8 wide(const Eight<T>& r) {
  return __builtin_convertvector(r.x, f32x8);
}

}  // namespace rs
