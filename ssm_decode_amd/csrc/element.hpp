// Element types of the prompt-side operators: fp32, bf16 and fp16 rows in memory, fp32 in registers.
#pragma once

#include "device.hpp"

namespace rs {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct F32 {
  typedef float type;
};
struct Bf16 {
  typedef __bf16 type;
};
struct F16 {
  typedef _Float16 type;
};

// Eight consecutive elements at a 16-byte aligned address (fp32: two 16-byte loads).
__device__ __forceinline__ f32x8 load8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ f32x8 load8(const __bf16* p) {
  return __builtin_convertvector(*reinterpret_cast<const bf16x8*>(p), f32x8);
}
__device__ __forceinline__ f32x8 load8(const _Float16* p) {
  return __builtin_convertvector(*reinterpret_cast<const f16x8*>(p), f32x8);
}

// Rounded once, to nearest even.
__device__ __forceinline__ void store8(float* p, const f32x8& x) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store8(__bf16* p, const f32x8& x) {
  *reinterpret_cast<bf16x8*>(p) = __builtin_convertvector(x, bf16x8);
}
__device__ __forceinline__ void store8(_Float16* p, const f32x8& x) {
  *reinterpret_cast<f16x8*>(p) = __builtin_convertvector(x, f16x8);
}

}  // namespace rs
