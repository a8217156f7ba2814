// Numbers that the serving kernels share: conversions with one rounding, order-keeping keys, lanes' sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbm {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(uint16_t u) {
  if constexpr (__is_same(T, __bf16)) return __uint_as_float((uint32_t)u << 16);
  else return (float)__builtin_bit_cast(_Float16, u);
}

// 64 bits to 32 with what those cannot hold gathered in their lowest bit (round to odd): a further rounding to fewer
// bits then sees on which side of a border the value was.
__device__ __forceinline__ float to_odd(double y) {
  uint64_t b = __builtin_bit_cast(uint64_t, y);
  const uint32_t low = (uint32_t)b & 0x1FFFFFFFu;
  b = (b & ~0x1FFFFFFFull) | (low ? 0x20000000u : 0u);
  return (float)__builtin_bit_cast(double, b);
}

// One rounding to T.
template <typename T>
__device__ __forceinline__ uint16_t round_once(float y) {
  return __builtin_bit_cast(uint16_t, (T)y);
}
template <typename T>
__device__ __forceinline__ uint16_t round_once(double y) {
  return round_once<T>(to_odd(y));
}

// 1 / sqrt(x): the hardware's estimate and one step of third order (2^-23 to below 2^-60).
__device__ __forceinline__ double inverse_root(double x) {
  const double y = __builtin_amdgcn_rsq(x), e = __builtin_fma(-x * y, y, 1.0);
  const double z = __builtin_fma(y * e, __builtin_fma(e, 0.375, 0.5), y);
  return x == 0. || x == (double)INFINITY ? y : z;
}
__device__ __forceinline__ float inverse_root(float x) {
  if (!(x > 1e-30f && x < 1e30f)) return 1.f / sqrtf(x);
  const float y = __builtin_amdgcn_rsqf(x), e = __builtin_fmaf(-x * y, y, 1.f);
  return __builtin_fmaf(y * e, 0.5f, y);
}

__device__ __forceinline__ float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fused(double a, double b, double c) { return __builtin_fma(a, b, c); }

}  // namespace
}  // namespace sbm
