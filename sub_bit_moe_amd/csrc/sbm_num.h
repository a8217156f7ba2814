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
// bits then sees on which side of a border the value was.  Of numbers from 2^-126 on; those below are rounded to the nearest.
__device__ __forceinline__ float to_odd(double y) {
  constexpr uint32_t kBelow = 0x1FFFFFFFu;
  const uint64_t b = __builtin_bit_cast(uint64_t, y);
  const uint32_t low = (uint32_t)b, carry = (low & kBelow) + kBelow;       // into the lowest bit that stays, if any below it is set
  return (float)__builtin_bit_cast(double, b >> 32 << 32 | ((low | carry) & ~kBelow));
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

// Eight numbers, also those of bf16 below 2^-126.
template <typename T>
__device__ __forceinline__ void round_once8(const double* x, uint16_t* y) {
  float odd[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) odd[j] = to_odd(x[j]);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = round_once<T>(odd[j]);
  if constexpr (__is_same(T, __bf16)) {
    bool small = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) small = small || __builtin_isfpclass(odd[j], 0x0090);        // subnormal
    if (small) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double steps = __builtin_rint(__builtin_fabs(x[j]) * 0x1p133);
        if (__builtin_fabs(x[j]) < 0x1p-126) y[j] = (uint16_t)((uint32_t)steps | (__float_as_uint(odd[j]) >> 31) << 15);
      }
    }
  }
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

// The 32-bit parts of 64.
using Halves = uint32_t __attribute__((ext_vector_type(2)));

// 2^(x by), to 4e-14 of itself, for x by within -1000 .. 1000: its whole part goes to the exponent, 2^f for the rest, |f| <= 1/2, is
// a polynomial of degree 9 that interpolates it at Chebyshev's points (3.7e-14 off at most) and is 1 at 0.  f64 runs at the rate of
// unpacked f32 here.
__device__ __forceinline__ double exp2_f64(double x, double by) {
  // n's low bits are the nearest whole number
  const double n = __builtin_fma(x, by, 0x1.8p52), y = __builtin_fma(x, by, -(n - 0x1.8p52));
  // as one block, since the compiler would copy each coefficient into the register of the sum, an instruction more
  double p;
  asm("v_fma_f64 %0, %2, %1, %3\n\tv_fma_f64 %0, %0, %1, %4\n\tv_fma_f64 %0, %0, %1, %5\n\tv_fma_f64 %0, %0, %1, %6\n\t"
      "v_fma_f64 %0, %0, %1, %7\n\tv_fma_f64 %0, %0, %1, %8\n\tv_fma_f64 %0, %0, %1, %9\n\tv_fma_f64 %0, %0, %1, %10\n\t"
      "v_fma_f64 %0, %0, %1, 1.0"
      : "=&v"(p)
      : "v"(y), "v"(0x1.b63880a30e9ffp-24), "s"(0x1.63d136366db24p-20), "s"(0x1.ffcb9515a8016p-17), "s"(0x1.4308ac85aa947p-13),
        "s"(0x1.5d87fe86fe88ep-10), "s"(0x1.3b2ab7181b755p-7), "s"(0x1.c6b08d7047e52p-5), "s"(0x1.ebfbdff823cedp-3),
        "s"(0x1.62e42fefa39efp-1));
  Halves u = __builtin_bit_cast(Halves, p);
  u[1] += __builtin_bit_cast(Halves, n)[0] << 20;
  return __builtin_bit_cast(double, u);
}
// 2^x; below -1000 it stays 2^-1000, for -inf and NaN too.
__device__ __forceinline__ double exp2_f64(double x) { return exp2_f64(fmax(x, -1000.), 1.); }

// 1 / x of normal numbers: the hardware's estimate and two of Newton's steps.
__device__ __forceinline__ double inverse(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = __builtin_fma(__builtin_fma(-x, y, 1.), y, y);
  return __builtin_fma(__builtin_fma(-x, y, 1.), y, y);
}

// 32 bits that order as the numbers do; both zeros are one.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// Sums over a wave's lanes up to each (row shifts, then rows' and halves' last lanes to what is behind them).
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xF, false);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ uint64_t moved(uint64_t v) {
  return (uint64_t)moved<kCtrl, kRows>((uint32_t)(v >> 32)) << 32 | moved<kCtrl, kRows>((uint32_t)v);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float(moved<kCtrl, kRows>(__float_as_uint(v)));
}
template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double v) {
  return __builtin_bit_cast(double, moved<kCtrl, kRows>(__builtin_bit_cast(uint64_t, v)));
}
template <typename V>
__device__ __forceinline__ V wave_scan(V v) {
  v += moved<0x111, 0xF>(v);
  v += moved<0x112, 0xF>(v);
  v += moved<0x114, 0xF>(v);
  v += moved<0x118, 0xF>(v);
  v += moved<0x142, 0xA>(v);
  v += moved<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ uint32_t of_lane(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ __forceinline__ uint64_t of_lane(uint64_t v, int lane) {
  return (uint64_t)of_lane((uint32_t)(v >> 32), lane) << 32 | of_lane((uint32_t)v, lane);
}
__device__ __forceinline__ float of_lane(float v, int lane) { return __uint_as_float(of_lane(__float_as_uint(v), lane)); }
__device__ __forceinline__ double of_lane(double v, int lane) {
  return __builtin_bit_cast(double, of_lane(__builtin_bit_cast(uint64_t, v), lane));
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
  return of_lane(wave_scan(v), 63);
}

template <int kCtrl, int kRows>
__device__ __forceinline__ float larger(float v) {
  return fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(v), (int)__float_as_uint(v), kCtrl, kRows, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = larger<0x111, 0xF>(v);
  v = larger<0x112, 0xF>(v);
  v = larger<0x114, 0xF>(v);
  v = larger<0x118, 0xF>(v);
  v = larger<0x142, 0xA>(v);
  v = larger<0x143, 0xC>(v);
  return __uint_as_float(of_lane(__float_as_uint(v), 63));
}

// Up to 64 different numbers of a wave's lanes, n of them, in order.
__device__ __forceinline__ uint64_t wave_sorted(uint64_t o, uint32_t n, uint64_t* space) {
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t rank = 0;
  for (uint32_t j = 0; j < n; ++j) rank += of_lane(o, (int)j) < o;
  if (lane < n) space[rank] = o;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  return lane < n ? space[lane] : ~0ull;
}

}  // namespace
}  // namespace sbm
