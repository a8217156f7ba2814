// The norm between a decoder's parts: the residual's addition, the sum over a
// token's experts, root-mean-square norm, and results in 16 or in 8 bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sbm_internal.h"
#include "sbm_num.h"

namespace sbm {
namespace {

constexpr int kMostDim = 32768;
constexpr int kMostThreads = 1024;
constexpr int kMostGrid = 1 << 21;             // a launch has fewer than 2^32 threads
constexpr int kFewThreads = 256;               // of a workgroup that has several rows

struct NormArgs {
  const void* x;
  const void* residual;
  void* residual_out;
  const uint16_t* weight;
  const float* gates;
  void* out;
  void* scales;
  int64_t x_stride, r_stride, ro_stride, o_stride;      // elements
  int64_t first;                                        // the launch's first row
  double eps;
  int32_t dim, k, repeat, block;                        // block: elements that share a scale, the row's if `whole`
  int32_t n_tokens, lanes;                              // lanes: threads of a row
  bool whole, powers;                                   // powers: scales are bytes
};

// Eight elements as they are in memory.  Rows may start anywhere an element may: the hardware takes a 16-byte access at any
// address.
template <bool kF32>
struct Raw {
  uint32_t v[kF32 ? 8 : 4];
};

template <bool kF32>
__device__ __forceinline__ Raw<kF32> load_raw(const void* row, int d0, int dim) {
  Raw<kF32> r;
  if (d0 + 8 <= dim) {
    __builtin_memcpy(&r, (const char*)row + (int64_t)d0 * (kF32 ? 4 : 2), sizeof r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (kF32) {
        r.v[j] = d0 + j < dim ? ((const uint32_t*)row)[d0 + j] : 0u;
      } else {
        const uint32_t u = d0 + j < dim ? ((const uint16_t*)row)[d0 + j] : 0u;
        r.v[j >> 1] = j & 1 ? r.v[j >> 1] | u << 16 : u;
      }
    }
  }
  return r;
}

template <typename T, bool kF32>
__device__ __forceinline__ float value(const Raw<kF32>& r, int j) {
  if constexpr (kF32) return __uint_as_float(r.v[j]);
  else return to_f32<T>((uint16_t)(r.v[j >> 1] >> 16 * (j & 1)));
}

// The first n of eight elements of kBytes each.
template <int kBytes>
__device__ __forceinline__ void store_raw(void* p, const void* x, int n) {
  if (n >= 8) {
    __builtin_memcpy(p, x, 8 * kBytes);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < n) __builtin_memcpy((char*)p + j * kBytes, (const char*)x + j * kBytes, kBytes);
    }
  }
}

struct Sum {
  __device__ double operator()(double a, double b) const { return a + b; }
};
// Magnitudes order as their bits do, NaN above infinity.
__device__ __forceinline__ uint64_t magnitude(double x) { return __builtin_bit_cast(uint64_t, x) & 0x7FFFFFFFFFFFFFFFull; }
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
struct Most {
  template <typename V>
  __device__ V operator()(V a, V b) const {
    return a > b ? a : b;
  }
};

// v joined over a row's threads, in all of them, in an order that does not change.
template <typename Op, bool kFew, typename C>
__device__ __forceinline__ C over_row(C v, C* shared, int lanes) {
  Op op;
  if constexpr (kFew) {
    for (int d = 1; d < lanes; d <<= 1) v = op(v, __shfl_xor(v, d, 64));
    return v;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = op(v, __shfl_xor(v, d, 64));
  const int waves = lanes >> 6;
  if (waves > 1) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = shared[0];
    for (int w = 1; w < waves; ++w) v = op(v, shared[w]);
  }
  return v;
}

// Eight elements of a row as codes, and the scale where a block begins; V: the scale's type.
template <typename V>
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t t, int d0, int n_blocks, const float* q, float by, bool bad, V scale) {
  if (d0 >= a.dim) return;
  uint32_t y[2] = {0u, 0u};
  if (!bad) {
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = fminf(fmaxf(q[j] * by, -448.f), 448.f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      y[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * j], c[4 * j + 1], 0, false);
      y[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * j + 2], c[4 * j + 3], (int)y[j], true);
    }
  }
  for (int r = 0; r < a.repeat; ++r) {
    const int64_t row = t * a.repeat + r;
    store_raw<1>((uint8_t*)a.out + row * a.o_stride + d0, y, a.dim - d0);
    if (d0 % a.block == 0) ((V*)a.scales)[row * n_blocks + d0 / a.block] = scale;
  }
}

//   h = residual + sum over e of gate_e x_e,  residual_out = h rounded,  out = h (mean(h^2) + eps)^-1/2 weight
// The norm takes h as it was before its rounding.  8-bit results: out / scale to e4m3, the scale from a block's largest magnitude.
// A workgroup holds a row in its registers, kN times eight elements a thread: everything is read once and written once.  The
// mean of squares is summed in 64 bits (f64 runs at the rate of unpacked f32 here), so that no row of finite numbers
// overflows it; what becomes 8 bits is computed in 64 bits throughout (C), so that a code beside the border of two does not
// depend on the order of a sum.
// What bounds it: memory for prompts (8191 x 4096 with residual in and out, 268 MB: 50.7 us, 5.3 TB/s; vector units busy for 68 %;
// 8192 x 4096 of eight fp32 rows each, 1.41 GB: 272 us, 5.2 TB/s); for 8 bits the 64-bit arithmetic, near to memory (4096 x 8192, 236 MB,
// bytes of scales: 58 us, 4.1 TB/s, vector units busy for 85 %; fp32 scales of 128 elements 58, of a row 60); for few tokens one row's
// latency (3.5 us a token alone, 5.0 us 64 tokens of two experts; 9 us with the host's call).
template <typename T, bool kXF, bool kRF, bool k8, int kN, bool kFew>
__global__ __launch_bounds__(kMostThreads) void norm_kernel(NormArgs a) {
  using C = std::conditional_t<k8, double, float>;
  __shared__ double s_sum[kMostThreads / 64];
  // a workgroup has one row, or (kFew) several of fewer threads than a wave each
  const int G = kFew ? a.lanes : (int)blockDim.x, tid = kFew ? (int)threadIdx.x & (G - 1) : (int)threadIdx.x;
  int64_t t = a.first + blockIdx.x;
  if constexpr (kFew) {
    t = a.first + (int64_t)blockIdx.x * (kFewThreads / G) + threadIdx.x / (uint32_t)G;
    if (t >= a.n_tokens) return;
  }
  C h[kN][8];
  if (a.residual) {
    const char* row = (const char*)a.residual + t * a.r_stride * (kRF ? 4 : 2);
    Raw<kRF> r[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) r[i] = load_raw<kRF>(row, (tid + i * G) * 8, a.dim);
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = (C)value<T, kRF>(r[i], j);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = (C)0;
  }
  for (int e = 0; e < a.k; ++e) {
    const float gate = a.gates ? a.gates[t * a.k + e] : 1.f;
    if (gate == 0.f) continue;
    const char* row = (const char*)a.x + (t * a.k + e) * a.x_stride * (kXF ? 4 : 2);
    Raw<kXF> r[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) r[i] = load_raw<kXF>(row, (tid + i * G) * 8, a.dim);
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = fused((C)gate, (C)value<T, kXF>(r[i], j), h[i][j]);
  }
  if (a.residual_out) {
    char* row = (char*)a.residual_out + t * a.ro_stride * (kRF ? 4 : 2);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int d0 = (tid + i * G) * 8;
      if constexpr (kRF) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (float)h[i][j];
        store_raw<4>(row + (int64_t)d0 * 4, y, a.dim - d0);
      } else {
        uint16_t y[8];
        if constexpr (k8) {
          round_once8<T>(h[i], y);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = round_once<T>(h[i][j]);
        }
        store_raw<2>(row + (int64_t)d0 * 2, y, a.dim - d0);
      }
    }
  }
  double ss = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)h[i][j], (double)h[i][j], ss);
  const double mean = over_row<Sum, kFew>(ss, s_sum, G) / (double)a.dim + a.eps;
  const double inv = inverse_root(mean);
  // weights; what is behind the row's end is zero
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int d0 = (tid + i * G) * 8;
    Raw<false> w;
    if (a.weight) w = load_raw<false>(a.weight, d0, a.dim);
    if (k8 || (mean > 1e-30 && mean < 1e30)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = (h[i][j] * (C)inv) * (a.weight ? (C)value<T, false>(w, j) : (C)1);
    } else {                                            // its root is no normal number of 32 bits
#pragma unroll
      for (int j = 0; j < 8; ++j)
        h[i][j] = (C)((double)h[i][j] * inv) * (a.weight ? (C)value<T, false>(w, j) : (C)1);
    }
  }
  if constexpr (!k8) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int d0 = (tid + i * G) * 8;
      uint16_t y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = round_once<T>(h[i][j]);
      for (int r = 0; r < a.repeat; ++r)
        store_raw<2>((uint16_t*)a.out + (t * a.repeat + r) * a.o_stride + d0, y, a.dim - d0);
    }
  } else {
    const int n_blocks = (a.dim + a.block - 1) / a.block;
    if (a.powers) {
      // a power of two does not change what is rounded: all the rest in 32 bits, with what is below gathered in the lowest
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int d0 = (tid + i * G) * 8;
        float q[8];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          q[j] = to_odd(h[i][j]);
          top = Most()(top, magnitude(q[j]));
        }
        top = Most()(top, (uint32_t)__shfl_xor((int)top, 1, 64));          // four neighbouring lanes hold a block
        top = Most()(top, (uint32_t)__shfl_xor((int)top, 2, 64));
        // the least power of two at which nothing passes 448 = 1.75 * 2^8
        int e = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u), -126);
        float by = __builtin_amdgcn_ldexpf(1.f, -e);
        bool bad = false;
        // From 64 bits where 32 do not hold the block, or where codes could come from numbers below their least normal one, 2^-126, which
        // have fewer bits (with a scale of 2^-115 or more those are below half the least code).  Four lanes are here together.
        constexpr uint32_t kLeast = (uint32_t)(127 - 115 + 8) << 23;
        if (top && top - kLeast >= 0x7F800000u - kLeast) {
          uint64_t all = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) all = Most()(all, magnitude(h[i][j]));
          all = Most()(all, (uint64_t)__shfl_xor(all, 1, 64));
          all = Most()(all, (uint64_t)__shfl_xor(all, 2, 64));
          bad = all >= 0x7FF0000000000000ull;
          e = bad ? 128 : max((int)(all >> 52) - 1023 - 8 + ((all & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull), -126);
          by = 1.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = to_odd(__builtin_amdgcn_ldexp(h[i][j], -e));
        }
        store_codes(a, t, d0, n_blocks, q, by, bad, (uint8_t)(e + 127));
      }
    } else {
      uint64_t top[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        top[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top[i] = Most()(top[i], magnitude(h[i][j]));
      }
      if (a.whole) {
        uint64_t all = top[0];
#pragma unroll
        for (int i = 1; i < kN; ++i) all = Most()(all, top[i]);
        all = over_row<Most, kFew>(all, (uint64_t*)s_sum, G);
#pragma unroll
        for (int i = 0; i < kN; ++i) top[i] = all;
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)                    // 16 neighbouring lanes hold a block
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) top[i] = Most()(top[i], (uint64_t)__shfl_xor(top[i], d, 64));
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const double most = __builtin_bit_cast(double, top[i]);
        const bool bad = !(most < (double)INFINITY);
        const float scale = fmaxf((float)(most / 448.), 0x1p-126f);
        const double unit = (double)scale, by = 1. / unit;
        float q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // a quotient that 64 bits hold, the middle between two codes among them, comes out as itself
          const double about = h[i][j] * by;
          q[j] = to_odd(fused(fused(-about, unit, h[i][j]), by, about));
        }
        store_codes(a, t, (tid + i * G) * 8, n_blocks, q, 1.f, bad, bad ? __builtin_nanf("") : scale);
      }
    }
  }
}

// Rows of a call: n of them, each `bytes` long, `stride` bytes apart.
struct Rows {
  const void* p;
  int64_t n, bytes, stride;
};

bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  const uintptr_t xe = x + (uintptr_t)((a.n - 1) * a.stride + a.bytes), ye = y + (uintptr_t)((b.n - 1) * b.stride + b.bytes);
  if (xe <= y || ye <= x) return false;
  if (a.stride != b.stride || a.stride < a.bytes + b.bytes) return true;
  // columns of one array: the second's begin behind the first's end in every row, and end before its next row
  const uintptr_t off = x <= y ? (y - x) % (uintptr_t)a.stride : (uintptr_t)a.stride - (x - y) % (uintptr_t)a.stride;
  return off < (uintptr_t)a.bytes || off + (uintptr_t)b.bytes > (uintptr_t)a.stride;
}

template <typename T, bool kXF, bool kRF, bool k8>
void launch_norm(NormArgs a, int32_t n_tokens, hipStream_t s) {
  // Eight elements a thread as long as a workgroup has that many threads.  8-bit results, which keep the vector units busy, take
  // sixteen from 256 threads on, so that more rows are in one CU (8192 rows of 4096: 55 instead of 61 us, 2080: 38 and 39); 16-bit
  // ones do not (4096: 54 instead of 50).
  const int chunks = (a.dim + 7) / 8, n = chunks > 2048 ? 4 : chunks > (k8 ? 256 : 1024) ? 2 : 1;
  // rows of up to 256 elements share a wave (65536 rows of 64: 10 instead of 34 us); 16 lanes at least have a block of 128
  a.lanes = ((chunks + n - 1) / n + 63) / 64 * 64;
  if (chunks <= 32)
    for (a.lanes = k8 ? 16 : 8; a.lanes < chunks;) a.lanes *= 2;
  const int rows = a.lanes < 64 ? kFewThreads / a.lanes : 1;
  const dim3 block((unsigned)(a.lanes * rows));
  for (; a.first < n_tokens; a.first += (int64_t)kMostGrid * rows) {
    const dim3 grid((unsigned)std::min<int64_t>((n_tokens - a.first + rows - 1) / rows, kMostGrid));
#define SBM_NORM(N, FEW) hipLaunchKernelGGL((norm_kernel<T, kXF, kRF, k8, N, FEW>), grid, block, 0, s, a)
    if (rows > 1) SBM_NORM(1, true);
    else if (n == 1) SBM_NORM(1, false);
    else if (n == 2) SBM_NORM(2, false);
    else SBM_NORM(4, false);
  }
#undef SBM_NORM
}

template <typename T>
void launch_norm(const NormArgs& a, int32_t n_tokens, uint32_t flags, hipStream_t s) {
  const bool xf = flags & SBM_F_IN_F32, rf = flags & SBM_F_RESIDUAL_F32, f8 = flags & SBM_F_OUT_FP8;
#define SBM_NORM(X, R, E) \
  if (xf == X && rf == R && f8 == E) launch_norm<T, X, R, E>(a, n_tokens, s)
  SBM_NORM(false, false, false);
  SBM_NORM(false, false, true);
  SBM_NORM(false, true, false);
  SBM_NORM(false, true, true);
  SBM_NORM(true, false, false);
  SBM_NORM(true, false, true);
  SBM_NORM(true, true, false);
  SBM_NORM(true, true, true);
#undef SBM_NORM
}

}  // namespace
}  // namespace sbm

using namespace sbm;

extern "C" int sbm_add_rms_norm(const sbm_norm_args* args, void* stream) {
  if (!args) return fail(SBM_EINVAL, "null pointer");
  const auto [x, x_stride, gates, residual, residual_stride, weight, residual_out, residual_out_stride, out, out_stride, scales, eps,
              n_tokens, dim, k, repeat, scale_block, flags] = *args;
  if (flags & ~(SBM_F_IN_BF16 | SBM_F_IN_F32 | SBM_F_RESIDUAL_F32 | SBM_F_OUT_FP8))
    return fail(SBM_EINVAL, "unknown flags 0x%x", flags);
  if (n_tokens < 0 || dim < 1 || dim > kMostDim)
    return fail(SBM_EINVAL, "bad n_tokens=%d or dim=%d (1..%d)", n_tokens, dim, kMostDim);
  if (k < 1 || k > 64 || repeat < 1 || repeat > 64) return fail(SBM_EINVAL, "k=%d or repeat=%d outside 1..64", k, repeat);
  if (!(eps >= 0.)) return fail(SBM_EINVAL, "bad eps");
  const bool xf = flags & SBM_F_IN_F32, rf = flags & SBM_F_RESIDUAL_F32, f8 = flags & SBM_F_OUT_FP8;
  if (f8 ? scale_block != 0 && scale_block != 32 && scale_block != 128 : scale_block != 0)
    return fail(SBM_EINVAL, "scale_block=%d is not 0, 32 or 128 (0 for 16-bit results)", scale_block);
  const int64_t most = (int64_t)1 << 40;
  if (x_stride < 0 || residual_stride < 0 || residual_out_stride < 0 || out_stride < 0 || x_stride > most ||
      residual_stride > most || residual_out_stride > most || out_stride > most)
    return fail(SBM_EINVAL, "bad row stride");
  if (n_tokens == 0) return SBM_OK;
  if (k > 1 && !gates) return fail(SBM_EINVAL, "k=%d rows of a token need gates", k);
  if (!x || !out || (f8 && !scales)) return fail(SBM_EINVAL, "null pointer");
  if ((n_tokens > 1 && ((residual_out && residual_out_stride < dim) || out_stride < dim)) || (repeat > 1 && out_stride < dim))
    return fail(SBM_EINVAL, "rows of a result overlap");
  const int32_t block = scale_block ? scale_block : dim;
  const int64_t xb = xf ? 4 : 2, rb = rf ? 4 : 2, ob = f8 ? 1 : 2, sb = scale_block == 32 ? 1 : 4;
  const int64_t n_blocks = (dim + block - 1) / block, T = n_tokens;
  if ((uintptr_t)x % xb || (uintptr_t)residual % rb || (uintptr_t)residual_out % rb ||
      (uintptr_t)weight % 2 || (uintptr_t)out % ob || (f8 && (uintptr_t)scales % sb) || (uintptr_t)gates % 4)
    return fail(SBM_EINVAL, "misaligned array");
  const Rows ins[] = {{x, T * k, dim * xb, x_stride * xb}, {residual, T, dim * rb, residual_stride * rb},
                      {weight, 1, dim * 2, 0}, {gates, 1, T * k * 4, 0}};
  const Rows outs[] = {{residual_out, T, dim * rb, residual_out_stride * rb}, {out, T * repeat, dim * ob, out_stride * ob},
                       {f8 ? scales : nullptr, 1, T * repeat * n_blocks * sb, 0}};
  // a row's workgroup has read the row before it writes
  const bool in_place = residual_out == residual && (residual_out_stride == residual_stride || T == 1);
  const bool over_x = out == x && k == 1 && repeat == 1 && xb == ob && (out_stride == x_stride || T == 1);
  for (const Rows& o : outs) {
    for (const Rows& i : ins)
      if (!(in_place && &o == outs && &i == ins + 1) && !(over_x && &o == outs + 1 && &i == ins) && overlap(o, i))
        return fail(SBM_EINVAL, "an output overlaps an input");
    for (const Rows& other : outs)
      if (&other < &o && overlap(o, other)) return fail(SBM_EINVAL, "outputs overlap");
  }
  const NormArgs a{x, residual, residual_out, weight, gates, out, scales, x_stride, residual_stride, residual_out_stride,
                   out_stride, 0, eps, dim, k, repeat, block, n_tokens, 0, scale_block == 0, scale_block == 32};
  if (flags & SBM_F_IN_BF16) launch_norm<__bf16>(a, n_tokens, flags, (hipStream_t)stream);
  else launch_norm<_Float16>(a, n_tokens, flags, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "add_rms_norm launch: %s", hipGetErrorString(e));
  return SBM_OK;
}
