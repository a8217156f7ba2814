// The next token: temperature, top-k, min-p and top-p, and the draw by a given number.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sbm_internal.h"
#include "sbm_num.h"

namespace sbm {
namespace {

constexpr int kMostVocab = 1 << 20;
constexpr int kSThreads = 1024;
constexpr int kSWaves = kSThreads / 64;

struct SampleArgs {
  const void* logits;
  int64_t stride;
  const float *uniforms, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* logprobs;
  uint32_t* error;
  int32_t vocab;
};

// Weights are whole numbers of 2^-42, so that their sums (at most 2^20 of at most 1) do not depend on an order.
constexpr double kUnit = 0x1p42;

template <typename T>
__device__ __forceinline__ float logit_at(const void* row, int i) {
  if constexpr (__is_same(T, float)) return ((const float*)row)[i];
  else return to_f32<T>(((const uint16_t*)row)[i]);
}

// 32 bits that order as the numbers do; both zeros are one.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Exclusive sums over the workgroup's threads, and the whole.
__device__ __forceinline__ uint64_t scan(uint64_t v, uint64_t* waves, uint64_t* all) {
  const int lane = (int)threadIdx.x & 63;
  uint64_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) waves[threadIdx.x >> 6] = x;
  __syncthreads();
  uint64_t before = 0, sum = 0;
  for (int w = 0; w < kSWaves; ++w) {
    if (w < (int)(threadIdx.x >> 6)) before += waves[w];
    sum += waves[w];
  }
  *all = sum;
  return before + x - v;
}

// A row's parameters.  Tokens are ordered by falling logit, equal ones by rising index; every filter keeps a beginning of
// that order: the tokens above `key`, and the first `ties` of those at it, with a weight of at least `least`.
struct Row {
  double most, least;
  uint32_t key;
  uint32_t ties;
};

template <typename T>
__global__ __launch_bounds__(kSThreads) void sample_kernel(SampleArgs a) {
  __shared__ uint64_t s_sum[256], s_waves[kSWaves];
  __shared__ uint32_t s_count[256], s_bad, s_key;
  __shared__ uint64_t s_found[4];
  const int tid = (int)threadIdx.x, V = a.vocab;
  const int64_t r = blockIdx.x;
  const char* row = (const char*)a.logits + r * a.stride * (__is_same(T, float) ? 4 : 2);
  const float u = a.uniforms[r], temperature = a.temperature ? a.temperature[r] : 1.f;
  const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
  const int32_t top_k = a.top_k ? a.top_k[r] : 0;
  if (tid == 0) s_bad = u != u || !(temperature >= 0.f) || top_p != top_p || min_p != min_p, s_key = 0;
  __syncthreads();
  // the largest
  uint32_t key = 0, bad = 0;
  for (int i = tid; i < V; i += kSThreads) {
    const float l = logit_at<T>(row, i);
    if (!(l < INFINITY)) bad = 1;
    else key = max(key, key_of(l));
  }
  if (bad) atomicOr(&s_bad, 1u);
  atomicMax(&s_key, key);
  __syncthreads();
  key = s_key;
  const uint32_t none = key_of(-INFINITY);
  if (s_bad || key == none) {
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.logprobs) a.logprobs[r] = __builtin_nanf("");
      if (a.error) atomicAdd(a.error, 1u);
    }
    return;
  }
  const float most = __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
  Row f{(double)most, min_p > 0.f ? fmin((double)min_p, 1.) : 0., none + 1, ~0u};
  if (temperature == 0.f) f.key = key, f.ties = 1;
  const auto weight = [&](float l) { return exp(((double)l - f.most) / (double)temperature); };
  const auto units = [&](float l) { return temperature == 0.f ? (uint64_t)kUnit : (uint64_t)rint(weight(l) * kUnit); };

  // For each bit group of the key: where the running count (or sum) from above reaches `target`.
  const auto descend = [&](bool sums, uint64_t target) {
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (tid < 256) s_sum[tid] = 0, s_count[tid] = 0;
      __syncthreads();
      for (int i = tid; i < V; i += kSThreads) {
        const float l = logit_at<T>(row, i);
        const uint32_t k = key_of(l);
        if (k < f.key || (shift < 24 && (k >> (shift + 8)) != (prefix >> (shift + 8)))) continue;
        const double w = f.least > 0. ? weight(l) : 1.;
        if (w < f.least) continue;
        atomicAdd(&s_count[(k >> shift) & 255u], 1u);
        if (sums) atomicAdd((unsigned long long*)&s_sum[(k >> shift) & 255u], (unsigned long long)units(l));
      }
      __syncthreads();
      if (tid == 0) {
        int b = 255;
        uint64_t have = 0;
        for (; b > 0; --b) {
          const uint64_t more = sums ? s_sum[b] : s_count[b];
          if (have + more >= target) break;
          have += more;
        }
        s_found[0] = (uint64_t)b;
        s_found[1] = target - have;
        s_found[2] = s_count[b];
        s_found[3] = have + (sums ? s_sum[b] : s_count[b]) < target;
      }
      __syncthreads();
      if (s_found[3]) return;                           // fewer than that: all stay
      prefix |= (uint32_t)s_found[0] << shift;
      target = s_found[1];
    }
    const uint64_t n = s_found[2];
    f.ties = prefix == f.key ? f.ties : ~0u;
    f.key = prefix;
    if (sums) {
      const uint32_t u = prefix & 0x80000000u ? prefix ^ 0x80000000u : ~prefix;
      const uint64_t w = units(__uint_as_float(u));
      target = w ? (target + w - 1) / w : n;
    }
    f.ties = (uint32_t)min((uint64_t)f.ties, min(target, n));
  };

  // Each thread has a run of neighbouring tokens: ties are counted, and weights summed, in the tokens' order.
  const int per = (V + kSThreads - 1) / kSThreads, i0 = min(V, tid * per), i1 = min(V, i0 + per);
  uint64_t ties_before = 0, before = 0, total = 0;
  const auto kept = [&](float l, uint64_t& ties) {
    const uint32_t k = key_of(l);
    if (k < f.key || weight(l) < f.least) return false;
    return k > f.key || ties++ < f.ties;
  };
  const auto sum_up = [&]() {
    uint64_t n = 0, sum = 0, all;
    for (int i = i0; i < i1; ++i) n += key_of(logit_at<T>(row, i)) == f.key;
    ties_before = scan(n, s_waves, &all);
    uint64_t ties = ties_before;
    for (int i = i0; i < i1; ++i) {
      const float l = logit_at<T>(row, i);
      if (kept(l, ties)) sum += units(l);
    }
    before = scan(sum, s_waves, &total);
  };

  if (temperature > 0.f) {
    if (top_k > 0 && top_k < V) descend(false, (uint64_t)top_k);
    if (top_p < 1.f) {
      sum_up();
      const double want = ceil(fmax((double)top_p, 0.) * (double)total);
      descend(true, max((uint64_t)want, (uint64_t)1));
    }
  }
  sum_up();
  // the first token whose running sum passes u * total
  const uint64_t at = min((uint64_t)(fmin(fmax((double)u, 0.), 1.) * (double)total), total - 1);
  uint64_t ties = ties_before, upto = before;
  for (int i = i0; i < i1 && upto <= at; ++i) {
    const float l = logit_at<T>(row, i);
    if (!kept(l, ties)) continue;
    upto += units(l);
    if (upto > at && before <= at) {
      a.tokens[r] = i;
      if (a.logprobs)
        a.logprobs[r] = temperature == 0.f ? 0.f : (float)(((double)l - f.most) / (double)temperature - log((double)total / kUnit));
    }
  }
}

bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

}  // namespace
}  // namespace sbm

using namespace sbm;

extern "C" {

size_t sbm_sample_workspace_bytes(int32_t n_rows, int32_t vocab) {
  if (n_rows < 0 || vocab < 1 || vocab > kMostVocab) return 0;
  return 256;
}

int sbm_sample(const void* logits, int64_t row_stride, int32_t n_rows, int32_t vocab, const float* uniforms,
               const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
               float* logprobs, uint32_t flags, void* workspace, size_t workspace_bytes, uint32_t* error, void* stream) {
  if (flags & ~(SBM_F_IN_BF16 | SBM_F_IN_F32)) return fail(SBM_EINVAL, "unknown flags 0x%x", flags);
  if ((flags & SBM_F_IN_BF16) && (flags & SBM_F_IN_F32)) return fail(SBM_EINVAL, "logits of two types");
  if (n_rows < 0 || vocab < 1 || vocab > kMostVocab)
    return fail(SBM_EINVAL, "bad n_rows=%d or vocab=%d (1..%d)", n_rows, vocab, kMostVocab);
  if (row_stride < 0 || row_stride > ((int64_t)1 << 40)) return fail(SBM_EINVAL, "bad row_stride");
  if (n_rows == 0) return SBM_OK;
  if (!logits || !uniforms || !tokens || !workspace) return fail(SBM_EINVAL, "null pointer");
  const int64_t size = flags & SBM_F_IN_F32 ? 4 : 2, n = 4 * (int64_t)n_rows;
  if ((uintptr_t)logits % size || ((uintptr_t)uniforms | (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p |
                                   (uintptr_t)min_p | (uintptr_t)tokens | (uintptr_t)logprobs | (uintptr_t)error) % 4)
    return fail(SBM_EINVAL, "misaligned array");
  if ((uintptr_t)workspace % 16) return fail(SBM_EINVAL, "workspace must be 16-byte aligned");
  const size_t need = sbm_sample_workspace_bytes(n_rows, vocab);
  if (workspace_bytes < need) return fail(SBM_ENOSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
  const struct {
    const void* p;
    int64_t bytes;
  } ins[] = {{logits, ((n_rows - 1) * row_stride + vocab) * size}, {uniforms, n}, {temperature, n}, {top_k, n}, {top_p, n}, {min_p, n}},
    outs[] = {{tokens, n}, {logprobs, n}, {workspace, (int64_t)need}, {error, 4}};
  for (const auto& o : outs) {
    for (const auto& i : ins)
      if (overlap(o.p, o.bytes, i.p, i.bytes)) return fail(SBM_EINVAL, "an output overlaps an input");
    for (const auto& other : outs)
      if (&other < &o && overlap(o.p, o.bytes, other.p, other.bytes)) return fail(SBM_EINVAL, "outputs overlap");
  }
  const SampleArgs a{logits, row_stride, uniforms, temperature, top_p, min_p, top_k, tokens, logprobs, error, vocab};
  const dim3 grid((unsigned)n_rows), block(kSThreads);
  hipStream_t s = (hipStream_t)stream;
  if (flags & SBM_F_IN_F32) hipLaunchKernelGGL((sample_kernel<float>), grid, block, 0, s, a);
  else if (flags & SBM_F_IN_BF16) hipLaunchKernelGGL((sample_kernel<__bf16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((sample_kernel<_Float16>), grid, block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "sample launch: %s", hipGetErrorString(e));
  return SBM_OK;
}

}  // extern "C"
