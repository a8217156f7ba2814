// Routing of tokens to experts: scores, choice with a bias and groups, weights.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sbm_internal.h"
#include "sbm_num.h"

namespace sbm {
namespace {

constexpr int kMostExperts = 4096;
constexpr int kMostChosen = 32;
constexpr int kMostGroups = 64;
constexpr int kRThreads = 256;

struct RouteArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  const int32_t* requests;
  int32_t* ids;
  float* gates;
  uint32_t* error;
  float scale;
  int32_t n_tokens, n_experts, k, n_groups, top_groups, group_best;
  bool sigmoid, renorm;
};

template <typename T>
__device__ __forceinline__ float logit_at(const void* row, int e) {
  if constexpr (__is_same(T, float)) return ((const float*)row)[e];
  else return to_f32<T>(((const uint16_t*)row)[e]);
}

// The larger of two choices, of equal ones the lower expert; no choice is -inf with any expert.
struct Choice {
  double c;
  int e;
};
__device__ __forceinline__ Choice better(Choice a, Choice b) { return b.c > a.c || (b.c == a.c && b.e < a.e) ? b : a; }
__device__ __forceinline__ Choice best_of_wave(Choice v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = better(v, Choice{__shfl_xor(v.c, d, 64), __shfl_xor(v.e, d, 64)});
  return v;
}

// A wave has a token, kN experts a lane (expert i * 64 + lane).
template <typename T, int kN>
__global__ __launch_bounds__(kRThreads) void route_kernel(RouteArgs a) {
  const int lane = (int)threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (kRThreads / 64) + (threadIdx.x >> 6);
  if (t >= a.n_tokens) return;
  const double kNone = -(double)INFINITY;
  int32_t* ids = a.ids + t * a.k;
  float* gates = a.gates + t * a.k;
  if (a.requests && a.requests[t] < 0) {
    if (lane < a.k) ids[lane] = -1, gates[lane] = 0.f;
    return;
  }
  const char* row = (const char*)a.logits + t * a.stride * (__is_same(T, float) ? 4 : 2);
  double s[kN], c[kN], most = kNone;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int e = i * 64 + lane;
    const float l = e < a.n_experts ? logit_at<T>(row, e) : -INFINITY;
    bad = bad || !(l < INFINITY);
    s[i] = (double)l;
    most = fmax(most, s[i]);
  }
  double sum = 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmax(most, __shfl_xor(most, d, 64));
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    c[i] = s[i];
    if (a.sigmoid) s[i] = 1. / (1. + exp(-s[i]));
    else s[i] = s[i] == kNone ? 0. : exp(s[i] - most);
    sum += s[i];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (!a.sigmoid) s[i] = sum > 0 ? s[i] / sum : 0.;
    if (a.bias && c[i] != kNone) {
      c[i] = s[i] + (double)a.bias[i * 64 + lane];
      bad = bad || !(c[i] < (double)INFINITY);
    }
  }
  if (__any(bad)) {
    if (lane < a.k) ids[lane] = -1, gates[lane] = 0.f;
    if (lane == 0 && a.error) atomicAdd(a.error, 1u);
    return;
  }
  if (a.n_groups > 1) {
    // a group's value: the sum of its largest choices (scores where there is no bias); lane g keeps group g's
    const int per = a.n_experts / a.n_groups;
    double mine = kNone;
    for (int g = 0; g < a.n_groups; ++g) {
      double value = kNone;
      int taken = -1;
      for (int b = 0; b < a.group_best; ++b) {
        Choice v{kNone, kMostExperts};
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int e = i * 64 + lane;
          if (e >= g * per && e < (g + 1) * per && e != taken && c[i] != kNone) v = better(v, Choice{a.bias ? c[i] : s[i], e});
        }
        v = best_of_wave(v);
        if (v.c == kNone) break;
        value = b ? value + v.c : v.c;
        taken = v.e;
      }
      if (lane == g) mine = value;
    }
    // the groups that stay, as bits
    uint64_t stay = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const Choice v = best_of_wave(Choice{(stay >> lane) & 1 ? kNone : mine, lane});
      if (v.c == kNone) break;
      stay |= 1ull << v.e;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = i * 64 + lane;
      if (e < a.n_experts && !((stay >> (e / per)) & 1)) c[i] = kNone;
    }
  }
  // the k best in turn; lane j keeps the j-th
  int my_id = -1;
  double my_score = 0, total = 0;
  for (int j = 0; j < a.k; ++j) {
    Choice v{kNone, kMostExperts};
#pragma unroll
    for (int i = 0; i < kN; ++i) v = better(v, Choice{c[i], i * 64 + lane});
    v = best_of_wave(v);
    if (v.c == kNone) break;
    double score = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (i * 64 + lane == v.e) {
        c[i] = kNone;
        score = s[i];
      }
    }
    score = __shfl(score, v.e & 63, 64);
    total += score;
    if (lane == j) my_id = v.e, my_score = score;
  }
  if (lane < a.k) {
    double g = my_score;
    if (a.renorm && total > 0) g /= total;
    ids[lane] = my_id;
    gates[lane] = (float)(g * (double)a.scale);
  }
}

template <typename T>
void launch_route(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.n_tokens + kRThreads / 64 - 1) / (kRThreads / 64))), block(kRThreads);
#define SBM_ROUTE(N) hipLaunchKernelGGL((route_kernel<T, N>), grid, block, 0, s, a)
  if (a.n_experts <= 64) SBM_ROUTE(1);
  else if (a.n_experts <= 128) SBM_ROUTE(2);
  else if (a.n_experts <= 256) SBM_ROUTE(4);
  else if (a.n_experts <= 512) SBM_ROUTE(8);
  else if (a.n_experts <= 1024) SBM_ROUTE(16);
  else if (a.n_experts <= 2048) SBM_ROUTE(32);
  else SBM_ROUTE(64);
#undef SBM_ROUTE
}

bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

}  // namespace
}  // namespace sbm

using namespace sbm;

extern "C" int sbm_moe_route(const void* logits, int64_t row_stride, const float* bias, const int32_t* requests,
                             int32_t n_tokens, int32_t n_experts, int32_t k, int32_t n_groups, int32_t top_groups,
                             int32_t group_best, float scale, int32_t* ids, float* gates, uint32_t flags, uint32_t* error,
                             void* stream) {
  if (flags & ~(SBM_F_IN_BF16 | SBM_F_IN_F32 | SBM_F_SIGMOID | SBM_F_RENORM)) return fail(SBM_EINVAL, "unknown flags 0x%x", flags);
  if ((flags & SBM_F_IN_BF16) && (flags & SBM_F_IN_F32)) return fail(SBM_EINVAL, "logits of two types");
  if (n_tokens < 0 || n_experts < 1 || n_experts > kMostExperts)
    return fail(SBM_EINVAL, "bad n_tokens=%d or n_experts=%d (1..%d)", n_tokens, n_experts, kMostExperts);
  if (n_groups < 1 || n_groups > kMostGroups || n_experts % n_groups || top_groups < 1 || top_groups > n_groups)
    return fail(SBM_EINVAL, "n_groups=%d (1..%d, a divisor of n_experts=%d) or top_groups=%d does not fit", n_groups, kMostGroups,
                n_experts, top_groups);
  if (group_best != 1 && group_best != 2) return fail(SBM_EINVAL, "group_best=%d is not 1 or 2", group_best);
  if (k < 1 || k > kMostChosen || k > n_experts / n_groups * top_groups)
    return fail(SBM_EINVAL, "k=%d outside 1..%d or above the %d experts of %d groups", k, kMostChosen,
                n_experts / n_groups * top_groups, top_groups);
  const int64_t size = flags & SBM_F_IN_F32 ? 4 : 2;
  if (row_stride < 0 || row_stride > ((int64_t)1 << 40)) return fail(SBM_EINVAL, "bad row_stride");
  if (!(scale - scale == 0.f)) return fail(SBM_EINVAL, "bad scale");
  if (n_tokens == 0) return SBM_OK;
  if (!logits || !ids || !gates) return fail(SBM_EINVAL, "null pointer");
  if ((uintptr_t)logits % size || ((uintptr_t)bias | (uintptr_t)requests | (uintptr_t)ids | (uintptr_t)gates | (uintptr_t)error) % 4)
    return fail(SBM_EINVAL, "misaligned array");
  const int64_t n = 4 * (int64_t)n_tokens * k;
  const struct {
    const void* p;
    int64_t bytes;
  } ins[] = {{logits, ((n_tokens - 1) * row_stride + n_experts) * size}, {bias, 4 * (int64_t)n_experts}, {requests, 4 * (int64_t)n_tokens}};
  for (const auto& i : ins)
    if (overlap(ids, n, i.p, i.bytes) || overlap(gates, n, i.p, i.bytes) || overlap(error, 4, i.p, i.bytes))
      return fail(SBM_EINVAL, "an output overlaps an input");
  if (overlap(ids, n, gates, n) || overlap(error, 4, ids, n) || overlap(error, 4, gates, n)) return fail(SBM_EINVAL, "outputs overlap");
  const RouteArgs a{logits, row_stride, bias, requests, ids, gates, error, scale, n_tokens, n_experts, k, n_groups, top_groups,
                    group_best, (flags & SBM_F_SIGMOID) != 0, (flags & SBM_F_RENORM) != 0};
  if (flags & SBM_F_IN_F32) launch_route<float>(a, (hipStream_t)stream);
  else if (flags & SBM_F_IN_BF16) launch_route<__bf16>(a, (hipStream_t)stream);
  else launch_route<_Float16>(a, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "moe_route launch: %s", hipGetErrorString(e));
  return SBM_OK;
}
