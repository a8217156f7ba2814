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

constexpr int kRWaves = kRThreads / 64;

template <typename T>
__device__ __forceinline__ float logit_at(const void* row, int e) {
  if constexpr (__is_same(T, float)) return ((const float*)row)[e];
  else return to_f32<T>(((const uint16_t*)row)[e]);
}

// What a lane has of a token's kN * 64 experts: runs of four neighbours (single ones up to 128 experts), so that a wave reads
// whole lines.
template <int kN>
__device__ __forceinline__ int expert(int i, int lane) {
  if constexpr (kN < 4) return i * 64 + lane;
  else return (i >> 2) * 256 + lane * 4 + (i & 3);
}

// The elements of a row as they are in memory; `none` behind its end.
template <typename T, int kN>
struct Row {
  static constexpr int kWords = __is_same(T, float) ? kN : (kN + 1) / 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* row, int n, uint32_t none, int lane) {
    constexpr bool kF = __is_same(T, float);
    if constexpr (kN < 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int e = expert<kN>(i, lane);
        uint32_t u = none;
        if (e < n) u = kF ? ((const uint32_t*)row)[e] : ((const uint16_t*)row)[e];
        if constexpr (kF) w[i] = u;
        else w[i >> 1] = i & 1 ? w[i >> 1] | u << 16 : u;
      }
    } else {
      // a run that passes the end is read from the row's last four elements (there are more than 128), then moved down
#pragma unroll
      for (int i = 0; i < kN; i += 4)
        __builtin_memcpy(&w[kF ? i : i / 2], (const char*)row + min(expert<kN>(i, lane), n - 4) * (kF ? 4 : 2), kF ? 16 : 8);
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        if (i / 4 * 256 + 256 <= n) continue;
        const int past = expert<kN>(i, lane) - (n - 4);
        if constexpr (kF) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool move = past > j;
            w[i] = move ? w[i + 1] : w[i];
            w[i + 1] = move ? w[i + 2] : w[i + 1];
            w[i + 2] = move ? w[i + 3] : w[i + 2];
            w[i + 3] = move ? none : w[i + 3];
          }
        } else {
          const uint64_t all = none * 0x0001000100010001ull, v = (uint64_t)w[i / 2 + 1] << 32 | w[i / 2];
          const int by = 16 * max(past, 0);
          const uint64_t u = by >= 64 ? all : by == 0 ? v : v >> by | all << (64 - by);
          w[i / 2] = (uint32_t)u;
          w[i / 2 + 1] = (uint32_t)(u >> 32);
        }
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (__is_same(T, float)) return __uint_as_float(w[i]);
    else return to_f32<T>((uint16_t)(w[i >> 1] >> 16 * (i & 1)));
  }
};

// 2^x, to 2^-22 of itself.
__device__ __forceinline__ float exp2_f32(float x) { return __builtin_amdgcn_exp2f(x); }
constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596303e-8f;     // log2(e) and what is left of it

// 2^x as 64 bits hold it, below 2^-1000 as well, which exp2_f64 does not go: as a denormal, or 0 where there is none.
__device__ __forceinline__ double exp2_any(double x) {
  double y = exp2_f64(x);
  if (__any(x < -1000.)) y = x < -1000. ? exp2_f64(x + 200.) * 0x1p-200 : y;
  return y;
}

// A score of an expert's logit in 64 bits; most, sum: the softmax's.  Where e^-l is no number of 64 bits the sigmoid is 0.
__device__ __forceinline__ double score_of(const RouteArgs& a, float l, float most, double sum) {
  constexpr double kLog2e64 = 1.4426950408889634;
  if (!a.sigmoid) return exp2_any(((double)l - (double)most) * kLog2e64) * inverse(sum);
  const double x = -(double)l * kLog2e64;
  if (__any(x > 1000.)) return x >= 1024. ? 0. : x > 1000. ? exp2_any(-x) : inverse(1. + exp2_f64(x));
  return inverse(1. + exp2_f64(x));
}

// e^(l - most) in 32 bits, and the sum over a wave's experts: fours in 32 bits, those in 64.  An exponent's roundings come
// to 2^-23 of it, the rest to 6 of 2^-24: less than 2^-19 of the sum (the weights' average exponent is 8 at most), mostly less than 2^-24.
// (The exponentials in 64 bits took 40 instead of 26 us for 16384 x 2048, and 71 instead of 34 with a bias.)
__device__ __forceinline__ float weight_f32(float l, float most) {
  const float d = l - most;
  return exp2_f32(fused(d, kLog2e, d * kLog2eLow));
}
template <int kN, typename F>
__device__ __forceinline__ double sum_f32(F w) {
  double sum = 0;
#pragma unroll
  for (int i = 0; i < kN; i += 4) {
    float part;
    if constexpr (kN == 1) part = w(0);
    else if constexpr (kN == 2) part = w(0) + w(1);
    else {
      const float a = w(i), b = w(i + 1), c = w(i + 2);
      part = (a + b) + (c + w(i + 3));
    }
    sum += (double)part;
  }
  return wave_sum(sum);
}

// The softmax's sum in 64 bits.
template <typename T>
__device__ double sum_of(const RouteArgs& a, const void* row, float most) {
  double sum = 0;
  for (int e = (int)threadIdx.x & 63; e < a.n_experts; e += 64) {
    const float l = logit_at<T>(row, e);
    sum += l == -INFINITY ? 0. : score_of(a, l, most, 1.);
  }
  return wave_sum(sum);
}

// The larger of two choices, of equal ones the lower expert.
struct Choice {
  double c;
  int e;
};
__device__ __forceinline__ bool before(Choice a, Choice b) { return a.c > b.c || (a.c == b.c && a.e < b.e); }
__device__ __forceinline__ Choice best_of_wave(Choice v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const Choice o{__shfl_xor(v.c, d, 64), __shfl_xor(v.e, d, 64)};
    if (before(o, v)) v = o;
  }
  return v;
}

// As many neighbouring lanes for each group as a wave has.
__device__ __forceinline__ int lanes_of(int n_groups) {
  int lanes = 1;
  while (2 * lanes * n_groups <= 64) lanes *= 2;
  return lanes;
}

// A group's value, and how large the choices are that it is the sum of: what it may be off by goes by those, not by what is left
// of them.
template <typename C>
struct Group {
  C value, size;
};

// The groups that stay, as bits, from what the groups' lanes have; `near`: whether one that stays and one that does not are too near
// to tell apart, where a value may be off by `off` and by roundings of what it is the sum of.
template <typename C>
__device__ __forceinline__ uint64_t best_groups(const RouteArgs& a, Group<C> v, int lanes, C off, bool* near) {
  const int lane = (int)threadIdx.x & 63, g = lane / lanes;
  int place = 0;
  for (int h = 0; h < a.n_groups; ++h) {
    const C o = of_lane(v.value, h * lanes);
    place += o > v.value || (o == v.value && h < g);
  }
  const bool is = g < a.n_groups && lane % lanes == 0 && v.value > -(C)INFINITY;
  const uint64_t kept = __ballot(is && place < a.top_groups);
  if (near) {
    // two choices and their sum, each rounded to 2^-24 of itself, and the additions here
    const float by = (float)(off + (C)0x1p-22f * v.size);
    const float least = -wave_max(is && place < a.top_groups ? by - (float)v.value : -INFINITY);
    const float next = wave_max(is && place >= a.top_groups ? (float)v.value + by : -INFINITY);
    *near = next > -INFINITY && !(least > next);
  }
  uint64_t stay = 0;
  for (uint64_t m = kept; m; m &= m - 1) stay |= 1ull << (__builtin_ctzll(m) / lanes);
  return stay;
}

// What a lane's group is worth, from its two largest choices.
template <typename C, typename F>
__device__ __forceinline__ Group<C> group_value(const RouteArgs& a, int lanes, F choice) {
  const int lane = (int)threadIdx.x & 63, g = lane / lanes, per = a.n_experts / a.n_groups;
  C one = -(C)INFINITY, two = one;
  if (g < a.n_groups) {
    for (int e = lane % lanes; e < per; e += lanes) {
      const C v = choice(g * per + e), less = one < v ? one : v;
      two = two > less ? two : less;
      one = one > v ? one : v;
    }
  }
  for (int d = 1; d < lanes; d <<= 1) {
    const C o1 = __shfl_xor(one, d, 64), o2 = __shfl_xor(two, d, 64), less = one < o1 ? one : o1;
    two = two > o2 ? two : o2;
    two = two > less ? two : less;
    one = one > o1 ? one : o1;
  }
  const C first = one < 0 ? -one : one;
  if (a.group_best == 2 && two > -(C)INFINITY) {
    // a sum past the type's lowest is a group still; its size says that it cannot be told from others
    const C sum = one + two;
    return Group<C>{sum > -(C)INFINITY ? sum : -(C)3.402823466e38f, first + (two < 0 ? -two : two)};
  }
  return Group<C>{one, first};
}

template <typename T>
__device__ uint64_t groups_exactly(const RouteArgs& a, const void* row, float most) {
  const double sum = a.sigmoid ? 1. : sum_of<T>(a, row, most);
  const int lanes = lanes_of(a.n_groups);
  const Group<double> value = group_value<double>(a, lanes, [&](int e) {
    const float l = logit_at<T>(row, e);
    return l == -INFINITY ? -(double)INFINITY : score_of(a, l, most, sum) + (a.bias ? (double)a.bias[e] : 0.);
  });
  return best_groups(a, value, lanes, 0., nullptr);
}

// The choice of a token's experts in 64 bits, where more are beside each other than a wave has lanes: lane j has the j-th expert, or
// -1.  Nothing is kept, so that it takes few registers: every round computes the scores again.
template <typename T>
__device__ int choose_exactly(const RouteArgs& a, const void* row, float most) {
  const int lane = (int)threadIdx.x & 63, per = a.n_groups > 1 ? a.n_experts / a.n_groups : kMostExperts;
  const double kNone = -(double)INFINITY;
  const double sum = a.sigmoid ? 1. : sum_of<T>(a, row, most);
  const uint64_t stay = a.n_groups > 1 ? groups_exactly<T>(a, row, most) : ~0ull;
  int id = -1;
  Choice last{(double)INFINITY, -1};
  for (int j = 0; j < a.k; ++j) {
    Choice v{kNone, kMostExperts};
    for (int e = lane; e < a.n_experts; e += 64) {
      const float l = logit_at<T>(row, e);
      if (l == -INFINITY || !((stay >> (e / per)) & 1)) continue;
      const Choice o{a.bias ? score_of(a, l, most, sum) + (double)a.bias[e] : (double)l, e};
      if (o.c > kNone && before(last, o) && before(o, v)) v = o;
    }
    v = best_of_wave(v);
    if (v.c == kNone) break;
    if (lane == j) id = v.e;
    last = v;
  }
  return id;
}

// Lanes' space in LDS for a wave: tokens' candidates, and choices by expert for the groups' sums.
template <int kN, bool kGroups>
struct WaveSpace {
  uint64_t order[64];
  float choice[kGroups ? kN * 64 : 1];
};

// A wave takes tokens, and has all of one in its lanes.  The k best: the (k + 1)-th largest of the lanes' largest choices is not
// above the (k + 1)-th largest of all, so what is not below it (some k + 1 experts) holds those; they go to LDS, a lane each, and
// are put in order.  Choices with a bias are compared in 32 bits, with what these may be off added to the candidates; where two
// that follow each other are nearer than that (one token in some hundred to some thousand), the candidates' choices are computed
// in 64, as the groups' values are where two at the border are.  With more than 64 candidates the whole token is.
// What bounds it: 16384 x 2048 in fp32 (134 MB) takes 33 to 40 us from one allocation to another (26 us of memory at its copy's rate,
// which it reaches without a bias): a token's choices fill the registers, so that four waves are in a SIMD, their vector units busy for
// 72 %, and all of them wait for rows at about the same time; with room for five or six the registers spill (39.6 and 57.8 us beside
// 35.3), the next token's row read ahead takes the room of a wave (67 us, when this took 50), and by way of LDS it was slower (40
// beside 37).  8192 x 256 in groups: 18.3 us, vector units 83 %.  64 x 2048: 4.9 us, one token's latency.  Where more than 64 choices are
// the same within what 32 bits tell apart, choose_exactly looks k times at the row: 16384 x 2048 of equal logits 212 us, with a bias
// 289, in groups 542; 64 x 2048 36, 50 and 80.
template <typename T, int kN, bool kGroups>
__global__ __launch_bounds__(kRThreads, kN > 32 ? 2 : 4) void route_kernel(RouteArgs a) {
  __shared__ WaveSpace<kN, kGroups> s_space[kRWaves];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  WaveSpace<kN, kGroups>& s = s_space[wave];
  constexpr uint32_t kNoneBits = __is_same(T, float) ? 0xFF800000u : __is_same(T, __bf16) ? 0xFF80u : 0xFC00u;
  constexpr int kSize = __is_same(T, float) ? 4 : 2;
  // The bias goes to LDS once (16384 x 2048: 36.7 us, from memory for each token 49), unless groups' choices leave too little room
  // there for four workgroups in a CU (16384 x 2048 in groups: 109 us and from memory 92, now 85).
  // One that is no number or +inf refuses the tokens that it could be chosen for.
  constexpr bool kHere = !kGroups || kN < 32;
  __shared__ alignas(16) float s_bias[kHere ? kN * 64 : 1];
  bool odd = false;
  if (a.bias) {
    for (int e = (int)threadIdx.x; e < (kHere ? kN * 64 : a.n_experts); e += kRThreads) {
      const float b = e < a.n_experts ? a.bias[e] : 0.f;
      odd = odd || !(b < INFINITY);
      if constexpr (kHere) s_bias[e] = b;
    }
    odd = __syncthreads_or(odd);
  }
  const int64_t step = (int64_t)gridDim.x * kRWaves;
  for (int64_t t = (int64_t)blockIdx.x * kRWaves + wave; t < a.n_tokens; t += step) {
    const char* row = (const char*)a.logits + t * a.stride * kSize;
    // what depends on it is made anew for each token: kept, it would fill the registers
    int lane = (int)threadIdx.x & 63;
    asm("" : "+v"(lane));
    Row<T, kN> x;
    x.load(row, a.n_experts, kNoneBits, lane);
    const bool padding = a.requests && a.requests[t] < 0;
    float most = x[0], low = x[0];
    bool bad = !(x[0] < INFINITY);
#pragma unroll
    for (int i = 1; i < kN; ++i) {
      most = fmaxf(most, x[i]);
      low = fminf(low, x[i]);
    }
    most = wave_max(most);
    // else the softmax's sum tells, unless there is nothing but -inf beside
    if (a.sigmoid || (!a.bias && !kGroups && a.renorm) || most == -INFINITY) {
#pragma unroll
      for (int i = 1; i < kN; ++i) bad = bad || x[i] != x[i];
    }
    bad = __any(bad) || most == INFINITY;
    const bool masked = __any(low == -INFINITY);
    uint32_t hidden[(kN + 31) / 32] = {};    // a bit for each -inf, so that the logits need not be kept beside the choices
    if (masked) {
#pragma unroll
      for (int i = 0; i < kN; ++i) hidden[i / 32] |= (x[i] == -INFINITY ? 1u : 0u) << (i % 32);
    }
    __builtin_amdgcn_sched_barrier(0);       // steps mixed with one another would take more registers than there are
    // choices
    float c[kN];
    double z = 1.;
    float score_most = 1.f;
    if (a.bias || kGroups) {
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < kN; ++i) c[i] = __builtin_amdgcn_rcpf(1.f + exp2_f32(-x[i] * kLog2e));
      } else {
        z = sum_f32<kN>([&](int i) { return c[i] = weight_f32(x[i], most); });
        score_most = 1.f / (float)z;
      }
      const float by = a.sigmoid ? 1.f : score_most;
      __builtin_amdgcn_sched_barrier(0);
      if (a.bias) {
        if constexpr (kHere) {
#pragma unroll
          for (int i = 0; i < kN; ++i) c[i] = fused(c[i], by, s_bias[expert<kN>(i, lane)]);
        } else {
          Row<float, kN> bias;
          bias.load(a.bias, a.n_experts, 0u, lane);
#pragma unroll
          for (int i = 0; i < kN; ++i) c[i] = fused(c[i], by, bias[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) c[i] *= by;
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < kN; ++i) c[i] = (hidden[i / 32] >> (i % 32)) & 1u ? -INFINITY : c[i];
      }
      if (odd) {
#pragma unroll
        for (int i = 0; i < kN; ++i) bad = bad || !(c[i] < INFINITY);
        bad = __any(bad);
      }
    } else {
      if (!a.sigmoid && !a.renorm) z = sum_f32<kN>([&](int i) { return weight_f32(x[i], most); });
#pragma unroll
      for (int i = 0; i < kN; ++i) c[i] = x[i];
    }
    bad = bad || (z != z && most > -INFINITY);
    if (bad || padding) {
      if (lane < a.k) a.ids[t * a.k + lane] = -1, a.gates[t * a.k + lane] = 0.f;
      if (!padding && lane == 0 && a.error) atomicAdd(a.error, 1u);
      continue;
    }
    __builtin_amdgcn_sched_barrier(0);
    // more than what two scores may be off together: exponentials of numbers rounded to 32 bits, and their sum's
    const float off = a.sigmoid ? 0x1p-19f : 0x1p-17f * score_most;
    uint64_t stay = ~0ull;
    const int per = kGroups ? a.n_experts / a.n_groups : 1;
    if constexpr (kGroups) {
#pragma unroll
      for (int i = 0; i < kN; ++i) s.choice[expert<kN>(i, lane)] = c[i];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      const int lanes = lanes_of(a.n_groups);
      bool near;
      stay = best_groups(a, group_value<float>(a, lanes, [&](int e) { return s.choice[e]; }), lanes, off, &near);
      if (near) stay = groups_exactly<T>(a, row, most);
    }
    if constexpr (kGroups) {
      if (!a.bias) {                         // the order is the logits': read again, rather than kept
        x.load(row, a.n_experts, kNoneBits, lane);
#pragma unroll
        for (int i = 0; i < kN; ++i) c[i] = x[i];
      }
    }
    if constexpr (kGroups) {
      const uint32_t magic = per > 1 ? (uint32_t)((0x100000000ull + per - 1) / per) : 0u;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t e = (uint32_t)expert<kN>(i, lane), g = per > 1 ? __umulhi(e, magic) : e;
        c[i] = (stay >> (g & 63u)) & 1 ? c[i] : -INFINITY;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // the (k + 1)-th largest of the lanes' largest
    float mine = c[0], border = -INFINITY;
#pragma unroll
    for (int i = 1; i < kN; ++i) mine = fmaxf(mine, c[i]);
    for (int j = 0; j <= a.k; ++j) {
      border = wave_max(mine);
      if (border == -INFINITY) break;
      if (lane == __builtin_ctzll(__ballot(mine == border))) mine = -INFINITY;
    }
    __builtin_amdgcn_sched_barrier(0);
    // candidates
    if (a.bias) border -= off + 0x1p-22f * fabsf(border);
    border = fmaxf(border, -3.402823466e38f);          // never -inf
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const bool is = c[i] >= border;
      const uint64_t m = __ballot(is);
      if (!m) continue;
      const uint32_t at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
      if (is && at < 64) s.order[at] = (uint64_t)~key_of(c[i]) << 32 | (uint32_t)expert<kN>(i, lane);
      n += (uint32_t)__popcll(m);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const uint32_t held = min(n, 64u);
    const bool there = (uint32_t)lane < held;
    const uint64_t o = wave_sorted(there ? s.order[lane] : ~0ull, held, s.order);
    float l = there ? logit_at<T>(row, (int)(uint32_t)o) : 0.f;
    int id = there && lane < a.k ? (int)(uint32_t)o : -1;
    bool near = false;
    if (a.bias) {
      const float v = of_key(~(uint32_t)(o >> 32)), w = __shfl_down(v, 1, 64);
      near = __any(lane < a.k && (uint32_t)lane + 1 < held && !(v - w > off + 0x1p-22f * fmaxf(fabsf(v), fabsf(w))));
    }
    __builtin_amdgcn_wave_barrier();
    // out of the way of the others up to 1024 experts (16384 x 256: 16.8 instead of 17.6 us); above it costs registers (16384 x 2048 34.4
    // instead of 33.4, in groups 96 instead of 86)
    const bool rare = n > 64 || near;
    if (kN < 32 ? __builtin_expect(rare, 0) : rare) {
      if (n > 64) {
        id = choose_exactly<T>(a, row, most);
      } else {
        const double sum = a.sigmoid ? 1. : sum_of<T>(a, row, most);
        const int e = (int)(uint32_t)o;
        const Choice v{there ? score_of(a, l, most, sum) + (double)a.bias[e] : -(double)INFINITY, there ? e : kMostExperts + lane};
        uint32_t at = 0;
        for (uint32_t j = 0; j < held; ++j) at += before(Choice{of_lane(v.c, (int)j), (int)of_lane((uint32_t)v.e, (int)j)}, v);
        if (there) s.order[at] = (uint32_t)e;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        id = there && lane < a.k ? (int)s.order[lane] : -1;
        __builtin_amdgcn_wave_barrier();
      }
      if (id >= 0) l = logit_at<T>(row, id);
    }
    // gates of the chosen, in 64 bits but for the terms of the sum over all experts
    double g = id < 0 ? 0. : score_of(a, l, most, a.renorm ? 1. : z);
    if (a.renorm) {
      const double total = wave_sum(g);
      if (total > 0x1p-900) g *= inverse(total);
      else if (total > 0.) g = g * 0x1p150 * inverse(total * 0x1p150);     // 1 / total may be no number of 64 bits
    }
    if (lane < a.k) {
      a.ids[t * a.k + lane] = id;
      a.gates[t * a.k + lane] = (float)(g * (double)a.scale);
    }
  }
}

// The most workgroups; each wave goes on to further tokens.  Above 1024 experts registers hold four waves of each SIMD, and more
// workgroups only bring the bias to LDS more often (16384 x 2048, by workgroups: 1024 36.7 us, 2048 38.8, 4096 41.2); below more
// waves fit, and tokens of different lengths even out (65536 x 256 in groups: 1024 124 us, 2048 109, 4096 100, 16384 102).
constexpr int most_workgroups(int n) { return n > 16 ? 1024 : 4096; }

template <typename T, int kN>
void launch_route(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>(((int64_t)a.n_tokens + kRWaves - 1) / kRWaves, most_workgroups(kN))), block(kRThreads);
  if (a.n_groups > 1) hipLaunchKernelGGL((route_kernel<T, kN, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_kernel<T, kN, false>), grid, block, 0, s, a);
}

template <typename T>
void launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.n_experts <= 64) launch_route<T, 1>(a, s);
  else if (a.n_experts <= 128) launch_route<T, 2>(a, s);
  else if (a.n_experts <= 256) launch_route<T, 4>(a, s);
  else if (a.n_experts <= 512) launch_route<T, 8>(a, s);
  else if (a.n_experts <= 1024) launch_route<T, 16>(a, s);
  else if (a.n_experts <= 2048) launch_route<T, 32>(a, s);
  else launch_route<T, 64>(a, s);
}

bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

}  // namespace
}  // namespace sbm

using namespace sbm;

extern "C" int sbm_moe_route(const sbm_route_args* args, void* stream) {
  if (!args) return fail(SBM_EINVAL, "null pointer");
  const auto [logits, row_stride, bias, requests, ids, gates, error, scale, n_tokens, n_experts, k, n_groups, top_groups, group_best,
              flags] = *args;
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
