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
constexpr int kTile = 1024;                  // tokens that a wave takes together, 16 a lane
constexpr int kPer = kTile / 64;
constexpr int kMostTiles = kMostVocab / kTile;
constexpr int kBins = 4096;                  // of the distance below the largest logit: 128 to a doubling, from 2^-12 on
constexpr int kDigits = 1024;                // ten bits of an order at a time
constexpr int kList = 6144;                  // tokens of a row that are put in order in LDS
constexpr int kMostParts = 64;               // workgroups of a row
static_assert(kMostTiles <= kSThreads && kDigits == kSThreads, "a thread has a tile, or a digit");

struct SampleArgs {
  const void* logits;
  int64_t stride;
  const float *uniforms, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* logprobs;
  uint32_t* error;
  uint8_t* workspace;
  int64_t ws_row;                            // workspace bytes of a row
  int32_t vocab, parts;
};

// What a row keeps between its filters: tokens in bins below lo stay (as far as min_p lets them), tokens in lo .. hi are put
// in order to see.
struct Range {
  uint32_t lo, hi;
  uint64_t target;                           // how many of those in order, or how much weight
};

// A row's workspace, where several workgroups share a row.
struct RowSpace {
  uint32_t done[2], n_list, first;           // workgroups that ended; tokens to be ordered; the first of the largest
  Range range;
  float part_max[kMostParts];
  uint64_t bins[kBins];
  uint64_t list[kList];
  uint64_t tiles[1];                         // one for each kTile tokens
};

constexpr int64_t row_space(int vocab) { return ((int64_t)sizeof(RowSpace) + 8 * ((vocab + kTile - 1) / kTile) + 255) / 256 * 256; }

// Weights are whole numbers of 2^-42, so that their sums (at most 2^20 of at most 1) do not depend on an order.
constexpr double kUnit = 0x1p42;

// 32 bits that order as the numbers do; both zeros are one.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// A token's place in a row's order, rising: falling logits, of equal ones rising indices.  52 bits, no two are the same.
__device__ __forceinline__ uint64_t order_of(float l, uint32_t i) { return (uint64_t)~key_of(l) << 20 | i; }
__device__ __forceinline__ float logit_of(uint64_t order) { return of_key(~(uint32_t)(order >> 20)); }
__device__ __forceinline__ uint32_t index_of(uint64_t order) { return (uint32_t)order & 0xFFFFFu; }

// The bin of a logit d below the largest (d >= 0, or NaN where both are -inf).
__device__ __forceinline__ uint32_t bin_of(float most, float l) {
  const uint32_t b = __float_as_uint(most - l) >> 16, from = (127 - 12) << 7;
  return min(max(b, from) - from, (uint32_t)kBins - 1);
}

// A row's parameters.
struct Row {
  const char* at;
  double most, slope, least;                 // the largest logit; log2(e) / temperature; min_p
  float u, top_p, temperature;
  int32_t top_k;                             // 0: all
  bool bad;
};

__device__ __forceinline__ Row row_of(const SampleArgs& a, int64_t r, int bytes) {
  Row f;
  f.at = (const char*)a.logits + r * a.stride * bytes;
  f.u = a.uniforms[r];
  f.temperature = a.temperature ? a.temperature[r] : 1.f;
  f.top_p = a.top_p ? a.top_p[r] : 1.f;
  const float min_p = a.min_p ? a.min_p[r] : 0.f;
  f.top_k = a.top_k ? a.top_k[r] : 0;
  if (f.top_k < 0 || f.top_k >= a.vocab) f.top_k = 0;
  f.bad = f.u != f.u || !(f.temperature >= 0.f) || f.top_p != f.top_p || min_p != min_p;
  f.least = min_p > 0.f ? fmin((double)min_p, 1.) : 0.;
  f.slope = f.temperature > 0.f ? 1.4426950408889634 / (double)f.temperature : 0.;
  f.most = 0;
  return f;
}

// exp((l - most) / temperature) = 2^x, to 4e-14 of itself: x's whole part goes to the exponent, 2^f for the rest, |f| <= 1/2,
// is a polynomial of degree 9 that interpolates it at Chebyshev's points (3.7e-14 off at most) and is 1 at 0.
__device__ __forceinline__ double weight(const Row& f, float l) {
  const double x = fmax(((double)l - f.most) * f.slope, -100.);
  const double n = rint(x), y = x - n;
  double p = 0x1.b63880a30e9ffp-24;
  p = __builtin_fma(p, y, 0x1.63d136366db24p-20);
  p = __builtin_fma(p, y, 0x1.ffcb9515a8016p-17);
  p = __builtin_fma(p, y, 0x1.4308ac85aa947p-13);
  p = __builtin_fma(p, y, 0x1.5d87fe86fe88ep-10);
  p = __builtin_fma(p, y, 0x1.3b2ab7181b755p-7);
  p = __builtin_fma(p, y, 0x1.c6b08d7047e52p-5);
  p = __builtin_fma(p, y, 0x1.ebfbdff823cedp-3);
  p = __builtin_fma(p, y, 0x1.62e42fefa39efp-1);
  p = __builtin_fma(p, y, 1.);
  return __builtin_amdgcn_ldexp(p, (int)n);
}
// The low bits of 2^10 + w are w in units of 2^-42, rounded.
__device__ __forceinline__ uint64_t units(double w) {
  return __builtin_bit_cast(uint64_t, w + 0x1p10) - __builtin_bit_cast(uint64_t, 0x1p10);
}

// What a lane has of a wave's tile: 16 logits in runs of 16 bytes; -inf past the vocabulary's end.
template <typename T>
struct Tile {
  static constexpr int kRun = __is_same(T, float) ? 4 : 8;
  float l[kPer];

  __device__ __forceinline__ static int index(int i) {
    return (i / kRun) * 64 * kRun + ((int)threadIdx.x & 63) * kRun + i % kRun;
  }
  __device__ __forceinline__ void load(const char* row, int first, int vocab) {
    constexpr int kBytes = 16 / kRun;
    if (first + kTile <= vocab) {
      uint32_t raw[kPer / kRun][4];
#pragma unroll
      for (int j = 0; j < kPer / kRun; ++j) __builtin_memcpy(raw[j], row + (int64_t)(first + index(j * kRun)) * kBytes, 16);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if constexpr (kRun == 4) l[i] = __uint_as_float(raw[i / 4][i % 4]);
        else l[i] = to_f32<T>((uint16_t)(raw[i / 8][i % 8 / 2] >> 16 * (i & 1)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = first + index(i);
        l[i] = -INFINITY;
        if (at < vocab) {
          if constexpr (kRun == 4) l[i] = ((const float*)row)[at];
          else l[i] = to_f32<T>(((const uint16_t*)row)[at]);
        }
      }
    }
  }
};

__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The LDS of a workgroup.
struct Shared {
  union {
    uint64_t bins[kBins];
    uint64_t list[kList];
  };
  uint64_t tiles[kMostTiles];
  uint64_t sums[kDigits];
  uint32_t counts[kDigits];
  uint64_t waves[kSWaves];
  uint64_t found[4];
  float wave_max[kSWaves];
  uint32_t n_list, first, last;
  Range range;
};

// Exclusive sums over the workgroup's threads, and the whole.
__device__ __forceinline__ uint64_t scan(uint64_t v, Shared& s, uint64_t* all) {
  const int lane = (int)threadIdx.x & 63;
  uint64_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) s.waves[threadIdx.x >> 6] = x;
  __syncthreads();
  uint64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kSWaves; ++w) {
    if (w < (int)(threadIdx.x >> 6)) before += s.waves[w];
    sum += s.waves[w];
  }
  *all = sum;
  return before + x - v;
}

// What the workgroups of a row tell each other within a launch goes past the caches of the chip's parts: a fence would write
// those back as a whole (with one, 200 x 50021 took 215 us in this step alone).
template <typename V>
__device__ __forceinline__ void tell(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V read_back(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this workgroup is the row's last to come here; what the others told before is then there to be read.
__device__ bool is_last(uint32_t* done, int parts, Shared& s) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0x0F70);                  // vmcnt(0): told
  __syncthreads();
  if (threadIdx.x == 0)
    s.last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)parts - 1;
  __syncthreads();
  return s.last != 0;
}

// ------------------------------------------------------------------ first: the largest

// The largest logit of a workgroup's tiles, NaN where one is NaN or +inf.
template <typename T>
__device__ float largest(const Row& f, const SampleArgs& a, int part, Shared& s) {
  const int wave = (int)threadIdx.x >> 6, tiles = (a.vocab + kTile - 1) / kTile;
  float most = -INFINITY;
  bool bad = false;
  for (int t = part * kSWaves + wave; t < tiles; t += a.parts * kSWaves) {
    Tile<T> x;
    x.load(f.at, t * kTile, a.vocab);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      bad = bad || !(x.l[i] < INFINITY);
      most = fmaxf(most, x.l[i]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
  if (__any(bad)) most = __builtin_nanf("");
  if ((threadIdx.x & 63) == 0) s.wave_max[wave] = most;
  __syncthreads();
  most = s.wave_max[0];
#pragma unroll
  for (int w = 1; w < kSWaves; ++w) most = s.wave_max[w] != s.wave_max[w] ? s.wave_max[w] : most != most ? most : fmaxf(most, s.wave_max[w]);
  return most + 0.f;                         // one zero
}

// ------------------------------------------------------------------ second: where a filter ends

// Tokens (top_k) or weights (top_p) by bins.
template <typename T>
__device__ void fill_bins(const Row& f, const SampleArgs& a, int part, Shared& s) {
  const int tid = (int)threadIdx.x, wave = tid >> 6, tiles = (a.vocab + kTile - 1) / kTile;
  for (int b = tid; b < kBins; b += kSThreads) s.bins[b] = 0;
  __syncthreads();
  const float most = (float)f.most;
  for (int t = part * kSWaves + wave; t < tiles; t += a.parts * kSWaves) {
    Tile<T> x;
    x.load(f.at, t * kTile, a.vocab);
    if (f.top_k) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (x.l[i] > -INFINITY) atomicAdd((uint32_t*)&s.bins[bin_of(most, x.l[i])], 1u);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const double w = weight(f, x.l[i]);
        if (x.l[i] > -INFINITY && w >= f.least)
          atomicAdd((unsigned long long*)&s.bins[bin_of(most, x.l[i])], (unsigned long long)units(w));
      }
    }
  }
  __syncthreads();
}

// The bins in which the filters' ends are, from all the row's tokens in s.bins.
__device__ Range find_bins(const Row& f, Shared& s) {
  constexpr int kMine = kBins / kSThreads;
  const int tid = (int)threadIdx.x;
  uint64_t mine[kMine], sum = 0, total;
#pragma unroll
  for (int j = 0; j < kMine; ++j) sum += mine[j] = s.bins[tid * kMine + j];
  uint64_t before = scan(sum, s, &total);
  const uint64_t want = f.top_k ? (uint64_t)f.top_k : max((uint64_t)ceil(fmax((double)f.top_p, 0.) * (double)total), (uint64_t)1);
  if (tid == 0 && total < want) s.range = Range{0, kBins - 1, want};            // all of fewer
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (before < want && before + mine[j] >= want) {
      const uint32_t b = (uint32_t)(tid * kMine + j);
      // the tokens of top_k: all in order, where there are few, or a top_p applies to them
      const bool whole = f.top_k && (before + mine[j] <= kList || f.top_p < 1.f);
      s.range = whole ? Range{0, b, want} : Range{b, b, want - before};
    }
    before += mine[j];
  }
  __syncthreads();
  return s.range;
}

// ------------------------------------------------------------------ third: order, sums, draw

// Each tile's sum of the weights that stay for certain, and a list of the tokens to be put in order.
template <typename T, bool kOne>
__device__ void sum_tiles(const Row& f, const SampleArgs& a, int part, const Range& r, uint64_t* sums, Shared& s) {
  const int tid = (int)threadIdx.x, wave = tid >> 6, tiles = (a.vocab + kTile - 1) / kTile;
  if (tid == 0) s.n_list = 0, s.first = ~0u;
  __syncthreads();
  const float most = (float)f.most;
  for (int t = part * kSWaves + wave; t < tiles; t += a.parts * kSWaves) {
    Tile<T> x;
    x.load(f.at, t * kTile, a.vocab);
    if (f.temperature == 0.f) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (x.l[i] == most) atomicMin(&s.first, (uint32_t)(t * kTile + Tile<T>::index(i)));
      continue;
    }
    uint64_t sum = 0;
    if (r.lo > 0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const double w = weight(f, x.l[i]);
        sum += x.l[i] > -INFINITY && bin_of(most, x.l[i]) < r.lo && w >= f.least ? units(w) : 0ull;
      }
    }
    if (r.lo < kBins) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t b = bin_of(most, x.l[i]);
        if (x.l[i] > -INFINITY && b >= r.lo && b <= r.hi) {
          const uint32_t n = atomicAdd(&s.n_list, 1u);
          if (n < kList) s.list[n] = order_of(x.l[i], (uint32_t)(t * kTile + Tile<T>::index(i)));
        }
      }
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) {
      if constexpr (kOne) sums[t] = sum;
      else tell(&sums[t], sum);
    }
  }
  __syncthreads();
}

// Tokens in order: those of the list, or all of the row.
template <typename T>
struct Source {
  const char* row;                           // NULL: the list
  uint32_t n;
  const uint64_t* list;
  __device__ __forceinline__ uint64_t operator[](uint32_t i) const {
    if (!row) return list[i];
    float l;
    if constexpr (__is_same(T, float)) l = ((const float*)row)[i];
    else l = to_f32<T>(((const uint16_t*)row)[i]);
    return l > -INFINITY ? order_of(l, i) : ~0ull;
  }
};

// The place in the order at which `target` tokens, or units of weight, are reached among those up to `end`: ten bits at a
// time, from the highest in which two differ.
template <typename T>
__device__ uint64_t descend(const Source<T>& from, const Row& f, bool weights, uint64_t target, uint64_t end, Shared& s) {
  const int tid = (int)threadIdx.x;
  uint64_t low = ~0ull, high = 0;
  if (!from.row) {
    for (uint32_t i = tid; i < from.n; i += kSThreads) {
      const uint64_t o = from.list[i];
      low = min(low, o);
      high = max(high, o);
    }
    __syncthreads();
    if (tid == 0) s.found[0] = ~0ull, s.found[1] = 0;
    __syncthreads();
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      low = min(low, (uint64_t)__shfl_xor(low, d, 64));
      high = max(high, (uint64_t)__shfl_xor(high, d, 64));
    }
    if ((tid & 63) == 0) {
      atomicMin((unsigned long long*)&s.found[0], (unsigned long long)low);
      atomicMax((unsigned long long*)&s.found[1], (unsigned long long)high);
    }
    __syncthreads();
    low = s.found[0];
    high = s.found[1];
  } else {
    low = 0;
    high = (1ull << 52) - 1;
  }
  int top = low == high ? 0 : 64 - __builtin_clzll(low ^ high);        // bits that are not known yet
  uint64_t prefix = top < 52 ? low >> top : 0;
  while (top > 0) {
    const int shift = max(top - 10, 0);
    __syncthreads();
    s.sums[tid] = 0;
    s.counts[tid] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < from.n; i += kSThreads) {
      const uint64_t o = from[i];
      if (o > end || o >> top != prefix) continue;
      const uint32_t digit = (uint32_t)(o >> shift) & ((1u << (top - shift)) - 1u);
      atomicAdd(&s.counts[digit], 1u);
      if (weights) {
        const double w = weight(f, logit_of(o));
        if (w >= f.least) atomicAdd((unsigned long long*)&s.sums[digit], (unsigned long long)units(w));
      }
    }
    __syncthreads();
    const uint64_t mine = weights ? s.sums[tid] : s.counts[tid];
    uint64_t all;
    const uint64_t before = scan(mine, s, &all);
    if (before < target && before + mine >= target) {
      s.found[0] = (uint64_t)tid;
      s.found[1] = target - before;
      s.found[2] = s.counts[tid];
    }
    __syncthreads();
    prefix = prefix << (top - shift) | s.found[0];
    target = s.found[1];
    top = shift;
    if (s.found[2] == 1 && top > 0) {        // one token: the rest of its bits
      for (uint32_t i = tid; i < from.n; i += kSThreads) {
        const uint64_t o = from[i];
        if (o <= end && o >> top == prefix) s.found[3] = o;
      }
      __syncthreads();
      prefix = s.found[3];
      top = 0;
    }
  }
  __syncthreads();
  return prefix;
}

__device__ void refuse(const SampleArgs& a, int64_t r) {
  a.tokens[r] = -1;
  if (a.logprobs) a.logprobs[r] = __builtin_nanf("");
  if (a.error) atomicAdd(a.error, 1u);
}

// The token of a row from its tiles' sums (s.tiles) and the tokens to be ordered (s.list, s.n_list of them).
template <typename T>
__device__ void draw(const Row& f, const SampleArgs& a, int64_t r, const Range& range, Shared& s) {
  const int tid = (int)threadIdx.x, wave = tid >> 6, tiles = (a.vocab + kTile - 1) / kTile;
  if (f.temperature == 0.f) {
    if (tid == 0) {
      a.tokens[r] = (int32_t)s.first;
      if (a.logprobs) a.logprobs[r] = 0.f;
    }
    return;
  }
  const bool few = s.n_list <= kList;
  const bool ordered = f.top_k || f.top_p < 1.f;
  uint64_t end = ~0ull - 1;                  // the last that stays; ~0 is no token
  if (ordered) {
    // more than the list holds: the whole row, bit by bit
    const Source<T> from{few ? nullptr : f.at, few ? s.n_list : (uint32_t)a.vocab, s.list};
    const auto sum_of = [&]() {
      uint64_t sum = 0, all;
      for (uint32_t i = tid; i < from.n; i += kSThreads) {
        const uint64_t o = from[i];
        if (o > end) continue;
        const double w = weight(f, logit_of(o));
        if (w >= f.least) sum += units(w);
      }
      scan(sum, s, &all);
      return all;
    };
    if (f.top_k) {
      uint64_t target = few ? range.target : (uint64_t)f.top_k, there = 0, all;
      for (uint32_t i = tid; i < from.n; i += kSThreads) there += from[i] != ~0ull;
      scan(there, s, &all);
      if (all >= target) end = descend(from, f, false, target, end, s);
    }
    if (f.top_p < 1.f) {
      uint64_t target = range.target;
      if (f.top_k || !few) target = max((uint64_t)ceil(fmax((double)f.top_p, 0.) * (double)sum_of()), (uint64_t)1);
      end = descend(from, f, true, target, end, s);
    }
    if (few) {
      for (uint32_t i = tid; i < s.n_list; i += kSThreads) {
        const uint64_t o = s.list[i];
        const double w = weight(f, logit_of(o));
        if (o <= end && w >= f.least) atomicAdd((unsigned long long*)&s.tiles[index_of(o) / kTile], (unsigned long long)units(w));
      }
    } else {
      for (int t = wave; t < tiles; t += kSWaves) {
        Tile<T> x;
        x.load(f.at, t * kTile, a.vocab);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const double w = weight(f, x.l[i]);
          if (x.l[i] > -INFINITY && order_of(x.l[i], (uint32_t)(t * kTile + Tile<T>::index(i))) <= end && w >= f.least) sum += units(w);
        }
        sum = wave_sum(sum);
        if ((tid & 63) == 0) s.tiles[t] = sum;
      }
    }
    __syncthreads();
  }
  // the first token whose running sum passes u * total
  uint64_t mine = tid < tiles ? s.tiles[tid] : 0, total, all;
  uint64_t before = scan(mine, s, &total);
  const uint64_t at = min((uint64_t)(fmin(fmax((double)f.u, 0.), 1.) * (double)total), total - 1);
  if (before <= at && before + mine > at) {
    s.found[0] = (uint64_t)tid;
    s.found[1] = at - before;
  }
  __syncthreads();
  const int i = (int)s.found[0] * kTile + tid;
  const uint64_t left = s.found[1], o = i < a.vocab ? Source<T>{f.at, 0, nullptr}[(uint32_t)i] : ~0ull;
  mine = 0;
  if (o <= end) {
    const double w = weight(f, logit_of(o));
    if (w >= f.least) mine = units(w);
  }
  before = scan(mine, s, &all);
  if (before <= left && before + mine > left) {
    a.tokens[r] = i;
    if (a.logprobs)
      a.logprobs[r] = (float)(((double)logit_of(o) - f.most) / (double)f.temperature - log((double)total * (1. / kUnit)));
  }
}

// ------------------------------------------------------------------ kernels

// A workgroup has a row.
template <typename T>
__global__ __launch_bounds__(kSThreads) void sample_row_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x;
  Row f = row_of(a, r, __is_same(T, float) ? 4 : 2);
  const float most = largest<T>(f, a, 0, s);
  if (f.bad || !(most > -INFINITY)) {
    if (threadIdx.x == 0) refuse(a, r);
    return;
  }
  f.most = (double)most;
  Range range{kBins, 0, 0};
  if (f.temperature > 0.f && (f.top_k || f.top_p < 1.f)) {
    fill_bins<T>(f, a, 0, s);
    range = find_bins(f, s);
  }
  sum_tiles<T, true>(f, a, 0, range, s.tiles, s);
  draw<T>(f, a, r, range, s);
}

__device__ __forceinline__ RowSpace* space_of(const SampleArgs& a, int64_t r) { return (RowSpace*)(a.workspace + r * a.ws_row); }

// The parts' largest logits; NaN where one is.
__device__ __forceinline__ float joined(const RowSpace* w, int parts) {
  const int lane = (int)threadIdx.x & 63;
  const float v = lane < parts ? w->part_max[lane] : -INFINITY;
  float most = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
  return __any(v != v) ? __builtin_nanf("") : most;
}

// Several workgroups share a row; three launches, and the last workgroup of a row to end the second and the third joins what
// they found.
template <typename T>
__global__ __launch_bounds__(kSThreads) void sample_max_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - r * a.parts), tid = (int)threadIdx.x;
  RowSpace* w = space_of(a, r);
  if (part == 0 && tid == 0) w->done[0] = w->done[1] = w->n_list = 0, w->first = ~0u;
  for (int b = part * kSThreads + tid; b < kBins; b += a.parts * kSThreads) w->bins[b] = 0;
  const Row f = row_of(a, r, __is_same(T, float) ? 4 : 2);
  const float most = largest<T>(f, a, part, s);
  if (tid == 0) w->part_max[part] = most;
}

template <typename T>
__global__ __launch_bounds__(kSThreads) void sample_bins_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - r * a.parts), tid = (int)threadIdx.x;
  RowSpace* w = space_of(a, r);
  Row f = row_of(a, r, __is_same(T, float) ? 4 : 2);
  const float most = joined(w, a.parts);
  if (f.bad || !(most > -INFINITY) || f.temperature == 0.f || (!f.top_k && !(f.top_p < 1.f))) return;
  f.most = (double)most;
  fill_bins<T>(f, a, part, s);
  for (int b = tid; b < kBins; b += kSThreads)
    if (s.bins[b]) atomicAdd((unsigned long long*)&w->bins[b], (unsigned long long)s.bins[b]);
  if (!is_last(&w->done[0], a.parts, s)) return;
  for (int b = tid; b < kBins; b += kSThreads) s.bins[b] = read_back(&w->bins[b]);
  __syncthreads();
  const Range range = find_bins(f, s);
  if (tid == 0) w->range = range;
}

template <typename T>
__global__ __launch_bounds__(kSThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - r * a.parts), tid = (int)threadIdx.x;
  RowSpace* w = space_of(a, r);
  Row f = row_of(a, r, __is_same(T, float) ? 4 : 2);
  const float most = joined(w, a.parts);
  if (f.bad || !(most > -INFINITY)) {
    if (part == 0 && tid == 0) refuse(a, r);
    return;
  }
  f.most = (double)most;
  Range range{kBins, 0, 0};
  if (f.temperature > 0.f && (f.top_k || f.top_p < 1.f)) range = w->range;
  sum_tiles<T, false>(f, a, part, range, w->tiles, s);
  const uint32_t n = s.n_list;
  if (tid == 0) {
    s.found[0] = n ? atomicAdd(&w->n_list, n) : 0u;
    if (s.first != ~0u) atomicMin(&w->first, s.first);
  }
  __syncthreads();
  const uint32_t at = (uint32_t)s.found[0];
  for (uint32_t i = tid; i < min(n, (uint32_t)kList) && at + i < kList; i += kSThreads) tell(&w->list[at + i], s.list[i]);
  if (!is_last(&w->done[1], a.parts, s)) return;
  if (tid == 0) {
    s.n_list = read_back(&w->n_list);
    s.first = read_back(&w->first);
  }
  __syncthreads();
  if (s.n_list <= kList)
    for (uint32_t i = tid; i < s.n_list; i += kSThreads) s.list[i] = read_back(&w->list[i]);
  for (int t = tid; t < (a.vocab + kTile - 1) / kTile; t += kSThreads) s.tiles[t] = read_back(&w->tiles[t]);
  __syncthreads();
  draw<T>(f, a, r, range, s);
}

// Workgroups of a row: one where there are rows enough to fill the card, or a row is short.
constexpr int kFull = 512;
int parts_of(int32_t n_rows, int32_t vocab) {
  const int tiles = (vocab + kTile - 1) / kTile;
  return std::max(1, std::min({(int)kMostParts, kFull / std::max(n_rows, 1), tiles / kSWaves}));
}

template <typename T>
void launch_sample(const SampleArgs& a, int32_t n_rows, hipStream_t s) {
  const dim3 grid((unsigned)(n_rows * a.parts)), block(kSThreads);
  if (a.parts == 1) {
    hipLaunchKernelGGL((sample_row_kernel<T>), grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((sample_max_kernel<T>), grid, block, 0, s, a);
    hipLaunchKernelGGL((sample_bins_kernel<T>), grid, block, 0, s, a);
    hipLaunchKernelGGL((sample_draw_kernel<T>), grid, block, 0, s, a);
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
  // what fewer rows and a shorter vocabulary need too
  return parts_of(1, vocab) > 1 ? std::max<size_t>((size_t)std::min(n_rows, kFull / 2) * (size_t)row_space(vocab), 256) : 256;
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
  const SampleArgs a{logits, row_stride, uniforms, temperature, top_p, min_p, top_k, tokens, logprobs, error, (uint8_t*)workspace,
                     row_space(vocab), vocab, parts_of(n_rows, vocab)};
  if (flags & SBM_F_IN_F32) launch_sample<float>(a, n_rows, (hipStream_t)stream);
  else if (flags & SBM_F_IN_BF16) launch_sample<__bf16>(a, n_rows, (hipStream_t)stream);
  else launch_sample<_Float16>(a, n_rows, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "sample launch: %s", hipGetErrorString(e));
  return SBM_OK;
}

}  // extern "C"
