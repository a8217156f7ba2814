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
constexpr int kHeld = 2;                     // tiles of a wave that stay in its registers: a workgroup's 32768 tokens
constexpr int kBeside = 4;                   // logits of a lane that are passed over together (2 and 8 take the same time)
constexpr int kGroup = kPer;                 // neighbours of which one counts for a top_k
constexpr int kMostGroups = 2048;
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
  int64_t first;                             // the first row of a launch of sample_row_kernel
  int32_t vocab, parts;
};

constexpr float kLowest = -3.402823466e38f;  // of the numbers; from there on is all but -inf

// Where the last token that stays is: logits from `from` on stay, those below it from `to` on are put in order to see.
struct Range {
  float from, to;
  uint64_t target;                           // how many of those in order, or how much weight
};

// A row's workspace, where several workgroups share a row.
struct RowSpace {
  uint32_t done[2], n_list, first;           // workgroups that ended; tokens to be ordered; the first of the largest
  Range range;
  float part_max[kMostParts];
  uint64_t bins[kBins];                      // weights; counts in the first 4 bytes each
  uint64_t list[kList];
  uint64_t tiles[1];                         // one for each kTile tokens
};

constexpr int64_t row_space(int vocab) { return ((int64_t)sizeof(RowSpace) + 8 * ((vocab + kTile - 1) / kTile) + 255) / 256 * 256; }

// Weights are whole numbers of a unit, so that their sums do not depend on an order: 2^-62 times the least power of two that is
// not below the vocabulary (or 2048), 2^-42 for the largest.
struct Unit {
  double magic;                              // 2^52 units: the low bits of magic + w are w in units, rounded
  // w in units above what none() is
  __device__ __forceinline__ uint64_t above(double w) const { return __builtin_bit_cast(uint64_t, w + magic); }
  __device__ __forceinline__ uint64_t none() const { return (uint64_t)__double2hiint(magic) << 32; }
  __device__ __forceinline__ uint64_t operator()(double w) const {
    Halves u = __builtin_bit_cast(Halves, w + magic);
    u[1] -= (uint32_t)__double2hiint(magic);
    return __builtin_bit_cast(uint64_t, u);
  }
};

// A token's place in a row's order, rising: falling logits, of equal ones rising indices.  52 bits, no two are the same.
__device__ __forceinline__ uint64_t order_of(float l, uint32_t i) { return (uint64_t)~key_of(l) << 20 | i; }
__device__ __forceinline__ float logit_of(uint64_t order) { return of_key(~(uint32_t)(order >> 20)); }
__device__ __forceinline__ uint32_t index_of(uint64_t order) { return (uint32_t)order & 0xFFFFFu; }

// The bin of a logit below the largest, by their distance; and the distance at which a bin begins.
constexpr uint32_t kFirstBin = (127 - 12) << 7;
__device__ __forceinline__ uint32_t bin_of(float most, float l) {
  const uint32_t b = __float_as_uint(most - l) >> 16;
  return min(max(b, kFirstBin) - kFirstBin, (uint32_t)kBins - 1);
}
__device__ __forceinline__ float begin_of(uint32_t bin) {
  return bin == 0 ? 0.f : bin >= kBins ? INFINITY : __uint_as_float((bin + kFirstBin) << 16);
}

// A row's parameters.
struct Row {
  const char* at;
  double most, slope, least;                 // the largest logit; log2(e) / temperature; -1000 / slope
  Unit units;
  float u, top_p, min_p, temperature;
  float low;                                 // the least logit that stays by min_p; above -inf
  int32_t top_k;                             // 0: all
  bool bad;
};

__device__ __forceinline__ Row row_of(const SampleArgs& a, int64_t r, int bytes) {
  Row f;
  f.at = (const char*)a.logits + r * a.stride * bytes;
  f.u = a.uniforms[r];
  f.temperature = a.temperature ? a.temperature[r] : 1.f;
  f.top_p = a.top_p ? a.top_p[r] : 1.f;
  f.min_p = a.min_p ? a.min_p[r] : 0.f;
  f.top_k = a.top_k ? a.top_k[r] : 0;
  if (f.top_k < 0 || f.top_k >= a.vocab) f.top_k = 0;
  f.bad = f.u != f.u || !(f.temperature >= 0.f) || f.top_p != f.top_p || f.min_p != f.min_p;
  f.low = kLowest;
  f.slope = f.temperature > 0.f ? fmax(1.4426950408889634 / (double)f.temperature, 1e-300) : 0.;      // not 0 * -inf
  f.least = f.temperature > 0.f ? -1000. / f.slope : 0.;
  f.most = 0;
  const int bits = max(32 - __builtin_clz(max((unsigned)a.vocab, 2u) - 1u), 11);
  f.units.magic = __builtin_amdgcn_ldexp(1., bits - 10);
  return f;
}

// exp((l - most) / temperature), to 4e-14 of itself; 2^-1000, which is no unit, for what is below that.
__device__ __forceinline__ double weight(const Row& f, float l) { return exp2_f64(fmax((double)l - f.most, f.least), f.slope); }

// The least key from lo to hi at which something holds that holds from there on, hi among it: 64 places at a time.
template <typename F>
__device__ __forceinline__ uint32_t first_key(uint32_t lo, uint32_t hi, F holds) {
  const uint32_t lane = threadIdx.x & 63u;
  while (lo < hi) {
    const uint32_t step = (hi - lo + 62u) / 63u;
    const uint32_t k = (uint32_t)min((uint64_t)lo + (uint64_t)lane * step, (uint64_t)hi);
    const uint32_t j = (uint32_t)__builtin_ctzll(__ballot(holds(k)));
    if (j == 0) return lo;
    hi = (uint32_t)min((uint64_t)lo + (uint64_t)j * step, (uint64_t)hi);
    lo += (j - 1u) * step + 1u;
  }
  return lo;
}

// What a lane has of a wave's tile: 16 logits in runs of 16 bytes; -inf past the vocabulary's end.
template <typename T>
struct Tile {
  static constexpr int kRun = __is_same(T, float) ? 4 : 8;
  static constexpr uint32_t kNone = __is_same(T, float) ? 0xFF800000u : __is_same(T, __bf16) ? 0xFF80u : 0xFC00u;
  uint32_t raw[kPer / kRun][4];

  __device__ __forceinline__ static int index(int i) {
    return (i / kRun) * 64 * kRun + ((int)threadIdx.x & 63) * kRun + i % kRun;
  }
  __device__ __forceinline__ void load(const char* row, int first, int vocab) {
    constexpr int kBytes = 16 / kRun;
    if (first + kTile <= vocab) {
#pragma unroll
      for (int j = 0; j < kPer / kRun; ++j) __builtin_memcpy(raw[j], row + (int64_t)(first + index(j * kRun)) * kBytes, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = first + index(i);
        uint32_t u = kNone;
        if (at < vocab) {
          if constexpr (kRun == 4) u = ((const uint32_t*)row)[at];
          else u = ((const uint16_t*)row)[at];
        }
        if constexpr (kRun == 4) raw[i / 4][i % 4] = u;
        else raw[i / 8][i % 8 / 2] = i & 1 ? raw[i / 8][i % 8 / 2] | u << 16 : u;
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (kRun == 4) return __uint_as_float(raw[i / 4][i % 4]);
    else return to_f32<T>((uint16_t)(raw[i / 8][i % 8 / 2] >> 16 * (i & 1)));
  }
};

// A wave's tiles, part, part + parts, ... of kSWaves each: loaded once and held in registers (kHold, which then has to be all),
// or loaded whenever they are looked at.
template <typename T, int kHold>
struct Tiles {
  Tile<T> held[kHold ? kHold : 1];
  const char* row;
  int vocab, first, step, n;

  __device__ __forceinline__ Tiles(const Row& f, const SampleArgs& a, int part) {
    row = f.at;
    vocab = a.vocab;
    n = (a.vocab + kTile - 1) / kTile;
    first = part * kSWaves + (int)(threadIdx.x >> 6);
    step = a.parts * kSWaves;
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if (first + j * step < n) held[j].load(row, (first + j * step) * kTile, vocab);
  }
  template <typename F>
  __device__ __forceinline__ void each(F fn) const {
    if constexpr (kHold > 0) {
#pragma unroll
      for (int j = 0; j < kHold; ++j)
        if (first + j * step < n) fn(first + j * step, held[j]);
    } else {
      for (int t = first; t < n; t += step) {
        Tile<T> x;
        x.load(row, t * kTile, vocab);
        fn(t, x);
      }
    }
  }
};

// The LDS of a workgroup.
struct alignas(16) Shared {
  union {
    uint64_t bins[kBins];                    // weights
    uint32_t counts_of[kBins];
    uint64_t list[kList];
  };
  uint64_t tiles[kMostTiles];
  uint64_t sums[kDigits];
  uint32_t counts[kDigits];
  uint64_t waves[kSWaves];
  uint64_t found[4], few[64];
  float wave_max[kSWaves];
  uint32_t n_list, n_few, first, last;
  float low;
  Range range;
};

// Exclusive sums over the workgroup's threads, and the whole.
template <typename V>
__device__ __forceinline__ V scan(V v, Shared& s, V* all) {
  V* waves = (V*)s.waves;
  const V x = wave_scan(v);
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  __syncthreads();
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  V w = lane < kSWaves ? waves[lane] : 0;
  w += moved<0x111, 0xF>(w);                 // within 16 lanes
  w += moved<0x112, 0xF>(w);
  w += moved<0x114, 0xF>(w);
  w += moved<0x118, 0xF>(w);
  *all = of_lane(w, kSWaves - 1);
  return (wave ? of_lane(w, wave - 1) : 0) + x - v;
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

// The largest of n <= 64 numbers, NaN where one is.
__device__ __forceinline__ float join_max(const float* p, int n) {
  const int lane = (int)threadIdx.x & 63;
  const float v = lane < n ? p[lane] : -INFINITY;
  return __any(v != v) ? __builtin_nanf("") : wave_max(v) + 0.f;              // one zero
}

// The largest logit of a workgroup's tiles, NaN where one is NaN or +inf.
template <typename X>
__device__ float largest(const X& tiles, Shared& s) {
  const int wave = (int)threadIdx.x >> 6;
  float most = -INFINITY;
  bool bad = false;
  tiles.each([&](int, const auto& x) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      bad = bad || !(x[i] < INFINITY);
      most = fmaxf(most, x[i]);
    }
  });
  most = wave_max(most);
  if (__any(bad)) most = __builtin_nanf("");
  if ((threadIdx.x & 63) == 0) s.wave_max[wave] = most;
  __syncthreads();
  return join_max(s.wave_max, kSWaves);
}

// The least logit that stays by min_p, into f.low.
__device__ void find_low(Row& f, Shared& s) {
  if (!(f.min_p > 0.f) || f.temperature == 0.f) return;
  if (threadIdx.x < 64) {
    const double least = fmin((double)f.min_p, 1.);
    s.low = of_key(first_key(key_of(f.low), key_of((float)f.most), [&](uint32_t k) { return weight(f, of_key(k)) >= least; }));
  }
  __syncthreads();
  f.low = s.low;
}

// ------------------------------------------------------------------ second: where a filter ends

// A top_k that is found from the largest of each group of 16 neighbours: at least k tokens are not below the k-th largest of
// those, and about as many as long as most groups have none (k up to half the groups).  That takes a sixteenth of the counting.
__device__ __forceinline__ bool by_groups(const Row& f, const SampleArgs& a) {
  return f.top_k <= min(kMostGroups, a.vocab / (2 * kGroup));
}

// Tokens or groups (top_k), or weights (top_p), by bins.  Whole numbers: the LDS adds fp32 numbers to a common place far slower
// (64 x 131072: 48 instead of 15 us).
template <typename X>
__device__ void fill_bins(const X& tiles, const Row& f, const SampleArgs& a, Shared& s) {
  const int tid = (int)threadIdx.x;
  for (int b = tid; b < kBins; b += kSThreads) s.bins[b] = 0;
  __syncthreads();
  const float most = (float)f.most;
  if (f.top_k && by_groups(f, a)) {
    tiles.each([&](int, const auto& x) {
      float l = x[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) l = fmaxf(l, x[i]);
      if (l > -INFINITY) atomicAdd(&s.counts_of[bin_of(most, l)], 1u);
    });
  } else if (f.top_k) {
    tiles.each([&](int, const auto& x) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (x[i] > -INFINITY) atomicAdd(&s.counts_of[bin_of(most, x[i])], 1u);
    });
  } else {
    tiles.each([&](int, const auto& x) {
#pragma unroll
      for (int i = 0; i < kPer; i += kBeside) {
        uint64_t u[kBeside];
#pragma unroll
        for (int j = 0; j < kBeside; ++j) u[j] = f.units(weight(f, x[i + j]));
#pragma unroll
        for (int j = 0; j < kBeside; ++j)
          if (x[i + j] >= f.low) atomicAdd((unsigned long long*)&s.bins[bin_of(most, x[i + j])], (unsigned long long)u[j]);
      }
    });
  }
  __syncthreads();
}

// What a top_p of a whole weight reaches.
__device__ __forceinline__ uint64_t part_of(const Row& f, uint64_t total) {
  return max((uint64_t)ceil(fmax((double)f.top_p, 0.) * (double)total), (uint64_t)1);
}

// The bins in which the filters' ends are, from all the row's tokens.
template <typename V>
__device__ Range find_bins(const V* bins, const Row& f, const SampleArgs& a, Shared& s) {
  constexpr int kMine = kBins / kSThreads;
  const int tid = (int)threadIdx.x;
  V mine[kMine], sum = 0, total;
#pragma unroll
  for (int j = 0; j < kMine; ++j) sum += mine[j] = bins[tid * kMine + j];
  V before = scan(sum, s, &total);
  const V want = f.top_k ? (V)f.top_k : (V)part_of(f, total);
  if (tid == 0) s.found[0] = 0, s.found[1] = kBins, s.found[2] = want;             // all of fewer
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (before < want && before + mine[j] >= want) {
      const uint32_t b = (uint32_t)(tid * kMine + j);
      // the tokens of a top_k: all in order, where there are few, or a top_p applies to them
      const bool whole = f.top_k && (by_groups(f, a) || before + mine[j] <= kList || f.top_p < 1.f);
      s.found[0] = whole ? 0 : b;
      s.found[1] = b + 1;
      s.found[2] = whole ? want : want - before;
    }
    before += mine[j];
  }
  __syncthreads();
  // the bins' beginnings as logits, one by a wave each
  if (tid < 128) {
    const float most = (float)f.most, below = begin_of((uint32_t)s.found[tid >> 6]);
    float l = below > 0.f ? kLowest : INFINITY;
    if (below > 0.f && below < INFINITY)
      l = of_key(first_key(key_of(l), key_of(most), [&](uint32_t k) { return most - of_key(k) < below; }));
    l = fmaxf(l, f.low);
    if (tid == 0) s.range.from = l, s.range.target = s.found[2];
    if (tid == 64) s.range.to = l;
  }
  __syncthreads();
  return s.range;
}
__device__ __forceinline__ Range find_bins(const Row& f, const SampleArgs& a, Shared& s) {
  return f.top_k ? find_bins(s.counts_of, f, a, s) : find_bins(s.bins, f, a, s);
}

// ------------------------------------------------------------------ third: order, sums, draw

// Each tile's sum of the weights that stay for certain, and a list of the tokens to be put in order.
template <bool kOne, typename X>
__device__ void sum_tiles(const X& tiles, const Row& f, const Range& r, uint64_t* sums, Shared& s) {
  const int tid = (int)threadIdx.x;
  if (tid == 0) s.n_list = 0, s.first = ~0u;
  __syncthreads();
  tiles.each([&](int t, const auto& x) {
    if (f.temperature == 0.f) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (x[i] == (float)f.most) atomicMin(&s.first, (uint32_t)(t * kTile + x.index(i)));
      return;
    }
    uint64_t sum = 0;
    if (r.from == kLowest) {                 // all: -inf weighs nothing
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += f.units.above(weight(f, x[i]));
      sum -= kPer * f.units.none();
    } else {
#pragma unroll
      for (int i = 0; i < kPer; i += kBeside) {
        float top = x[i];
#pragma unroll
        for (int j = 1; j < kBeside; ++j) top = fmaxf(top, x[i + j]);
        if (!__any(top >= r.to)) continue;
        if (__any(top >= r.from)) {
#pragma unroll
          for (int j = 0; j < kBeside; ++j) {
            sum += f.units.above(weight(f, x[i + j] >= r.from ? x[i + j] : -INFINITY));
          }
          sum -= kBeside * f.units.none();
        }
#pragma unroll
        for (int j = 0; j < kBeside; ++j) {
          if (x[i + j] >= r.to && x[i + j] < r.from) {
            const uint32_t n = atomicAdd(&s.n_list, 1u);
            if (n < kList) s.list[n] = order_of(x[i + j], (uint32_t)(t * kTile + x.index(i + j)));
          }
        }
      }
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) {
      if constexpr (kOne) sums[t] = sum;
      else tell(&sums[t], sum);
    }
  });
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

// Where in the order a filter ends.
struct Reached {
  uint64_t order, sum;                       // the last that stays; the weight up to it
};

// Where `target` tokens, or units of weight (by_weight; 0: top_p of all of it), are reached among those of orders base .. base + last
// up to `end`; all of them where they are fewer.  The stretch is cut into 1024 equal parts, each with its tokens and (sums) their
// weight, and the part in which the end is into 1024 again, until a wave can put a part's tokens in order: after six times at most,
// since an order has 52 bits.
template <typename T>
__device__ Reached reach(const Source<T>& from, const Row& f, uint64_t base, uint64_t last, bool by_weight, bool sums, uint64_t target,
                         uint64_t end, Shared& s) {
  const uint32_t tid = threadIdx.x;
  uint64_t sum_before = 0;
  for (int level = 0; level < 6; ++level) {
    const int shift = max(54 - __builtin_clzll(last | 1), 0);
    __syncthreads();
    s.sums[tid] = 0;
    s.counts[tid] = 0;
    if (tid == 0) s.n_few = 0;
    __syncthreads();
    for (uint32_t i = tid; i < from.n; i += kSThreads) {
      const uint64_t o = from[i], off = o - base;
      if (o > end || off > last) continue;
      atomicAdd(&s.counts[off >> shift], 1u);
      if (sums && logit_of(o) >= f.low)
        atomicAdd((unsigned long long*)&s.sums[off >> shift], (unsigned long long)f.units(weight(f, logit_of(o))));
    }
    __syncthreads();
    const uint32_t count = s.counts[tid];
    const uint64_t sum = s.sums[tid];
    uint32_t all = 0, place = 0;
    uint64_t total = 0, before = 0;
    if (!by_weight) place = scan(count, s, &all);
    if (sums) before = scan(sum, s, &total);
    if (level == 0) {
      if (by_weight && target == 0) target = part_of(f, total);
      if (!by_weight && all < target) return Reached{end, total};
    }
    const uint64_t here = by_weight ? before : place, more = by_weight ? sum : count;
    if (here < target && here + more >= target) {
      s.found[0] = tid;
      s.found[1] = target - here;
      s.found[2] = count;
      s.found[3] = before;
    }
    __syncthreads();
    base += s.found[0] << shift;
    last = (1ull << shift) - 1;
    target = s.found[1];
    const uint32_t there = (uint32_t)s.found[2];
    sum_before += s.found[3];
    if (there > 64) continue;
    for (uint32_t i = tid; i < from.n; i += kSThreads) {
      const uint64_t o = from[i];
      if (o > end || o - base > last) continue;
      const uint32_t at = atomicAdd(&s.n_few, 1u);
      if (at < 64) s.few[at] = o;
    }
    __syncthreads();
    if (tid < 64) {
      const uint64_t o = wave_sorted(tid < there ? s.few[tid] : ~0ull, there, s.few);
      const uint64_t u = sums && tid < there && logit_of(o) >= f.low ? f.units(weight(f, logit_of(o))) : 0, upto = wave_scan(u);
      if (by_weight ? upto - u < target && upto >= target : tid + 1 == target) s.found[0] = o, s.found[1] = sum_before + upto;
    }
    __syncthreads();
    return Reached{s.found[0], s.found[1]};
  }
  return Reached{base, sum_before};
}

__device__ void refuse(const SampleArgs& a, int64_t r) {
  a.tokens[r] = -1;
  if (a.logprobs) a.logprobs[r] = __builtin_nanf("");
  if (a.error) atomicAdd(a.error, 1u);
}

// The token of a row from its tiles' sums (s.tiles) and the tokens to be ordered (s.list, s.n_list of them).  Where the list does not
// hold those (a top_k from some thousand on beside a top_p; more than 6144 logits alike where a filter ends, such as masks of the type's
// lowest number under a top_k above what is left) one workgroup orders them from the row itself: 64 x 131072 in 0.44 to 0.58 ms, 1.05
// where all are alike and a top_p ends among them; with -inf for the masks it is 0.023.
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
  uint64_t mine, before, want = range.target, total, all;
  if (ordered && s.n_list <= 64) {           // a wave puts them in order; none where min_p lets none of a bin stay
    if (tid == 0) s.found[3] = end;
    if (tid < 64 && s.n_list > 0) {
      const uint32_t n = s.n_list, held = f.top_k && range.target < n ? (uint32_t)range.target : n;
      const uint64_t o = wave_sorted((uint32_t)tid < n ? s.list[tid] : ~0ull, n, s.few);
      const uint64_t u = (uint32_t)tid < held ? f.units(weight(f, logit_of(o))) : 0, upto = wave_scan(u);
      if (f.top_k) want = f.top_p < 1.f ? part_of(f, of_lane(upto, 63)) : ~0ull;
      const bool stays = (uint32_t)tid < held && upto - u < want;
      if (stays) atomicAdd((unsigned long long*)&s.tiles[index_of(o) / kTile], (unsigned long long)u);
      const uint64_t last = of_lane(o, 63 - __builtin_clzll(__ballot(stays)));
      if (tid == 0) s.found[3] = last;
    }
    __syncthreads();
    end = s.found[3];
  } else if (ordered) {
    // the list, or the whole row where the list does not hold what there is
    const Source<T> from{few ? nullptr : f.at, few ? s.n_list : (uint32_t)a.vocab, s.list};
    const float high = few ? fminf(range.from, (float)f.most) : (float)f.most, low = few ? range.to : f.low;
    const uint64_t base = (uint64_t)~key_of(high) << 20, last = ((uint64_t)~key_of(low) << 20 | 0xFFFFFu) - base;
    if (f.top_k) {
      const Reached r = reach(from, f, base, last, false, f.top_p < 1.f, few ? range.target : (uint64_t)f.top_k, end, s);
      end = r.order;
      want = part_of(f, r.sum);
    }
    if (f.top_p < 1.f) end = reach(from, f, base, last, true, true, f.top_k || few ? want : 0ull, end, s).order;
    if (few) {
      for (uint32_t i = tid; i < s.n_list; i += kSThreads) {
        const uint64_t o = s.list[i];
        if (o <= end)
          atomicAdd((unsigned long long*)&s.tiles[index_of(o) / kTile], (unsigned long long)f.units(weight(f, logit_of(o))));
      }
    } else {
      for (int t = wave; t < tiles; t += kSWaves) {
        Tile<T> x;
        x.load(f.at, t * kTile, a.vocab);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (x[i] >= f.low && order_of(x[i], (uint32_t)(t * kTile + x.index(i))) <= end) sum += f.units(weight(f, x[i]));
        }
        sum = wave_sum(sum);
        if ((tid & 63) == 0) s.tiles[t] = sum;
      }
    }
    __syncthreads();
  }
  // the first token whose running sum passes u * total
  mine = tid < tiles ? s.tiles[tid] : 0;
  before = scan(mine, s, &total);
  const uint64_t at = min((uint64_t)(fmin(fmax((double)f.u, 0.), 1.) * (double)total), total - 1);
  if (before <= at && before + mine > at) {
    s.found[0] = (uint64_t)tid;
    s.found[1] = at - before;
  }
  __syncthreads();
  const int i = (int)s.found[0] * kTile + tid;
  const uint64_t left = s.found[1], o = i < a.vocab ? Source<T>{f.at, 0, nullptr}[(uint32_t)i] : ~0ull;
  mine = o <= end && logit_of(o) >= f.low ? f.units(weight(f, logit_of(o))) : 0;
  before = scan(mine, s, &all);
  if (before <= left && before + mine > left) {
    a.tokens[r] = i;
    if (a.logprobs)
      a.logprobs[r] = (float)(((double)logit_of(o) - f.most) / (double)f.temperature - log((double)total * (f.units.magic * 0x1p-52)));
  }
}

// ------------------------------------------------------------------ kernels
//
// A token stays if it is among the top_k, its weight w = exp((l - most) / temperature) is min_p at least, and the weights before it
// in falling order are below top_p of those that stay so far; drawn is the first, by index, whose running sum of the weights that stay
// passes u of their sum.  No row is sorted: the logits' distances from the largest, in bins of 1 / 128 of a doubling, say in which bin
// the filter ends; the tokens above stay, those of the bin are put in order in LDS, and each tile's weights are summed on the way.  The
// draw looks at the tiles' sums and then at one tile.  So a row is read three times: largest, bins, sums (once, as long as it stays in
// registers).
// What bounds it: 1 x 32000 in fp16 takes 11.3 us of one workgroup's steps after one another; 64 x 131072 in bf16 three launches of
// 4.1, 14.2 and 21 us, of which the vector units are busy for 44, 47 and 36 % and the rest is the launches' ends and the last workgroup
// of a row, which puts the list in order.  256 x 150001 in fp32 takes 105 us, the time of the row of which most stays: 22 for the
// largest (memory, 7 TB/s), 34 for the bins, 41 for the sums (18 instructions of 64 bits a weight; 12 where few stay), 7 for the rest;
// 200 x 50021 without filters 20 us, 5 of a pass over memory and 10 of one of weights.  The largest alone (temperature 0): 1 x 32000
// 4.8 us, 64 x 131072 11.4, 256 x 150001 43.

// A workgroup has a row.
template <typename T, int kHold>
__global__ __launch_bounds__(kSThreads) void sample_row_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = a.first + blockIdx.x;
  Row f = row_of(a, r, __is_same(T, float) ? 4 : 2);
  const Tiles<T, kHold> tiles(f, a, 0);
  const float most = largest(tiles, s);
  if (f.bad || !(most > -INFINITY)) {
    if (threadIdx.x == 0) refuse(a, r);
    return;
  }
  f.most = (double)most;
  find_low(f, s);
  Range range{f.low, f.low, 0};
  if (f.temperature > 0.f && (f.top_k || f.top_p < 1.f)) {
    fill_bins(tiles, f, a, s);
    range = find_bins(f, a, s);
  }
  sum_tiles<true>(tiles, f, range, s.tiles, s);
  draw<T>(f, a, r, range, s);
}

__device__ __forceinline__ RowSpace* space_of(const SampleArgs& a, int64_t r) { return (RowSpace*)(a.workspace + r * a.ws_row); }

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
  const float most = largest(Tiles<T, 0>(f, a, part), s);
  if (tid == 0) w->part_max[part] = most;
}

template <typename T>
__global__ __launch_bounds__(kSThreads) void sample_bins_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - r * a.parts), tid = (int)threadIdx.x;
  RowSpace* w = space_of(a, r);
  Row f = row_of(a, r, __is_same(T, float) ? 4 : 2);
  const float most = join_max(w->part_max, a.parts);
  if (f.bad || !(most > -INFINITY) || f.temperature == 0.f || (!f.top_k && !(f.top_p < 1.f))) return;
  f.most = (double)most;
  find_low(f, s);
  fill_bins(Tiles<T, 0>(f, a, part), f, a, s);
  for (int b = tid; b < kBins; b += kSThreads) {
    if (f.top_k && s.counts_of[b])
      __hip_atomic_fetch_add((uint32_t*)&w->bins[b], s.counts_of[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (!f.top_k && s.bins[b]) __hip_atomic_fetch_add(&w->bins[b], s.bins[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (!is_last(&w->done[0], a.parts, s)) return;
  for (int b = tid; b < kBins; b += kSThreads) {
    if (f.top_k) s.counts_of[b] = read_back((uint32_t*)&w->bins[b]);
    else s.bins[b] = read_back(&w->bins[b]);
  }
  __syncthreads();
  const Range range = find_bins(f, a, s);
  if (tid == 0) w->range = range;
}

template <typename T>
__global__ __launch_bounds__(kSThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - r * a.parts), tid = (int)threadIdx.x;
  RowSpace* w = space_of(a, r);
  Row f = row_of(a, r, __is_same(T, float) ? 4 : 2);
  const float most = join_max(w->part_max, a.parts);
  if (f.bad || !(most > -INFINITY)) {
    if (part == 0 && tid == 0) refuse(a, r);
    return;
  }
  f.most = (double)most;
  find_low(f, s);
  Range range{f.low, f.low, 0};
  if (f.temperature > 0.f && (f.top_k || f.top_p < 1.f)) range = w->range;
  sum_tiles<false>(Tiles<T, 0>(f, a, part), f, range, w->tiles, s);
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

// Workgroups of a row: one below 48 tiles or where there are rows enough to fill the card, else one for each 16 tiles, as far as the card's
// 256 CUs go.  Us by the rule's several workgroups and by one (bf16; no filter; a top_p; users' different wishes):
//    1 x 40000    15 and 12, 23 and 19, 23 and 18        64 x 40000    16 and 13, 33 and 30, 34 and 31
//    1 x 49152    13 and 14, 22 and 22, 21 and 21        64 x 49152    14 and 14, 32 and 36, 31 and 36
//    1 x 131072   13 and 29, 22 and 45, 22 and 42        64 x 131072   18 and 30, 41 and 75, 39 and 73
// A small top_k in every row leaves little to share: up to 98304 tokens one is faster (65536: 16 instead of 21), which the host does not
// see.  64 x 131072 with 128 workgroups in all takes 54 us, with 256 39, with 512 42; 200 x 50021 with up to 512, which is two a row and
// three launches instead of one, 36 instead of 22.
constexpr int kFull = 256;
constexpr int kLeastShared = 3 * kSWaves;
int parts_of(int32_t n_rows, int32_t vocab) {
  const int tiles = (vocab + kTile - 1) / kTile;
  if (tiles < kLeastShared) return 1;
  return std::max(1, std::min({(int)kMostParts, kFull / std::max(n_rows, 1), tiles / kSWaves}));
}

// A launch has fewer than 2^32 threads.
constexpr int kMostRows = 1 << 21;

template <typename T>
void launch_sample(SampleArgs a, int32_t n_rows, hipStream_t s) {
  const dim3 block(kSThreads);
  if (a.parts == 1) {
    for (; a.first < n_rows; a.first += kMostRows) {
      const dim3 grid((unsigned)std::min<int64_t>(n_rows - a.first, kMostRows));
      if (a.vocab <= kHeld * kSWaves * kTile) hipLaunchKernelGGL((sample_row_kernel<T, kHeld>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((sample_row_kernel<T, 0>), grid, block, 0, s, a);
    }
  } else {
    const dim3 grid((unsigned)(n_rows * a.parts));
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

int sbm_sample(const sbm_sample_args* args, void* stream) {
  if (!args) return fail(SBM_EINVAL, "null pointer");
  const auto [logits, row_stride, uniforms, temperature, top_k, top_p, min_p, tokens, logprobs, workspace, workspace_bytes, error, n_rows,
              vocab, flags, reserved] = *args;
  if (reserved) return fail(SBM_EINVAL, "reserved must be 0");
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
                     row_space(vocab), 0, vocab, parts_of(n_rows, vocab)};
  if (flags & SBM_F_IN_F32) launch_sample<float>(a, n_rows, (hipStream_t)stream);
  else if (flags & SBM_F_IN_BF16) launch_sample<__bf16>(a, n_rows, (hipStream_t)stream);
  else launch_sample<_Float16>(a, n_rows, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "sample launch: %s", hipGetErrorString(e));
  return SBM_OK;
}

}  // extern "C"
