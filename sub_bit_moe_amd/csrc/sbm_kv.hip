// The serving operators around the attention: the plan of a step over a paged
// cache, norms and rotation of queries and keys with the 4-bit cache's writer,
// and the cache's reader.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sbm_kv4.h"

namespace sbm {
namespace {

// ------------------------------------------------------------------ the plan

constexpr int kPThreads = 256;

struct PlanArgs {
  const int32_t* ctx;
  const int32_t* fresh;
  const int32_t* free_blocks;
  const int32_t* n_free;
  int32_t* table;
  int32_t* slots;
  int32_t* positions;
  int32_t* requests;
  int32_t* cu_q;
  int32_t* kv_lens;
  int32_t* n_free_out;
  uint32_t* error;
  int32_t n_requests, free_capacity, width, n_blocks, shift, max_tokens;   // block_size = 1 << shift
};

// Sums of lengths that stop at 2^31 - 1 instead of wrapping (a + b of two such
// values fits 32 bits unsigned).
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, 0x7FFFFFFFu); }

__device__ __forceinline__ uint32_t blocks_of(uint32_t tokens, int shift) {
  return (tokens >> shift) + ((tokens & ((1u << shift) - 1u)) != 0);
}

// The largest i with p[i] <= v among p[0 .. n - 1], p[0] = 0 and rising.
__device__ __forceinline__ int last_at_most(const uint32_t* p, int n, uint32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Every workgroup scans all the lengths (at most 4096, so one to sixteen
// rounds) into its LDS and then fills its share of the tokens and new blocks by
// binary search: one launch, no workgroup waits for another.  Bound by latency:
// lengths, scan, search, free list, store (64 requests 4 us, 512 requests with
// 60512 new tokens 6 us).
__global__ __launch_bounds__(kPThreads) void plan_kernel(PlanArgs a) {
  __shared__ uint32_t s_tok[kMaxRequests + 1], s_need[kMaxRequests + 1];
  __shared__ uint32_t s_wave[2][kPThreads / 64], s_bad;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, R = a.n_requests;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  uint32_t tok0 = 0, need0 = 0;                  // sums before these lengths
  for (int base = 0; base < R; base += kPThreads) {
    const int r = base + tid;
    uint32_t tok = 0, need = 0;
    if (r < R) {
      const int32_t c = a.ctx[r], n = a.fresh[r];
      if (c < 0 || c > (1 << 30) || n < 0) {
        atomicOr(&s_bad, SBM_PLAN_ELENGTH);
      } else if (n > a.max_tokens) {
        atomicOr(&s_bad, SBM_PLAN_ETOKENS);
      } else {
        const uint32_t total = blocks_of((uint32_t)c + (uint32_t)n, a.shift);
        if (total > (uint32_t)a.width) atomicOr(&s_bad, SBM_PLAN_EWIDTH);
        tok = (uint32_t)n;
        need = total - blocks_of((uint32_t)c, a.shift);
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t t = __shfl_up(tok, d, 64), n = __shfl_up(need, d, 64);
      if (lane >= d) {
        tok = add_sat(tok, t);
        need = add_sat(need, n);
      }
    }
    if (lane == 63) {
      s_wave[0][wave] = tok;
      s_wave[1][wave] = need;
    }
    __syncthreads();
    uint32_t tb = tok0, nb = need0;
#pragma unroll
    for (int w = 0; w < kPThreads / 64; ++w) {
      if (w == wave) {
        tok = add_sat(tok, tb);
        need = add_sat(need, nb);
      }
      tb = add_sat(tb, s_wave[0][w]);
      nb = add_sat(nb, s_wave[1][w]);
    }
    if (r < R) {
      s_tok[r + 1] = tok;
      s_need[r + 1] = need;
    }
    if (r == 0) s_tok[0] = s_need[0] = 0;
    tok0 = tb;
    need0 = nb;
    __syncthreads();
  }
  const int32_t nf = *a.n_free;
  uint32_t bad = s_bad;
  if (tok0 > (uint32_t)a.max_tokens) bad |= SBM_PLAN_ETOKENS;
  if (nf < 0 || nf > a.free_capacity || need0 > (uint32_t)nf) bad |= SBM_PLAN_EPOOL;
  const int64_t g0 = (int64_t)blockIdx.x * kPThreads + tid, step = (int64_t)gridDim.x * kPThreads;
  if (g0 == 0) {
    *a.n_free_out = bad ? nf : nf - (int32_t)need0;
    a.cu_q[0] = 0;
    if (bad && a.error) atomicOr(a.error, bad);
  }
  for (int64_t r = g0; r < R; r += step) {
    const int32_t c = a.ctx[r];
    a.cu_q[r + 1] = bad ? 0 : (int32_t)s_tok[r + 1];
    a.kv_lens[r] = bad ? max(c, 0) : c + a.fresh[r];
  }
  const uint32_t n_tok = bad ? 0u : tok0, n_need = bad ? 0u : need0;
  for (int64_t t = g0; t < a.max_tokens; t += step) {
    int32_t slot = -1, pos = 0, req = -1;
    if (t < n_tok) {
      req = last_at_most(s_tok, R, (uint32_t)t);
      const int32_t c = a.ctx[req];
      pos = c + (int32_t)((uint32_t)t - s_tok[req]);
      const uint32_t col = (uint32_t)pos >> a.shift, held = blocks_of((uint32_t)c, a.shift);
      // a column of this step comes from the free list: the table's entry may not be written yet
      const int32_t b = col < held ? a.table[(int64_t)req * a.width + col]
                                   : a.free_blocks[nf - 1 - (int32_t)(s_need[req] + col - held)];
      if ((uint32_t)b < (uint32_t)a.n_blocks) slot = (b << a.shift) + (pos & ((1 << a.shift) - 1));
      else if (a.error) atomicOr(a.error, SBM_PLAN_EBLOCK);
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
    a.requests[t] = req;
  }
  for (int64_t f = g0; f < n_need; f += step) {
    const int req = last_at_most(s_need, R, (uint32_t)f);
    const uint32_t held = blocks_of((uint32_t)a.ctx[req], a.shift);
    a.table[(int64_t)req * a.width + held + ((uint32_t)f - s_need[req])] = a.free_blocks[nf - 1 - (int32_t)f];
  }
}

// ------------------------------------------------------------------ norms, rotation, cache

constexpr int kQThreads = 256;

struct QkArgs {
  const uint16_t *q, *k, *v, *qw, *kw;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  uint16_t *q_out, *k_out;
  int64_t qo_ts, qo_hs, ko_ts, ko_hs;
  const int32_t* positions;
  const float* rope;
  const int32_t* slots;
  uint8_t* cache;
  uint32_t* error;
  double eps;
  int32_t rope_rows, rot, n_tokens, heads, kv_heads, n_blocks, shift, neighbours;
  int32_t per_token;     // log2 of the groups of lanes that a token has in a workgroup
};

template <typename T>
__device__ __forceinline__ float to_f32(uint16_t u) {
  if constexpr (__is_same(T, __bf16)) return __uint_as_float((uint32_t)u << 16);
  else return (float)__builtin_bit_cast(_Float16, u);
}

// Eight elements: one 16-byte access where every address allows it (kVec), else eight.
template <bool kVec>
__device__ __forceinline__ void load8(const uint16_t* p, uint16_t* x) {
  if constexpr (kVec) {
    *(uint4*)x = *(const uint4*)p;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = p[j];
  }
}

template <bool kVec>
__device__ __forceinline__ void store8(uint16_t* p, const uint16_t* x) {
  if constexpr (kVec) {
    *(uint4*)p = *(const uint4*)x;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = x[j];
  }
}

// One rounding to T.  From 64 bits the way goes over 32, so what those cannot
// hold is first gathered in their lowest bit (round to odd): the second
// rounding then sees on which side of a border the value was.
template <typename T>
__device__ __forceinline__ uint16_t round_once(float y) {
  return __builtin_bit_cast(uint16_t, (T)y);
}
template <typename T>
__device__ __forceinline__ uint16_t round_once(double y) {
  uint64_t b = __builtin_bit_cast(uint64_t, y);
  const uint32_t low = (uint32_t)b & 0x1FFFFFFFu;
  b = (b & ~0x1FFFFFFFull) | (low ? 0x20000000u : 0u);
  return round_once<T>((float)__builtin_bit_cast(double, b));
}

// v summed over groups of kL lanes, in all of them.
template <int kCtrl>
__device__ __forceinline__ float other_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xF, 0xF, true));
}
template <int kCtrl>
__device__ __forceinline__ double other_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int kL, typename C>
__device__ __forceinline__ C group_sum(C v) {
  v += other_lane<0xB1>(v);                        // neighbours, neighbouring pairs, mirrored eights and sixteens
  v += other_lane<0x4E>(v);
  v += other_lane<0x141>(v);
  if constexpr (kL > 8) v += other_lane<0x140>(v);
  if constexpr (kL > 16) v += __shfl_xor(v, 16, 64);
  return v;
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

// What a lane keeps of its token and its eight dimensions for all the heads it takes.
struct QkLane {
  float cos[8], sin[8];
  int d0, p0;                // its first dimension, and that of the partners (halves)
  bool turn, split, low;     // rotated; with partners eight apart or more; those are the higher ones
};

// A lane's eight elements after the norm, x, and their partners z become x * own + z * with: weight and rotation in one
// factor each, the same for all the heads.  An element that is not rotated is its own partner, times 0.
template <typename C>
struct QkTurn {
  C own[8], with[8];
};

template <typename T, typename C, bool kVec>
__device__ __forceinline__ void load_turn(QkTurn<C>& r, const uint16_t* weight, const QkLane& l) {
  constexpr uint16_t kOne = __is_same(T, __bf16) ? 0x3F80 : 0x3C00;
  uint16_t w[8], z[8];
  if (weight) {
    load8<kVec>(weight + l.d0, w);
    load8<kVec>(weight + l.p0, z);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = z[j] = kOne;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) r.own[j] = (C)to_f32<T>(w[j]), r.with[j] = (C)0;
  if (l.split) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r.own[j] *= (C)l.cos[j];
      r.with[j] = (C)to_f32<T>(z[j]) * (C)(l.low ? -l.sin[j] : l.sin[j]);
    }
  } else if (l.turn) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r.own[j] *= (C)l.cos[j >> 1];
      r.with[j] = (C)to_f32<T>(w[j ^ 1]) * (C)(j & 1 ? l.sin[j >> 1] : -l.sin[j >> 1]);
    }
  }
}

__device__ __forceinline__ float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fused(double a, double b, double c) { return __builtin_fma(a, b, c); }

// Norm and rotation of a lane's eight elements of one head; C: the type it is computed in.
template <typename T, typename C, int D>
__device__ __forceinline__ void norm_rope8(const uint16_t* raw, uint16_t* other, const QkTurn<C>& r, const QkLane& l,
                                           const QkArgs& a, uint16_t* out) {
  C x[8], ss = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = (C)to_f32<T>(raw[j]);
    ss = fused(x[j], x[j], ss);
  }
  ss = group_sum<D / 8>(ss);
  if (l.turn && !l.split) {
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = raw[j ^ 1];
  }
  const C mean = ss * ((C)1 / (C)D) + (C)a.eps;
  if constexpr (sizeof(C) == 4 && __is_same(T, __bf16)) {
    // squares that 32 bits do not hold (beyond 1e15 and, with an eps of 0, below 1e-15): the mean in 64; a head's lanes all
    // come here or none
    if (__builtin_expect(!(mean > 1e-30f && mean < 1e30f), 0)) {
      double sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fused((double)x[j], (double)x[j], sum);
      const double inv = inverse_root(group_sum<D / 8>(sum) * (1. / D) + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        out[j] = round_once<T>(fused((float)((double)to_f32<T>(other[j]) * inv), r.with[j],
                                     (float)((double)x[j] * inv) * r.own[j]));
      return;
    }
  }
  const C inv = inverse_root(mean);
  // the norm first: its results are sqrt(D) at most, whatever the elements and the weights are
#pragma unroll
  for (int j = 0; j < 8; ++j)
    out[j] = round_once<T>(fused((C)to_f32<T>(other[j]) * inv, r.with[j], (x[j] * inv) * r.own[j]));
}

// Eight of a block's 32 values (four neighbouring lanes hold them) to codes and the block's scale.
template <typename T>
__device__ __forceinline__ uint32_t quantise8(const uint16_t* x, uint32_t* scale) {
  constexpr uint32_t most = __is_same(T, __bf16) ? 252 : 140;
  float f[8];
  uint32_t top = 0;                               // magnitudes order as their bits do, NaN above infinity
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = to_f32<T>(x[j]);
    top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  }
  top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
  if (top >= 0x7F800000u) {
    *scale = kScaleNaN;
    return 0;
  }
  // 7 * 2^e = 1.75 * 2^(e + 2)
  const int32_t e = (int32_t)(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x600000u);
  const uint32_t s = (uint32_t)min(max(e, 1), (int32_t)most);
  *scale = s;
  // the conversion rounds to nearest, ties to even, and takes 7 down to 6; the division is by the multiplication, which keeps
  // what is below the normal numbers
  const float by = __uint_as_float((254u - s) << 23);
  uint32_t codes = 0;
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[0] * by, f[1] * by, 1.f, 0);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[2] * by, f[3] * by, 1.f, 1);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[4] * by, f[5] * by, 1.f, 2);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[6] * by, f[7] * by, 1.f, 3);
  return codes;
}

// D / 8 lanes hold a head (16-byte accesses) and take every so-manieth head of one token, so that its cosines and sines
// and the weights are read, and multiplied with each other, once for all of them.  A wave has a token to itself: with the
// groups of a workgroup on one token a group has too few heads for that (2000 tokens of 32 + 8 + 8 heads of 128: 14.8, not
// 11.9 us).  A few tokens' heads are shared out over gridDim.y.  The instructions count: with the products of weight and
// rotation made for each head, and codes by comparing, 8191 tokens of 40 + 8 + 8 heads of 128 took 59 us, 98 % of them
// issuing vector instructions; now 42 us (5.0 TB/s) and 79 %.  Bound by HBM for prompts (4096 tokens of 32 + 8 heads, 86 MB:
// 17.2 us, 5.0 TB/s),
// by latency for a few tokens (64 tokens: 4 us).
template <typename T, int D, bool kVec>
__global__ __launch_bounds__(kQThreads, 4) void qk_kernel(QkArgs a) {
  constexpr int L = D / 8, kGroups = kQThreads / L;
  const uint32_t group = threadIdx.x / L;
  const uint32_t t = blockIdx.x * ((uint32_t)kGroups >> a.per_token) + (group >> a.per_token);
  uint32_t h = (group & ((1u << a.per_token) - 1u)) + (blockIdx.y << a.per_token);
  const uint32_t step = gridDim.y << a.per_token;
  const uint32_t heads = (uint32_t)a.heads, kv_heads = (uint32_t)a.kv_heads;
  const uint32_t all = heads + kv_heads + (a.cache ? kv_heads : 0);
  if (t >= (uint32_t)a.n_tokens || h >= all) return;
  QkLane l;
  l.d0 = (int)(threadIdx.x % L) * 8;
  const int half = a.rot >> 1;
  l.turn = l.d0 < a.rot;
  l.split = l.turn && !a.neighbours;
  l.low = l.d0 < half;
  l.p0 = !l.split ? l.d0 : l.low ? l.d0 + half : l.d0 - half;
  const float* rope = a.rope;
  bool ok = true;
  if (a.rot) {
    const int32_t pos = a.positions[t];
    ok = (uint32_t)pos < (uint32_t)a.rope_rows;
    if (ok) rope += (int64_t)pos * a.rot;
  }
  int64_t slot = -1;
  if (a.cache) {
    slot = a.slots[t];
    if (slot >= ((int64_t)a.n_blocks << a.shift)) {
      if (h == 0 && l.d0 == 0 && a.error) atomicAdd(a.error, 1u);
      slot = -1;
    }
  }
  if (!ok) {
    if (h == 0 && l.d0 == 0 && a.error) atomicAdd(a.error, 1u);
    return;
  }
  if (l.turn) {
    // neighbours: four of each
    const float* cs = rope + (a.neighbours ? l.d0 >> 1 : l.low ? l.d0 : l.d0 - half);
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      if (j && a.neighbours) break;
      if constexpr (kVec) {
        const float4 c = *(const float4*)(cs + j), s = *(const float4*)(cs + half + j);
        l.cos[j] = c.x, l.cos[j + 1] = c.y, l.cos[j + 2] = c.z, l.cos[j + 3] = c.w;
        l.sin[j] = s.x, l.sin[j + 1] = s.y, l.sin[j + 2] = s.z, l.sin[j + 3] = s.w;
      } else {
#pragma unroll
        for (int k = j; k < j + 4; ++k) l.cos[k] = cs[k], l.sin[k] = cs[half + k];
      }
    }
  }
  uint16_t y[8];
  if (h < heads) {
    QkTurn<float> r;
    load_turn<T, float, kVec>(r, a.qw, l);
    // kAhead heads are read together
    constexpr int kAhead = 2;
    for (; h < heads; h += kAhead * step) {
      uint16_t raw[kAhead][8], other[kAhead][8];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint32_t at = h + i * step < heads ? h + i * step : h;
        const uint16_t* q = a.q + t * a.q_ts + at * a.q_hs;
        load8<kVec>(q + l.d0, raw[i]);
        load8<kVec>(q + l.p0, other[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        norm_rope8<T, float, D>(raw[i], other[i], r, l, a, y);
        if (h + i * step < heads) store8<kVec>(a.q_out + t * a.qo_ts + (h + i * step) * a.qo_hs + l.d0, y);
      }
    }
    // the first that is not a query's
    h -= ((h - heads) / step) * step;
  }
  if (h >= all) return;
  QkTurn<double> r;
  load_turn<T, double, kVec>(r, a.kw, l);
  const int64_t bs = 1ll << a.shift, row = slot & (bs - 1);
  for (; h < all; h += step) {
    const bool is_v = h >= heads + kv_heads;
    const uint32_t kh = h - heads - (is_v ? kv_heads : 0);
    if (is_v) {
      if (slot < 0) return;
      load8<kVec>(a.v + t * a.v_ts + kh * a.v_hs + l.d0, y);
    } else {
      uint16_t raw[8], other[8];
      load8<kVec>(a.k + t * a.k_ts + kh * a.k_hs + l.d0, raw);
      load8<kVec>(a.k + t * a.k_ts + kh * a.k_hs + l.p0, other);
      norm_rope8<T, double, D>(raw, other, r, l, a, y);
      if (a.k_out) store8<kVec>(a.k_out + t * a.ko_ts + kh * a.ko_hs + l.d0, y);
      if (slot < 0) continue;
    }
    uint32_t scale;
    const uint32_t codes = quantise8<T>(y, &scale);
    uint8_t* rec = a.cache + ((slot >> a.shift) * a.kv_heads + kh) * kv_record_bytes((int32_t)bs, D);
    *(uint32_t*)(rec + (is_v ? bs * (D / 2) : 0) + row * (D / 2) + l.d0 / 2) = codes;
    if ((l.d0 & 31) == 0) rec[bs * D + (is_v ? bs * (D / 32) : 0) + row * (D / 32) + l.d0 / 32] = (uint8_t)scale;
  }
}

// ------------------------------------------------------------------ the cache's reader

// A lane has eight values of a head: 4 bytes of codes read, 16 of values written.  Bound by HBM for prompts (8191 tokens of
// 8 + 8 heads of 128: 10.5 us, 4.0 TB/s), by latency for a few tokens (64: 2.9 us).
template <typename T, int D>
__global__ __launch_bounds__(kQThreads) void load_kernel(const uint8_t* cache, int32_t n_blocks, int32_t kv_heads,
                                                         int32_t shift, const int32_t* slots, uint32_t n_tokens,
                                                         uint16_t* k, uint16_t* v, uint32_t* error) {
  constexpr int L = D / 8;
  const uint32_t both = k && v ? 2u * (uint32_t)kv_heads : (uint32_t)kv_heads;
  const uint32_t unit = blockIdx.x * (kQThreads / L) + threadIdx.x / L;
  const uint32_t t = unit / both, h = unit - t * both;
  if (t >= n_tokens) return;
  const int d0 = (int)(threadIdx.x % L) * 8;
  const bool is_v = !k || h >= (uint32_t)kv_heads;
  const uint32_t kh = h >= (uint32_t)kv_heads ? h - (uint32_t)kv_heads : h;
  int64_t slot = slots[t];
  if (slot >= ((int64_t)n_blocks << shift)) {
    if (h == 0 && d0 == 0 && error) atomicAdd(error, 1u);
    slot = -1;
  }
  uint4 out = make_uint4(0u, 0u, 0u, 0u);
  if (slot >= 0) {
    const int64_t bs = 1ll << shift, row = slot & (bs - 1);
    const uint8_t* rec = cache + ((slot >> shift) * kv_heads + kh) * kv_record_bytes((int32_t)bs, D);
    const uint32_t codes = *(const uint32_t*)(rec + (is_v ? bs * (D / 2) : 0) + row * (D / 2) + d0 / 2);
    const uint32_t s = rec[bs * D + (is_v ? bs * (D / 32) : 0) + row * (D / 32) + d0 / 32];
    const float scale = __uint_as_float(s << 23);
    out.x = cvt_fp4<T, 0>(codes, scale);
    out.y = cvt_fp4<T, 1>(codes, scale);
    out.z = cvt_fp4<T, 2>(codes, scale);
    out.w = cvt_fp4<T, 3>(codes, scale);
  }
  *(uint4*)((is_v ? v : k) + ((int64_t)t * kv_heads + kh) * D + d0) = out;
}

// int32 arrays of a plan.
struct Ints {
  const void* p;
  int64_t n;
};

bool overlap(Ints a, Ints b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.n > 0 && b.n > 0 && x < y + 4 * (uintptr_t)b.n && y < x + 4 * (uintptr_t)a.n;
}

bool vec_ok(const void* p, int64_t ts, int64_t hs) {
  return !p || (((uintptr_t)p & 15u) == 0 && ts % 8 == 0 && hs % 8 == 0);
}

// Workgroups that fill the chip: with fewer tokens their heads are shared out.
constexpr int64_t kQFull = 1024;

template <typename T, int D>
void launch_qk(QkArgs a, bool vec, hipStream_t s) {
  constexpr int kGroups = kQThreads / (D / 8);
  const int64_t all = a.heads + a.kv_heads + (a.cache ? a.kv_heads : 0);
  // as many groups of lanes for a token as it has heads, a wave's at most
  a.per_token = 0;
  while ((1 << a.per_token) < 64 / (D / 8) && (1 << a.per_token) < all) ++a.per_token;
  const int64_t tokens = kGroups >> a.per_token, x = (a.n_tokens + tokens - 1) / tokens;
  const int64_t rounds = (all + (1 << a.per_token) - 1) >> a.per_token;
  const int64_t y = std::min<int64_t>(std::min<int64_t>(rounds, std::max<int64_t>(kQFull / x, 1)), 65535);
  const dim3 grid((unsigned)x, (unsigned)y);
  if (vec) hipLaunchKernelGGL((qk_kernel<T, D, true>), grid, dim3(kQThreads), 0, s, a);
  else hipLaunchKernelGGL((qk_kernel<T, D, false>), grid, dim3(kQThreads), 0, s, a);
}

}  // namespace
}  // namespace sbm

using namespace sbm;

extern "C" {

size_t sbm_kv_cache_bytes(int32_t n_blocks, int32_t n_kv_heads, int32_t block_size, int32_t head_dim) {
  if (n_blocks <= 0 || n_kv_heads <= 0 || !kv_shape_ok(block_size, head_dim)) return 0;
  return (size_t)n_blocks * (size_t)n_kv_heads * (size_t)kv_record_bytes(block_size, head_dim);
}

int sbm_kv_plan(const int32_t* context_lens, const int32_t* new_lens, int32_t n_requests,
                const int32_t* free_blocks, int32_t free_capacity, const int32_t* n_free,
                int32_t* block_table, int32_t table_width, int32_t n_blocks, int32_t block_size,
                int32_t max_tokens, int32_t* slots, int32_t* positions, int32_t* requests, int32_t* cu_q,
                int32_t* kv_lens, int32_t* n_free_out, uint32_t* error, void* stream) {
  if (n_requests < 0 || n_requests > kMaxRequests)
    return fail(SBM_EINVAL, "n_requests=%d outside 0..%d", n_requests, kMaxRequests);
  if (!kv_shape_ok(block_size, 64)) return fail(SBM_EINVAL, "block_size=%d is no power of two from 16 to 4096", block_size);
  if (free_capacity < 0 || table_width < 0 || n_blocks < 0 || max_tokens < 0 || max_tokens >= (1 << 30))
    return fail(SBM_EINVAL, "bad free_capacity=%d, table_width=%d, n_blocks=%d or max_tokens=%d", free_capacity,
                table_width, n_blocks, max_tokens);
  if ((int64_t)n_blocks * block_size > 0x7FFFFFFF)
    return fail(SBM_ERANGE, "%d blocks of %d tokens do not fit 32-bit slots", n_blocks, block_size);
  if (!n_free || !cu_q || !n_free_out || (n_requests && (!context_lens || !new_lens || !kv_lens)) ||
      (n_requests && table_width && !block_table) || (free_capacity && !free_blocks) ||
      (max_tokens && (!slots || !positions || !requests)))
    return fail(SBM_EINVAL, "null pointer");
  if (n_free == n_free_out) return fail(SBM_EINVAL, "n_free_out must not be n_free");
  if (n_requests && (kv_lens == context_lens || kv_lens == new_lens))
    return fail(SBM_EINVAL, "kv_lens must not be one of the input lengths");
  // lengths are read again where blocks are filled in: overwritten by then, they would index past the table
  const Ints ins[] = {{context_lens, n_requests}, {new_lens, n_requests}, {free_blocks, free_capacity}, {n_free, 1}};
  const Ints outs[] = {{block_table, (int64_t)n_requests * table_width}, {slots, max_tokens}, {positions, max_tokens},
                       {requests, max_tokens}, {cu_q, (int64_t)n_requests + 1}, {kv_lens, n_requests}, {n_free_out, 1},
                       {error, error ? 1 : 0}};
  for (const Ints& o : outs) {
    for (const Ints& i : ins)
      if (overlap(o, i)) return fail(SBM_EINVAL, "an output overlaps an input");
    for (const Ints& other : outs)
      if (&other < &o && overlap(o, other)) return fail(SBM_EINVAL, "outputs overlap");
  }
  PlanArgs a{context_lens, new_lens, free_blocks, n_free, block_table, slots, positions, requests, cu_q, kv_lens,
             n_free_out, error, n_requests, free_capacity, table_width, n_blocks, __builtin_ctz((unsigned)block_size),
             max_tokens};
  const int64_t most = std::max<int64_t>(max_tokens, n_requests);
  const unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>((most + kPThreads - 1) / kPThreads, 1), 512);
  hipLaunchKernelGGL(plan_kernel, dim3(grid), dim3(kPThreads), 0, (hipStream_t)stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "plan launch: %s", hipGetErrorString(e));
  return SBM_OK;
}

int sbm_qk_norm_rope(const sbm_heads* q, const sbm_heads* k, const sbm_heads* v, const uint16_t* q_weight,
                     const uint16_t* k_weight, const int32_t* positions, const float* rope, int32_t rope_rows,
                     int32_t rot_dim, double eps, int32_t n_tokens, int32_t n_heads, int32_t n_kv_heads,
                     int32_t head_dim, const sbm_heads* q_out, const sbm_heads* k_out, const int32_t* slots,
                     uint8_t* cache, int32_t n_blocks, int32_t block_size, uint32_t flags, uint32_t* error,
                     void* stream) {
  if (flags & ~(SBM_F_IN_BF16 | SBM_F_NEIGHBOURS)) return fail(SBM_EINVAL, "unknown flags 0x%x", flags);
  if (n_tokens < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads > 65536 || n_kv_heads > 65536)
    return fail(SBM_EINVAL, "bad n_tokens=%d, n_heads=%d or n_kv_heads=%d", n_tokens, n_heads, n_kv_heads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(SBM_EINVAL, "head_dim=%d is not 64, 128 or 256", head_dim);
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
    return fail(SBM_EINVAL, "rot_dim=%d is no multiple of 16 up to head_dim=%d", rot_dim, head_dim);
  if (!(eps >= 0.)) return fail(SBM_EINVAL, "bad eps");
  if (rot_dim && rope_rows < 0) return fail(SBM_EINVAL, "rope_rows=%d", rope_rows);
  if (cache) {
    if (!kv_shape_ok(block_size, head_dim))
      return fail(SBM_EINVAL, "block_size=%d is no power of two from 16 to 4096", block_size);
    if (n_blocks <= 0) return fail(SBM_EINVAL, "n_blocks=%d", n_blocks);
    if ((int64_t)n_blocks * block_size > 0x7FFFFFFF)
      return fail(SBM_ERANGE, "%d blocks of %d tokens do not fit 32-bit slots", n_blocks, block_size);
    if ((uintptr_t)cache & 15u) return fail(SBM_EINVAL, "cache must be 16-byte aligned");
  }
  if (n_tokens == 0) return SBM_OK;
  if ((int64_t)n_tokens * ((int64_t)n_heads + 2 * (int64_t)n_kv_heads) > 0x7FFFFFFF)
    return fail(SBM_ERANGE, "too many heads of tokens");
  if (!q || !q->data || !k || !k->data || !q_out || !q_out->data || (rot_dim && (!positions || !rope)) ||
      (cache && (!v || !v->data || !slots)) || (!cache && (!k_out || !k_out->data)))
    return fail(SBM_EINVAL, "null pointer");
  const sbm_heads none{nullptr, 0, 0};
  const sbm_heads vv = cache ? *v : none, ko = k_out ? *k_out : none;
  for (const sbm_heads* p : {q, k, (const sbm_heads*)&vv, q_out, (const sbm_heads*)&ko})
    if ((uintptr_t)p->data & 1u) return fail(SBM_EINVAL, "misaligned heads");
  QkArgs a{(const uint16_t*)q->data, (const uint16_t*)k->data, (const uint16_t*)vv.data, q_weight, k_weight,
           q->token_stride, q->head_stride, k->token_stride, k->head_stride, vv.token_stride, vv.head_stride,
           (uint16_t*)q_out->data, (uint16_t*)ko.data, q_out->token_stride, q_out->head_stride, ko.token_stride,
           ko.head_stride, positions, rope, slots, cache, error, eps, rope_rows, rot_dim, n_tokens, n_heads,
           n_kv_heads, n_blocks, cache ? __builtin_ctz((unsigned)block_size) : 0,
           (flags & SBM_F_NEIGHBOURS) ? 1 : 0, 0};
  bool vec = (((uintptr_t)rope | (uintptr_t)q_weight | (uintptr_t)k_weight) & 15u) == 0;
  for (const sbm_heads* p : {q, k, (const sbm_heads*)&vv, q_out, (const sbm_heads*)&ko})
    vec = vec && vec_ok(p->data, p->token_stride, p->head_stride);
  hipStream_t s = (hipStream_t)stream;
  if (flags & SBM_F_IN_BF16) {
    if (head_dim == 64) launch_qk<__bf16, 64>(a, vec, s);
    else if (head_dim == 128) launch_qk<__bf16, 128>(a, vec, s);
    else launch_qk<__bf16, 256>(a, vec, s);
  } else {
    if (head_dim == 64) launch_qk<_Float16, 64>(a, vec, s);
    else if (head_dim == 128) launch_qk<_Float16, 128>(a, vec, s);
    else launch_qk<_Float16, 256>(a, vec, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "qk_norm_rope launch: %s", hipGetErrorString(e));
  return SBM_OK;
}

int sbm_kv_load(const uint8_t* cache, int32_t n_blocks, int32_t n_kv_heads, int32_t block_size, int32_t head_dim,
                const int32_t* slots, int32_t n_tokens, uint16_t* k, uint16_t* v, uint32_t flags, uint32_t* error,
                void* stream) {
  if (flags & ~SBM_F_IN_BF16) return fail(SBM_EINVAL, "unknown flags 0x%x", flags);
  if (n_tokens < 0 || n_kv_heads <= 0 || n_kv_heads > 65536 || n_blocks <= 0 || !kv_shape_ok(block_size, head_dim))
    return fail(SBM_EINVAL, "bad shape: n_tokens=%d, n_kv_heads=%d, n_blocks=%d, block_size=%d, head_dim=%d", n_tokens,
                n_kv_heads, n_blocks, block_size, head_dim);
  if ((int64_t)n_blocks * block_size > 0x7FFFFFFF)
    return fail(SBM_ERANGE, "%d blocks of %d tokens do not fit 32-bit slots", n_blocks, block_size);
  if ((int64_t)n_tokens * n_kv_heads * 2 > 0x7FFFFFFF) return fail(SBM_ERANGE, "too many heads of tokens");
  if (n_tokens == 0 || (!k && !v)) return SBM_OK;
  if (!cache || !slots) return fail(SBM_EINVAL, "null pointer");
  if (((uintptr_t)cache | (uintptr_t)k | (uintptr_t)v) & 15u)
    return fail(SBM_EINVAL, "cache, k and v must be 16-byte aligned");
  const int64_t units = (int64_t)n_tokens * n_kv_heads * (k && v ? 2 : 1);
  const int per = kQThreads / (head_dim / 8), shift = __builtin_ctz((unsigned)block_size);
  const dim3 grid((unsigned)((units + per - 1) / per)), threads(kQThreads);
  hipStream_t s = (hipStream_t)stream;
#define SBM_LOAD(T, D)                                                                                            \
  hipLaunchKernelGGL((load_kernel<T, D>), grid, threads, 0, s, cache, n_blocks, n_kv_heads, shift, slots,         \
                     (uint32_t)n_tokens, k, v, error)
  if (flags & SBM_F_IN_BF16) {
    if (head_dim == 64) SBM_LOAD(__bf16, 64);
    else if (head_dim == 128) SBM_LOAD(__bf16, 128);
    else SBM_LOAD(__bf16, 256);
  } else {
    if (head_dim == 64) SBM_LOAD(_Float16, 64);
    else if (head_dim == 128) SBM_LOAD(_Float16, 128);
    else SBM_LOAD(_Float16, 256);
  }
#undef SBM_LOAD
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "kv_load launch: %s", hipGetErrorString(e));
  return SBM_OK;
}

}  // extern "C"
