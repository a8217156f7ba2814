// Attention over the 4-bit paged cache.
//
// A wave takes 16 rows (query heads of one key head, and their tokens) as the
// columns of the matrix products, and walks the cached tokens 32 at a time,
// everything in registers:
//   S^T [32 tokens x 16 rows] = K Q^T   two v_mfma_f32_16x16x32 per 32 dimensions
//   P^T = exp2(S^T - m)                 the running maximum m of a row (= lane & 15)
//   O^T [D x 16] += V^T P^T             one v_mfma_f32_16x16x32 per 16 dimensions
// A lane of S^T holds, for its row, tokens 4g .. 4g + 3 of both halves (g = lane
// / 16): that is already the operand of the second product if its inner index
// is numbered the same way, so P never leaves its lanes.  V is read in the same
// numbering: eight tokens' codes of the same D / 16 dimensions, converted two
// dimensions at a time (v_cvt_scalef32_pk_*_fp4) and paired by token (v_perm_b32).
// K's dimensions are numbered so that a lane's codes are contiguous.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sbm_kv4.h"

namespace sbm {
namespace {

constexpr int kAThreads = 256;
constexpr int kAWaves = kAThreads / 64;
// P is held as exp2(z - m) with m = (the row's maximum when m was last raised)
// - kBias, and m is raised when a score passes that maximum by kSlack: P stays
// below 2^15, which fp16 holds, and a score has to be 32 below the maximum (in
// powers of two) before fp16 drops it.
constexpr float kBias = 8.f, kSlack = 7.f;
constexpr float kLowest = -3.0e38f;       // m before the first score
constexpr float kLn2 = 0.693147180559945309f;
constexpr uint32_t kErrBlock = 1, kErrLength = 2, kErrCuQ = 4;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct AttnArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  uint16_t* out;
  float* lse;
  uint32_t* error;
  float scale2;          // scale * log2(e)
  int32_t n_blocks, shift, width, n_requests, n_tokens, heads, kv_heads, group;
};

template <typename T>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (__is_same(T, __bf16)) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  } else {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef T v2 __attribute__((ext_vector_type(2)));
  const v2 v = {(T)a, (T)b};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float exponent(uint32_t s) { return __uint_as_float(s << 23); }

// What a wave has read of 32 cached tokens.
template <int D>
struct Raw {
  uint32_t k[2][D / 32];       // a lane's D / 4 K codes of token (lane & 15), both halves
  uint32_t ks[2];              // their scale bytes (one, or two with D = 256)
  uint32_t v[2][4][D > 128 ? 2 : 1];   // D / 16 V codes of tokens 4g + i
  uint32_t vs[2][4];           // the scale byte of each (in the low byte)
  bool ok[2];                  // the block exists (the same in all lanes)
};

// Where the 32 tokens from t0 are (t0 a multiple of 32); `end`: the tokens that there are.
template <int D>
__device__ __forceinline__ void load_tokens(Raw<D>& r, const AttnArgs& a, const int32_t* table, int kh, int t0,
                                            int end, int lane) {
  const int m = lane & 15, g = lane >> 4;
  const int bs = 1 << a.shift;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = t0 + 16 * x;
    int32_t b = t < end ? table[t >> a.shift] : 0;
    b = __builtin_amdgcn_readfirstlane(b);
    r.ok[x] = (uint32_t)b < (uint32_t)a.n_blocks;
    if (!r.ok[x]) b = 0;
    const int row = t & (bs - 1);                  // t past the end stays inside block 0's rows
    const uint8_t* rec = a.cache + ((int64_t)b * a.kv_heads + kh) * kv_record_bytes(bs, D);
    const uint8_t* kc = rec + (row + m) * (D / 2) + g * (D / 8);
    if constexpr (D == 64) {
      const uint2 w = *(const uint2*)kc;
      r.k[x][0] = w.x, r.k[x][1] = w.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 w = *(const uint4*)(kc + 16 * i);
        r.k[x][4 * i] = w.x, r.k[x][4 * i + 1] = w.y, r.k[x][4 * i + 2] = w.z, r.k[x][4 * i + 3] = w.w;
      }
    }
    const uint8_t* ks = rec + bs * D + (row + m) * (D / 32);
    if constexpr (D == 64) r.ks[x] = ks[g >> 1];
    else if constexpr (D == 128) r.ks[x] = ks[g];
    else r.ks[x] = *(const uint16_t*)(ks + 2 * g);
    const uint8_t* vc = rec + bs * (D / 2) + (row + 4 * g) * (D / 2) + m * (D / 32);
    const uint8_t* vs = rec + bs * D + bs * (D / 32) + (row + 4 * g) * (D / 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (D == 64) {
        r.v[x][i][0] = *(const uint16_t*)(vc + i * (D / 2));
      } else if constexpr (D == 128) {
        r.v[x][i][0] = *(const uint32_t*)(vc + i * (D / 2));
      } else {
        const uint2 w = *(const uint2*)(vc + i * (D / 2));
        r.v[x][i][0] = w.x, r.v[x][i][1] = w.y;
      }
      r.vs[x][i] = vs[i * (D / 32) + m * (D / 16) / 32];
    }
  }
}

// 16 kNQ rows of one key head: queries, running maxima, sums and outputs.
template <typename T, int D, int kNQ>
struct Rows {
  static constexpr int E = D / 16;
  u32x4 q[kNQ][D / 32];
  f32x4 o[kNQ][E];
  float m[kNQ], l[kNQ];
  int last[kNQ];               // the last position that the lane's row sees, -1: none
};

// NaN for the rows that see a token whose values have one, where that token
// went into the products as if it had none (a masked step, some rows not seeing it).
template <typename T, int D, int kNQ>
__device__ __forceinline__ void nan_values(Rows<T, D, kNQ>& s, const AttnArgs& a, const int32_t* table, int kh, int t0,
                                        int end, int lane) {
  const int bs = 1 << a.shift, g = lane >> 4;
  for (int t = t0; t < min(t0 + 32, end); ++t) {
    const int32_t b = table[t >> a.shift];
    if ((uint32_t)b >= (uint32_t)a.n_blocks) continue;
    const uint8_t* vs = a.cache + ((int64_t)b * a.kv_heads + kh) * kv_record_bytes(bs, D) + bs * D + bs * (D / 32) +
                        (t & (bs - 1)) * (D / 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // rows 4g + i of an output tile are dimensions (4g + i) D / 16 and on
      if (vs[(4 * g + i) * (D / 16) / 32] != kScaleNaN) continue;
#pragma unroll
      for (int c = 0; c < kNQ; ++c) {
        if (t > s.last[c]) continue;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) s.o[c][e][i] = NAN;
      }
    }
  }
}

template <typename T, int D, int kNQ>
__device__ __forceinline__ void step(Rows<T, D, kNQ>& s, Raw<D>& r, const AttnArgs& a, const int32_t* table,
                                     int kh, int t0, int end, int first, int lane) {
  constexpr int E = D / 16;
  const int g = lane >> 4;
  // some token of the 32 is hidden from some row (`first`: the first row's last position)
  const bool masked = t0 + 31 > first || !r.ok[0] || !r.ok[1];
  // K Q^T
  f32x4 sc[kNQ][2];
#pragma unroll
  for (int c = 0; c < kNQ; ++c) sc[c][0] = sc[c][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      const float ks = exponent(D == 256 ? (r.ks[x] >> (kk / 4 * 8)) & 255u : r.ks[x]);
      const uint32_t w = r.k[x][kk];
      const u32x4 k = {cvt_fp4<T, 0>(w, ks), cvt_fp4<T, 1>(w, ks), cvt_fp4<T, 2>(w, ks), cvt_fp4<T, 3>(w, ks)};
#pragma unroll
      for (int c = 0; c < kNQ; ++c) sc[c][x] = mfma<T>(k, s.q[c][kk], sc[c][x]);
    }
  }
  bool odd_v = false;            // a NaN among the values of tokens that not every row sees
  if (masked) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + 16 * x + 4 * g + i;
        const bool there = r.ok[x] && t < end;
        odd_v = odd_v || (there && r.vs[x][i] == kScaleNaN);
        // 0 * NaN is NaN: what is not seen has to be finite
        if (!there || r.vs[x][i] == kScaleNaN) r.vs[x][i] = 127;
      }
    }
  }
  // P^T = exp2(scale2 * S^T - m)
  u32x4 p[kNQ];
#pragma unroll
  for (int c = 0; c < kNQ; ++c) {
    float z[8], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = sc[c][j >> 2][j & 3] * a.scale2;
    if (masked) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = t0 + 16 * (j >> 2) + 4 * g + (j & 3);
        if (t > s.last[c] || !r.ok[j >> 2]) z[j] = -INFINITY;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, z[j]);
    if (__any(top > s.m[c] + (kBias + kSlack))) {
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float m = fmaxf(s.m[c], top - kBias), by = __builtin_amdgcn_exp2f(s.m[c] - m);
      s.m[c] = m;
      s.l[c] *= by;
#pragma unroll
      for (int e = 0; e < E; ++e) s.o[c][e] *= by;
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[j] = __builtin_amdgcn_exp2f(z[j] - s.m[c]);
      sum += z[j];
    }
    s.l[c] += sum;
    // rounded to the values' type: off by half a step of it, as the output is
    p[c] = u32x4{pack2<T>(z[0], z[1]), pack2<T>(z[2], z[3]), pack2<T>(z[4], z[5]), pack2<T>(z[6], z[7])};
  }
  // V^T P^T
  float vs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) vs[j] = exponent(r.vs[j >> 2][j & 3]);
  auto pair = [&](auto byte) {               // dimensions 2 byte and 2 byte + 1 of the lane's E
    constexpr int kB = decltype(byte)::value;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = cvt_fp4<T, kB & 3>(r.v[j >> 2][j & 3][kB >> 2], vs[j]);
    u32x4 lo, hi;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x05040100u);
      hi[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x07060302u);
    }
#pragma unroll
    for (int c = 0; c < kNQ; ++c) {
      s.o[c][2 * kB] = mfma<T>(lo, p[c], s.o[c][2 * kB]);
      s.o[c][2 * kB + 1] = mfma<T>(hi, p[c], s.o[c][2 * kB + 1]);
    }
  };
  pair(std::integral_constant<int, 0>{});
  pair(std::integral_constant<int, 1>{});
  if constexpr (E > 4) {
    pair(std::integral_constant<int, 2>{});
    pair(std::integral_constant<int, 3>{});
  }
  if constexpr (E > 8) {
    pair(std::integral_constant<int, 4>{});
    pair(std::integral_constant<int, 5>{});
    pair(std::integral_constant<int, 6>{});
    pair(std::integral_constant<int, 7>{});
  }
  if (masked && __any(odd_v)) nan_values<T, D, kNQ>(s, a, table, kh, t0, end, lane);
}

template <typename T, int D, int kNQ>
__device__ __forceinline__ void init_rows(Rows<T, D, kNQ>& s, const AttnArgs& a, int kh, int q0, int n, int kv,
                                          int row0, int lane) {
  const int g = lane >> 4;
#pragma unroll
  for (int c = 0; c < kNQ; ++c) {
    const int row = row0 + 16 * c + (lane & 15), i = row / a.group;
    s.last[c] = i < n ? min(kv - n + i, kv - 1) : -1;
    s.m[c] = kLowest;
    s.l[c] = 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) s.o[c][e] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint16_t* q = a.q + (int64_t)(q0 + min(i, n - 1)) * a.q_ts + (int64_t)(kh * a.group + row % a.group) * a.q_hs;
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) s.q[c][kk] = *(const u32x4*)(q + (D / 4) * g + 8 * kk);
  }
}

template <typename T, int D, int kNQ>
__device__ __forceinline__ void write_rows(Rows<T, D, kNQ>& s, const AttnArgs& a, int kh, int q0, int n, int row0,
                                           int lane) {
  constexpr int E = D / 16;
  const int g = lane >> 4;
#pragma unroll
  for (int c = 0; c < kNQ; ++c) {
    float l = s.l[c];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    const int row = row0 + 16 * c + (lane & 15), i = row / a.group;
    if (i >= n) continue;
    const int64_t at = (int64_t)(q0 + i) * a.heads + kh * a.group + row % a.group;
    const float by = l == 0.f ? 0.f : 1.f / l;
    uint16_t* out = a.out + at * D + (D / 4) * g;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) w[e / 2] = pack2<T>(s.o[c][e][j] * by, s.o[c][e + 1][j] * by);
#pragma unroll
      for (int e = 0; e < E / 2; e += 2) *(uint2*)(out + E * j + 2 * e) = make_uint2(w[e], w[e + 1]);
    }
    if (a.lse && g == 0) a.lse[at] = l == 0.f ? -INFINITY : (s.m[c] + __log2f(l)) * kLn2;
  }
}

// One workgroup for each request and key head, its waves taking 16 rows at a time.
template <typename T, int D>
__global__ __launch_bounds__(kAThreads) void attn_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = blockIdx.x, kh = blockIdx.y;
  // tokens of no request
  const int c0 = a.cu_q ? min(max(a.cu_q[0], 0), a.n_tokens) : 0;
  const int c1 = a.cu_q ? min(max(a.cu_q[a.n_requests], 0), a.n_tokens) : a.n_tokens;
  for (int t = r; t < a.n_tokens; t += a.n_requests) {
    if (t >= c0 && t < c1) continue;
    for (int d = threadIdx.x; d < a.group * D; d += kAThreads)
      a.out[((int64_t)t * a.heads + kh * a.group) * D + d] = 0;
    if (a.lse)
      for (int h = threadIdx.x; h < a.group; h += kAThreads) a.lse[(int64_t)t * a.heads + kh * a.group + h] = -INFINITY;
  }
  int q0 = r, n = 1;
  if (a.cu_q) {
    q0 = a.cu_q[r];
    const int q1 = a.cu_q[r + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.n_tokens) {
      if (threadIdx.x == 0 && a.error) atomicOr(a.error, kErrCuQ);
      return;
    }
    n = q1 - q0;
  }
  int kv = a.kv_lens[r];
  if (kv > (int64_t)a.width << a.shift) {
    if (threadIdx.x == 0 && a.error) atomicOr(a.error, kErrLength);
    kv = (int)((int64_t)a.width << a.shift);
  }
  kv = max(kv, 0);
  const int32_t* table = a.table + (int64_t)r * a.width;
  for (int row0 = 16 * wave; row0 < n * a.group; row0 += 16 * kAWaves) {
    Rows<T, D, 1> s;
    init_rows(s, a, kh, q0, n, kv, row0, lane);
    const int first = max(kv - n + row0 / a.group, -1);
    const int end = kv - n + min((row0 + 15) / a.group, n - 1) + 1;
    for (int t0 = 0; t0 < end; t0 += 32) {
      Raw<D> raw;
      load_tokens<D>(raw, a, table, kh, t0, end, lane);
      if ((!raw.ok[0] || !raw.ok[1]) && lane == 0 && a.error) atomicOr(a.error, kErrBlock);
      step(s, raw, a, table, kh, t0, end, first, lane);
    }
    write_rows(s, a, kh, q0, n, row0, lane);
  }
}

template <typename T>
void launch_attn(const AttnArgs& a, int32_t head_dim, hipStream_t s) {
  const dim3 grid((unsigned)a.n_requests, (unsigned)a.kv_heads), threads(kAThreads);
  if (head_dim == 64) hipLaunchKernelGGL((attn_kernel<T, 64>), grid, threads, 0, s, a);
  else if (head_dim == 128) hipLaunchKernelGGL((attn_kernel<T, 128>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((attn_kernel<T, 256>), grid, threads, 0, s, a);
}

}  // namespace
}  // namespace sbm

using namespace sbm;

extern "C" {

size_t sbm_attention_kv4_workspace_bytes(int32_t n_requests, int32_t n_tokens, int32_t n_heads, int32_t n_kv_heads,
                                         int32_t head_dim) {
  if (n_requests < 0 || n_tokens < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads ||
      !kv_shape_ok(16, head_dim))
    return 0;
  return 16;
}

int sbm_attention_kv4(const sbm_heads* q, const uint8_t* cache, int32_t n_blocks, int32_t block_size,
                      const int32_t* block_table, int32_t table_width, const int32_t* kv_lens, const int32_t* cu_q,
                      int32_t n_requests, int32_t n_tokens, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                      float scale, uint16_t* out, float* lse, uint32_t flags, void* workspace,
                      size_t workspace_bytes, uint32_t* error, void* stream) {
  if (flags & ~SBM_F_IN_BF16) return fail(SBM_EINVAL, "unknown flags 0x%x", flags);
  if (n_requests < 0 || n_requests > kMaxRequests)
    return fail(SBM_EINVAL, "n_requests=%d outside 0..%d", n_requests, kMaxRequests);
  if (n_tokens < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads > 65535 || n_heads % n_kv_heads)
    return fail(SBM_EINVAL, "bad n_tokens=%d, n_heads=%d or n_kv_heads=%d", n_tokens, n_heads, n_kv_heads);
  if (n_blocks <= 0 || table_width < 0 || !kv_shape_ok(block_size, head_dim))
    return fail(SBM_EINVAL, "bad cache: n_blocks=%d, block_size=%d, head_dim=%d, table_width=%d", n_blocks, block_size,
                head_dim, table_width);
  if ((int64_t)table_width * block_size > 0x7FFFFF00)
    return fail(SBM_ERANGE, "%d blocks of %d tokens in one request", table_width, block_size);
  if ((int64_t)n_tokens * (n_heads / n_kv_heads) > 0x7FFFFF00) return fail(SBM_ERANGE, "too many rows");
  if (!cu_q && n_tokens != n_requests)
    return fail(SBM_EINVAL, "without cu_q each request has one token: n_tokens=%d, n_requests=%d", n_tokens, n_requests);
  if (n_tokens == 0) return SBM_OK;
  if (n_requests == 0) return fail(SBM_EINVAL, "%d tokens without a request", n_tokens);
  if (!q || !q->data || !cache || !kv_lens || (table_width && !block_table) || !out || !workspace)
    return fail(SBM_EINVAL, "null pointer");
  if (((uintptr_t)q->data | (uintptr_t)cache | (uintptr_t)out | (uintptr_t)workspace) & 15u)
    return fail(SBM_EINVAL, "q, cache, out and workspace must be 16-byte aligned");
  if (q->token_stride % 8 || q->head_stride % 8) return fail(SBM_EINVAL, "q's strides must be multiples of 8 elements");
  const size_t need = sbm_attention_kv4_workspace_bytes(n_requests, n_tokens, n_heads, n_kv_heads, head_dim);
  if (workspace_bytes < need) return fail(SBM_ENOSPACE, "workspace %zu < %zu bytes", workspace_bytes, need);
  AttnArgs a{(const uint16_t*)q->data, q->token_stride, q->head_stride, cache, block_table, kv_lens, cu_q, out, lse,
             error, scale * 1.44269504088896341f, n_blocks, __builtin_ctz((unsigned)block_size), table_width,
             n_requests, n_tokens, n_heads, n_kv_heads, n_heads / n_kv_heads};
  if (flags & SBM_F_IN_BF16) launch_attn<__bf16>(a, head_dim, (hipStream_t)stream);
  else launch_attn<_Float16>(a, head_dim, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SBM_EHIP, "attention launch: %s", hipGetErrorString(e));
  return SBM_OK;
}

}  // extern "C"
