// The 4-bit cache's layout and what its kernels share (include/sbm.h has the
// format).  One head of one block is a record of block_size * D * 17 / 16
// bytes: K codes, V codes, K scales, V scales, each block_size rows.
#pragma once

#include <hip/hip_runtime.h>

#include "sbm_internal.h"

namespace sbm {

constexpr int kMaxRequests = 4096;        // lengths of a call that a workgroup scans into its LDS
constexpr uint32_t kScaleNaN = 255;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

inline bool kv_shape_ok(int32_t block_size, int32_t head_dim) {
  return block_size >= 16 && block_size <= 4096 && (block_size & (block_size - 1)) == 0 &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256);
}

__host__ __device__ constexpr int64_t kv_record_bytes(int32_t block_size, int32_t head_dim) {
  return (int64_t)block_size * head_dim / 16 * 17;
}

// Two codes of a byte (byte `kSel` of src) times the power of two in scale's
// exponent; exponent 255 gives NaN, 0 gives 2^-127: E8M0 as it stands.
template <typename T, int kSel>
__device__ __forceinline__ uint32_t cvt_fp4(uint32_t src, float scale) {
  if constexpr (sizeof(T) == 2 && __is_same(T, __bf16)) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(src, scale, kSel));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(src, scale, kSel));
  }
}

}  // namespace sbm
