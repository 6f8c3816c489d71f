// Host: tensor maps of the rows of 16-bit tensors, shared by the tile kernels.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "kv_internal.h"

namespace vdx {

// A [n3][n2][n1] grid of rows of D channels (element strides s1, s2, s3) as a map with boxes of
// b1 x b2 rows of `channels` channels (64: 128-byte swizzle, 32: 64-byte).
template <typename T>
inline bool encode_rows(EncodeTiledFn encode, CUtensorMap* map, const void* base, int D, long long n1, long long s1, long long n2,
                 long long s2, long long n3, long long s3, int channels, int b1, int b2) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2),
                              static_cast<cuuint64_t>(n3)};
  auto bytes = [&](long long n, long long s) { return static_cast<cuuint64_t>(n > 1 ? s : D) * 2; };   // unused where n = 1
  const cuuint64_t strides[3] = {bytes(n1, s1), bytes(n2, s2), bytes(n3, s3)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(channels), static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(map, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                channels == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace vdx
