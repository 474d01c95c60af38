// What the tensor-core attention kernels share: the arithmetic of a row's softmax and the tensor maps of packed rows.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ts_tc.cuh"

namespace ts {

__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  uint64_t s = pack_f2(a, b), t = pack_f2(x, y), r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(s), "l"(t));
  unpack_f2(r, a, b);
}

__device__ __forceinline__ float pr_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Base-2 maxima that fp32 holds to no better than 1 (or not at all: infinities): the rounding of the maximum is then
// a factor of 2 or more in the weights, and of nothing but zeros and infinities from 2^31 on. The weights of such
// rows are taken from the scores less the unscaled maximum, which is exact for the scores that matter.
__device__ __forceinline__ bool far(float m2) { return !(fabsf(m2) <= 16777216.f); }

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  return encode;
}

// bf16 [rows][heads][d] with `stride` elements between rows, boxes of 64 elements x bh heads x bt rows.
inline bool rows_map(CUtensorMap* map, const void* p, int64_t rows, int heads, int d, int64_t stride, int bh, int bt) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)bt};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ts
