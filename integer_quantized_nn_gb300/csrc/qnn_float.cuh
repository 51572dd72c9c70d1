// qnn_float.cuh -- the float types of the weight-only product and the block norm:
// their sizes, and conversions to and from fp32.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "qnn.h"

namespace qnn {

inline bool is_float_dt(int dt) { return dt == QNN_F32 || dt == QNN_F16 || dt == QNN_BF16; }
__host__ __device__ inline int float_bytes(int dt) { return dt == QNN_F32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// round to nearest even, the one rounding of a result
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace qnn
