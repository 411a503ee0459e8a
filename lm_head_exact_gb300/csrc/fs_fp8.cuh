// Device helpers of the 8-bit path: 16-, 32- and 8-bit elements in groups, and
// the scale of a block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "flashsample.h"

namespace fs {

template <typename T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// The largest finite value of an 8-bit type.
__host__ __device__ constexpr float fp8_largest(int type) { return type == FS_TYPE_E5M2 ? 57344.0f : 448.0f; }

// Scale of a block whose largest magnitude is amax, and its reciprocal.  Both
// are rounded once, so that every implementation of the formula finds the same
// 8-bit values.  The least scale keeps the reciprocal finite; a block below
// 2^-100 loses what lies under 2^-110.  An infinity makes its block's scale
// infinite and all of its values NaN; NaNs are not counted into amax and stay
// NaN where they are.
struct BlockScale {
  float scale, inverse;
};

__device__ __forceinline__ BlockScale block_scale(float amax, float largest) {
  BlockScale s;
  s.scale = fmaxf(__fdiv_rn(amax, largest), 0x1p-100f);
  s.inverse = __frcp_rn(s.scale);
  return s;
}

// Two values times the reciprocal, to nearest even, the first in the low byte.
template <int kType>
__device__ __forceinline__ uint16_t fp8_pair(float a, float b, float inverse) {
  return __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(a, inverse), __fmul_rn(b, inverse)), __NV_SATFINITE,
                                  kType == FS_TYPE_E5M2 ? __NV_E5M2 : __NV_E4M3);
}

template <int kType>
__device__ __forceinline__ uint32_t fp8_quad(float a, float b, float c, float d, float inverse) {
  return fp8_pair<kType>(a, b, inverse) | static_cast<uint32_t>(fp8_pair<kType>(c, d, inverse)) << 16;
}

template <int kType>
__device__ __forceinline__ uint8_t fp8_one(float a, float inverse) {
  return static_cast<uint8_t>(fp8_pair<kType>(a, 0.0f, inverse));
}

// Elements of one 16-byte access.
template <typename T> constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// kVec<T> elements at p, 16-byte aligned, as floats.
template <typename T>
__device__ __forceinline__ void unpack(uint4 raw, float (&v)[kVec<T>]) {
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j) v[j] = to_float<T>(e[j]);
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[kVec<T>]) {
  uint4 raw;
  T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j) e[j] = from_float<T>(v[j]);
  return raw;
}

}  // namespace fs
