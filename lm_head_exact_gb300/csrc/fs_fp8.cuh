// Device helpers of the 8-bit path: 16-, 32- and 8-bit elements in groups, and
// the scale of a block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "flashsample.h"
#include "fs_device.cuh"

namespace fs {

// Waits for what lies ahead in the stream, then lets the next kernel start: one
// that reads weights before its own wait must not begin while a kernel ahead of
// this one may still write them.  For kernels whose own results no such reader
// takes: 8-bit matrices, samples.  One that writes a caller's matrix of 16- or
// 32-bit elements waits only: it lets the next kernel start by its end, for
// whatever follows may, before its wait, let one start that reads the matrix
// as an LM head before its own.
__device__ __forceinline__ void pdl_wait_then_launch() {
  pdl_wait();
  pdl_launch_dependents();
}

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

// Eight elements of a row as they lie in memory.
template <typename T>
struct Eight {
  uint4 raw[8 / kVec<T>];

  __device__ __forceinline__ T at(int j) const { return reinterpret_cast<const T*>(raw)[j]; }
  __device__ __forceinline__ float value(int j) const { return to_float<T>(at(j)); }
};

// Largest magnitudes of eights; NaNs do not count.  16-bit types are compared two
// at a time.
__device__ __forceinline__ uint32_t abs2(uint32_t v) { return v & 0x7fff7fffu; }
template <typename T> __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t max2<__nv_bfloat16>(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
template <> __device__ __forceinline__ uint32_t max2<__half>(uint32_t a, uint32_t b) {
  const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Magnitudes by column, and their joins: eight columns.
template <typename T>
struct Tops {
  uint32_t two[4];
  __device__ __forceinline__ void clear() { two[0] = two[1] = two[2] = two[3] = 0u; }
  __device__ __forceinline__ void add(const Eight<T>& e) {
    two[0] = max2<T>(two[0], abs2(e.raw[0].x));
    two[1] = max2<T>(two[1], abs2(e.raw[0].y));
    two[2] = max2<T>(two[2], abs2(e.raw[0].z));
    two[3] = max2<T>(two[3], abs2(e.raw[0].w));
  }
  __device__ __forceinline__ void join(int lanes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) two[i] = max2<T>(two[i], __shfl_xor_sync(0xffffffffu, two[i], lanes));
  }
  __device__ __forceinline__ float column(int j) const { return to_float<T>(reinterpret_cast<const T*>(two)[j]); }
  __device__ __forceinline__ float all() const {
    const uint32_t m = max2<T>(max2<T>(two[0], two[1]), max2<T>(two[2], two[3]));
    return fmaxf(to_float<T>(reinterpret_cast<const T*>(&m)[0]), to_float<T>(reinterpret_cast<const T*>(&m)[1]));
  }
};
template <>
struct Tops<float> {
  float one[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) one[i] = 0.0f;
  }
  __device__ __forceinline__ void add(const Eight<float>& e) {
#pragma unroll
    for (int i = 0; i < 8; ++i) one[i] = fmaxf(one[i], fabsf(e.value(i)));
  }
  __device__ __forceinline__ void join(int lanes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) one[i] = fmaxf(one[i], __shfl_xor_sync(0xffffffffu, one[i], lanes));
  }
  __device__ __forceinline__ float column(int j) const { return one[j]; }
  __device__ __forceinline__ float all() const {
    float m = one[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, one[i]);
    return m;
  }
};

// The largest of value[i] over the 16 lanes of a half warp for each of kN values
// (a power of two up to 16), and its scale: lane l ends with that of value
// l / (16 / kN) of its half.  Each step sends the half of the values that the other
// lane keeps: for 8 values 8 shuffles and one division instead of 32 and 8.
template <int kN>
__device__ __forceinline__ BlockScale spread_scale(float (&value)[kN], int lane, float largest) {
  int n = kN;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        if (i >= n) break;
        const float mine = up ? value[i + n] : value[i], other = up ? value[i] : value[i + n];
        value[i] = fmaxf(mine, __shfl_xor_sync(0xffffffffu, other, o));
      }
    } else {
      value[0] = fmaxf(value[0], __shfl_xor_sync(0xffffffffu, value[0], o));
    }
  }
  return block_scale(value[0], largest);
}
template <int kN>
__device__ __forceinline__ float spread_get(float v, int i, int lane) {
  return __shfl_sync(0xffffffffu, v, (lane & 16) + i * (16 / kN));
}

}  // namespace fs
