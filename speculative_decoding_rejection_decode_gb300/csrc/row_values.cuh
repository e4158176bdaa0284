// Eight neighbouring values of a 16-bit row in 32 bits, and the axes of rotary pairs:
// what the kernels that turn rows share (cache.cu, rotary.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"

namespace specdec {

struct Vec8 {
  float x[8];
};

__device__ __forceinline__ float2 unpack(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
__device__ __forceinline__ uint32_t pack(float a, float b, __nv_bfloat16) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack(float a, float b, __half) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ Vec8 widen(uint4 w) {
  Vec8 v;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack(u[i], T());
    v.x[2 * i] = f.x;
    v.x[2 * i + 1] = f.y;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ uint4 narrow(const Vec8& v) {
  return make_uint4(pack(v.x[0], v.x[1], T()), pack(v.x[2], v.x[3], T()),
                    pack(v.x[4], v.x[5], T()), pack(v.x[6], v.x[7], T()));
}

// Axis of a rotary pair (at most kMaxPairs).
__device__ __forceinline__ int axis_of(const RotaryAxes& a, int pair) {
  return (int)(a.word[pair >> 4] >> ((pair & 15) * 2)) & 3;
}

}  // namespace specdec
