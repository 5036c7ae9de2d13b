// Device helpers of the sequence-layer kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "laplex_device.hpp"

namespace laplex {

using bf16 = __bf16;

template <typename T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v) { return (T)v; }  // round to nearest even

// sum over the 64 lanes, the same value in every lane
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// A rate as the kernels use it: +Inf becomes the largest float, so that a lag
// of zero weighs exp(0) = 1 and any other 0.  NaN stays.
__device__ __forceinline__ float attn_rate(float r) { return r > 3.402823466e38f ? 3.402823466e38f : r; }

}  // namespace laplex
