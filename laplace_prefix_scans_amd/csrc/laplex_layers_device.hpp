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

// exp(-rate n) as the sum of two floats.  A carry is multiplied by it once per
// segment, or per single token: with one float, the rounding of a weight near 1
// would add up, the same way each time, over the thousands of them that a slow
// decay reaches (rate 1e-4, 6000 single tokens: 8e-5 of the state).
struct AttnDecay {
  float hi, lo;
  __device__ __forceinline__ float of(float s) const { return fmaf(s, hi, s * lo); }
};
__device__ __forceinline__ AttnDecay attn_decay(float rate, int64_t n) {
  const double w = exp(-(double)rate * (double)n);
  return {(float)w, (float)(w - (double)(float)w)};
}

}  // namespace laplex
