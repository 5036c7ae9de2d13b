// Layer norm, forward and backward, with the reduction of the weight's gradient.
#include "laplex_layers.hpp"
#include "laplex_layers_device.hpp"

namespace laplex {

constexpr int kNormBlock = 256;
constexpr uint32_t kNormParts = 512;  // row groups of the weight gradient's partial sums

__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = wave_sum(v);
  __syncthreads();
  if (lane_id() == 0) sh[threadIdx.x / kWave] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < kNormBlock / kWave; ++i) t += sh[i];
  return t;
}

// One row per block, read three times (the row stays in the caches).
template <typename T>
__global__ __launch_bounds__(kNormBlock) void k_norm(uint64_t rows, uint32_t width, const T* __restrict__ x, const T* __restrict__ w,
                                                     const T* __restrict__ b, float eps, T* __restrict__ y,
                                                     float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float sh[kNormBlock / kWave];
  for (uint64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * width;
    float s = 0.f;
    for (uint32_t i = threadIdx.x; i < width; i += kNormBlock) s += to_f32(xr[i]);
    const float m = block_sum(s, sh) / (float)width;
    float v = 0.f;
    for (uint32_t i = threadIdx.x; i < width; i += kNormBlock) {
      const float d = to_f32(xr[i]) - m;
      v = fmaf(d, d, v);
    }
    const float rs = 1.f / sqrtf(block_sum(v, sh) / (float)width + eps);
    for (uint32_t i = threadIdx.x; i < width; i += kNormBlock) {
      const float z = (to_f32(xr[i]) - m) * rs;
      y[row * width + i] = from_f32<T>(fmaf(z, w ? to_f32(w[i]) : 1.f, b ? to_f32(b[i]) : 0.f));
    }
    if (threadIdx.x == 0) {
      if (mean) mean[row] = m;
      if (rstd) rstd[row] = rs;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kNormBlock) void k_norm_dx(uint64_t rows, uint32_t width, const T* __restrict__ x,
                                                        const T* __restrict__ dy, const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, const T* __restrict__ w,
                                                        T* __restrict__ dx) {
  __shared__ float sh[kNormBlock / kWave];
  for (uint64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * width, *gr = dy + row * width;
    const float m = mean[row], rs = rstd[row];
    float a = 0.f, c = 0.f;
    for (uint32_t i = threadIdx.x; i < width; i += kNormBlock) {
      const float u = to_f32(gr[i]) * (w ? to_f32(w[i]) : 1.f);
      a += u;
      c = fmaf(u, (to_f32(xr[i]) - m) * rs, c);
    }
    a = block_sum(a, sh) / (float)width;
    c = block_sum(c, sh) / (float)width;
    for (uint32_t i = threadIdx.x; i < width; i += kNormBlock) {
      const float u = to_f32(gr[i]) * (w ? to_f32(w[i]) : 1.f), z = (to_f32(xr[i]) - m) * rs;
      dx[row * width + i] = from_f32<T>(rs * (u - a - z * c));
    }
  }
}

// Column sums of one group of rows; thread per column.
template <typename T>
__global__ __launch_bounds__(kNormBlock) void k_norm_dw(uint64_t rows, uint32_t width, const T* __restrict__ x,
                                                        const T* __restrict__ dy, const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, float* __restrict__ part) {
  const uint32_t i = blockIdx.x * kNormBlock + threadIdx.x;
  if (i >= width) return;
  float dw = 0.f, db = 0.f;
  for (uint64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float g = to_f32(dy[row * width + i]);
    dw = fmaf(g, (to_f32(x[row * width + i]) - mean[row]) * rstd[row], dw);
    db += g;
  }
  part[((uint64_t)blockIdx.y * 2) * width + i] = dw;
  part[((uint64_t)blockIdx.y * 2 + 1) * width + i] = db;
}

__global__ __launch_bounds__(kNormBlock) void k_norm_dw_sum(const float* __restrict__ part, uint32_t parts, uint32_t width,
                                                            float* __restrict__ dw, float* __restrict__ db) {
  const uint32_t i = blockIdx.x * kNormBlock + threadIdx.x;
  if (i >= width) return;
  float a = 0.f, b = 0.f;
  for (uint32_t p = 0; p < parts; ++p) {
    a += part[(uint64_t)(2 * p) * width + i];
    b += part[(uint64_t)(2 * p + 1) * width + i];
  }
  if (dw) dw[i] = a;
  if (db) db[i] = b;
}

static uint32_t norm_parts(uint64_t rows) { return (uint32_t)std::min<uint64_t>((rows + 15) / 16, kNormParts); }

size_t layer_norm_backward_bytes(uint64_t rows, uint32_t width) { return (size_t)norm_parts(rows) * 2 * width * 4 + 256; }

hipError_t layer_norm(int dtype, uint64_t rows, uint32_t width, const void* x, const void* w, const void* b, float eps, void* y,
                      float* mean, float* rstd, hipStream_t s) {
  const unsigned blocks = (unsigned)std::min<uint64_t>(rows, 1u << 20);
  LAPLEX_LAUNCH("k_norm", rows, s, {
    if (dtype == LAPLEX_BF16)
      k_norm<bf16><<<blocks, kNormBlock, 0, s>>>(rows, width, (const bf16*)x, (const bf16*)w, (const bf16*)b, eps, (bf16*)y, mean, rstd);
    else
      k_norm<float><<<blocks, kNormBlock, 0, s>>>(rows, width, (const float*)x, (const float*)w, (const float*)b, eps, (float*)y, mean,
                                                  rstd);
  });
  return hipGetLastError();
}

hipError_t layer_norm_backward(int dtype, uint64_t rows, uint32_t width, const void* x, const void* dy, const float* mean,
                               const float* rstd, const void* w, void* dx, float* dw, float* db, void* ws, hipStream_t s) {
  const unsigned blocks = (unsigned)std::min<uint64_t>(rows, 1u << 20);
  const uint32_t parts = norm_parts(rows);
  float* part = static_cast<float*>(ws);
  const unsigned cols = (width + kNormBlock - 1) / kNormBlock;
  if (rows) {
    LAPLEX_LAUNCH("k_norm_dx", rows, s, {
      if (dtype == LAPLEX_BF16)
        k_norm_dx<bf16><<<blocks, kNormBlock, 0, s>>>(rows, width, (const bf16*)x, (const bf16*)dy, mean, rstd, (const bf16*)w, (bf16*)dx);
      else
        k_norm_dx<float><<<blocks, kNormBlock, 0, s>>>(rows, width, (const float*)x, (const float*)dy, mean, rstd, (const float*)w,
                                                       (float*)dx);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!dw && !db) return hipSuccess;
    LAPLEX_LAUNCH("k_norm_dw", rows, s, {
      const dim3 grid(cols, parts);
      if (dtype == LAPLEX_BF16)
        k_norm_dw<bf16><<<grid, kNormBlock, 0, s>>>(rows, width, (const bf16*)x, (const bf16*)dy, mean, rstd, part);
      else
        k_norm_dw<float><<<grid, kNormBlock, 0, s>>>(rows, width, (const float*)x, (const float*)dy, mean, rstd, part);
    });
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (dw || db)
    LAPLEX_LAUNCH("k_norm_dw_sum", width, s, k_norm_dw_sum<<<cols, kNormBlock, 0, s>>>(part, parts, width, dw, db));
  return hipGetLastError();
}

}  // namespace laplex
