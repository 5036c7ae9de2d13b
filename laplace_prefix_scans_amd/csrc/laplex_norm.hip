// Layer norm, forward and backward, with the reduction of the weight's gradient.
//
//   y = (x - mean) rstd w + b;   with z = (x - mean) rstd, u = dy w:
//   dx = rstd (u - mean(u) - z mean(u z)),   dw = sum_rows dy z,   db = sum_rows dy.
//
// Both passes move each tensor once and are bound by HBM: a row lives in the
// registers of the threads that share it (a wave up to 2048 bfloat16 elements,
// then 256 or 1024 threads), so its mean, the centred second moment and the
// result need one read.  Statistics and all sums are float32.  The backward
// keeps each column's dw and db in the same registers over all the rows a
// block takes and writes one partial per block; a second launch adds the
// partials.  16384 rows of 4096 bfloat16: forward 49 us, 5.4 TB/s; backward 84 us,
// 4.8 TB/s, and 5 us for the partials.  Rows longer than 32768 bfloat16 (16384 float) elements are
// read again instead of held.
// The backward holds less than it should of long rows: a thread of 1024 has 128 registers, and above 8192 bfloat16 or
// float elements 76 to 325 of its values spill to scratch.  TB/s, forward and backward, of tensors of 67 to 268 MB: bfloat16
// 1024 columns 5.3, 5.4; 2048 4.6, 4.8; 8192 5.1, 4.1; 12288 3.8, 1.4; 32768 3.2, 0.7 (read again: 1.3, 1.0); float 1024 to
// 8192 5.6 to 5.8, 4.8 to 5.3; 12288 and 16384 5.8, 2.2 and 2.4 (read again: 2.0, 2.0).
#include "laplex_layers.hpp"
#include "laplex_layers_device.hpp"

namespace laplex {

constexpr int kNormBlock = 256;
constexpr uint32_t kNormBlocks = 2048;  // 256-thread blocks of a forward pass (eight a CU), each taking rows in turn
constexpr uint32_t kNormParts = 512;  // at most so many partials of the weight gradient (two 256-thread blocks a CU; the
                                      // shapes of 1025 to 2048 and 4097 to 8192 bfloat16 elements have registers for one or two)

// ------------------------------------------------------------------ rows in registers
// VEC: every row begins at a multiple of 16 bytes and has whole 16-byte pieces.  Without, the pieces are the same
// ones, read and written at the alignment of T but for the row's last: columns keep their threads, so that a row's
// sums, and with them its results, are the same bits whatever its alignment.
template <typename T, int TPR, int VPT, bool VEC>
struct NormRow {
  static constexpr int E = 16 / sizeof(T), N = VPT * E;
  static constexpr int THREADS = TPR < 256 ? 256 : TPR, ROWS = THREADS / TPR;
  T e[N];
  // column of element k of thread t of the row
  static __device__ __forceinline__ uint32_t col(int k, int t) {
    return (uint32_t)((k / E * TPR + t) * E + k % E);
  }
  __device__ __forceinline__ void load(const T* p, uint32_t width, int t) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (col(i * E, t) < width) q = *reinterpret_cast<const uint4*>(p + col(i * E, t));
        __builtin_memcpy(e + i * E, &q, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const uint32_t c = col(i * E, t);
        if (c + E <= width) {
          __builtin_memcpy(e + i * E, p + c, 16);
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j) e[i * E + j] = c + j < width ? p[c + j] : T(0.f);
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* p, uint32_t width, int t) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        uint4 q;
        __builtin_memcpy(&q, e + i * E, 16);
        if (col(i * E, t) < width) *reinterpret_cast<uint4*>(p + col(i * E, t)) = q;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const uint32_t c = col(i * E, t);
        if (c + E <= width) {
          __builtin_memcpy(p + c, e + i * E, 16);
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (c + j < width) p[c + j] = e[i * E + j];
        }
      }
    }
  }
};

// sum over the TPR threads of a row; sh: one float2 per wave, two buffers used in turn
template <int TPR>
__device__ __forceinline__ float2 row_sum(float a, float b, float2 (*sh)[16], int& turn) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (TPR > kWave) {
    constexpr int W = TPR / kWave;
    if (lane_id() == 0) sh[turn][threadIdx.x / kWave] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a += sh[turn][i].x;
      b += sh[turn][i].y;
    }
    turn ^= 1;  // the other buffer's readers are past the barrier before the one after next writes it
  }
  return make_float2(a, b);
}

template <typename T, int TPR, int VPT, bool VEC>
__global__ __launch_bounds__((TPR < 256 ? 256 : TPR)) void k_norm(uint64_t rows, uint32_t width, const T* __restrict__ x,
                                                                 const T* __restrict__ w, const T* __restrict__ b, float eps,
                                                                 T* __restrict__ y, float* __restrict__ mean,
                                                                 float* __restrict__ rstd) {
  using Row = NormRow<T, TPR, VPT, VEC>;
  __shared__ float2 sh[2][16];
  int turn = 0;
  const int t = threadIdx.x % TPR;
  Row r, rw, rb;
  if (w) rw.load(w, width, t);
  if (b) rb.load(b, width, t);
  // uniform over the threads of a row, and over the block where a row takes all of it
  const uint64_t stride = (uint64_t)gridDim.x * Row::ROWS;
  uint64_t row = (uint64_t)blockIdx.x * Row::ROWS + threadIdx.x / TPR;
  Row next;  // on its way while this row is reduced
  if (row < rows) next.load(x + row * width, width, t);
  for (; row < rows; row += stride) {
    r = next;
    if (row + stride < rows) next.load(x + (row + stride) * width, width, t);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < Row::N; ++k) s += to_f32(r.e[k]);
    const float m = row_sum<TPR>(s, 0.f, sh, turn).x / (float)width;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < Row::N; ++k) {
      const float d = Row::col(k, t) < width ? to_f32(r.e[k]) - m : 0.f;
      v = fmaf(d, d, v);
    }
    const float rs = 1.f / sqrtf(row_sum<TPR>(v, 0.f, sh, turn).x / (float)width + eps);
#pragma unroll
    for (int k = 0; k < Row::N; ++k) {
      const float z = (to_f32(r.e[k]) - m) * rs;
      r.e[k] = from_f32<T>(fmaf(z, w ? to_f32(rw.e[k]) : 1.f, b ? to_f32(rb.e[k]) : 0.f));
    }
    r.store(y + row * width, width, t);
    if (t == 0) {
      if (mean) mean[row] = m;
      if (rstd) rstd[row] = rs;
    }
  }
}

// part: per block, width sums of dy z and then width sums of dy; null where no weight gradient is asked for
template <typename T, int TPR, int VPT, bool VEC>
__global__ __launch_bounds__((TPR < 256 ? 256 : TPR)) void k_norm_back(uint64_t rows, uint32_t width, const T* __restrict__ x,
                                                                      const T* __restrict__ dy, const float* __restrict__ mean,
                                                                      const float* __restrict__ rstd, const T* __restrict__ w,
                                                                      T* __restrict__ dx, float* __restrict__ part) {
  using Row = NormRow<T, TPR, VPT, VEC>;
  constexpr int N = Row::N;
  __shared__ float2 sh[2][16];
  __shared__ float comb[Row::ROWS > 1 ? 2 * TPR * N : 1];
  int turn = 0;
  const int t = threadIdx.x % TPR, wr = threadIdx.x / TPR;
  const uint64_t stride = (uint64_t)gridDim.x * Row::ROWS;
  uint64_t row = (uint64_t)blockIdx.x * Row::ROWS + wr;
  Row rw;
  if (w) rw.load(w, width, t);
  float dw[N], db[N];
#pragma unroll
  for (int k = 0; k < N; ++k) dw[k] = db[k] = 0.f;
  Row nx, ng;  // the next row, on its way while this one is reduced
  float nm = 0.f, nr = 0.f;
  auto fetch = [&](uint64_t at) {
    nx.load(x + at * width, width, t);
    ng.load(dy + at * width, width, t);
    nm = mean[at];
    nr = rstd[at];
  };
  if (row < rows) fetch(row);
  for (; row < rows; row += stride) {  // uniform over the threads of a row, and over the block where rows share barriers
    Row rx = nx, rg = ng;
    const float m = nm, rs = nr;
    if (row + stride < rows) fetch(row + stride);
    float a = 0.f, c = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float g = to_f32(rg.e[k]), u = g * (w ? to_f32(rw.e[k]) : 1.f);
      const float z = Row::col(k, t) < width ? (to_f32(rx.e[k]) - m) * rs : 0.f;
      a += u;
      c = fmaf(u, z, c);
      dw[k] = fmaf(g, z, dw[k]);
      db[k] += g;
    }
    const float2 s = row_sum<TPR>(a, c, sh, turn);
    a = s.x / (float)width;
    c = s.y / (float)width;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float u = to_f32(rg.e[k]) * (w ? to_f32(rw.e[k]) : 1.f), z = (to_f32(rx.e[k]) - m) * rs;
      rx.e[k] = from_f32<T>(rs * (u - a - z * c));
    }
    rx.store(dx + row * width, width, t);
  }
  if (!part) return;
  if constexpr (Row::ROWS > 1) {  // the block's rows one after the other into one sum
    for (int r = 0; r < Row::ROWS; ++r) {
      if (wr == r) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          float* at = comb + 2 * (k * TPR + t);
          at[0] = r ? at[0] + dw[k] : dw[k];
          at[1] = r ? at[1] + db[k] : db[k];
        }
      }
      __syncthreads();
    }
    if (wr != 0) return;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      dw[k] = comb[2 * (k * TPR + t)];
      db[k] = comb[2 * (k * TPR + t) + 1];
    }
  }
  float* out = part + (uint64_t)blockIdx.x * 2 * width;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t c = Row::col(k, t);
    if (c < width) {
      out[c] = dw[k];
      out[width + c] = db[k];
    }
  }
}

// dw and db from their partials: 64 columns (of the 2 x width) by 16 groups of partials per block
__global__ __launch_bounds__(1024) void k_norm_dw_sum(const float* __restrict__ part, uint32_t parts, uint32_t width,
                                                      float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sh[16][64];
  const uint64_t c = (uint64_t)blockIdx.x * 64 + threadIdx.x % 64;
  const uint32_t g = threadIdx.x / 64;
  float a = 0.f;
  if (c < 2ull * width) {
#pragma unroll 8
    for (uint32_t p = g; p < parts; p += 16) a += part[(uint64_t)p * 2 * width + c];
  }
  sh[g][threadIdx.x % 64] = a;
  __syncthreads();
  if (g || c >= 2ull * width) return;
  a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a += sh[i][threadIdx.x];
  if (c < width) {
    if (dw) dw[c] = a;
  } else if (db) {
    db[c - width] = a;
  }
}

// ------------------------------------------------------------------ rows too long for registers
__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = wave_sum(v);
  __syncthreads();
  if (lane_id() == 0) sh[threadIdx.x / kWave] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < kNormBlock / kWave; ++i) t += sh[i];
  return t;
}

template <typename T>
__global__ __launch_bounds__(kNormBlock) void k_norm_long(uint64_t rows, uint32_t width, const T* __restrict__ x,
                                                          const T* __restrict__ w, const T* __restrict__ b, float eps,
                                                          T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
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
__global__ __launch_bounds__(kNormBlock) void k_norm_long_dx(uint64_t rows, uint32_t width, const T* __restrict__ x,
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

// column sums of every gridDim.y-th row
template <typename T>
__global__ __launch_bounds__(kNormBlock) void k_norm_long_dw(uint64_t rows, uint32_t width, const T* __restrict__ x,
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

// ------------------------------------------------------------------ launches
// Calls f.template operator()<TPR, VPT>() with the smallest shape that holds a row; false if none does.
template <typename T, typename F>
static bool norm_shape(uint32_t width, F&& f) {
  constexpr uint32_t E = 16 / sizeof(T);
  const uint32_t v = (width + E - 1) / E;  // 16-byte pieces of a row
  if (v <= 64) f.template operator()<64, 1>();
  else if (v <= 128) f.template operator()<64, 2>();
  else if (v <= 256) f.template operator()<64, 4>();
  else if (v <= 512) f.template operator()<256, 2>();
  else if (v <= 1024) f.template operator()<256, 4>();
  else if (v <= 2048) f.template operator()<1024, 2>();
  else if (v <= 4096) f.template operator()<1024, 4>();
  else return false;
  return true;
}
static uint64_t norm_rows_per_block(uint32_t width, size_t e) { return (uint64_t)width * e <= 256 * 16 ? 4 : 1; }
static uint32_t norm_parts(uint64_t rows) { return (uint32_t)std::min<uint64_t>(rows, kNormParts); }

size_t layer_norm_backward_bytes(uint64_t rows, uint32_t width) { return (size_t)norm_parts(rows) * 2 * width * 4 + 256; }

static bool norm_vec(uint32_t width, size_t e, std::initializer_list<const void*> ps) {
  if (width * e % 16) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

template <typename T>
struct NormForward {
  uint64_t rows;
  uint32_t width;
  const T *x, *w, *b;
  float eps;
  T* y;
  float *mean, *rstd;
  bool vec;
  hipStream_t s;
  template <int TPR, int VPT>
  void operator()() const {
    constexpr int TH = TPR < 256 ? 256 : TPR, R = TH / TPR;
    const unsigned blocks = (unsigned)std::min<uint64_t>((rows + R - 1) / R, kNormBlocks * 256 / TH);
    if (vec) k_norm<T, TPR, VPT, true><<<blocks, TH, 0, s>>>(rows, width, x, w, b, eps, y, mean, rstd);
    else k_norm<T, TPR, VPT, false><<<blocks, TH, 0, s>>>(rows, width, x, w, b, eps, y, mean, rstd);
  }
};
template <typename T>
struct NormBackward {
  uint64_t rows;
  uint32_t width;
  const T *x, *dy;
  const float *mean, *rstd;
  const T* w;
  T* dx;
  float* part;
  unsigned blocks;
  bool vec;
  hipStream_t s;
  template <int TPR, int VPT>
  void operator()() const {
    constexpr int TH = TPR < 256 ? 256 : TPR;
    if (vec) k_norm_back<T, TPR, VPT, true><<<blocks, TH, 0, s>>>(rows, width, x, dy, mean, rstd, w, dx, part);
    else k_norm_back<T, TPR, VPT, false><<<blocks, TH, 0, s>>>(rows, width, x, dy, mean, rstd, w, dx, part);
  }
};

template <typename T>
static void norm_forward(uint64_t rows, uint32_t width, const void* x, const void* w, const void* b, float eps, void* y,
                         float* mean, float* rstd, hipStream_t s) {
  const NormForward<T> f{rows, width, (const T*)x, (const T*)w, (const T*)b, eps, (T*)y, mean, rstd,
                         norm_vec(width, sizeof(T), {x, w, b, y}), s};
  if (!norm_shape<T>(width, f))
    k_norm_long<T><<<(unsigned)std::min<uint64_t>(rows, 1u << 20), kNormBlock, 0, s>>>(rows, width, f.x, f.w, f.b, eps, f.y, mean, rstd);
}

hipError_t layer_norm(int dtype, uint64_t rows, uint32_t width, const void* x, const void* w, const void* b, float eps, void* y,
                      float* mean, float* rstd, hipStream_t s) {
  LAPLEX_LAUNCH("k_norm", rows, s, {
    if (dtype == LAPLEX_BF16) norm_forward<bf16>(rows, width, x, w, b, eps, y, mean, rstd, s);
    else norm_forward<float>(rows, width, x, w, b, eps, y, mean, rstd, s);
  });
  return hipGetLastError();
}

template <typename T>
static uint32_t norm_backward(uint64_t rows, uint32_t width, const void* x, const void* dy, const float* mean, const float* rstd,
                              const void* w, void* dx, float* part, hipStream_t s) {
  const uint64_t per = norm_rows_per_block(width, sizeof(T));
  const unsigned blocks = (unsigned)std::min<uint64_t>((rows + per - 1) / per, kNormParts);
  const NormBackward<T> f{rows, width, (const T*)x, (const T*)dy, mean, rstd, (const T*)w, (T*)dx, part, blocks,
                          norm_vec(width, sizeof(T), {x, dy, w, dx}), s};
  if (norm_shape<T>(width, f)) return blocks;
  k_norm_long_dx<T><<<(unsigned)std::min<uint64_t>(rows, 1u << 20), kNormBlock, 0, s>>>(rows, width, f.x, f.dy, mean, rstd, f.w, f.dx);
  const uint32_t parts = norm_parts(rows);
  if (part) k_norm_long_dw<T><<<dim3((width + kNormBlock - 1) / kNormBlock, parts), kNormBlock, 0, s>>>(rows, width, f.x, f.dy, mean, rstd, part);
  return parts;
}

hipError_t layer_norm_backward(int dtype, uint64_t rows, uint32_t width, const void* x, const void* dy, const float* mean,
                               const float* rstd, const void* w, void* dx, float* dw, float* db, void* ws, hipStream_t s) {
  float* part = dw || db ? static_cast<float*>(ws) : nullptr;
  uint32_t parts = 0;
  if (rows)
    LAPLEX_LAUNCH("k_norm_back", rows, s, {
      parts = dtype == LAPLEX_BF16 ? norm_backward<bf16>(rows, width, x, dy, mean, rstd, w, dx, part, s)
                                   : norm_backward<float>(rows, width, x, dy, mean, rstd, w, dx, part, s);
    });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (dw || db)
    LAPLEX_LAUNCH("k_norm_dw_sum", width, s,
                  k_norm_dw_sum<<<(unsigned)((2ull * width + 63) / 64), 1024, 0, s>>>(part, parts, width, dw, db));
  return hipGetLastError();
}

}  // namespace laplex
