// AdamW over many tensors in one launch, with states in float32 or in 8 bits.
//
//   g' = s g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// A block takes 2048 elements of a tensor at a time and reads and writes
// everything once.  With float moments a thread has two pieces of four
// consecutive elements, so that a wave's floats are whole 1024-byte stretches;
// with 8-bit ones eight consecutive elements.
//
// 8-bit states: a block of 256 values (32 threads) shares a float scale, its
// largest magnitude / 448; m and sqrt(v) are e4m3 codes of the values over it.
// Rounding is stochastic if asked for: 16 random bits below the kept mantissa are
// added and the rest cut off, so that a state's expectation is the value itself --
// rounded to nearest (half a step is added, so that ties go away from zero), a
// second moment that changes by a thousandth a step would never leave its code.  sqrt(v) > 0 never becomes 0, or a step would be divided by eps.
// The new parameters are made from the moments before they are rounded.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "laplex_layers_device.hpp"
#include "laplex_train.hpp"

namespace laplex {

constexpr int kAdamBlock = 256, kAdamChunk = 2048;
constexpr int kAdamGroup = 40;  // tensors of a launch: its arguments stay below 4 KB
// Tensors of more bytes than the Infinity Cache keeps from one step to the next are moved past the caches (float moments
// and parameters, 268 MB: 81 us, through them 73; 335 MB: 101, 128; 4.3 GB: 1307, 1605).
constexpr uint64_t kAdamCached = 288ull << 20;
constexpr uint64_t kAdamBlocks = (1u << 24) - 1;  // (a launch has fewer than 2^32 threads)

struct AdamTensor {
  void* p;
  const void* g;
  void *m, *v;
  float *m_scale, *v_scale, *master;
  uint64_t n;
  float keep;        // 1 - lr wd
  float wd;          // (with lr from the device)
  uint32_t chunk0;   // chunks of the launch's tensors before this one
  uint32_t number;   // in the caller's list
};
struct AdamArgs {
  AdamTensor t[kAdamGroup];
  uint32_t count, chunks;
  float b1, one_b1, b2, one_b2, eps, rate, inv_c2;  // (inv_c2: of the square root of 1 - beta2^step)
  bool divide;  // eps is so small that its reciprocal may be infinite
  uint32_t seed;
  int32_t stochastic;
  uint64_t step;
  double lr, beta1, beta2;
  const int32_t* step_dev;
  const float *lr_dev, *grad_scale;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

// MurmurHash3's 32-bit finalizer (public domain)
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}

// 4, 8 or 16 bytes at the alignment of T; NT: past the caches
template <typename T, int BYTES>
using Words = uint32_t __attribute__((ext_vector_type(BYTES / 4), aligned(sizeof(T))));
template <bool NT, int BYTES, typename T>
__device__ __forceinline__ void load_bytes(const T* p, void* to) {
  constexpr int W = BYTES < 16 ? BYTES : 16;
  using V = Words<T, W>;
#pragma unroll
  for (int i = 0; i < BYTES / W; ++i) {
    const V* q = reinterpret_cast<const V*>(reinterpret_cast<const char*>(p) + i * W);
    const V v = NT ? __builtin_nontemporal_load(q) : *q;
    __builtin_memcpy(static_cast<char*>(to) + i * W, &v, W);
  }
}
template <bool NT, int BYTES, typename T>
__device__ __forceinline__ void store_bytes(T* p, const void* from) {
  constexpr int W = BYTES < 16 ? BYTES : 16;
  using V = Words<T, W>;
#pragma unroll
  for (int i = 0; i < BYTES / W; ++i) {
    V v, *q = reinterpret_cast<V*>(reinterpret_cast<char*>(p) + i * W);
    __builtin_memcpy(&v, static_cast<const char*>(from) + i * W, W);
    if (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
  }
}
// N consecutive elements, of which `left` are the tensor's
template <bool NT, int N, typename T>
__device__ __forceinline__ void load_some(const T* p, int64_t left, float (&v)[N]) {
  T e[N];
  if (left >= N) {
    load_bytes<NT, sizeof e>(p, e);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = i < left ? p[i] : T(0.f);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_f32(e[i]);
}
template <bool NT, int N, typename T>
__device__ __forceinline__ void store_some(T* p, int64_t left, const float (&v)[N]) {
  T e[N];
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = from_f32<T>(v[i]);
  if (left >= N) {
    store_bytes<NT, sizeof e>(p, e);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) p[i] = e[i];
  }
}

// ------------------------------------------------------------------ e4m3 codes
template <bool NT, int N>
__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t left, float scale, float (&v)[N]) {
  uint32_t w[N / 4] = {};
  if (left >= N) {
    load_bytes<NT, N>(p, w);
  } else {
    for (int i = 0; i < (int)left; ++i) w[i / 4] |= (uint32_t)p[i] << i % 4 * 8;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
    v[4 * i] = a[0] * scale;
    v[4 * i + 1] = a[1] * scale;
    v[4 * i + 2] = b[0] * scale;
    v[4 * i + 3] = b[1] * scale;
  }
}
template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t left, const uint32_t (&c)[8]) {
  if (left >= 8) {
    const uint32_t w[2] = {c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24};
    store_bytes<NT, 8>(p, w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint8_t)c[i];
  }
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.402823466e38f; }
// the largest of the 32 threads' magnitudes (NaN is passed over); finite_only: of those that are finite
__device__ __forceinline__ float block_most(const float (&v)[8], bool finite_only) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_only && !finite(v[i]) ? 0.f : fabsf(v[i]));
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  return m;
}
// Magnitudes below 2^-100 are kept as zeros (the reciprocal of their scale would be infinite).
__device__ __forceinline__ float inverse_scale(float most) { return most >= 0x1p-100f ? 448.f / most : 0.f; }
// e4m3 magnitude of |x| / scale; r: 16 random bits (0x8000: to nearest).  Subnormals, multiples of 2^-9, are those
// of the binade from 2^-6 on, moved there by an addition.
__device__ __forceinline__ uint32_t code_of(float x, float inverse, uint32_t r) {
  const float y = fminf(fabsf(x) * inverse, 448.f);
  const bool small = y < 0x1p-6f;
  return ((__float_as_uint(small ? y + 0x1p-6f : y) + (r << 4)) >> 20) - (small ? 968u : 960u);
}

// ------------------------------------------------------------------ the step
template <typename P, typename G, int BITS, bool NT>
__global__ __launch_bounds__(kAdamBlock) void k_adamw(AdamArgs a) {
  __shared__ float sh[2];
  constexpr int N = BITS == 8 ? 8 : 4, PIECES = 8 / N;
  const float scale = a.grad_scale ? *a.grad_scale : 1.f;
  if (!finite(scale)) return;  // the step is skipped
  float rate = a.rate, inv_c2 = a.inv_c2;
  uint64_t step = a.step;
  double lr = a.lr;
  if (a.step_dev || a.lr_dev) {
    if (a.step_dev) step = (uint64_t)max(*a.step_dev, 1);
    if (a.lr_dev) lr = (double)*a.lr_dev;
    if (threadIdx.x == 0) {
      sh[0] = (float)(lr / (1.0 - pow(a.beta1, (double)step)));
      sh[1] = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)step)));
    }
    __syncthreads();
    rate = sh[0];
    inv_c2 = sh[1];
  }
  uint32_t k = 0;  // the tensor of the chunk before
  for (uint32_t chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    while (k + 1 < a.count && a.t[k + 1].chunk0 <= chunk) ++k;
    const AdamTensor& t = a.t[k];
    const float keep = a.lr_dev ? (float)(1.0 - lr * (double)t.wd) : t.keep;
    float p[PIECES][N] = {}, g[PIECES][N] = {}, m[PIECES][N] = {}, v[PIECES][N] = {};
    const uint64_t at0 = (uint64_t)(chunk - t.chunk0) * kAdamChunk + threadIdx.x * N;
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const uint64_t at = at0 + q * (kAdamBlock * N);
      const int64_t left = (int64_t)t.n - (int64_t)at;
      if (left <= 0) continue;
      if (t.master) load_some<NT>(t.master + at, left, p[q]);
      else load_some<NT>(static_cast<const P*>(t.p) + at, left, p[q]);
      load_some<NT>(static_cast<const G*>(t.g) + at, left, g[q]);
      if constexpr (BITS == 32) {
        load_some<NT>(static_cast<const float*>(t.m) + at, left, m[q]);
        load_some<NT>(static_cast<const float*>(t.v) + at, left, v[q]);
      } else {
        load_codes<NT>(static_cast<const uint8_t*>(t.m) + at, left, t.m_scale[at / 256], m[q]);
        load_codes<NT>(static_cast<const uint8_t*>(t.v) + at, left, t.v_scale[at / 256], v[q]);
#pragma unroll
        for (int i = 0; i < N; ++i) v[q][i] *= v[q][i];
      }
    }
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const uint64_t at = at0 + q * (kAdamBlock * N);
      const int64_t left = (int64_t)t.n - (int64_t)at;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float gi = a.grad_scale ? g[q][i] * scale : g[q][i];
        m[q][i] = a.b1 * m[q][i] + a.one_b1 * gi;
        v[q][i] = a.b2 * v[q][i] + a.one_b2 * (gi * gi);
        const float root = sqrtf(v[q][i]), d = fmaf(root, inv_c2, a.eps), up = rate * m[q][i];
        // (a reciprocal's last bit is nothing beside lr)
        p[q][i] = p[q][i] * keep - (a.divide ? up / d : up * __builtin_amdgcn_rcpf(d));
        if constexpr (BITS == 8) v[q][i] = root;
      }
      if (left > 0) {
        store_some<NT>(static_cast<P*>(t.p) + at, left, p[q]);
        if (t.master) store_some<NT>(t.master + at, left, p[q]);
        if constexpr (BITS == 32) {
          store_some<NT>(static_cast<float*>(t.m) + at, left, m[q]);
          store_some<NT>(static_cast<float*>(t.v) + at, left, v[q]);
        }
      }
    }
    if constexpr (BITS == 8) {
      const uint64_t at = at0;
      const int64_t left = (int64_t)t.n - (int64_t)at;
      if (left < N) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i >= left) m[0][i] = v[0][i] = 0.f;
      }
      float mm = block_most(m[0], false), vm = block_most(v[0], false);
      // (a NaN, which has no part in a maximum, shows in sums; a square that is too large only costs the second look)
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) all = fmaf(m[0][i], m[0][i], all + v[0][i]);
      const bool bad = __any(!finite(all) || !finite(mm));
      if (bad) {
        mm = block_most(m[0], true);
        vm = block_most(v[0], true);
      }
      const float mi = inverse_scale(mm), vi = inverse_scale(vm);
      const uint32_t key = mix32(mix32(t.number * 0x9E3779B9u + (uint32_t)step) ^ a.seed) ^ (uint32_t)(at >> 32) * 0x85EBCA6Bu;
      uint32_t cm[N], cv[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t r = a.stochastic ? mix32((uint32_t)(at + i) ^ key) : 0x80008000u;
        cm[i] = code_of(m[0][i], mi, r & 0xFFFFu) | (m[0][i] < 0.f ? 128u : 0u);
        cv[i] = code_of(v[0][i], vi, r >> 16);
        if (v[0][i] > 0.f && cv[i] == 0) cv[i] = 1;
        if (bad) {
          if (!finite(m[0][i])) cm[i] = 0x7F;  // NaN
          if (!finite(v[0][i])) cv[i] = 0x7F;
        }
      }
      if (left > 0) {
        store_codes<NT>(static_cast<uint8_t*>(t.m) + at, left, cm);
        store_codes<NT>(static_cast<uint8_t*>(t.v) + at, left, cv);
        if (threadIdx.x % 32 == 0) {
          t.m_scale[at / 256] = mm / 448.f;
          t.v_scale[at / 256] = vm / 448.f;
        }
      }
    }
  }
}

// Launches `run` for groups of tensors, in at most so many blocks; each holds chunks of its own.
template <typename F>
static hipError_t by_groups(AdamArgs& a, const laplex_adamw_tensor* t, uint32_t count, double lr, uint64_t most, F run) {
  for (uint32_t i = 0; i < count;) {
    a.count = 0;
    uint64_t chunks = 0;
    for (; i < count && a.count < kAdamGroup; ++i) {
      if (t[i].n == 0) continue;
      const uint64_t more = (t[i].n + kAdamChunk - 1) / kAdamChunk;
      if (a.count && chunks + more > 0x7FFFFFFFu) break;
      a.t[a.count++] = {t[i].p, t[i].g, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale, t[i].master, t[i].n,
                        (float)(1.0 - lr * (double)t[i].weight_decay), t[i].weight_decay, (uint32_t)chunks, i};
      chunks += more;
    }
    if (a.count == 0) continue;
    a.chunks = (uint32_t)chunks;
    run((unsigned)std::min<uint64_t>(chunks, most));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t adamw(const laplex_adamw_args& o, const laplex_adamw_tensor* t, uint32_t count, hipStream_t s) {
  AdamArgs a{};
  a.b1 = (float)o.beta1;
  a.one_b1 = (float)(1.0 - o.beta1);
  a.b2 = (float)o.beta2;
  a.one_b2 = (float)(1.0 - o.beta2);
  a.eps = (float)o.eps;
  a.rate = (float)(o.lr / (1.0 - std::pow(o.beta1, (double)o.step)));
  a.inv_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(o.beta2, (double)o.step)));
  a.divide = o.eps < 1e-30;
  a.seed = o.seed;
  a.stochastic = o.stochastic;
  a.step = o.step;
  a.lr = o.lr;
  a.beta1 = o.beta1;
  a.beta2 = o.beta2;
  a.step_dev = o.step_dev;
  a.lr_dev = o.lr_dev;
  a.grad_scale = o.grad_scale;
  const bool pb = o.dtype == LAPLEX_BF16, gb = o.grad_dtype == LAPLEX_BF16;
  uint64_t bytes = 0;
  for (uint32_t i = 0; i < count; ++i) bytes += t[i].n * ((pb ? 2 : 4) + (gb ? 2 : 4) + o.state_bits / 4 + (t[i].master ? 4 : 0));
  // (a block takes one chunk; with the step or rate on the device, several, for each block forms the powers of beta)
  return by_groups(a, t, count, o.lr, o.step_dev || o.lr_dev ? 8192 : kAdamBlocks, [&](unsigned blocks) {
    const auto bits = [&](auto p, auto g, auto nt) {
      using P = decltype(p);
      using G = decltype(g);
      if (o.state_bits == 32) k_adamw<P, G, 32, decltype(nt)::value><<<blocks, kAdamBlock, 0, s>>>(a);
      else k_adamw<P, G, 8, decltype(nt)::value><<<blocks, kAdamBlock, 0, s>>>(a);
    };
    const auto types = [&](auto nt) {
      if (pb) gb ? bits(bf16{}, bf16{}, nt) : bits(bf16{}, float{}, nt);
      else gb ? bits(float{}, bf16{}, nt) : bits(float{}, float{}, nt);
    };
    LAPLEX_LAUNCH("k_adamw", a.chunks, s, bytes > kAdamCached ? types(std::true_type{}) : types(std::false_type{}));
  });
}

// ------------------------------------------------------------------ 8-bit moments as floats
// (p and master hold the outputs)
template <bool NT>
__global__ __launch_bounds__(kAdamBlock) void k_adamw_moments(AdamArgs a) {
  constexpr int N = 4;
  uint32_t k = 0;
  for (uint32_t chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    while (k + 1 < a.count && a.t[k + 1].chunk0 <= chunk) ++k;
    const AdamTensor& t = a.t[k];
    const uint64_t at0 = (uint64_t)(chunk - t.chunk0) * kAdamChunk + threadIdx.x * N;
    const auto move = [&](const void* codes, const float* scales, float* out, bool square) {
      float v[2][N];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint64_t at = at0 + q * kAdamBlock * N;
        if (at < t.n) load_codes<NT>(static_cast<const uint8_t*>(codes) + at, (int64_t)(t.n - at), scales[at / 256], v[q]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint64_t at = at0 + q * kAdamBlock * N;
        if (square)
#pragma unroll
          for (int i = 0; i < N; ++i) v[q][i] *= v[q][i];
        if (at < t.n) store_some<NT>(out + at, (int64_t)(t.n - at), v[q]);
      }
    };
    if (t.p) move(t.m, t.m_scale, static_cast<float*>(t.p), false);
    if (t.master) move(t.v, t.v_scale, t.master, true);
  }
}

hipError_t adamw_moments(const laplex_adamw_tensor* t, uint32_t count, hipStream_t s) {
  AdamArgs a{};
  uint64_t bytes = 0;
  for (uint32_t i = 0; i < count; ++i) bytes += t[i].n * 10;
  return by_groups(a, t, count, 0.0, kAdamBlocks, [&](unsigned blocks) {
    LAPLEX_LAUNCH("k_adamw_moments", a.chunks, s,
                  bytes > kAdamCached ? k_adamw_moments<true><<<blocks, kAdamBlock, 0, s>>>(a) : k_adamw_moments<false><<<blocks, kAdamBlock, 0, s>>>(a));
  });
}

}  // namespace laplex
