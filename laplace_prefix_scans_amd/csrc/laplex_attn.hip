// Decayed linear attention: the recurrence S_u = w S_{u-1} + y_u z_u^T,
// out_u = x_u S_u of a matrix-valued carry.
#include "laplex_layers.hpp"
#include "laplex_layers_device.hpp"

namespace laplex {

// Tokens [first, last) of a packed sequence, clamped into the buffer whatever the offsets hold.
__device__ __forceinline__ void seq_range(const int32_t* offsets, uint64_t tokens, uint32_t seqs, uint32_t s, int64_t& first,
                                          int64_t& last) {
  if (!offsets) {
    const int64_t len = (int64_t)(tokens / seqs);
    first = s * len;
    last = first + len;
    return;
  }
  const int64_t t = (int64_t)tokens;
  first = min(max((int64_t)offsets[s], (int64_t)0), t);
  last = min(max((int64_t)offsets[s + 1], first), t);
}

constexpr int kCols = 64;  // columns of the carry per block
constexpr int kRows = 4;   // threads per column
constexpr int kMaxK = 256;

// Token by token: thread (c, r) holds rows r, r + 4, .. of column c of the carry.
template <typename T, bool RATE>
__global__ __launch_bounds__(kCols * kRows) void k_attn_scan(AttnPass p) {
  __shared__ float xs[kMaxK], ys[kMaxK], red[2][kRows][kCols];
  const int c = threadIdx.x % kCols, r = threadIdx.x / kCols;
  const uint32_t h = blockIdx.y, col = blockIdx.z * kCols + c;
  const bool live = col < p.V;
  const int K = (int)p.K;
  auto put = [&](int64_t t, float v) {
    const uint64_t at = ((uint64_t)t * p.heads + h) * p.V + col;
    if (p.out_f32)
      static_cast<float*>(p.out)[at] = v;
    else
      static_cast<T*>(p.out)[at] = from_f32<T>(v);
  };
  int64_t first, last;
  if (blockIdx.x >= p.seqs) {  // tokens outside every sequence
    const int64_t lo = min(max((int64_t)p.offsets[0], (int64_t)0), (int64_t)p.tokens);
    int64_t f, hi;
    seq_range(p.offsets, p.tokens, p.seqs, p.seqs - 1, f, hi);
    if (live && r == 0 && p.out) {
      for (int64_t t = 0; t < lo; ++t) put(t, 0.f);
      for (int64_t t = hi; t < (int64_t)p.tokens; ++t) put(t, 0.f);
    }
    return;
  }
  seq_range(p.offsets, p.tokens, p.seqs, blockIdx.x, first, last);
  const float rate = attn_rate(p.rate[h]), w1 = decay(-rate);
  const uint64_t sbase = ((uint64_t)blockIdx.x * p.heads + h) * (uint64_t)p.K * p.V;
  auto sat = [&](int row) { return sbase + (p.s_trans ? (uint64_t)col * p.K + row : (uint64_t)row * p.V + col); };
  float s[kMaxK / kRows], d[RATE ? kMaxK / kRows : 1];
#pragma unroll
  for (int i = 0; i < kMaxK / kRows; ++i) {
    const int row = i * kRows + r;
    s[i] = (live && row < K && p.s_in) ? p.s_in[sat(row)] : 0.f;
    if constexpr (RATE) d[i] = 0.f;
  }
  const T *x = static_cast<const T*>(p.x.p) + (int64_t)(h / p.x.div) * p.x.head,
          *y = static_cast<const T*>(p.y.p) + (int64_t)(h / p.y.div) * p.y.head,
          *z = static_cast<const T*>(p.z.p) + (int64_t)(h / p.z.div) * p.z.head;
  double dr = 0.0;
  for (int64_t u = 0; u < last - first; ++u) {
    const int64_t t = p.reverse ? last - 1 - u : first + u;
    __syncthreads();
    for (int i = threadIdx.x; i < K; i += kCols * kRows) {
      xs[i] = to_f32(x[t * p.x.token + i]);
      ys[i] = to_f32(y[t * p.y.token + i]);
    }
    __syncthreads();
    const float zv = live ? to_f32(z[t * p.z.token + col]) : 0.f;
    const float w = (p.reverse && u == 0) ? 1.f : w1;
    float acc = 0.f, accd = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxK / kRows; ++i) {
      const int row = i * kRows + r;
      if (row < K) {
        if constexpr (RATE) {
          d[i] = w * (d[i] + s[i]);
          accd = fmaf(xs[row], d[i], accd);
        }
        s[i] = fmaf(w, s[i], p.c_add * ys[row] * zv);
        acc = fmaf(xs[row], s[i], acc);
      }
    }
    red[0][r][c] = acc;
    red[1][r][c] = accd;
    __syncthreads();
    if (r == 0 && live) {
      // c_in == c_pair / c_add in every pass, so the carry's output factor is c_in
      if (p.out) put(t, p.c_in * (red[0][0][c] + red[0][1][c] + red[0][2][c] + red[0][3][c]));
      if constexpr (RATE) {
        const T* dot = static_cast<const T*>(p.dot) + (int64_t)(h / p.dot_view.div) * p.dot_view.head;
        dr += (double)to_f32(dot[t * p.dot_view.token + col]) *
              (double)(p.c_in * (red[1][0][c] + red[1][1][c] + red[1][2][c] + red[1][3][c]));
      }
    }
  }
  const float wf = (p.reverse && last > first) ? w1 : 1.f;
#pragma unroll
  for (int i = 0; i < kMaxK / kRows; ++i) {
    const int row = i * kRows + r;
    if (live && row < K) {
      if (p.s_out) p.s_out[sat(row)] = wf * s[i];
      if constexpr (RATE)
        if (p.ds_out) dr += (double)d[i] * (double)p.ds_out[sat(row)];
    }
  }
  if constexpr (RATE) {
    __shared__ double all[kCols * kRows];
    all[threadIdx.x] = dr;
    __syncthreads();
    if (threadIdx.x == 0) {
      double sum = 0.0;
      for (int i = 0; i < kCols * kRows; ++i) sum += all[i];
      p.drate_part[((uint64_t)blockIdx.x * gridDim.z + blockIdx.z) * p.heads + h] = (float)-sum;
    }
  }
}

__global__ void k_attn_drate(const float* __restrict__ part, uint64_t parts, uint32_t heads, float* __restrict__ drate) {
  const uint32_t h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= heads) return;
  double s = 0.0;
  for (uint64_t i = 0; i < parts; ++i) s += (double)part[i * heads + h];
  drate[h] = (float)s;
}

size_t attn_pass_bytes(uint32_t, uint32_t, uint32_t, uint32_t, uint64_t) { return 0; }
uint64_t attn_drate_parts(uint32_t seqs, uint32_t, uint32_t, uint32_t V, uint64_t) {
  return (uint64_t)seqs * ((V + kCols - 1) / kCols);
}

hipError_t attn_drate_reduce(const float* part, uint64_t parts, uint32_t heads, float* drate, hipStream_t s) {
  LAPLEX_LAUNCH("k_attn_drate", heads, s, k_attn_drate<<<(heads + 63) / 64, 64, 0, s>>>(part, parts, heads, drate));
  return hipGetLastError();
}

hipError_t attn_pass(const AttnPass& p, void*, hipStream_t s) {
  const dim3 grid(p.seqs + (p.offsets ? 1 : 0), p.heads, (p.V + kCols - 1) / kCols);
  LAPLEX_LAUNCH("k_attn_scan", p.tokens, s, {
    if (p.dtype == LAPLEX_BF16)
      p.drate_part ? k_attn_scan<bf16, true><<<grid, kCols * kRows, 0, s>>>(p)
                   : k_attn_scan<bf16, false><<<grid, kCols * kRows, 0, s>>>(p);
    else
      p.drate_part ? k_attn_scan<float, true><<<grid, kCols * kRows, 0, s>>>(p)
                   : k_attn_scan<float, false><<<grid, kCols * kRows, 0, s>>>(p);
  });
  return hipGetLastError();
}

template <typename T>
__global__ void k_attn_group_sum(const float* __restrict__ src, uint64_t count, uint32_t group, uint32_t width, T* __restrict__ dst) {
  const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
  for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < count; i += stride) {
    const uint64_t row = i / width;
    const float* q = src + row * group * width + i % width;
    float a = 0.f;
    for (uint32_t g = 0; g < group; ++g) a += q[(uint64_t)g * width];
    dst[i] = from_f32<T>(a);
  }
}

hipError_t attn_group_sum(int dtype, const float* src, uint64_t tokens, uint32_t kv_heads, uint32_t group, uint32_t width,
                          void* dst, hipStream_t s) {
  const uint64_t count = tokens * kv_heads * width;
  const unsigned blocks = (unsigned)std::min<uint64_t>((count + 255) / 256, 16384);
  LAPLEX_LAUNCH("k_attn_group_sum", count, s, {
    if (dtype == LAPLEX_BF16)
      k_attn_group_sum<bf16><<<blocks, 256, 0, s>>>(src, count, group, width, static_cast<bf16*>(dst));
    else
      k_attn_group_sum<float><<<blocks, 256, 0, s>>>(src, count, group, width, static_cast<float*>(dst));
  });
  return hipGetLastError();
}

// ------------------------------------------------------------------ one token
template <typename T>
__global__ __launch_bounds__(256) void k_attn_step(AttnStep p) {
  __shared__ float part[4][64];
  const uint32_t row = blockIdx.x, h = blockIdx.y;
  const int c = threadIdx.x % 64, r = threadIdx.x / 64;
  const uint32_t col = blockIdx.z * 64 + c;
  const bool live = col < p.V;
  const int64_t slot = p.slots ? (int64_t)p.slots[row] : (int64_t)row;
  const uint64_t at = ((uint64_t)row * p.heads + h) * p.V + col;
  T* out = static_cast<T*>(p.out);
  if (slot < 0 || slot >= (int64_t)p.pool) {
    if (live && r == 0) out[at] = from_f32<T>(0.f);
    return;
  }
  const float w = decay(-attn_rate(p.rate[h]));
  const T *q = static_cast<const T*>(p.q.p) + row * p.q.token + (int64_t)(h / p.q.div) * p.q.head,
          *k = static_cast<const T*>(p.k.p) + row * p.k.token + (int64_t)(h / p.k.div) * p.k.head,
          *v = static_cast<const T*>(p.v.p) + row * p.v.token + (int64_t)(h / p.v.div) * p.v.head;
  float* st = p.state + ((uint64_t)slot * p.heads + h) * (uint64_t)p.K * p.V + col;
  float acc = 0.f;
  if (live) {
    const float vv = to_f32(v[col]);
    for (uint32_t i = r; i < p.K; i += 4) {
      const float n = fmaf(w, st[(uint64_t)i * p.V], to_f32(k[i]) * vv);
      st[(uint64_t)i * p.V] = n;
      acc = fmaf(to_f32(q[i]), n, acc);
    }
  }
  part[r][c] = acc;
  __syncthreads();
  if (r == 0 && live) out[at] = from_f32<T>(p.scale * (part[0][c] + part[1][c] + part[2][c] + part[3][c]));
}

hipError_t attn_step(const AttnStep& p, hipStream_t s) {
  const dim3 grid(p.rows, p.heads, (p.V + 63) / 64);
  LAPLEX_LAUNCH("k_attn_step", p.rows, s, {
    if (p.dtype == LAPLEX_BF16)
      k_attn_step<bf16><<<grid, 256, 0, s>>>(p);
    else
      k_attn_step<float><<<grid, 256, 0, s>>>(p);
  });
  return hipGetLastError();
}

}  // namespace laplex
