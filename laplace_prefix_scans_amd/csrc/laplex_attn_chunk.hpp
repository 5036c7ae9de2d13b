// The chunked recurrence pass of decayed attention: one kernel for every pass
// (forward, dq, dk, dv, states alone), instantiated per type in its own
// source file.
#pragma once
#include <type_traits>

#include "laplex_layers.hpp"
#include "laplex_layers_device.hpp"

namespace laplex {

// ------------------------------------------------------------------ segments
// A sequence is cut into segments of seg_len tokens (a multiple of the
// chunk) so that few long sequences still fill the chip.  Slot b of the grid
// is a segment of some sequence: sequence i's segments start at slot
// bound(i) / seg_len + i, which leaves room for each of them whatever the
// lengths, so nothing about the lengths is needed on the host.  With offsets,
// "sequence" 0 and seqs + 1 are the tokens before the first and after the
// last real one; their outputs are zeroed.
struct AttnSegs {
  const int32_t* offsets;
  uint64_t tokens;
  uint32_t seqs;
  int64_t seg_len;
};
// start of (virtual) sequence i, clamped into the buffer whatever the offsets hold
__device__ __forceinline__ int64_t seq_bound(const AttnSegs& g, int64_t i) {
  if (!g.offsets) return i * (int64_t)(g.tokens / g.seqs);
  if (i == 0) return 0;
  if (i >= (int64_t)g.seqs + 2) return (int64_t)g.tokens;
  return min(max((int64_t)g.offsets[i - 1], (int64_t)0), (int64_t)g.tokens);
}
inline uint64_t attn_slots(const AttnSegs& g) {
  if (!g.offsets) {
    const uint64_t len = g.tokens / g.seqs;
    return g.seqs * std::max<uint64_t>(1, (len + g.seg_len - 1) / g.seg_len);
  }
  return g.tokens / g.seg_len + g.seqs + 3;
}
// Boundaries between two segments of one sequence lie at least seg_len tokens
// apart over all sequences, so position / seg_len numbers them uniquely.
inline uint64_t attn_bounds(uint64_t tokens, int64_t seg_len) { return tokens / seg_len + 1; }

struct AttnSeg {
  int64_t first, len;  // the sequence's tokens
  int64_t u0, n;       // the segment's first token in processing order, its length
  uint32_t seq;
  bool outside, valid;
};
// The segment of slot b (the whole wave calls this with the same b).
__device__ __forceinline__ AttnSeg find_seg(const AttnSegs& g, uint64_t b) {
  AttnSeg s;
  int64_t i, seg;
  if (!g.offsets) {
    const int64_t len = (int64_t)(g.tokens / g.seqs), per = max((int64_t)1, (len + g.seg_len - 1) / g.seg_len);
    i = (int64_t)b / per;
    seg = (int64_t)b % per;
    s.first = i * len;
    s.len = len;
    s.outside = false;
    s.seq = (uint32_t)i;
    s.valid = i < (int64_t)g.seqs;
  } else {
    // 64-ary search for the last sequence whose first slot is <= b
    int64_t lo = 0, cnt = (int64_t)g.seqs + 2;
    while (cnt > 1) {
      const int64_t step = (cnt + kWave - 1) / kWave, at = lo + lane_id() * step;
      const bool le = at < lo + cnt && seq_bound(g, at) / g.seg_len + at <= (int64_t)b;
      const int64_t k = (int64_t)__popcll(__ballot(le)) - 1;
      const int64_t skip = max(k, (int64_t)0) * step;
      lo += skip;
      cnt = min(step, cnt - skip);
    }
    i = lo;
    s.first = seq_bound(g, i);
    s.len = max((int64_t)0, seq_bound(g, i + 1) - s.first);
    seg = (int64_t)b - (s.first / g.seg_len + i);
    s.outside = i == 0 || i == (int64_t)g.seqs + 1;
    s.seq = (uint32_t)(i - 1);
    // an empty sequence still has one segment: its final state is its initial one
    s.valid = seg >= 0 && (seg == 0 || seg * g.seg_len < s.len);
  }
  s.u0 = seg * g.seg_len;
  s.n = min(g.seg_len, s.len - s.u0);
  return s;
}

// ------------------------------------------------------------------ tiles in LDS
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// Rows of a tile are 16-byte chunks; chunk c of row r is kept at c ^ swz(r), so
// that both kinds of reads meet 64 different banks: 16 bytes from each of 16
// rows (row operands), and for the transposed operands 64 contiguous bytes
// from each of 4 rows (bf16) or 128 from two rows 4 apart (float).
template <typename T, int P>
__device__ __forceinline__ int swz(int r) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (P == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    else return ((r & 3) << 2) | ((r >> 2) & 3);
  } else {
    return (((r >> 2) & 1) << 3) | (((r >> 3) & 1) << 2) | (r & 3);
  }
}
// element offset of column c (any) of row r
template <typename T, int P>
__device__ __forceinline__ int tile_at(int r, int c) {
  constexpr int E = 16 / sizeof(T);
  return r * P + (((c / E) ^ swz<T, P>(r)) * E) + c % E;
}

// A tile's 16-byte pieces on their way from memory to LDS.
template <typename T, int ROWS, int P, int THREADS>
struct Stage {
  static constexpr int E = 16 / sizeof(T), N = ROWS * P / E / THREADS;
  static_assert(ROWS * P / E % THREADS == 0, "pieces divide evenly");
  uint4 v[N];
  // Rows [0, rows) of the chunk that starts at processing position u (row r is
  // token base + r * step), columns [col0, width); the rest is zero.
  __device__ __forceinline__ void load(const T* p, int64_t stride, int64_t token, int step, int rows, int col0, int width, bool vec) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * THREADS + threadIdx.x, r = at / (P / E), c = col0 + at % (P / E) * E;
      uint4 q = make_uint4(0, 0, 0, 0);
      if (r < rows && c < width) {
        const T* src = p + (token + (int64_t)r * step) * stride + c;
        if (vec) {
          q = *reinterpret_cast<const uint4*>(src);
        } else {
          T e[E];
#pragma unroll
          for (int j = 0; j < E; ++j) e[j] = c + j < width ? src[j] : T(0.f);
          __builtin_memcpy(&q, e, 16);
        }
      }
      v[i] = q;
    }
  }
  __device__ __forceinline__ void store(T* tile) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * THREADS + threadIdx.x, r = at / (P / E), c = at % (P / E);
      *reinterpret_cast<uint4*>(tile + r * P + ((c ^ swz<T, P>(r)) * E)) = v[i];
    }
  }
  // whether any piece holds an infinity or NaN
  __device__ __forceinline__ bool nonfinite() const {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) bad |= (w[j] & 0x7F80u) == 0x7F80u;
        bad |= (w[j] & 0x7F800000u) == 0x7F800000u;
      }
    }
    return bad;
  }
};

// x = hi + lo (+ lo2) in bfloat16 parts, 2^-17 (2^-25) of x left over.
__device__ __forceinline__ void split_pair(float a, float b, bf16x2& hi, f32x2& rest) {
  hi = bf16x2{(__bf16)a, (__bf16)b};
  rest = f32x2{a - (float)hi[0], b - (float)hi[1]};
}

struct AttnChunkArgs {
  AttnPass p;
  AttnSegs g;
  uint32_t slices;   // blocks across the V columns
  uint64_t tiles;    // slots x heads x slices
  float* bound;      // states at segment boundaries ([boundary][head][K][V]), or null
  float* bound_d;    // the lag-weighted ones (rate gradient)
  bool vec_x, vec_y, vec_z, vec_dot, vec_out;  // 16-byte loads and 4-element stores are aligned
  double* drate;     // Rate: partials [slot][slice][head]
};

template <typename T>
constexpr int kAttnC = sizeof(T) == 2 ? 64 : 32;  // tokens per chunk

// Row of the carry that register (r, e) of a 32-row tile holds in lane half h.
// bf16: the order in which 8 consecutive channels of x form one operand.
template <typename T>
__device__ __forceinline__ int carry_row(int r, int e, int h) {
  if constexpr (sizeof(T) == 2) return 16 * (r >> 1) + 8 * h + 4 * (r & 1) + e;
  else return 8 * r + 4 * h + e;
}

// transposed operand: column 16 * (lane / 16 % 2) + lane % 16 (bf16 carry order if PERM) of rows row0 + 4 h + {0..3}
template <int P, bool PERM>
__device__ __forceinline__ s16x4 read_tr(const __bf16* tile, int l, int row0, int col0) {
  const int q = l & 3, row = row0 + 4 * (l >> 5) + ((l >> 2) & 3);
  const int quad = PERM ? ((q & 1) << 1 | (q >> 1)) : q;
  const int c = col0 + 16 * ((l >> 4) & 1) + 4 * quad;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(tile + tile_at<__bf16, P>(row, c)));
}
template <int P, bool PERM>
__device__ __forceinline__ bf16x8 read_tr8(const __bf16* tile, int l, int row0, int col0) {
  struct { s16x4 a, b; } v = {read_tr<P, PERM>(tile, l, row0, col0), read_tr<P, PERM>(tile, l, row0 + 8, col0)};
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(float a, float b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

// A 32 x 32 tile of the carry (KT of them per wave, one under the other): a
// float register per element, column = lane % 32.
template <typename T, int KP, int NW, bool FULL, bool RATE>
__global__ __launch_bounds__(NW * kWave, KP == 256 || RATE ? 1 : 2) void k_attn_chunk(AttnChunkArgs a) {
  constexpr int C = kAttnC<T>, KT = KP / 32, BV = 32 * NW, THREADS = NW * kWave, IT = C / 32;
  constexpr bool BF = sizeof(T) == 2, DOT = FULL && RATE;
  const AttnPass& p = a.p;
  __shared__ __attribute__((aligned(16))) T xs[FULL ? C * KP : 8];
  __shared__ __attribute__((aligned(16))) T ys[C * KP];
  __shared__ __attribute__((aligned(16))) T zs[C * BV];
  __shared__ __attribute__((aligned(16))) T dots[DOT ? C * BV : 8];
  __shared__ __attribute__((aligned(16))) float down[C], downlag[RATE ? C : 4];
  __shared__ float wt[FULL ? 2 * C : 1];
  __shared__ int bad_chunk[2];
  __shared__ double red[NW];

  uint64_t tile;
  if (!xcd_tile(a.tiles, tile)) return;
  const uint32_t slice = (uint32_t)(tile % a.slices), h = (uint32_t)(tile / a.slices % p.heads);
  const uint64_t slot = tile / a.slices / p.heads;
  const AttnSeg sg = find_seg(a.g, slot);
  const int wave = threadIdx.x / kWave, lane = lane_id(), half = lane >> 5, lc = lane & 31;
  const int col = slice * BV + wave * 32 + lc;  // this lane's column of the carry
  const int K = (int)p.K, V = (int)p.V;
  const bool active = (int)slice * BV + wave * 32 < V;  // the wave has columns (all waves move tiles)
  if (DOT && threadIdx.x == 0 && (!sg.valid || sg.outside)) a.drate[(slot * a.slices + slice) * p.heads + h] = 0.0;
  if (!sg.valid) return;
  if (sg.outside) {
    if constexpr (FULL) {
      if (!p.out) return;
      const int cols = min(BV, V - (int)slice * BV);
      for (int64_t i = threadIdx.x; i < sg.n * cols; i += THREADS) {
        const uint64_t at = ((uint64_t)(sg.first + sg.u0 + i / cols) * p.heads + h) * V + slice * BV + i % cols;
        if (p.out_f32) static_cast<float*>(p.out)[at] = 0.f;
        else static_cast<T*>(p.out)[at] = T(0.f);
      }
    }
    return;
  }
  const bool last_seg = sg.u0 + sg.n >= sg.len;
  if (!FULL && last_seg) return;  // nothing reads this segment's state
  const float rate = attn_rate(p.rate[h]);
  const int lead = p.reverse ? 0 : 1;
  const bool keep = !last_seg || p.s_out || (DOT && p.ds_out);  // the carry after the last chunk is needed
  const uint64_t sbase = ((uint64_t)sg.seq * p.heads + h) * (uint64_t)K * V;
  // element (row, column) of a state in the caller's layout
  auto sat = [&](int row, int c) { return sbase + (p.s_trans ? (uint64_t)c * K + row : (uint64_t)row * V + c); };
  const uint64_t per_bound = (uint64_t)K * V;
  auto bound_at = [&](int64_t u) { return ((uint64_t)((sg.first + u) / a.g.seg_len) * p.heads + h) * per_bound; };

  f32x16 S[KT], D[RATE ? KT : 1];
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 32 * t + carry_row<T>(i / 4, i % 4, half);
      float v = 0.f, d = 0.f;
      if (row < K && col < V) {
        if (FULL && sg.u0 > 0) {
          const uint64_t at = bound_at(sg.u0) + (uint64_t)row * V + col;
          v = a.bound[at];
          if constexpr (RATE) d = a.bound_d[at];
        } else if (FULL && p.s_in) {
          v = p.s_in[sat(row, col)];
        }
      }
      S[t][i] = v;
      if constexpr (RATE) D[t][i] = d;
    }

  // weights of a pair inside a chunk by its lag, 0 for the pairs above the diagonal
  if constexpr (FULL)
    for (int i = threadIdx.x; i < 2 * C; i += THREADS) wt[i] = i >= C ? p.c_pair * decay(-rate * (float)(i - C)) : 0.f;
  float up[IT];
  if constexpr (FULL)
#pragma unroll
    for (int t = 0; t < IT; ++t) up[t] = p.c_in * decay(-rate * (float)(32 * t + lc + lead));
  const AttnDecay wc = attn_decay(rate, C);  // the carry's decay over a chunk
  auto set_down = [&](int n) {
    if (threadIdx.x < C) {
      const int j = threadIdx.x, lag = n - 1 - j;
      down[j] = lag >= 0 ? p.c_add * decay(-rate * (float)(lag + 1 - lead)) : 0.f;
      if constexpr (RATE) downlag[j] = lag >= 0 ? (float)lag * down[j] : 0.f;
    }
  };

  const T* x = static_cast<const T*>(p.x.p) + (int64_t)(h / p.x.div) * p.x.head;
  const T* y = static_cast<const T*>(p.y.p) + (int64_t)(h / p.y.div) * p.y.head;
  const T* z = static_cast<const T*>(p.z.p) + (int64_t)(h / p.z.div) * p.z.head;
  const T* dot = DOT ? static_cast<const T*>(p.dot) + (int64_t)(h / p.dot_view.div) * p.dot_view.head : nullptr;
  const int step = p.reverse ? -1 : 1;
  auto token = [&](int64_t u) { return p.reverse ? sg.first + sg.len - 1 - u : sg.first + u; };

  Stage<T, C, KP, THREADS> sx, sy;
  Stage<T, C, BV, THREADS> sz, sd;
  auto load = [&](int64_t u) {
    const int rows = (int)min((int64_t)C, sg.u0 + sg.n - u);
    const int64_t t = token(u);
    if constexpr (FULL) sx.load(x, p.x.token, t, step, rows, 0, K, a.vec_x);
    sy.load(y, p.y.token, t, step, rows, 0, K, a.vec_y);
    sz.load(z, p.z.token, t, step, rows, slice * BV, V, a.vec_z);
    if constexpr (DOT) sd.load(dot, p.dot_view.token, t, step, rows, slice * BV, V, a.vec_dot);
  };
  double dr = 0.0;
  if (threadIdx.x < 2) bad_chunk[threadIdx.x] = 0;
  set_down((int)min((int64_t)C, sg.n));
  if (sg.n > 0) load(sg.u0);
  int parity = 0;
  for (int64_t u = sg.u0; u < sg.u0 + sg.n; u += C, parity ^= 1) {
    const int n = (int)min((int64_t)C, sg.u0 + sg.n - u);
    __syncthreads();  // the previous chunk's reads are done
    if constexpr (FULL) sx.store(xs);
    sy.store(ys);
    sz.store(zs);
    if constexpr (DOT) sd.store(dots);
    if (FULL && sz.nonfinite()) bad_chunk[parity] = 1;
    if (threadIdx.x == 0) bad_chunk[parity ^ 1] = 0;
    if (n < C && u > sg.u0) set_down(n);
    __syncthreads();
    const bool more = u + C < sg.u0 + sg.n;
    if (more) load(u + C);
    // a masked pair weighs 0, but 0 times an infinity is NaN: a chunk with one in z takes care
    const bool bad = FULL && bad_chunk[parity] != 0;
    if (!active) continue;
    // the lane as the compiler sees it changes with every chunk: the many LDS offsets made from it are
    // then formed where they are used (an xor each) instead of each holding a register over the loop
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int half = ln >> 5, lc = ln & 31;

    f32x16 O[FULL ? IT : 1], OD[DOT ? IT : 1], Pd[FULL ? IT : 1], Po;
    if constexpr (FULL) {
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        O[t] = f32x16{};
        Pd[t] = f32x16{};
        if constexpr (RATE) OD[t] = f32x16{};
      }
      Po = f32x16{};
      // P^T = y x^T (rows j, columns i) and out^T = S^T x^T (rows V, columns i): x is the same operand in both
      if constexpr (BF) {
#pragma unroll
        for (int ks = 0; ks < KP / 16; ++ks) {
          __builtin_amdgcn_sched_barrier(0);  // operands are read as they are needed: held ahead they would spill
          bf16x8 xf[IT], yf[IT], sh, sl, dh, dl;
#pragma unroll
          for (int t = 0; t < IT; ++t) {
            xf[t] = *reinterpret_cast<const bf16x8*>(xs + tile_at<T, KP>(32 * t + lc, 16 * ks + 8 * half));
            yf[t] = *reinterpret_cast<const bf16x8*>(ys + tile_at<T, KP>(32 * t + lc, 16 * ks + 8 * half));
          }
#pragma unroll
          for (int t = 0; t < IT; ++t) Pd[t] = mfma(yf[t], xf[t], Pd[t]);
          if constexpr (IT == 2) Po = mfma(yf[0], xf[1], Po);
          // the carry enters as two bfloat16 parts: with one, its rounding would show beside the output's own
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            bf16x2 hi;
            f32x2 rest;
            split_pair(S[ks / 2][8 * (ks % 2) + e], S[ks / 2][8 * (ks % 2) + e + 1], hi, rest);
            sh[e] = hi[0], sh[e + 1] = hi[1];
            sl[e] = (__bf16)rest[0], sl[e + 1] = (__bf16)rest[1];
            if constexpr (RATE) {
              split_pair(D[ks / 2][8 * (ks % 2) + e], D[ks / 2][8 * (ks % 2) + e + 1], hi, rest);
              dh[e] = hi[0], dh[e + 1] = hi[1];
              dl[e] = (__bf16)rest[0], dl[e + 1] = (__bf16)rest[1];
            }
          }
#pragma unroll
          for (int t = 0; t < IT; ++t) {
            O[t] = mfma(sh, xf[t], O[t]);
            O[t] = mfma(sl, xf[t], O[t]);
            if constexpr (RATE) {
              OD[t] = mfma(dh, xf[t], OD[t]);
              OD[t] = mfma(dl, xf[t], OD[t]);
            }
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            __builtin_amdgcn_sched_barrier(0);
            const float4 xf = *reinterpret_cast<const float4*>(xs + tile_at<T, KP>(lc, 32 * t + 8 * r + 4 * half));
            const float4 yf = *reinterpret_cast<const float4*>(ys + tile_at<T, KP>(lc, 32 * t + 8 * r + 4 * half));
            const float xe[4] = {xf.x, xf.y, xf.z, xf.w}, ye[4] = {yf.x, yf.y, yf.z, yf.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              Pd[0] = mfma(ye[e], xe[e], Pd[0]);
              O[0] = mfma(S[t][4 * r + e], xe[e], O[0]);
              if constexpr (RATE) OD[0] = mfma(D[t][4 * r + e], xe[e], OD[0]);
            }
          }
      }
#pragma unroll
      for (int t = 0; t < IT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if constexpr (RATE) OD[t][i] = up[t] * fmaf((float)(32 * t + lc + lead), O[t][i], OD[t][i]);
          O[t][i] *= up[t];
          const float w = wt[C + lc - (8 * (i / 4) + 4 * half + i % 4)];
          Pd[t][i] = w != 0.f ? Pd[t][i] * w : 0.f;  // a masked pair is 0 whatever its product
        }
      if constexpr (IT == 2)
#pragma unroll
        for (int i = 0; i < 16; ++i) Po[i] *= wt[C + 32 + lc - (8 * (i / 4) + 4 * half + i % 4)];
    }

    // the carry over the chunk, with the lag-weighted one ahead of it
    const bool carry = !FULL || more || keep;
    if (carry) {
      AttnDecay w = wc;
      if (n != C) w = attn_decay(rate, n);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if constexpr (RATE) {
            D[t][i] = w.of(fmaf((float)n, S[t][i], D[t][i]));
          }
          S[t][i] = w.of(S[t][i]);
        }
    }
    if constexpr (BF) {
#pragma unroll
      for (int js = 0; js < C / 16; ++js) {
        __builtin_amdgcn_sched_barrier(0);
        const bf16x8 zf = read_tr8<BV, false>(zs, ln, 16 * js, wave * 32);
        if constexpr (FULL) {
          bf16x8 zp = zf, zn;
          if (bad) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool hit = bits_nonfinite(__float_as_uint((float)zf[e]));
              zn[e] = hit ? (__bf16)3.3e38f : (__bf16)0.f;
              if (hit) zp[e] = (__bf16)0.f;
            }
          }
#pragma unroll
          for (int t = 0; t < IT; ++t) {
            if (js >= 2 * (t + 1)) continue;  // pairs above the diagonal
            const f32x16& P = js >= 2 * t ? Pd[t] : Po;
            bf16x8 ph, pl, rh, rl;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const int i = 8 * (js % 2) + e;
              bf16x2 hi;
              f32x2 rest;
              // two parts, as for the carry
              split_pair(P[i], P[i + 1], hi, rest);
              ph[e] = hi[0], ph[e + 1] = hi[1];
              pl[e] = (__bf16)rest[0], pl[e + 1] = (__bf16)rest[1];
              if constexpr (RATE) {
                const int j = 8 * (i / 4) + 4 * half + i % 4 - (js >= 2 * t ? 0 : 32);
                split_pair(P[i] * (float)(lc - j), P[i + 1] * (float)(lc - j - 1), hi, rest);
                rh[e] = hi[0], rh[e + 1] = hi[1];
                rl[e] = (__bf16)rest[0], rl[e + 1] = (__bf16)rest[1];
              }
            }
            O[t] = mfma(zp, ph, O[t]);
            O[t] = mfma(zp, pl, O[t]);
            if constexpr (RATE) {
              OD[t] = mfma(zp, rh, OD[t]);
              OD[t] = mfma(zp, rl, OD[t]);
            }
            if (bad) {  // large finite stand-ins times 0 or 1, often enough to overflow
              bf16x8 one;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int i = 8 * (js % 2) + e, j = 8 * (i / 4) + 4 * half + i % 4;
                one[e] = js < 2 * t || lc >= j ? (__bf16)1.f : (__bf16)0.f;
              }
#pragma unroll
              for (int k = 0; k < 3; ++k) {
                O[t] = mfma(zn, one, O[t]);
                if constexpr (RATE) OD[t] = mfma(zn, one, OD[t]);
              }
            }
          }
        }
        if (carry) {
          // z weighted by its decay to the chunk's end, as three bfloat16 parts: the carry keeps float32's bits
          bf16x8 z0, z1, z2, l0, l1;
          const float4 da = *reinterpret_cast<const float4*>(down + 16 * js + 4 * half),
                       db = *reinterpret_cast<const float4*>(down + 16 * js + 8 + 4 * half);
          const float dw[8] = {da.x, da.y, da.z, da.w, db.x, db.y, db.z, db.w};
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            bf16x2 hi;
            f32x2 rest, rest2;
            split_pair((float)zf[e] * dw[e], (float)zf[e + 1] * dw[e + 1], hi, rest);
            z0[e] = hi[0], z0[e + 1] = hi[1];
            split_pair(rest[0], rest[1], hi, rest2);
            z1[e] = hi[0], z1[e + 1] = hi[1];
            z2[e] = (__bf16)rest2[0], z2[e + 1] = (__bf16)rest2[1];
          }
          if constexpr (RATE) {
            const float4 la = *reinterpret_cast<const float4*>(downlag + 16 * js + 4 * half),
                         lb = *reinterpret_cast<const float4*>(downlag + 16 * js + 8 + 4 * half);
            const float lw[8] = {la.x, la.y, la.z, la.w, lb.x, lb.y, lb.z, lb.w};
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              bf16x2 hi;
              f32x2 rest;
              split_pair((float)zf[e] * lw[e], (float)zf[e + 1] * lw[e + 1], hi, rest);
              l0[e] = hi[0], l0[e + 1] = hi[1];
              l1[e] = (__bf16)rest[0], l1[e + 1] = (__bf16)rest[1];
            }
          }
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const bf16x8 yt = read_tr8<KP, true>(ys, ln, 16 * js, 32 * t);
            S[t] = mfma(yt, z0, S[t]);
            S[t] = mfma(yt, z1, S[t]);
            S[t] = mfma(yt, z2, S[t]);
            if constexpr (RATE) {
              D[t] = mfma(yt, l0, D[t]);
              D[t] = mfma(yt, l1, D[t]);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        const int j = 8 * (i / 4) + 4 * half + i % 4;
        const float zf = zs[tile_at<T, BV>(j, wave * 32 + lc)];
        if constexpr (FULL) {
          const bool hit = bad && bits_nonfinite(__float_as_uint(zf));
          const float zp = hit ? 0.f : zf;
          O[0] = mfma(zp, Pd[0][i], O[0]);
          if constexpr (RATE) OD[0] = mfma(zp, Pd[0][i] * (float)(lc - j), OD[0]);
          if (bad) {  // large finite stand-ins times 0 or 1, often enough to overflow
            const float zn = hit ? 3.3e38f : 0.f, one = lc >= j ? 1.f : 0.f;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              O[0] = mfma(zn, one, O[0]);
              if constexpr (RATE) OD[0] = mfma(zn, one, OD[0]);
            }
          }
        }
        if (carry) {
          const float zw = zf * down[j];
          float zl = 0.f;
          if constexpr (RATE) zl = zf * downlag[j];
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const float yt = ys[tile_at<T, KP>(j, 32 * t + lc)];
            S[t] = mfma(yt, zw, S[t]);
            if constexpr (RATE) D[t] = mfma(yt, zl, D[t]);
          }
        }
      }
    }

    if constexpr (FULL) {
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const int i = 32 * t + lc;  // this lane's token
        if (i >= n) continue;
        const int64_t tok = token(u + i);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int c0 = wave * 32 + 8 * r + 4 * half, c = slice * BV + c0;
          const float o[4] = {O[t][4 * r], O[t][4 * r + 1], O[t][4 * r + 2], O[t][4 * r + 3]};
          if constexpr (RATE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) dr += (double)(OD[t][4 * r + e] * to_f32(dots[tile_at<T, BV>(i, c0 + e)]));
          }
          if (!p.out || c >= V) continue;
          const uint64_t at = ((uint64_t)tok * p.heads + h) * V + c;
          if (p.out_f32 || !BF) {
            float* dst = static_cast<float*>(p.out) + at;
            if (a.vec_out) *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
            else
              for (int e = 0; e < 4; ++e)
                if (c + e < V) dst[e] = o[e];
          } else {
            T* dst = static_cast<T*>(p.out) + at;
            if (a.vec_out) {
              const bf16x4 v = {(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
              *reinterpret_cast<bf16x4*>(dst) = v;
            } else {
              for (int e = 0; e < 4; ++e)
                if (c + e < V) dst[e] = from_f32<T>(o[e]);
            }
          }
        }
      }
    }
  }

  // the carry after the segment
  float* to = nullptr;
  int colf = col, halff = half;
  asm volatile("" : "+v"(colf), "+v"(halff));  // the row and column tests are made again, not kept over the loop
  if (!FULL) to = a.bound + bound_at(sg.u0 + sg.n);
  else if (last_seg && p.s_out) to = p.s_out;
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 32 * t + carry_row<T>(i / 4, i % 4, halff);
      if (row >= K || colf >= V) continue;
      if (to) to[FULL ? sat(row, colf) : (uint64_t)row * V + colf] = S[t][i];
      if constexpr (RATE && !FULL) a.bound_d[bound_at(sg.u0 + sg.n) + (uint64_t)row * V + colf] = D[t][i];
      if constexpr (DOT)
        if (last_seg && p.ds_out) dr += (double)(D[t][i] * p.ds_out[sat(row, colf)]);
    }
  if constexpr (DOT) {
    for (int off = 32; off; off >>= 1) dr += __shfl_xor(dr, off);
    if (lane == 0) red[wave] = dr;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int i = 0; i < NW; ++i) s += red[i];
      a.drate[(slot * a.slices + slice) * p.heads + h] = -s;
    }
  }
}

// kp: K rounded up to 64, 128 or 256; nw: waves per block, 32 columns each (4, or 2 where K and V are at most 64)
template <typename T>
void attn_chunk_launch(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);

template <typename T, int KP, int NW>
void attn_chunk_launch_at(const AttnChunkArgs& a, bool full, bool rate, hipStream_t s) {
  const dim3 grid((unsigned)xcd_blocks(a.tiles)), block(NW * kWave);
  if (full) {
    if (rate) k_attn_chunk<T, KP, NW, true, true><<<grid, block, 0, s>>>(a);
    else k_attn_chunk<T, KP, NW, true, false><<<grid, block, 0, s>>>(a);
  } else {
    if (rate) k_attn_chunk<T, KP, NW, false, true><<<grid, block, 0, s>>>(a);
    else k_attn_chunk<T, KP, NW, false, false><<<grid, block, 0, s>>>(a);
  }
}
#define LAPLEX_ATTN_CHUNK_SIZES(T)                                                                         \
  template <>                                                                                              \
  void attn_chunk_launch<T>(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s) { \
    if (kp == 64 && nw == 2) attn_chunk_launch_at<T, 64, 2>(a, full, rate, s);                             \
    else if (kp == 64) attn_chunk_launch_at<T, 64, 4>(a, full, rate, s);                                   \
    else if (kp == 128) attn_chunk_launch_at<T, 128, 4>(a, full, rate, s);                                 \
    else attn_chunk_launch_at<T, 256, 4>(a, full, rate, s);                                                \
  }

}  // namespace laplex
