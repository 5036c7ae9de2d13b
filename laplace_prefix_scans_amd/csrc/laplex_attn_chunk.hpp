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
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
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

// A tile's 16-byte pieces on their way from memory to LDS: thread -> column
// piece threadIdx.x % (P / E) of every RPI-th row.
template <typename T, int ROWS, int P, int THREADS, bool VEC>
struct Stage {
  static constexpr int E = 16 / sizeof(T), RPI = THREADS / (P / E), N = ROWS / RPI;
  static_assert(THREADS % (P / E) == 0 && ROWS % RPI == 0, "pieces divide evenly");
  uint4 v[N];
  const T* at;       // this thread's first piece in the next chunk
  int64_t rows_it;   // elements from one of its pieces to the next
  int cols;          // columns from its piece's first to the end of the row
  // p: the row of the first token, col0: the tile's first column, stride: elements from a row of the tile to the next
  __device__ __forceinline__ void init(const T* p, int64_t stride, int col0, int width) {
    const int r = threadIdx.x / (P / E), c = col0 + threadIdx.x % (P / E) * E;
    at = p + r * stride + c;
    rows_it = RPI * stride;
    cols = width - c;
  }
  // The next chunk's rows [0, rows); rows and columns past the end are zero.  whole: every column is there.
  __device__ __forceinline__ void load(int rows, bool whole) {
    const int r0 = threadIdx.x / (P / E);
    const T* src = at;
    if (VEC && whole && rows == ROWS) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = *reinterpret_cast<const uint4*>(src);
        src += rows_it;
      }
      at = src;
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if constexpr (VEC) {
        if (r0 + i * RPI < rows && cols > 0) q = *reinterpret_cast<const uint4*>(src);
      } else {
        T e[E];
#pragma unroll
        for (int j = 0; j < E; ++j) e[j] = r0 + i * RPI < rows && j < cols ? src[j] : T(0.f);
        __builtin_memcpy(&q, e, 16);
      }
      v[i] = q;
      src += rows_it;
    }
    at = src;
  }
  __device__ __forceinline__ void store(T* tile) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = threadIdx.x / (P / E) + i * RPI, c = threadIdx.x % (P / E);
      *reinterpret_cast<uint4*>(tile + r * P + ((c ^ swz<T, P>(r)) * E)) = v[i];
    }
  }
  // Replaces infinities and NaN by 0 and lowers first[column of the tile] to their row; whether there were any.
  __device__ __forceinline__ bool clean(int* first) {
    // the largest magnitude, as an integer: infinities and NaN are above every finite one
    bool bad;
    if constexpr (sizeof(T) == 2) {
      u16x2 top = {0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[j] & 0x7FFF7FFFu));
      }
      bad = top[0] >= 0x7F80u || top[1] >= 0x7F80u;
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) top = max(max(max(top, v[i].x & 0x7FFFFFFFu), max(v[i].y & 0x7FFFFFFFu, v[i].z & 0x7FFFFFFFu)), v[i].w & 0x7FFFFFFFu);
      bad = top >= 0x7F800000u;
    }
    if (!bad) return false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      T e[E];
      __builtin_memcpy(e, &v[i], 16);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (bits_nonfinite(__float_as_uint(to_f32(e[j])))) {
          e[j] = T(0.f);
          atomicMin(first + threadIdx.x % (P / E) * E + j, (int)threadIdx.x / (P / E) + i * RPI);
        }
      __builtin_memcpy(&v[i], e, 16);
    }
    return true;
  }
};

// Two floats as a pair of bfloat16, and what the pair leaves over: x = hi + lo
// (+ lo2) in two (three) parts loses 2^-17 (2^-25) of x.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ uint32_t split_pair(float& a, float& b) {
  const uint32_t w = pack_bf16(a, b);
  a -= __uint_as_float(w << 16);
  b -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}
struct Parts2 {
  bf16x8 hi, lo;
};
__device__ __forceinline__ Parts2 split2(const float (&x)[8]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
    h[i] = split_pair(a, b);
    l[i] = pack_bf16(a, b);
  }
  return {__builtin_bit_cast(bf16x8, make_uint4(h[0], h[1], h[2], h[3])), __builtin_bit_cast(bf16x8, make_uint4(l[0], l[1], l[2], l[3]))};
}
struct Parts3 {
  bf16x8 hi, lo, lo2;
};
__device__ __forceinline__ Parts3 split3(const float (&x)[8]) {
  uint32_t h[4], l[4], m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
    h[i] = split_pair(a, b);
    l[i] = split_pair(a, b);
    m[i] = pack_bf16(a, b);
  }
  return {__builtin_bit_cast(bf16x8, make_uint4(h[0], h[1], h[2], h[3])), __builtin_bit_cast(bf16x8, make_uint4(l[0], l[1], l[2], l[3])),
          __builtin_bit_cast(bf16x8, make_uint4(m[0], m[1], m[2], m[3]))};
}

struct AttnChunkArgs {
  AttnPass p;
  AttnSegs g;
  uint32_t slices;   // blocks across the V columns
  uint32_t group;    // query heads per shared head
  uint64_t slots;    // segments, with room for unused ones
  float* bound;      // states at segment boundaries ([boundary][head][K][V]), or null
  float* bound_d;    // the lag-weighted ones (rate gradient)
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
template <typename T, int KP, int NW, bool FULL, bool RATE, bool VEC>
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
  // bf16: operand [tile][channel half][part] of a lane (the lag-weighted ones behind them); float: [wave][register quad]
  using Pair = std::conditional_t<BF, bf16x8, float4>;
  __shared__ Pair pairs[(FULL ? (BF ? (RATE ? 24 : 12) : NW * 4) : 1) * kWave];
  __shared__ int bad_chunk[2], bad_row[2][FULL ? BV : 1];
  __shared__ double red[NW];

  // Blocks that read the same rows (the column slices and the heads of one shared head) follow each other on
  // one XCD; these units go to the XCDs in turn, so that unused slots leave none of them with less work.
  const uint32_t per = a.group * a.slices, at_xcd = blockIdx.x / kXcds;
  const uint64_t unit = (uint64_t)(at_xcd / per) * kXcds + blockIdx.x % kXcds, shared = p.heads / a.group;
  const uint32_t slice = at_xcd % a.slices, h = (uint32_t)(unit % shared) * a.group + at_xcd % per / a.slices;
  const uint64_t slot = unit / shared;
  if (slot >= a.slots) return;
  const AttnSeg sg = find_seg(a.g, slot);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id(), half = lane >> 5, lc = lane & 31;
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
  // states in memory: element (row, column) at row * rs + column * cs of the caller's ([seq][head], either order) or of a boundary's
  const uint64_t sbase = ((uint64_t)sg.seq * p.heads + h) * (uint64_t)K * V;
  const int rs = p.s_trans ? 1 : V, cs = p.s_trans ? K : 1;
  const uint64_t per_bound = (uint64_t)K * V;
  auto bound_at = [&](int64_t u) { return ((uint64_t)((sg.first + u) / a.g.seg_len) * p.heads + h) * per_bound; };
  auto load_state = [&](f32x16 (&s)[KT], const float* src, int rs, int cs) {
    if (col >= V) return;
    src += (int64_t)col * cs;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = 32 * t + carry_row<T>(i / 4, i % 4, half);
        const float v = src[min(row, K - 1) * rs];
        s[t][i] = row < K ? v : 0.f;
      }
  };

  f32x16 S[KT], D[RATE ? KT : 1];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    S[t] = f32x16{};
    if constexpr (RATE) D[t] = f32x16{};
  }
  if constexpr (FULL) {
    if (sg.u0 > 0) {
      const uint64_t at = bound_at(sg.u0);
      load_state(S, a.bound + at, V, 1);
      if constexpr (RATE) load_state(D, a.bound_d + at, V, 1);
    } else if (p.s_in) {
      load_state(S, p.s_in + sbase, rs, cs);
    }
  }

  // weights of a pair inside a chunk by its lag, 0 for the pairs above the diagonal
  if constexpr (FULL)
    for (int i = threadIdx.x; i < 2 * C; i += THREADS) wt[i] = i >= C ? p.c_pair * decay(-rate * (float)(i - C)) : 0.f;
  float up[IT];
  if constexpr (FULL)
#pragma unroll
    for (int t = 0; t < IT; ++t) up[t] = p.c_in * decay(-rate * (float)(32 * t + lc + lead));
  // The carry's decay over a chunk.  As one float its rounding would add up, the same way each time, over the
  // thousands of chunks that a slow decay reaches: each chunk takes the float nearest to what brings the product
  // so far back to the exact one.
  const double wc = exp(-(double)rate * (double)C);
  double owed = 1.0;
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

  Stage<T, C, KP, THREADS, VEC> sx, sy;
  Stage<T, C, BV, THREADS, VEC> sz, sd;
  const bool whole_v = ((int)slice + 1) * BV <= V;
  const int64_t t0 = token(sg.u0);
  if constexpr (FULL) sx.init(x + t0 * p.x.token, step * p.x.token, 0, K);
  sy.init(y + t0 * p.y.token, step * p.y.token, 0, K);
  sz.init(z + t0 * p.z.token, step * p.z.token, slice * BV, V);
  if constexpr (DOT) sd.init(dot + t0 * p.dot_view.token, step * p.dot_view.token, slice * BV, V);
  auto load = [&](int64_t u) {
    const int rows = (int)min((int64_t)C, sg.u0 + sg.n - u);
    if constexpr (FULL) sx.load(rows, K == KP);
    sy.load(rows, K == KP);
    sz.load(rows, whole_v);
    if constexpr (DOT) sd.load(rows, whole_v);
  };
  f32x16 O[FULL ? IT : 1];
  // Writes the outputs of the chunk at u.  Called when the next chunk is in LDS: stores are counted with the
  // loads, so writing before would make the wait for the next chunk's rows one for the stores too.
  auto put = [&](int64_t u) {
    if (!active || !p.out) return;
    const int n = (int)min((int64_t)C, sg.u0 + sg.n - u);
#pragma unroll
    for (int t = 0; t < IT; ++t) {
      const int i = 32 * t + lc;  // this lane's token
      if (i >= n) continue;
      const int c0 = slice * BV + wave * 32 + 4 * half;
      const uint64_t at = ((uint64_t)token(u + i) * p.heads + h) * V + c0;
      if (p.out_f32 || !BF) {
        float* dst = static_cast<float*>(p.out) + at;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (VEC) {
            if (c0 + 8 * r < V)
              *reinterpret_cast<float4*>(dst + 8 * r) = make_float4(O[t][4 * r], O[t][4 * r + 1], O[t][4 * r + 2], O[t][4 * r + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c0 + 8 * r + e < V) dst[8 * r + e] = O[t][4 * r + e];
          }
        }
      } else {
        T* dst = static_cast<T*>(p.out) + at;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (VEC) {
            if (c0 + 8 * r < V)
              *reinterpret_cast<uint2*>(dst + 8 * r) = make_uint2(pack_bf16(O[t][4 * r], O[t][4 * r + 1]), pack_bf16(O[t][4 * r + 2], O[t][4 * r + 3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c0 + 8 * r + e < V) dst[8 * r + e] = from_f32<T>(O[t][4 * r + e]);
          }
        }
      }
    }
  };
  double dr = 0.0;
  if (threadIdx.x < 2) bad_chunk[threadIdx.x] = 0;
  if constexpr (FULL)
    for (int i = threadIdx.x; i < 2 * BV; i += THREADS) bad_row[i / BV][i % BV] = C;
  set_down((int)min((int64_t)C, sg.n));
  if (sg.n > 0) load(sg.u0);
  int parity = 0;
  for (int64_t u = sg.u0; u < sg.u0 + sg.n; u += C, parity ^= 1) {
    const int n = (int)min((int64_t)C, sg.u0 + sg.n - u);
    __syncthreads();  // the previous chunk's reads are done
    if constexpr (FULL) sx.store(xs);
    sy.store(ys);
    // A masked pair weighs 0, but 0 times an infinity is NaN: infinities and NaN in z are taken out of the
    // tile, and what they reach -- their own and later tokens of their column, the carry -- is set to NaN below.
    if (FULL && sz.clean(bad_row[parity])) bad_chunk[parity] = 1;
    sz.store(zs);
    if constexpr (DOT) sd.store(dots);
    if (threadIdx.x == 0) bad_chunk[parity ^ 1] = 0;
    if (FULL && (int)threadIdx.x < BV) bad_row[parity ^ 1][threadIdx.x] = C;
    if (n < C && u > sg.u0) set_down(n);
    __syncthreads();
    const bool more = u + C < sg.u0 + sg.n;
    if (FULL && u > sg.u0) put(u - C);
    if (more) load(u + C);
    const bool bad = FULL && bad_chunk[parity] != 0;
    // the lane as the compiler sees it changes with every chunk: the many LDS offsets made from it are
    // then formed where they are used (an xor each) instead of each holding a register over the loop
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int half = ln >> 5, lc = ln & 31;

    f32x16 OD[DOT ? IT : 1];
    if constexpr (FULL) {
      // The weighted pairs are the same for every column: the waves share them out and pass them on through LDS.
      if constexpr (BF) {
        // P^T tiles (rows j, columns i): (0, 0), (1, 1) on the diagonal and (0, 1), as operands of two bfloat16 parts
        for (int tile = wave; tile < 3; tile += NW) {
          const int j0 = tile == 1 ? 32 : 0, i0 = tile == 0 ? 0 : 32;
          f32x16 P = {};
#pragma unroll
          for (int ks = 0; ks < KP / 16; ++ks) {
            const bf16x8 xf = *reinterpret_cast<const bf16x8*>(xs + tile_at<T, KP>(i0 + lc, 16 * ks + 8 * half));
            const bf16x8 yf = *reinterpret_cast<const bf16x8*>(ys + tile_at<T, KP>(j0 + lc, 16 * ks + 8 * half));
            P = mfma(yf, xf, P);
          }
          const float* w0 = wt + C + i0 - j0 + lc - 4 * half;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float pv[8], pd[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int i = 8 * s + e, j = 8 * (i / 4) + i % 4;
              const float w = w0[-j];
              pv[e] = w != 0.f ? P[i] * w : 0.f;  // a masked pair is 0 whatever its product
              if constexpr (RATE) pd[e] = pv[e] * (float)(i0 - j0 + lc - 4 * half - j);
            }
            const Parts2 p2 = split2(pv);
            pairs[((tile * 2 + s) * 2) * kWave + ln] = p2.hi;
            pairs[((tile * 2 + s) * 2 + 1) * kWave + ln] = p2.lo;
            if constexpr (RATE) {
              const Parts2 d2 = split2(pd);
              pairs[((6 + tile * 2 + s) * 2) * kWave + ln] = d2.hi;
              pairs[((6 + tile * 2 + s) * 2 + 1) * kWave + ln] = d2.lo;
            }
          }
        }
      } else {
        // each wave adds a share of the channels of P^T
        f32x16 P = {};
#pragma unroll
        for (int k = 0; k < KP / NW / 8; ++k) {
          const int ch = wave * (KP / NW) + 8 * k + 4 * half;
          const float4 xf = *reinterpret_cast<const float4*>(xs + tile_at<T, KP>(lc, ch));
          const float4 yf = *reinterpret_cast<const float4*>(ys + tile_at<T, KP>(lc, ch));
          P = mfma(yf.x, xf.x, P);
          P = mfma(yf.y, xf.y, P);
          P = mfma(yf.z, xf.z, P);
          P = mfma(yf.w, xf.w, P);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          pairs[(wave * 4 + r) * kWave + ln] = make_float4(P[4 * r], P[4 * r + 1], P[4 * r + 2], P[4 * r + 3]);
      }
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        O[t] = f32x16{};
        if constexpr (RATE) OD[t] = f32x16{};
      }
      if (active) {
        // out^T = S^T x^T (rows V, columns i)
        if constexpr (BF) {
#pragma unroll
          for (int ks = 0; ks < KP / 16; ++ks) {
            bf16x8 xf[IT];
#pragma unroll
            for (int t = 0; t < IT; ++t) xf[t] = *reinterpret_cast<const bf16x8*>(xs + tile_at<T, KP>(32 * t + lc, 16 * ks + 8 * half));
            // the carry enters as two bfloat16 parts: with one, its rounding would show beside the output's own
            float sv[8], dv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              sv[e] = S[ks / 2][8 * (ks % 2) + e];
              if constexpr (RATE) dv[e] = D[ks / 2][8 * (ks % 2) + e];
            }
            const Parts2 s2 = split2(sv);
#pragma unroll
            for (int t = 0; t < IT; ++t) O[t] = mfma(s2.hi, xf[t], O[t]);
#pragma unroll
            for (int t = 0; t < IT; ++t) O[t] = mfma(s2.lo, xf[t], O[t]);
            if constexpr (RATE) {
              const Parts2 d2 = split2(dv);
#pragma unroll
              for (int t = 0; t < IT; ++t) {
                OD[t] = mfma(d2.hi, xf[t], OD[t]);
                OD[t] = mfma(d2.lo, xf[t], OD[t]);
              }
            }
          }
        } else {
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float4 xf = *reinterpret_cast<const float4*>(xs + tile_at<T, KP>(lc, 32 * t + 8 * r + 4 * half));
              const float xe[4] = {xf.x, xf.y, xf.z, xf.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
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
          }
      }
      __syncthreads();  // every wave's share of the pairs is there
    }
    if (!active) continue;

    // the carry over the chunk, with the lag-weighted one ahead of it
    const bool carry = !FULL || more || keep;
    if (carry) {
      const double exact = (n == C ? wc : exp(-(double)rate * (double)n)) * owed;
      const float w = (float)exact;
      owed = w != 0.f ? exact / (double)w : 1.0;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if constexpr (RATE) {
            D[t][i] = w * fmaf((float)n, S[t][i], D[t][i]);
          }
          S[t][i] *= w;
        }
    }
    if constexpr (BF) {
#pragma unroll
      for (int js = 0; js < C / 16; ++js) {
        const bf16x8 zf = read_tr8<BV, false>(zs, ln, 16 * js, wave * 32);
        if constexpr (FULL) {
#pragma unroll
          for (int t = 0; t < IT; ++t) {
            if (js >= 2 * (t + 1)) continue;  // pairs above the diagonal
            const bf16x8* pf = pairs + (((js >= 2 * t ? t : 2) * 2 + js % 2) * 2) * kWave + ln;
            O[t] = mfma(zf, pf[0], O[t]);
            O[t] = mfma(zf, pf[kWave], O[t]);
            if constexpr (RATE) {
              OD[t] = mfma(zf, pf[12 * kWave], OD[t]);
              OD[t] = mfma(zf, pf[13 * kWave], OD[t]);
            }
          }
        }
        if (carry) {
          // z weighted by its decay to the chunk's end, as three bfloat16 parts: the carry keeps float32's bits
          auto weighted = [&](const float* w, float (&out)[8]) {
            const float4 wa = *reinterpret_cast<const float4*>(w + 16 * js + 4 * half),
                         wb = *reinterpret_cast<const float4*>(w + 16 * js + 8 + 4 * half);
            const float ws[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = (float)zf[e] * ws[e];
          };
          float zw[8], zl[8];
          weighted(down, zw);
          const Parts3 z3 = split3(zw);
          Parts2 l2;
          if constexpr (RATE) {
            weighted(downlag, zl);
            l2 = split2(zl);
          }
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const bf16x8 yt = read_tr8<KP, true>(ys, ln, 16 * js, 32 * t);
            S[t] = mfma(yt, z3.hi, S[t]);
            S[t] = mfma(yt, z3.lo, S[t]);
            S[t] = mfma(yt, z3.lo2, S[t]);
            if constexpr (RATE) {
              D[t] = mfma(yt, l2.hi, D[t]);
              D[t] = mfma(yt, l2.lo, D[t]);
            }
          }
        }
      }
    } else {
      f32x16 P = {};
      if constexpr (FULL) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float4 s = pairs[r * kWave + ln];
#pragma unroll
          for (int k = 1; k < NW; ++k) {
            const float4 v = pairs[(k * 4 + r) * kWave + ln];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
          }
          const float* w = wt + C + lc - 4 * half - 8 * r;
          const float pv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) P[4 * r + e] = w[-e] != 0.f ? pv[e] * w[-e] : 0.f;  // a masked pair is 0 whatever its product
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 8 * (i / 4) + 4 * half + i % 4;
        const float zf = zs[tile_at<T, BV>(j, wave * 32 + lc)];
        if constexpr (FULL) {
          O[0] = mfma(zf, P[i], O[0]);
          if constexpr (RATE) OD[0] = mfma(zf, P[i] * (float)(lc - j), OD[0]);
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
      if (bad) {
        const float nan = __builtin_nanf("");
        const int* first = bad_row[parity] + wave * 32;
        const bool gone = first[lc] < C;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
          for (int t = 0; t < IT; ++t) {
            const bool hit = 32 * t + lc >= first[8 * (i / 4) + 4 * half + i % 4];
            O[t][i] = hit ? nan : O[t][i];
            if constexpr (RATE) OD[t][i] = hit ? nan : OD[t][i];
          }
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            S[t][i] = gone ? nan : S[t][i];
            if constexpr (RATE) D[t][i] = gone ? nan : D[t][i];
          }
        }
      }
      if constexpr (DOT) {
#pragma unroll
        for (int t = 0; t < IT; ++t)
#pragma unroll
          for (int k = 0; k < 16; ++k)  // rows past the end are zero in the tile
            dr += (double)(OD[t][k] * to_f32(dots[tile_at<T, BV>(32 * t + lc, wave * 32 + 8 * (k / 4) + 4 * half + k % 4)]));
      }
    }
  }
  if (FULL && sg.n > 0) put(sg.u0 + (sg.n - 1) / C * C);

  // the carry after the segment
  int colf = col, halff = half;
  asm volatile("" : "+v"(colf), "+v"(halff));  // the row and column tests are made again, not kept over the loop
  auto each = [&](int rs, int cs, auto&& f) {
    if (colf >= V) return;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = 32 * t + carry_row<T>(i / 4, i % 4, halff);
        if (row < K) f(t, i, row * rs + colf * cs);
      }
  };
  if constexpr (!FULL) {
    const uint64_t at = bound_at(sg.u0 + sg.n);
    float* to = a.bound + at;
    each(V, 1, [&](int t, int i, int o) { to[o] = S[t][i]; });
    if constexpr (RATE) {
      float* tod = a.bound_d + at;
      each(V, 1, [&](int t, int i, int o) { tod[o] = D[t][i]; });
    }
  } else if (last_seg) {
    if (p.s_out) {
      float* to = p.s_out + sbase;
      each(rs, cs, [&](int t, int i, int o) { to[o] = S[t][i]; });
    }
    if constexpr (RATE)
      if (p.ds_out) {
        const float* g = p.ds_out + sbase;
        each(rs, cs, [&](int t, int i, int o) { dr += (double)(D[t][i] * g[o]); });
      }
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
template <typename T, int KP, int NW, bool VEC>
void attn_chunk_launch_at(const AttnChunkArgs& a, bool full, bool rate, hipStream_t s) {
  const uint64_t units = a.slots * (a.p.heads / a.group);
  const dim3 grid((unsigned)(xcd_blocks(units) * a.group * a.slices)), block(NW * kWave);
  if (full) {
    if (rate) k_attn_chunk<T, KP, NW, true, true, VEC><<<grid, block, 0, s>>>(a);
    else k_attn_chunk<T, KP, NW, true, false, VEC><<<grid, block, 0, s>>>(a);
  } else {
    if (rate) k_attn_chunk<T, KP, NW, false, true, VEC><<<grid, block, 0, s>>>(a);
    else k_attn_chunk<T, KP, NW, false, false, VEC><<<grid, block, 0, s>>>(a);
  }
}
template <typename T, bool VEC>
void attn_chunk_launch(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s) {
  if (kp == 64 && nw == 2) attn_chunk_launch_at<T, 64, 2, VEC>(a, full, rate, s);
  else if (kp == 64) attn_chunk_launch_at<T, 64, 4, VEC>(a, full, rate, s);
  else if (kp == 128) attn_chunk_launch_at<T, 128, 4, VEC>(a, full, rate, s);
  else attn_chunk_launch_at<T, 256, 4, VEC>(a, full, rate, s);
}

// The instantiations, each in a source file of its own.  vec: every row of x, y, z, dot and out is 16-byte aligned.
void attn_chunk_bf16_vec(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);
void attn_chunk_bf16_any(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);
void attn_chunk_f32_vec(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);
void attn_chunk_f32_any(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);

}  // namespace laplex
