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
// apart over all sequences, so position / seg_len numbers them uniquely (AttnPlan::bounds).

// a value that every lane holds, in scalar registers
template <typename V>
__device__ __forceinline__ V uniform(V v) {
  static_assert(sizeof(V) == 8, "two words");
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
}

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
  // every lane has found the same: what follows from it then needs no vector registers
  s.first = uniform(s.first);
  s.len = uniform(s.len);
  s.seq = __builtin_amdgcn_readfirstlane(s.seq);
  s.u0 = uniform(seg) * g.seg_len;
  s.n = min(g.seg_len, s.len - s.u0);
  return s;
}

// ------------------------------------------------------------------ tiles in LDS
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// Rows of a tile are 16-byte pieces; piece c of row r is kept at c ^ swz(r), so
// that the reads spread over the 64 banks: 16 bytes from each of 16 rows (row
// operands), and for the transposed operands 8 rows of 32 bytes (bf16) or four
// rows 4 apart of 64 (float).
template <typename T, int P>
__device__ __forceinline__ int swz(int r) {
  if constexpr (sizeof(T) == 2) {
    const int low = (((r >> 2) & 1) << 1) | ((r >> 3) & 1);
    if constexpr (P == 64) return (((r >> 1) & 1) << 2) | low;
    else return ((r & 3) << 2) | low;
  } else {
    return (((r >> 2) & 3) << 2) | (r & 3);
  }
}
// element offset of column c (any) of row r
template <typename T, int P>
__device__ __forceinline__ int tile_at(int r, int c) {
  constexpr int E = 16 / sizeof(T);
  return r * P + (((c / E) ^ swz<T, P>(r)) * E) + c % E;
}

// Memory by a descriptor of its first byte and its length, both the same for every thread, and 32 bits of each
// thread's own: one vector register an address, and the hardware's bounds check in place of branches -- a read
// past the length is 0 and a write there is dropped.  kNowhere is past every length, by a chunk's rows to either side.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const void* first, uint32_t bytes) {
  void* p = reinterpret_cast<void*>(uniform((uint64_t)reinterpret_cast<uintptr_t>(first)));
  return __builtin_amdgcn_make_buffer_rsrc(p, 0, __builtin_amdgcn_readfirstlane(bytes), 0x00027000);  // raw, 32-bit words
}

template <typename T>
constexpr int kAttnC = sizeof(T) == 2 ? 64 : 32;  // tokens per chunk

// The ten 16 x 16 tiles of the weighted pairs on and below the diagonal, as operands over 32 rows j: per operand three
// parts of 64 lanes' 16 bytes, and 8 bytes in the two whose second 16 rows lie above the diagonal.  15 KB, so that two
// blocks of eight waves and 128 rows of the carry fit the LDS of a CU.  First 8-byte word of tile i's operand of rows 32 s on:
__device__ __forceinline__ constexpr int pair_at(int i, int s) {
  return i == 2 * s ? (4 * 2 + s) * 3 * kWave : (i == 1 ? 0 : i - 1 + (i == 3 ? s : 0)) * 2 * 3 * kWave;
}

// The first rows with an infinity or NaN, a byte per column of a tile (kNoRow: none; a chunk has at most 64 rows).
constexpr uint32_t kNoRow = 0x40404040u;
__device__ __forceinline__ int row_byte(const uint32_t* rows, int col) { return (rows[col / 4] >> col % 4 * 8) & 0xFF; }
__device__ __forceinline__ void lower_row_byte(uint32_t* rows, int col, uint32_t row) {
  uint32_t* at = rows + col / 4;
  const int shift = col % 4 * 8;
  uint32_t old = *at;
  while ((old >> shift & 0xFF) > row) {  // (a swap fails only where another lowered a byte of the word: a bounded number of times)
    const uint32_t seen = atomicCAS(at, old, (old & ~(0xFFu << shift)) | row << shift);
    if (seen == old) break;
    old = seen;
  }
}

// The thread's number, as something the compiler takes to change with every call: what is made from it is
// then formed where it is used instead of holding a register over the loop.
__device__ __forceinline__ int thread_now() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// A tile's 16-byte pieces on their way from memory to LDS: thread -> column
// piece threadIdx.x % (P / E) of every RPI-th row.
template <typename T, int ROWS, int P, int THREADS, bool VEC>
struct Stage {
  static constexpr int E = 16 / sizeof(T), RPI = THREADS / (P / E), N = ROWS / RPI;
  static_assert(THREADS % (P / E) == 0 && ROWS % RPI == 0, "pieces divide evenly");
  uint4 v[N];
  // All of these are the same for every thread; a thread's own offsets are formed anew each time.
  using Bytes = std::conditional_t<VEC, int32_t, int64_t>;  // (VEC: the host has seen that a chunk's rows span less than 2^30 bytes)
  const char* at;  // the next chunk's first row, at the tile's first column
  Bytes pitch;     // bytes from a row to the next token's: negative where the tokens run backwards
  __device__ __forceinline__ void init(const T* p, int64_t stride, int step, int col0) {
    pitch = (Bytes)(stride * step) * (Bytes)sizeof(T);
    at = reinterpret_cast<const char*>(p + col0);
  }
  // The next chunk's rows [0, rows); rows, and columns from `width` on, are zero.
  __device__ __forceinline__ void load(int rows, int width) {
    const int t = thread_now(), r0 = t / (P / E), c = t % (P / E) * E;
    if constexpr (VEC) {
      // (rows do not overlap, so those outside [0, rows) lie outside the descriptor's bytes)
      const int32_t back = min((rows - 1) * pitch, 0), span = abs((rows - 1) * pitch);
      const __amdgpu_buffer_rsrc_t m = rows_at(at + back, (uint32_t)span + (uint32_t)width * (uint32_t)sizeof(T));
      const uint32_t off = c < width ? (uint32_t)(r0 * pitch - back) + c * (uint32_t)sizeof(T) : kNowhere;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(m, off + (uint32_t)(i * RPI * pitch), 0, 0));
    } else {
      // Pieces at the alignment of T.  A row's last one is read 16 bytes before its end and shifted down; rows
      // shorter than a piece are read one by one.
      const char* p = at + r0 * pitch;
      const int past = max(c + E - width, 0);  // elements of the piece behind the row's end
#pragma unroll
      for (int i = 0; i < N; ++i) {
        unsigned __int128 w = 0;
        if (r0 + i * RPI < rows && c < width) {
          const T* q = reinterpret_cast<const T*>(p + i * RPI * pitch);
          if (width >= E) {
            __builtin_memcpy(&w, q + (c - past), 16);
            if (past) w >>= past * (int)sizeof(T) * 8;
          } else {
            for (int j = width - 1; j >= 0; --j) {
              uint32_t one = 0;
              __builtin_memcpy(&one, q + j, sizeof(T));
              w = w << sizeof(T) * 8 | one;
            }
          }
        }
        __builtin_memcpy(&v[i], &w, 16);
      }
    }
    at += (int64_t)(ROWS * pitch);
  }
  __device__ __forceinline__ void store(T* tile) const {
    const int t = thread_now();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = t / (P / E) + i * RPI, c = t % (P / E);
      *reinterpret_cast<uint4*>(tile + r * P + ((c ^ swz<T, P>(r)) * E)) = v[i];
    }
  }
  // Replaces infinities and NaN by 0 and lowers the byte of their column in `first` to their row; whether there were any.
  __device__ __forceinline__ bool clean(uint32_t* first) {
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
    const int t = thread_now();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      T e[E];
      __builtin_memcpy(e, &v[i], 16);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (bits_nonfinite(__float_as_uint(to_f32(e[j])))) {
          e[j] = T(0.f);
          lower_row_byte(first, t % (P / E) * E + j, t / (P / E) + i * RPI);
        }
      __builtin_memcpy(&v[i], e, 16);
    }
    return true;
  }
};

// Two floats as a pair of bfloat16, and what the pair leaves over.  Three parts of 8 bits, x = hi + lo + lo2, hold the
// 24 of a float (short of 2^-110): carries, pairs and weighted rows enter bfloat16 products with all of their bits, and
// every sum is float32's.  Two parts would lose 2^-18 of each, a thousandth of a bfloat16 result's own rounding, but more than
// float32 does (65536 tokens x 8 heads, 128 x 128: whole pass 193 us, with two parts 154; states alone 73 and 66).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ uint32_t split_pair(float& a, float& b) {
  const uint32_t w = pack_bf16(a, b);
  a -= __uint_as_float(w << 16);
  b -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}
struct Parts {
  bf16x8 hi, lo, lo2;
};
__device__ __forceinline__ Parts split(const f32x4& u, const f32x4& v) {
  const float x[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
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
  bool bound_trans;  // they are [V][K], from a pass with the roles of K and V exchanged
  float* bound_d;    // the lag-weighted ones (rate gradient)
  double* drate;     // Rate: partials [slot][slice][head]
};

// row of the carry that register r of 16-row tile t holds in lane group g
__device__ __forceinline__ int carry_row(int t, int g, int r) { return 16 * t + 4 * g + r; }

// Operands from LDS.  The piece index of a tile is xored with swz(row), and every
// step over channels changes only bits above the ones that a lane group or quad
// sets: a lane's byte offset for step k is its first xor (k << 6), and steps of 16
// rows, which swz does not see, are constants.  So three offsets per lane
// serve all reads of a chunk.
template <typename T, int P>
__device__ __forceinline__ uint32_t row_operand(int l) {  // row l % 16, channels 4 (l / 16) + {0..3}
  return tile_at<T, P>(l & 15, (l >> 4) * 4) * sizeof(T);
}
template <typename T>
__device__ __forceinline__ const T& lds_at(const void* tile, uint32_t bytes) {
  return *reinterpret_cast<const T*>(static_cast<const char*>(tile) + bytes);
}
// Row operand of a bf16 product over 32 channels: those of the carry's tiles 2k and 2k + 1 in lane group g,
// 32 k + 4 g + {0..3} and 16 on, so that the carry's registers are the other operand as they are.
__device__ __forceinline__ bf16x8 read_row(const __bf16* tile, uint32_t bytes) {
  // (volatile: the compiler would join the reads of two row tiles into one and move the halves about after it)
  typedef const volatile __attribute__((address_space(3))) u32x2* Lds;
  struct { u32x2 a, b; } v = {*(Lds)(reinterpret_cast<const char*>(tile) + bytes), *(Lds)(reinterpret_cast<const char*>(tile) + (bytes ^ 32))};
  return __builtin_bit_cast(bf16x8, v);
}
// Transposed (bf16): a group of 16 lanes reads 4 rows x 16 columns, each lane 4 columns of one row, and gets
// its column's 4 rows back.  Rows 4 (l / 16) + l / 4 % 4, columns from `col` (< 32).
template <int P>
__device__ __forceinline__ uint32_t tr_operand(int l, int col) {
  return tile_at<__bf16, P>(4 * (l >> 4) + ((l >> 2) & 3), col) * 2;
}
template <int P>  // those rows and the ones 16 on
__device__ __forceinline__ bf16x8 read_tr(const __bf16* tile, uint32_t bytes) {
  struct { s16x4 a, b; } v = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(reinterpret_cast<const char*>(tile) + bytes)),
                              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(reinterpret_cast<const char*>(tile) + bytes + 32 * P))};
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x4 mfma(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// sum of a tile's four registers' products and the like: loops over the registers of KT tiles
#define LAPLEX_EACH(t, n, r)   \
  _Pragma("unroll") for (int t = 0; t < (n); ++t) _Pragma("unroll") for (int r = 0; r < 4; ++r)

// One block: a segment's chunks in turn, one head, 16 columns of the carry per
// wave.  The carry's 16 x 16 tiles stay in the accumulators' layout (column =
// lane % 16, row = 4 (lane / 16) + register), which is that of an operand of
// the same column and consecutive rows: the carry enters the products of the
// next chunk without leaving the registers.
//   P^T = y x^T, weighted        (the waves share its tiles out)
//   out^T = up (S^T x^T)
//   S = w(n) S + y^T (down z)
//   out^T += z^T P
// With 16 columns a wave holds 32 registers of a 128-row carry, so that four
// waves share a SIMD and one's conversions run beside another's products;
// 32 columns in half as many waves took as long without the rate's gradient, and a quarter longer with it.
// Measured (bfloat16, 128 x 128; averages).  States alone, 65536 tokens x 8 heads: 73 us for 302 MB, 4.1 TB/s.  The whole
// pass there: 187 us for 570 MB, 3.0 TB/s.  Reads and writes alone take 110 us; the rest is what the four waves of a SIMD do
// not hide of 119 products and about 650 vector instructions a chunk and wave.  Products that do not follow one they add to, and
// fewer instructions to split a float (by two-element dot products), changed nothing.  With the rate's
// gradient, 16384 tokens x 16 heads: 207 us, against 103 without; it has a second carry in three parts and registers for two
// waves a SIMD.
template <typename T, int KP, int NW, bool FULL, bool RATE, bool VEC>
__global__ __launch_bounds__(NW * kWave, KP == 256 || RATE || (KP == 128 && NW == 4) ? 2 : 4) void k_attn_chunk(AttnChunkArgs a) {
  constexpr int C = kAttnC<T>, KT = KP / 16, BV = 16 * NW, THREADS = NW * kWave, IT = C / 16;
  constexpr bool BF = sizeof(T) == 2, DOT = FULL && RATE;
  constexpr int WK = KP / 16 < 4 ? KP / 16 : 4;    // float: waves that share the channels of P^T
  constexpr int ZB = FULL ? 2 : 1;                 // buffers of z
  const AttnPass& p = a.p;
  __shared__ __attribute__((aligned(16))) T xs[FULL ? C * KP : 8];
  __shared__ __attribute__((aligned(16))) T ys[C * KP];
  __shared__ __attribute__((aligned(16))) T zs[ZB][C * BV];
  __shared__ __attribute__((aligned(16))) T dots[2][DOT ? C * BV : 8];
  __shared__ __attribute__((aligned(16))) float down[C], downlag[RATE ? C : 4];
  // Weights of pairs by their lag and of the carry.  bf16: exp(-rate n) alone, for its LDS is full; float: the products,
  // 0 for lags below 0, for its registers are (formed anew, 32 of the eight-wave pass spill).
  __shared__ float dec[FULL && BF ? C + 1 : 1], wt[FULL && !BF ? 2 * C : 1], up[FULL && !BF ? C : 1];
  // bf16: operands of the weighted pairs (pair_at; the lag-weighted ones behind them); float: [wave][tile]
  constexpr int PAIRS = 10 * 3 * kWave;  // 8-byte words
  __shared__ __attribute__((aligned(16))) uint2 pairs[FULL ? (BF ? (RATE ? 2 : 1) * PAIRS : WK * 3 * kWave * 2) : 2];
  __shared__ int bad_chunk[2];
  __shared__ uint32_t bad_row[2][FULL ? BV / 4 : 1];  // a byte per column
  __shared__ double red[DOT ? NW : 1];

  // Blocks that read the same rows (the column slices and the heads of one shared head) follow each other on
  // one XCD; these units go to the XCDs in turn, so that unused slots leave none of them with less work.
  const uint32_t per = a.group * a.slices, at_xcd = blockIdx.x / kXcds;
  const uint64_t unit = (uint64_t)(at_xcd / per) * kXcds + blockIdx.x % kXcds, shared = p.heads / a.group;
  const uint32_t slice = at_xcd % a.slices, h = (uint32_t)(unit % shared) * a.group + at_xcd % per / a.slices;
  const uint64_t slot = unit / shared;
  if (slot >= a.slots) return;
  const AttnSeg sg = find_seg(a.g, slot);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id(), g = lane >> 4, lc = lane & 15;
  const int col = slice * BV + wave * 16 + lc;  // this lane's column of the carry
  const int K = (int)p.K, V = (int)p.V;
  const bool active = (int)slice * BV + wave * 16 < V;  // the wave has columns (all waves move tiles)
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
  const float rate = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(attn_rate(p.rate[h]))));
  const int lead = p.reverse ? 0 : 1;
  const bool keep = !last_seg || p.s_out || (DOT && p.ds_out);  // the carry after the last chunk is needed
  // states in memory: element (row, column) at row * rs + column * cs of the caller's ([seq][head], either order) or of a boundary's
  const uint64_t sbase = ((uint64_t)sg.seq * p.heads + h) * (uint64_t)K * V;
  const int rs = p.s_trans ? 1 : V, cs = p.s_trans ? K : 1;
  const uint64_t per_bound = (uint64_t)K * V;
  const int brs = a.bound_trans ? 1 : V, bcs = a.bound_trans ? K : 1;
  auto bound_at = [&](int64_t u) { return ((uint64_t)((sg.first + u) / a.g.seg_len) * p.heads + h) * per_bound; };
  auto load_state = [&](f32x4 (&s)[KT], const float* src, int rs, int cs) {
    if (col >= V) return;
    src += (int64_t)col * cs;
    LAPLEX_EACH(t, KT, r) {
      const int row = carry_row(t, g, r);
      const float v = src[min(row, K - 1) * rs];
      s[t][r] = row < K ? v : 0.f;
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
  const int64_t t0 = token(sg.u0);
  if constexpr (FULL) sx.init(x + t0 * p.x.token, p.x.token, step, 0);
  sy.init(y + t0 * p.y.token, p.y.token, step, 0);
  sz.init(z + t0 * p.z.token, p.z.token, step, slice * BV);
  if constexpr (DOT) sd.init(dot + t0 * p.dot_view.token, p.dot_view.token, step, slice * BV);
  auto load = [&](int rows) {
    if constexpr (FULL) sx.load(rows, K);
    sy.load(rows, K);
    sz.load(rows, V - (int)slice * BV);
    if constexpr (DOT) sd.load(rows, V - (int)slice * BV);
  };
  const int tail = __builtin_amdgcn_readfirstlane((int)((sg.n - 1) % C) + 1);  // tokens of the last chunk
  const uint32_t chunks = sg.n > 0 ? __builtin_amdgcn_readfirstlane((uint32_t)((sg.n + C - 1) / C)) : 0;  // (the last of `tail` tokens)
  if (chunks) load(chunks > 1 ? C : tail);  // on their way while the states are read and the weights formed
  f32x4 S[KT], D[RATE ? KT : 1];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    S[t] = f32x4{};
    if constexpr (RATE) D[t] = f32x4{};
  }
  if constexpr (FULL) {
    if (sg.u0 > 0) {
      const uint64_t at = bound_at(sg.u0);
      load_state(S, a.bound + at, brs, bcs);
      if constexpr (RATE) load_state(D, a.bound_d + at, V, 1);
    } else if (p.s_in) {
      load_state(S, p.s_in + sbase, rs, cs);
    }
  }

  if constexpr (FULL) {
    if constexpr (BF) {
      if (threadIdx.x <= C) dec[threadIdx.x] = decay(-rate * (float)threadIdx.x);
    } else {
      for (int i = threadIdx.x; i < 2 * C; i += THREADS) wt[i] = i >= C ? p.c_pair * decay(-rate * (float)(i - C)) : 0.f;
      if (threadIdx.x < C) up[threadIdx.x] = p.c_in * decay(-rate * (float)((int)threadIdx.x + lead));
    }
  }
  auto pair_weight = [&](int lag) {
    if constexpr (BF) return lag >= 0 ? p.c_pair * dec[lag] : 0.f;
    else return wt[C + lag];
  };
  // The carry's decay over a chunk.  As one float its rounding would add up, the same way each time, over the
  // thousands of chunks that a slow decay reaches: each chunk takes the float nearest to what brings the product
  // so far back to the exact one.
  const double wc = uniform(exp(-(double)rate * (double)C)), wtail = uniform(exp(-(double)rate * (double)tail));
  double owed = 1.0;
  auto set_down = [&](int n) {
    const int j = thread_now(), lag = n - 1 - j;
    if (j >= C) return;
    down[j] = lag >= 0 ? p.c_add * decay(-rate * (float)(lag + 1 - lead)) : 0.f;
    if constexpr (RATE) downlag[j] = lag >= 0 ? (float)lag * down[j] : 0.f;
  };

  f32x4 O[FULL ? IT : 1];
  // where the next chunk's first output row goes, and bytes to the next (64 rows of at most 4096 x 256 floats)
  const bool wide = p.out_f32 || !BF, puts = active && p.out;
  const int32_t out_pitch = (int32_t)(p.heads * V) * (wide ? 4 : 2) * step;
  char* out = static_cast<char*>(p.out) + (t0 * p.heads + h) * V * (wide ? 4 : 2);
  // Writes the outputs of a chunk of n tokens.  Called when the next chunk is in LDS: stores are counted with the
  // loads, so writing before would make the wait for the next chunk's rows one for the stores too.
  auto put = [&](int n) {
    if (!puts) return;
    const int ln = thread_now() & (kWave - 1), g = ln >> 4, lc = ln & 15, c = slice * BV + wave * 16 + 4 * g;
    if constexpr (VEC) {
      const int32_t back = min((n - 1) * out_pitch, 0), span = abs((n - 1) * out_pitch), size = wide ? 4 : 2;
      const __amdgpu_buffer_rsrc_t m = rows_at(out + back, (uint32_t)(span + V * size));
      const uint32_t off = c < V ? (uint32_t)(lc * out_pitch - back + c * size) : kNowhere;
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const uint32_t at = off + (uint32_t)(16 * t * out_pitch);
        if (wide) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[t]), m, at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(O[t][0], O[t][1]), pack_bf16(O[t][2], O[t][3])}, m, at, 0, 0);
      }
    } else {
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        if (16 * t + lc >= n || c >= V) continue;
        char* to = out + (int64_t)((16 * t + lc) * out_pitch) + c * (wide ? 4 : 2);
        const int left = min(V - c, 4);
        if (wide) {
          if (left == 4) {
            __builtin_memcpy(reinterpret_cast<float*>(to), &O[t], 16);
          } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (e < left) reinterpret_cast<float*>(to)[e] = O[t][e];
          }
        } else {
          const u32x2 w = {pack_bf16(O[t][0], O[t][1]), pack_bf16(O[t][2], O[t][3])};
          if (left == 4) {
            __builtin_memcpy(reinterpret_cast<uint16_t*>(to), &w, 8);
          } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (e < left) reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(w[e / 2] >> 16 * (e % 2));
          }
        }
      }
    }
    out += (int64_t)(C * out_pitch);
  };
  double dr = 0.0;
  if (threadIdx.x < 2) bad_chunk[threadIdx.x] = 0;
  if constexpr (FULL)
    for (int i = threadIdx.x; i < 2 * BV / 4; i += THREADS) bad_row[i / (BV / 4)][i % (BV / 4)] = kNoRow;
  __syncthreads();
  // the loaded rows of a chunk into LDS, z and dot into buffer `to`
  auto fill = [&](int to) {
    if constexpr (FULL) sx.store(xs);
    sy.store(ys);
    // A masked pair weighs 0, but 0 times an infinity is NaN: infinities and NaN in z are taken out of the
    // tile, and what they reach -- their own and later tokens of their column, the carry -- is set to NaN below.
    if (FULL && sz.clean(bad_row[to])) bad_chunk[to] = 1;
    sz.store(zs[FULL ? to : 0]);
    if constexpr (DOT) sd.store(dots[to]);
  };
  if (chunks) {
    fill(0);
    set_down(chunks > 1 ? C : tail);
  }
  __syncthreads();
  // Two barriers a chunk: between the first and the second the next chunk's rows go to LDS beside the products
  // of the pairs, which are all that is left of this one (z has two buffers).
  int now = 0;
  for (uint32_t left = chunks; left; --left, now ^= 1) {
    const int n = left > 1 ? C : tail;
    const bool more = left > 1;
    if (more) load(left > 2 ? C : tail);
    if (FULL && left < chunks) put(C);
    const bool bad = FULL && bad_chunk[now] != 0;
    const int tid = thread_now(), ln = tid & (kWave - 1);
    if (tid == 0) bad_chunk[now ^ 1] = 0;
    if (FULL && tid < BV / 4) bad_row[now ^ 1][tid] = kNoRow;
    const int g = ln >> 4, lc = ln & 15;

    // byte offsets of this lane's operands
    const uint32_t row_at = row_operand<T, KP>(ln);
    const uint32_t y_at = BF ? tr_operand<KP>(ln, 4 * (ln & 3)) : tile_at<float, KP>(4 * g, lc) * 4;
    const uint32_t z_at = BF ? tr_operand<BV>(ln, wave * 16 % 32 + 4 * (ln & 3)) ^ (wave / 2 << 6) : 0;

    f32x4 OD[DOT ? IT : 1];
    if constexpr (FULL) {
      // The weighted pairs are the same for every column: the waves share them out and pass them on through LDS.
      if constexpr (BF) {
        // the ten 16 x 16 tiles of P^T (rows j, columns i) on and below the diagonal, as operands of three bfloat16 parts
        for (int tile = wave; tile < IT * (IT + 1) / 2; tile += NW) {
          const int it = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, jt = tile - it * (it + 1) / 2;
          f32x4 P = {};
          bf16x8 f[2][2];
          auto read = [&](int ks) {
            f[ks & 1][0] = read_row(ys + 16 * jt * KP, row_at ^ (ks << 6));
            f[ks & 1][1] = read_row(xs + 16 * it * KP, row_at ^ (ks << 6));
          };
          read(0);
#pragma unroll
          for (int ks = 0; ks < KP / 32; ++ks) {
            if (ks + 1 < KP / 32) read(ks + 1);
            __builtin_amdgcn_sched_barrier(0);
            P = mfma(f[ks & 1][0], f[ks & 1][1], P);
          }
          const int lag0 = 16 * (it - jt) + lc - 4 * g;
          float pv[4], pd[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = pair_weight(lag0 - r);
            pv[r] = w != 0.f ? P[r] * w : 0.f;  // a masked pair is 0 whatever its product
            if constexpr (RATE) pd[r] = pv[r] * (float)(lag0 - r);
          }
          auto put_pair = [&](float (&v)[4], int base) {
            const bool half = jt == it && !(it & 1);
            uint2* dst = pairs + base + pair_at(it, jt >> 1) + (half ? ln : 2 * ln + (jt & 1));
            const int part = half ? kWave : 2 * kWave;
            uint32_t w0 = split_pair(v[0], v[1]), w1 = split_pair(v[2], v[3]);
            dst[0] = make_uint2(w0, w1);
            w0 = split_pair(v[0], v[1]), w1 = split_pair(v[2], v[3]);
            dst[part] = make_uint2(w0, w1);
            dst[2 * part] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          };
          put_pair(pv, 0);
          if constexpr (RATE) put_pair(pd, PAIRS);
        }
      } else if (wave < WK) {
        // each of WK waves adds a share of the channels of the tiles (0, 0), (0, 1), (1, 1)
        f32x4 P[3] = {};
#pragma unroll
        for (int k = 0; k < KP / WK / 16; ++k) {
          const uint32_t at = row_at ^ ((wave * (KP / WK / 16) + k) << 6);
          f32x4 xf[2], yf[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            xf[t] = lds_at<f32x4>(xs + 16 * t * KP, at);
            yf[t] = lds_at<f32x4>(ys + 16 * t * KP, at);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            P[0] = mfma(yf[0][e], xf[0][e], P[0]);
            P[1] = mfma(yf[0][e], xf[1][e], P[1]);
            P[2] = mfma(yf[1][e], xf[1][e], P[2]);
          }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) reinterpret_cast<f32x4*>(pairs)[(wave * 3 + i) * kWave + ln] = P[i];
      }
      if (active) {
        // out^T = S^T x^T (rows V, columns i)
        if constexpr (BF) {
          constexpr int STEPS = KP / 32 * IT;
          bf16x8 xf[2];
          auto read = [&](int i) { xf[i & 1] = read_row(xs + 16 * (i % IT) * KP, row_at ^ (i / IT << 6)); };
          Parts sp, dp;
          read(0);
#pragma unroll
          for (int i = 0; i < STEPS; ++i) {
            const int ks = i / IT, t = i % IT;
            if (i + 1 < STEPS) read(i + 1);
            __builtin_amdgcn_sched_barrier(0);
            if (t == 0) {
              sp = split(S[2 * ks], S[2 * ks + 1]);
              if constexpr (RATE) dp = split(D[2 * ks], D[2 * ks + 1]);
            }
            auto add = [&](f32x4& o, const Parts& c) {
              o = mfma(c.hi, xf[i & 1], ks ? o : f32x4{});
              o = mfma(c.lo, xf[i & 1], o);
              o = mfma(c.lo2, xf[i & 1], o);
            };
            add(O[t], sp);
            if constexpr (RATE) add(OD[t], dp);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int t = 0; t < IT; ++t) {
              const f32x4 xf = lds_at<f32x4>(xs + 16 * t * KP, row_at ^ (k << 6));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                O[t] = mfma(S[k][e], xf[e], k + e ? O[t] : f32x4{});
                if constexpr (RATE) OD[t] = mfma(D[k][e], xf[e], k + e ? OD[t] : f32x4{});
              }
            }
        }
#pragma unroll
        for (int t = 0; t < IT; ++t) {
          const float f = BF ? p.c_in * dec[16 * t + lc + lead] : up[16 * t + lc];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (RATE) OD[t][r] = f * fmaf((float)(16 * t + lc + lead), O[t][r], OD[t][r]);
            O[t][r] *= f;
          }
        }
      }
    }
    // the carry over the chunk
    const T* z = zs[FULL ? now : 0];
    if (active && (!FULL || more || keep)) {
      const double exact = uniform((more ? wc : wtail) * owed);
      const float w = (float)exact;
      // (a subnormal w has no reciprocal, and nothing that a later chunk could show)
      owed = __builtin_amdgcn_readfirstlane(__float_as_uint(w)) >= 0x00800000u ? 1.0 + (double)((float)(exact - (double)w) * __builtin_amdgcn_rcpf(w)) : 1.0;
      LAPLEX_EACH(t, KT, r) {
        if constexpr (RATE) D[t][r] = w * fmaf((float)n, S[t][r], D[t][r]);  // the lag-weighted carry ahead of the other
        S[t][r] *= w;
      }
      if constexpr (BF) {
        constexpr int STEPS = C / 32 * KT;
        bf16x8 zf, yt[2];
        auto read = [&](int i) {
          const int t = i % KT;
          yt[i & 1] = read_tr<KP>(ys + 32 * (i / KT) * KP, y_at ^ (t >> 1 << 6 | (t & 1) << 5));
          if (t == 0) zf = read_tr<BV>(z + 32 * (i / KT) * BV, z_at);
        };
        read(0);
        Parts zp, lp;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const int s = i / KT, t = i % KT;
          if (i + 1 < STEPS) read(i + 1);
          __builtin_amdgcn_sched_barrier(0);
          if (t == 0) {
            // z weighted by its decay to the chunk's end
            auto weighted = [&](const float* w, f32x4& lo, f32x4& hi) {
              lo = *reinterpret_cast<const f32x4*>(w + 32 * s + 4 * g);
              hi = *reinterpret_cast<const f32x4*>(w + 32 * s + 16 + 4 * g);
#pragma unroll
              for (int e = 0; e < 4; ++e) lo[e] *= (float)zf[e], hi[e] *= (float)zf[4 + e];
            };
            f32x4 z0, z1;
            weighted(down, z0, z1);
            zp = split(z0, z1);
            if constexpr (RATE) {
              weighted(downlag, z0, z1);
              lp = split(z0, z1);
            }
          }
          auto add = [&](f32x4& s, const Parts& p) {
            s = mfma(yt[i & 1], p.hi, s);
            s = mfma(yt[i & 1], p.lo, s);
            s = mfma(yt[i & 1], p.lo2, s);
          };
          add(S[t], zp);
          if constexpr (RATE) add(D[t], lp);
        }
      } else {
        f32x4 zw[C / 16], zl[C / 16];
#pragma unroll
        for (int s = 0; s < C / 16; ++s) {
          f32x4 zf;
#pragma unroll
          for (int r = 0; r < 4; ++r) zf[r] = z[tile_at<T, BV>(16 * s + 4 * g + r, wave * 16 + lc)];
          if constexpr (RATE) zl[s] = zf * *reinterpret_cast<const f32x4*>(downlag + 16 * s + 4 * g);
          zw[s] = zf * *reinterpret_cast<const f32x4*>(down + 16 * s + 4 * g);
        }
        LAPLEX_EACH(s, C / 16, r) {
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const float yt = lds_at<float>(ys + (16 * s + r) * KP, y_at ^ (t << 6 | r << 4));
            S[t] = mfma(yt, zw[s][r], S[t]);
            if constexpr (RATE) D[t] = mfma(yt, zl[s][r], D[t]);
          }
        }
      }
      if (bad && row_byte(bad_row[now], wave * 16 + lc) < C) {
        LAPLEX_EACH(t, KT, r) {
          S[t][r] = __builtin_nanf("");
          if constexpr (RATE) D[t][r] = __builtin_nanf("");
        }
      }
    }
    __syncthreads();  // every wave's share of the pairs is there, and x and y are read
    if (more) {
      fill(now ^ 1);
      if (left == 2 && tail != C) set_down(tail);
    }
    if (FULL && active) {
      // out^T += z^T P
      if constexpr (BF) {
#pragma unroll
        for (int s = 0; s < C / 32; ++s) {
          const bf16x8 zf = read_tr<BV>(z + 32 * s * BV, z_at);
#pragma unroll
          for (int t = 2 * s; t < IT; ++t) {
            auto add = [&](f32x4& o, int base) {
              const uint2* from = pairs + base + pair_at(t, s);
#pragma unroll
              for (int part = 0; part < 3; ++part) {
                bf16x8 w;
                if (t == 2 * s) {  // (the other 16 rows lie above the diagonal)
                  const uint2 half = from[part * kWave + ln];
                  w = __builtin_bit_cast(bf16x8, make_uint4(half.x, half.y, 0, 0));
                } else {
                  w = __builtin_bit_cast(bf16x8, reinterpret_cast<const uint4*>(from)[part * kWave + ln]);
                }
                o = mfma(zf, w, o);
              }
            };
            add(O[t], 0);
            if constexpr (RATE) add(OD[t], PAIRS);
          }
        }
      } else {
        f32x4 P[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const f32x4* parts = reinterpret_cast<const f32x4*>(pairs) + i * kWave + ln;
          P[i] = parts[0];
#pragma unroll
          for (int k = 1; k < WK; ++k) P[i] += parts[k * 3 * kWave];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = pair_weight((i == 1 ? 16 : 0) + lc - 4 * g - r);
            P[i][r] = w != 0.f ? P[i][r] * w : 0.f;  // a masked pair is 0 whatever its product
          }
        }
        LAPLEX_EACH(s, C / 16, r) {
          const float zf = z[tile_at<T, BV>(16 * s + 4 * g + r, wave * 16 + lc)];
#pragma unroll
          for (int t = s; t < IT; ++t) {
            O[t] = mfma(zf, P[s + t][r], O[t]);
            if constexpr (RATE) OD[t] = mfma(zf, P[s + t][r] * (float)(16 * (t - s) + lc - 4 * g - r), OD[t]);
          }
        }
      }
      if (bad) {
        LAPLEX_EACH(t, IT, r) {
          const bool hit = 16 * t + lc >= row_byte(bad_row[now], wave * 16 + 4 * g + r);
          O[t][r] = hit ? __builtin_nanf("") : O[t][r];
          if constexpr (RATE) OD[t][r] = hit ? __builtin_nanf("") : OD[t][r];
        }
      }
      if constexpr (DOT) {
        LAPLEX_EACH(t, IT, r)  // rows past the end are zero in the tile
          dr += (double)(OD[t][r] * to_f32(dots[now][tile_at<T, BV>(16 * t + lc, wave * 16 + 4 * g + r)]));
      }
    }
    __syncthreads();
  }
  if (FULL && chunks) put(tail);

  // the carry after the segment
  const int lnf = thread_now() & (kWave - 1), gf = lnf >> 4, colf = slice * BV + wave * 16 + (lnf & 15);
  auto each = [&](int rs, int cs, auto&& f) {
    if (colf >= V) return;
    LAPLEX_EACH(t, KT, r) {
      const int row = carry_row(t, gf, r);
      if (row < K) f(t, r, row * rs + colf * cs);
    }
  };
  if constexpr (!FULL) {
    const uint64_t at = bound_at(sg.u0 + sg.n);
    float* to = a.bound + at;
    each(V, 1, [&](int t, int r, int o) { to[o] = S[t][r]; });
    if constexpr (RATE) {
      float* tod = a.bound_d + at;
      each(V, 1, [&](int t, int r, int o) { tod[o] = D[t][r]; });
    }
  } else if (last_seg) {
    if (p.s_out) {
      float* to = p.s_out + sbase;
      each(rs, cs, [&](int t, int r, int o) { to[o] = S[t][r]; });
    }
    if constexpr (RATE)
      if (p.ds_out) {
        const float* gd = p.ds_out + sbase;
        each(rs, cs, [&](int t, int r, int o) { dr += (double)(D[t][r] * gd[o]); });
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

// kp: K rounded up to 64, 128 or 256; nw: waves per block, 16 columns each (8, or 4 where V is at most 64 or blocks are few)
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
  if (kp == 64 && nw == 4) attn_chunk_launch_at<T, 64, 4, VEC>(a, full, rate, s);
  else if (kp == 64) attn_chunk_launch_at<T, 64, 8, VEC>(a, full, rate, s);
  else if (kp == 128 && nw == 4) attn_chunk_launch_at<T, 128, 4, VEC>(a, full, rate, s);
  else if (kp == 128) attn_chunk_launch_at<T, 128, 8, VEC>(a, full, rate, s);
  else attn_chunk_launch_at<T, 256, 8, VEC>(a, full, rate, s);
}

// The instantiations, each in a source file of its own.  vec: every row of x, y, z, dot and out is 16-byte aligned.
void attn_chunk_bf16_vec(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);
void attn_chunk_bf16_any(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);
void attn_chunk_f32_vec(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);
void attn_chunk_f32_any(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s);

}  // namespace laplex
