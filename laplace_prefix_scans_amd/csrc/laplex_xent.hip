// Softmax cross entropy of rows against a linear output table, forward and backward, without the logits in memory.
//
//   l_tv = c x_t . W_v,  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_{t y_t},
//   G_tv = c [(dloss_t + dlse_t) exp(l_tv - lse_t) - dloss_t [v = y_t]],  dx = G W,  dW = G^T x.
//
// Four matrix products (the logits twice), all of one kernel: C[n][m] = sum_k A[m][k] B[n][k] on the matrix cores, A and B
// each contiguous along k or along their rows.  What follows the product is fused: the forward keeps a maximum and a sum
// of exponentials per token and tile of the vocabulary, the backward writes a tile of G.  Tensors are read as they lie; rows
// that are not whole 128-byte pieces are filled up with zeros first, and the backward takes a copy of x in which the
// tokens that take no part are zeros.
#include <algorithm>
#include <type_traits>

#include "laplex_host.hpp"
#include "laplex_layers_device.hpp"
#include "laplex_train.hpp"

namespace laplex {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

template <typename T>
struct Frag;
template <>
struct Frag<bf16> {
  using V = bf16x8;
  static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <>
struct Frag<float> {
  using V = f32x4;
  // (which k of the 16 a lane's four values have does not matter, as A and B agree)
  static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

enum { XENT_STATS, XENT_GRAD, XENT_OUT };

struct ProductArgs {
  const void *A, *B;
  int64_t lda, ldb;  // elements; rows are whole 128-byte pieces (zeros beyond their end)
  uint32_t M, N;     // C's
  uint64_t K;        // a multiple of a step's
  uint64_t k_rows;   // rows that A has where it lies along M; those up to K count as its last one (B's are zeros there)
  uint32_t tiles_m, tiles_n, splits;
  uint64_t k_split;  // k of a split, the same multiple
  // XENT_STATS, XENT_GRAD: rows of A are vocabulary entries from v0 on, rows of B tokens
  const void* targets;
  int id_bytes;
  uint32_t vocab, v0;
  float scale;
  float2* stats;     // [tile of M][token]: maximum, sum of exp(l - maximum)
  float* hit;        // [token]: the target's logit
  const float *lse, *dloss, *dlse;
  void* G;           // [token][ldg]
  int64_t ldg;
  int64_t rest;      // bytes from G (XENT_OUT: B) to a second part of it, what its rounding left out; 0: there is none
  uint32_t n_fill, m_fill;  // rows and columns that are written, zeros from N and M on
  // XENT_OUT
  void* out;         // [N][ldo], of type out_f32 ? float : T; splits of out_f32 follow each other
  int64_t ldo, out_split;
  bool out_f32, add;
  bool live_rows;    // rows of tokens whose target is outside the vocabulary are zero
};

__device__ __forceinline__ int64_t target_of(const void* ids, int bytes, uint32_t t) {
  return bytes == 8 ? static_cast<const int64_t*>(ids)[t] : (int64_t) static_cast<const int32_t*>(ids)[t];
}
__device__ __forceinline__ bool live(const ProductArgs& a, uint32_t t) {
  const int64_t y = target_of(a.targets, a.id_bytes, t);
  return y >= 0 && y < (int64_t)a.vocab;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
// exp(l - m) with 1 where both are the same infinity
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.f : exp_of(l - m); }

// Tile and split number `id`: groups of 8 tiles of M by all of N, of which the ones that run at once share rows of both
// factors in an XCD's L2.
__device__ __forceinline__ void tile_of(const ProductArgs& a, uint32_t id, uint32_t& tm, uint32_t& tn, uint32_t& split) {
  constexpr uint32_t GROUP = 8;
  const uint32_t total = a.tiles_m * a.tiles_n;
  split = id / total;
  id %= total;
  const uint32_t group = id / (GROUP * a.tiles_n), first = group * GROUP, rows = min(GROUP, a.tiles_m - first);
  const uint32_t in = id - first * a.tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// ------------------------------------------------------------------ the product
// A block of WM x WN waves makes BM x BN of C, and then of other tiles, whose first bytes are on their way while it finishes
// one.  128 bytes of k of its rows are on their way from memory straight to LDS
// while those before are multiplied; a row's eight 16-byte pieces lie at piece ^ (row & 7), so that the reads of 16
// rows' pieces spread over the banks.  A step's 128 bytes are two halves, and a half's operands are read one half ahead of
// their products, across the step's one barrier: it stands in the middle of a step, where both halves of it have been read
// and the next one's bytes have arrived.  (16384 tokens, 65536 x 2048 in bfloat16, forward and backward: 13.6 to 13.7 ms by card,
// 1290 TFLOP/s; forward of 2043 tokens 383 to 425 us by card and clock, the matrix cores busy in 0.7 of the cycles.  Four steps in LDS instead of two for
// the 64 x 32 tiles: 4096 tokens, 257 x 513 in float 91 us instead of 88.)
template <int M, int N, int WAVES_M, int WAVES_N, int BLOCKS>
struct Tile {
  static constexpr int PER_CU = BLOCKS;  // that fit a CU at once
  static constexpr int BM = M, BN = N, WM = WAVES_M, WN = WAVES_N, THREADS = WM * WN * kWave;
  static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  static constexpr int LOADS = (BM + BN) / 8 / (WM * WN);  // of a wave and step: 8 rows each
  static constexpr int STEP_BYTES = (BM + BN) * 128;
  static_assert((BM + BN) % (8 * WM * WN) == 0 && BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "whole operands");
};
using TileL = Tile<256, 256, 2, 4, 1>;
using TileM = Tile<128, 128, 2, 2, 2>;
using TileS = Tile<64, 64, 2, 2, 4>;
using TileT = Tile<64, 32, 2, 2, 6>;

// 16 bytes of each lane, from `off` bytes past a base that the wave shares, to 16 lane past an LDS address that it shares.
// (Written out, for with the builtin the compiler waits for these loads before every transposing read of LDS.  They give
// no register a value; what they bring is waited for by arrived().  Nothing else here uses m0.)
__device__ __forceinline__ void to_lds(uint64_t base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(lds), "v"(off), "s"(base) : "memory");
}
// 4 bytes of each lane, to 4 lane past the LDS address
__device__ __forceinline__ void word_to_lds(uint64_t base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" : : "s"(lds), "v"(off), "s"(base) : "memory");
}
// Two addresses that the wave shares, in scalar registers; the wait states that a load has to keep from the vector
// instructions that write them are here, once for all the loads that follow.
__device__ __forceinline__ void share(const char* p, const char* q, uint64_t& a, uint64_t& b) {
  const uint64_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  // (the builtin returns a signed word)
  const auto word = [](uint64_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v); };
  a = (uint64_t)word(x >> 32) << 32 | word(x);
  b = (uint64_t)word(y >> 32) << 32 | word(y);
  asm volatile("s_nop 4" : "+s"(a), "+s"(b));
}
// (the address of LDS leaves the compiler's sight here, so that it takes to_lds to write there)
__device__ __forceinline__ uint32_t lds_address(char* p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)p));
}

// The thread's number, as something the compiler takes to change with every call: what is made from it is
// then formed where it is used instead of holding a register over the loop.
__device__ __forceinline__ int thread_now() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}
// Every wave's reads of LDS are done, and its bytes on their way to LDS are there.
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The same for LDS alone.
__device__ __forceinline__ void written() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

constexpr int kPieceK = 128;

// One factor's rows of a step in LDS, R0 of them (of M or N).
// Along k: row r is 128 bytes, its eight 16-byte pieces at piece ^ (r & 7), so that reads of 16 rows' pieces spread over
// the banks.  Along its rows (ALONG): row k of the step is R0 elements, in blocks of 16 at block ^ mix(k), so that the
// operand reads, which go across the rows, do.  A lane's operand of a half is the same elements either way: row lane % 16 and
// k = 8 (lane / 16) .. + 7 of 32 (bfloat16; across rows by the transposing read, which gives each of 16 lanes one of
// 16 columns of four rows) or 4 (lane / 16) .. + 3 of 16 (float).
template <typename T, int R0, bool ALONG>
struct Factor {
  static constexpr int ROW = R0 * (int)sizeof(T), BLOCK = 16 * (int)sizeof(T), BLOCKS = R0 / 16;
  static constexpr int READS = !ALONG ? 1 : sizeof(T) == 2 ? 2 : 4;  // of an operand
  static __device__ __forceinline__ int mix(int k) {
    const int m = sizeof(T) == 2 ? (k & 3) | (k >> 3 & 1) << 2 : k >> 2 & 3;
    return m & (BLOCKS - 1);
  }
  // where the 16 bytes at `at` of a step (a multiple of 16) come from: offset of row and column, in elements
  static __device__ __forceinline__ void source(int at, int& row, int& col) {
    constexpr int E = 16 / sizeof(T);
    if constexpr (ALONG) {
      row = at / ROW;
      const int block = at % ROW / BLOCK ^ mix(row);
      col = block * 16 + at % BLOCK / 16 * E;
    } else {
      row = at / kPieceK;
      col = (at % kPieceK / 16 ^ (row & 7)) * E;
    }
  }
  // the lane's first byte of operand 0 (rows r0 .. r0 + 15) of half 0
  static __device__ __forceinline__ uint32_t first(int r0, int lane) {
    if constexpr (!ALONG) return (r0 + lane % 16) * kPieceK + ((lane / 16) ^ (lane & 7)) * 16;
    const int k = sizeof(T) == 2 ? 8 * (lane / 16) + (lane >> 2 & 3) : 4 * (lane / 16);
    return k * ROW + ((r0 / 16) ^ mix(k)) * BLOCK + (sizeof(T) == 2 ? (lane & 3) * 8 : lane % 16 * 4);
  }
  // operand i of a half (r0 a multiple of the operands' rows, so that i only flips bits of the block)
  static __device__ __forceinline__ typename Frag<T>::V read(const char* step, uint32_t first, int half, int i) {
    using V = typename Frag<T>::V;
    if constexpr (!ALONG) {
      return *reinterpret_cast<const V*>(step + (first ^ half * 64) + i * 16 * kPieceK);
    } else if constexpr (sizeof(T) == 2) {
      const char* p = step + (first ^ i * BLOCK) + half * 32 * ROW;
      struct { s16x4 a, b; } v = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p), __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 4 * ROW))};
      return __builtin_bit_cast(V, v);
    } else {
      const char* p = step + (first ^ i * BLOCK) + half * 16 * ROW;
      V v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float*>(p + j * ROW);
      return v;
    }
  }
};

// What the logits' products need of each token of a tile, in LDS: words of the target, lse, dloss, dlse.
enum { INFO_LOW, INFO_HIGH, INFO_LSE, INFO_DLOSS, INFO_DLSE, INFO_WORDS };

// A_ALONG: A is [k][M]; B_ALONG: B is [k][N]
template <typename T, int EPI, typename C, bool A_ALONG, bool B_ALONG>
__global__ __launch_bounds__(C::THREADS) void k_product(ProductArgs a) {
  constexpr int BM = C::BM, BN = C::BN, MI = C::MI, NI = C::NI, W = C::WM * C::WN, BK = kPieceK / sizeof(T), E = 16 / sizeof(T);
  constexpr int INFO = EPI == XENT_OUT ? 0 : EPI == XENT_STATS ? INFO_LSE : INFO_WORDS;
  using FA = Factor<T, BM, A_ALONG>;
  using FB = Factor<T, BN, B_ALONG>;
  __shared__ __attribute__((aligned(16))) char lds[2 * C::STEP_BYTES];
  __shared__ uint32_t info[INFO ? INFO : 1][INFO ? (BN + 63) / 64 * 64 : 1];
  __shared__ float2 part[EPI == XENT_STATS ? C::WM : 1][EPI == XENT_STATS ? BN : 1];
  using V = typename Frag<T>::V;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  // Blocks are dispatched to the 8 XCDs in turn; each XCD's blocks take a stretch of the tiles, one after the other.
  const uint32_t all = a.tiles_m * a.tiles_n * a.splits, xcd = blockIdx.x % kXcds, rest = all % kXcds;
  const uint32_t next_id = gridDim.x / kXcds + (xcd < gridDim.x % kXcds), end = (xcd + 1) * (all / kXcds) + min(xcd + 1, rest);
  uint32_t id = xcd * (all / kXcds) + min(xcd, rest) + blockIdx.x / kXcds;

  // this lane's 16 bytes of each of the wave's stretches of 1024, from the tile's first element on; LOADS_A of them are A's
  constexpr int LOADS_A = BM / 8 / W;
  static_assert(BM % (8 * W) == 0, "a wave's stretches are A's and then B's");
  const int64_t row_a = a.lda * (int64_t)sizeof(T), row_b = a.ldb * (int64_t)sizeof(T);
  const int64_t next_a = A_ALONG ? row_a * BK : kPieceK, next_b = B_ALONG ? row_b * BK : kPieceK;
  const uint32_t to0 = lds_address(lds) + wave * 1024;
  uint32_t off[C::LOADS], tm, tn, split;
  const char *base_a, *base_b;
  uint64_t k0;
  int steps, turn, first = 0;  // steps of one part of B; the buffer of step 0
  const auto choose = [&] {
    tile_of(a, id, tm, tn, split);
    k0 = split * a.k_split;
    steps = (int)((min(a.K, k0 + a.k_split) - k0) / BK);
    if (EPI == XENT_OUT) {
      turn = steps;
      if (a.rest) steps *= 2;
    }
    base_a = static_cast<const char*>(a.A) + (A_ALONG ? (int64_t)k0 * row_a + (int64_t)tm * BM * sizeof(T) : (int64_t)tm * BM * row_a + (int64_t)k0 * sizeof(T));
    base_b = static_cast<const char*>(a.B) + (B_ALONG ? (int64_t)k0 * row_b + (int64_t)tn * BN * sizeof(T) : (int64_t)tn * BN * row_b + (int64_t)k0 * sizeof(T));
#pragma unroll
    for (int i = 0; i < C::LOADS; ++i) {
      const int at = (i * W + wave) * 1024 + thread_now() % kWave * 16;
      int row, col;
      if (i < LOADS_A) {
        FA::source(at, row, col);
        if (A_ALONG) col = min((int64_t)col, a.lda - E - (int64_t)tm * BM);
        else row = min((uint32_t)row, a.M - 1 - tm * BM);
        off[i] = (uint32_t)row * (uint32_t)row_a + (uint32_t)col * (uint32_t)sizeof(T);
      } else {
        FB::source(at - BM * kPieceK, row, col);
        if (B_ALONG) col = min((int64_t)col, a.ldb - E - (int64_t)tn * BN);
        else row = min((uint32_t)row, max(a.N, tn * BN + 1) - 1 - tn * BN);
        off[i] = (uint32_t)row * (uint32_t)row_b + (uint32_t)col * (uint32_t)sizeof(T);
      }
    }
  };
  auto load = [&](int step) {
    const uint32_t to = to0 + ((first + step) & 1) * C::STEP_BYTES;
    const char* from_b = base_b;
    if (EPI == XENT_OUT && step >= turn) {  // B's second part, by the same rows of A
      step -= turn;
      from_b += a.rest;
    }
    uint64_t p, q;
    share(base_a + step * next_a, from_b + step * next_b, p, q);
    if (A_ALONG && k0 + (uint64_t)(step + 1) * BK > a.k_rows) {  // the last step has rows beyond the last: that one again
      const int rows = (int)((int64_t)a.k_rows - (int64_t)(k0 + (uint64_t)step * BK));
#pragma unroll
      for (int i = 0; i < LOADS_A; ++i) {
        int row, col;
        FA::source((i * W + wave) * 1024 + thread_now() % kWave * 16, row, col);
        to_lds(p, off[i] - (uint32_t)max(row - (rows - 1), 0) * (uint32_t)row_a, to + i * W * 1024);
      }
    } else {
#pragma unroll
      for (int i = 0; i < LOADS_A; ++i) to_lds(p, off[i], to + i * W * 1024);
    }
#pragma unroll
    for (int i = LOADS_A; i < C::LOADS; ++i) to_lds(q, off[i], to + i * W * 1024);
  };
  // the tile's tokens' words, an array a wave
  const auto load_info = [&] {
#pragma unroll
    for (int w = 0; w < INFO; ++w) {
      if (wave != w % W || (w == INFO_HIGH && a.id_bytes == 4) || (w == INFO_DLSE && !a.dlse)) continue;
      const char* p = w <= INFO_HIGH ? static_cast<const char*>(a.targets) + w * 4 : reinterpret_cast<const char*>(w == INFO_LSE ? a.lse : w == INFO_DLOSS ? a.dloss : a.dlse);
      const uint32_t pitch = w <= INFO_HIGH ? a.id_bytes : 4, to = lds_address(reinterpret_cast<char*>(info[w]));
      uint64_t base, none;
      share(p, p, base, none);
#pragma unroll
      for (int i = 0; i < (BN + 63) / 64; ++i) word_to_lds(base, min(tn * BN + i * kWave + lane, a.N - 1) * pitch, to + i * 256);
    }
  };
  const int wm = wave % C::WM * (BM / C::WM), wn = wave / C::WM * (BN / C::WN);
  const uint32_t at_a = FA::first(wm, lane), at_b = FB::first(wn, lane);
  if (id >= end) return;
  choose();
  if (steps > 0) load(0);
  if (steps > 1) load(1);
  for (;;) {
    f32x4 acc[MI][NI] = {};
    if (steps > 0) {
      V fa[2][MI], fb[2][NI];
      auto read = [&](int step, int half) {
        const char* base = lds + ((first + step) & 1) * C::STEP_BYTES;
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[half][j] = FB::read(base + BM * kPieceK, at_b, half, j);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[half][i] = FA::read(base, at_a, half, i);
      };
      auto multiply = [&](int half) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NI; ++j) acc[i][j] = Frag<T>::mul(fa[half][i], fb[half][j], acc[i][j]);
        // a read after every few products
        constexpr int READS = MI * FA::READS + NI * FB::READS, PRODUCTS = MI * NI * (sizeof(T) == 4 ? 4 : 1);
#pragma unroll
        for (int r = 0; r < READS; ++r) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x8, PRODUCTS / READS ? PRODUCTS / READS : 1, 0);
        }
      };
      arrived();
      if (INFO) load_info();  // (every wave is past the tile before; it is there after the next arrived())
      read(0, 0);
      for (int k = 0; k < steps; ++k) {
        read(k, 1);
        multiply(0);
        arrived();
        if (k + 2 < steps) load(k + 2);
        read(k + 1, 0);  // (after the last step: bytes that nothing uses)
        multiply(1);
      }
    }
    // the next tile's first bytes: every wave has read all it will of this one's
    const uint32_t m_tile = tm * BM, n_tile = tn * BN, this_split = split;
    id += next_id;
    const bool more = id < end;
    if (more) {
      first = (first + steps) & 1;
      choose();
      if (steps > 0) load(0);
      if (steps > 1) load(1);
    }
    // a lane holds column n = lane % 16 and rows m = lane / 16 * 4 .. + 3 of each 16 x 16 tile
    const uint32_t m0 = m_tile + wm + lane / 16 * 4, n0 = n_tile + wn + lane % 16;
    const bool whole = m_tile + BM <= a.M;
    if constexpr (EPI != XENT_OUT) {
      // which of the wave's rows is the token's target, in this lane: the element's number, or -1
      const auto target = [&](int j, bool& in) {
        const int c = wn + j * 16 + lane % 16;
        const int64_t y = a.id_bytes == 4 ? (int64_t)(int32_t)info[INFO_LOW][c] : (int64_t)((uint64_t)info[INFO_HIGH][c] << 32 | info[INFO_LOW][c]);
        in = n_tile + c < a.N && y >= 0 && y < (int64_t)a.vocab;
        const int64_t at = y - a.v0 - (m_tile + wm);
        return in && at >= 0 && at < BM / C::WM && (at >> 2 & 3) == lane / 16 ? (int)((at >> 4) * 4 + (at & 3)) : -1;
      };
      if constexpr (EPI == XENT_STATS) {
        // Maxima and sums of exp(l - max), l = scale acc: an element takes a maximum, a product and sum, an exponential of
        // base 2 and a sum.
        float scale = a.scale;
        const auto all_of = [&](auto f) {
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[i][j][r] = f(acc[i][j][r], m0 + i * 16 + r);
        };
        if (scale < 0.f) {
          scale = -scale;
          all_of([](float x, uint32_t) { return -x; });
        }
        if (scale == 0.f) {
          scale = 1.f;
          all_of([](float x, uint32_t) { return 0.f * x; });
        }
        if (!whole) all_of([&](float x, uint32_t v) { return v < a.M ? x : -INFINITY; });
        const float s2 = scale * kLog2e;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          bool in;
          const int hit = target(j, in);
          if (__any(hit >= 0)) {
            float l = 0.f;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int r = 0; r < 4; ++r) l = hit == i * 4 + r ? acc[i][j][r] : l;
            if (hit >= 0) a.hit[n0 + j * 16] = scale * l;
          }
          float most = -INFINITY, sum = 0.f;
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) most = fmaxf(most, acc[i][j][r]);
          most = fmaxf(most, __shfl_xor(most, 16));
          most = fmaxf(most, __shfl_xor(most, 32));
          const float m2 = most * s2;
          const bool odd = !(fabsf(m2) < 0x1p18f);  // (m2's rounding is that of the maximum in the result, but for this in the exponents)
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], s2, -m2));
          if (__any(odd)) {
            float again = 0.f;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int r = 0; r < 4; ++r) again += exp_below(acc[i][j][r] * scale, most * scale);
            sum = odd ? again : sum;
          }
          sum += __shfl_xor(sum, 16);
          sum += __shfl_xor(sum, 32);
          if (lane < 16) part[wave % C::WM][wn + j * 16 + lane] = make_float2(most * scale, sum);
        }
        written();
        if (threadIdx.x < BN && n_tile + threadIdx.x < a.N) {
          float m = part[0][threadIdx.x].x, sum = 0.f;
#pragma unroll
          for (int w = 1; w < C::WM; ++w) m = fmaxf(m, part[w][threadIdx.x].x);
#pragma unroll
          for (int w = 0; w < C::WM; ++w) sum += part[w][threadIdx.x].y * exp_below(part[w][threadIdx.x].x, m);
          a.stats[(uint64_t)(m_tile / BM) * a.N + n_tile + threadIdx.x] = make_float2(m, sum);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int c = wn + j * 16 + lane % 16;
          const uint32_t t = n0 + j * 16;
          bool in;
          const int hit = target(j, in);
          const float lse = __uint_as_float(info[INFO_LSE][c]), d = a.scale * __uint_as_float(info[INFO_DLOSS][c]);
          const float f = a.dlse ? d + a.scale * __uint_as_float(info[INFO_DLSE][c]) : d;
          T* row = static_cast<T*>(a.G) + (int64_t)t * a.ldg;
          const auto column = [&](auto plain) {  // without a target, inside the vocabulary
#pragma unroll
            for (int i = 0; i < MI; ++i) {
              T g[4], left[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float x = f * exp_of(fmaf(acc[i][j][r], a.scale, -lse));
                if (!decltype(plain)::value) {
                  if (hit == i * 4 + r) x -= d;
                  if (m0 + i * 16 + r >= a.M) x = 0.f;
                }
                g[r] = from_f32<T>(in ? x : 0.f);
                left[r] = from_f32<T>((in ? x : 0.f) - to_f32(g[r]));
              }
              const uint32_t v = m0 + i * 16;
              if (t < a.n_fill && (decltype(plain)::value || v < a.m_fill)) {
                __builtin_memcpy(row + v, g, sizeof g);
                if (a.rest) __builtin_memcpy(reinterpret_cast<char*>(row + v) + a.rest, left, sizeof left);
              }
            }
          };
          if (whole && !__any(hit >= 0)) column(std::true_type{});
          else column(std::false_type{});
        }
      }
    } else {
      typedef T Four __attribute__((ext_vector_type(4), aligned(sizeof(T))));
      typedef float Four32 __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const uint32_t n = n0 + j * 16;
        if (n >= a.N) continue;
        const bool zero = a.live_rows && !live(a, n);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const uint32_t m = m0 + i * 16;
          const uint64_t at = (uint64_t)n * a.ldo + m;
          f32x4 x = zero ? f32x4{} : acc[i][j];
          float* o = static_cast<float*>(a.out) + this_split * a.out_split + at;
          if (m + 4 <= a.M) {
            if (a.out_f32) {
              if (a.add) x += *reinterpret_cast<const Four32*>(o);
              *reinterpret_cast<Four32*>(o) = x;
            } else {
              Four y;
#pragma unroll
              for (int r = 0; r < 4; ++r) y[r] = from_f32<T>(x[r]);
              *reinterpret_cast<Four*>(static_cast<T*>(a.out) + at) = y;
            }
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (m + r < a.M) {
                if (a.out_f32) o[r] = a.add ? o[r] + x[r] : x[r];
                else static_cast<T*>(a.out)[at + r] = from_f32<T>(x[r]);
              }
          }
        }
      }
    }
    if (!more) return;
  }
}

// ------------------------------------------------------------------ few tokens
// The statistics where the table's bytes are all that counts: at most 4 tokens, whose rows lie in LDS.  A wave takes four
// rows of the table at a time as they lie, 1024 bytes a load, and a block joins its waves' maxima and sums.  Up to 2 tokens
// where a product reads rows as they lie too (65536 x 2048 in bfloat16, 1 token: 57 us, by a product's tiles 67; 2000 x 1024, 2 tokens:
// 9.5 and 10.0, 3: 12.8 and 10.1), up to 4 where it would have to copy them (15167 x 442 in float, 4 tokens: 15 and 26 us, 8: 33 and 27).
constexpr int kFewTokens = 4, kFewTokensWhole = 2, kFewRows = 4;
constexpr uint32_t kFewBytes = 128 << 10;  // of tokens in LDS
template <typename T, int N>
__global__ __launch_bounds__(256) void k_xent_few(ProductArgs a, uint32_t width, uint32_t fill) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ __attribute__((aligned(16))) char shared[];
  T* const x = reinterpret_cast<T*>(shared);  // [N][fill], zeros from `width` on
  __shared__ float2 part[4][N];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  for (uint32_t i = threadIdx.x; i < N * fill; i += 256) {
    const uint32_t n = i / fill, c = i % fill;
    x[i] = c < width && n < a.N ? static_cast<const T*>(a.B)[(uint64_t)n * width + c] : T(0.f);
  }
  __syncthreads();
  int64_t y[N];
  float most[N], sum[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    y[n] = (uint32_t)n < a.N ? target_of(a.targets, a.id_bytes, n) : -1;
    most[n] = -INFINITY;
    sum[n] = 0.f;
  }
  const uint32_t stride = gridDim.x * 4 * kFewRows;
  for (uint64_t v0 = (blockIdx.x * 4 + wave) * kFewRows; v0 < a.M; v0 += stride) {
    float acc[kFewRows][N] = {};
    const T* row[kFewRows];
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) row[r] = static_cast<const T*>(a.A) + min(v0 + r, (uint64_t)a.M - 1) * width;
    // (the last stretch, which a row need not fill, on its own)
    const auto stretch = [&](uint32_t c, auto full) {
      float w[kFewRows][E];
#pragma unroll
      for (int r = 0; r < kFewRows; ++r) {
        T e[E];
        if (decltype(full)::value || c + E <= width) {
          __builtin_memcpy(e, row[r] + c, 16);
        } else {
#pragma unroll
          for (int k = 0; k < E; ++k) e[k] = c + k < width ? row[r][c + k] : T(0.f);
        }
#pragma unroll
        for (int k = 0; k < E; ++k) w[r][k] = to_f32(e[k]);
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        T e[E];
        __builtin_memcpy(e, __builtin_assume_aligned(x + n * fill + c, 16), 16);
#pragma unroll
        for (int k = 0; k < E; ++k)
#pragma unroll
          for (int r = 0; r < kFewRows; ++r) acc[r][n] = fmaf(w[r][k], to_f32(e[k]), acc[r][n]);
      }
    };
    uint32_t c = lane * E;
#pragma unroll 4
    for (; c - lane * E + kWave * E <= width; c += kWave * E) stretch(c, std::true_type{});
    if (c - lane * E < width) stretch(c, std::false_type{});
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float l = a.scale * wave_sum(acc[r][n]);
        if (v0 + r < a.M) {
          const float m = fmaxf(most[n], l);
          sum[n] = sum[n] * exp_below(most[n], m) + exp_below(l, m);
          most[n] = m;
          if ((int64_t)(v0 + r) == y[n] && lane == 0) a.hit[n] = l;
        }
      }
  }
  if (lane == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) part[wave][n] = make_float2(most[n], sum[n]);
  }
  __syncthreads();
  if (threadIdx.x < a.N) {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, part[w][threadIdx.x].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) s += part[w][threadIdx.x].y * exp_below(part[w][threadIdx.x].x, m);
    a.stats[(uint64_t)blockIdx.x * a.N + threadIdx.x] = make_float2(m, s);
  }
}

// ------------------------------------------------------------------ layouts
// dst[r][c] = src[r][c], zeros for columns from `cols` to `fill`; targets: zeros also for rows of tokens that are left
// out and from `rows` on.  Two tensors a launch, of which either may have no rows.
struct RowsCopy {
  const void* src;
  void* dst;
  uint64_t rows, rows_fill;
  uint32_t cols, fill;
  const void* targets;
  int id_bytes;
  uint32_t vocab;
};
struct RowsCopies {
  RowsCopy c[2];
};
template <typename T>
__global__ __launch_bounds__(256) void k_xent_rows(RowsCopies a) {
  constexpr int E = 16 / sizeof(T);
  const uint64_t n0 = a.c[0].rows_fill * (a.c[0].fill / E), n = n0 + a.c[1].rows_fill * (a.c[1].fill / E), stride = (uint64_t)gridDim.x * 256;
  for (uint64_t k = (uint64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += stride) {
    const RowsCopy& q = a.c[k >= n0];
    const uint64_t i = k >= n0 ? k - n0 : k, r = i / (q.fill / E);
    const uint32_t c = (uint32_t)(i % (q.fill / E)) * E;
    bool in = r < q.rows;
    if (in && q.targets) {
      const int64_t y = target_of(q.targets, q.id_bytes, (uint32_t)r);
      in = y >= 0 && y < (int64_t)q.vocab;
    }
    T v[E];
    const T* p = static_cast<const T*>(q.src) + r * q.cols + c;
    if (in && c + E <= q.cols) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = in && c + e < q.cols ? p[e] : T(0.f);
    }
    __builtin_memcpy(static_cast<T*>(q.dst) + r * q.fill + c, v, 16);
  }
}

// ------------------------------------------------------------------ logits of a split product
// Where tokens and vocabulary are too few tiles for the chip, the logits' products are split over the width, and what follows
// them is done here, from the parts, which are the only place where logits are in memory (kPartFloats at most).
struct LogitParts {
  const float* part;  // [split][N][M]
  uint32_t splits;
};
constexpr int kStretch = 4 * kWave;  // vocabulary entries of a wave
// The sums of the parts at N places, a part's loads together and four parts' on their way
template <int N>
__device__ __forceinline__ void sum_parts(const LogitParts& p, const ProductArgs& a, const uint64_t (&at)[N], float (&x)[N]) {
  const uint64_t size = (uint64_t)a.N * a.M;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = p.part[at[i]];
  uint32_t k = 1;
  for (; k + 4 <= p.splits; k += 4) {
    float y[4][N];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < N; ++i) y[q][i] = p.part[(k + q) * size + at[i]];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += y[q][i];
  }
  for (; k < p.splits; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += p.part[k * size + at[i]];
}
// A wave's token and stretch of the vocabulary: maximum and sum, in the place of a tile's.
__global__ __launch_bounds__(256) void k_xent_parts_stats(ProductArgs a, LogitParts p) {
  const uint32_t stretches = (a.M + kStretch - 1) / kStretch, unit = blockIdx.x * 4 + threadIdx.x / kWave;
  const uint32_t t = unit / stretches, c = unit % stretches, lane = lane_id();
  if (t >= a.N) return;
  const int64_t y = target_of(a.targets, a.id_bytes, t);
  float l[4], m = -INFINITY, s = 0.f;
  uint64_t at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) at[i] = (uint64_t)t * a.M + min(c * kStretch + i * kWave + lane, a.M - 1);
  sum_parts(p, a, at, l);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = c * kStretch + i * kWave + lane;
    l[i] = v < a.M ? a.scale * l[i] : -INFINITY;
    if ((int64_t)v == y && v < a.M) a.hit[t] = l[i];
    m = fmaxf(m, l[i]);
  }
#pragma unroll
  for (int off = 32; off; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c * kStretch + i * kWave + lane < a.M) s += exp_below(l[i], m);
  s = wave_sum(s);
  if (lane == 0) a.stats[(uint64_t)c * a.N + t] = make_float2(m, s);
}
template <typename T>
__global__ __launch_bounds__(256) void k_xent_parts_grad(ProductArgs a, LogitParts p) {
  const uint64_t n = (uint64_t)a.n_fill * a.m_fill, stride = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
    const uint32_t t = (uint32_t)(i / a.m_fill), v = (uint32_t)(i % a.m_fill);
    float x[1] = {};
    if (t < a.N && v < a.M && live(a, t)) {
      const uint64_t at[1] = {(uint64_t)t * a.M + v};
      sum_parts(p, a, at, x);
      const float d = a.scale * a.dloss[t], f = a.dlse ? d + a.scale * a.dlse[t] : d;
      x[0] = f * exp_of(fmaf(x[0], a.scale, -a.lse[t]));
      if ((int64_t)a.v0 + v == target_of(a.targets, a.id_bytes, t)) x[0] -= d;
    }
    T* const to = static_cast<T*>(a.G) + (uint64_t)t * a.ldg + v;
    *to = from_f32<T>(x[0]);
    if (a.rest) *reinterpret_cast<T*>(reinterpret_cast<char*>(to) + a.rest) = from_f32<T>(x[0] - to_f32(*to));
  }
}

// ------------------------------------------------------------------ joins
// lse and loss of each token from t0 on from its tiles' maxima and sums: TOKENS of them a block, 256 / TOKENS threads each
template <int TOKENS>
__global__ __launch_bounds__(256) void k_xent_join(const float2* __restrict__ stats, uint32_t tiles, uint32_t t0, uint32_t tokens, const float* __restrict__ hit,
                                                   const void* targets, int id_bytes, uint32_t vocab, float* __restrict__ loss, float* __restrict__ lse) {
  constexpr int PARTS = 256 / TOKENS, N = 4;  // (loads on their way)
  __shared__ float2 sh[PARTS][TOKENS + 1];
  const uint32_t i = threadIdx.x % TOKENS, k = threadIdx.x / TOKENS, t = t0 + blockIdx.x * TOKENS + i;
  float m = -INFINITY, s = 0.f;
  const auto add = [&](float2 p) {
    const float n = fmaxf(m, p.x);
    s = s * exp_below(m, n) + p.y * exp_below(p.x, n);
    m = n;
  };
  if (t < tokens)
    for (uint32_t j = k; j < tiles; j += PARTS * N) {
      float2 p[N];
#pragma unroll
      for (int q = 0; q < N; ++q) p[q] = stats[(uint64_t)min(j + q * PARTS, tiles - 1) * tokens + t];
#pragma unroll
      for (int q = 0; q < N; ++q)
        if (j + q * PARTS < tiles) add(p[q]);
    }
  sh[k][i] = make_float2(m, s);
#pragma unroll
  for (int half = PARTS / 2; half; half /= 2) {
    __syncthreads();
    if (k < (uint32_t)half) {
      add(sh[k + half][i]);
      sh[k][i] = make_float2(m, s);
    }
  }
  if (k || t >= tokens) return;
  const int64_t y = target_of(targets, id_bytes, t);
  const bool in = y >= 0 && y < (int64_t)vocab;
  const float e = in ? m + logf(s) : 0.f;
  if (loss) loss[t] = in ? e - hit[t] : 0.f;
  if (lse) lse[t] = e;
}
// dst = the sum of the splits
template <typename T>
__global__ __launch_bounds__(256) void k_xent_sum(const float* __restrict__ part, uint32_t splits, uint64_t n, T* __restrict__ dst) {
  const uint64_t stride = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
    float s = part[i];
    for (uint32_t k = 1; k < splits; ++k) s += part[k * n + i];
    dst[i] = from_f32<T>(s);
  }
}

// ------------------------------------------------------------------ plan
constexpr uint32_t kTile = 128;
// bytes of G (16384 tokens, 65536 x 2048 in bfloat16, forward and backward, on one card in turn: 13.60 ms; twice as many 13.77, half 13.81)
constexpr uint64_t kPiece = 1ull << 29;
static uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }
static uint32_t tiles(uint64_t n, uint32_t of = kTile) { return (uint32_t)((n + of - 1) / of); }

// Sizes that a call with this many tokens keeps in its workspace; each grows with the tokens.
// G in two parts of bfloat16, which hold 16 of its bits, for so many tokens: half a step of the one that a token's row of dx
// is mostly made of shows in the row, and among few tokens in the whole (11 tokens, 227 x 2696: dx off by 0.0030 of its size, with
// two parts 0.0017, which is its own rounding; the backward of 200 tokens, 500 x 4096 takes 33 us instead of 26, of 64, 65536 x 2048 404
// instead of 278, of 1000, 8000 x 1024 128 instead of 90).  Among 600 it still is up to 1.5 times its own rounding.  Among more it is
// 1.44 times that and no more, G's half step beside its own, and the products, which the matrix cores bound, would be six
// instead of four (16384 tokens, 65536 x 2048, forward and backward: off by 0.0024 and 0.0022 of dx and dtable, 13.65 ms; with two
// parts 0.0017 and 0.0017, 20.85 ms; 2049, 8000 x 1024: 0.0024 and 0.0023, 256 us; 0.0017 and 0.0017, 378).  A gradient
// of the table in float32 has no rounding beside which one part's could be lost: its product takes two always.
constexpr uint64_t kTwoParts = 2048;
struct XentPlan {
  uint64_t k_width, k_tokens;  // extents of k, whole pieces
  uint32_t parts;              // of G
  uint32_t piece;              // vocabulary entries at a time
};
static XentPlan xent_plan(int dtype, uint64_t tokens, uint32_t vocab, uint32_t width) {
  const uint64_t e = dtype == LAPLEX_BF16 ? 2 : 4, bk = kPieceK / e;
  XentPlan p;
  p.k_width = up(width, bk);
  p.k_tokens = up(tokens, bk);
  p.parts = dtype == LAPLEX_BF16 && tokens <= kTwoParts ? 2 : 1;
  const uint64_t fit = kPiece / (e * p.parts * std::max<uint64_t>(p.k_tokens, 1)) / kTile * kTile;
  p.piece = (uint32_t)std::min<uint64_t>(up(vocab, bk), std::max<uint64_t>(kTile, fit));
  return p;
}

// Blocks of k_xent_few: one turn of rows a wave at least (4 tokens, 2418 x 1770 in float: 18 us; with four turns 37), and at
// most four a CU (1 token, 65536 x 2048 in bfloat16: 57.5 us; eight 60).
static uint32_t few_blocks(uint32_t vocab) { return std::min(1024u, (vocab + 4 * kFewRows - 1) / (4 * kFewRows)); }

// ------------------------------------------------------------------ tiles and splits of a product
// By a model of its time: rounds of blocks over the CUs, each at the rate that its tile reaches, and for a split product the
// pass that adds the parts.  Rates, in 10^6 operations a us and CU, are those of large products with one tile for all of them:
// 16384 x 16384 x 2048 in bfloat16, forward (along k) 1371, 974, 716 and 443 TFLOP/s by tiles L, M, S and T, with the
// backward (a third of it along k, the rest across) 1266, 974, 550 and 284; 4096 x 16384 x 1024 in float 147, 140, 138 and 129, and
// 106, 136, 135 and 124.  A step takes kStepLeast us however little there is to do in it (32 tokens, 2000 x 2048 in bfloat16: the
// forward unsplit 12.5 us, split 11.5; the backward 31.7 and 26.8).
struct Tiling {
  int tile;         // TILE_L .. TILE_T
  uint32_t splits;  // of k
};
enum { TILE_L, TILE_M, TILE_S, TILE_T };
constexpr uint32_t kTileM[] = {TileL::BM, TileM::BM, TileS::BM, TileT::BM}, kTileN[] = {TileL::BN, TileM::BN, TileS::BN, TileT::BN};
static double rate_of(bool bf, bool across, int tile) {
  const double rates[2][2][4] = {{{.57, .55, .54, .50}, {.41, .53, .53, .48}}, {{5.4, 3.8, 2.8, 1.7}, {4.9, 3.8, 2.1, 1.1}}};
  return rates[bf][across][tile];
}
// tokens of a launch of the join, which has 16 threads for each (a launch has fewer than 2^32)
constexpr uint64_t kJoinMost = 1ull << 27;
// partial sums of a split product, in floats
constexpr uint64_t kPartFloats = 8ull << 20, kMostSplits = 64;
constexpr double kStepLeast = 0.25;
static Tiling tiling(bool bf, bool across, uint64_t M, uint64_t N, uint64_t K, bool may_split) {
  const uint64_t bk = kPieceK / (bf ? 2 : 4), steps = std::max<uint64_t>(1, K / bk);
  Tiling best{TILE_S, 1};
  double least = 1e300;
  for (int t = TILE_L; t <= TILE_T; ++t) {
    const uint64_t blocks = tiles(M, kTileM[t]) * (uint64_t)tiles(N, kTileN[t]);
    for (uint64_t s = 1; s <= kMostSplits; s *= 2) {
      if (s > 1 && (!may_split || s * 4 > steps || s * M * N > kPartFloats)) break;
      const double step = 2e-6 * kTileM[t] * kTileN[t] * bk / rate_of(bf, across, t);
      const double us = (double)((steps + s - 1) / s) * std::max((double)((blocks * s + 255) / 256) * step, kStepLeast) +
                        (s > 1 ? 4.0 + s * M * N * 8e-6 / 4.0 : 0.0) + 2.0;
      if (us < least) {
        least = us;
        best = {t, (uint32_t)s};
      }
    }
  }
  return best;
}

// Whether the forward goes by the table row after row
static bool few_tokens(uint64_t tokens, uint64_t width, uint64_t e) {
  return tokens <= (uint64_t)(width * e % kPieceK ? kFewTokens : kFewTokensWhole) && kFewTokens * up(width, kWave * 16 / e) * e <= kFewBytes;
}

struct XentWorkspace {
  void *x_rows, *table_rows;  // filled up copies, where rows are not whole pieces
  float2* stats;
  float* hit;
  void* G;
  uint64_t g_bytes;
  float* dx;    // dx while pieces of the vocabulary are added to it
  float* part;  // parts of a split product
};
static bool whole_rows(const void* p, uint64_t width, uint64_t e) { return width * e % kPieceK == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// aligned: x and the table begin at multiples of 16 bytes, so that rows of whole pieces need no copies
static XentWorkspace xent_carve(void* ws, int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width, bool aligned, size_t* total) {
  const uint64_t e = dtype == LAPLEX_BF16 ? 2 : 4;
  const XentPlan p = xent_plan(dtype, tokens, vocab, width);
  Carver c(ws);
  XentWorkspace w{};
  const bool few = pass == 0 && few_tokens(tokens, width, e), lie = few || (aligned && whole_rows(nullptr, width, e));
  if (pass == 1 || !lie) w.x_rows = c.take<void>(p.k_tokens * p.k_width * e);
  if (!lie) w.table_rows = c.take<void>(vocab * p.k_width * e);
  if (pass == 0) {
    // (of the smallest tiles, or of a few tokens' blocks)
    w.stats = c.take<float2>(std::max<uint64_t>(tiles(vocab, TileS::BM) * tokens, few_blocks(vocab) * std::min<uint64_t>(tokens, kFewTokens)) * 8);
    w.hit = c.take<float>(tokens * 4);
    if (!few) w.part = c.take<float>(std::min<uint64_t>(kPartFloats, kMostSplits * tokens * vocab) * 4);
  } else {
    // (a piece has at most kPiece bytes, or one tile of the vocabulary, or all of it)
    const uint64_t bk = kPieceK / e;
    const auto g = [&](uint64_t rows) { return std::max<uint64_t>(std::min<uint64_t>(kPiece, up(vocab, bk) * rows * e), kTile * rows * e); };
    // (of more tokens' one part, or those at the switch, of which there are two)
    const uint64_t two = dtype == LAPLEX_BF16 ? up(std::min(tokens, kTwoParts), bk) * 2 : 0;
    w.g_bytes = std::max(g(p.k_tokens), g(two));
    w.G = c.take<void>(w.g_bytes);
    w.dx = c.take<float>(tokens * width * 4);
    w.part = c.take<float>(kPartFloats * 4);
  }
  *total = (c.off + 255) & ~size_t(255);
  return w;
}
size_t xent_bytes(int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width, bool aligned) {
  size_t total = 0;
  xent_carve(nullptr, pass, dtype, tokens, vocab, width, aligned, &total);
  return total;
}
bool xent_aligned(const void* x, const void* table) { return (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(table)) % 16 == 0; }

enum Product { LOGITS_STATS, LOGITS_GRAD, LOGITS_PARTS, DX, DTABLE };
template <typename T, typename C>
static hipError_t product_of(const char* name, Product epi, ProductArgs& a, hipStream_t s) {
  a.tiles_m = tiles(a.M, C::BM);
  a.tiles_n = tiles(epi == LOGITS_GRAD ? std::max(a.N, a.n_fill) : a.N, C::BN);
  const uint64_t all = (uint64_t)a.tiles_m * a.tiles_n * a.splits, blocks = std::min<uint64_t>(all, 256 * C::PER_CU);
  LAPLEX_LAUNCH(name, all, s, {
    if (epi == LOGITS_STATS) k_product<T, XENT_STATS, C, false, false><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
    else if (epi == LOGITS_GRAD) k_product<T, XENT_GRAD, C, false, false><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
    else if (epi == LOGITS_PARTS) k_product<T, XENT_OUT, C, false, false><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
    else if (epi == DX) k_product<T, XENT_OUT, C, true, false><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
    else k_product<T, XENT_OUT, C, true, true><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
  });
  return hipGetLastError();
}
template <typename T>
static hipError_t product(const char* name, Product epi, ProductArgs& a, const Tiling& t, hipStream_t s) {
  constexpr uint64_t bk = kPieceK / sizeof(T);
  a.k_split = std::max(bk, up((a.K + t.splits - 1) / t.splits, bk));
  a.splits = (uint32_t)std::max<uint64_t>(1, (a.K + a.k_split - 1) / a.k_split);
  switch (t.tile) {
    case TILE_L: return product_of<T, TileL>(name, epi, a, s);
    case TILE_M: return product_of<T, TileM>(name, epi, a, s);
    case TILE_S: return product_of<T, TileS>(name, epi, a, s);
    default: return product_of<T, TileT>(name, epi, a, s);
  }
}
static unsigned some_blocks(uint64_t n) { return (unsigned)std::min<uint64_t>((n + 255) / 256, 16384); }

// x and the table in rows of whole pieces, as they lie or copied (x in the backward always: without the tokens that are
// left out, and with rows of zeros up to a whole step)
template <typename T>
static hipError_t whole(const XentShape& x, const XentPlan& p, const XentWorkspace& w, bool back, const void** rows, const void** table, hipStream_t s) {
  RowsCopies c{};
  *rows = x.x;
  *table = x.table;
  const auto copy = [&](int i, const void** at, void* to, uint64_t n, uint64_t fill) {
    c.c[i] = {*at, to, n, fill, x.width, (uint32_t)p.k_width, i == 0 && back ? x.targets : nullptr, x.id_bytes, x.vocab};
    *at = to;
  };
  if (back || !whole_rows(x.x, x.width, sizeof(T))) copy(0, rows, w.x_rows, x.tokens, back ? p.k_tokens : x.tokens);
  if (!whole_rows(x.table, x.width, sizeof(T))) copy(1, table, w.table_rows, x.vocab, x.vocab);
  const uint64_t n = (c.c[0].rows_fill + c.c[1].rows_fill) * p.k_width * sizeof(T) / 16;
  for (RowsCopy& q : c.c) q.fill = (uint32_t)p.k_width;
  if (n) LAPLEX_LAUNCH("k_xent_rows", n, s, k_xent_rows<T><<<some_blocks(n), 256, 0, s>>>(c));
  return hipGetLastError();
}

template <typename T, int N = kFewTokens>
static hipError_t few(ProductArgs& a, uint32_t width, hipStream_t s) {
  if constexpr (N > 1)
    if (a.N <= N / 2) return few<T, N / 2>(a, width, s);
  const uint32_t fill = (uint32_t)up(width, kWave * 16 / sizeof(T)), bytes = N * fill * (uint32_t)sizeof(T);
  const uint32_t blocks = few_blocks(a.M);
  if (bytes > (48u << 10)) {
    const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(k_xent_few<T, N>), hipFuncAttributeMaxDynamicSharedMemorySize, (int)kFewBytes);
    if (err != hipSuccess) return err;
  }
  LAPLEX_LAUNCH("k_xent_few", a.M, s, k_xent_few<T, N><<<blocks, 256, bytes, s>>>(a, width, fill));
  a.tiles_m = blocks;
  return hipGetLastError();
}
// Whether the logits' product is better split, and how it is tiled
template <typename T>
static bool in_parts(const ProductArgs& l, uint64_t n_tiles, Tiling& t) {
  t = tiling(sizeof(T) == 2, false, l.M, n_tiles, l.K, true);
  return t.splits > 1;
}
template <typename T>
static hipError_t logit_parts(const ProductArgs& l, const Tiling& t, float* part, LogitParts& p, hipStream_t s) {
  ProductArgs a = l;
  a.rest = 0;
  a.out = part;
  a.out_f32 = true;
  a.ldo = a.M;
  a.out_split = (int64_t)a.N * a.M;
  const hipError_t err = product<T>("k_product_logits", LOGITS_PARTS, a, t, s);
  p = {part, a.splits};
  return err;
}
template <typename T>
static hipError_t forward(const XentShape& x, float* loss, float* lse, void* ws, hipStream_t s) {
  size_t total;
  const XentPlan p = xent_plan(x.dtype, x.tokens, x.vocab, x.width);
  const XentWorkspace w = xent_carve(ws, 0, x.dtype, x.tokens, x.vocab, x.width, xent_aligned(x.x, x.table), &total);
  ProductArgs a{};
  a.A = x.table;
  a.B = x.x;
  a.M = x.vocab;
  a.N = (uint32_t)x.tokens;
  a.targets = x.targets;
  a.id_bytes = x.id_bytes;
  a.vocab = x.vocab;
  a.scale = x.scale;
  a.stats = w.stats;
  a.hit = w.hit;
  hipError_t err;
  if (few_tokens(x.tokens, x.width, sizeof(T))) {
    if ((err = few<T>(a, x.width, s)) != hipSuccess) return err;
  } else {
    if ((err = whole<T>(x, p, w, false, &a.B, &a.A, s)) != hipSuccess) return err;
    a.lda = a.ldb = (int64_t)p.k_width;
    a.K = p.k_width;
    Tiling t;
    if (in_parts<T>(a, a.N, t)) {
      LogitParts parts;
      if ((err = logit_parts<T>(a, t, w.part, parts, s)) != hipSuccess) return err;
      a.tiles_m = tiles(a.M, kStretch);
      LAPLEX_LAUNCH("k_xent_parts_stats", a.N, s, k_xent_parts_stats<<<(unsigned)((x.tokens * a.tiles_m + 3) / 4), 256, 0, s>>>(a, parts));
      if ((err = hipGetLastError()) != hipSuccess) return err;
    } else if ((err = product<T>("k_product_stats", LOGITS_STATS, a, t, s)) != hipSuccess) {
      return err;
    }
  }
  const auto join = [&](auto tokens, uint64_t t0, uint64_t n) {
    constexpr int TOKENS = decltype(tokens)::value;
    LAPLEX_LAUNCH("k_xent_join", n, s,
                  k_xent_join<TOKENS><<<(unsigned)((n + TOKENS - 1) / TOKENS), 256, 0, s>>>(w.stats, a.tiles_m, (uint32_t)t0, a.N, w.hit, x.targets, x.id_bytes,
                                                                                          x.vocab, loss, lse));
  };
  if (x.tokens <= 64) join(std::integral_constant<int, 1>{}, 0, x.tokens);
  else for (uint64_t t0 = 0; t0 < x.tokens; t0 += kJoinMost) join(std::integral_constant<int, 16>{}, t0, std::min(kJoinMost, x.tokens - t0));
  return hipGetLastError();
}
template <typename T>
static hipError_t backward(const XentShape& x, const float* lse, const float* dloss, const float* dlse, void* dx, int table_dtype,
                           void* dtable, void* ws, hipStream_t s) {
  size_t total;
  XentPlan p = xent_plan(x.dtype, x.tokens, x.vocab, x.width);
  const XentWorkspace w = xent_carve(ws, 1, x.dtype, x.tokens, x.vocab, x.width, xent_aligned(x.x, x.table), &total);
  const uint32_t tokens = (uint32_t)x.tokens;
  const void *table = x.table, *rows = x.x;
  hipError_t err;
  const bool dx_parts = p.parts > 1;  // (the table's gradient in float32 takes two where dx has one: G's place then holds fewer entries)
  if (sizeof(T) == 2 && tokens && dtable && table_dtype == LAPLEX_F32 && !dx_parts) {
    p.parts = 2;
    const uint64_t fit = w.g_bytes / (2 * sizeof(T) * p.k_tokens);  // (at least 64: there is room for 128 of one part)
    p.piece = (uint32_t)std::min<uint64_t>(p.piece, fit >= kTile ? fit / kTile * kTile : kTile / 2);
  }
  if (tokens) {  // (without, dtable is a sum of nothing)
    if ((err = whole<T>(x, p, w, true, &rows, &table, s)) != hipSuccess) return err;
  } else {
    dx = nullptr;
  }
  ProductArgs l{};
  l.B = rows;
  l.lda = l.ldb = (int64_t)p.k_width;
  l.K = p.k_width;
  l.N = tokens;
  l.targets = x.targets;
  l.id_bytes = x.id_bytes;
  l.vocab = x.vocab;
  l.scale = x.scale;
  l.lse = lse;
  l.dloss = dloss;
  l.dlse = dlse;
  l.G = w.G;
  l.n_fill = (uint32_t)p.k_tokens;
  // A product that may be split: to its place, or its parts and then their sum
  const auto output = [&](const char* name, Product epi, ProductArgs& a) {
    const Tiling t = tiling(sizeof(T) == 2, true, a.M, a.N, a.rest ? 2 * a.K : a.K, !a.add);
    if (t.splits == 1) return product<T>(name, epi, a, t, s);
    void* const out = a.out;
    const bool f32 = a.out_f32;
    a.out = w.part;
    a.out_f32 = true;
    a.out_split = (int64_t)a.N * a.ldo;
    const hipError_t e = product<T>(name, epi, a, t, s);
    if (e != hipSuccess) return e;
    const uint64_t n = (uint64_t)a.out_split;
    LAPLEX_LAUNCH("k_xent_sum", n, s, {
      if (f32) k_xent_sum<float><<<some_blocks(n), 256, 0, s>>>(w.part, a.splits, n, static_cast<float*>(out));
      else k_xent_sum<T><<<some_blocks(n), 256, 0, s>>>(w.part, a.splits, n, static_cast<T*>(out));
    });
    return hipGetLastError();
  };
  const bool once = p.piece >= x.vocab;  // dx is one product
  for (uint32_t v0 = 0; v0 < x.vocab; v0 += p.piece) {
    const uint32_t n = std::min(p.piece, x.vocab - v0);
    const uint64_t fill = up(n, kPieceK / sizeof(T));
    l.A = static_cast<const T*>(table) + v0 * p.k_width;
    l.M = n;
    l.v0 = v0;
    l.ldg = (int64_t)fill;
    l.m_fill = (uint32_t)fill;
    l.rest = p.parts > 1 ? (int64_t)(p.k_tokens * fill * sizeof(T)) : 0;
    Tiling t;
    if (tokens && in_parts<T>(l, l.n_fill, t)) {
      LogitParts parts;
      if ((err = logit_parts<T>(l, t, w.part, parts, s)) != hipSuccess) return err;
      const uint64_t all = (uint64_t)l.n_fill * l.m_fill;
      LAPLEX_LAUNCH("k_xent_parts_grad", l.N, s, k_xent_parts_grad<T><<<some_blocks(all), 256, 0, s>>>(l, parts));
      if ((err = hipGetLastError()) != hipSuccess) return err;
    } else if (tokens && (err = product<T>("k_product_grad", LOGITS_GRAD, l, t, s)) != hipSuccess) {
      return err;
    }
    if (dx) {
      ProductArgs a{};
      a.A = l.A;
      a.lda = l.lda;
      a.B = w.G;
      a.ldb = (int64_t)fill;
      a.rest = dx_parts ? l.rest : 0;
      a.K = fill;
      a.k_rows = n;
      a.M = x.width;
      a.N = tokens;
      a.targets = x.targets;
      a.id_bytes = x.id_bytes;
      a.vocab = x.vocab;
      a.live_rows = true;
      a.ldo = x.width;
      a.out = once ? dx : w.dx;
      a.out_f32 = !once || sizeof(T) == 4;
      a.add = v0 > 0;
      if ((err = output("k_product_dx", DX, a)) != hipSuccess) return err;
    }
    if (dtable) {
      ProductArgs a{};
      a.A = rows;
      a.lda = (int64_t)p.k_width;
      a.B = w.G;
      a.ldb = (int64_t)fill;
      a.rest = l.rest;
      a.K = a.k_rows = p.k_tokens;
      a.M = x.width;
      a.N = n;
      a.ldo = x.width;
      a.out_f32 = table_dtype == LAPLEX_F32;
      a.out = static_cast<char*>(dtable) + (uint64_t)v0 * x.width * (a.out_f32 ? 4 : 2);
      if ((err = output("k_product_dtable", DTABLE, a)) != hipSuccess) return err;
    }
  }
  if (dx && !once) {
    const uint64_t n = x.tokens * x.width;
    LAPLEX_LAUNCH("k_xent_sum", n, s, k_xent_sum<T><<<some_blocks(n), 256, 0, s>>>(w.dx, 1, n, static_cast<T*>(dx)));
  }
  return hipGetLastError();
}

hipError_t xent(const XentShape& x, float* loss, float* lse, void* ws, hipStream_t s) {
  return x.dtype == LAPLEX_BF16 ? forward<bf16>(x, loss, lse, ws, s) : forward<float>(x, loss, lse, ws, s);
}
hipError_t xent_backward(const XentShape& x, const float* lse, const float* dloss, const float* dlse, void* dx, int table_dtype,
                         void* dtable, void* ws, hipStream_t s) {
  return x.dtype == LAPLEX_BF16 ? backward<bf16>(x, lse, dloss, dlse, dx, table_dtype, dtable, ws, s)
                                : backward<float>(x, lse, dloss, dlse, dx, table_dtype, dtable, ws, s);
}

}  // namespace laplex
