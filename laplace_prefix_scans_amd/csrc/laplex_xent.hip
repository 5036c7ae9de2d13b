// Softmax cross entropy of rows against a linear output table, forward and backward, without the logits in memory.
//
//   l_tv = c x_t . W_v,  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_{t y_t},
//   G_tv = c [(dloss_t + dlse_t) exp(l_tv - lse_t) - dloss_t [v = y_t]],  dx = G W,  dW = G^T x.
//
// Four matrix products (the logits twice), all of one kernel: C[n][m] = sum_k A[m][k] B[n][k] on the matrix cores, rows
// of A and B contiguous in k.  What follows the product is fused: the forward keeps a maximum and a sum of exponentials
// per token and tile of the vocabulary, the backward writes a tile of G and its transpose.  For the products with G the
// other factor is laid out along k first (W and x transposed, one pass over each), which also leaves out the tokens that
// take no part and fills odd sizes up with zeros.
#include <algorithm>

#include "laplex_host.hpp"
#include "laplex_layers_device.hpp"
#include "laplex_train.hpp"

namespace laplex {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

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
  int64_t lda, ldb;  // elements; rows are whole 128-byte pieces (or zeros beyond their end)
  uint32_t M, N;     // rows of A, of B
  uint64_t K;        // a multiple of a 128-byte piece
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
  void *G, *Gt;      // [token][ldg], [vocabulary entry][ldgt]
  int64_t ldg, ldgt;
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

// Tile and split of this block.  Blocks are dispatched to the 8 XCDs in turn; each XCD takes a stretch of the tiles, in
// groups of 8 tiles of M by all of N, of which the ones that run at once share rows of both factors in its L2.
__device__ __forceinline__ void tile_of_block(const ProductArgs& a, uint32_t& tm, uint32_t& tn, uint32_t& split) {
  constexpr uint32_t GROUP = 8;
  const uint32_t total = a.tiles_m * a.tiles_n, all = total * a.splits;
  const uint32_t per = all / kXcds, rest = all % kXcds, x = blockIdx.x % kXcds, y = blockIdx.x / kXcds;
  uint32_t id = x * per + min(x, rest) + y;  // (XCD x has per blocks, and one more where x < rest)
  split = id / total;
  id %= total;
  const uint32_t group = id / (GROUP * a.tiles_n), first = group * GROUP, rows = min(GROUP, a.tiles_m - first);
  const uint32_t in = id - first * a.tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// ------------------------------------------------------------------ the product
// A block of WM x WN waves makes BM x BN of C.  128 bytes of k of its rows are on their way from memory straight to LDS
// while those before are multiplied; a row's eight 16-byte pieces lie at piece ^ (row & 7), so that the reads of 16
// rows' pieces spread over the banks.  A step's 128 bytes are two halves, and a half's operands are read one half ahead of
// their products, across the step's one barrier: it stands in the middle of a step, where both halves of it have been read
// and the next one's bytes have arrived.
template <int M, int N, int WAVES_M, int WAVES_N>
struct Tile {
  static constexpr int BM = M, BN = N, WM = WAVES_M, WN = WAVES_N, THREADS = WM * WN * kWave;
  static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  static constexpr int LOADS = (BM + BN) / 8 / (WM * WN);  // of a wave and step: 8 rows each
  static constexpr int STEP_BYTES = (BM + BN) * 128;
  static_assert((BM + BN) % (8 * WM * WN) == 0 && BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "whole operands");
};
using TileL = Tile<256, 256, 2, 4>;
using TileM = Tile<128, 128, 2, 2>;
using TileS = Tile<64, 64, 2, 2>;
using TileT = Tile<128, 32, 4, 1>;

// 16 bytes of each lane from memory to lds + 16 lane
__device__ __forceinline__ void to_lds(const char* from, char* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// Every wave's reads of LDS are done, and its bytes on their way to LDS are there.
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

constexpr int kPieceK = 128;
template <typename T, int EPI, typename C>
__global__ __launch_bounds__(C::THREADS) void k_product(ProductArgs a) {
  constexpr int BM = C::BM, BN = C::BN, MI = C::MI, NI = C::NI, W = C::WM * C::WN;
  __shared__ __attribute__((aligned(16))) char lds[2 * C::STEP_BYTES];
  using V = typename Frag<T>::V;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  uint32_t tm, tn, split;
  tile_of_block(a, tm, tn, split);
  const uint64_t k0 = split * a.k_split, k1 = min(a.K, k0 + a.k_split);
  const int steps = (int)((k1 - k0) * sizeof(T) / kPieceK);
  // this lane's 16 bytes of each of the wave's groups of 8 rows
  const char* from[C::LOADS];
#pragma unroll
  for (int i = 0; i < C::LOADS; ++i) {
    const int row = (i * W + wave) * 8 + lane / 8;
    const T* p = row < BM ? static_cast<const T*>(a.A) + (int64_t)min(tm * BM + row, a.M - 1) * a.lda
                          : static_cast<const T*>(a.B) + (int64_t)min(tn * BN + row - BM, a.N - 1) * a.ldb;
    from[i] = reinterpret_cast<const char*>(p + k0) + ((lane % 8) ^ (lane / 8)) * 16;
  }
  auto load = [&](int step) {
#pragma unroll
    for (int i = 0; i < C::LOADS; ++i) to_lds(from[i] + (int64_t)step * kPieceK, lds + (step & 1) * C::STEP_BYTES + (i * W + wave) * 8 * kPieceK);
  };
  f32x4 acc[MI][NI] = {};
  const int wm = wave % C::WM * (BM / C::WM), wn = wave / C::WM * (BN / C::WN);
  if (steps > 0) {
    V fa[2][MI], fb[2][NI];
    // (a row's number & 7 is the lane's)
    const uint32_t at_a = (wm + lane % 16) * kPieceK, at_b = (BM + wn + lane % 16) * kPieceK;
    const uint32_t piece[2] = {(uint32_t)((lane / 16) ^ (lane % 8)) * 16, (uint32_t)((4 + lane / 16) ^ (lane % 8)) * 16};
    auto read = [&](int step, int half) {
      const char* base = lds + (step & 1) * C::STEP_BYTES;
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[half][j] = *reinterpret_cast<const V*>(base + at_b + piece[half] + j * 16 * kPieceK);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[half][i] = *reinterpret_cast<const V*>(base + at_a + piece[half] + i * 16 * kPieceK);
    };
    auto multiply = [&](int half) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = Frag<T>::mul(fa[half][i], fb[half][j], acc[i][j]);
      // a read after every few products
#pragma unroll
      for (int r = 0; r < MI + NI; ++r) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x8, MI * NI * (sizeof(T) == 4 ? 4 : 1) / (MI + NI), 0);
      }
    };
    load(0);
    arrived();
    if (steps > 1) load(1);
    read(0, 0);
    for (int k = 0; k < steps; ++k) {
      read(k, 1);
      multiply(0);
      arrived();
      if (k + 2 < steps) load(k + 2);
      read(k + 1, 0);  // (after the last step: bytes that nothing uses)
      multiply(1);
    }
    __syncthreads();
  }
  // a lane holds column n = lane % 16 and rows m = lane / 16 * 4 .. + 3 of each 16 x 16 tile
  const uint32_t m0 = tm * BM + wm + lane / 16 * 4, n0 = tn * BN + wn + lane % 16;
  if constexpr (EPI == XENT_STATS) {
    float2* sh = reinterpret_cast<float2*>(lds);  // [wave of M][BN]
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const uint32_t t = n0 + j * 16;
      const int64_t y = t < a.N ? target_of(a.targets, a.id_bytes, t) : -1;
      float most = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t v = m0 + i * 16 + r;
          const float l = a.scale * acc[i][j][r];
          acc[i][j][r] = v < a.M ? l : -INFINITY;
          if ((int64_t)v + a.v0 == y && v < a.M) a.hit[t] = l;
          most = fmaxf(most, acc[i][j][r]);
        }
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum += exp_below(acc[i][j][r], most);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (lane < 16) sh[(wave % C::WM) * BN + wn + j * 16 + lane] = make_float2(most, sum);
    }
    __syncthreads();
    if (threadIdx.x < BN && tn * BN + threadIdx.x < a.N) {
      float m = sh[threadIdx.x].x, sum = 0.f;
#pragma unroll
      for (int w = 1; w < C::WM; ++w) m = fmaxf(m, sh[w * BN + threadIdx.x].x);
#pragma unroll
      for (int w = 0; w < C::WM; ++w) sum += sh[w * BN + threadIdx.x].y * exp_below(sh[w * BN + threadIdx.x].x, m);
      a.stats[(uint64_t)tm * a.N + tn * BN + threadIdx.x] = make_float2(m, sum);
    }
  } else if constexpr (EPI == XENT_GRAD) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const uint32_t t = n0 + j * 16;
      const int64_t y = t < a.N ? target_of(a.targets, a.id_bytes, t) : -1;
      const bool in = y >= 0 && y < (int64_t)a.vocab;
      const float lse = in ? a.lse[t] : 0.f, d = in ? a.scale * a.dloss[t] : 0.f, f = in ? d + (a.dlse ? a.scale * a.dlse[t] : 0.f) : 0.f;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        T g[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t v = m0 + i * 16 + r;
          float x = f * exp_of(a.scale * acc[i][j][r] - lse);
          if ((int64_t)v + a.v0 == y) x -= d;
          g[r] = from_f32<T>(in && v < a.M ? x : 0.f);
        }
        const uint32_t v = m0 + i * 16;
        if (t < a.N && v < a.m_fill) __builtin_memcpy(static_cast<T*>(a.G) + (int64_t)t * a.ldg + v, g, sizeof g);
        if (t < a.n_fill) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (v + r < a.M) static_cast<T*>(a.Gt)[(int64_t)(v + r) * a.ldgt + t] = g[r];
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const uint32_t n = n0 + j * 16;
      if (n >= a.N) continue;
      const bool zero = a.live_rows && !live(a, n);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t m = m0 + i * 16 + r;
          if (m >= a.M) continue;
          float x = zero ? 0.f : acc[i][j][r];
          const uint64_t at = (uint64_t)n * a.ldo + m;
          if (a.out_f32) {
            float* o = static_cast<float*>(a.out) + split * a.out_split + at;
            *o = a.add ? *o + x : x;
          } else {
            static_cast<T*>(a.out)[at] = from_f32<T>(x);
          }
        }
    }
  }
}

// ------------------------------------------------------------------ layouts
// dst[r][c] = src[r][c], zeros for columns from `cols` to `fill`
template <typename T>
__global__ __launch_bounds__(256) void k_xent_rows(const T* __restrict__ src, uint64_t rows, uint32_t cols, uint32_t fill, T* __restrict__ dst) {
  const uint64_t n = rows * fill, stride = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
    const uint64_t r = i / fill;
    const uint32_t c = (uint32_t)(i % fill);
    dst[i] = c < cols ? src[r * cols + c] : T(0.f);
  }
}
// dst[c][r] = src[r][c] for r < rows, zeros from `rows` to `fill`; targets: rows of tokens that are left out are zeros
template <typename T>
__global__ __launch_bounds__(256) void k_xent_transposed(const T* __restrict__ src, uint32_t rows, uint32_t cols, uint32_t fill, T* __restrict__ dst,
                                                         const void* targets, int id_bytes, uint32_t vocab) {
  __shared__ T sh[64][65];
  const uint32_t tiles_c = (cols + 63) / 64, r0 = blockIdx.x / tiles_c * 64, c0 = blockIdx.x % tiles_c * 64;
  for (uint32_t i = threadIdx.x; i < 64 * 64; i += 256) {
    const uint32_t r = r0 + i / 64, c = c0 + i % 64;
    T v = T(0.f);
    if (r < rows && c < cols) {
      bool in = true;
      if (targets) {
        const int64_t y = target_of(targets, id_bytes, r);
        in = y >= 0 && y < (int64_t)vocab;
      }
      if (in) v = src[(uint64_t)r * cols + c];
    }
    sh[i / 64][i % 64] = v;
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 64 * 64; i += 256) {
    const uint32_t c = c0 + i / 64, r = r0 + i % 64;
    if (c < cols && r < fill) dst[(uint64_t)c * fill + r] = sh[i % 64][i / 64];
  }
}

// ------------------------------------------------------------------ joins
// lse and loss of each token from its tiles' maxima and sums: 16 threads a token, 16 tokens a block
__global__ __launch_bounds__(256) void k_xent_join(const float2* __restrict__ stats, uint32_t tiles, uint32_t tokens, const float* __restrict__ hit,
                                                   const void* targets, int id_bytes, uint32_t vocab, float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 sh[16][17];
  const uint32_t i = threadIdx.x % 16, k = threadIdx.x / 16, t = blockIdx.x * 16 + i;
  float m = -INFINITY, s = 0.f;
  if (t < tokens)
    for (uint32_t j = k; j < tiles; j += 16) {
      const float2 p = stats[(uint64_t)j * tokens + t];
      const float n = fmaxf(m, p.x);
      s = s * exp_below(m, n) + p.y * exp_below(p.x, n);
      m = n;
    }
  sh[k][i] = make_float2(m, s);
  __syncthreads();
  if (k || t >= tokens) return;
  for (int j = 1; j < 16; ++j) {
    const float2 p = sh[j][i];
    const float n = fmaxf(m, p.x);
    s = s * exp_below(m, n) + p.y * exp_below(p.x, n);
    m = n;
  }
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
constexpr uint64_t kPiece = 1ull << 30;  // bytes of G and its transpose
static uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }
static uint32_t tiles(uint64_t n, uint32_t of = kTile) { return (uint32_t)((n + of - 1) / of); }

// Sizes that a call with this many tokens keeps in its workspace; each grows with the tokens.
struct XentPlan {
  uint64_t k_width, k_tokens, k_piece;  // extents of k, whole pieces
  uint32_t piece;                       // vocabulary entries at a time
  uint32_t splits;                      // of dx's product over them
};
static XentPlan xent_plan(int dtype, uint64_t tokens, uint32_t vocab, uint32_t width) {
  const uint64_t e = dtype == LAPLEX_BF16 ? 2 : 4, bk = kPieceK / e;
  XentPlan p;
  p.k_width = up(width, bk);
  p.k_tokens = up(tokens, bk);
  const uint64_t fit = kPiece / (2 * e * std::max<uint64_t>(p.k_tokens, 1)) / kTile * kTile;
  p.piece = (uint32_t)std::min<uint64_t>(up(vocab, bk), std::max<uint64_t>(kTile, fit));
  p.k_piece = up(p.piece, bk);
  // Where dx has fewer tiles than the chip has CUs, its sums over the vocabulary are split.
  const uint64_t t = (uint64_t)tiles(std::max<uint64_t>(tokens, 1)) * tiles(width);
  p.splits = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(512 / t, p.k_piece / bk));
  return p;
}
struct XentWorkspace {
  void *x_rows, *table_rows;  // filled up copies, where rows are not whole pieces
  float2* stats;
  float* hit;
  void *G, *Gt, *x_t, *table_t;
  float* dx;
};
static bool whole_rows(const void* p, uint64_t width, uint64_t e) { return width * e % kPieceK == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; }
static XentWorkspace xent_carve(void* ws, int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width, size_t* total) {
  const uint64_t e = dtype == LAPLEX_BF16 ? 2 : 4;
  const XentPlan p = xent_plan(dtype, tokens, vocab, width);
  Carver c(ws);
  XentWorkspace w{};
  w.x_rows = c.take<void>(tokens * p.k_width * e);
  w.table_rows = c.take<void>(vocab * p.k_width * e);
  if (pass == 0) {
    w.stats = c.take<float2>((uint64_t)tiles(vocab, TileS::BM) * tokens * 8);
    w.hit = c.take<float>(tokens * 4);
  } else {
    // (a piece has at most kPiece bytes, or one tile of the vocabulary, or all of it)
    const uint64_t bk = kPieceK / e, g = std::max<uint64_t>(std::min<uint64_t>(kPiece / 2, up(vocab, bk) * p.k_tokens * e), kTile * p.k_tokens * e);
    w.G = c.take<void>(g);
    w.Gt = c.take<void>(g);
    w.x_t = c.take<void>(width * p.k_tokens * e);
    w.table_t = c.take<void>((uint64_t)width * up(vocab, bk) * e);
    w.dx = c.take<float>((std::min<uint64_t>(tokens * 513, tokens + 512 * kTile)) * width * 4);
  }
  *total = (c.off + 255) & ~size_t(255);
  return w;
}
size_t xent_bytes(int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width) {
  size_t total = 0;
  xent_carve(nullptr, pass, dtype, tokens, vocab, width, &total);
  return total;
}

template <typename T, typename C>
static hipError_t product_of(const char* name, int epi, ProductArgs& a, hipStream_t s) {
  a.tiles_m = tiles(a.M, C::BM);
  a.tiles_n = tiles(epi == XENT_GRAD ? std::max(a.N, a.n_fill) : a.N, C::BN);
  const uint64_t blocks = (uint64_t)a.tiles_m * a.tiles_n * a.splits;
  LAPLEX_LAUNCH(name, blocks, s, {
    if (epi == XENT_STATS) k_product<T, XENT_STATS, C><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
    else if (epi == XENT_GRAD) k_product<T, XENT_GRAD, C><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
    else k_product<T, XENT_OUT, C><<<(unsigned)blocks, C::THREADS, 0, s>>>(a);
  });
  return hipGetLastError();
}
template <typename T>
static hipError_t product(const char* name, int epi, ProductArgs& a, uint32_t splits, hipStream_t s) {
  constexpr uint64_t bk = kPieceK / sizeof(T);
  a.k_split = std::max(bk, up((a.K + splits - 1) / splits, bk));
  a.splits = (uint32_t)std::max<uint64_t>(1, (a.K + a.k_split - 1) / a.k_split);
  const uint64_t l = (uint64_t)tiles(a.M, 256) * tiles(a.N, 256) * a.splits, m = (uint64_t)tiles(a.M, 128) * tiles(a.N, 128) * a.splits;
  if (a.N <= 32) return product_of<T, TileT>(name, epi, a, s);
  if (l >= 200) return product_of<T, TileL>(name, epi, a, s);
  if (m >= 200) return product_of<T, TileM>(name, epi, a, s);
  return product_of<T, TileS>(name, epi, a, s);
}
static unsigned some_blocks(uint64_t n) { return (unsigned)std::min<uint64_t>((n + 255) / 256, 16384); }

// x and the table with rows of whole pieces
template <typename T>
static hipError_t whole(const void** p, uint64_t rows, uint32_t width, uint64_t k, void* copy, hipStream_t s) {
  if (whole_rows(*p, width, sizeof(T))) return hipSuccess;
  LAPLEX_LAUNCH("k_xent_rows", rows, s,
                k_xent_rows<T><<<some_blocks(rows * k), 256, 0, s>>>(static_cast<const T*>(*p), rows, width, (uint32_t)k, static_cast<T*>(copy)));
  *p = copy;
  return hipGetLastError();
}
template <typename T>
static hipError_t forward(const XentShape& x, float* loss, float* lse, void* ws, hipStream_t s) {
  size_t total;
  const XentPlan p = xent_plan(x.dtype, x.tokens, x.vocab, x.width);
  const XentWorkspace w = xent_carve(ws, 0, x.dtype, x.tokens, x.vocab, x.width, &total);
  ProductArgs a{};
  a.A = x.table;
  a.B = x.x;
  hipError_t err;
  if ((err = whole<T>(&a.A, x.vocab, x.width, p.k_width, w.table_rows, s)) != hipSuccess) return err;
  if ((err = whole<T>(&a.B, x.tokens, x.width, p.k_width, w.x_rows, s)) != hipSuccess) return err;
  a.lda = a.ldb = (int64_t)p.k_width;
  a.K = p.k_width;
  a.M = x.vocab;
  a.N = (uint32_t)x.tokens;
  a.targets = x.targets;
  a.id_bytes = x.id_bytes;
  a.vocab = x.vocab;
  a.scale = x.scale;
  a.stats = w.stats;
  a.hit = w.hit;
  if ((err = product<T>("k_product_stats", XENT_STATS, a, 1, s)) != hipSuccess) return err;
  LAPLEX_LAUNCH("k_xent_join", x.tokens, s,
                k_xent_join<<<(unsigned)((x.tokens + 15) / 16), 256, 0, s>>>(w.stats, a.tiles_m, a.N, w.hit, x.targets, x.id_bytes, x.vocab, loss, lse));
  return hipGetLastError();
}
template <typename T>
static hipError_t transposed(const void* src, uint64_t rows, uint32_t cols, uint64_t fill, void* dst, const XentShape* tokens, hipStream_t s) {
  const uint64_t blocks = (fill + 63) / 64 * ((cols + 63) / 64);
  LAPLEX_LAUNCH("k_xent_transposed", rows, s,
                k_xent_transposed<T><<<(unsigned)blocks, 256, 0, s>>>(static_cast<const T*>(src), (uint32_t)rows, cols, (uint32_t)fill, static_cast<T*>(dst),
                                                                      tokens ? tokens->targets : nullptr, tokens ? tokens->id_bytes : 0, tokens ? tokens->vocab : 0));
  return hipGetLastError();
}
template <typename T>
static hipError_t backward(const XentShape& x, const float* lse, const float* dloss, const float* dlse, void* dx, int table_dtype,
                           void* dtable, void* ws, hipStream_t s) {
  size_t total;
  const XentPlan p = xent_plan(x.dtype, x.tokens, x.vocab, x.width);
  const XentWorkspace w = xent_carve(ws, 1, x.dtype, x.tokens, x.vocab, x.width, &total);
  const uint32_t tokens = (uint32_t)x.tokens;
  ProductArgs l{};
  l.A = x.table;
  l.B = x.x;
  hipError_t err;
  if (tokens) {  // (without, dtable is a sum of nothing)
    if ((err = whole<T>(&l.A, x.vocab, x.width, p.k_width, w.table_rows, s)) != hipSuccess) return err;
    if ((err = whole<T>(&l.B, x.tokens, x.width, p.k_width, w.x_rows, s)) != hipSuccess) return err;
    if (dtable && (err = transposed<T>(x.x, x.tokens, x.width, p.k_tokens, w.x_t, &x, s)) != hipSuccess) return err;
  } else {
    dx = nullptr;
  }
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
  l.Gt = w.Gt;
  l.ldgt = (int64_t)p.k_tokens;
  l.n_fill = (uint32_t)p.k_tokens;
  const char* table = static_cast<const char*>(l.A);
  const bool once = p.splits == 1 && p.piece >= x.vocab;  // dx is one product
  uint32_t used = 1;
  for (uint32_t v0 = 0; v0 < x.vocab; v0 += p.piece) {
    const uint32_t n = std::min(p.piece, x.vocab - v0);
    const uint64_t fill = up(n, kPieceK / sizeof(T));
    l.A = table + (uint64_t)v0 * p.k_width * sizeof(T);
    l.M = n;
    l.v0 = v0;
    l.ldg = (int64_t)fill;
    l.m_fill = (uint32_t)fill;
    if (tokens && (err = product<T>("k_product_grad", XENT_GRAD, l, 1, s)) != hipSuccess) return err;
    if (dx) {
      if ((err = transposed<T>(static_cast<const T*>(x.table) + (uint64_t)v0 * x.width, n, x.width, fill, w.table_t, nullptr, s)) != hipSuccess) return err;
      ProductArgs a{};
      a.A = w.table_t;
      a.B = w.G;
      a.lda = a.ldb = (int64_t)fill;
      a.K = fill;
      a.M = x.width;
      a.N = tokens;
      a.targets = x.targets;
      a.id_bytes = x.id_bytes;
      a.vocab = x.vocab;
      a.live_rows = true;
      a.ldo = x.width;
      a.out = once ? dx : w.dx;
      a.out_f32 = !once || sizeof(T) == 4;
      a.out_split = (int64_t)x.tokens * x.width;
      a.add = v0 > 0;
      if ((err = product<T>("k_product_dx", XENT_OUT, a, p.splits, s)) != hipSuccess) return err;
      used = std::max(used, a.splits);
    }
    if (dtable) {
      ProductArgs a{};
      a.A = w.x_t;
      a.B = w.Gt;
      a.lda = a.ldb = (int64_t)p.k_tokens;
      a.K = p.k_tokens;
      a.M = x.width;
      a.N = n;
      a.ldo = x.width;
      a.out_f32 = table_dtype == LAPLEX_F32;
      a.out = static_cast<char*>(dtable) + (uint64_t)v0 * x.width * (a.out_f32 ? 4 : 2);
      if ((err = product<T>("k_product_dtable", XENT_OUT, a, 1, s)) != hipSuccess) return err;
    }
  }
  if (dx && !once) {
    const uint64_t n = x.tokens * x.width;
    LAPLEX_LAUNCH("k_xent_sum", n, s, k_xent_sum<T><<<some_blocks(n), 256, 0, s>>>(w.dx, used, n, static_cast<T*>(dx)));
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
