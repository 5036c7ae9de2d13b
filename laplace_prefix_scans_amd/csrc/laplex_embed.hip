// Embedding lookup and its gradient by sorted tokens.
//
// Forward: y_t = scale table[id_t], a copy of rows, bound by HBM.
// Backward: the tokens are sorted by id (stable), so a table row's terms are a
// stretch of the sorted order; stretches are cut into chunks of kEmbedChunk
// tokens so that a frequent id is added by many blocks.  A stretch inside
// one chunk is written at once; one over several chunks leaves a float32
// partial row per chunk, and a second launch adds those in order.  Rows
// without a token are zeroed by the same launch that adds the chunks, so every
// element of the gradient is written once and nothing is cleared first.
#include "laplex_layers.hpp"
#include "laplex_layers_device.hpp"

namespace laplex {

constexpr int kEmbedBlock = 256;
constexpr int kEmbedZeroRows = 8;  // table rows a thread group looks at for zeroing

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, uint64_t t) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
}

// `E` consecutive elements where rows are 16-byte aligned, else one
template <typename T, int E>
struct Piece {
  T e[E];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (E > 1) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      __builtin_memcpy(e, &q, 16);
    } else {
      e[0] = *p;
    }
  }
};
template <typename O, int E>
__device__ __forceinline__ void store_row(O* p, const float (&v)[E], float scale) {
  O o[E];
#pragma unroll
  for (int j = 0; j < E; ++j) o[j] = from_f32<O>(scale * v[j]);
  if constexpr (E == 1) {
    *p = o[0];
  } else {
    uint4 q[(E * sizeof(O) + 15) / 16];
    __builtin_memcpy(q, o, E * sizeof(O));
#pragma unroll
    for (int i = 0; i < (int)(E * sizeof(O) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = q[i];
  }
}

// Thread per piece of a row; `lanes` threads share a token and step over its pieces.
template <typename T, int E>
__global__ __launch_bounds__(kEmbedBlock) void k_embed(const void* __restrict__ ids, int id_bytes, uint64_t tokens,
                                                       const T* __restrict__ table, uint32_t vocab, uint32_t width, float scale,
                                                       T* __restrict__ y, uint32_t lanes) {
  const uint32_t per = kEmbedBlock / lanes;
  for (uint64_t t = (uint64_t)blockIdx.x * per + threadIdx.x / lanes; t < tokens; t += (uint64_t)gridDim.x * per) {
    const int64_t id = load_id(ids, id_bytes, t);
    const bool live = id >= 0 && id < (int64_t)vocab;
    for (uint32_t c = threadIdx.x % lanes * E; c < width; c += lanes * E) {
      float v[E];
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = 0.f;
      if (live) {
        Piece<T, E> p;
        p.load(table + (uint64_t)id * width + c);
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = to_f32(p.e[j]);
      }
      store_row<T, E>(y + t * width + c, v, live ? scale : 0.f);
    }
  }
}

// Ids as sort keys; those outside the table sort behind every row.
__global__ void k_embed_keys(const void* __restrict__ ids, int id_bytes, uint64_t tokens, uint32_t vocab, uint32_t* __restrict__ keys) {
  const uint64_t t = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= tokens) return;
  const int64_t id = load_id(ids, id_bytes, t);
  keys[t] = (id >= 0 && id < (int64_t)vocab) ? (uint32_t)id : vocab;
}

// starts[v] = first sorted position whose key is >= v, for v = 0 .. vocab.
__global__ void k_embed_starts(const uint32_t* __restrict__ keys, uint64_t tokens, uint32_t vocab, uint32_t* __restrict__ starts) {
  const uint64_t v = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (v > vocab) return;
  uint64_t lo = 0, hi = tokens;
  while (lo < hi) {
    const uint64_t mid = (lo + hi) / 2;
    if (keys[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  starts[v] = (uint32_t)lo;
}

struct EmbedGrad {
  const uint32_t *keys, *perm, *starts;
  uint64_t tokens;
  uint32_t vocab, width, chunk, lanes;
  uint64_t chunk_blocks;  // blocks of the chunks; the rest zero rows
  float scale;
  float* part;  // [chunk][0: the stretch begun earlier, 1: the one that goes on][width]
};

template <typename T, typename O, int E>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_grad(EmbedGrad g, const T* __restrict__ dy, O* __restrict__ dtable) {
  const uint32_t groups = kEmbedBlock / g.lanes, group = threadIdx.x / g.lanes;
  const uint32_t c = (blockIdx.y * g.lanes + threadIdx.x % g.lanes) * E;
  if (c >= g.width) return;
  if (blockIdx.x >= g.chunk_blocks) {
    const uint64_t v0 = ((blockIdx.x - g.chunk_blocks) * groups + group) * kEmbedZeroRows;
    float zero[E];
#pragma unroll
    for (int j = 0; j < E; ++j) zero[j] = 0.f;
    for (uint64_t v = v0; v < v0 + kEmbedZeroRows && v < g.vocab; ++v)
      if (g.starts[v] == g.starts[v + 1]) store_row<O, E>(dtable + v * g.width + c, zero, 0.f);
    return;
  }
  const uint64_t ch = (uint64_t)blockIdx.x * groups + group, p0 = ch * g.chunk;
  if (p0 >= g.tokens) return;
  const uint64_t p1 = min(p0 + g.chunk, g.tokens);
  uint32_t cur = g.keys[p0];
  bool head = p0 > 0 && g.keys[p0 - 1] == cur;
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.f;
  auto flush = [&](bool goes_on) {
    if (cur >= g.vocab) return;
    if (head || goes_on) store_row<float, E>(g.part + (ch * 2 + (head ? 0 : 1)) * g.width + c, acc, 1.f);
    else store_row<O, E>(dtable + (uint64_t)cur * g.width + c, acc, g.scale);
  };
  constexpr int B = 8;  // rows in flight
  for (uint64_t q = p0; q < p1; q += B) {
    uint32_t key[B];
    Piece<T, E> row[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const uint64_t at = min(q + i, p1 - 1);
      key[i] = g.keys[at];
      row[i].load(dy + (uint64_t)g.perm[at] * g.width + c);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (q + i >= p1) break;
      if (key[i] != cur) {
        flush(false);
        cur = key[i];
        head = false;
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] += to_f32(row[i].e[j]);
    }
  }
  flush(p1 < g.tokens && g.keys[p1] == cur);
}

// Adds the partials of a stretch that begins in this block's chunk and goes on: 64 columns of four rows groups.
template <typename O>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_join(EmbedGrad g, O* __restrict__ dtable) {
  __shared__ float sh[4][64];
  const uint64_t ch = blockIdx.x, p0 = ch * g.chunk, p1 = p0 + g.chunk;
  if (p1 >= g.tokens) return;
  const uint32_t v = g.keys[p1 - 1];
  if (v >= g.vocab || g.keys[p1] != v || g.starts[v] < p0) return;
  const uint64_t last = ((uint64_t)g.starts[v + 1] - 1) / g.chunk;
  const uint32_t r = threadIdx.x / 64;
  for (uint32_t c = blockIdx.y * 64 + threadIdx.x % 64; c - threadIdx.x % 64 < g.width; c += gridDim.y * 64) {
    float a = 0.f;
    if (c < g.width) {
      if (r == 0) a = g.part[(ch * 2 + 1) * g.width + c];
#pragma unroll 4
      for (uint64_t k = ch + 1 + r; k <= last; k += 4) a += g.part[k * 2 * g.width + c];
    }
    sh[r][threadIdx.x % 64] = a;
    __syncthreads();
    if (r == 0 && c < g.width)
      dtable[(uint64_t)v * g.width + c] = from_f32<O>(g.scale * (sh[0][threadIdx.x] + sh[1][threadIdx.x] + sh[2][threadIdx.x] + sh[3][threadIdx.x]));
    __syncthreads();
  }
}

// ------------------------------------------------------------------ launches
static bool embed_vec(uint32_t width, size_t e, size_t out, std::initializer_list<const void*> ps) {
  if (width * e % 16 || width * out % 16) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}
// threads that share a row of `pieces`: the power of two that covers it, up to a block
static uint32_t embed_lanes(uint32_t pieces) {
  uint32_t l = 1;
  while (l < pieces && l < (uint32_t)kEmbedBlock) l *= 2;
  return l;
}

template <typename T, int E>
static void embed_launch(const void* ids, int id_bytes, uint64_t tokens, const void* table, uint32_t vocab, uint32_t width,
                         float scale, void* y, hipStream_t s) {
  const uint32_t lanes = embed_lanes((width + E - 1) / E), per = kEmbedBlock / lanes;
  k_embed<T, E><<<(unsigned)std::min<uint64_t>((tokens + per - 1) / per, 1u << 20), kEmbedBlock, 0, s>>>(ids, id_bytes, tokens, (const T*)table, vocab, width,
                                                                            scale, (T*)y, lanes);
}

hipError_t embedding(int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* table, uint32_t vocab, uint32_t width,
                     float scale, void* y, hipStream_t s) {
  const size_t e = dtype == LAPLEX_BF16 ? 2 : 4;
  const bool vec = embed_vec(width, e, e, {table, y});
  LAPLEX_LAUNCH("k_embed", tokens, s, {
    if (dtype == LAPLEX_BF16)
      vec ? embed_launch<bf16, 8>(ids, id_bytes, tokens, table, vocab, width, scale, y, s)
          : embed_launch<bf16, 1>(ids, id_bytes, tokens, table, vocab, width, scale, y, s);
    else
      vec ? embed_launch<float, 4>(ids, id_bytes, tokens, table, vocab, width, scale, y, s)
          : embed_launch<float, 1>(ids, id_bytes, tokens, table, vocab, width, scale, y, s);
  });
  return hipGetLastError();
}

uint32_t embed_chunk(uint64_t tokens) { return tokens <= 32768 ? 32 : 64; }
uint64_t embed_part_floats(uint64_t tokens, uint32_t width) {
  const uint32_t c = embed_chunk(tokens);
  return (tokens + c - 1) / c * 2 * width;
}

template <typename T, typename O, int E>
static void embed_grad_launch(EmbedGrad g, const void* dy, void* dtable, hipStream_t s) {
  const uint32_t pieces = (g.width + E - 1) / E;
  g.lanes = embed_lanes(pieces);
  const uint32_t groups = kEmbedBlock / g.lanes;
  const uint64_t chunks = (g.tokens + g.chunk - 1) / g.chunk;
  g.chunk_blocks = (chunks + groups - 1) / groups;
  const uint64_t zero_blocks = ((uint64_t)g.vocab + groups * kEmbedZeroRows - 1) / (groups * kEmbedZeroRows);
  const dim3 grid((unsigned)(g.chunk_blocks + zero_blocks), (pieces + g.lanes - 1) / g.lanes);
  k_embed_grad<T, O, E><<<grid, kEmbedBlock, 0, s>>>(g, (const T*)dy, (O*)dtable);
  if (chunks > 1) {
    const dim3 jgrid((unsigned)(chunks - 1), std::min<uint32_t>((g.width + 63) / 64, 8));
    k_embed_join<O><<<jgrid, kEmbedBlock, 0, s>>>(g, (O*)dtable);
  }
}

hipError_t embedding_backward(const EmbedWorkspace& w, int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* dy,
                              uint32_t vocab, uint32_t width, float scale, int table_dtype, void* dtable, hipStream_t s) {
  hipError_t e;
  if (tokens) {
    LAPLEX_LAUNCH("k_embed_keys", tokens, s,
                  k_embed_keys<<<(unsigned)((tokens + 255) / 256), 256, 0, s>>>(ids, id_bytes, tokens, vocab, w.keys));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = sort_indices(w.sort, w.keys, tokens, vocab, w.keys_s, w.perm, s)) != hipSuccess) return e;
  }
  LAPLEX_LAUNCH("k_embed_starts", vocab, s, k_embed_starts<<<vocab / 256 + 1, 256, 0, s>>>(w.keys_s, tokens, vocab, w.starts));
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const size_t te = table_dtype == LAPLEX_BF16 ? 2 : 4;
  const bool vec = embed_vec(width, dtype == LAPLEX_BF16 ? 2 : 4, te, {dy, dtable});
  const EmbedGrad g{w.keys_s, w.perm, w.starts, tokens, vocab, width, embed_chunk(tokens), 0, 0, scale, w.part};
  LAPLEX_LAUNCH("k_embed_grad", tokens, s, {
    if (dtype != LAPLEX_BF16)
      vec ? embed_grad_launch<float, float, 4>(g, dy, dtable, s) : embed_grad_launch<float, float, 1>(g, dy, dtable, s);
    else if (table_dtype == LAPLEX_F32)
      vec ? embed_grad_launch<bf16, float, 8>(g, dy, dtable, s) : embed_grad_launch<bf16, float, 1>(g, dy, dtable, s);
    else
      vec ? embed_grad_launch<bf16, bf16, 8>(g, dy, dtable, s) : embed_grad_launch<bf16, bf16, 1>(g, dy, dtable, s);
  });
  return hipGetLastError();
}

}  // namespace laplex
