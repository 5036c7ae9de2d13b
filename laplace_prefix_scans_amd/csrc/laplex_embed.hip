// Embedding lookup and its gradient by sorted tokens.
//
// Forward: y_t = scale table[id_t], a copy of rows, bound by HBM (16384 tokens,
// 65536 x 2048 bfloat16, ids as frequent as words are: 26 us for 67 MB written and
// 42 MB read).
// Backward: the tokens are sorted by id (stable), so a table row's terms are a
// stretch of the sorted order; stretches are cut into chunks of kEmbedChunk
// tokens so that a frequent id is added by many blocks.  A stretch inside
// one chunk is written at once; one over several chunks leaves a float32
// partial row per chunk, and a second launch adds those in order.  Rows
// without a token are zeroed by the same launch that adds the chunks, so every
// element of the gradient is written once and nothing is cleared first; where the general sort gave up, that launch
// writes NaN to every row and nothing reads the undefined order (the
// same size: 67 us for 66 MB read and 272 MB written, 5.0 TB/s; the sort
// 16 us, the partials 12 us).
#include "laplex_layers.hpp"
#include "laplex_layers_device.hpp"

namespace laplex {

constexpr int kEmbedBlock = 256;
constexpr size_t kEmbedLong = 2560;  // bytes from which rows that are not whole aligned pieces are moved in 16 bytes
constexpr int kEmbedZeroRows = 8;  // table rows a thread group looks at for zeroing

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, uint64_t t) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
}

// Rows are moved in pieces of E elements.  WHOLE: they are 16 bytes, aligned and whole.  Otherwise they are read and
// written at the alignment of an element: long rows in 16 bytes too, of which a row's last begin E elements before its
// end (two threads then form and write the same values in some columns), short ones an element a thread, for there the
// threads on the way count.  Lookup and gradient, 16384 tokens: 65536 x 2047 bfloat16 166 us, by elements 272; 5000 x
// 1001 float 61 and 65; but 257 x 513 float, 4096 tokens, 25.6 and 24, and 23748 x 107, 17368 tokens, 45 and 36.
template <int E, bool WHOLE>
__device__ __forceinline__ uint32_t piece_at(uint32_t c, uint32_t width) {
  return WHOLE || width < (uint32_t)E ? c : min(c, width - E);
}
template <typename T, int E, bool WHOLE>
struct Piece {
  T e[E];
  __device__ __forceinline__ void load(const T* p, uint32_t left) {
    if constexpr (WHOLE) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      __builtin_memcpy(e, &q, 16);
    } else if (left >= (uint32_t)E) {
      __builtin_memcpy(e, p, sizeof(e));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) e[j] = j < (int)left ? p[j] : T(0.f);
    }
  }
};
template <typename O, int E, bool WHOLE>
__device__ __forceinline__ void store_row(O* p, const float (&v)[E], float scale, uint32_t left) {
  O o[E];
#pragma unroll
  for (int j = 0; j < E; ++j) o[j] = from_f32<O>(scale * v[j]);
  if constexpr (WHOLE) {
    uint4 q[E * sizeof(O) / 16];
    __builtin_memcpy(q, o, E * sizeof(O));
#pragma unroll
    for (int i = 0; i < (int)(E * sizeof(O) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = q[i];
  } else if (left >= (uint32_t)E) {
    __builtin_memcpy(p, o, E * sizeof(O));
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < (int)left) p[j] = o[j];
  }
}

// Thread per piece of a row; `lanes` threads share a token and step over its pieces.
template <typename T, int E, bool WHOLE>
__global__ __launch_bounds__(kEmbedBlock) void k_embed(const void* __restrict__ ids, int id_bytes, uint64_t tokens,
                                                       const T* __restrict__ table, uint32_t vocab, uint32_t width, float scale,
                                                       T* __restrict__ y, uint32_t lanes) {
  const uint32_t per = kEmbedBlock / lanes;
  for (uint64_t t = (uint64_t)blockIdx.x * per + threadIdx.x / lanes; t < tokens; t += (uint64_t)gridDim.x * per) {
    const int64_t id = load_id(ids, id_bytes, t);
    const bool live = id >= 0 && id < (int64_t)vocab;
    for (uint32_t c0 = threadIdx.x % lanes * E; c0 < width; c0 += lanes * E) {
      const uint32_t c = piece_at<E, WHOLE>(c0, width);
      float v[E];
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = 0.f;
      if (live) {
        Piece<T, E, WHOLE> p;
        p.load(table + (uint64_t)id * width + c, width - c);
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = to_f32(p.e[j]);
      }
      store_row<T, E, WHOLE>(y + t * width + c, v, live ? scale : 0.f, width - c);
    }
  }
}

// Sort keys.  Any order that brings equal ids together will do, and frequent
// ids are often neighbours (a vocabulary in order of frequency), so an id's 6
// lowest bits become its key's highest: key ranges of equal size then hold
// about as many tokens.  Keys have `bits` bits; ids outside the table get the
// key 2^bits, behind every row.
constexpr int kTopBits = 6, kTops = 1 << kTopBits;
__host__ __device__ __forceinline__ int key_bits(uint32_t vocab) {
  int b = kTopBits;
  while ((1u << b) < vocab) ++b;
  return b;
}
__device__ __forceinline__ uint32_t key_of(int64_t id, uint32_t vocab, int bits) {
  if (id < 0 || id >= (int64_t)vocab) return 1u << bits;
  return ((uint32_t)id & (kTops - 1)) << (bits - kTopBits) | (uint32_t)id >> kTopBits;
}
__device__ __forceinline__ uint32_t row_of(uint32_t key, int bits) {
  return (key & ((1u << (bits - kTopBits)) - 1)) << kTopBits | key >> (bits - kTopBits);
}

__global__ void k_embed_keys(const void* __restrict__ ids, int id_bytes, uint64_t tokens, uint32_t vocab, int bits,
                             uint32_t* __restrict__ keys) {
  const uint64_t t = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (t < tokens) keys[t] = key_of(load_id(ids, id_bytes, t), vocab, bits);
}

// Stable sort of a tile of up to kEmbedSmall tokens by key in one launch: block b reads
// all of them, takes those of the key range b (range kTops: outside the table)
// in order, counts those of the ranges before it -- where its part of the
// result starts -- and sorts its own in LDS by the remaining bits (stable LSD
// passes of 6), and for vocabularies up to 2^kFindBits writes its keys' first
// positions too.  No block waits for another.  A whole gradient over 16384
// tokens (65536 x 128) takes 36 us with the lookup, 66 with the general sort's
// nine launches in place of this one; over 4096 tokens (257 x 513) 24 and 51.
// More tokens are sorted in tiles of kEmbedSmall and joined (k_embed_merge).
constexpr int kFindBits = 18, kEmbedTiles = 8;
constexpr int kEmbedSmall = 16384, kSortThreads = 1024, kSortWaves = kSortThreads / kWave, kSortBits = 6, kSortBins = 1 << kSortBits;

// lanes whose digit is this lane's
__device__ __forceinline__ uint64_t peers6(uint32_t d) {
  uint64_t peers = ~0ull;
#pragma unroll
  for (int b = 0; b < kSortBits; ++b) {
    const uint64_t m = __ballot((d >> b) & 1);
    peers &= (d >> b) & 1 ? m : ~m;
  }
  return peers;
}

// LDS written by one lane and read by another of the same wave
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int E>
__global__ __launch_bounds__(kSortThreads) void k_embed_sort(const void* __restrict__ ids, int id_bytes, uint32_t all, uint32_t vocab,
                                                             int bits, uint32_t* __restrict__ keys, uint32_t* __restrict__ perm,
                                                             uint32_t* __restrict__ starts) {
  const uint32_t t0 = blockIdx.y * kEmbedSmall, tokens = min(all - t0, (uint32_t)kEmbedSmall);
  keys += t0;
  perm += t0;
  if (starts) starts += (uint64_t)blockIdx.y * ((1u << bits) + 1);
  __shared__ uint32_t sk[E * kSortThreads];
  __shared__ uint16_t sp[E * kSortThreads];
  __shared__ uint32_t count[kSortWaves][kSortBins];
  __shared__ uint32_t base[kSortBins], mine[kSortWaves], below[kSortWaves];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int low = bits - kTopBits;
  uint32_t k[E], v[E];
  uint32_t in = 0, under = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {  // wave w reads [w * 64 E, (w + 1) * 64 E)
    const uint32_t at = (wave * E + e) * kWave + lane;
    k[e] = at < tokens ? key_of(load_id(ids, id_bytes, (uint64_t)t0 + at), vocab, bits) : 0xFFFFFFFFu;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t at = (wave * E + e) * kWave + lane;
    in += (uint32_t)__popcll(__ballot(at < tokens && k[e] >> low == blockIdx.x));
    under += (uint32_t)__popcll(__ballot(at < tokens && k[e] >> low < blockIdx.x));
  }
  if (lane == 0) {
    mine[wave] = in;
    below[wave] = under;
  }
  __syncthreads();
  uint32_t start = 0, m = 0, to = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    to += w < wave ? mine[w] : 0;
    m += mine[w];
    start += below[w];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t at = (wave * E + e) * kWave + lane;
    const bool own = at < tokens && k[e] >> low == blockIdx.x;
    const uint64_t b = __ballot(own);
    if (own) {
      sk[to + lanes_below(b)] = k[e];
      sp[to + lanes_below(b)] = (uint16_t)at;
    }
    to += (uint32_t)__popcll(b);
  }
  const int per = (int)((m + kSortThreads - 1) / kSortThreads);  // of the m taken, wave w holds [w * 64 per, (w + 1) * 64 per)
  const bool one_key = blockIdx.x == kTops;
  for (int shift = 0; shift < low && !one_key; shift += kSortBits) {
    __syncthreads();
    count[wave][lane] = 0;  // a wave's own row
    wave_sync();
    uint32_t rank[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (e >= per) break;
      const uint32_t at = (wave * per + e) * kWave + lane;
      k[e] = at < m ? sk[at] : 0xFFFFFFFFu;  // past the end: behind every key of the range
      v[e] = at < m ? sp[at] : 0;
      const uint32_t d = at < m ? (k[e] >> shift) & (kSortBins - 1) : kSortBins - 1;
      const uint64_t peers = peers6(d);
      const uint32_t before = count[wave][d];
      rank[e] = before + lanes_below(peers);
      wave_sync();
      if (lanes_below(peers) == 0) count[wave][d] = before + (uint32_t)__popcll(peers);
      wave_sync();
    }
    __syncthreads();
    if (threadIdx.x < kSortBins) {  // one wave: totals over the waves, then their exclusive scan over the digits
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = count[w][lane];
        count[w][lane] = sum;
        sum += c;
      }
      base[lane] = wave_incl_sum_u32(sum) - sum;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (e >= per) break;
      const uint32_t at = (wave * per + e) * kWave + lane;
      if (at >= m) continue;
      const uint32_t d = (k[e] >> shift) & (kSortBins - 1), dst = base[d] + count[wave][d] + rank[e];
      sk[dst] = k[e];
      sp[dst] = (uint16_t)v[e];
    }
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < m; i += kSortThreads) {
    keys[start + i] = sk[i];
    perm[start + i] = t0 + sp[i];
  }
  if (!starts) return;
  // the first position of each key of the range
  const uint32_t k0 = blockIdx.x << low, n = one_key ? 1 : 1u << low;
  for (uint32_t i = threadIdx.x; i < n; i += kSortThreads) {
    uint32_t lo = 0, hi = m;
    while (lo < hi) {
      const uint32_t mid = (lo + hi) / 2;
      if (sk[mid] < k0 + i) lo = mid + 1;
      else hi = mid;
    }
    starts[k0 + i] = start + lo;
  }
}

// Joins sorted tiles: an element's place is its place among its tile's equal keys, behind all smaller keys and the
// equal ones of earlier tiles.  The tiles' starts give every term, so an element needs no search; the last blocks
// add them up to the starts of the whole.
__global__ __launch_bounds__(256) void k_embed_merge(const uint32_t* __restrict__ tile_keys, const uint32_t* __restrict__ tile_perm,
                                                     const uint32_t* __restrict__ tile_starts, uint32_t tokens, uint32_t tiles, int bits,
                                                     uint32_t* __restrict__ keys, uint32_t* __restrict__ perm, uint32_t* __restrict__ starts) {
  const uint32_t n = 1u << bits, blocks = (tokens + 255) / 256;
  if (blockIdx.x >= blocks) {
    const uint32_t u = (blockIdx.x - blocks) * 256 + threadIdx.x;
    if (u > n) return;
    uint32_t s = 0;
    for (uint32_t j = 0; j < tiles; ++j) s += tile_starts[(uint64_t)j * (n + 1) + u];
    starts[u] = s;
    return;
  }
  const uint32_t p = blockIdx.x * 256 + threadIdx.x;
  if (p >= tokens) return;
  const uint32_t tile = p / kEmbedSmall, u = tile_keys[p];
  uint32_t to = p % kEmbedSmall;
  for (uint32_t j = 0; j < tiles; ++j) {
    const uint32_t* st = tile_starts + (uint64_t)j * (n + 1) + u;
    const uint32_t first = st[0];
    if (j < tile) to += u < n ? st[1] : min(tokens - j * kEmbedSmall, (uint32_t)kEmbedSmall);  // all up to its equal keys
    else if (j > tile) to += first;
  }
  keys[to] = u;
  perm[to] = tile_perm[p];
}

// starts[u] = first sorted position whose key is >= u, for u = 0 .. 2^bits.
__global__ void k_embed_starts(const uint32_t* __restrict__ keys, uint64_t tokens, int bits, uint32_t* __restrict__ starts) {
  const uint64_t u = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (u > (1ull << bits)) return;
  uint64_t lo = 0, hi = tokens;
  while (lo < hi) {
    const uint64_t mid = (lo + hi) / 2;
    if (keys[mid] < u) lo = mid + 1;
    else hi = mid;
  }
  starts[u] = (uint32_t)lo;
}

struct EmbedGrad {
  const uint32_t *keys, *perm, *starts;
  uint64_t tokens;
  uint32_t vocab, width, chunk, lanes;
  int bits;  // of a key
  uint64_t chunk_blocks;  // blocks of the chunks; the rest zero rows
  float scale;
  float* part;  // [chunk][0: the stretch begun earlier, 1: the one that goes on][width]
  const uint32_t* stop;  // set where the general sort gave up (its keys and places are then undefined), or null
  __device__ __forceinline__ bool stalled() const { return stop && *stop != 0; }
};

template <typename T, typename O, int E, bool WHOLE>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_grad(EmbedGrad g, const T* __restrict__ dy, O* __restrict__ dtable) {
  const uint32_t groups = kEmbedBlock / g.lanes, group = threadIdx.x / g.lanes;
  const uint32_t c0 = (blockIdx.y * g.lanes + threadIdx.x % g.lanes) * E;
  if (c0 >= g.width) return;
  const uint32_t c = piece_at<E, WHOLE>(c0, g.width), left = g.width - c;
  const bool stalled = g.stalled();
  if (blockIdx.x >= g.chunk_blocks) {
    const uint64_t v0 = ((blockIdx.x - g.chunk_blocks) * groups + group) * kEmbedZeroRows;
    float none[E];
#pragma unroll
    for (int j = 0; j < E; ++j) none[j] = stalled ? __builtin_nanf("") : 0.f;
    for (uint64_t v = v0; v < v0 + kEmbedZeroRows && v < g.vocab; ++v) {
      const uint32_t u = key_of((int64_t)v, g.vocab, g.bits);
      if (stalled || g.starts[u] == g.starts[u + 1]) store_row<O, E, WHOLE>(dtable + v * g.width + c, none, 1.f, left);
    }
    return;
  }
  if (stalled) return;
  const uint64_t ch = (uint64_t)blockIdx.x * groups + group, p0 = ch * g.chunk;
  if (p0 >= g.tokens) return;
  const uint64_t p1 = min(p0 + g.chunk, g.tokens);
  uint32_t cur = g.keys[p0];
  bool head = p0 > 0 && g.keys[p0 - 1] == cur;
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.f;
  auto flush = [&](bool goes_on) {
    if (cur >> g.bits) return;  // outside the table
    if (head || goes_on) store_row<float, E, WHOLE>(g.part + (ch * 2 + (head ? 0 : 1)) * g.width + c, acc, 1.f, left);
    else store_row<O, E, WHOLE>(dtable + (uint64_t)row_of(cur, g.bits) * g.width + c, acc, g.scale, left);
  };
  constexpr int B = 8;  // rows in flight
  for (uint64_t q = p0; q < p1; q += B) {
    uint32_t key[B];
    Piece<T, E, WHOLE> row[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const uint64_t at = min(q + i, p1 - 1);
      key[i] = g.keys[at];
      row[i].load(dy + (uint64_t)g.perm[at] * g.width + c, left);
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
  if (p1 >= g.tokens || g.stalled()) return;
  const uint32_t u = g.keys[p1 - 1];
  if (u >> g.bits || g.keys[p1] != u || g.starts[u] < p0) return;
  const uint64_t last = ((uint64_t)g.starts[u + 1] - 1) / g.chunk, v = row_of(u, g.bits);
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
      dtable[v * g.width + c] = from_f32<O>(g.scale * (sh[0][threadIdx.x] + sh[1][threadIdx.x] + sh[2][threadIdx.x] + sh[3][threadIdx.x]));
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

template <typename T, int E, bool WHOLE>
static void embed_launch(const void* ids, int id_bytes, uint64_t tokens, const void* table, uint32_t vocab, uint32_t width,
                         float scale, void* y, hipStream_t s) {
  const uint32_t lanes = embed_lanes((width + E - 1) / E), per = kEmbedBlock / lanes;
  k_embed<T, E, WHOLE><<<(unsigned)std::min<uint64_t>((tokens + per - 1) / per, 1u << 20), kEmbedBlock, 0, s>>>(ids, id_bytes, tokens, (const T*)table, vocab, width,
                                                                            scale, (T*)y, lanes);
}

hipError_t embedding(int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* table, uint32_t vocab, uint32_t width,
                     float scale, void* y, hipStream_t s) {
  const size_t e = dtype == LAPLEX_BF16 ? 2 : 4;
  const bool vec = embed_vec(width, e, e, {table, y}), wide = width * e >= kEmbedLong;
  auto run = [&](auto f) { f(ids, id_bytes, tokens, table, vocab, width, scale, y, s); };
  LAPLEX_LAUNCH("k_embed", tokens, s, {
    if (dtype == LAPLEX_BF16) run(vec ? embed_launch<bf16, 8, true> : wide ? embed_launch<bf16, 8, false> : embed_launch<bf16, 1, false>);
    else run(vec ? embed_launch<float, 4, true> : wide ? embed_launch<float, 4, false> : embed_launch<float, 1, false>);
  });
  return hipGetLastError();
}

// Tokens of a chunk.  Gradient with chunks of 32 and of 64: 4096 tokens, 257 x 513 float, 16.5 us and 18.7; 16384,
// 65536 x 128 bfloat16, 30 and 35, but 65536 x 2048 93 and 87; 32768, 65536 x 512, 44.7 and 45.1; 65536, the same,
// 64 and 57; 131072, 5000 x 1024, 144 and 114 (with 128: 99).
constexpr uint64_t kEmbedShort = 32768;
uint32_t embed_chunk(uint64_t tokens) { return tokens <= kEmbedShort ? 32 : 64; }
uint64_t embed_starts(uint32_t vocab) { return (1ull << key_bits(vocab)) + 1; }
// The general sort takes seven to nine launches whatever the size; tiles take two, and reads of every tile's starts
// by every token (lookup and gradient, 49625 tokens, 58298 x 136: 82 -> 53 us; 131072 tokens, 65536 x 64: 88 -> 74).
constexpr uint64_t kEmbedTiled = kEmbedTiles * (uint64_t)kEmbedSmall;
uint64_t embed_tiled_most(uint64_t tokens, uint32_t vocab) {
  return tokens > (uint64_t)kEmbedSmall && key_bits(vocab) <= kFindBits ? std::min(tokens, kEmbedTiled) : 0;
}
uint32_t embed_tiles_of(uint64_t tiled) { return (uint32_t)((tiled + kEmbedSmall - 1) / kEmbedSmall); }
uint32_t embed_tiles(uint64_t tokens, uint32_t vocab) {
  return tokens <= kEmbedTiled ? embed_tiles_of(embed_tiled_most(tokens, vocab)) : 0;
}
uint64_t embed_part_floats(uint64_t tokens, uint32_t width) {
  auto chunks = [](uint64_t n) { return (n + embed_chunk(n) - 1) / embed_chunk(n); };
  return std::max(chunks(tokens), chunks(std::min(tokens, kEmbedShort))) * 2 * width;
}

template <typename T, typename O, int E, bool WHOLE>
static void embed_grad_launch(EmbedGrad g, const void* dy, void* dtable, hipStream_t s) {
  const uint32_t pieces = (g.width + E - 1) / E;
  g.lanes = embed_lanes(pieces);
  const uint32_t groups = kEmbedBlock / g.lanes;
  const uint64_t chunks = (g.tokens + g.chunk - 1) / g.chunk;
  g.chunk_blocks = (chunks + groups - 1) / groups;
  const uint64_t zero_blocks = ((uint64_t)g.vocab + groups * kEmbedZeroRows - 1) / (groups * kEmbedZeroRows);
  const dim3 grid((unsigned)(g.chunk_blocks + zero_blocks), (pieces + g.lanes - 1) / g.lanes);
  k_embed_grad<T, O, E, WHOLE><<<grid, kEmbedBlock, 0, s>>>(g, (const T*)dy, (O*)dtable);
  if (chunks > 1) {
    const dim3 jgrid((unsigned)(chunks - 1), std::min<uint32_t>((g.width + 63) / 64, 32));
    k_embed_join<O><<<jgrid, kEmbedBlock, 0, s>>>(g, (O*)dtable);
  }
}

hipError_t embedding_backward(const EmbedWorkspace& w, int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* dy,
                              uint32_t vocab, uint32_t width, float scale, int table_dtype, void* dtable, hipStream_t s) {
  hipError_t e;
  const int bits = key_bits(vocab);
  const uint32_t tiles = embed_tiles(tokens, vocab);
  const uint32_t* stop = nullptr;
  uint32_t* starts = tiles || (tokens && tokens <= (uint64_t)kEmbedSmall && bits <= kFindBits) ? w.starts : nullptr;  // found by the sort
  if (tiles) {
    const uint32_t n = (uint32_t)tokens;
    LAPLEX_LAUNCH("k_embed_sort", tokens, s,
                  k_embed_sort<16><<<dim3(kTops + 1, tiles), kSortThreads, 0, s>>>(ids, id_bytes, n, vocab, bits, w.keys, w.tile_perm, w.tile_starts));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    LAPLEX_LAUNCH("k_embed_merge", tokens, s,
                  k_embed_merge<<<(n + 255) / 256 + (1u << bits) / 256 + 1, 256, 0, s>>>(w.keys, w.tile_perm, w.tile_starts, n, tiles, bits, w.keys_s, w.perm, starts));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else if (tokens && tokens <= (uint64_t)kEmbedSmall) {
    LAPLEX_LAUNCH("k_embed_sort", tokens, s, {
      const uint32_t n = (uint32_t)tokens;
      if (n <= kSortThreads) k_embed_sort<1><<<kTops + 1, kSortThreads, 0, s>>>(ids, id_bytes, n, vocab, bits, w.keys_s, w.perm, starts);
      else if (n <= 4 * kSortThreads) k_embed_sort<4><<<kTops + 1, kSortThreads, 0, s>>>(ids, id_bytes, n, vocab, bits, w.keys_s, w.perm, starts);
      else k_embed_sort<16><<<kTops + 1, kSortThreads, 0, s>>>(ids, id_bytes, n, vocab, bits, w.keys_s, w.perm, starts);
    });
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else if (tokens) {
    LAPLEX_LAUNCH("k_embed_keys", tokens, s,
                  k_embed_keys<<<(unsigned)((tokens + 255) / 256), 256, 0, s>>>(ids, id_bytes, tokens, vocab, bits, w.keys));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = sort_indices(w.sort, w.keys, tokens, 1u << bits, w.keys_s, w.perm, s)) != hipSuccess) return e;
    stop = w.sort.header + kHdrStop;
  }
  if (!starts)
    LAPLEX_LAUNCH("k_embed_starts", vocab, s, k_embed_starts<<<(1u << bits) / 256 + 1, 256, 0, s>>>(w.keys_s, tokens, bits, w.starts));
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const size_t te = table_dtype == LAPLEX_BF16 ? 2 : 4;
  const size_t de = dtype == LAPLEX_BF16 ? 2 : 4;
  const bool vec = embed_vec(width, de, te, {dy, dtable}), wide = width * de >= kEmbedLong;
  const EmbedGrad g{w.keys_s, w.perm, w.starts, tokens, vocab, width, embed_chunk(tokens), 0, bits, 0, scale, w.part, stop};
  auto run = [&](auto f) { f(g, dy, dtable, s); };
  LAPLEX_LAUNCH("k_embed_grad", tokens, s, {
    if (dtype != LAPLEX_BF16)
      run(vec ? embed_grad_launch<float, float, 4, true> : wide ? embed_grad_launch<float, float, 4, false> : embed_grad_launch<float, float, 1, false>);
    else if (table_dtype == LAPLEX_F32)
      run(vec ? embed_grad_launch<bf16, float, 8, true> : wide ? embed_grad_launch<bf16, float, 8, false> : embed_grad_launch<bf16, float, 1, false>);
    else
      run(vec ? embed_grad_launch<bf16, bf16, 8, true> : wide ? embed_grad_launch<bf16, bf16, 8, false> : embed_grad_launch<bf16, bf16, 1, false>);
  });
  return hipGetLastError();
}

}  // namespace laplex
