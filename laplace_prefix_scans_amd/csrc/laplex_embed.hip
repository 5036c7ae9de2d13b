// Embedding lookup and its gradient by sorted tokens.
#include "laplex_layers.hpp"
#include "laplex_layers_device.hpp"

namespace laplex {

constexpr int kEmbedBlock = 256;

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, uint64_t t) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
}

template <typename T>
__global__ __launch_bounds__(kEmbedBlock) void k_embed(const void* __restrict__ ids, int id_bytes, uint64_t tokens,
                                                       const T* __restrict__ table, uint32_t vocab, uint32_t width, float scale,
                                                       T* __restrict__ y) {
  for (uint64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    const int64_t id = load_id(ids, id_bytes, t);
    const bool live = id >= 0 && id < (int64_t)vocab;
    const T* row = table + (uint64_t)(live ? id : 0) * width;
    for (uint32_t i = threadIdx.x; i < width; i += kEmbedBlock)
      y[t * width + i] = from_f32<T>(live ? scale * to_f32(row[i]) : 0.f);
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

template <typename T, typename O>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_grad(const uint32_t* __restrict__ perm, const uint32_t* __restrict__ starts,
                                                            const T* __restrict__ dy, uint32_t vocab, uint32_t width, float scale,
                                                            O* __restrict__ dtable) {
  for (uint64_t v = blockIdx.x; v < vocab; v += gridDim.x) {
    const uint32_t a = starts[v], b = starts[v + 1];
    for (uint32_t i = threadIdx.x; i < width; i += kEmbedBlock) {
      float s = 0.f;
      for (uint32_t j = a; j < b; ++j) s += to_f32(dy[(uint64_t)perm[j] * width + i]);
      dtable[v * width + i] = from_f32<O>(scale * s);
    }
  }
}

hipError_t embedding(int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* table, uint32_t vocab, uint32_t width,
                     float scale, void* y, hipStream_t s) {
  const unsigned blocks = (unsigned)std::min<uint64_t>(tokens, 1u << 20);
  LAPLEX_LAUNCH("k_embed", tokens, s, {
    if (dtype == LAPLEX_BF16)
      k_embed<bf16><<<blocks, kEmbedBlock, 0, s>>>(ids, id_bytes, tokens, (const bf16*)table, vocab, width, scale, (bf16*)y);
    else
      k_embed<float><<<blocks, kEmbedBlock, 0, s>>>(ids, id_bytes, tokens, (const float*)table, vocab, width, scale, (float*)y);
  });
  return hipGetLastError();
}

hipError_t embedding_backward(const EmbedWorkspace& w, int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* dy,
                              uint32_t vocab, uint32_t width, float scale, int table_dtype, void* dtable, hipStream_t s) {
  hipError_t e;
  if (tokens) {
    LAPLEX_LAUNCH("k_embed_keys", tokens, s,
                  k_embed_keys<<<(unsigned)((tokens + 255) / 256), 256, 0, s>>>(ids, id_bytes, tokens, vocab, w.keys));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // a nonnegative int's bits, read as a float, sort in the same order
    if ((e = sort_anchors(w.sort, reinterpret_cast<const float*>(w.keys), tokens, w.keys_s, w.perm, nullptr, s)) != hipSuccess)
      return e;
  }
  LAPLEX_LAUNCH("k_embed_starts", vocab, s,
                k_embed_starts<<<vocab / 256 + 1, 256, 0, s>>>(reinterpret_cast<const uint32_t*>(w.keys_s), tokens, vocab, w.starts));
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned blocks = std::min<uint32_t>(vocab, 1u << 20);
  LAPLEX_LAUNCH("k_embed_grad", tokens, s, {
    if (dtype != LAPLEX_BF16)
      k_embed_grad<float, float><<<blocks, kEmbedBlock, 0, s>>>(w.perm, w.starts, (const float*)dy, vocab, width, scale, (float*)dtable);
    else if (table_dtype == LAPLEX_F32)
      k_embed_grad<bf16, float><<<blocks, kEmbedBlock, 0, s>>>(w.perm, w.starts, (const bf16*)dy, vocab, width, scale, (float*)dtable);
    else
      k_embed_grad<bf16, bf16><<<blocks, kEmbedBlock, 0, s>>>(w.perm, w.starts, (const bf16*)dy, vocab, width, scale, (bf16*)dtable);
  });
  return hipGetLastError();
}

}  // namespace laplex
