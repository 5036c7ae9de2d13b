// Decayed linear attention: the passes over a sequence (segments, their join,
// the launches), the sums over shared heads, and the single-token form.
#include "laplex_attn_chunk.hpp"

namespace laplex {

// Turns the segments' own final states into the states before each segment,
// S_k+1 = w(L) S_k + T_k, in place; thread per element.  With lag-weighted
// states, D_k+1 = w(L) (D_k + L S_k) + E_k.  One read and one write of the states: bound by HBM (512 boundaries of
// 128 x 128 floats, 67 MB: 14 us, 4.8 TB/s).  Joined in the next pass's first lines instead, each segment reads
// all of its predecessors: 100 us of that pass became 134.
template <bool RATE>
__global__ __launch_bounds__(256) void k_attn_join(AttnChunkArgs a) {
  __shared__ AttnDecay sw;
  const AttnPass& p = a.p;
  const uint32_t per = p.K * p.V, at = blockIdx.x * 256 + threadIdx.x;
  const uint32_t h = blockIdx.y;
  const int64_t L = a.g.seg_len;
  if (threadIdx.x == 0) sw = attn_decay(attn_rate(p.rate[h]), L);
  __syncthreads();
  const AttnDecay w = sw;
  if (at >= per) return;
  const uint64_t step = (uint64_t)p.heads * per;  // from a boundary to the next
  for (uint32_t s = blockIdx.z; s < p.seqs; s += gridDim.z) {
    const int64_t i = (int64_t)s + (a.g.offsets ? 1 : 0), first = seq_bound(a.g, i), len = seq_bound(a.g, i + 1) - first;
    if (len <= L) continue;  // no boundary inside the sequence
    const int nb = (int)((len - 1) / L);
    float cur = 0.f, d = 0.f;
    if (p.s_in) cur = p.s_in[((uint64_t)s * p.heads + h) * per + (p.s_trans ? at % p.V * p.K + at / p.V : at)];
    uint64_t q = ((uint64_t)(first / L + 1) * p.heads + h) * per + at;
    auto join = [&](uint64_t q, float t, float e) {
      if constexpr (RATE) {
        d = w.of(fmaf((float)L, cur, d)) + e;
        a.bound_d[q] = d;
      }
      cur = w.of(cur) + t;
      a.bound[q] = cur;
    };
    constexpr int N = 8;  // loads in flight
    int k = 0;
    for (; k + N <= nb; k += N) {
      float t[N], e[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        t[j] = a.bound[q + j * step];
        e[j] = RATE ? a.bound_d[q + j * step] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) join(q + j * step, t[j], e[j]);
      q += N * step;
    }
    for (; k < nb; ++k, q += step) join(q, a.bound[q], RATE ? a.bound_d[q] : 0.f);
  }
}

// ------------------------------------------------------------------ launches
struct AttnPlan {
  int kp, nw;
  uint32_t slices;
  int64_t seg_len;
  uint64_t bounds;
  bool split;
};
// The split depends on K and V alike, so that a pass and the one with K and V exchanged share their segments.
struct AttnSplit {
  uint64_t least;   // tokens of a segment, at least
  uint64_t across;  // blocks across heads and columns
  uint64_t blocks;  // that run at once
};
static AttnSplit attn_split(int dtype, uint32_t heads, uint32_t K, uint32_t V, bool rate) {
  const uint32_t wide = std::max(K, V), slices = wide > 128 ? 2 : 1;
  // Blocks that run at once: 256 CUs with two of eight waves or four of four; half with the lag-weighted carry.
  // (65536 tokens x 8 heads, 128 x 128: 252 us; with half as many blocks 275, with twice as many 274.  8 x 2048 tokens
  // x 16 heads forward and backward: 600, 719, 685.)  At least two chunks each (1000 tokens x 8 heads of
  // floats, 128 x 128, forward and backward: 139 us, with one chunk 138, with four 185; 4000 x 8 heads in bfloat16: 174, 191, 189).
  return {dtype == LAPLEX_BF16 ? 128u : 64u, (uint64_t)heads * slices, (wide <= 64 ? 1024u : 512u) / (rate ? 2 : 1)};
}
static int64_t attn_seg_len(int dtype, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens, bool rate) {
  const AttnSplit f = attn_split(dtype, heads, K, V, rate);
  uint64_t len = std::max<uint64_t>(f.least, tokens * f.across / f.blocks);
  len = (len + 63) / 64 * 64;
  // Two segments cost more than one of twice the length (2048 tokens x 256 heads: 222 us, 197; 256 x 8: 23.9, 21.9),
  // three do not (300 x 4 heads, 64 x 64, forward and backward: 89 us, unsplit 102; 2048 x 200 heads: 198, 197).
  return (int64_t)(2 * len < tokens ? len : std::max<uint64_t>(64, (tokens + 63) / 64 * 64));
}
// Boundaries between segments (tokens / seg_len + 1, none without a split), the most over all smaller numbers of tokens,
// so that a workspace for many tokens serves fewer.  seg_len is at least `least`, and at least 64 / 65 of tokens *
// across / blocks (that quotient is rounded down, then up to a multiple of 64).
static uint64_t attn_bounds_most(int dtype, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens, bool rate) {
  const AttnSplit f = attn_split(dtype, heads, K, V, rate);
  if (tokens <= 2 * f.least || 128 * f.across >= 65 * f.blocks) return 0;  // two segments are not less than the tokens
  return std::min(tokens / f.least, f.blocks * 65 / (f.across * 64)) + 1;
}
static AttnPlan attn_plan(int dtype, uint32_t seqs, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens, bool rate) {
  AttnPlan q;
  q.kp = K <= 64 ? 64 : K <= 128 ? 128 : 256;
  q.seg_len = attn_seg_len(dtype, heads, K, V, tokens, rate);
  // V of at most 64 needs four waves (16384 tokens x 16 heads, 64 x 64, forward and backward: 333 us with eight, 300;
  // in float 624, 533; 128 x 64: 427 either way).  Where blocks of 128 columns would leave a good part of the 256 CUs
  // idle, blocks of 64 share a chunk's work out among twice as many (131 tokens x 4 heads, 80 x 96, float: 34 -> 25 us;
  // 2048 x 8 heads, 128 x 128, bfloat16, 136 blocks, forward and backward: 157 -> 138; at 264 blocks 175 -> 197).  In
  // between it depends: at 152 blocks 2304 tokens in bfloat16 take 155 -> 176, for the rate's gradient has one block a CU
  // and then two rounds of them, but without backward 36.0 -> 36.1, and 1200 tokens in float 190 -> 175.
  const uint64_t blocks = (tokens / q.seg_len + seqs) * heads * ((V + 127) / 128);
  q.nw = q.kp <= 128 && (V <= 64 || blocks <= 160) ? 4 : 8;
  q.slices = (V + 16 * q.nw - 1) / (16 * q.nw);
  q.split = (uint64_t)q.seg_len < tokens;
  q.bounds = q.split ? tokens / q.seg_len + 1 : 0;
  return q;
}

size_t attn_pass_bytes(int dtype, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens, bool rate) {
  return (size_t)attn_bounds_most(dtype, heads, K, V, tokens, rate) * heads * K * V * 4 * (rate ? 2 : 1);
}
uint64_t attn_drate_parts_most(int dtype, uint32_t seqs, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens) {
  // attn_slots with or without offsets, by the slices of the narrowest blocks
  return (std::max<uint64_t>(attn_bounds_most(dtype, heads, K, V, tokens, true), 1) + seqs + 3) * ((V + 63) / 64);
}
uint64_t attn_drate_parts(int dtype, uint32_t seqs, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens, const int32_t* offsets) {
  const AttnPlan q = attn_plan(dtype, seqs, heads, K, V, tokens, true);
  return attn_slots({offsets, tokens, seqs, q.seg_len}) * q.slices;
}

static bool aligned16(const void* p, int64_t token, int64_t head, uint32_t width, size_t e) {
  // (and rows follow each other without overlap, a chunk's 64 within 2^30 bytes)
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token >= (int64_t)width && (uint64_t)token * e < (1u << 24) && token * e % 16 == 0 && head * e % 16 == 0 && width * e % 16 == 0;
}

hipError_t attn_pass(const AttnPass& p, void* ws, hipStream_t s) {
  const bool rate = p.drate_part != nullptr, bf = p.dtype == LAPLEX_BF16;
  const size_t e = bf ? 2 : 4;
  const AttnPlan q = attn_plan(p.dtype, p.seqs, p.heads, p.K, p.V, p.tokens, rate);
  if (q.bounds > attn_bounds_most(p.dtype, p.heads, p.K, p.V, p.tokens, rate) ||
      (rate && attn_drate_parts(p.dtype, p.seqs, p.heads, p.K, p.V, p.tokens, p.offsets) >
                   attn_drate_parts_most(p.dtype, p.seqs, p.heads, p.K, p.V, p.tokens)))
    return hipErrorInvalidValue;  // (more than the workspace was laid out for)
  AttnChunkArgs a{};
  a.p = p;
  a.g = {p.offsets, p.tokens, p.seqs, q.seg_len};
  a.slices = q.slices;
  a.slots = attn_slots(a.g);
  a.group = std::max(p.x.div, std::max(p.y.div, p.z.div));
  if (q.split) {
    a.bound = static_cast<float*>(ws);
    a.bound_d = a.bound + q.bounds * p.heads * p.K * p.V;
  }
  const bool vec = aligned16(p.x.p, p.x.token, p.x.head, p.K, e) && aligned16(p.y.p, p.y.token, p.y.head, p.K, e) &&
                   aligned16(p.z.p, p.z.token, p.z.head, p.V, e) &&
                   (!rate || aligned16(p.dot, p.dot_view.token, p.dot_view.head, p.V, e)) &&
                   reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  a.bound_trans = p.bound_ready;
  a.drate = p.drate_part;
  auto run = [&](const char* name, bool full) {
    LAPLEX_LAUNCH(name, p.tokens, s, {
      if (bf) (vec ? attn_chunk_bf16_vec : attn_chunk_bf16_any)(a, q.kp, q.nw, full, rate, s);
      else (vec ? attn_chunk_f32_vec : attn_chunk_f32_any)(a, q.kp, q.nw, full, rate, s);
    });
    return hipGetLastError();
  };
  hipError_t err;
  if (q.split && !p.bound_ready) {
    if ((err = run("k_attn_chunk_state", false)) != hipSuccess) return err;
    const uint64_t longest = p.offsets ? p.tokens : p.tokens / p.seqs;  // at most
    const dim3 grid((unsigned)(((uint64_t)p.K * p.V + 255) / 256), p.heads, std::min(p.seqs, 8u));
    if ((int64_t)longest > q.seg_len)
      LAPLEX_LAUNCH("k_attn_join", q.bounds, s, rate ? k_attn_join<true><<<grid, 256, 0, s>>>(a) : k_attn_join<false><<<grid, 256, 0, s>>>(a));
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  return run("k_attn_chunk", true);
}

// drate_h = the sum of its partials in a fixed order (a launch's latency: 5 us)
__global__ __launch_bounds__(256) void k_attn_drate(const double* __restrict__ part, uint64_t parts, uint32_t heads,
                                                    float* __restrict__ drate) {
  __shared__ double sh[256];
  const uint32_t h = blockIdx.x;
  double s = 0.0;
  for (uint64_t i = threadIdx.x; i < parts; i += 256) s += part[i * heads + h];
  sh[threadIdx.x] = s;
  for (int off = 128; off; off >>= 1) {
    __syncthreads();
    if (threadIdx.x < off) sh[threadIdx.x] += sh[threadIdx.x + off];
  }
  if (threadIdx.x == 0) drate[h] = (float)sh[0];
}

hipError_t attn_drate_reduce(const double* part, uint64_t parts, uint32_t heads, float* drate, hipStream_t s) {
  LAPLEX_LAUNCH("k_attn_drate", heads, s, k_attn_drate<<<heads, 256, 0, s>>>(part, parts, heads, drate));
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
// S = w S + k v^T in place, o = scale q S: the state is read and written once,
// everything else is small, so the step is bound by HBM (256 rows x 16 heads x
// 128 x 128, 541 MB: 99 us, 5.4 TB/s).  A block takes one head of one row; a
// thread holds E consecutive columns of every R-th row of the state, kStepRows
// rows on the way at a time (1: 103 us, 8: 146); the R partial outputs meet in LDS.
// NT: loads and stores that leave the caches alone, for states larger than the
// Infinity Cache (470 MB: 178 us instead of 190; 117 MB, which stay in it from
// one step to the next: 45 instead of 43).
constexpr int kStepBlock = 256, kStepRows = 4;
constexpr uint64_t kStepCached = 256ull << 20;
template <typename T, int E, bool NT>
__global__ __launch_bounds__(kStepBlock) void k_attn_step(AttnStep p, uint32_t lanes) {
  __shared__ float qs[256], ks[256], part[kStepBlock * E];
  typedef float vec __attribute__((ext_vector_type(E)));
  const uint32_t row = blockIdx.x, h = blockIdx.y;
  const int64_t slot = p.slots ? (int64_t)p.slots[row] : (int64_t)row;
  T* out = static_cast<T*>(p.out) + ((uint64_t)row * p.heads + h) * p.V;
  if (slot < 0 || slot >= (int64_t)p.pool) {
    for (uint32_t c = threadIdx.x; c < p.V; c += kStepBlock) out[c] = from_f32<T>(0.f);
    return;
  }
  const T *q = static_cast<const T*>(p.q.p) + row * p.q.token + (int64_t)(h / p.q.div) * p.q.head,
          *k = static_cast<const T*>(p.k.p) + row * p.k.token + (int64_t)(h / p.k.div) * p.k.head,
          *v = static_cast<const T*>(p.v.p) + row * p.v.token + (int64_t)(h / p.v.div) * p.v.head;
  const AttnDecay w = attn_decay(attn_rate(p.rate[h]), 1);
  for (uint32_t i = threadIdx.x; i < p.K; i += kStepBlock) {
    qs[i] = to_f32(q[i]);
    ks[i] = to_f32(k[i]);
  }
  const uint32_t R = kStepBlock / lanes, r = threadIdx.x / lanes, c = threadIdx.x % lanes * E;
  float* st = p.state + ((uint64_t)slot * p.heads + h) * (uint64_t)p.K * p.V + c;
  vec vv, acc = {};
#pragma unroll
  for (int e = 0; e < E; ++e) vv[e] = c + e < p.V ? to_f32(v[c + e]) : 0.f;
  __syncthreads();
  if (c < p.V)
    for (uint32_t i0 = r; i0 < p.K; i0 += R * kStepRows) {
      vec s[kStepRows];
#pragma unroll
      for (int j = 0; j < kStepRows; ++j)
        if (i0 + j * R < p.K) {
          const vec* at = reinterpret_cast<const vec*>(st + (uint64_t)(i0 + j * R) * p.V);
          s[j] = NT ? __builtin_nontemporal_load(at) : *at;
        }
#pragma unroll
      for (int j = 0; j < kStepRows; ++j) {
        const uint32_t i = i0 + j * R;
        if (i >= p.K) break;
        const float kk = ks[i], qq = qs[i];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          s[j][e] = fmaf(w.hi, s[j][e], fmaf(w.lo, s[j][e], kk * vv[e]));
          acc[e] = fmaf(qq, s[j][e], acc[e]);
        }
        vec* at = reinterpret_cast<vec*>(st + (uint64_t)i * p.V);
        if (NT) __builtin_nontemporal_store(s[j], at);
        else *at = s[j];
      }
    }
#pragma unroll
  for (int e = 0; e < E; ++e) part[(r * lanes + threadIdx.x % lanes) * E + e] = acc[e];
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < p.V; o += kStepBlock) {
    float a = 0.f;
    for (uint32_t i = 0; i < R; ++i) a += part[i * lanes * E + o];
    out[o] = from_f32<T>(p.scale * a);
  }
}

template <typename T, int E>
static void step_launch(const AttnStep& p, hipStream_t s) {
  uint32_t lanes = 1;  // threads across a row of the state
  while (lanes * E < p.V) lanes *= 2;
  const dim3 grid(p.rows, p.heads);
  if ((uint64_t)p.rows * p.heads * p.K * p.V * 4 > kStepCached) k_attn_step<T, E, true><<<grid, kStepBlock, 0, s>>>(p, lanes);
  else k_attn_step<T, E, false><<<grid, kStepBlock, 0, s>>>(p, lanes);
}

hipError_t attn_step(const AttnStep& p, hipStream_t s) {
  const bool vec = p.V % 4 == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0;
  LAPLEX_LAUNCH("k_attn_step", p.rows, s, {
    if (p.dtype == LAPLEX_BF16) vec ? step_launch<bf16, 4>(p, s) : step_launch<bf16, 1>(p, s);
    else vec ? step_launch<float, 4>(p, s) : step_launch<float, 1>(p, s);
  });
  return hipGetLastError();
}

}  // namespace laplex
