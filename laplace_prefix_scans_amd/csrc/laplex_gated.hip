// Gated linear recurrence: forward, backward, and the single-token form.
//
//   h_t = a_t h_{t-1} + w_t x_t,   rate: a = exp(-r), w = 1;   sigmoid: a = s(z), w = 1 - a.
//   l_t = dh_t + a_{t+1} l_{t+1},  dx = w l,  dr = -a h_{t-1} l,  dz = a w (h_{t-1} - x) l.
//
// A wave takes 64 lanes' channels of one segment of the packed tokens, 16 tokens
// at a time, so that 16 rows of each tensor are on their way at once; nothing is
// exchanged between lanes.  Where sequences and channels alone do not fill the
// chip, the tokens are cut into segments: a pass over their aggregates (the
// decay over a segment and its state from zero), then the whole pass, each
// wave of which first joins the aggregates before its own.  Segments are cut
// without regard to sequences: a token that begins a sequence replaces the
// state before it, whatever that is.
#include "laplex_layers_device.hpp"
#include "laplex_train.hpp"

namespace laplex {

constexpr int kGateU = (int)kGateChunk;
constexpr int kGateWaves = 4;  // of a block

// ------------------------------------------------------------------ decays
// A decay a near 1 is kept as c = -(1 - a), with the sign bit set, and any other as
// c = a: over the thousands of tokens that a slow decay reaches, the rounding of
// a itself would add up (each of 4000 steps by up to 2^-25), that of 1 - a does not.
__device__ __forceinline__ bool near_one(float c) { return __float_as_int(c) < 0; }
// a s
__device__ __forceinline__ float decayed(float c, float s) { return fmaf(c, s, near_one(c) ? s : 0.f); }
__device__ __forceinline__ float decay_value(float c) { return near_one(c) ? 1.f + c : c; }
// the product of two decays
__device__ __forceinline__ float decay_join(float c, float d) {
  if (near_one(c) && near_one(d)) {
    const float q = fmaf(c, d, c + d);  // -(1 - a b)
    return q >= -0.5f ? (q == 0.f ? -0.f : q) : 1.f + q;
  }
  return near_one(c) ? fmaf(c, d, d) : near_one(d) ? fmaf(c, d, c) : c * d;
}

template <int KIND>
struct Gate {
  float c, a, w;  // the decay as above, itself, and the input's weight
};
template <int KIND>
__device__ __forceinline__ Gate<KIND> gate_of(float g) {
  Gate<KIND> r;
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (KIND == LAPLEX_GATE_RATE) {
    const float e = __builtin_amdgcn_exp2f(-g * kLog2e);
    // 1 - exp(-g): its series up to g = 0.3, where the first term left out is below 2^-25 of it
    float p = fmaf(g, -1.f / 8, 1.f);
    p = fmaf(g * p, -1.f / 7, 1.f);
    p = fmaf(g * p, -1.f / 6, 1.f);
    p = fmaf(g * p, -1.f / 5, 1.f);
    p = fmaf(g * p, -1.f / 4, 1.f);
    p = fmaf(g * p, -1.f / 3, 1.f);
    p = fmaf(g * p, -1.f / 2, 1.f);
    const float q = g < 0.3f ? g * p : 1.f - e;
    r.a = e;
    r.w = 1.f;
    r.c = g >= 0.f && q <= 0.5f ? -q : e;
  } else {
    const float e = __builtin_amdgcn_exp2f(-fabsf(g) * kLog2e), d = 1.f + e;
    float big = __builtin_amdgcn_rcpf(d);
    big = fmaf(fmaf(-d, big, 1.f), big, big);
    const float small = e * big;
    const bool up = g >= 0.f;
    r.a = up ? big : small;
    r.w = up ? small : big;
    r.c = up ? -small : small;
  }
  return r;
}

// The decay over the tokens of a tile.
struct TileDecay {
  float p = 1.f, q = 0.f, most = -1.f;  // their product, one minus it, and the largest that is not near 1
  __device__ __forceinline__ void add(float c, float a) {
    p *= a;
    q = fmaf(-c, 1.f - q, q);
    most = fmaxf(most, c);
  }
  __device__ __forceinline__ float coded() const { return p < 0.5f || most > 0.f ? p : -q; }
};

// ------------------------------------------------------------------ sequences
struct GateSeqs {
  const int32_t* offsets;
  int64_t len;  // tokens of each sequence, without offsets
  int32_t seqs;
  __device__ __forceinline__ int64_t at(int64_t j) const { return offsets ? (int64_t)offsets[j] : j * len; }
  // first j in 0 .. seqs whose start (the last one's end) is at least t, or seqs + 1; the whole wave with the same t
  __device__ __forceinline__ int32_t lower(int64_t t) const {
    if (!offsets && len > 0) return (int32_t)min((int64_t)seqs + 1, max((int64_t)0, (t + len - 1) / len));
    int32_t lo = 0, cnt = seqs + 1;  // the answer is in lo .. lo + cnt
    while (cnt > 0) {
      const int32_t step = (cnt + kWave - 1) / kWave, j = lo + lane_id() * step;
      const bool below = j < lo + cnt && at(j) < t;
      const int32_t k = (int32_t)__popcll(__ballot(below));
      if (k == 0) return lo;
      const int32_t skip = (k - 1) * step + 1;  // at(lo + skip - 1) < t
      lo += skip;
      cnt = min(step - 1, cnt - skip);
    }
    return lo;
  }
  // the sequence that holds token t (which lies in one)
  __device__ __forceinline__ int32_t of(int64_t t) const {
    return __builtin_amdgcn_readfirstlane(min(max(lower(t + 1) - 1, 0), seqs - 1));
  }
};
__device__ __forceinline__ uint32_t wave_or(uint32_t v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v |= __shfl_xor(v, off);
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  // (the builtin returns a signed word)
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32)), lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Which of a tile's tokens begin and end sequences, and which lie in none; tiles are taken in turn, so most need only `clear`.
struct GateMarks {
  uint32_t starts, ends, outside;
  int64_t first, last;  // tokens of all sequences
  int64_t clear_lo, clear_hi;  // no boundary b with clear_lo < b < clear_hi
  __device__ __forceinline__ void init(const GateSeqs& s) {
    first = uniform64(s.at(0));
    last = uniform64(s.at(s.seqs));
    clear_lo = 1;
    clear_hi = 0;
  }
  __device__ __forceinline__ void tile(const GateSeqs& s, int64_t t0) {
    constexpr int64_t U = kGateU;
    starts = ends = outside = 0;
    if (t0 > clear_lo && t0 + U < clear_hi) {  // (a boundary at t0 + U is an end inside)
      if (t0 >= last || t0 + U <= first) outside = (1u << U) - 1;
      return;
    }
    const int32_t lo = __builtin_amdgcn_readfirstlane(s.lower(t0));
    uint32_t m = 0;
    int64_t above = INT64_MAX;
    for (int32_t base = lo; base <= s.seqs; base += kWave) {
      const int32_t j = base + lane_id();
      const bool real = j <= s.seqs;
      const int64_t o = real ? s.at(j) : INT64_MAX;
      if (real && o <= t0 + U) {
        if (o < t0 + U && j < s.seqs && s.at(j + 1) > o) m |= 1u << (o - t0);
        if (o > t0 && j > 0 && s.at(j - 1) < o) m |= 0x10000u << (o - 1 - t0);
      }
      const uint64_t beyond = __ballot(real && o > t0 + U);
      if (beyond) {
        above = s.at(base + __builtin_ctzll(beyond));
        break;
      }
    }
    clear_lo = uniform64(lo > 0 ? s.at(lo - 1) : INT64_MIN);
    clear_hi = uniform64(above);
    m = wave_or(m);
    if (m || (lo <= s.seqs && uniform64(s.at(lo)) <= t0 + U)) {  // boundaries inside: what is clear begins after them, or before
      starts = m & 0xFFFFu;
      ends = m >> 16;
      clear_lo = 1;
      clear_hi = 0;
    }
    if (t0 < first) outside |= first - t0 >= U ? (1u << U) - 1 : (1u << (first - t0)) - 1;
    if (t0 + U > last) outside |= last <= t0 ? (1u << U) - 1 : ((1u << U) - 1) & ~((1u << (last - t0)) - 1);
  }
};
static_assert(kGateU == 16, "marks of a tile are 16 bits");

// ------------------------------------------------------------------ rows
// CV channels a lane, the row's last ones one by one.
template <typename T>
constexpr int kGateCV = 4 / sizeof(T);
template <typename T>
struct Piece {
  T e[kGateCV<T>];
};
template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T* p, int left) {
  Piece<T> r;
  if (left >= kGateCV<T>) {
    __builtin_memcpy(r.e, p, sizeof r.e);
  } else {
#pragma unroll
    for (int i = 0; i < kGateCV<T>; ++i) r.e[i] = i < left ? p[i] : T(0.f);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void store_piece(T* p, int left, const float (&v)[kGateCV<T>]) {
  Piece<T> r;
#pragma unroll
  for (int i = 0; i < kGateCV<T>; ++i) r.e[i] = from_f32<T>(v[i]);
  if (left >= kGateCV<T>) {
    __builtin_memcpy(p, r.e, sizeof r.e);
  } else {
#pragma unroll
    for (int i = 0; i < kGateCV<T>; ++i)
      if (i < left) p[i] = r.e[i];
  }
}
template <typename T>
struct Rows {
  const T* p;  // of the lane's first channel
  int64_t token;
  int left;
  __device__ __forceinline__ void load(Piece<T> (&v)[kGateU], int64_t t0, int64_t tokens) const {
#pragma unroll
    for (int i = 0; i < kGateU; ++i) v[i] = load_piece(p + min(t0 + i, tokens - 1) * token, left);
  }
};

struct GateArgs {
  GateShape g;
  int64_t seg_len;  // a multiple of the tile
  uint32_t segs, ctiles;
  float *agg_c, *agg_b;  // segs x channels: decay over a segment (coded), its state from zero
  uint32_t* reset;       // segs: whether a segment holds a boundary, so that nothing passes through it
  const float* state_in;
  float* state_out;
  void* h;
  float* carries;
  // backward
  const float* carries_in;
  const void* dh;
  const float* dstate_out;
  void *dgate, *dx;
  float* dstate_in;
};

template <typename T>
struct Lane {
  uint32_t seg, ctile;
  int64_t c0, t_lo, t_hi;  // first channel, the segment's tokens
  int left;                // channels from c0 on
  bool valid;
  __device__ __forceinline__ Lane(const GateArgs& a) {
    const uint64_t unit = (uint64_t)blockIdx.x * kGateWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    seg = (uint32_t)(unit / a.ctiles);
    ctile = (uint32_t)(unit % a.ctiles);
    valid = seg < a.segs;
    c0 = ((int64_t)ctile * kWave + lane_id()) * kGateCV<T>;
    left = (int)max((int64_t)0, min((int64_t)a.g.channels - c0, (int64_t)kGateCV<T>));
    if (left == 0) c0 = 0;
    t_lo = (int64_t)seg * a.seg_len;
    t_hi = min((int64_t)a.g.tokens, t_lo + a.seg_len);
  }
};

// What comes into segment `seg` from those before it (BACK: after it): aggregates joined in turn, 8 on their way.
template <typename T, bool BACK>
__device__ __forceinline__ void joined(const GateArgs& a, const Lane<T>& l, float (&s)[kGateCV<T>]) {
  constexpr int CV = kGateCV<T>, N = 8;
#pragma unroll
  for (int e = 0; e < CV; ++e) s[e] = 0.f;
  const int32_t n = BACK ? (int32_t)(a.segs - 1 - l.seg) : (int32_t)l.seg;
  for (int32_t k = 0; k < n; k += N) {
    float c[N][CV], b[N][CV];
    uint32_t r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t at = min(k + i, n - 1), seg = BACK ? a.segs - 1 - at : at;
      r[i] = a.reset[seg];
#pragma unroll
      for (int e = 0; e < CV; ++e) {
        const uint64_t p = (uint64_t)seg * a.g.channels + l.c0 + (e < l.left ? e : 0);
        c[i][e] = a.agg_c[p];
        b[i][e] = a.agg_b[p];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (k + i < n) {
#pragma unroll
        for (int e = 0; e < CV; ++e) s[e] = r[i] ? b[i][e] : decayed(c[i][e], s[e]) + b[i][e];
      }
  }
}

// ------------------------------------------------------------------ forward
// WHOLE: outputs; without, the segment's aggregate alone.
template <typename T, int KIND, bool WHOLE>
__global__ __launch_bounds__(kWave* kGateWaves) void k_gated(GateArgs a) {
  constexpr int CV = kGateCV<T>, U = kGateU;
  const Lane<T> l(a);
  if (!l.valid) return;
  const GateSeqs seqs{a.g.offsets, a.g.offsets ? 0 : (int64_t)(a.g.tokens / a.g.seqs), (int32_t)a.g.seqs};
  const int64_t T_ = (int64_t)a.g.tokens;
  const Rows<T> rg{static_cast<const T*>(a.g.gate) + l.c0, a.g.gate_token, l.left}, rx{static_cast<const T*>(a.g.x) + l.c0, a.g.x_token, l.left};
  float s[CV] = {}, total[CV];
#pragma unroll
  for (int e = 0; e < CV; ++e) total[e] = -0.f;  // a decay of 1
  uint32_t cut = 0;
  Piece<T> g[U], x[U];
  rg.load(g, l.t_lo, T_);
  rx.load(x, l.t_lo, T_);
  if (WHOLE && l.seg) joined<T, false>(a, l, s);
  GateMarks m;
  m.init(seqs);
  for (int64_t t0 = l.t_lo; t0 < l.t_hi; t0 += U) {
    float c[U][CV], b[U][CV];
    TileDecay d[CV];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < CV; ++e) {
        const Gate<KIND> q = gate_of<KIND>(to_f32(g[i].e[e]));
        c[i][e] = q.c;
        b[i][e] = KIND == LAPLEX_GATE_RATE ? to_f32(x[i].e[e]) : q.w * to_f32(x[i].e[e]);
        if (!WHOLE) d[e].add(q.c, q.a);
      }
    if (t0 + U < l.t_hi) {
      rg.load(g, t0 + U, T_);
      rx.load(x, t0 + U, T_);
    }
    m.tile(seqs, t0);
    if (WHOLE && a.carries && l.left) {
      float* q = a.carries + (uint64_t)(t0 / U) * a.g.channels + l.c0;
#pragma unroll
      for (int e = 0; e < CV; ++e)
        if (e < l.left) q[e] = s[e];
    }
    const uint32_t special = m.starts | m.ends | m.outside;
    const int n = (int)min((int64_t)U, l.t_hi - t0);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i < n) {
        if (__builtin_expect(special >> i & 1, 0)) {
          if (m.starts >> i & 1) {
            const int32_t q = seqs.of(t0 + i);
#pragma unroll
            for (int e = 0; e < CV; ++e) s[e] = a.state_in && e < l.left ? a.state_in[(uint64_t)q * a.g.channels + l.c0 + e] : 0.f;
            cut = 1;
          }
          if (m.outside >> i & 1) {
            cut = 1;
#pragma unroll
            for (int e = 0; e < CV; ++e) s[e] = c[i][e] = b[i][e] = 0.f;
          }
        }
#pragma unroll
        for (int e = 0; e < CV; ++e) s[e] = decayed(c[i][e], s[e]) + b[i][e];
        if constexpr (WHOLE) {
          if (l.left) store_piece(static_cast<T*>(a.h) + (uint64_t)(t0 + i) * a.g.channels + l.c0, l.left, s);
          if (__builtin_expect(a.state_out && (m.ends >> i & 1), 0)) {
            const int32_t q = seqs.of(t0 + i);
#pragma unroll
            for (int e = 0; e < CV; ++e)
              if (e < l.left) a.state_out[(uint64_t)q * a.g.channels + l.c0 + e] = s[e];
          }
        }
      }
    }
    if (!WHOLE) {
#pragma unroll
      for (int e = 0; e < CV; ++e) total[e] = decay_join(total[e], d[e].coded());
    }
  }
  if constexpr (!WHOLE) {
#pragma unroll
    for (int e = 0; e < CV; ++e)
      if (e < l.left) {
        const uint64_t p = (uint64_t)l.seg * a.g.channels + l.c0 + e;
        a.agg_c[p] = total[e];
        a.agg_b[p] = s[e];
      }
    if (l.ctile == 0 && lane_id() == 0) a.reset[l.seg] = cut;
  }
}

// ------------------------------------------------------------------ backward
// The carry is mu_t = a_t l_t, which token t - 1 receives: mu_t = a_t mu_{t+1} + a_t dh_t.
template <typename T, int KIND>
__global__ __launch_bounds__(kWave* kGateWaves) void k_gated_back_aggregate(GateArgs a) {
  constexpr int CV = kGateCV<T>, U = kGateU;
  const Lane<T> l(a);
  if (!l.valid) return;
  const GateSeqs seqs{a.g.offsets, a.g.offsets ? 0 : (int64_t)(a.g.tokens / a.g.seqs), (int32_t)a.g.seqs};
  const int64_t T_ = (int64_t)a.g.tokens;
  const Rows<T> rg{static_cast<const T*>(a.g.gate) + l.c0, a.g.gate_token, l.left},
      rd{static_cast<const T*>(a.dh) + l.c0, (int64_t)a.g.channels, l.left};
  float mu[CV] = {}, total[CV];
#pragma unroll
  for (int e = 0; e < CV; ++e) total[e] = -0.f;
  uint32_t cut = 0;
  Piece<T> g[U], y[U];
  int64_t t0 = l.t_lo + (l.t_hi - l.t_lo - 1) / U * U;
  rg.load(g, t0, T_);
  rd.load(y, t0, T_);
  GateMarks m;
  m.init(seqs);
  for (; t0 >= l.t_lo; t0 -= U) {
    float c[U][CV], dh[U][CV];
    TileDecay d[CV];
    const int n = (int)min((int64_t)U, l.t_hi - t0);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < CV; ++e) {
        const Gate<KIND> q = gate_of<KIND>(to_f32(g[i].e[e]));
        c[i][e] = q.c;
        dh[i][e] = to_f32(y[i].e[e]);
        if (i < n) d[e].add(q.c, q.a);
      }
    if (t0 > l.t_lo) {
      rg.load(g, t0 - U, T_);
      rd.load(y, t0 - U, T_);
    }
    m.tile(seqs, t0);
    const uint32_t special = m.ends | m.outside;
#pragma unroll
    for (int i = U - 1; i >= 0; --i) {
      if (i < n) {
        if (__builtin_expect(special >> i & 1, 0)) {
          cut = 1;
          const int32_t q = m.ends >> i & 1 ? seqs.of(t0 + i) : 0;
#pragma unroll
          for (int e = 0; e < CV; ++e) {
            mu[e] = m.ends >> i & 1 && a.dstate_out && e < l.left ? a.dstate_out[(uint64_t)q * a.g.channels + l.c0 + e] : 0.f;
            if (m.outside >> i & 1) c[i][e] = dh[i][e] = 0.f;
          }
        }
#pragma unroll
        for (int e = 0; e < CV; ++e) mu[e] = decayed(c[i][e], mu[e] + dh[i][e]);
      }
    }
#pragma unroll
    for (int e = 0; e < CV; ++e) total[e] = decay_join(total[e], d[e].coded());
  }
#pragma unroll
  for (int e = 0; e < CV; ++e)
    if (e < l.left) {
      const uint64_t p = (uint64_t)l.seg * a.g.channels + l.c0 + e;
      a.agg_c[p] = total[e];
      a.agg_b[p] = mu[e];
    }
  if (l.ctile == 0 && lane_id() == 0) a.reset[l.seg] = cut;
}

template <typename T, int KIND>
__global__ __launch_bounds__(kWave* kGateWaves) void k_gated_back(GateArgs a) {
  constexpr int CV = kGateCV<T>, U = kGateU;
  const Lane<T> l(a);
  if (!l.valid) return;
  const GateSeqs seqs{a.g.offsets, a.g.offsets ? 0 : (int64_t)(a.g.tokens / a.g.seqs), (int32_t)a.g.seqs};
  const int64_t T_ = (int64_t)a.g.tokens;
  const Rows<T> rg{static_cast<const T*>(a.g.gate) + l.c0, a.g.gate_token, l.left}, rx{static_cast<const T*>(a.g.x) + l.c0, a.g.x_token, l.left},
      rd{static_cast<const T*>(a.dh) + l.c0, (int64_t)a.g.channels, l.left};
  float mu[CV];
  Piece<T> g[U], x[U], y[U];
  float before[CV];
  auto load_carry = [&](int64_t t0) {
    const float* q = a.carries_in + (uint64_t)(t0 / U) * a.g.channels + l.c0;
#pragma unroll
    for (int e = 0; e < CV; ++e) before[e] = q[e < l.left ? e : 0];
  };
  int64_t t0 = l.t_lo + (l.t_hi - l.t_lo - 1) / U * U;
  rg.load(g, t0, T_);
  rx.load(x, t0, T_);
  rd.load(y, t0, T_);
  load_carry(t0);
  joined<T, true>(a, l, mu);
  GateMarks m;
  m.init(seqs);
  for (; t0 >= l.t_lo; t0 -= U) {
    const int n = (int)min((int64_t)U, l.t_hi - t0);
    m.tile(seqs, t0);
    Gate<KIND> q[U][CV];
    float hb[U][CV], s[CV], xs[U][CV], dh[U][CV];
#pragma unroll
    for (int e = 0; e < CV; ++e) s[e] = before[e];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < CV; ++e) {
        q[i][e] = gate_of<KIND>(to_f32(g[i].e[e]));
        xs[i][e] = to_f32(x[i].e[e]);
        dh[i][e] = to_f32(y[i].e[e]);
      }
    if (t0 > l.t_lo) {
      rg.load(g, t0 - U, T_);
      rx.load(x, t0 - U, T_);
      rd.load(y, t0 - U, T_);
      load_carry(t0 - U);
    }
    // the states before each token, from the one that the forward pass kept
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (__builtin_expect(m.starts >> i & 1, 0)) {
        const int32_t j = seqs.of(t0 + i);
#pragma unroll
        for (int e = 0; e < CV; ++e) s[e] = a.state_in && e < l.left ? a.state_in[(uint64_t)j * a.g.channels + l.c0 + e] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < CV; ++e) {
        hb[i][e] = s[e];
        s[e] = decayed(q[i][e].c, s[e]) + (KIND == LAPLEX_GATE_RATE ? xs[i][e] : q[i][e].w * xs[i][e]);
      }
    }
#pragma unroll
    for (int i = U - 1; i >= 0; --i) {
      if (i < n) {
        if (__builtin_expect((m.ends | m.outside) >> i & 1, 0)) {
          const int32_t j = m.ends >> i & 1 ? seqs.of(t0 + i) : 0;
#pragma unroll
          for (int e = 0; e < CV; ++e)
            mu[e] = m.ends >> i & 1 && a.dstate_out && e < l.left ? a.dstate_out[(uint64_t)j * a.g.channels + l.c0 + e] : 0.f;
        }
        float dg[CV], dx[CV];
#pragma unroll
        for (int e = 0; e < CV; ++e) {
          const float lam = dh[i][e] + mu[e];
          if (KIND == LAPLEX_GATE_RATE) {
            dg[e] = -q[i][e].a * (hb[i][e] * lam);
            dx[e] = lam;
          } else {
            dx[e] = q[i][e].w * lam;
            dg[e] = q[i][e].a * ((hb[i][e] - xs[i][e]) * dx[e]);
          }
          mu[e] = decayed(q[i][e].c, lam);
        }
        if (__builtin_expect(m.outside >> i & 1, 0)) {
#pragma unroll
          for (int e = 0; e < CV; ++e) dg[e] = dx[e] = mu[e] = 0.f;
        }
        if (l.left) {
          const uint64_t at = (uint64_t)(t0 + i) * a.g.channels + l.c0;
          store_piece(static_cast<T*>(a.dgate) + at, l.left, dg);
          store_piece(static_cast<T*>(a.dx) + at, l.left, dx);
        }
        if (__builtin_expect(a.dstate_in && (m.starts >> i & 1), 0)) {
          const int32_t j = seqs.of(t0 + i);
#pragma unroll
          for (int e = 0; e < CV; ++e)
            if (e < l.left) a.dstate_in[(uint64_t)j * a.g.channels + l.c0 + e] = mu[e];
        }
      }
    }
  }
}

// Empty sequences: what comes in goes out.
__global__ __launch_bounds__(256) void k_gated_empty(GateSeqs s, uint32_t channels, const float* __restrict__ in, float* __restrict__ out) {
  for (int32_t j = blockIdx.x; j < s.seqs; j += gridDim.x) {
    if (s.at(j + 1) > s.at(j)) continue;
    for (uint32_t c = threadIdx.x; c < channels; c += 256) {
      const uint64_t at = (uint64_t)j * channels + c;
      out[at] = in ? in[at] : 0.f;
    }
  }
}

// ------------------------------------------------------------------ launches
struct GatePlan {
  uint32_t segs, ctiles;
  int64_t seg_len;
};
// About as many waves as the chip holds at once (256 CUs x 8), segments of at least four tiles.
constexpr uint64_t kGateUnits = 2048, kGateLeast = 64;
static GatePlan gate_plan(uint32_t channels, uint64_t tokens, int cv) {
  GatePlan p;
  p.ctiles = (channels + kWave * cv - 1) / (kWave * cv);
  const uint64_t want = std::max<uint64_t>(1, kGateUnits / p.ctiles);
  uint64_t len = std::max<uint64_t>(kGateLeast, (tokens + want - 1) / want);
  len = (len + kGateChunk - 1) / kGateChunk * kGateChunk;
  p.seg_len = (int64_t)len;
  p.segs = (uint32_t)((tokens + len - 1) / len);
  return p;
}
// (a segment is at least tokens / want long, so there are at most `want`, and at most tokens / least rounded up)
size_t gated_scan_bytes(uint32_t channels, uint64_t tokens) {
  const uint64_t ctiles = (channels + kWave * 2 - 1) / (kWave * 2);  // the fewest, with two channels a lane
  const uint64_t segs = std::min<uint64_t>(std::max<uint64_t>(1, kGateUnits / ctiles), (tokens + kGateLeast - 1) / kGateLeast);
  if (segs <= 1) return 0;
  return ((size_t)segs * channels * 8 + segs * 4 + 255) & ~size_t(255);
}

static hipError_t gate_ready(GateArgs& a, const GateShape& g, void* ws) {
  const GatePlan p = gate_plan(g.channels, g.tokens, g.dtype == LAPLEX_BF16 ? 2 : 1);
  a.g = g;
  a.seg_len = p.seg_len;
  a.segs = p.segs;
  a.ctiles = p.ctiles;
  if (p.segs > 1) {
    if ((size_t)p.segs * (g.channels * 8ull + 4) > gated_scan_bytes(g.channels, g.tokens)) return hipErrorInvalidValue;
    a.agg_c = static_cast<float*>(ws);
    a.agg_b = a.agg_c + (size_t)p.segs * g.channels;
    a.reset = reinterpret_cast<uint32_t*>(a.agg_b + (size_t)p.segs * g.channels);
  }
  return hipSuccess;
}
template <typename F>
static void by_type(const GateShape& g, F f) {
  const bool rate = g.kind == LAPLEX_GATE_RATE;
  if (g.dtype == LAPLEX_BF16) rate ? f(bf16{}, std::integral_constant<int, LAPLEX_GATE_RATE>{}) : f(bf16{}, std::integral_constant<int, LAPLEX_GATE_SIGMOID>{});
  else rate ? f(float{}, std::integral_constant<int, LAPLEX_GATE_RATE>{}) : f(float{}, std::integral_constant<int, LAPLEX_GATE_SIGMOID>{});
}
static hipError_t gate_empty(const GateShape& g, const float* in, float* out, hipStream_t s) {
  if (!out || (!g.offsets && g.tokens)) return hipSuccess;  // (equal lengths of at least one token: no empty sequence)
  const GateSeqs q{g.offsets, g.offsets ? 0 : (int64_t)(g.tokens / g.seqs), (int32_t)g.seqs};
  LAPLEX_LAUNCH("k_gated_empty", g.seqs, s, k_gated_empty<<<std::min(g.seqs, 2048u), 256, 0, s>>>(q, g.channels, in, out));
  return hipGetLastError();
}

hipError_t gated_scan(const GateShape& g, const float* state_in, float* state_out, void* h, float* carries, void* ws, hipStream_t s) {
  hipError_t err = gate_empty(g, state_in, state_out, s);
  if (err != hipSuccess || g.tokens == 0) return err;
  GateArgs a{};
  if ((err = gate_ready(a, g, ws)) != hipSuccess) return err;
  a.state_in = state_in;
  a.state_out = state_out;
  a.h = h;
  a.carries = carries;
  const unsigned blocks = (unsigned)(((uint64_t)a.segs * a.ctiles + kGateWaves - 1) / kGateWaves);
  by_type(g, [&](auto t, auto kind) {
    using T = decltype(t);
    if (a.segs > 1) LAPLEX_LAUNCH("k_gated_aggregate", g.tokens, s, k_gated<T, kind(), false><<<blocks, kWave * kGateWaves, 0, s>>>(a));
    LAPLEX_LAUNCH("k_gated", g.tokens, s, k_gated<T, kind(), true><<<blocks, kWave * kGateWaves, 0, s>>>(a));
  });
  return hipGetLastError();
}

hipError_t gated_scan_backward(const GateShape& g, const float* carries, const void* dh, const float* state_in,
                               const float* dstate_out, void* dgate, void* dx, float* dstate_in, void* ws, hipStream_t s) {
  hipError_t err = gate_empty(g, dstate_out, dstate_in, s);
  if (err != hipSuccess || g.tokens == 0) return err;
  GateArgs a{};
  if ((err = gate_ready(a, g, ws)) != hipSuccess) return err;
  a.state_in = state_in;
  a.carries_in = carries;
  a.dh = dh;
  a.dstate_out = dstate_out;
  a.dgate = dgate;
  a.dx = dx;
  a.dstate_in = dstate_in;
  const unsigned blocks = (unsigned)(((uint64_t)a.segs * a.ctiles + kGateWaves - 1) / kGateWaves);
  by_type(g, [&](auto t, auto kind) {
    using T = decltype(t);
    if (a.segs > 1)
      LAPLEX_LAUNCH("k_gated_back_aggregate", g.tokens, s, k_gated_back_aggregate<T, kind()><<<blocks, kWave * kGateWaves, 0, s>>>(a));
    LAPLEX_LAUNCH("k_gated_back", g.tokens, s, k_gated_back<T, kind()><<<blocks, kWave * kGateWaves, 0, s>>>(a));
  });
  return hipGetLastError();
}

// ------------------------------------------------------------------ one token
template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_gated_step(GateShape g, const int32_t* __restrict__ slots, uint32_t pool,
                                                    float* __restrict__ state, T* __restrict__ h) {
  const uint32_t per = (g.channels + 255) / 256, row = blockIdx.x / per, c = blockIdx.x % per * 256 + threadIdx.x;
  if (c >= g.channels) return;
  const int64_t slot = slots ? (int64_t)slots[row] : (int64_t)row;
  T* out = h + (uint64_t)row * g.channels + c;
  if (slot < 0 || slot >= (int64_t)pool) {
    *out = from_f32<T>(0.f);
    return;
  }
  const Gate<KIND> q = gate_of<KIND>(to_f32(static_cast<const T*>(g.gate)[row * g.gate_token + c]));
  const float x = to_f32(static_cast<const T*>(g.x)[row * g.x_token + c]);
  float* at = state + (uint64_t)slot * g.channels + c;
  const float s = decayed(q.c, *at) + (KIND == LAPLEX_GATE_RATE ? x : q.w * x);
  *at = s;
  *out = from_f32<T>(s);
}

hipError_t gated_scan_step(const GateShape& g, const int32_t* slots, uint32_t pool, float* state, void* h, hipStream_t s) {
  const uint64_t blocks = (uint64_t)g.seqs * ((g.channels + 255) / 256);
  by_type(g, [&](auto t, auto kind) {
    using T = decltype(t);
    LAPLEX_LAUNCH("k_gated_step", g.seqs, s, k_gated_step<T, kind()><<<(unsigned)blocks, 256, 0, s>>>(g, slots, pool, state, static_cast<T*>(h)));
  });
  return hipGetLastError();
}

}  // namespace laplex
