// Gated linear recurrence: forward, backward, and the single-token form.
//
//   h_t = a_t h_{t-1} + w_t x_t,   rate: a = exp(-r), w = 1;   sigmoid: a = s(z), w = 1 - a.
//   l_t = dh_t + a_{t+1} l_{t+1},  dx = w l,  dr = -a h_{t-1} l,  dz = a w (h_{t-1} - x) l.
//
// A wave takes 64 channels of one segment of the packed tokens, 16 tokens at a
// time, so that 16 rows of each tensor are on their way at once; nothing is
// exchanged between lanes.  Where sequences and channels alone do not fill the
// chip, the tokens are cut into segments: a pass over their aggregates (the
// decay over a segment and its state from zero), their join, then the whole
// pass.  Segments are cut without regard to sequences: a token that begins a
// sequence replaces the state before it, whatever that is.
//
// Memory bounds the passes: under the profiler 8 x 2048 tokens x 4096 channels in
// bfloat16 take 52 us for the forward's aggregates (5.1 TB/s), 78 for the whole
// pass (5.4), 46 and 128 for the backward's (5.9 with what the caches hold, 5.4),
// 6 for each join, 316 together; without it the calls take 303, where the bytes
// that cannot be done without take 169 at the rate of a plain copy (6.35 TB/s).
#include <algorithm>
#include <type_traits>

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

// exp(-y) of a gate's y.  Base 2 takes y log2 e: at y = 80 that product's rounding alone would put the result off by up to
// 44 2^-24 of it, and the constant's by 18.  So y meets a head of log2 e, in bfloat16 16 bits, whose product with the 8 of y is
// exact, and what is left out (in float also what the product rounds off) goes into a factor next to 1; decays are then off by
// 4 2^-24.  The head is rounded down, by more than the product's rounding can make up: for y >= 0 the factor is 1 at most, and
// the limits of a y without a sign (ABS) cost nothing.  They keep it a number where the result is 0 (or infinite) and
// it would not be one.  (16384 tokens x 4096 channels in bfloat16, forward and backward: 306 us, without the factor 304.)
template <typename T, bool ABS>
__device__ __forceinline__ float exp_of_minus(float y) {
  constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.6931471805599453094;
  constexpr float kHead = sizeof(T) == 2 ? 0x1.7154p0f : 0x1.715474p0f;
  const float t = -y * kHead;
  float factor;
  if constexpr (sizeof(T) == 2) factor = fmaf(-y, (float)((kLog2e - kHead) * kLn2), 1.f);
  else factor = fmaf(fmaf(-y, (float)(kLog2e - kHead), fmaf(-y, kHead, -t)), (float)kLn2, 1.f);
  factor = ABS ? __builtin_amdgcn_fmed3f(factor, 0.f, 1.f) : __builtin_amdgcn_fmed3f(factor, 0.5f, 2.f);
  return __builtin_amdgcn_exp2f(t) * factor;
}

template <int KIND>
struct Gate {
  float c, w;  // the decay as above, the input's weight
  bool near;   // near_one(c)
};
template <int KIND>
__device__ __forceinline__ float decayed(const Gate<KIND>& q, float s) { return fmaf(q.c, s, q.near ? s : 0.f); }
template <typename T, int KIND>
__device__ __forceinline__ Gate<KIND> gate_of(float g) {
  Gate<KIND> r;
  if constexpr (KIND == LAPLEX_GATE_RATE) {
    const float e = exp_of_minus<T, false>(g);
    // 1 - exp(-g): its series up to g = 0.3, where the first term left out is below 2^-25 of it
    float p = fmaf(g, -1.f / 8, 1.f);
    p = fmaf(g * p, -1.f / 7, 1.f);
    p = fmaf(g * p, -1.f / 6, 1.f);
    p = fmaf(g * p, -1.f / 5, 1.f);
    p = fmaf(g * p, -1.f / 4, 1.f);
    p = fmaf(g * p, -1.f / 3, 1.f);
    p = fmaf(g * p, -1.f / 2, 1.f);
    const float q = g < 0.3f ? g * p : 1.f - e;
    r.w = 1.f;
    r.near = g >= 0.f && q <= 0.5f;
    r.c = r.near ? -fabsf(q) : e;  // (a rate of -0.0 has a distance of -0.0, which would lose the mark)
  } else {
    const float e = exp_of_minus<T, true>(fabsf(g));
    const float big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
    r.near = g >= 0.f;
    r.w = r.near ? small : big;
    r.c = r.near ? -small : small;
  }
  return r;
}

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
        if (o >= t0 && o < t0 + U && j < s.seqs && s.at(j + 1) > o) m |= 1u << (o - t0);  // (offsets need not ascend)
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
// A lane has one channel; lanes past the last one have that one too, and write what it writes.  Rows are taken one after
// the other (STEP 1 or -1): their address is the wave's, and moves on by scalar additions, to which a load adds 32 bits.
// Rows past the last token are read as it.  What the whole pass reads (LAST) and writes goes past the caches, which are left
// to what the aggregates have read (16384 tokens x 4096 channels in bfloat16, forward and backward: 316 us, through the
// caches 350; 65536 x 256 in float 74, 83; the loads alone, as all of this is now: 303 and 306, 69 and 72 for inputs that change from
// call to call; for the same ones again, which a part of the caches still holds, 304 and 300, 65 and 62).
// A bfloat16 is held as the word that its load makes, and becomes a float where it is used: held as what it is, two are packed
// into a register, or masked, as soon as they arrive, which is waited for at the end of each tile (16384 tokens x 4096 channels,
// aggregates of the forward and the backward: 84 and 67 us so, 52 and 46 now).  Which width avoids that differs by loop.
template <typename T, bool LAST>
using Raw = std::conditional_t<sizeof(T) == 2, std::conditional_t<LAST, uint32_t, uint16_t>, float>;
__device__ __forceinline__ float value_of(float v) { return v; }
__device__ __forceinline__ float value_of(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float value_of(uint16_t v) { return value_of((uint32_t)v); }
template <typename T, int STEP, bool LAST>
struct Rows {
  typedef __attribute__((address_space(1))) char* Global;
  Global at;      // the first channel of the row that is next
  int64_t token;  // bytes
  int32_t left;   // tokens behind it
  __device__ __forceinline__ Rows(const void* p, int64_t stride, int64_t t0, int64_t tokens)
      : token(STEP * stride * (int64_t)sizeof(T)), left((int32_t)(tokens - 1 - t0)) {
    at = (Global)(uintptr_t)uniform64(reinterpret_cast<int64_t>(p) + min(t0, tokens - 1) * stride * (int64_t)sizeof(T));
  }
  // (INSIDE: neither this row nor the next one is past the last token)
  template <bool INSIDE>
  __device__ __forceinline__ void move() {
    at += INSIDE || (STEP > 0 ? left > 0 : left >= 0) ? token : 0;
    left -= STEP;
  }
  template <bool INSIDE>
  __device__ __forceinline__ Raw<T, LAST> get(uint32_t off) {
    using W = std::conditional_t<sizeof(T) == 2, uint16_t, float>;
    const __attribute__((address_space(1))) W* p = (const __attribute__((address_space(1))) W*)(at + off);
    const Raw<T, LAST> v = LAST ? __builtin_nontemporal_load(p) : *p;
    move<INSIDE>();
    return v;
  }
  template <bool INSIDE>
  __device__ __forceinline__ void put(uint32_t off, bool real, float v) {
    if (real) __builtin_nontemporal_store(from_f32<T>(v), (__attribute__((address_space(1))) T*)(at + off));
    move<INSIDE>();
  }
};
// bytes to the lane's channel, given anew for each tile: else its 64-bit form is kept, and each row's address is formed in
// vector registers
struct Off {
  uint32_t bytes;
  template <typename T>
  __device__ __forceinline__ Off(T, int64_t channel) : bytes((uint32_t)channel * (uint32_t)sizeof(T)) {}
  __device__ __forceinline__ uint32_t now() {
    asm volatile("" : "+v"(bytes));
    return bytes;
  }
};

// Keeps loads from being moved ahead over more than a few tokens, where they would need registers of their own.
__device__ __forceinline__ void every_fourth(int i) {
  if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
}

// The rows of a tile of two tensors, token by token, as they will be used
template <bool INSIDE, typename T, int STEP, bool LAST>
__device__ __forceinline__ void load_tile(uint32_t off, Rows<T, STEP, LAST>& p, Raw<T, LAST> (&v)[kGateU], Rows<T, STEP, LAST>& q, Raw<T, LAST> (&w)[kGateU]) {
#pragma unroll
  for (int j = 0; j < kGateU; ++j) {
    const int i = STEP > 0 ? j : kGateU - 1 - j;
    v[i] = p.template get<INSIDE>(off);
    w[i] = q.template get<INSIDE>(off);
    every_fourth(j);
  }
}
// A value that is there before what follows: a loop's first one that was still on its way would be waited for, with all
// that is, in every round; and one that is needed only later would be formed later, after the loads that follow it.
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

struct GateArgs {
  GateShape g;
  int64_t seg_len;  // a multiple of the tile
  uint32_t segs, ctiles;
  float *agg_c, *agg_b;  // segs x channels: decay over a segment, its state from zero and then what comes into it
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

struct Lane {
  uint32_t seg, ctile;
  int64_t c0, t_lo, t_hi;  // the channel, the segment's tokens
  bool valid;
  __device__ __forceinline__ Lane(const GateArgs& a) {
    const uint64_t unit = (uint64_t)blockIdx.x * kGateWaves + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    seg = (uint32_t)(unit / a.ctiles);
    ctile = (uint32_t)(unit % a.ctiles);
    valid = seg < a.segs;
    c0 = min((int64_t)ctile * kWave + lane_id(), (int64_t)a.g.channels - 1);
    t_lo = (int64_t)seg * a.seg_len;
    t_hi = min((int64_t)a.g.tokens, t_lo + a.seg_len);
  }
  // the channel of row j of a tensor of floats (null: 0)
  __device__ __forceinline__ float load(const GateArgs& a, const float* p, int64_t j) const { return p ? p[j * a.g.channels + c0] : 0.f; }
  __device__ __forceinline__ void store(const GateArgs& a, float* p, int64_t j, float v) const { p[j * a.g.channels + c0] = v; }
};
__device__ __forceinline__ GateSeqs gate_seqs(const GateArgs& a) {
  return {a.g.offsets, a.g.offsets ? 0 : (int64_t)(a.g.tokens / a.g.seqs), (int32_t)a.g.seqs};
}
// Values by a bit that all lanes share, without branches: v where the bit is set, else `other` (or 0).
__device__ __forceinline__ float where_bit(uint32_t bits, int i, float v, float other) {
  const uint32_t m = (uint32_t)((int32_t)(bits << (31 - i)) >> 31);
  return __uint_as_float((__float_as_uint(v) & m) | (__float_as_uint(other) & ~m));
}
__device__ __forceinline__ float unless_bit(uint32_t bits, int i, float v) {
  return __uint_as_float(__float_as_uint(v) & ~(uint32_t)((int32_t)(bits << (31 - i)) >> 31));
}
// For each set bit of a mask, in turn, a token of a tile: f(its sequence, the bit)
template <typename F>
__device__ __forceinline__ void each_marked(uint32_t mask, const GateSeqs& seqs, int64_t t0, F f) {
  while (mask) {
    f(seqs.of(t0 + __builtin_ctz(mask)), mask & -mask);
    mask &= mask - 1;
  }
}
// Empty sequences: what comes in goes out.  A unit's share of them.
__device__ __forceinline__ void pass_empty(const GateArgs& a, const Lane& l, const GateSeqs& seqs, const float* in, float* out) {
  if (!a.g.offsets || !out) return;
  for (int32_t j = l.seg; j < seqs.seqs; j += a.segs)
    if (seqs.at(j + 1) <= seqs.at(j)) l.store(a, out, j, l.load(a, in, j));
}

// ------------------------------------------------------------------ aggregates
// A segment's decay and its state from zero, b_n + a_n b_{n-1} + a_n a_{n-1} b_{n-2} + ..., from its last token to its first
// (BACK: mu from zero, a_1 dh_1 + a_1 a_2 dh_2 + ..., from the first to the last): one product and one sum a token, it ends where
// a sequence begins (BACK: ends), and it leaves in the caches what the whole pass, which goes the other way, reads first.
template <typename T, int KIND, bool BACK>
__global__ __launch_bounds__(kWave* kGateWaves) void k_gated_aggregate(GateArgs a) {
  constexpr int U = kGateU;
  const Lane l(a);
  if (!l.valid || l.seg == (BACK ? 0 : a.segs - 1)) return;  // (nothing comes after it)
  const GateSeqs seqs = gate_seqs(a);
  const int64_t T_ = (int64_t)a.g.tokens;
  float p = 1.f, s = 0.f;
  Raw<T, false> g[U], v[U];
  const int64_t tiles = (l.t_hi - l.t_lo + U - 1) / U, step = BACK ? U : -U;
  int64_t t0 = BACK ? l.t_lo : l.t_lo + (tiles - 1) * U;
  const int64_t from = BACK ? t0 : t0 + U - 1;
  Rows<T, BACK ? 1 : -1, false> rg(a.g.gate, a.g.gate_token, from, T_), rv(BACK ? a.dh : a.g.x, BACK ? (int64_t)a.g.channels : a.g.x_token, from, T_);
  Off off(T{}, l.c0);
  load_tile<false>(off.now(), rg, g, rv, v);
  GateMarks m;
  m.init(seqs);
  uint32_t none, stop;
  const auto marks = [&] {
    m.tile(seqs, t0);
    const int n = (int)min((int64_t)U, l.t_hi - t0);
    none = m.outside | (n < U ? ~0u << n & (1u << U) - 1 : 0u);
    stop = (BACK ? m.ends : m.starts) | none;
  };
  const auto input = [&](const Gate<KIND>& q, int i) { return BACK || KIND == LAPLEX_GATE_RATE ? value_of(v[i]) : q.w * value_of(v[i]); };
  // a tile, four tokens at a time, whose places the next one's rows take
  const auto tile = [&](auto inside) {
    const uint32_t o = off.now();
#pragma unroll
    for (int j0 = 0; j0 < U; j0 += 4) {
#pragma unroll
      for (int j = j0; j < j0 + 4; ++j) {
        const int i = BACK ? j : U - 1 - j;
        const Gate<KIND> q = gate_of<T, KIND>(value_of(g[i]));
        const float b = input(q, i);
        if (BACK) p = decayed(q, p);
        s = fmaf(p, b, s);
        if (!BACK) p = decayed(q, p);
      }
      settle(p);
      settle(s);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = j0; j < j0 + 4; ++j) {
        const int i = BACK ? j : U - 1 - j;
        g[i] = rg.template get<decltype(inside)::value>(o);
        v[i] = rv.template get<decltype(inside)::value>(o);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  marks();
  for (int64_t k = 0; k + 1 < tiles && !stop; ++k) {
    tile(std::integral_constant<bool, !BACK>{});  // (backwards, the next one may be the last)
    t0 += step;
    marks();
  }
  // The last tile, or the one where a sequence ends it.  The first to be met of what does: that token counts if it is one, with
  // what comes into its sequence, those beyond do not.
  const bool cut = stop != 0;
  const int h = BACK ? __builtin_ctz(stop | 1u << U) : 31 - __builtin_clz(stop | 1u);
  const uint32_t bit = cut ? 1u << h : 0u, gone = cut ? (BACK ? ~0u << h : (bit << 1) - 1) & ~(bit & ~none) : 0u;
  const float w = bit & ~none ? l.load(a, BACK ? a.dstate_out : a.state_in, seqs.of(t0 + h)) : 0.f;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int i = BACK ? j : U - 1 - j;
    const Gate<KIND> q = gate_of<T, KIND>(value_of(g[i]));
    const float b = input(q, i);
    const float c = unless_bit(gone, i, q.c), d = unless_bit(gone, i, where_bit(bit, i, BACK ? b + w : decayed(q, w) + b, b));
    if (BACK) p = decayed(c, p);
    s = fmaf(p, d, s);
    if (!BACK) p = decayed(c, p);
  }
  l.store(a, a.agg_c, l.seg, p);
  l.store(a, a.agg_b, l.seg, s);
  if (l.ctile == 0 && lane_id() == 0) a.reset[l.seg] = cut;
}

// ------------------------------------------------------------------ forward
template <typename T, int KIND>
__global__ __launch_bounds__(kWave* kGateWaves) void k_gated(GateArgs a) {
  constexpr int U = kGateU;
  const Lane l(a);
  if (!l.valid) return;
  const GateSeqs seqs = gate_seqs(a);
  const int64_t T_ = (int64_t)a.g.tokens;
  Rows<T, 1, true> rg(a.g.gate, a.g.gate_token, l.t_lo, T_), rx(a.g.x, a.g.x_token, l.t_lo, T_), rh(a.h, a.g.channels, l.t_lo, T_);
  Off off(T{}, l.c0);
  float s = l.seg ? l.load(a, a.agg_b, l.seg) : 0.f;
  Raw<T, true> g[U], x[U];
  load_tile<false>(off.now(), rg, g, rx, x);
  settle(s);
  pass_empty(a, l, seqs, a.state_in, a.state_out);
  GateMarks m;
  m.init(seqs);
  const auto input = [&](const Gate<KIND>& q, int i) { return KIND == LAPLEX_GATE_RATE ? value_of(x[i]) : q.w * value_of(x[i]); };
  for (int64_t t0 = l.t_lo;; t0 += U) {
    // tiles without a mark but the last, and but one that has the last tokens behind it
    for (;; t0 += U) {
      m.tile(seqs, t0);
      if (a.carries) l.store(a, a.carries, t0 / U, s);
      if (m.starts | m.ends | m.outside || t0 + U >= l.t_hi || t0 + 2 * U >= T_) break;
      const uint32_t o = off.now();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const Gate<KIND> q = gate_of<T, KIND>(value_of(g[i]));
        s = decayed(q, s) + input(q, i);
        g[i] = rg.template get<true>(o);  // a row of the next tile takes the place of each as it is used
        x[i] = rx.template get<true>(o);
        rh.template put<true>(o, true, s);
        every_fourth(i);
      }
    }
    const int n = (int)min((int64_t)U, l.t_hi - t0);
    float c[U], b[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const Gate<KIND> q = gate_of<T, KIND>(value_of(g[i]));
      c[i] = q.c;
      b[i] = input(q, i);
    }
    // a token that begins a sequence is its own state: the initial one goes into its input
    each_marked(m.starts, seqs, t0, [&](int32_t j, uint32_t bit) {
      const float v = l.load(a, a.state_in, j);
#pragma unroll
      for (int i = 0; i < U; ++i) b[i] = where_bit(bit, i, decayed(c[i], v) + b[i], b[i]);
    });
    const uint32_t fresh = m.starts | m.outside;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      s = unless_bit(m.outside, i, decayed(c[i], unless_bit(fresh, i, s)) + b[i]);
      b[i] = s;
      rh.template put<false>(off.bytes, i < n, s);
    }
    if (a.state_out)
      each_marked(m.ends, seqs, t0, [&](int32_t j, uint32_t bit) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) v = where_bit(bit, i, b[i], v);
        l.store(a, a.state_out, j, v);
      });
    if (t0 + U >= l.t_hi) return;
    load_tile<false>(off.now(), rg, g, rx, x);
  }
}

// ------------------------------------------------------------------ backward
// The carry is mu_t = a_t l_t, which token t - 1 receives: mu_t = a_t (mu_{t+1} + dh_t).
template <typename T, int KIND>
__global__ __launch_bounds__(kWave* kGateWaves) void k_gated_back(GateArgs a) {
  constexpr int U = kGateU;
  const Lane l(a);
  if (!l.valid) return;
  const GateSeqs seqs = gate_seqs(a);
  const int64_t T_ = (int64_t)a.g.tokens;
  float mu = l.seg + 1 < a.segs ? l.load(a, a.agg_b, l.seg) : 0.f;
  Raw<T, true> g[U], x[U], y[U];
  int64_t t0 = l.t_lo + (l.t_hi - l.t_lo - 1) / U * U;
  const int64_t from = t0 + U - 1;
  Rows<T, -1, true> rg(a.g.gate, a.g.gate_token, from, T_), rx(a.g.x, a.g.x_token, from, T_), rd(a.dh, a.g.channels, from, T_),
      out_g(a.dgate, a.g.channels, from, T_), out_x(a.dx, a.g.channels, from, T_);
  Off off(T{}, l.c0);
  const auto rows = [&](auto inside, uint32_t o) {
#pragma unroll
    for (int i = U - 1; i >= 0; --i) {
      g[i] = rg.template get<decltype(inside)::value>(o);
      x[i] = rx.template get<decltype(inside)::value>(o);
      y[i] = rd.template get<decltype(inside)::value>(o);
    }
  };
  rows(std::false_type{}, off.now());
  float before = l.load(a, a.carries_in, t0 / U);
  settle(mu);
  pass_empty(a, l, seqs, a.dstate_out, a.dstate_in);
  GateMarks m;
  m.init(seqs);
  for (; t0 >= l.t_lo; t0 -= U) {
    const int n = (int)min((int64_t)U, l.t_hi - t0);
    m.tile(seqs, t0);
    // each token's decay, the state before it, its input and gradient (and, with marks, what it hands on)
    float c[U], hb[U] = {}, xs[U], dh[U], s = before;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      c[i] = value_of(g[i]);
      xs[i] = value_of(x[i]);
      dh[i] = value_of(y[i]);
    }
    const uint32_t o = off.now();
    if (t0 > l.t_lo) {
      rows(std::true_type{}, o);
      before = l.load(a, a.carries_in, t0 / U - 1);
    }
    const uint32_t none = m.outside | (n < U ? ~0u << n : 0u);
    const auto tile = [&](auto all) {
      constexpr bool ALL = decltype(all)::value;  // no marks
      // the states before each token, from the one that the forward pass kept
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const Gate<KIND> q = gate_of<T, KIND>(c[i]);
        c[i] = q.c;
        if (!ALL) s = where_bit(m.starts, i, hb[i], s);
        hb[i] = s;
        s = decayed(q, s) + (KIND == LAPLEX_GATE_RATE ? xs[i] : q.w * xs[i]);
      }
#pragma unroll
      for (int i = U - 1; i >= 0; --i) {
        const float lam = dh[i] + (ALL ? mu : unless_bit(m.ends, i, mu)), av = decay_value(c[i]);
        float dg, dx;
        if (KIND == LAPLEX_GATE_RATE) {
          dx = lam;
          dg = -av * (hb[i] * lam);
        } else {
          dx = (near_one(c[i]) ? -c[i] : 1.f - c[i]) * lam;  // (a decay near 1 is kept as a - 1)
          dg = av * ((hb[i] - xs[i]) * dx);
        }
        mu = decayed(c[i], lam);
        if (!ALL) {
          dg = unless_bit(none, i, dg);
          dx = unless_bit(none, i, dx);
          dh[i] = mu = unless_bit(none, i, mu);
        }
        out_g.template put<ALL>(o, ALL || i < n, dg);
        out_x.template put<ALL>(o, ALL || i < n, dx);
      }
    };
    if (__builtin_expect(!(m.starts | m.ends | m.outside) && n == U, 1)) {
      tile(std::true_type{});
    } else {
      // initial states in the places of those before; what comes into a sequence's last token goes into its gradient
      each_marked(m.starts, seqs, t0, [&](int32_t j, uint32_t bit) {
        const float v = l.load(a, a.state_in, j);
#pragma unroll
        for (int i = 0; i < U; ++i) hb[i] = where_bit(bit, i, v, hb[i]);
      });
      each_marked(m.ends, seqs, t0, [&](int32_t j, uint32_t bit) {
        const float v = l.load(a, a.dstate_out, j);
#pragma unroll
        for (int i = 0; i < U; ++i) dh[i] = where_bit(bit, i, dh[i] + v, dh[i]);
      });
      tile(std::false_type{});
      if (a.dstate_in)
        each_marked(m.starts, seqs, t0, [&](int32_t j, uint32_t bit) {
          float v = 0.f;
#pragma unroll
          for (int i = 0; i < U; ++i) v = where_bit(bit, i, dh[i], v);
          l.store(a, a.dstate_in, j, v);
        });
    }
  }
}

// ------------------------------------------------------------------ join
// The segments' aggregates joined in turn: agg_b becomes what comes into each segment from those before it (BACK: after
// it).  A block takes a few channels, each of them in many stretches at once: a stretch's own aggregate, those of the
// stretches before it joined in steps of 1, 2, 4, ..., and then its segments, which registers hold meanwhile (1024 segments of
// 256 channels: 8.5 us of what is mostly latency; stretch after stretch, with 8 segments held, 13.3).
constexpr int kJoinChannels = 16, kJoinParts = 64, kJoinHeld = 16;
template <bool BACK>
__global__ __launch_bounds__(kJoinChannels* kJoinParts) void k_gated_join(GateArgs a) {
  __shared__ float sc[2][kJoinParts][kJoinChannels], sb[2][kJoinParts][kJoinChannels];
  __shared__ uint32_t sr[2][kJoinParts];
  const uint32_t lane = threadIdx.x % kJoinChannels, part = threadIdx.x / kJoinChannels;
  const uint64_t at = (uint64_t)blockIdx.x * kJoinChannels + lane, ch = min(at, (uint64_t)a.g.channels - 1);
  // (nothing comes after the last segment)
  const int32_t n = a.segs - 1, per = (n + kJoinParts - 1) / kJoinParts, lo = min(n, (int32_t)part * per), hi = min(n, lo + per);
  const auto seg = [&](int32_t k) { return (uint32_t)(BACK ? n - k : k); };
  constexpr int N = kJoinHeld;  // on their way
  float c = 1.f, b = 0.f, vc[N], vb[N];
  uint32_t r = 0, vr[N];
  const auto load = [&](int32_t k) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t q = seg(min(k + i, hi - 1));
      vr[i] = a.reset[q];
      vc[i] = a.agg_c[(uint64_t)q * a.g.channels + ch];
      vb[i] = a.agg_b[(uint64_t)q * a.g.channels + ch];
    }
  };
  for (int32_t k = lo; k < hi; k += N) {
    load(k);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (k + i < hi) {
        b = vr[i] ? vb[i] : fmaf(vc[i], b, vb[i]);
        c *= vc[i];
        r |= vr[i];
      }
  }
  // aggregates of all stretches up to this one
  int buf = 0;
#pragma unroll
  for (int step = 1; step <= kJoinParts; step *= 2, buf ^= 1) {
    sc[buf][part][lane] = c;
    sb[buf][part][lane] = b;
    if (lane == 0) sr[buf][part] = r;
    __syncthreads();
    if (step < kJoinParts && part >= (uint32_t)step) {
      const uint32_t q = part - step;
      if (!r) b = fmaf(c, sb[buf][q][lane], b);
      c *= sc[buf][q][lane];
      r |= sr[buf][q];
    }
  }
  float s = part ? sb[buf ^ 1][part - 1][lane] : 0.f;
  for (int32_t k = lo; k < hi; k += N) {
    if (hi - lo > N) load(k);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (k + i < hi) {
        if (at < a.g.channels) a.agg_b[(uint64_t)seg(k + i) * a.g.channels + ch] = s;
        s = vr[i] ? vb[i] : fmaf(vc[i], s, vb[i]);
      }
  }
  if (hi == n && lo < hi && at < a.g.channels) a.agg_b[(uint64_t)seg(n) * a.g.channels + ch] = s;
}

// Sequences that are all empty (there are no tokens): what comes in goes out.
__global__ __launch_bounds__(256) void k_gated_empty(uint64_t count, const float* __restrict__ in, float* __restrict__ out) {
  const uint64_t stride = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += stride) out[i] = in ? in[i] : 0.f;
}

// ------------------------------------------------------------------ launches
struct GatePlan {
  uint32_t segs, ctiles;
  int64_t seg_len;
};
// As many waves as the chip holds at once of the passes with 88 registers (five a SIMD), segments of at least four tiles
// (16384 tokens x 4096 channels in bfloat16, forward and backward: 304 us; 4096 waves 331, 6144 307, 8192 342).
constexpr uint64_t kGateUnits = 5120, kGateLeast = 64;
static GatePlan gate_plan(uint32_t channels, uint64_t tokens) {
  GatePlan p;
  p.ctiles = (channels + kWave - 1) / kWave;
  const uint64_t want = std::max<uint64_t>(1, kGateUnits / p.ctiles);
  uint64_t len = std::max<uint64_t>(kGateLeast, (tokens + want - 1) / want);
  len = (len + kGateChunk - 1) / kGateChunk * kGateChunk;
  p.seg_len = (int64_t)len;
  p.segs = (uint32_t)((tokens + len - 1) / len);
  return p;
}
// (a segment is at least tokens / want long, so there are at most `want`, and at most tokens / least rounded up)
size_t gated_scan_bytes(uint32_t channels, uint64_t tokens) {
  const uint64_t ctiles = (channels + kWave - 1) / kWave;
  const uint64_t segs = std::min<uint64_t>(std::max<uint64_t>(1, kGateUnits / ctiles), (tokens + kGateLeast - 1) / kGateLeast);
  if (segs <= 1) return 0;
  return ((size_t)segs * channels * 8 + segs * 4 + 255) & ~size_t(255);
}

static hipError_t gate_ready(GateArgs& a, const GateShape& g, void* ws) {
  const GatePlan p = gate_plan(g.channels, g.tokens);
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
  const uint64_t n = (uint64_t)g.seqs * g.channels;
  if (out) LAPLEX_LAUNCH("k_gated_empty", g.seqs, s, k_gated_empty<<<(unsigned)std::min<uint64_t>((n + 255) / 256, 4096), 256, 0, s>>>(n, in, out));
  return hipGetLastError();
}

hipError_t gated_scan(const GateShape& g, const float* state_in, float* state_out, void* h, float* carries, void* ws, hipStream_t s) {
  if (g.tokens == 0) return gate_empty(g, state_in, state_out, s);
  GateArgs a{};
  const hipError_t err = gate_ready(a, g, ws);
  if (err != hipSuccess) return err;
  a.state_in = state_in;
  a.state_out = state_out;
  a.h = h;
  a.carries = carries;
  const unsigned blocks = (unsigned)(((uint64_t)a.segs * a.ctiles + kGateWaves - 1) / kGateWaves);
  by_type(g, [&](auto t, auto kind) {
    using T = decltype(t);
    if (a.segs > 1) {
      LAPLEX_LAUNCH("k_gated_aggregate", g.tokens, s, k_gated_aggregate<T, kind(), false><<<blocks, kWave * kGateWaves, 0, s>>>(a));
      LAPLEX_LAUNCH("k_gated_join", a.segs, s, k_gated_join<false><<<(g.channels + kJoinChannels - 1) / kJoinChannels, kJoinChannels * kJoinParts, 0, s>>>(a));
    }
    LAPLEX_LAUNCH("k_gated", g.tokens, s, k_gated<T, kind()><<<blocks, kWave * kGateWaves, 0, s>>>(a));
  });
  return hipGetLastError();
}

hipError_t gated_scan_backward(const GateShape& g, const float* carries, const void* dh, const float* state_in,
                               const float* dstate_out, void* dgate, void* dx, float* dstate_in, void* ws, hipStream_t s) {
  if (g.tokens == 0) return gate_empty(g, dstate_out, dstate_in, s);
  GateArgs a{};
  const hipError_t err = gate_ready(a, g, ws);
  if (err != hipSuccess) return err;
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
    if (a.segs > 1) {
      LAPLEX_LAUNCH("k_gated_aggregate", g.tokens, s, k_gated_aggregate<T, kind(), true><<<blocks, kWave * kGateWaves, 0, s>>>(a));
      LAPLEX_LAUNCH("k_gated_join", a.segs, s, k_gated_join<true><<<(g.channels + kJoinChannels - 1) / kJoinChannels, kJoinChannels * kJoinParts, 0, s>>>(a));
    }
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
  const Gate<KIND> q = gate_of<T, KIND>(to_f32(static_cast<const T*>(g.gate)[row * g.gate_token + c]));
  const float x = to_f32(static_cast<const T*>(g.x)[row * g.x_token + c]);
  float* at = state + (uint64_t)slot * g.channels + c;
  const float s = decayed(q, *at) + (KIND == LAPLEX_GATE_RATE ? x : q.w * x);
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
