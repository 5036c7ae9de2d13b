// C-ABI entry points of the training-step operators: argument checks, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "../../include/laplex.h"
#include "laplex_host.hpp"
#include "laplex_train.hpp"

namespace {

using namespace laplex;

constexpr uint64_t kMaxTokens = 0x7FFFFFFFull;  // int32 offsets
constexpr uint32_t kMaxSeqs = 1u << 20, kMaxWidth = 1u << 24, kMaxVocab = 1u << 26, kMaxXentWidth = 1u << 20;
constexpr uint64_t kMaxXentTokens = 1ull << 28, kMaxTiles = (1ull << 24) - 1, kMaxBlocks = (1ull << 24) - 1;  // a launch has fewer than 2^32 threads

inline size_t elem(int dtype) { return dtype == LAPLEX_BF16 ? 2 : 4; }
inline bool is_dtype(int dtype) { return dtype == LAPLEX_F32 || dtype == LAPLEX_BF16; }

struct Extent {
  const void* p;
  size_t bytes;
};
template <size_t N, size_t M>
bool any_overlap(const Extent (&outs)[N], const Extent (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
    for (const Extent& x : ins)
      if (overlaps(outs[i].p, outs[i].bytes, x.p, x.bytes)) return true;
  }
  return false;
}
template <size_t N>
bool any_misaligned(const Extent (&v)[N], size_t a) {
  for (const Extent& x : v)
    if (misaligned(x.p, a)) return true;
  return false;
}

// ------------------------------------------------------------------ gated linear recurrence
laplex_status check_scan(const laplex_scan_shape* a) {
  if (!a) return LAPLEX_ERR_NULL;
  if (!is_dtype(a->dtype) || (a->gate != LAPLEX_GATE_RATE && a->gate != LAPLEX_GATE_SIGMOID) || a->channels == 0) return LAPLEX_ERR_ARG;
  if (a->tokens > kMaxTokens || a->seqs > kMaxSeqs || a->channels > kMaxWidth) return LAPLEX_ERR_SIZE;
  return LAPLEX_OK;
}
bool rows_bytes(const laplex_scan_shape& a, int64_t token, size_t* bytes) {
  *bytes = 0;
  if (token < 0) return false;
  if (a.tokens == 0) return true;
  const unsigned __int128 n = (unsigned __int128)(a.tokens - 1) * (uint64_t)token + a.channels;
  if (n > ((uint64_t)1 << 60)) return false;
  *bytes = (size_t)n * elem(a.dtype);
  return true;
}
GateShape gate_shape(const laplex_scan_shape& a, const void* gate, const void* x) {
  return {a.dtype, a.gate, a.seqs, a.channels, a.tokens, a.offsets, gate, x, a.gate_token, a.x_token};
}
inline uint64_t carries_of(const laplex_scan_shape& a) { return (a.tokens + kGateChunk - 1) / kGateChunk * a.channels; }

}  // namespace

extern "C" size_t laplex_gated_scan_workspace_bytes(const laplex_scan_shape* shape) {
  return check_scan(shape) == LAPLEX_OK ? gated_scan_bytes(shape->channels, shape->tokens) : 0;
}

extern "C" laplex_status laplex_gated_scan(const laplex_scan_shape* shape, const void* gate, const void* x, const float* state_in,
                                           float* state_out, void* h, float* carries, void* ws, size_t ws_bytes, hipStream_t stream) {
  const laplex_status st = check_scan(shape);
  if (st != LAPLEX_OK) return st;
  const laplex_scan_shape& a = *shape;
  if (a.seqs == 0) return a.tokens == 0 ? LAPLEX_OK : LAPLEX_ERR_ARG;
  if (!a.offsets && a.tokens % a.seqs != 0) return LAPLEX_ERR_ARG;
  if (a.tokens && (!gate || !x || !h)) return LAPLEX_ERR_NULL;
  if (a.tokens == 0 && !state_out) return LAPLEX_OK;
  const size_t e = elem(a.dtype), need = gated_scan_bytes(a.channels, a.tokens), sb = (size_t)a.seqs * a.channels * 4;
  if (need && !ws) return LAPLEX_ERR_NULL;
  size_t gb, xb;
  if (!rows_bytes(a, a.gate_token, &gb) || !rows_bytes(a, a.x_token, &xb)) return LAPLEX_ERR_ARG;
  const Extent words[] = {{a.offsets, (a.seqs + 1ull) * 4}, {state_in, sb}, {state_out, sb}, {carries, carries_of(a) * 4}};
  const Extent elems[] = {{gate, gb}, {x, xb}, {h, a.tokens * a.channels * e}};
  if (any_misaligned(words, 4) || any_misaligned(elems, e) || (need && misaligned(ws, 256))) return LAPLEX_ERR_ALIGN;
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  const Extent outs[] = {elems[2], words[2], words[3], {ws, need}}, ins[] = {elems[0], elems[1], words[0], words[1]};
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(gated_scan(gate_shape(a, gate, x), state_in, state_out, h, carries, ws, stream));
}

extern "C" laplex_status laplex_gated_scan_backward(const laplex_scan_shape* shape, const void* gate, const void* x,
                                                    const float* carries, const void* dh, const float* state_in,
                                                    const float* dstate_out, void* dgate, void* dx, float* dstate_in, void* ws,
                                                    size_t ws_bytes, hipStream_t stream) {
  const laplex_status st = check_scan(shape);
  if (st != LAPLEX_OK) return st;
  const laplex_scan_shape& a = *shape;
  if (a.seqs == 0) return a.tokens == 0 ? LAPLEX_OK : LAPLEX_ERR_ARG;
  if (!a.offsets && a.tokens % a.seqs != 0) return LAPLEX_ERR_ARG;
  if (a.tokens && (!gate || !x || !carries || !dh || !dgate || !dx)) return LAPLEX_ERR_NULL;
  if (a.tokens == 0 && !dstate_in) return LAPLEX_OK;
  const size_t e = elem(a.dtype), need = gated_scan_bytes(a.channels, a.tokens), sb = (size_t)a.seqs * a.channels * 4,
               tb = a.tokens * a.channels * e;
  if (need && !ws) return LAPLEX_ERR_NULL;
  size_t gb, xb;
  if (!rows_bytes(a, a.gate_token, &gb) || !rows_bytes(a, a.x_token, &xb)) return LAPLEX_ERR_ARG;
  const Extent words[] = {{a.offsets, (a.seqs + 1ull) * 4}, {state_in, sb}, {dstate_out, sb}, {carries, carries_of(a) * 4}, {dstate_in, sb}};
  const Extent elems[] = {{gate, gb}, {x, xb}, {dh, tb}, {dgate, tb}, {dx, tb}};
  if (any_misaligned(words, 4) || any_misaligned(elems, e) || (need && misaligned(ws, 256))) return LAPLEX_ERR_ALIGN;
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  const Extent outs[] = {elems[3], elems[4], words[4], {ws, need}},
               ins[] = {elems[0], elems[1], elems[2], words[0], words[1], words[2], words[3]};
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(gated_scan_backward(gate_shape(a, gate, x), carries, dh, state_in, dstate_out, dgate, dx, dstate_in, ws, stream));
}

extern "C" laplex_status laplex_gated_scan_step(const laplex_scan_shape* shape, const void* gate, const void* x, const int32_t* slots,
                                                uint32_t pool, float* state, void* h, hipStream_t stream) {
  const laplex_status st = check_scan(shape);
  if (st != LAPLEX_OK) return st;
  const laplex_scan_shape& a = *shape;
  if (a.tokens != a.seqs || (!slots && a.seqs > pool)) return LAPLEX_ERR_ARG;
  if (a.seqs == 0) return LAPLEX_OK;
  if ((uint64_t)a.seqs * ((a.channels + 255) / 256) > kMaxBlocks) return LAPLEX_ERR_SIZE;
  if (!gate || !x || !h || (!state && pool)) return LAPLEX_ERR_NULL;
  const size_t e = elem(a.dtype);
  size_t gb, xb;
  if (!rows_bytes(a, a.gate_token, &gb) || !rows_bytes(a, a.x_token, &xb)) return LAPLEX_ERR_ARG;
  const Extent outs[] = {{h, a.tokens * a.channels * e}, {state, (size_t)pool * a.channels * 4}};
  const Extent ins[] = {{gate, gb}, {x, xb}, {slots, a.seqs * 4ull}};
  if (misaligned(h, e) || misaligned(gate, e) || misaligned(x, e) || misaligned(state, 4) || misaligned(slots, 4)) return LAPLEX_ERR_ALIGN;
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(gated_scan_step(gate_shape(a, gate, x), slots, pool, state, h, stream));
}

// ------------------------------------------------------------------ linear softmax cross entropy
namespace {
laplex_status check_xent(int dtype, int id_bytes, uint64_t tokens, uint32_t vocab, uint32_t width) {
  if (!is_dtype(dtype) || (id_bytes != 4 && id_bytes != 8) || vocab == 0 || width == 0) return LAPLEX_ERR_ARG;
  if (tokens > kMaxXentTokens || vocab > kMaxVocab || width > kMaxXentWidth) return LAPLEX_ERR_SIZE;
  // logits: 2^38 of them, in tiles of 128 x 128
  if ((tokens / 128 + 1) * (vocab / 128 + 1) > kMaxTiles) return LAPLEX_ERR_SIZE;
  // tiles of the gradients' products, at the smallest 64 of the width by 32, are counted in 32 bits
  if ((width / 64 + 1ull) * (std::max<uint64_t>(tokens, vocab) / 32 + 1) >= 1ull << 31) return LAPLEX_ERR_SIZE;
  return LAPLEX_OK;
}
}  // namespace

namespace {
size_t xent_workspace(int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width, bool aligned) {
  if ((pass != 0 && pass != 1) || check_xent(dtype, 4, tokens, vocab, width) != LAPLEX_OK) return 0;
  return xent_bytes(pass, dtype, tokens, vocab, width, aligned);
}
}  // namespace

extern "C" size_t laplex_linear_cross_entropy_workspace_bytes(int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width) {
  return xent_workspace(pass, dtype, tokens, vocab, width, false);
}
extern "C" size_t laplex_linear_cross_entropy_workspace_bytes_aligned(int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width) {
  return xent_workspace(pass, dtype, tokens, vocab, width, true);
}

extern "C" laplex_status laplex_linear_cross_entropy(int dtype, const void* targets, int id_bytes, uint64_t tokens, const void* x,
                                                     const void* table, uint32_t vocab, uint32_t width, float scale, float* loss,
                                                     float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  const laplex_status st = check_xent(dtype, id_bytes, tokens, vocab, width);
  if (st != LAPLEX_OK) return st;
  if (tokens == 0) return LAPLEX_OK;
  if (!targets || !x || !table || !ws || (!loss && !lse)) return LAPLEX_ERR_NULL;
  const size_t e = elem(dtype), need = xent_bytes(0, dtype, tokens, vocab, width, xent_aligned(x, table));
  if (misaligned(targets, id_bytes) || misaligned(x, e) || misaligned(table, e) || misaligned(loss, 4) || misaligned(lse, 4) || misaligned(ws, 256))
    return LAPLEX_ERR_ALIGN;
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  const Extent outs[] = {{loss, tokens * 4}, {lse, tokens * 4}, {ws, need}},
               ins[] = {{targets, tokens * id_bytes}, {x, tokens * width * e}, {table, (size_t)vocab * width * e}};
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(xent({dtype, id_bytes, tokens, vocab, width, targets, x, table, scale}, loss, lse, ws, stream));
}

extern "C" laplex_status laplex_linear_cross_entropy_backward(int dtype, const void* targets, int id_bytes, uint64_t tokens, const void* x,
                                                              const void* table, uint32_t vocab, uint32_t width, float scale,
                                                              const float* lse, const float* dloss, const float* dlse, void* dx,
                                                              int table_dtype, void* dtable, void* ws, size_t ws_bytes,
                                                              hipStream_t stream) {
  const laplex_status st = check_xent(dtype, id_bytes, tokens, vocab, width);
  if (st != LAPLEX_OK) return st;
  if (table_dtype != dtype && table_dtype != LAPLEX_F32) return LAPLEX_ERR_ARG;
  if ((!dx || tokens == 0) && !dtable) return LAPLEX_OK;
  if (!ws || (tokens && (!targets || !x || !table || !lse || !dloss))) return LAPLEX_ERR_NULL;
  const size_t e = elem(dtype), te = elem(table_dtype), need = xent_bytes(1, dtype, tokens, vocab, width, xent_aligned(x, table));
  if ((tokens && misaligned(targets, id_bytes)) || misaligned(x, e) || misaligned(table, e) || misaligned(dx, e) || misaligned(dtable, te) ||
      misaligned(lse, 4) || misaligned(dloss, 4) || misaligned(dlse, 4) || misaligned(ws, 256))
    return LAPLEX_ERR_ALIGN;
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  const Extent outs[] = {{dx, tokens * width * e}, {dtable, (size_t)vocab * width * te}, {ws, need}},
               ins[] = {{targets, tokens * id_bytes}, {x, tokens * width * e}, {table, (size_t)vocab * width * e},
                        {lse, tokens * 4},            {dloss, tokens * 4},     {dlse, tokens * 4}};
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(xent_backward({dtype, id_bytes, tokens, vocab, width, targets, x, table, scale}, lse, dloss, dlse, dx, table_dtype, dtable, ws, stream));
}

// ------------------------------------------------------------------ AdamW
namespace {
// Whether two of the extents overlap of which at least one is written.  Sorted by their starts, an extent meets one
// before it only if that reaches past its start: the furthest end so far, of those written and of all.
struct Span {
  uintptr_t at, end;
  bool out;
};
bool spans_overlap(std::vector<Span>& v) {
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
  uintptr_t any = 0, out = 0;
  for (const Span& s : v) {
    if (s.at < out || (s.out && s.at < any)) return true;
    any = std::max(any, s.end);
    if (s.out) out = std::max(out, s.end);
  }
  return false;
}
// Checks of the tensors of a step (args), or of the moments' floats.
laplex_status check_tensors(const laplex_adamw_args* a, const laplex_adamw_tensor* t, uint32_t count) {
  const bool eight = !a || a->state_bits == 8;
  const size_t pe = a ? elem(a->dtype) : 4, ge = a ? elem(a->grad_dtype) : 0, se = eight ? 1 : 4;
  try {
    std::vector<Span> spans;
    spans.reserve(count * 7ull + 3);
    const auto add = [&](const void* p, size_t bytes, bool out) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      if (p) spans.push_back({at, at + bytes, out});
    };
    if (a) {
      add(a->step_dev, 4, false);
      add(a->lr_dev, 4, false);
      add(a->grad_scale, 4, false);
    }
    for (uint32_t i = 0; i < count; ++i) {
      const laplex_adamw_tensor& x = t[i];
      if (x.n == 0) continue;
      if (x.n > (1ull << 40)) return LAPLEX_ERR_SIZE;
      if ((a && (!x.p || !x.g)) || !x.m || !x.v || (eight && (!x.m_scale || !x.v_scale))) return LAPLEX_ERR_NULL;
      if (a && !std::isfinite(x.weight_decay)) return LAPLEX_ERR_ARG;
      if (misaligned(x.p, pe) || (a && misaligned(x.g, ge)) || misaligned(x.m, se) || misaligned(x.v, se) || misaligned(x.master, 4) ||
          (eight && (misaligned(x.m_scale, 4) || misaligned(x.v_scale, 4))))
        return LAPLEX_ERR_ALIGN;
      const size_t scales = (x.n + 255) / 256 * 4;
      add(x.p, x.n * pe, true);
      add(x.master, x.n * 4, true);
      if (a) add(x.g, x.n * ge, false);
      add(x.m, x.n * se, a != nullptr);
      add(x.v, x.n * se, a != nullptr);
      if (eight) {
        add(x.m_scale, scales, a != nullptr);
        add(x.v_scale, scales, a != nullptr);
      }
    }
    return spans_overlap(spans) ? LAPLEX_ERR_OVERLAP : LAPLEX_OK;
  } catch (const std::bad_alloc&) {
    return LAPLEX_ERR_SIZE;
  }
}
}  // namespace

extern "C" laplex_status laplex_adamw(const laplex_adamw_args* args, const laplex_adamw_tensor* tensors, uint32_t count, hipStream_t stream) {
  if (!args || (count && !tensors)) return LAPLEX_ERR_NULL;
  const laplex_adamw_args& a = *args;
  if (!is_dtype(a.dtype) || !is_dtype(a.grad_dtype) || (a.state_bits != 32 && a.state_bits != 8) || a.step == 0) return LAPLEX_ERR_ARG;
  if (!(a.beta1 >= 0 && a.beta1 < 1) || !(a.beta2 >= 0 && a.beta2 < 1) || !(a.eps >= 0) || !std::isfinite(a.eps) || !std::isfinite(a.lr))
    return LAPLEX_ERR_ARG;
  if (misaligned(a.step_dev, 4) || misaligned(a.lr_dev, 4) || misaligned(a.grad_scale, 4)) return LAPLEX_ERR_ALIGN;
  const laplex_status st = check_tensors(&a, tensors, count);
  if (st != LAPLEX_OK) return st;
  return from_hip(adamw(a, tensors, count, stream));
}

extern "C" laplex_status laplex_adamw_moments(const laplex_adamw_tensor* tensors, uint32_t count, hipStream_t stream) {
  if (count && !tensors) return LAPLEX_ERR_NULL;
  const laplex_status st = check_tensors(nullptr, tensors, count);
  if (st != LAPLEX_OK) return st;
  return from_hip(adamw_moments(tensors, count, stream));
}
