// C-ABI entry points of the sequence layers: argument checks, workspace
// layout, launches.
#include <hip/hip_runtime.h>

#include "../../include/laplex.h"
#include "laplex_host.hpp"
#include "laplex_layers.hpp"

namespace {

using namespace laplex;

constexpr uint64_t kMaxTokens = 0x7FFFFFFFull;  // int32 offsets
constexpr uint32_t kMaxSeqs = 1u << 20, kMaxHeads = 4096, kMaxChannels = 256, kMaxWidth = 1u << 24;
constexpr uint64_t kMaxBlocks = 1ull << 22;  // sequences x heads: a launch has fewer than 2^32 threads
constexpr uint64_t kMaxRows = 0xFFFFFFFFull;
constexpr uint32_t kMaxVocab = 1u << 26;
constexpr uint64_t kMaxEmbedTokens = 1ull << 28;

inline size_t elem(int dtype) { return dtype == LAPLEX_BF16 ? 2 : 4; }
inline bool is_dtype(int dtype) { return dtype == LAPLEX_F32 || dtype == LAPLEX_BF16; }

// Sizes alone; LAPLEX_OK also where there is nothing to do.
laplex_status check_shape(const laplex_attn_shape* a) {
  if (!a) return LAPLEX_ERR_NULL;
  if (!is_dtype(a->dtype)) return LAPLEX_ERR_ARG;
  if (a->heads == 0 || a->kv_heads == 0 || a->heads % a->kv_heads != 0 || a->dk == 0 || a->dv == 0) return LAPLEX_ERR_ARG;
  if (a->tokens > kMaxTokens || a->seqs > kMaxSeqs || a->heads > kMaxHeads || a->dk > kMaxChannels || a->dv > kMaxChannels)
    return LAPLEX_ERR_SIZE;
  if ((a->seqs + 1024ull) * a->heads > kMaxBlocks) return LAPLEX_ERR_SIZE;
  return LAPLEX_OK;
}

// Bytes from a view's first element to the end of its last; false if a stride is negative or the extent overflows.
bool view_bytes(uint64_t tokens, uint32_t heads, uint32_t width, int64_t token, int64_t head, size_t e, size_t* bytes) {
  *bytes = 0;
  if (token < 0 || head < 0) return false;
  if (tokens == 0) return true;
  const unsigned __int128 n = (unsigned __int128)(tokens - 1) * (uint64_t)token + (unsigned __int128)(heads - 1) * (uint64_t)head + width;
  if (n > ((uint64_t)1 << 60)) return false;
  *bytes = (size_t)n * e;
  return true;
}

struct Extent {
  const void* p;
  size_t bytes;
};
// whether one of `outs` overlaps another of them or one of `ins`
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

struct AttnWorkspace {
  void* pass;    // of one recurrence pass at a time
  float* sum;    // per query head gradients before they are added over a shared head
  double* drate; // partials of the rate gradient
};
AttnWorkspace carve_attn(void* ws, int pass, const laplex_attn_shape& a, size_t* total) {
  Carver c(ws);
  AttnWorkspace w{};
  size_t b = attn_pass_bytes(a.dtype, a.heads, a.dk, a.dv, a.tokens, false);
  if (pass == LAPLEX_ATTN_BACKWARD) b = std::max({b, attn_pass_bytes(a.dtype, a.heads, a.dv, a.dk, a.tokens, false), attn_pass_bytes(a.dtype, a.heads, a.dv, a.dk, a.tokens, true)});
  w.pass = c.take<void>(b);
  if (pass == LAPLEX_ATTN_BACKWARD) {
    if (a.heads != a.kv_heads) w.sum = c.take<float>(a.tokens * a.heads * std::max(a.dk, a.dv) * 4);
    w.drate = c.take<double>(a.seqs ? attn_drate_parts_most(a.dtype, a.seqs, a.heads, a.dv, a.dk, a.tokens) * a.heads * 8 : 0);
  }
  *total = (c.off + 255) & ~size_t(255);
  return w;
}

AttnPass base_pass(const laplex_attn_shape& a) {
  AttnPass p{};
  p.dtype = a.dtype;
  p.seqs = a.seqs;
  p.heads = a.heads;
  p.tokens = a.tokens;
  p.offsets = a.offsets;
  p.rate = a.rate;
  return p;
}

}  // namespace

extern "C" size_t laplex_decay_attn_workspace_bytes(int pass, const laplex_attn_shape* shape) {
  if (check_shape(shape) != LAPLEX_OK || (pass != LAPLEX_ATTN_FORWARD && pass != LAPLEX_ATTN_BACKWARD)) return 0;
  size_t total = 0;
  carve_attn(nullptr, pass, *shape, &total);
  return total;
}

extern "C" laplex_status laplex_decay_attn(const laplex_attn_shape* shape, const void* q, const void* k, const void* v,
                                           const float* state_in, float* state_out, void* o, void* ws, size_t ws_bytes,
                                           hipStream_t stream) {
  laplex_status st = check_shape(shape);
  if (st != LAPLEX_OK) return st;
  const laplex_attn_shape& a = *shape;
  if (a.seqs == 0) return a.tokens == 0 ? LAPLEX_OK : LAPLEX_ERR_ARG;
  if (!a.offsets && a.tokens % a.seqs != 0) return LAPLEX_ERR_ARG;
  if (!a.rate || (a.tokens && (!q || !k || !v || !o))) return LAPLEX_ERR_NULL;
  if (a.tokens == 0 && !state_out) return LAPLEX_OK;
  const size_t e = elem(a.dtype);
  size_t need = 0, qb, kb, vb;
  const AttnWorkspace w = carve_attn(ws, LAPLEX_ATTN_FORWARD, a, &need);
  if (need && !ws) return LAPLEX_ERR_NULL;
  if (!view_bytes(a.tokens, a.heads, a.dk, a.q_token, a.q_head, e, &qb) ||
      !view_bytes(a.tokens, a.kv_heads, a.dk, a.k_token, a.k_head, e, &kb) ||
      !view_bytes(a.tokens, a.kv_heads, a.dv, a.v_token, a.v_head, e, &vb))
    return LAPLEX_ERR_ARG;
  const size_t sb = (size_t)a.seqs * a.heads * a.dk * a.dv * 4;
  const Extent words[] = {{a.offsets, (a.seqs + 1ull) * 4}, {a.rate, a.heads * 4ull}, {state_in, sb}, {state_out, sb}};
  const Extent elems[] = {{q, qb}, {k, kb}, {v, vb}, {o, a.tokens * a.heads * a.dv * e}};
  if (any_misaligned(words, 4) || any_misaligned(elems, e) || misaligned(ws, 256)) return LAPLEX_ERR_ALIGN;
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  const Extent outs[] = {elems[3], words[3], {ws, need}}, ins[] = {elems[0], elems[1], elems[2], words[0], words[1], words[2]};
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  AttnPass p = base_pass(a);
  const uint32_t group = a.heads / a.kv_heads;
  p.K = a.dk;
  p.V = a.dv;
  p.x = {q, a.q_token, a.q_head, 1};
  p.y = {k, a.k_token, a.k_head, group};
  p.z = {v, a.v_token, a.v_head, group};
  p.c_pair = p.c_in = a.scale;
  p.c_add = 1.f;
  p.out = a.tokens ? o : nullptr;
  p.s_in = state_in;
  p.s_out = state_out;
  return from_hip(attn_pass(p, w.pass, stream));
}

extern "C" laplex_status laplex_decay_attn_backward(const laplex_attn_shape* shape, const void* q, const void* k, const void* v,
                                                    const void* go, const float* state_in, const float* dstate_out, void* dq,
                                                    void* dk, void* dv, float* drate, float* dstate_in, void* ws,
                                                    size_t ws_bytes, hipStream_t stream) {
  laplex_status st = check_shape(shape);
  if (st != LAPLEX_OK) return st;
  const laplex_attn_shape& a = *shape;
  if (a.seqs == 0 && a.tokens != 0) return LAPLEX_ERR_ARG;
  if (a.seqs && !a.offsets && a.tokens % a.seqs != 0) return LAPLEX_ERR_ARG;
  if (!a.rate || (a.tokens && (!q || !k || !v || !go || !dq || !dk || !dv))) return LAPLEX_ERR_NULL;
  const size_t e = elem(a.dtype);
  size_t need = 0, qb, kb, vb;
  const AttnWorkspace w = carve_attn(ws, LAPLEX_ATTN_BACKWARD, a, &need);
  if (need && !ws) return LAPLEX_ERR_NULL;
  if (!view_bytes(a.tokens, a.heads, a.dk, a.q_token, a.q_head, e, &qb) ||
      !view_bytes(a.tokens, a.kv_heads, a.dk, a.k_token, a.k_head, e, &kb) ||
      !view_bytes(a.tokens, a.kv_heads, a.dv, a.v_token, a.v_head, e, &vb))
    return LAPLEX_ERR_ARG;
  const size_t sb = (size_t)a.seqs * a.heads * a.dk * a.dv * 4, ob = a.tokens * a.heads * a.dv * e;
  const Extent outs[] = {{dq, a.tokens * a.heads * a.dk * e}, {dk, a.tokens * a.kv_heads * a.dk * e},
                         {dv, a.tokens * a.kv_heads * a.dv * e}, {drate, a.heads * 4ull}, {dstate_in, sb}, {ws, need}};
  const Extent ins[] = {{q, qb}, {k, kb}, {v, vb}, {go, ob}, {a.offsets, (a.seqs + 1ull) * 4}, {a.rate, a.heads * 4ull},
                        {state_in, sb}, {dstate_out, sb}};
  const Extent words[] = {outs[3], outs[4], ins[4], ins[5], ins[6], ins[7]};
  const Extent elems[] = {outs[0], outs[1], outs[2], ins[0], ins[1], ins[2], ins[3]};
  if (any_misaligned(words, 4) || any_misaligned(elems, e) || misaligned(ws, 256)) return LAPLEX_ERR_ALIGN;
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;

  const uint32_t group = a.heads / a.kv_heads;
  const AttnView vq = {q, a.q_token, a.q_head, 1}, vk = {k, a.k_token, a.k_head, group}, vv = {v, a.v_token, a.v_head, group},
                 vg = {go, (int64_t)a.heads * a.dv, (int64_t)a.dv, 1};
  if (a.seqs == 0) return drate ? from_hip(attn_drate_reduce(w.drate, 0, a.heads, drate, stream)) : LAPLEX_OK;
  hipError_t err;
  if (a.tokens || drate) {  // dq, and the rate's gradient
    AttnPass p = base_pass(a);
    p.K = a.dv;
    p.V = a.dk;
    p.x = vg;
    p.y = vv;
    p.z = vk;
    p.c_pair = p.c_in = a.scale;
    p.c_add = 1.f;
    p.out = a.tokens ? dq : nullptr;
    p.s_in = state_in;
    p.s_trans = true;
    if (drate) {
      p.dot = q;
      p.dot_view = vq;
      p.ds_out = dstate_out;
      p.drate_part = w.drate;
    }
    if ((err = attn_pass(p, w.pass, stream)) != hipSuccess) return from_hip(err);
    if (drate) {
      const uint64_t parts = attn_drate_parts(a.dtype, a.seqs, a.heads, a.dv, a.dk, a.tokens, a.offsets);
      if ((err = attn_drate_reduce(w.drate, parts, a.heads, drate, stream)) != hipSuccess) return from_hip(err);
    }
  }
  // dv with the initial state's gradient, then dk
  for (int i = 0; i < 2; ++i) {
    if (a.tokens == 0 && !(i == 0 && dstate_in)) continue;
    AttnPass p = base_pass(a);
    p.reverse = true;
    p.x = i == 0 ? vk : vv;
    p.y = i == 0 ? vq : vg;
    p.z = i == 0 ? vg : vq;
    p.K = i == 0 ? a.dk : a.dv;
    p.V = i == 0 ? a.dv : a.dk;
    p.s_trans = p.bound_ready = i == 1;
    p.c_pair = p.c_add = a.scale;
    p.c_in = 1.f;
    p.s_in = dstate_out;
    p.s_out = i == 0 ? dstate_in : nullptr;
    void* grad = i == 0 ? dv : dk;
    p.out = a.tokens == 0 ? nullptr : group > 1 ? w.sum : grad;
    p.out_f32 = group > 1;
    if ((err = attn_pass(p, w.pass, stream)) != hipSuccess) return from_hip(err);
    if (group > 1 && a.tokens)
      if ((err = attn_group_sum(a.dtype, w.sum, a.tokens, a.kv_heads, group, p.V, grad, stream)) != hipSuccess) return from_hip(err);
  }
  return LAPLEX_OK;
}

extern "C" laplex_status laplex_decay_attn_step(const laplex_attn_shape* shape, const void* q, const void* k, const void* v,
                                                const int32_t* slots, uint32_t pool, float* state, void* o,
                                                hipStream_t stream) {
  laplex_status st = check_shape(shape);
  if (st != LAPLEX_OK) return st;
  const laplex_attn_shape& a = *shape;
  if (a.tokens != a.seqs || (!slots && a.seqs > pool)) return LAPLEX_ERR_ARG;
  if (a.seqs == 0) return LAPLEX_OK;
  if (!a.rate || !q || !k || !v || !o || (!state && pool)) return LAPLEX_ERR_NULL;
  const size_t e = elem(a.dtype);
  size_t qb, kb, vb;
  if (!view_bytes(a.tokens, a.heads, a.dk, a.q_token, a.q_head, e, &qb) ||
      !view_bytes(a.tokens, a.kv_heads, a.dk, a.k_token, a.k_head, e, &kb) ||
      !view_bytes(a.tokens, a.kv_heads, a.dv, a.v_token, a.v_head, e, &vb))
    return LAPLEX_ERR_ARG;
  const Extent outs[] = {{o, a.tokens * a.heads * a.dv * e}, {state, (size_t)pool * a.heads * a.dk * a.dv * 4}};
  const Extent ins[] = {{q, qb}, {k, kb}, {v, vb}, {slots, a.seqs * 4ull}, {a.rate, a.heads * 4ull}};
  if (misaligned(o, e) || misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(state, 4) ||
      misaligned(slots, 4) || misaligned(a.rate, 4))
    return LAPLEX_ERR_ALIGN;
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  const uint32_t group = a.heads / a.kv_heads;
  AttnStep p{a.dtype, a.seqs, a.heads, a.dk, a.dv, pool, a.rate, {q, a.q_token, a.q_head, 1}, {k, a.k_token, a.k_head, group},
             {v, a.v_token, a.v_head, group}, a.scale, slots, state, o};
  return from_hip(attn_step(p, stream));
}

// ------------------------------------------------------------------ layer norm
extern "C" laplex_status laplex_layer_norm(int dtype, uint64_t rows, uint32_t width, const void* x, const void* weight,
                                           const void* bias, float eps, void* y, float* mean, float* rstd, hipStream_t stream) {
  if (!is_dtype(dtype) || width == 0) return LAPLEX_ERR_ARG;
  if (rows > kMaxRows || width > kMaxWidth) return LAPLEX_ERR_SIZE;
  if (rows == 0) return LAPLEX_OK;
  if (!x || !y) return LAPLEX_ERR_NULL;
  const size_t e = elem(dtype), xb = rows * width * e;
  const Extent outs[] = {{y, xb}, {mean, rows * 4}, {rstd, rows * 4}}, ins[] = {{x, xb}, {weight, width * e}, {bias, width * e}};
  if (misaligned(y, e) || any_misaligned(ins, e) || misaligned(mean, 4) || misaligned(rstd, 4)) return LAPLEX_ERR_ALIGN;
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(layer_norm(dtype, rows, width, x, weight, bias, eps, y, mean, rstd, stream));
}

extern "C" size_t laplex_layer_norm_workspace_bytes(uint64_t rows, uint32_t width) {
  if (width == 0 || rows > kMaxRows || width > kMaxWidth) return 0;
  return layer_norm_backward_bytes(rows, width);
}

extern "C" laplex_status laplex_layer_norm_backward(int dtype, uint64_t rows, uint32_t width, const void* x, const void* dy,
                                                    const float* mean, const float* rstd, const void* weight, void* dx,
                                                    float* dweight, float* dbias, void* ws, size_t ws_bytes,
                                                    hipStream_t stream) {
  if (!is_dtype(dtype) || width == 0) return LAPLEX_ERR_ARG;
  if (rows > kMaxRows || width > kMaxWidth) return LAPLEX_ERR_SIZE;
  if (rows && (!x || !dy || !mean || !rstd || !dx)) return LAPLEX_ERR_NULL;
  const bool sums = dweight || dbias;
  if (sums && rows && !ws) return LAPLEX_ERR_NULL;
  const size_t e = elem(dtype), xb = rows * width * e, need = sums && rows ? layer_norm_backward_bytes(rows, width) : 0;
  const Extent outs[] = {{dx, xb}, {dweight, width * 4ull}, {dbias, width * 4ull}, {ws, need}};
  const Extent ins[] = {{x, xb}, {dy, xb}, {mean, rows * 4}, {rstd, rows * 4}, {weight, width * e}};
  if (misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(weight, e) || misaligned(mean, 4) ||
      misaligned(rstd, 4) || misaligned(dweight, 4) || misaligned(dbias, 4) || (need && misaligned(ws, 256)))
    return LAPLEX_ERR_ALIGN;
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(layer_norm_backward(dtype, rows, width, x, dy, mean, rstd, weight, dx, dweight, dbias, ws, stream));
}

// ------------------------------------------------------------------ embedding
namespace {
EmbedWorkspace carve_embed(void* ws, uint64_t tokens, uint32_t vocab, uint32_t width, size_t* total) {
  Carver c(ws);
  EmbedWorkspace w{};
  char* sort_base = c.take<char>(sort_bytes(tokens));
  if (ws) w.sort = carve_sort(sort_base, tokens);
  w.keys = c.take<uint32_t>(tokens * 4);
  w.keys_s = c.take<uint32_t>(tokens * 4);
  w.perm = c.take<uint32_t>(tokens * 4);
  w.starts = c.take<uint32_t>(embed_starts(vocab) * 4);
  w.part = c.take<float>(embed_part_floats(tokens, width) * 4);
  const uint64_t tiled = embed_tiled_most(tokens, vocab);
  w.tile_perm = c.take<uint32_t>(tiled * 4);
  w.tile_starts = c.take<uint32_t>(embed_tiles_of(tiled) * embed_starts(vocab) * 4);
  *total = (c.off + 255) & ~size_t(255);
  return w;
}
}  // namespace

extern "C" laplex_status laplex_embedding(int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* table,
                                          uint32_t vocab, uint32_t width, float scale, void* y, hipStream_t stream) {
  if (!is_dtype(dtype) || (id_bytes != 4 && id_bytes != 8) || width == 0) return LAPLEX_ERR_ARG;
  if (tokens > kMaxEmbedTokens || vocab > kMaxVocab || width > kMaxWidth) return LAPLEX_ERR_SIZE;
  if (tokens == 0) return LAPLEX_OK;
  if (!ids || !y || (vocab && !table)) return LAPLEX_ERR_NULL;
  const size_t e = elem(dtype);
  if (misaligned(ids, id_bytes) || misaligned(table, e) || misaligned(y, e)) return LAPLEX_ERR_ALIGN;
  const Extent outs[] = {{y, tokens * width * e}}, ins[] = {{ids, tokens * id_bytes}, {table, (size_t)vocab * width * e}};
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(embedding(dtype, ids, id_bytes, tokens, table, vocab, width, scale, y, stream));
}

extern "C" size_t laplex_embedding_workspace_bytes(uint64_t tokens, uint32_t vocab, uint32_t width) {
  if (tokens > kMaxEmbedTokens || vocab > kMaxVocab || width > kMaxWidth || width == 0) return 0;
  size_t total = 0;
  carve_embed(nullptr, tokens, vocab, width, &total);
  return total;
}

extern "C" laplex_status laplex_embedding_backward(int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* dy,
                                                   uint32_t vocab, uint32_t width, float scale, int table_dtype, void* dtable,
                                                   void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!is_dtype(dtype) || (table_dtype != dtype && table_dtype != LAPLEX_F32) || (id_bytes != 4 && id_bytes != 8) || width == 0)
    return LAPLEX_ERR_ARG;
  if (tokens > kMaxEmbedTokens || vocab > kMaxVocab || width > kMaxWidth) return LAPLEX_ERR_SIZE;
  if (vocab == 0) return LAPLEX_OK;
  if (!dtable || !ws || (tokens && (!ids || !dy))) return LAPLEX_ERR_NULL;
  const size_t e = elem(dtype), te = elem(table_dtype);
  if ((tokens && misaligned(ids, id_bytes)) || misaligned(dy, e) || misaligned(dtable, te) || misaligned(ws, 256))
    return LAPLEX_ERR_ALIGN;
  size_t need = 0;
  const EmbedWorkspace w = carve_embed(ws, tokens, vocab, width, &need);
  if (ws_bytes < need) return LAPLEX_ERR_WORKSPACE;
  const Extent outs[] = {{dtable, (size_t)vocab * width * te}, {ws, need}}, ins[] = {{ids, tokens * id_bytes}, {dy, tokens * width * e}};
  if (any_overlap(outs, ins)) return LAPLEX_ERR_OVERLAP;
  return from_hip(embedding_backward(w, dtype, ids, id_bytes, tokens, dy, vocab, width, scale, table_dtype, dtable, stream));
}
