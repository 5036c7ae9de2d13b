// Host-visible launch interface of the sequence-layer kernels (internal to
// the library): decayed linear attention, layer norm, embedding.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/laplex.h"
#include "laplex_kernels.hpp"

namespace laplex {

// ------------------------------------------------------------------ decayed attention
// One pass of the attention recurrence over all sequences.  Rows x (K
// channels) read the carry, rows y (K) and z (V) are added to it, out (V) is
// written.  With u = 0 .. L-1 the tokens of a sequence in processing order and
// w(n) = exp(-rate n):
//   out_u = c_pair sum_{u' <= u} w(u - u') (x_u . y_u') z_u'  +  c_in w(u + lead) x_u S_in
//   S_out = w(L) S_in + c_add sum_u w(L - 1 - u + 1 - lead) y_u z_u^T
// Forward: (x, y, z) = (q, k, v), lead 1.  dq: (go, v, k) on S_in^T, lead 1.
// dk and dv: reversed tokens, (v, go, q) and (k, q, go), lead 0 (the gradient
// of the final state reaches the last token undecayed).
struct AttnView {
  const void* p;
  int64_t token, head;  // strides in elements
  uint32_t div;         // row of head h: head h / div of the tensor
};
struct AttnPass {
  int dtype;
  uint32_t seqs, heads, K, V;
  uint64_t tokens;
  const int32_t* offsets;
  const float* rate;
  AttnView x, y, z;
  float c_pair, c_in, c_add;
  bool reverse;        // processing order runs from the last token to the first
  void* out;           // tokens x heads x V, contiguous, or null (state only)
  bool out_f32;        // out holds floats whatever the dtype
  const float* s_in;   // seqs x heads x K x V, or null
  float* s_out;        // the same, or null
  bool s_trans;        // s_in, s_out are V x K per head
  bool bound_ready;    // the workspace holds the segments' states of the pass before, which had K and V (and y and z) exchanged
  // rate gradient (dq pass only): -c_pair sum_u <dot_u, sum_u' (u - u') w x.y z> and the final state's part
  const void* dot;     // rows (V) the lag-weighted outputs are multiplied with, strides as dot_view
  AttnView dot_view;
  const float* ds_out; // gradient of the final state, laid out as s_in, or null
  double* drate_part;  // partials of the rate gradient ([attn_drate_parts][head])
};
hipError_t attn_pass(const AttnPass& p, void* ws, hipStream_t s);
// bytes of workspace of a pass, and partials of the rate's gradient, that serve this many tokens and any fewer
size_t attn_pass_bytes(int dtype, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens, bool rate);
uint64_t attn_drate_parts_most(int dtype, uint32_t seqs, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens);
// number of partials per head an attn_pass with drate_part writes ([partial][head])
uint64_t attn_drate_parts(int dtype, uint32_t seqs, uint32_t heads, uint32_t K, uint32_t V, uint64_t tokens, const int32_t* offsets);
hipError_t attn_drate_reduce(const double* part, uint64_t parts, uint32_t heads, float* drate, hipStream_t s);
// dst[t][g][c] = sum of src[t][g * group + i][c] over i < group (src in float)
hipError_t attn_group_sum(int dtype, const float* src, uint64_t tokens, uint32_t kv_heads, uint32_t group, uint32_t width,
                          void* dst, hipStream_t s);
struct AttnStep {
  int dtype;
  uint32_t rows, heads, K, V, pool;
  const float* rate;
  AttnView q, k, v;
  float scale;
  const int32_t* slots;
  float* state;
  void* out;
};
hipError_t attn_step(const AttnStep& p, hipStream_t s);

// ------------------------------------------------------------------ layer norm
hipError_t layer_norm(int dtype, uint64_t rows, uint32_t width, const void* x, const void* w, const void* b, float eps, void* y,
                      float* mean, float* rstd, hipStream_t s);
size_t layer_norm_backward_bytes(uint64_t rows, uint32_t width);
hipError_t layer_norm_backward(int dtype, uint64_t rows, uint32_t width, const void* x, const void* dy, const float* mean,
                               const float* rstd, const void* w, void* dx, float* dw, float* db, void* ws, hipStream_t s);

// ------------------------------------------------------------------ embedding
hipError_t embedding(int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* table, uint32_t vocab, uint32_t width,
                     float scale, void* y, hipStream_t s);
// the sorted tokens of an embedding backward
struct EmbedWorkspace {
  SortWorkspace sort;
  uint32_t* keys;    // the ids' sort keys (tokens)
  uint32_t* keys_s;  // the same, sorted
  uint32_t* perm;    // tokens in that order
  uint32_t* starts;  // first sorted position of each key (embed_starts)
  float* part;       // partial rows (embed_part_floats)
  // where the tokens are sorted in tiles first (embed_tiles): each tile's tokens and starts (its keys are in `keys`)
  uint32_t *tile_perm, *tile_starts;
};
uint64_t embed_starts(uint32_t vocab);
// sizes that serve this many tokens and any fewer: tokens that are sorted in tiles, floats of partial rows
uint64_t embed_tiled_most(uint64_t tokens, uint32_t vocab);
uint64_t embed_part_floats(uint64_t tokens, uint32_t width);
uint32_t embed_tiles(uint64_t tokens, uint32_t vocab);
uint32_t embed_tiles_of(uint64_t tiled);
hipError_t embedding_backward(const EmbedWorkspace& w, int dtype, const void* ids, int id_bytes, uint64_t tokens, const void* dy,
                              uint32_t vocab, uint32_t width, float scale, int table_dtype, void* dtable, hipStream_t s);

}  // namespace laplex
