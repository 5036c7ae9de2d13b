// The chunked attention pass for bfloat16 tensors, rows aligned to 16 bytes.
#include "laplex_attn_chunk.hpp"

namespace laplex {
void attn_chunk_bf16_vec(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s) {
  attn_chunk_launch<bf16, true>(a, kp, nw, full, rate, s);
}
}  // namespace laplex
