// The chunked attention pass for float32 tensors, any alignment.
#include "laplex_attn_chunk.hpp"

namespace laplex {
void attn_chunk_f32_any(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s) {
  attn_chunk_launch<float, false>(a, kp, nw, full, rate, s);
}
}  // namespace laplex
