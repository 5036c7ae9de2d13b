// The chunked attention pass for float32 tensors, rows aligned to 16 bytes.
#include "laplex_attn_chunk.hpp"

namespace laplex {
void attn_chunk_f32_vec(const AttnChunkArgs& a, int kp, int nw, bool full, bool rate, hipStream_t s) {
  attn_chunk_launch<float, true>(a, kp, nw, full, rate, s);
}
}  // namespace laplex
