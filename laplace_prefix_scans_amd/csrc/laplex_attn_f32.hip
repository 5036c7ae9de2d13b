// The chunked attention pass for float32 tensors.
#include "laplex_attn_chunk.hpp"

namespace laplex {
LAPLEX_ATTN_CHUNK_SIZES(float)
}  // namespace laplex
