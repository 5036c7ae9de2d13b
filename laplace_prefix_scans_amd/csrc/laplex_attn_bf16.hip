// The chunked attention pass for bfloat16 tensors.
#include "laplex_attn_chunk.hpp"

namespace laplex {
LAPLEX_ATTN_CHUNK_SIZES(bf16)
}  // namespace laplex
