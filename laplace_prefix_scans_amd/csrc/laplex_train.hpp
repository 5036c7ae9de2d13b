// Host-visible launch interface of the training-step kernels (internal to the
// library): gated linear recurrence, linear softmax cross entropy, AdamW.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/laplex.h"
#include "laplex_kernels.hpp"

namespace laplex {

// ------------------------------------------------------------------ gated linear recurrence
// Tokens of a tile, and between two carries that the forward pass keeps for the backward.
constexpr uint32_t kGateChunk = LAPLEX_SCAN_CHUNK;
struct GateShape {
  int dtype, kind;
  uint32_t seqs, channels;
  uint64_t tokens;
  const int32_t* offsets;  // or null: equal lengths
  const void *gate, *x;
  int64_t gate_token, x_token;
};
size_t gated_scan_bytes(uint32_t channels, uint64_t tokens);
hipError_t gated_scan(const GateShape& g, const float* state_in, float* state_out, void* h, float* carries, void* ws, hipStream_t s);
hipError_t gated_scan_backward(const GateShape& g, const float* carries, const void* dh, const float* state_in,
                               const float* dstate_out, void* dgate, void* dx, float* dstate_in, void* ws, hipStream_t s);
hipError_t gated_scan_step(const GateShape& g, const int32_t* slots, uint32_t pool, float* state, void* h, hipStream_t s);

// ------------------------------------------------------------------ linear softmax cross entropy
struct XentShape {
  int dtype, id_bytes;
  uint64_t tokens;
  uint32_t vocab, width;
  const void *targets, *x, *table;
  float scale;
};
// aligned: of calls whose x and table begin at multiples of 16 bytes, as xent_aligned tells
size_t xent_bytes(int pass, int dtype, uint64_t tokens, uint32_t vocab, uint32_t width, bool aligned);
bool xent_aligned(const void* x, const void* table);
hipError_t xent(const XentShape& a, float* loss, float* lse, void* ws, hipStream_t s);
hipError_t xent_backward(const XentShape& a, const float* lse, const float* dloss, const float* dlse, void* dx, int table_dtype,
                         void* dtable, void* ws, hipStream_t s);

// ------------------------------------------------------------------ AdamW
hipError_t adamw(const laplex_adamw_args& a, const laplex_adamw_tensor* t, uint32_t count, hipStream_t s);
// floats of the 8-bit moments: of m to p, of v to master (either may be null)
hipError_t adamw_moments(const laplex_adamw_tensor* t, uint32_t count, hipStream_t s);

}  // namespace laplex
