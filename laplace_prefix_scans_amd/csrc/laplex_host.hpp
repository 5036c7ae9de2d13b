// Host-side helpers of the C-ABI entry points: workspace layout and argument checks.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/laplex.h"
#include "laplex_kernels.hpp"

namespace laplex {

// Carves 256-byte aligned regions out of a workspace (base 0: sizing only).
struct Carver {
  uintptr_t base;
  size_t off = 0;
  explicit Carver(void* b) : base(reinterpret_cast<uintptr_t>(b)) {}
  template <typename T>
  T* take(size_t bytes) {
    off = (off + 255) & ~size_t(255);
    T* p = reinterpret_cast<T*>(base + off);
    off += bytes;
    return p;
  }
};

inline SortWorkspace carve_sort(void* ws, uint64_t n) {
  Carver c(ws);
  SortWorkspace w;
  w.header = c.take<uint32_t>(kSortHeaderBytes);
  w.hist = w.header + kSortHistOffset / 4;
  w.offsets = w.header + kSortOffsOffset / 4;
  w.status = c.take<void>(sort_status_bytes(n));  // directly after the header
  for (int i = 0; i < 2; ++i) w.kv[i] = c.take<uint2>(n * 8);
  w.tcount = c.take<uint32_t>(sort_tiles_alloc(n) * 256 * 4);
  w.gsum = c.take<uint32_t>((size_t)kHistMaxBlocks * 256 * 4);
  return w;
}
inline size_t sort_bytes(uint64_t n) {
  Carver c(nullptr);
  c.take<uint32_t>(kSortHeaderBytes);
  c.take<void>(sort_status_bytes(n));
  for (int i = 0; i < 2; ++i) c.take<uint2>(n * 8);
  c.take<uint32_t>(sort_tiles_alloc(n) * 256 * 4);
  c.take<uint32_t>((size_t)kHistMaxBlocks * 256 * 4);
  return (c.off + 255) & ~size_t(255);
}

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

inline bool overlaps(const void* p, size_t pb, const void* q, size_t qb) {
  if (!p || !q || pb == 0 || qb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(p), a1 = a0 + pb;
  const uintptr_t b0 = reinterpret_cast<uintptr_t>(q), b1 = b0 + qb;
  return a0 < b1 && b0 < a1;
}

inline laplex_status from_hip(hipError_t e) { return e == hipSuccess ? LAPLEX_OK : LAPLEX_ERR_HIP; }

}  // namespace laplex
