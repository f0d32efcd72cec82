// The paged 4-bit cache of keys and values (its layout: include/qmm.h).
#pragma once

#include "attn.hpp"

namespace qmm {

constexpr int kCellTokens = 16;

inline bool kv_q4_shape(int64_t pages, int64_t page, int64_t Hk, int64_t D) {
  return Hk >= 1 && Hk <= 1024 && attn_head_dim(D) && page >= 16 && page <= (int64_t{1} << 20) && page % 16 == 0 &&
         pages >= 1 && pages <= 0x7fffffff;
}

// First byte of the cell that holds a slot's token for head h.
__device__ __forceinline__ int64_t kv_cell(int64_t slot, int64_t page, int h, int Hk, int D) {
  const int64_t p = slot / page;
  return ((p * Hk + h) * (page / kCellTokens) + (slot - p * page) / kCellTokens) * (20 * D);
}

// Memory that nothing writes while the kernel runs, read at addresses that are
// the same for the whole wave: through the scalar cache.
typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
__device__ __forceinline__ scalar_ints as_scalar(const int32_t* p) {
  return reinterpret_cast<scalar_ints>(reinterpret_cast<uintptr_t>(p));
}

// Where byte i of a quad's four value codes stands: tokens 0, 2, 1, 3.
__device__ __forceinline__ int kv_quad_byte(int t) { return (t & 1) * 2 + (t >> 1); }

}  // namespace qmm
