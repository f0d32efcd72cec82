// The paged 4-bit cache of keys and values (its layout: include/qmm.h).
#pragma once

#include "attn.hpp"

namespace qmm {

constexpr int kCellTokens = 16;

inline bool kv_q4_shape(int64_t pages, int64_t page, int64_t Hk, int64_t D) {
  return Hk >= 1 && Hk <= 1024 && attn_head_dim(D) && page >= 16 && page <= (int64_t{1} << 20) && page % 16 == 0 &&
         pages >= 1 && pages <= 0x7fffffff;
}

// First byte of the cell that holds a slot's token for head h.  `shift`: the page size is 2^shift, or -1.
__device__ __forceinline__ int64_t kv_cell(int64_t slot, int64_t page, int shift, int h, int Hk, int D) {
  const int64_t p = shift >= 0 ? slot >> shift
                    : slot < (int64_t{1} << 32) ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(page) : slot / page;
  const int cells = static_cast<int>(page) / kCellTokens, cell = static_cast<int>(slot - p * page) / kCellTokens;
  return ((p * Hk + h) * cells + cell) * (20 * D);
}
inline int page_shift(int64_t page) {
  int s = 0;
  while ((int64_t{1} << s) < page) ++s;
  return (int64_t{1} << s) == page ? s : -1;
}

// Memory that nothing writes while the kernel runs, read at addresses that are
// the same for the whole wave: through the scalar cache.
typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
__device__ __forceinline__ scalar_ints as_scalar(const int32_t* p) {
  return reinterpret_cast<scalar_ints>(reinterpret_cast<uintptr_t>(p));
}

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ h2 as_h2(uint32_t v) { return __builtin_bit_cast(h2, v); }

// Bytes 0 and 1 (or 2 and 3) of v, each 0..15, as f16 numbers.  A byte n read as
// an 8-bit float with three bits of fraction is n * 2^-9, below 8 a subnormal
// one; the conversion of two multiplies by 2^9.
template <bool UPPER>
__device__ __forceinline__ h2 codes_to_f16(uint32_t v) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.0f, UPPER);
}

// Where byte i of a quad's four value codes stands: tokens 0, 2, 1, 3.
__device__ __forceinline__ int kv_quad_byte(int t) { return (t & 1) * 2 + (t >> 1); }

}  // namespace qmm
