// Values of 32 and 16 bits behind one type code (QMM_F32, QMM_F16, QMM_BF16):
// widening loads, and stores rounded once to the nearest (ties to even).
#pragma once

#include "qmm_common.hpp"

namespace qmm {

inline bool known_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }

typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));

// Storage of a type code and of four of its values.
template <int TY> struct Typed;
template <> struct Typed<QMM_F32> { using one = float; using four = float4; };
template <> struct Typed<QMM_F16> { using one = _Float16; using four = v4h; };
template <> struct Typed<QMM_BF16> { using one = __bf16; using four = v4b; };

// Values 4i .. 4i + 3, widened (exact).
template <int TY>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
  const auto v = static_cast<const typename Typed<TY>::four*>(p)[i];
  return make_float4(static_cast<float>(v.x), static_cast<float>(v.y), static_cast<float>(v.z),
                     static_cast<float>(v.w));
}

// Values 4i .. 4i + 3, each rounded to the nearest (ties to even).
template <int TY>
__device__ __forceinline__ void store4(void* p, int64_t i, float4 v) {
  using one = typename Typed<TY>::one;
  typename Typed<TY>::four r;
  r.x = static_cast<one>(v.x);
  r.y = static_cast<one>(v.y);
  r.z = static_cast<one>(v.z);
  r.w = static_cast<one>(v.w);
  static_cast<typename Typed<TY>::four*>(p)[i] = r;
}

// The same with the type known only when the kernel runs (uniform over it).
__device__ __forceinline__ float4 load4(int type, const void* p, int64_t i) {
  if (type == QMM_F32) return load4<QMM_F32>(p, i);
  if (type == QMM_F16) return load4<QMM_F16>(p, i);
  return load4<QMM_BF16>(p, i);
}
__device__ __forceinline__ void store4(int type, void* p, int64_t i, float4 v) {
  if (type == QMM_F32) store4<QMM_F32>(p, i, v);
  else if (type == QMM_F16) store4<QMM_F16>(p, i, v);
  else store4<QMM_BF16>(p, i, v);
}

}  // namespace qmm
