// Values of 32 and 16 bits behind one type code (QMM_F32, QMM_F16, QMM_BF16):
// widening loads, and stores rounded once to the nearest (ties to even).
#pragma once

#include "qmm_common.hpp"

namespace qmm {

// Rows of heads: a stride of at least all of them, 16-byte steps for any type, and 64 rows' bytes within 32 bits.
inline bool strided_rows(int64_t stride, int64_t heads, int64_t D) {
  return stride >= heads * D && stride % 8 == 0 && stride < (int64_t{1} << 24);
}

// Lists of whole numbers are read one at a time, so any part of one may be passed.
inline bool aligned_list(const void* p, uintptr_t size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

// Tokens of a call, 32 lanes or a wave each: a grid has to stay below 2^32 of them.
constexpr int64_t kMostRows = int64_t{1} << 26;

inline bool known_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }

typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));

// Outputs larger than half of the last-level cache (256 MB) are stored past the
// caches: nothing finds all of them there.  65536 x 8 x 128 cached tokens read
// back to bf16, 268 MB: 60 us, with stores through the caches 91; a smaller one
// the next kernel finds.
inline bool large_output(int64_t values, int type) { return values * (type == QMM_F32 ? 4 : 2) >= (int64_t{128} << 20); }

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

__device__ __forceinline__ void load8(int type, const void* p, int64_t i, float (&v)[8]) {
  const float4 lo = load4(type, p, 2 * i), hi = load4(type, p, 2 * i + 1);
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}

// Eight values 8i .. 8i + 7 as they are stored.
template <int TY>
struct Raw8 {
  static constexpr int kWords = TY == QMM_F32 ? 2 : 1;
  uint4 v[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = static_cast<const uint4*>(p)[i * kWords + k];
  }
  // Data that is read once.  Only 16-bit values: the two loads of eight fp32 ones touch the same lines, and the second
  // would miss (16384 x 4096, bf16: 93 -> 87 us; 4096 x 11008, fp32: 57 -> 64).
  __device__ __forceinline__ void load_once(const void* p, int64_t i) {
    if constexpr (kWords == 1) v[0] = ld16_nt(static_cast<const uint4*>(p) + i);
    else load(p, i);
  }
  __device__ __forceinline__ void store_nt(void* p, int64_t i) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      v4u t;
      t.x = v[k].x;
      t.y = v[k].y;
      t.z = v[k].z;
      t.w = v[k].w;
      __builtin_nontemporal_store(t, static_cast<v4u*>(p) + i * kWords + k);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) static_cast<uint4*>(p)[i * kWords + k] = v[k];
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (TY == QMM_F32) {
      const uint4& q = v[j >> 2];
      return __builtin_bit_cast(float, (j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w);
    } else {
      const uint32_t d = (j >> 1) == 0 ? v[0].x : (j >> 1) == 1 ? v[0].y : (j >> 1) == 2 ? v[0].z : v[0].w;
      if constexpr (TY == QMM_F16) return h2f(j & 1 ? d >> 16 : d & 0xffffu);
      return __builtin_bit_cast(float, j & 1 ? d & 0xffff0000u : d << 16);
    }
  }
  // values f rounded to the type, to the nearest (ties to even)
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t d[4 * kWords];
#pragma unroll
    for (int j = 0; j < 4 * kWords; ++j) {
      if constexpr (TY == QMM_F32) d[j] = __builtin_bit_cast(uint32_t, f[j]);
      else if constexpr (TY == QMM_F16) d[j] = f2h_bits(f[2 * j]) | f2h_bits(f[2 * j + 1]) << 16;
      else
        d[j] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f[2 * j]))) |
               static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f[2 * j + 1]))) << 16;
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = make_uint4(d[4 * k], d[4 * k + 1], d[4 * k + 2], d[4 * k + 3]);
  }
};

}  // namespace qmm
