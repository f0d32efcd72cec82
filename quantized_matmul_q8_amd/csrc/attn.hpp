// Shared by the attention kernels: the running maximum and sum of a softmax
// over lanes, and the joining of partial results.
#pragma once

#include "typed.hpp"

#include <float.h>

namespace qmm {

typedef float v4f __attribute__((ext_vector_type(4)));

// No sequence is longer.  A window that is wider sees the same and is cut to
// this, so that the places of keys, less a window, stay in 32 bits.
constexpr int64_t kMostTokens = int64_t{1} << 30;

inline bool attn_head_dim(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

// Over lanes l and l ^ 32, in both: one exchange of the wave's halves.
template <typename F>
__device__ __forceinline__ float halves_join(float v, F f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return f(__builtin_bit_cast(float, static_cast<uint32_t>(b[0])), __builtin_bit_cast(float, static_cast<uint32_t>(b[1])));
}
// Over the four rows of 16 lanes, in all of them.
template <typename F>
__device__ __forceinline__ float rows_join(float v, F f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return halves_join(f(__builtin_bit_cast(float, static_cast<uint32_t>(a[0])),
                       __builtin_bit_cast(float, static_cast<uint32_t>(a[1]))), f);
}
__device__ __forceinline__ float rows_max(float v) {
  return rows_join(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float rows_sum(float v) {
  return rows_join(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float halves_max(float v) {
  return halves_join(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float halves_sum(float v) {
  return halves_join(v, [](float a, float b) { return a + b; });
}

// The sum over this lane and those before it, by moves within rows of 16 lanes and of their last lanes to the rows behind.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31 into rows 2 and 3
  return v;
}

// What the difference of two products q k is multiplied with for the exponent
// between their terms; 1 where that is 0 (the queries count as zeros then), and the
// largest number where it is past fp32 (infinity times no difference would be NaN).
// Differences are taken first, everywhere: of products past 2^24 or so, multiplied
// each by itself, only the rounding would be left.
constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ bool vanishes(float scale) { return fabsf(scale) * kLog2e == 0.0f; }
__device__ __forceinline__ float exponent_mul(float scale) {
  return vanishes(scale) ? 1.0f : fminf(fabsf(scale) * kLog2e, FLT_MAX);
}

// One row of four dims per lane from `count` partial results: at `part` + step *
// at(k) number k's sums of terms times values, in ml[at(k)] its largest product and
// its sum of terms.  The products and sums by the lanes, 64 at a time, then the
// partial results in order, four loads in flight.  The first loads begin with the
// object, so that what is done before join() hides them.
template <typename At>
struct Parts {
  const At at;
  const float* part;
  const float2* ml;
  int64_t step;
  int count, lane;
  float2 own;
  v4f x[4];

  __device__ __forceinline__ Parts(const At& at, const float* part, int64_t step, const float2* ml, int count, int lane)
      : at(at), part(part), ml(ml), step(step), count(count), lane(lane) {
    load_sums(0);
    load_rows(0);
  }
  __device__ __forceinline__ void load_sums(int k0) { own = ml[at(min(k0 + lane, count - 1))]; }
  __device__ __forceinline__ void load_rows(int k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const v4f*>(part + at(min(k + i, count - 1)) * step);
  }

  // The row; zeros if all sums are 0.
  __device__ __forceinline__ v4f join(float mul) {
    float m = -INFINITY, total = 0.0f;
    v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < count; k0 += 64) {
      const int here = min(64, count - k0);
      if (lane >= here) own = make_float2(-INFINITY, 0.0f);
      float most = fmaxf(m, rows_max(own.x));
#pragma unroll
      for (int k = 1; k < 16; k *= 2) most = fmaxf(most, __shfl_xor(most, k));
      const float base = most == -INFINITY ? 0.0f : most, keep = __builtin_amdgcn_exp2f((m - base) * mul);
      const float f = __builtin_amdgcn_exp2f((own.x - base) * mul);
      total = total * keep + wave_sum(own.y * f);
      y *= keep;
      m = most;
      if (k0 + 64 < count) load_sums(k0 + 64);
      for (int k = 0; k < here; k += 4) {
        v4f now[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) now[i] = x[i];
        if (k0 + k + 4 < count) load_rows(k0 + k + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k + i < here) y += now[i] * __shfl(f, k + i);
      }
    }
    return y * (total == 0.0f ? 0.0f : 1.0f / total);
  }
};

}  // namespace qmm
