// Matvec of 4-bit weights with group scales and Q8_1 activations.
//
//   y[t][m] = sum_b s[m][g(b)] * d[t][b] * (sum_i q_i a_i - z[m][g(b)] * S[t][b])
//
// over the 32-value blocks b of the row, with the block's integer sum S as
// stored in Q8_1: integer dot products, one fp32 rounding of the scales'
// product and one fma per block.
#include "typed.hpp"

namespace qmm {

struct Q4gArgs {
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;
  const uint8_t* xq;
  float* y;
  int64_t M;
  int nblk, group_blk, groups, T, scale_type;
};

constexpr uint32_t kEvenBytes = 0x06040200u, kOddBytes = 0x07050301u;

__global__ __launch_bounds__(256) void mmvq_q4g_kernel(Q4gArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (m >= a.M) return;
  float acc[QMM_MMVQ_MAX_T] = {};
  for (int b = lane; b < a.nblk; b += 64) {
    const int g = b / a.group_blk;
    const uint4 w = ld16_a16(a.w + (m * a.nblk + b) * 16);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    const float s = a.scale_type == QMM_F16 ? static_cast<float>(static_cast<const _Float16*>(a.scales)[m * a.groups + g])
                                            : static_cast<float>(static_cast<const __bf16*>(a.scales)[m * a.groups + g]);
    const int z = a.zeros ? (a.zeros[m * ((a.groups + 1) / 2) + (g >> 1)] >> (4 * (g & 1))) & 15 : 8;
#pragma unroll
    for (int t = 0; t < QMM_MMVQ_MAX_T; ++t) {
      if (t < a.T) {
        const uint8_t* x = a.xq + (static_cast<int64_t>(t) * a.nblk + b) * kQ8Bytes;
        const uint32_t* q = reinterpret_cast<const uint32_t*>(x + 4);
        int dot = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dot = dot4(ww[j] & 0x0f0f0f0fu, __builtin_amdgcn_perm(q[2 * j + 1], q[2 * j], kEvenBytes), dot);
          dot = dot4((ww[j] >> 4) & 0x0f0f0f0fu, __builtin_amdgcn_perm(q[2 * j + 1], q[2 * j], kOddBytes), dot);
        }
        const int S = reinterpret_cast<const int32_t*>(x + 36)[0];
        acc[t] = __builtin_fmaf(s * h2f(ld_u16(x)), static_cast<float>(dot - z * S), acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < QMM_MMVQ_MAX_T; ++t) {
    if (t < a.T) {
      const float v = wave_sum(acc[t]);
      if (lane == 0) a.y[t * a.M + m] = v;
    }
  }
}

}  // namespace qmm

using namespace qmm;

extern "C" int mmvq_q4g(const void* w, const void* scales, int scale_type, const void* zeros, const void* xq, float* y,
                        int64_t M, int64_t K, int64_t group, int64_t T, void* stream) {
  if (scale_type != QMM_F16 && scale_type != QMM_BF16) return QMM_ERR_UNSUPPORTED;
  if (M < 1 || M > (int64_t{1} << 26) || K < kQB || (K % kQB) != 0 || K > (int64_t{1} << 24) || group < kQB ||
      (group % kQB) != 0 || (K % group) != 0 || T < 1 || T > QMM_MMVQ_MAX_T)
    return QMM_ERR_SHAPE;
  if (!w || !scales || !xq || !y) return QMM_ERR_NULL;
  if (!aligned16(w) || !aligned16(scales) || !aligned16(zeros) || !aligned16(xq) || !aligned16(y))
    return QMM_ERR_ALIGN;
  const Q4gArgs a{static_cast<const uint8_t*>(w), scales, static_cast<const uint8_t*>(zeros),
                  static_cast<const uint8_t*>(xq), y, M, static_cast<int>(K / kQB), static_cast<int>(group / kQB),
                  static_cast<int>(K / group), static_cast<int>(T), scale_type};
  hipLaunchKernelGGL(mmvq_q4g_kernel, dim3(static_cast<unsigned>((M + 3) / 4)), dim3(256), 0, to_stream(stream), a);
  return launch_status();
}
