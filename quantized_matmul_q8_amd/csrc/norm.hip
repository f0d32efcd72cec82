// Root-mean-square norm with the residual's addition, written as Q8_1 rows,
// and Q8_1 rows read back.
//
//   h = x (+ r, rounded to r's type: the stored residual stream)
//   n = h * rstd * (w + offset),  rstd = 1 / sqrt(mean(h^2) + eps)
//   xq = Q8_1(n) with the steps of q8_1_quantize;  y = n rounded to y's type
//
// One workgroup per row; eight lanes own one 32-value block, four values
// each, as in q8_1_quantize.
#include "typed.hpp"

namespace qmm {

constexpr int kNormThreads = 256;
constexpr int64_t kMaxGrid = int64_t{1} << 22;  // workgroups of a launch: its threads are counted in 32 bits

struct NormArgs {
  const void* x;
  const void* res;
  void* res_out;
  const void* w;
  uint8_t* xq;
  void* y;
  int x_type, res_type, w_type, y_type;
  float offset, eps;
  int64_t T, K;
};

// Sum over the workgroup, in every thread (s: one float per wave).
__device__ __forceinline__ float block_sum(float v, float* s, int waves) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < waves; ++i) t += s[i];
  return t;
}

__global__ __launch_bounds__(kNormThreads) void rms_norm_q8_1_kernel(NormArgs a) {
  __shared__ float s[kNormThreads / 64];
  const int64_t n4 = a.K / 4;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
  const int64_t row4 = row * n4;
  float sum = 0.0f;
  for (int64_t i = threadIdx.x; i < n4; i += kNormThreads) {
    float4 h = load4(a.x_type, a.x, row4 + i);
    if (a.res) {
      const float4 r = load4(a.res_type, a.res, row4 + i);
      h = make_float4(h.x + r.x, h.y + r.y, h.z + r.z, h.w + r.w);
      store4(a.res_type, a.res_out, row4 + i, h);
      h = load4(a.res_type, a.res_out, row4 + i);
    }
    sum += (h.x * h.x + h.y * h.y) + (h.z * h.z + h.w * h.w);
  }
  sum = block_sum(sum, s, kNormThreads / 64);
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.K) + a.eps);
  for (int64_t i = threadIdx.x; i < n4; i += kNormThreads) {
    const float4 h = a.res ? load4(a.res_type, a.res_out, row4 + i) : load4(a.x_type, a.x, row4 + i);
    const float4 w = load4(a.w_type, a.w, i);
    const float4 n = make_float4(h.x * rstd * (w.x + a.offset), h.y * rstd * (w.y + a.offset),
                                 h.z * rstd * (w.z + a.offset), h.w * rstd * (w.w + a.offset));
    if (a.y) store4(a.y_type, a.y, row4 + i, n);
    const int64_t blk = (row4 + i) >> 3;
    q8_1_block_8lanes(n, static_cast<int>(i & 7), a.xq + blk * kQ8Bytes, true);
  }
  __syncthreads();
  }
}

__global__ __launch_bounds__(256) void q8_1_dequantize_kernel(const uint8_t* xq, void* x, int type, int64_t n4) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n4; i += static_cast<int64_t>(gridDim.x) * 256) {
  const uint8_t* b = xq + (i >> 3) * kQ8Bytes;
  const float d = h2f(ld_u16(b));
  const int q = reinterpret_cast<const int32_t*>(b + 4)[i & 7];
  store4(type, x, i,
         make_float4(d * static_cast<float>(static_cast<int8_t>(q)), d * static_cast<float>(static_cast<int8_t>(q >> 8)),
                     d * static_cast<float>(static_cast<int8_t>(q >> 16)), d * static_cast<float>(q >> 24)));
  }
}

}  // namespace qmm

using namespace qmm;

extern "C" int rms_norm_q8_1(const void* x, int x_type, const void* residual, void* residual_out, int res_type,
                             const void* weight, int w_type, float weight_offset, float eps, void* xq, void* y,
                             int y_type, int64_t T, int64_t K, void* stream) {
  if (!known_type(x_type) || !known_type(w_type) || ((residual || residual_out) && !known_type(res_type)) ||
      (y && !known_type(y_type)))
    return QMM_ERR_UNSUPPORTED;
  if (T < 0 || T > 0x7fffffff || K <= 0 || (K % kQB) != 0 || K > (int64_t{1} << 30)) return QMM_ERR_SHAPE;
  if (!(eps >= 0.0f)) return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!x || !weight || !xq || (residual == nullptr) != (residual_out == nullptr)) return QMM_ERR_NULL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(residual_out) || !aligned16(weight) || !aligned16(xq) ||
      !aligned16(y))
    return QMM_ERR_ALIGN;
  const NormArgs a{x, residual, residual_out, weight, static_cast<uint8_t*>(xq), y, x_type, res_type, w_type, y_type,
                   weight_offset, eps, T, K};
  hipLaunchKernelGGL(rms_norm_q8_1_kernel, dim3(static_cast<unsigned>(T < kMaxGrid ? T : kMaxGrid)), dim3(kNormThreads), 0, to_stream(stream), a);
  return launch_status();
}

extern "C" int q8_1_dequantize(const void* xq, void* x, int x_type, int64_t T, int64_t K, void* stream) {
  if (!known_type(x_type)) return QMM_ERR_UNSUPPORTED;
  if (T < 0 || K <= 0 || (K % kQB) != 0) return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!x || !xq) return QMM_ERR_NULL;
  if (!aligned16(x) || !aligned16(xq)) return QMM_ERR_ALIGN;
  if (T > (int64_t{1} << 40) / K) return QMM_ERR_SHAPE;
  const int64_t n4 = T * (K / 4);
  const int64_t need = (n4 + 255) / 256, grid = need < kMaxGrid ? need : kMaxGrid;
  hipLaunchKernelGGL(q8_1_dequantize_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, to_stream(stream),
                     static_cast<const uint8_t*>(xq), x, x_type, n4);
  return launch_status();
}
