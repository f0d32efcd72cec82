// Attention over whole prompts, packed sequences.
//
// One wave per query row and head: scores key by key, with the running maximum
// and sum of the softmax.
#include "typed.hpp"

#include <math.h>

namespace qmm {

inline bool prompt_head_dim(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* y;
  int64_t q_stride, k_stride, v_stride, window, Tq, Tk;
  float scale;
  int B, Hq, Hk, D, type, y_type;
  bool causal;
};

__device__ __forceinline__ float prompt_load(int type, const void* p, int64_t i) {
  if (type == QMM_F16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}

__global__ __launch_bounds__(64) void attn_prompt_kernel(PromptArgs a) {
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x / a.Hq;
  const int h = blockIdx.x % a.Hq, kh = h / (a.Hq / a.Hk);
  int b = 0;
  while (b < a.B && row >= a.cu_q[b + 1]) ++b;
  if (b == a.B || row < a.cu_q[b]) return;
  const auto within = [](int64_t x, int64_t lo, int64_t hi) { return max(lo, min(hi, x)); };
  const int64_t q0 = within(a.cu_q[b], 0, a.Tq), q1 = within(a.cu_q[b + 1], q0, a.Tq);
  const int64_t k0 = within(a.cu_k[b], 0, a.Tk), k1 = within(a.cu_k[b + 1], k0, a.Tk);
  const int64_t nk = k1 - k0, at = nk - (q1 - q0) + (row - q0);
  const int64_t first = a.window > 0 ? max(int64_t{0}, at - a.window + 1) : 0, last = a.causal ? at : nk - 1;
  float q[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, top = -INFINITY, sum = 0.0f;
  for (int r = 0; r < 4; ++r) {
    const int d = lane + 64 * r;
    q[r] = d < a.D ? prompt_load(a.type, a.q, row * a.q_stride + h * a.D + d) * a.scale : 0.0f;
  }
  for (int64_t j = first; j <= last; ++j) {
    float s = 0.0f, v[4];
    for (int r = 0; r < 4; ++r) {
      const int d = lane + 64 * r;
      v[r] = 0.0f;
      if (d >= a.D) continue;
      s += q[r] * prompt_load(a.type, a.k, (k0 + j) * a.k_stride + kh * a.D + d);
      v[r] = prompt_load(a.type, a.v, (k0 + j) * a.v_stride + kh * a.D + d);
    }
    s = wave_sum(s);
    if (s == -INFINITY) continue;
    const float up = fmaxf(top, s), keep = expf(top - up), p = expf(s - up);
    sum = sum * keep + p;
    for (int r = 0; r < 4; ++r) o[r] = o[r] * keep + p * v[r];
    top = up;
  }
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  for (int r = 0; r < 4; ++r) {
    const int d = lane + 64 * r;
    const int64_t i = (row * a.Hq + h) * a.D + d;
    if (d >= a.D) continue;
    if (a.y_type == QMM_F32) static_cast<float*>(a.y)[i] = o[r] * inv;
    else if (a.y_type == QMM_F16) static_cast<_Float16*>(a.y)[i] = static_cast<_Float16>(o[r] * inv);
    else static_cast<__bf16*>(a.y)[i] = static_cast<__bf16>(o[r] * inv);
  }
}

}  // namespace qmm

using namespace qmm;

extern "C" int attn_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, int type, const int32_t* cu_q, const int32_t* cu_k, int64_t B, float scale,
                           int causal, int64_t window, void* y, int y_type, int64_t Tq, int64_t Tk, int64_t Hq,
                           int64_t Hk, int64_t D, void* stream) {
  if ((type != QMM_F16 && type != QMM_BF16) || !known_type(y_type) || (window > 0 && !causal)) return QMM_ERR_UNSUPPORTED;
  if (B < 0 || Tq < 0 || Tk < 0 || Tq >= (int64_t{1} << 30) || Tk >= (int64_t{1} << 30)) return QMM_ERR_SHAPE;
  if (Hk < 1 || Hq < Hk || Hq > 1024 || Hq % Hk != 0 || !prompt_head_dim(D)) return QMM_ERR_SHAPE;
  if (B > 0x7fffffff || (Tq / 64 + B) * Hq > 0x7fffffff) return QMM_ERR_SHAPE;
  if (!strided_rows(q_stride, Hq, D) || !strided_rows(k_stride, Hk, D) || !strided_rows(v_stride, Hk, D))
    return QMM_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || window > 0x7fffffff) return QMM_ERR_SHAPE;
  if (B == 0 || Tq == 0) return QMM_OK;
  if (!q || !cu_q || !cu_k || !y || (Tk > 0 && (!k || !v))) return QMM_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cu_q) || !aligned16(cu_k) || !aligned16(y))
    return QMM_ERR_ALIGN;
  const PromptArgs a{q, k, v, cu_q, cu_k, y, q_stride, k_stride, v_stride, window, Tq, Tk, scale, static_cast<int>(B),
                     static_cast<int>(Hq), static_cast<int>(Hk), static_cast<int>(D), type, y_type, causal != 0};
  hipLaunchKernelGGL(attn_prompt_kernel, dim3(static_cast<unsigned>(Tq * Hq)), dim3(64), 0, to_stream(stream), a);
  return launch_status();
}
