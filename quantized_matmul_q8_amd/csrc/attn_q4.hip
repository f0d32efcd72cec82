// Attention of a sequence's last tokens over the paged 4-bit cache.
//
// One wave per query row: scores key by key, with the running maximum and sum
// of the softmax.
#include "kv_q4.hpp"

#include <algorithm>
#include <math.h>

namespace qmm {

struct AttnQ4Args {
  const void* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  void* y;
  int64_t q_stride, pages, page, W, window;
  float scale;
  int B, n, Hq, Hk, D, type, y_type;
};

__device__ __forceinline__ float load1(int type, const void* p, int64_t i) {
  if (type == QMM_F32) return static_cast<const float*>(p)[i];
  if (type == QMM_F16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}
__device__ __forceinline__ void store1(int type, void* p, int64_t i, float v) {
  if (type == QMM_F32) static_cast<float*>(p)[i] = v;
  else if (type == QMM_F16) static_cast<_Float16*>(p)[i] = static_cast<_Float16>(v);
  else static_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
}

__global__ __launch_bounds__(64) void attn_q4_kernel(AttnQ4Args a) {
  const int lane = threadIdx.x;
  const int h = blockIdx.x % a.Hq, row = blockIdx.x / a.Hq, b = row / a.n, i = row % a.n, kh = h / (a.Hq / a.Hk);
  const int64_t len = max(int64_t{0}, min(a.W * a.page, static_cast<int64_t>(a.lens[b])));
  const int64_t at = len - a.n + i, first = a.window > 0 ? max(int64_t{0}, at - a.window + 1) : 0;
  const int nb = a.D / 32;
  float q[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, top = -INFINITY, sum = 0.0f;
  for (int r = 0; r < 4; ++r) {
    const int d = lane + 64 * r;
    q[r] = d < a.D ? load1(a.type, a.q, row * a.q_stride + h * a.D + d) * a.scale : 0.0f;
  }
  for (int64_t j = first; j <= at; ++j) {
    const int64_t pg = a.table[b * a.W + j / a.page];
    if (pg < 0 || pg >= a.pages) continue;
    const uint8_t* cell = a.cache + kv_cell(pg * a.page + j % a.page, a.page, kh, a.Hk, a.D);
    const int t = static_cast<int>(j % kCellTokens), quad = t >> 2;
    float s = 0.0f, v[4];
    for (int r = 0; r < 4; ++r) {
      const int d = lane + 64 * r, blk = d >> 5, e = d & 7;
      v[r] = 0.0f;
      if (d >= a.D) continue;
      const uint32_t kb = cell[(blk * 16 + t) * 16 + (d & 31) / 8 * 4 + (e & 1) * 2 + (e >> 2)];
      const uint16_t* ks = reinterpret_cast<const uint16_t*>(cell + 8 * a.D + (blk * 16 + t) * 4);
      const float d16 = h2f(ks[0]), m16 = h2f(ks[1]);
      s += q[r] * h2f(f2h_bits(__builtin_fmaf(static_cast<float>((e & 2) ? kb >> 4 : kb & 15u), d16, m16)));
      const uint32_t vb = cell[10 * a.D + ((quad * 16 + (d & 15)) * nb + blk) * 4 + kv_quad_byte(t & 3)];
      const uint16_t* vs = reinterpret_cast<const uint16_t*>(cell + 18 * a.D + (quad * nb + blk) * 16) + (t & 3);
      v[r] = h2f(f2h_bits(__builtin_fmaf(static_cast<float>((d & 16) ? vb >> 4 : vb & 15u), h2f(vs[0]), h2f(vs[4]))));
    }
    s = wave_sum(s);
    const float up = fmaxf(top, s), keep = expf(top - up), p = expf(s - up);
    sum = sum * keep + p;
    for (int r = 0; r < 4; ++r) o[r] = o[r] * keep + p * v[r];
    top = up;
  }
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  for (int r = 0; r < 4; ++r) {
    const int d = lane + 64 * r;
    if (d < a.D) store1(a.y_type, a.y, (static_cast<int64_t>(row) * a.Hq + h) * a.D + d, o[r] * inv);
  }
}

static bool attn_q4_shape(int64_t B, int64_t n, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  return B >= 0 && n >= 1 && n <= QMM_ATTN_MAX_N && Hk >= 1 && Hq >= Hk && Hq <= 1024 && Hq % Hk == 0 &&
         attn_head_dim(D) && max_len >= 1 && max_len <= (int64_t{1} << 30) && B < (int64_t{1} << 26) / (n * Hq);
}

}  // namespace qmm

using namespace qmm;

extern "C" size_t attn_q4_workspace_bytes(int64_t B, int64_t n, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  if (!attn_q4_shape(B, n, Hq, Hk, D, max_len)) return 0;
  return 0;
}

extern "C" int attn_q4(const void* q, int64_t q_stride, int type, const void* cache, int64_t pages, int64_t page,
                       const int32_t* table, int64_t W, const int32_t* lens, float scale, int64_t window, void* y,
                       int y_type, int64_t B, int64_t n, int64_t Hq, int64_t Hk, int64_t D, void* ws, size_t ws_bytes,
                       void* stream) {
  if ((type != QMM_F16 && type != QMM_BF16) || !known_type(y_type)) return QMM_ERR_UNSUPPORTED;
  if (!kv_q4_shape(pages, page, Hk, D) || W < 1 || W > (int64_t{1} << 30) / page) return QMM_ERR_SHAPE;
  if (!attn_q4_shape(B, n, Hq, Hk, D, W * page) || !strided_rows(q_stride, Hq, D)) return QMM_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || window > 0x7fffffff) return QMM_ERR_SHAPE;
  if (B == 0) return QMM_OK;
  const size_t need = attn_q4_workspace_bytes(B, n, Hq, Hk, D, W * page);
  if (!q || !cache || !table || !lens || !y || (need > 0 && !ws)) return QMM_ERR_NULL;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(table) || !aligned16(lens) || !aligned16(y) || !aligned16(ws))
    return QMM_ERR_ALIGN;
  if (ws_bytes < need) return QMM_ERR_WORKSPACE;
  const AttnQ4Args a{q, static_cast<const uint8_t*>(cache), table, lens, y, q_stride, pages, page, W, window, scale,
                     static_cast<int>(B), static_cast<int>(n), static_cast<int>(Hq), static_cast<int>(Hk),
                     static_cast<int>(D), type, y_type};
  hipLaunchKernelGGL(attn_q4_kernel, dim3(static_cast<unsigned>(B * n * Hq)), dim3(64), 0, to_stream(stream), a);
  return launch_status();
}
