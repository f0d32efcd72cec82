// Norm of each query and key head with the position rotation, in one pass.
//
//   n = x * rstd * (w + offset),  rstd = 1 / sqrt(mean(x^2) + eps) over the head
//   out = n with each pair (a, b) turned: a c - b s, b c + a s
//
// A head of D values lies in D/16 lanes (rounded up to a power of two), as two
// chunks of eight each: those whose values are pairs, so a turn needs no other
// lane.  A wave holds one token's cosines and sines in registers while it goes
// over heads of that token.
//
// Bound by HBM: 16384 x 72 x 128 in bf16, 612 MB, 111 to 116 us on three cards,
// 5.3 to 5.5 TB/s, the rate of a copy; one token by the launch, 3.6 us.
#include "typed.hpp"

#include <algorithm>

namespace qmm {

struct RopeArgs {
  const void* x[2];  // q, k
  const void* w[2];
  void* y[2];
  int64_t x_stride[2], y_stride[2];
  int heads[2], units[2];  // a unit: as many heads as a wave holds
  const float* rope;
  const int32_t* positions;
  int64_t T, P;
  int D, rot, row_lanes, w_type, per_wave;
  bool interleaved, large;
  float offset, eps;
};

// The sum over the lanes of a head, in each of them.
__device__ __forceinline__ float row_sum(float v, int lanes) {
  for (int k = 1; k < lanes; k *= 2) v += __shfl_xor(v, k);
  return v;
}

// 1/rms of sixteen values per lane; `by` multiplies the values first where
// their squares leave fp32: past it (or NaN) 2^-70 keeps them below 2^58, and
// below a mean of 2^-96, where squares come near the subnormals, 2^96 keeps
// them below 2^53.
__device__ __forceinline__ float head_scale(const float (&v)[16], const RopeArgs& a, float& by) {
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) sum = __builtin_fmaf(v[j], v[j], sum);
  const float n = static_cast<float>(a.D), ms = row_sum(sum, a.row_lanes) / n + a.eps;
  by = 1.0f;
  if (ms >= 0x1p-96f && ms < INFINITY) return 1.0f / sqrtf(ms);
  by = ms < 0x1p-96f ? 0x1p96f : 0x1p-70f;
  sum = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) sum = __builtin_fmaf(v[j] * by, v[j] * by, sum);
  const float odd = row_sum(sum, a.row_lanes) / n + a.eps * by * by;
  return odd == 0.0f ? 0.0f : 1.0f / sqrtf(odd);
}

template <int XT, int YT>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(RopeArgs a) {
  const int lane = threadIdx.x & 63, groups = 64 / a.row_lanes;
  const int p = lane % a.row_lanes, group = lane / a.row_lanes;
  const int units = a.units[0] + a.units[1], segs = (units + a.per_wave - 1) / a.per_wave;
  const uint32_t item = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = item / static_cast<uint32_t>(segs);
  if (t >= a.T) return;
  const int u0 = static_cast<int>(item % static_cast<uint32_t>(segs)) * a.per_wave, u1 = min(units, u0 + a.per_wave);
  const bool in_head = p < a.D / 16, turned = p < a.rot / 16, halves = turned && !a.interleaved;
  const int ca = halves ? p : 2 * p, cb = halves ? p + a.rot / 16 : 2 * p + 1;
  float cos[8], sin[8];
  if (turned) {
    const int64_t row = max(int64_t{0}, min(a.P - 1, static_cast<int64_t>(a.positions[t])));
    load8(QMM_F32, a.rope, (row * a.rot) / 8 + p, cos);
    load8(QMM_F32, a.rope, (row * a.rot + a.rot / 2) / 8 + p, sin);
  }
  float w[16];
  int have = -1;  // the side whose weights these are
  for (int u = u0; u < u1; ++u) {
    const int side = u < a.units[0] ? 0 : 1;
    const int h = (u - (side ? a.units[0] : 0)) * groups + group;
    const bool on = in_head && h < a.heads[side];
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
    if (on) {
      const int64_t at = (t * a.x_stride[side] + static_cast<int64_t>(h) * a.D) / 8;
      Raw8<XT> lo, hi;
      // Large calls read past the caches too: what wrote the rows has filled these, and lines that are taken in push its
      // stores out (16384 x 72 x 128 behind their writer: 146 -> 124 us).  Not where two loads share lines.
      if (a.large && !a.interleaved) lo.load_once(a.x[side], at + ca), hi.load_once(a.x[side], at + cb);
      else lo.load(a.x[side], at + ca), hi.load(a.x[side], at + cb);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = lo.get(j), v[8 + j] = hi.get(j);
    }
    if (a.w[side]) {
      if (have != side && in_head) {
        float part[8];
        load8(a.w_type, a.w[side], ca, part);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = part[j] + a.offset;
        load8(a.w_type, a.w[side], cb, part);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[8 + j] = part[j] + a.offset;
      }
      have = side;
      float by;
      const float rstd = head_scale(v, a, by);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = v[j] * by * rstd * w[j];
    }
    if (turned) {
      float r[16];
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[2 * j] = v[2 * j] * cos[j] - v[2 * j + 1] * sin[j];
          r[2 * j + 1] = v[2 * j + 1] * cos[j] + v[2 * j] * sin[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[j] = v[j] * cos[j] - v[8 + j] * sin[j];
          r[8 + j] = v[8 + j] * cos[j] + v[j] * sin[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = r[j];
    }
    if (on) {
      const int64_t at = (t * a.y_stride[side] + static_cast<int64_t>(h) * a.D) / 8;
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) lo[j] = v[j], hi[j] = v[8 + j];
      Raw8<YT> o;
      o.set(lo);
      if (a.large) o.store_nt(a.y[side], at + ca);
      else o.store(a.y[side], at + ca);
      o.set(hi);
      if (a.large) o.store_nt(a.y[side], at + cb);
      else o.store(a.y[side], at + cb);
    }
  }
}

template <int XT>
static void launch_rope(const RopeArgs& a, int out_type, dim3 g, hipStream_t st) {
  if (out_type == QMM_F32) hipLaunchKernelGGL((qk_norm_rope_kernel<XT, QMM_F32>), g, dim3(256), 0, st, a);
  else if (out_type == QMM_F16) hipLaunchKernelGGL((qk_norm_rope_kernel<XT, QMM_F16>), g, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((qk_norm_rope_kernel<XT, QMM_BF16>), g, dim3(256), 0, st, a);
}

}  // namespace qmm

using namespace qmm;

extern "C" int qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int type,
                            const void* q_weight, const void* k_weight, int w_type, float weight_offset, float eps,
                            const float* rope, int64_t P, int64_t rot, int interleaved, const int32_t* positions,
                            void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, int out_type,
                            int64_t T, int64_t Hq, int64_t Hk, int64_t D, void* stream) {
  if (!known_type(type) || !known_type(out_type) || ((q_weight || k_weight) && !known_type(w_type)))
    return QMM_ERR_UNSUPPORTED;
  if (Hq < 1 || Hq > 1024 || (k && (Hk < 1 || Hk > 1024)) || D < 32 || D > 512 || D % 32 != 0) return QMM_ERR_SHAPE;
  if (T < 0 || T >= kMostRows || T > 0x7fffffff / (Hq + (k ? Hk : 0))) return QMM_ERR_SHAPE;
  if (rot < 0 || rot % 16 != 0 || rot > D || (rot > 0 && (P < 1 || P > 0x7fffffff))) return QMM_ERR_SHAPE;
  if (!(eps >= 0.0f)) return QMM_ERR_SHAPE;
  if (!strided_rows(q_stride, Hq, D) || !strided_rows(q_out_stride, Hq, D)) return QMM_ERR_SHAPE;
  if (k && (!strided_rows(k_stride, Hk, D) || !strided_rows(k_out_stride, Hk, D)))
    return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!q || !q_out || (k && !k_out) || (rot > 0 && (!rope || !positions))) return QMM_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(rope) ||
      !aligned_list(positions, 4) || !aligned16(q_out) || !aligned16(k_out))
    return QMM_ERR_ALIGN;
  int lanes = 2;
  while (lanes * 16 < D) lanes *= 2;
  const int groups = 64 / lanes;
  RopeArgs a{{q, k}, {q_weight, k_weight}, {q_out, k_out}, {q_stride, k_stride}, {q_out_stride, k_out_stride},
             {static_cast<int>(Hq), k ? static_cast<int>(Hk) : 0}, {0, 0}, rope, positions, T, P, static_cast<int>(D),
             static_cast<int>(rot), lanes, w_type, 1, interleaved != 0,
             large_output(T * (Hq + (k ? Hk : 0)) * D, out_type), weight_offset, eps};
  for (int s = 0; s < 2; ++s) a.units[s] = (a.heads[s] + groups - 1) / groups;
  const int64_t units = a.units[0] + a.units[1];
  a.per_wave = static_cast<int>(std::max<int64_t>(1, std::min(units, T * units / 16384)));
  const int64_t waves = T * ((units + a.per_wave - 1) / a.per_wave);
  const dim3 g(static_cast<unsigned>((waves + 3) / 4));
  hipStream_t st = to_stream(stream);
  if (type == QMM_F32) launch_rope<QMM_F32>(a, out_type, g, st);
  else if (type == QMM_F16) launch_rope<QMM_F16>(a, out_type, g, st);
  else launch_rope<QMM_BF16>(a, out_type, g, st);
  return launch_status();
}
