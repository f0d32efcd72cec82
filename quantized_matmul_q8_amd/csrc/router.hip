// Routing of tokens to experts: scores, a balancing bias, groups, top-k and
// weights, in the ids and expert_weights that the grouped calls take.
//
// One wave64 per token; lane l holds experts l*V .. l*V + V - 1 (V =
// ceil(E/64)), so the order of lanes is the order of experts and the lowest
// lane of several with the same value has the lowest expert.
#include "typed.hpp"

#include <float.h>

namespace qmm {

constexpr int kRouterMaxTopK = 64;
constexpr int kRouterMaxGroups = 64;
constexpr int kRouterWaves = 4;
constexpr int kRouterV = kMoeMaxE / 64;
constexpr double kMaskedOrder = -1e300;     // below every selection value
constexpr double kOutsideOrder = -DBL_MAX;  // an expert of a group that is not kept

struct RouterArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t T;
  int type, E, top_k, scoring, groups, keep, group_score, renorm;
  float scale;
};

__device__ __forceinline__ float load1(int type, const void* p, int64_t i) {
  if (type == QMM_F32) return static_cast<const float*>(p)[i];
  if (type == QMM_F16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}

__device__ __forceinline__ float wave_max(float v) {
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

__global__ __launch_bounds__(kRouterWaves * 64) void moe_router_kernel(RouterArgs a) {
  __shared__ double s_pick[kRouterWaves][kMoeMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWaves + wave;
  if (t >= a.T) return;
  const int V = (a.E + 63) / 64;
  float x[kRouterV];
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < kRouterV; ++v) {
    const int e = lane * V + v;
    x[v] = -INFINITY;
    if (v < V && e < a.E) {
      const float l = load1(a.type, a.logits, t * a.E + e);
      x[v] = l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;  // NaN counts as masked
    }
    top = fmaxf(top, x[v]);
  }
  top = wave_max(top);
  const bool none = !(top > -INFINITY);
  // scores in 64 bits for the order, selection values, order keys
  double ord[kRouterV], sum = 0.0;
#pragma unroll
  for (int v = 0; v < kRouterV; ++v) {
    const bool live = x[v] > -INFINITY;
    double sc = 0.0;
    if (live) sc = a.scoring == QMM_SCORE_SOFTMAX ? exp(static_cast<double>(x[v]) - static_cast<double>(top))
                                                  : 1.0 / (1.0 + exp(-static_cast<double>(x[v])));
    ord[v] = sc;
    sum += sc;
  }
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  uint64_t kept = ~0ull;
  const int per = a.E / a.groups;
#pragma unroll
  for (int v = 0; v < kRouterV; ++v) {
    const int e = lane * V + v;
    const bool in = v < V && e < a.E, live = x[v] > -INFINITY;
    double pick = ord[v];
    if (a.scoring == QMM_SCORE_SOFTMAX && !none) pick /= sum;
    if (in && a.bias) pick += static_cast<double>(a.bias[e]);
    ord[v] = !in ? kOutsideOrder : !live ? kMaskedOrder : a.bias ? pick : static_cast<double>(x[v]);
    if (in) s_pick[wave][e] = !live ? kMaskedOrder : a.bias || a.group_score != QMM_GROUP_MAX ? pick : x[v];
  }
  if (a.groups > 1) {
    __builtin_amdgcn_wave_barrier();
    double best = kOutsideOrder;
    if (lane < a.groups) {
      double b0 = kMaskedOrder, b1 = kMaskedOrder;
      for (int i = 0; i < per; ++i) {
        const double p = s_pick[wave][lane * per + i];
        b1 = fmax(b1, fmin(b0, p));
        b0 = fmax(b0, p);
      }
      best = b0;
      if (a.group_score != QMM_GROUP_MAX && b1 > kMaskedOrder) best += b1;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(best, g);
      rank += (o > best || (o == best && g < lane)) ? 1 : 0;
    }
    kept = __ballot(lane < a.groups && rank < a.keep);
#pragma unroll
    for (int v = 0; v < kRouterV; ++v) {
      const int e = lane * V + v;
      if (v < V && e < a.E && !((kept >> (e / per)) & 1)) ord[v] = kOutsideOrder;
    }
  }
  // top-k: the wave's largest each time, the lowest expert of equal ones
  int my_id = 0;
  float my_x = -INFINITY;
  for (int k = 0; k < a.top_k; ++k) {
    double best = kOutsideOrder;
    int at = kMoeMaxE;
    float bx = -INFINITY;
#pragma unroll
    for (int v = 0; v < kRouterV; ++v)
      if (ord[v] > best) { best = ord[v]; at = lane * V + v; bx = x[v]; }
    for (int d = 32; d; d >>= 1) {
      const double o = __shfl_xor(best, d);
      const int oa = __shfl_xor(at, d);
      const float ox = __shfl_xor(bx, d);
      if (o > best || (o == best && oa < at)) { best = o; at = oa; bx = ox; }
    }
#pragma unroll
    for (int v = 0; v < kRouterV; ++v)
      if (lane * V + v == at) ord[v] = kOutsideOrder;
    if (lane == k) { my_id = at; my_x = bx; }
  }
  // weights of the chosen, in lanes 0 .. top_k - 1
  const bool mine = lane < a.top_k, live = mine && my_x > -INFINITY;
  float w = 0.0f;
  if (a.scoring == QMM_SCORE_SOFTMAX) {
    const float ref = a.renorm ? wave_max(mine ? my_x : -INFINITY) : top;
    if (live) w = expf(my_x - ref);
    if (!a.renorm) {
      float z = 0.0f;
#pragma unroll
      for (int v = 0; v < kRouterV; ++v) z += x[v] > -INFINITY ? expf(x[v] - top) : 0.0f;
      z = wave_sum(z);
      if (live) w /= z;
    }
  } else if (live) {
    w = 1.0f / (1.0f + expf(-my_x));
  }
  if (a.renorm) {
    const float z = wave_sum(w);
    if (z > 0.0f) w /= z;
  }
  if (mine) {
    a.ids[t * a.top_k + lane] = my_id;
    a.weights[t * a.top_k + lane] = w * a.scale;
  }
}

}  // namespace qmm

using namespace qmm;

extern "C" int moe_router(const void* logits, int type, int64_t T, int64_t E, int64_t top_k, int scoring,
                          const float* bias, int64_t n_groups, int64_t topk_groups, int group_score, int renormalize,
                          float scale, int32_t* ids, float* weights, void* stream) {
  if (!known_type(type) || (scoring != QMM_SCORE_SOFTMAX && scoring != QMM_SCORE_SIGMOID) ||
      (group_score != QMM_GROUP_MAX && group_score != QMM_GROUP_TOP2))
    return QMM_ERR_UNSUPPORTED;
  if (T < 0 || T > (int64_t{1} << 26) || E < 1 || E > kMoeMaxE || n_groups < 1 || n_groups > kRouterMaxGroups ||
      (E % n_groups) != 0 || topk_groups < 1 || topk_groups > n_groups || top_k < 1 || top_k > kRouterMaxTopK ||
      top_k > topk_groups * (E / n_groups))
    return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!logits || !ids || !weights) return QMM_ERR_NULL;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(weights)) return QMM_ERR_ALIGN;
  const RouterArgs a{logits, bias, ids, weights, T, type, static_cast<int>(E), static_cast<int>(top_k), scoring,
                     static_cast<int>(n_groups), static_cast<int>(topk_groups), group_score, renormalize, scale};
  hipLaunchKernelGGL(moe_router_kernel, dim3(static_cast<unsigned>((T + kRouterWaves - 1) / kRouterWaves)),
                     dim3(kRouterWaves * 64), 0, to_stream(stream), a);
  return launch_status();
}
