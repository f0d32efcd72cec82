// Routing of tokens to experts: scores, a balancing bias, groups, top-k and
// weights, in the ids and expert_weights that the grouped calls take.
//
// The order has to be that of the exact values.  moe_router_kernel takes four
// tokens per wave, 16 lanes each, and finds the chosen in 32 bits; where two
// values at the border or in the order are closer than its rounding errors it
// leaves the token to route_token, which takes the whole wave and 64 bits.
//
// Its bytes are few: latency bounds it up to some thousand tokens (1 x 128:
// 3.3 us, 512 x 128: 4.4, most of it the launch; 4099 x 256 with a bias and
// groups 13.0), then the instructions: 16384 x 256, eight of them, no bias: 10.3
// us, 1.7 TB/s, 5.9 us of VALU time; 32768 x 384 with a bias: 22.1 us, 2.3 TB/s,
// 17.8 us of VALU time.  One token per wave in 64 bits throughout took 9.5, 43
// and 88 us for 1 x 128, 16384 x 256 and 32768 x 384; taking the best out one
// after the other instead of the candidates' ranks 12.0 and 35.8 for the latter
// two.
#include "typed.hpp"

#include <float.h>
#include <limits.h>

namespace qmm {

constexpr int kRouterMaxTopK = 64;
constexpr int kRouterMaxGroups = 64;
constexpr int kRouterWaves = 4;
constexpr int kRouterV = kMoeMaxE / 64;  // experts per lane where a wave has one token
constexpr double kMaskedValue = -1e300;  // below every selection value

struct RouterArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t T;
  int type, E, top_k, scoring, groups, keep, group_score, renorm;
  float scale;
  uint32_t magic;  // ceil(2^20 / (E / groups))
};

__device__ __forceinline__ float load1(int type, const void* p, int64_t i) {
  if (type == QMM_F32) return static_cast<const float*>(p)[i];
  if (type == QMM_F16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}

// LDS written before by the wave is read after: a wave's LDS instructions keep
// their order, so this holds the compiler alone.
__device__ __forceinline__ void wave_fence() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// Reductions over each row of 16 lanes (in all of its lanes) and over the wave
// (uniform).
template <int CTRL>
__device__ __forceinline__ int row_ror(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);
}
template <class Fn>
__device__ __forceinline__ int row_reduce(int v, Fn fn) {
  v = fn(v, row_ror<0x128>(v));
  v = fn(v, row_ror<0x124>(v));
  v = fn(v, row_ror<0x122>(v));
  return fn(v, row_ror<0x121>(v));
}
template <class Fn>
__device__ __forceinline__ float row_reduce_f(float v, Fn fn) {
  return __builtin_bit_cast(float, row_reduce(__builtin_bit_cast(int, v), [&](int x, int y) {
    return __builtin_bit_cast(int, fn(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)));
  }));
}
template <class Fn>
__device__ __forceinline__ int wave_reduce(int v, Fn fn) {
  v = row_reduce(v, fn);
  return fn(fn(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
            fn(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = row_reduce_f(v, [](float x, float y) { return fmaxf(x, y); });
  const int b = __builtin_bit_cast(int, v);
  return fmaxf(
      fmaxf(__builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0)), __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16))),
      fmaxf(__builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32)), __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48))));
}

// A float's (double's) bits as a signed integer of the same order, and back.
__device__ __forceinline__ int order_key(float c) {
  const int k = __builtin_bit_cast(int, c + 0.0f);  // -0 as 0
  return k ^ ((k >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) { return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7fffffff)); }
__device__ __forceinline__ int64_t order_key(double c) {
  const int64_t k = __builtin_bit_cast(int64_t, c + 0.0);
  return k ^ ((k >> 63) & INT64_MAX);
}

// Sigmoid scores of logits below this are taken in 64 bits for their shares of
// a sum: in fp32 they come near the subnormals (from -87.3), and from -88.7 on
// exp(-x) is infinite and all of them 0.  route_token takes such tokens.
constexpr float kSmallSigmoid = -80.0f;
__device__ __forceinline__ double sigmoid64(float x) { return 1.0 / (1.0 + exp(-static_cast<double>(x))); }

// One token by the whole wave, its order in 64 bits.  Lane l holds experts l*V
// .. l*V + V - 1 (V = ceil(E/64)): the lowest lane of several with the same
// value has the lowest expert.  s_pick: a double per expert.
__device__ __noinline__ void route_token(RouterArgs a, int64_t t, double* s_pick) {
  const int lane = threadIdx.x & 63;
  const int V = (a.E + 63) / 64;
  const bool softmax = a.scoring == QMM_SCORE_SOFTMAX;
  const bool scored = a.bias || (a.groups > 1 && a.group_score != QMM_GROUP_MAX);
  float x[kRouterV];
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < kRouterV; ++v) {
    x[v] = -INFINITY;
    if (v < V) {
      const int e = lane * V + v;
      const float l = load1(a.type, a.logits, t * a.E + min(e, a.E - 1));
      x[v] = l > -INFINITY && e < a.E ? fminf(l, FLT_MAX) : -INFINITY;  // NaN counts as masked
    }
    top = fmaxf(top, x[v]);
  }
  top = wave_max(top);
  const float ref = top > -INFINITY ? top : 0.0f;
  // selection values in 64 bits
  double pick[kRouterV], sum = 0.0;
#pragma unroll
  for (int v = 0; v < kRouterV; ++v) {
    pick[v] = static_cast<double>(x[v]);
    if (v < V && scored) {
      pick[v] = softmax ? exp(static_cast<double>(x[v]) - static_cast<double>(ref))
                        : sigmoid64(x[v]);
      sum += pick[v];
    }
  }
  if (scored) {
    if (softmax)
      for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    const double div = softmax && sum > 0.0 ? sum : 1.0;
#pragma unroll
    for (int v = 0; v < kRouterV; ++v) {
      if (v < V) {
        const int e = min(lane * V + v, a.E - 1);
        if (softmax) pick[v] /= div;
        if (a.bias) pick[v] += static_cast<double>(a.bias[e]);
      }
    }
  }
  uint64_t kept = ~0ull;
  const int per = a.E / a.groups;
  if (a.groups > 1) {
    wave_fence();
#pragma unroll
    for (int v = 0; v < kRouterV; ++v)
      if (v < V && lane * V + v < a.E) s_pick[lane * V + v] = x[v] > -INFINITY ? pick[v] : kMaskedValue;
    wave_fence();
    int span = 1;  // lanes that share a group
    while (span * 2 * a.groups <= 64) span *= 2;
    const int g = lane / span;
    double b0 = kMaskedValue, b1 = kMaskedValue;
    if (g < a.groups) {
#pragma unroll 4
      for (int i = lane % span; i < per; i += span) {
        const double p = s_pick[g * per + i];
        b1 = fmax(b1, fmin(b0, p));
        b0 = fmax(b0, p);
      }
    }
    for (int d = 1; d < span; d <<= 1) {
      const double o0 = __shfl_xor(b0, d), o1 = __shfl_xor(b1, d);
      b1 = fmax(fmin(b0, o0), fmax(b1, o1));
      b0 = fmax(b0, o0);
    }
    const double best = a.group_score != QMM_GROUP_MAX && b1 > kMaskedValue ? b0 + b1 : b0;
    wave_fence();
    if (g < a.groups) s_pick[g] = best;
    wave_fence();
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < a.groups; ++j) {
      const double o = s_pick[j];
      rank += (o > best || (o == best && j < g)) ? 1 : 0;
    }
    wave_fence();
    // bit g of the kept groups, from the first lane of each
    const uint64_t in = __ballot(g < a.groups && rank < a.keep);
    kept = 0;
    for (int j = 0; j < a.groups; ++j) kept |= (in >> (j * span) & 1) << j;
  }
  int64_t key[kRouterV];
#pragma unroll
  for (int v = 0; v < kRouterV; ++v) {
    const int e = lane * V + v;
    // without a bias the order is the logits'
    const int64_t k = order_key(a.bias ? pick[v] : static_cast<double>(x[v]));
    key[v] = INT64_MIN;
    if (v < V && e < a.E && ((kept >> (e / per)) & 1 || a.groups == 1))
      key[v] = x[v] > -INFINITY ? k : INT64_MIN + 1;
  }
  // top-k: the wave's largest each time
  const auto larger = [](int p, int q) { return max(p, q); };
  int my_id = 0;
  float my_x = -INFINITY;
  for (int k = 0; k < a.top_k; ++k) {
    int64_t best = key[0];
    int at = 0;
    float bx = x[0];
#pragma unroll
    for (int v = 1; v < kRouterV; ++v)
      if (v < V && key[v] > best) {
        best = key[v];
        at = v;
        bx = x[v];
      }
    const int hi = static_cast<int>(best >> 32);
    const int top_hi = wave_reduce(hi, larger);
    // the low half as signed: its order with the highest bit turned
    const int lo = hi == top_hi ? static_cast<int>(static_cast<uint32_t>(best) ^ 0x80000000u) : INT_MIN;
    const int top_lo = wave_reduce(lo, larger);
    const int owner = __ffsll(static_cast<unsigned long long>(__ballot(hi == top_hi && lo == top_lo))) - 1;
#pragma unroll
    for (int v = 0; v < kRouterV; ++v)
      if (lane == owner && v == at) key[v] = INT64_MIN;
    const int id = __builtin_amdgcn_readlane(lane * V + at, owner);
    const float px = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, bx), owner));
    if (lane == k) {
      my_id = id;
      my_x = px;
    }
  }
  // weights of the chosen, in lanes 0 .. top_k - 1
  const bool mine = lane < a.top_k, live = mine && my_x > -INFINITY;
  float w = 0.0f;
  if (softmax) {
    const float at = a.renorm ? wave_max(mine ? my_x : -INFINITY) : top;
    if (live) w = expf(my_x - at);
    if (!a.renorm) {
      float z = 0.0f;
#pragma unroll
      for (int v = 0; v < kRouterV; ++v) z += x[v] > -INFINITY ? expf(x[v] - ref) : 0.0f;
      z = wave_sum(z);
      if (live) w /= z;
    }
  } else if (live) {
    w = 1.0f / (1.0f + expf(-my_x));
  }
  if (a.renorm && !softmax && __any(live && my_x < kSmallSigmoid)) {
    const double s = live ? sigmoid64(my_x) : 0.0;
    double z = s;
    for (int d = 32; d; d >>= 1) z += __shfl_xor(z, d);
    w = z > 0.0 ? static_cast<float>(s / z) : 0.0f;
  } else if (a.renorm) {
    const float z = wave_sum(w);
    if (z > 0.0f) w /= z;
  }
  if (mine) {
    a.ids[t * a.top_k + lane] = my_id;
    a.weights[t * a.top_k + lane] = w * a.scale;
  }
  wave_fence();
}

__global__ __launch_bounds__(kRouterWaves * 64) void moe_router_wide_kernel(RouterArgs a) {
  __shared__ double s_pick[kRouterWaves][kMoeMaxE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWaves + wave;
  if (t < a.T) route_token(a, t, s_pick[wave]);
}

template <int N>
__device__ __forceinline__ int row_shr(int v) {  // lane i's from lane i - N of its row, 0 before the first
  return __builtin_amdgcn_update_dpp(0, v, 0x110 + N, 0xf, 0xf, true);
}
__device__ __forceinline__ float row_shl1(float v) {  // lane i's from lane i + 1 of its row
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x101, 0xf, 0xf, true));
}
// fn(value, its lane of the row) for the 15 other lanes of the row
template <int R = 1, class Fn>
__device__ __forceinline__ void for_others(int v, Fn fn) {
  if constexpr (R < 16) {
    fn(row_ror<0x120 + R>(v), ((threadIdx.x & 15) - R) & 15);
    for_others<R + 1>(v, fn);
  }
}
template <int R = 1, class Fn>
__device__ __forceinline__ void for_others2(int2 v, Fn fn) {
  if constexpr (R < 16) {
    fn(make_int2(row_ror<0x120 + R>(v.x), row_ror<0x120 + R>(v.y)));
    for_others2<R + 1>(v, fn);
  }
}

// order keys below those of all floats; masked experts have one each, the lower expert's the larger
constexpr int kTaken = INT_MIN, kMasked = INT_MIN + 1 + kMoeMaxE;

constexpr float kLog2e = 1.44269504088896340736f;

// Four tokens per wave, lane li of a token's 16 holds experts v*16 + li (v <
// V).
//
// The n best (n = top_k, with a bias two more) without n rounds over all
// experts: the n-th largest of the 16 lanes' maxima is a bound that n experts
// reach, so the experts that reach it are the candidates; they are few (nine
// for the best seven of 384), go one to a lane, and each lane counts those
// before its own.  Only where more than 16 reach the bound (n near 16, many
// equal values, masks) the n best are taken out one after the other.
//
// Without a bias the order is that of the logits and exact.  With one, c = s +
// b in fp32.  Error of s, with exp2 and the reciprocal good to 2^-23:
// softmax, relative, (2.5 |x - max| + 56) * 2^-24 (the difference, its product
// with log2 e, exp2, a sum with chains of V + 4 <= 36, its terms' errors, the
// division), and s * 2.5 |x - max| <= 1; sigmoid, 1/(1+e): s (1 - s) times e's
// relative error (1.5 |x| + 2) * 2^-24, and 3 s * 2^-24 of sum and reciprocal,
// with s (1 - s) |x| < 0.23.  So |error of c| <= (1 + kappa + |c|) * 2^-24 with
// kappa 56 times the largest probability, and 3.  Neighbours of the first top_k + 1 that are closer than
// both errors, or groups at the border of the kept, make the token unsure.
// The n best then get their exponentials in 64 bits and are ranked again; if
// that leaves a doubt (the softmax's sum, still in 32 bits; the n-th, whose
// 32-bit c bounds the rest, not clearly below the chosen), and for the groups,
// route_token takes the token.
template <int V>
__global__ __launch_bounds__(kRouterWaves * 64) void moe_router_kernel(RouterArgs a) {
  // with groups, per wave a float per token and expert, or route_token's double per expert
  extern __shared__ double s_values[];
  __shared__ float s_group[kRouterWaves][4][2][kRouterMaxGroups];  // a group's value, and its terms' magnitudes added
  __shared__ int2 s_cand[kRouterWaves][2][4][17];  // the 17th takes what is no candidate
  const int lane = threadIdx.x & 63, li = lane & 15, tok = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouterWaves + wave) * 4;
  if (t0 >= a.T) return;
  const int64_t t = min(t0 + tok, a.T - 1);
  double* s_pick = s_values + wave * 2 * a.E;
  const auto fmax2 = [](float x, float y) { return fmaxf(x, y); };
  const auto fmin2 = [](float x, float y) { return fminf(x, y); };
  const auto add2 = [](float x, float y) { return x + y; };
  const bool softmax = a.scoring == QMM_SCORE_SOFTMAX;
  // E > kFull * 16: this many v need no test for the last expert (the launch takes the smallest V)
  constexpr int kFull = V <= 2 ? 0 : V <= 4 ? 2 : V <= 8 ? 4 : V <= 12 ? 8 : V <= 16 ? 12 : V <= 24 ? 16 : 24;

  float x[V], bias[V];
  const uint32_t at = static_cast<uint32_t>(min(static_cast<int64_t>(tok), a.T - 1 - t0)) * a.E;  // from the first token
  const auto load = [&](const auto* p) {
    if (a.E == V * 16) {  // constant distances
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = static_cast<float>(p[at + v * 16 + li]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = static_cast<float>(p[at + min(v * 16 + li, a.E - 1)]);
    }
  };
  // one branch for all loads, so that they are in flight together
  if (a.type == QMM_F32) load(static_cast<const float*>(a.logits) + t0 * a.E);
  else if (a.type == QMM_F16) load(static_cast<const _Float16*>(a.logits) + t0 * a.E);
  else load(static_cast<const __bf16*>(a.logits) + t0 * a.E);
  if (a.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = a.bias[min(v * 16 + li, a.E - 1)];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = 0.0f;
  }
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // NaN and what is behind the last expert count as masked, +inf as the largest finite value
    x[v] = fminf(fmaxf(x[v], -INFINITY), FLT_MAX);
    if (v >= kFull) x[v] = v * 16 + li < a.E ? x[v] : -INFINITY;
    top = fmaxf(top, x[v]);
  }
  top = row_reduce_f(top, fmax2);
  const float ref = top > -INFINITY ? top : 0.0f;

  // scores, where the order or the weights need them for all experts
  const bool scored = a.bias || (a.groups > 1 && a.group_score != QMM_GROUP_MAX);
  float c[V], sum = 0.0f;
  if (softmax && (scored || !a.renorm)) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = __builtin_amdgcn_exp2f((x[v] - ref) * kLog2e);
      sum += c[v];
    }
    sum = row_reduce_f(sum, add2);
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  if (scored && softmax) {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = c[v] * inv + bias[v];
  } else if (scored) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      c[v] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[v] * -kLog2e)) + bias[v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = x[v];
  }

  // no score is larger: 1/sum is the largest logit's
  const float kappa = softmax ? 56.0f * inv : 3.0f;
  bool unsure = false;  // of the groups
  uint32_t inside = 0;  // bit v: expert v*16 + li is in a kept group
  if (a.groups > 1) {
    const int per = a.E / a.groups;
    int span = 1;  // lanes that share a group
    while (span * 2 * a.groups <= 16) span *= 2;
    float* mine = reinterpret_cast<float*>(s_pick) + tok * a.E;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 16 + li < a.E) mine[v * 16 + li] = x[v] > -INFINITY ? c[v] : -INFINITY;
    wave_fence();
    for (int g0 = 0; g0 < a.groups; g0 += 16) {
      const int g = g0 + li / span;
      float b0 = -INFINITY, b1 = -INFINITY;
      const auto take = [&](int i) {
        const float p = mine[g * per + i];
        b1 = fmaxf(b1, fminf(b0, p));
        b0 = fmaxf(b0, p);
      };
      if (g < a.groups) {
        const int all = per / span, first = li % span;  // rounds that every lane of a group has
#pragma unroll 8
        for (int i = 0; i < all; ++i) take(first + i * span);
        if (first < per - all * span) take(first + all * span);
      }
      for (int d = 1; d < span; d <<= 1) {
        const float o0 = __shfl_xor(b0, d), o1 = __shfl_xor(b1, d);
        b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
        b0 = fmaxf(b0, o0);
      }
      if (g < a.groups) {
        const float second = a.group_score != QMM_GROUP_MAX && b1 > -INFINITY ? b1 : 0.0f;
        s_group[wave][tok][0][g] = b0 + second;
        s_group[wave][tok][1][g] = b0 > -INFINITY ? fabsf(b0) + fabsf(second) : 0.0f;
      }
    }
    wave_fence();
    // Of the kept the least that one can be, of the others the most.  A group's error is that of its terms, which its sum
    // may be far smaller than: 2 (1 + kappa) * 2^-24, and twice their magnitudes for theirs and the sum's rounding (taken
    // twice, for the roundings here).  Terms that add up past fp32 can be anything; groups without unmasked experts are
    // all the same.
    float low = INFINITY, high = -INFINITY;
    uint64_t kept = 0;  // bit g: group g of the token
    for (int g0 = 0; g0 < a.groups; g0 += 16) {
      const int g = g0 + li;
      const float mine = s_group[wave][tok][0][min(g, a.groups - 1)], size = s_group[wave][tok][1][min(g, a.groups - 1)];
      const float err = 0x1p-23f * (1.0f + kappa) + 0x1p-22f * size, from = size < INFINITY ? mine : 0.0f;
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < a.groups; ++j) {
        const float o = s_group[wave][tok][0][j];
        rank += o > mine || (o == mine && j < g) ? 1 : 0;
      }
      const bool in = g < a.groups && rank < a.keep;
      kept |= (__ballot(in) >> (lane & 48) & 0xffff) << g0;
      if (in) low = fminf(low, from - err);
      else if (g < a.groups) high = fmaxf(high, from + err);
    }
    low = row_reduce_f(low, fmin2);
    high = row_reduce_f(high, fmax2);
    // where all others are masked, the kept are right; scores by the logits have no error
    if (scored) unsure = high > -INFINITY && !(low > high);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // e / per: exact, for e times the multiplier's error is below 2^9 * 2^9
      const uint32_t g = __umul24(static_cast<uint32_t>(v * 16 + li), a.magic) >> 20;
      inside |= static_cast<uint32_t>(kept >> (g & 63) & 1) << v;
    }
  }
  int key[V];
  const bool biased = a.bias != nullptr;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float by = biased ? c[v] : x[v];
    key[v] = x[v] > -INFINITY ? order_key(by) : kMasked - (v * 16 + li);
    if (v >= kFull) key[v] = v * 16 + li < a.E ? key[v] : kTaken;
  }
  if (a.groups > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = inside >> v & 1 ? key[v] : kTaken;
  }

  // lane j < n gets the j-th best
  const int n = a.top_k + (biased ? 2 : 0);
  int my_key = kTaken, my_id = 0;
  int m = key[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = max(m, key[v]);
  int rank = 0;
  for_others(m, [&](int o, int lane_o) { rank += o > m || (o == m && lane_o < li) ? 1 : 0; });
  const int bound = row_reduce(rank == n - 1 ? m : INT_MIN, [](int p, int q) { return max(p, q); });
  int count = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) count += key[v] >= bound ? 1 : 0;
  int upto = count;  // of this lane and those before it
  upto += row_shr<1>(upto);
  upto += row_shr<2>(upto);
  upto += row_shr<4>(upto);
  upto += row_shr<8>(upto);
  const int all = row_reduce(upto, [](int p, int q) { return max(p, q); });
  int2* cand = s_cand[wave][0][tok];
  int2* sorted = s_cand[wave][1][tok];
  if (!__any(all > 16)) {
    int at = upto - count;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool in = key[v] >= bound;
      cand[in ? at : 16] = make_int2(key[v], v * 16 + li);
      at += in ? 1 : 0;
    }
    wave_fence();
    const int2 own = li < all ? cand[li] : make_int2(kTaken, kMoeMaxE + li);
    int place = 0;
    for_others2(own, [&](int2 o) { place += o.x > own.x || (o.x == own.x && o.y < own.y) ? 1 : 0; });
    sorted[place] = own;
    wave_fence();
    const int2 got = sorted[li];
    my_key = got.x;
    my_id = got.y;
    wave_fence();
  } else {
    for (int k = 0; k < n; ++k) {
      if (k) {
        m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = max(m, key[v]);
      }
      const int best = row_reduce(m, [](int p, int q) { return max(p, q); });
      int at = V;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) at = key[v] == best ? v : at;
      const int mine = at * 16 + li;  // no expert of this lane: past all experts
      const int id = row_reduce(mine, [](int p, int q) { return min(p, q); });
      const int out = mine == id ? at : -1;
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = v == out ? kTaken : key[v];
      if (li == k) {
        my_key = best;
        my_id = id;
      }
    }
  }
  bool live = my_key > kMasked && li < n;
  float mine_x = -INFINITY;
  if (live) {
    mine_x = key_value(my_key);
    if (biased) mine_x = fminf(load1(a.type, a.logits, t * a.E + my_id), FLT_MAX);
  }

  rank = li;
  if (biased) {
    const float now = key_value(my_key), b = a.bias[min(my_id, a.E - 1)], next = row_shl1(now);
    const bool next_live = row_shl1(live ? 1.0f : 0.0f) > 0.0f;
    const float margin = 0x1p-23f * (1.0f + kappa + fmaxf(fabsf(now), fabsf(next)));
    const bool close = li < a.top_k && live && next_live && !(now - next > margin);
    const uint64_t closes = __ballot(close);
    if (closes) {  // any of the wave's tokens
      const bool token = (closes >> (lane & 48) & 0xffff) != 0;
      // The n best again, their exponentials in 64 bits; masked ones stay behind, in their order.  The softmax's sum keeps
      // a relative error below 56 * 2^-24 =: r, which moves the difference of two values by r |s - s'|.
      const double r = softmax ? 0x1p-24 * 56.0 : 0.0;
      double score64 = 0.0, d = -1e300 * (li + 1) / 64;
      if (live) {
        score64 = softmax ? exp(static_cast<double>(mine_x) - static_cast<double>(ref)) / static_cast<double>(sum)
                          : sigmoid64(mine_x);
        d = score64 + static_cast<double>(b);
      }
      if (li >= n) d = -DBL_MAX;
      int place = 0;
      bool doubt = false;
#pragma unroll
      for (int k = 1; k < 16; ++k) {
        const int src = (lane & 48) | ((li + k) & 15);
        const double od = __shfl(d, src), os = __shfl(score64, src);
        const int id = __shfl(my_id, src);
        place += od > d || (od == d && id < my_id) ? 1 : 0;
        doubt = doubt || (fabs(od - d) <= r * fabs(os - score64) && os != score64);
      }
      // every expert that is not among the n has a 32-bit c of at most the n-th's
      const int last = (lane & 48) | (n - 1);
      const float last_c = __shfl(now, last);
      const bool last_live = __shfl(live ? 1 : 0, last) != 0;
      const double above = static_cast<double>(last_c) + 0x1p-22 * (1.0 + kappa + fabs(last_c));
      // a bias that is not finite has no place among the others
      const bool bad = token && live && (!(fabs(d) < DBL_MAX) ||
                                         (place < a.top_k && (doubt || (last_live && !(d - r * score64 > above)))));
      if (token) rank = place;
      unsure = unsure || (__ballot(bad) >> (lane & 48) & 0xffff) != 0;
    }
  }

  // weights of the chosen
  const bool chosen = rank < a.top_k && li < n;
  live = live && chosen;
  float w = 0.0f;
  // NaNs of some bits have the key of what is taken
  bool again = unsure || (li < a.top_k && my_key == kTaken);
  if (softmax) {
    const float at = a.renorm ? row_reduce_f(live ? mine_x : -INFINITY, fmax2) : top;
    if (live) w = expf(mine_x - at);
    if (!a.renorm && live) w /= sum;
  } else if (live) {
    w = 1.0f / (1.0f + expf(-mine_x));
    if (a.renorm && mine_x < kSmallSigmoid) again = true;
  }
  if (a.renorm) {
    const float z = row_reduce_f(w, add2);
    if (z > 0.0f) w /= z;
  }
  const uint64_t redo = __ballot(again);
  if (chosen && t0 + tok < a.T && !(redo >> (lane & 48) & 0xffff)) {
    a.ids[t * a.top_k + rank] = my_id;
    a.weights[t * a.top_k + rank] = w * a.scale;
  }
  if (redo) {
    for (int i = 0; i < 4; ++i)
      if ((redo >> (16 * i) & 0xffff) && t0 + i < a.T) route_token(a, t0 + i, s_pick);
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
  if (T < 0 || T > (int64_t{1} << 25) || E < 1 || E > kMoeMaxE || n_groups < 1 || n_groups > kRouterMaxGroups ||
      (E % n_groups) != 0 || topk_groups < 1 || topk_groups > n_groups || top_k < 1 || top_k > kRouterMaxTopK ||
      top_k > topk_groups * (E / n_groups))
    return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!logits || !ids || !weights) return QMM_ERR_NULL;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(weights)) return QMM_ERR_ALIGN;
  const uint32_t per = static_cast<uint32_t>(E / n_groups);
  const RouterArgs a{logits, bias, ids, weights, T, type, static_cast<int>(E), static_cast<int>(top_k), scoring,
                     static_cast<int>(n_groups), static_cast<int>(topk_groups), group_score, renormalize, scale,
                     ((1u << 20) + per - 1) / per};
  hipStream_t st = to_stream(stream);
  const dim3 block(kRouterWaves * 64);
  if (top_k + (bias ? 2 : 0) > 16) {
    // more picks than a token's 16 lanes hold: one token per wave (16384 x 256, 32 of them: 103 us, bound by its 3600
    // VALU instructions a token)
    hipLaunchKernelGGL(moe_router_wide_kernel, dim3(static_cast<unsigned>((T + kRouterWaves - 1) / kRouterWaves)), block,
                       0, st, a);
    return launch_status();
  }
  const dim3 grid(static_cast<unsigned>((T + 4 * kRouterWaves - 1) / (4 * kRouterWaves)));
  const size_t lds = n_groups > 1 ? kRouterWaves * 2 * static_cast<size_t>(E) * sizeof(double) : 0;
  const int v = static_cast<int>((E + 15) / 16);  // experts per lane
  if (v <= 2) hipLaunchKernelGGL(moe_router_kernel<2>, grid, block, lds, st, a);
  else if (v <= 4) hipLaunchKernelGGL(moe_router_kernel<4>, grid, block, lds, st, a);
  else if (v <= 8) hipLaunchKernelGGL(moe_router_kernel<8>, grid, block, lds, st, a);
  else if (v <= 12) hipLaunchKernelGGL(moe_router_kernel<12>, grid, block, lds, st, a);
  else if (v <= 16) hipLaunchKernelGGL(moe_router_kernel<16>, grid, block, lds, st, a);
  else if (v <= 24) hipLaunchKernelGGL(moe_router_kernel<24>, grid, block, lds, st, a);
  else hipLaunchKernelGGL(moe_router_kernel<32>, grid, block, lds, st, a);
  return launch_status();
}
