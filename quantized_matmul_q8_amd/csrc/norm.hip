// Root-mean-square norm with the residual's addition, written as Q8_1 rows,
// and Q8_1 rows read back.
//
//   h = x (+ r, rounded to r's type: the stored residual stream)
//   n = h * rstd * (w + offset),  rstd = 1 / sqrt(mean(h^2) + eps)
//       (by powers of two where squares would leave fp32)
//   xq = Q8_1(n) with the steps of q8_1_quantize;  y = n rounded to y's type
//
// A row stays in registers between the sum of its squares and its output: 64
// to 1024 threads hold it, eight consecutive values per lane and chunk, up to
// four chunks.  A quad of lanes owns one 32-value block.  The split of a row
// depends on K alone, so its result does not depend on T.
//
// Bound by HBM: 16384 x 8192, bf16 with a bf16 residual, 7.25 bytes a value:
// 180 us, 5.4 TB/s (a copy of 1 GiB reaches 5.1); reading the row again after
// the sum took 306 us.  A few rows are bound by the launch and three round
// trips (1 x 4096: 3.0 us).  Reading 8192 x 11008 back to bf16: 44.5 us, 6.6
// TB/s, to fp32 82 us, 5.7 TB/s (asked of the memory side, where the last-level
// cache serves a part that the counters do not tell apart).
#include "typed.hpp"

#include <algorithm>

namespace qmm {

constexpr int64_t kMaxGrid = int64_t{1} << 20;  // workgroups of a launch: its threads are counted in 32 bits
constexpr int kNoType = -1;

struct NormArgs {
  const void* x;
  const void* res;
  void* res_out;
  const void* w;
  uint8_t* xq;
  void* y;
  int w_type, y_type;
  float offset, eps;
  int64_t T, K;
  int row_threads;  // 64, or the workgroup's threads
  bool large;       // the stream is larger than what the last-level cache (256 MB) would keep of it
};

// 1 / sqrt(mean + eps); 0 where the mean is 0 and there is no eps, and where it is infinite.
__device__ __forceinline__ float rms_scale(float sum, const NormArgs& a) {
  const float ms = sum / static_cast<float>(a.K) + a.eps;
  return ms == 0.0f ? 0.0f : 1.0f / sqrtf(ms);
}

// One 32-value block by a quad of lanes, eight values each: the steps and so
// the bytes of q8_1_block_8lanes.  Lane part p writes bytes 4 + 8p .. 11 + 8p,
// and the first and last the scale and the sum.
__device__ __forceinline__ void q8_1_block_4lanes(const float (&v)[8], int part, uint8_t* dst) {
#pragma clang fp contract(off)
  float am = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(v[j]));
  am = fmaxf(am, lane8_xchg<0xb1>(am));
  am = fmaxf(am, lane8_xchg<0x4e>(am));
  const float d = am / 127.0f;
  const float di = d >= 0x1p-126f ? 1.0f / d : 0.0f;
  uint32_t p[2] = {0u, 0u};
  int s = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int q = max(-128, min(127, static_cast<int>(rintf(v[j] * di))));
    s += q;
    p[j >> 2] |= (static_cast<uint32_t>(q) & 255u) << (8 * (j & 3));
  }
  s += lane8_xchg<0xb1>(s);
  s += lane8_xchg<0x4e>(s);
  struct __attribute__((aligned(4))) Two { uint32_t a, b; };
  *reinterpret_cast<Two*>(dst + 4 + 8 * part) = Two{p[0], p[1]};
  if (part == 0 || part == 3)
    *reinterpret_cast<uint32_t*>(dst + (part ? 36 : 0)) = part ? static_cast<uint32_t>(s) : f2h_bits(d);
}

// Whether a row has to be done again with its values scaled: where its mean
// square + eps is past fp32 (rstd 0 or NaN) or below 2^-96, where squares come
// near the subnormals (above it those that vanish move it by less than 2^-50).
__device__ __forceinline__ bool is_odd(float rstd) { return !(rstd > 0.0f && rstd <= 0x1p48f); }

// Such a row once more, from memory: each wave sums all of it and writes its
// part.  `by` multiplies the values and `sq` these again for their squares alone:
//   past fp32: values of at most 2^124 then, squares of up to 2^64, 1/rms above
//     2^-126; a value that loses bits has a result below 2^-126
//   below 2^-96: up to 2^30 values below 2^-33 give a sum below 2^126, the
//     smallest subnormal a square of 2^-106.
__device__ __forceinline__ void odd_row(const NormArgs& a, int type, const void* from, int64_t row, int tid, bool past) {
  __asm__ volatile("" : "+v"(tid));  // no address from it is worked out before the usual rows
  const int64_t n8 = a.K / 8, at = row * n8;
  const float by = past ? 0x1p-4f : 0x1p96f, sq = past ? 0x1p-92f : 1.0f, f = by * sq;
  float h[8], sum = 0.0f;
  for (int64_t i = tid & 63; i < n8; i += 64) {
    load8(type, from, at + i, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[j] * f, h[j] * f, sum);
  }
  const float ms = wave_sum(sum) / static_cast<float>(a.K) + a.eps * f * f;
  // a row of zeros without an eps stays zeros
  const float rstd = ms == 0.0f ? 0.0f : 1.0f / sqrtf(ms) * sq;
  for (int64_t i = tid; i < n8; i += a.row_threads) {
    float w[8];
    load8(type, from, at + i, h);
    load8(a.w_type, a.w, i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = h[j] * by * rstd * (w[j] + a.offset);
    if (a.y) {
      store4(a.y_type, a.y, 2 * (at + i), make_float4(h[0], h[1], h[2], h[3]));
      store4(a.y_type, a.y, 2 * (at + i) + 1, make_float4(h[4], h[5], h[6], h[7]));
    }
    q8_1_block_4lanes(h, static_cast<int>(i & 3), a.xq + ((at + i) >> 2) * kQ8Bytes);
  }
}

// The odd ones among a workgroup's rows, each wave its own, found by their sums,
// which are added up as norm_rows does.  A row's waves have waited for each
// other's stores of the stream at the barriers there.  Behind all rows, for
// within their loop this costs registers (4096 x 11008, fp32: 72 us for 57).
__device__ __forceinline__ void odd_rows(const NormArgs& a, int type, const void* from, int wave) {
  const int64_t n8 = a.K / 8;
  const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)), thread = wave * 64 + lane;
  const int tid = thread % a.row_threads, rows = blockDim.x / a.row_threads;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows + thread / a.row_threads; row < a.T;
       row += static_cast<int64_t>(gridDim.x) * rows) {
    float all = 0.0f;
    for (int k = 0; k < a.row_threads; k += 64) {
      float h[8], sum = 0.0f;
      for (int64_t i = k + lane; i < n8; i += a.row_threads) {
        load8(type, from, row * n8 + i, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[j], h[j], sum);
      }
      all += wave_sum(sum);
    }
    const float rstd = rms_scale(all, a);
    if (is_odd(rstd)) odd_row(a, type, from, row, tid, !(all / static_cast<float>(a.K) + a.eps < INFINITY));
  }
}

// True where a row of the wave is odd.
template <int XT, int RT, int WT, int C, bool LATE>
__device__ __forceinline__ bool norm_rows(const NormArgs& a, float* s_sum) {
  bool odd = false;
  const int64_t n8 = a.K / 8;
  const int tid = threadIdx.x % a.row_threads;
  const int rows = blockDim.x / a.row_threads;  // of the workgroup; above one where a wave has a row
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows; row0 < a.T; row0 += static_cast<int64_t>(gridDim.x) * rows) {
    const int64_t row = row0 + threadIdx.x / a.row_threads, at = row * n8;
    const bool on = row < a.T;
    Raw8<XT> x[C];
    Raw8<RT == kNoType ? QMM_F32 : RT> r[C];
    Raw8<WT> w[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * a.row_threads + tid;
      if (on && i < n8) {
        x[c].load_once(a.x, at + i);
        if constexpr (RT != kNoType) r[c].load_once(a.res, at + i);
        if constexpr (!LATE) w[c].load(a.w, i);
      }
    }
    float h[C][8], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * a.row_threads + tid;
      if (on && i < n8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = x[c].get(j);
        if constexpr (RT != kNoType) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] += r[c].get(j);
          r[c].set(h[c]);
          if (a.large) r[c].store_nt(a.res_out, at + i);
          else r[c].store(a.res_out, at + i);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = r[c].get(j);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[c][j], h[c][j], sum);
      }
    }
    sum = wave_sum(sum);
    if (a.row_threads > 64) {
      const int waves = a.row_threads >> 6, first = threadIdx.x / a.row_threads * waves;  // of the row
      if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
      __syncthreads();
      sum = 0.0f;
      for (int k = 0; k < waves; ++k) sum += s_sum[first + k];
      __syncthreads();  // before the next row's
    }
    const float rstd = rms_scale(sum, a);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * a.row_threads + tid;
      if (on && i < n8) {
        if constexpr (LATE) w[c].load(a.w, i);
        float n[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = h[c][j] * rstd * (w[c].get(j) + a.offset);
        if (a.y) {
          if (a.y_type == QMM_F32) {
            Raw8<QMM_F32> y;
            y.set(n);
            y.store(a.y, at + i);
          } else if (a.y_type == QMM_F16) {
            Raw8<QMM_F16> y;
            y.set(n);
            y.store(a.y, at + i);
          } else {
            Raw8<QMM_BF16> y;
            y.set(n);
            y.store(a.y, at + i);
          }
        }
        q8_1_block_4lanes(n, i & 3, a.xq + ((at + i) >> 2) * kQ8Bytes);
      }
    }
    odd = odd || (on && is_odd(rstd));
  }
  return odd;
}

// LATE: the weights are read after the sum, for fewer registers and so two
// workgroups of more than 512 threads per CU (4096 x 11008, fp32: 57 us, 66
// with the weights read with the row; 16384 x 8192 on 512 threads: 194 and 188).
template <int XT, int RT, int C, bool LATE>
__global__ __launch_bounds__(1024) void rms_norm_q8_1_kernel(NormArgs a) {
  __shared__ float s_sum[16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // not from the thread's number, a register more
  const bool odd = a.w_type == QMM_F32   ? norm_rows<XT, RT, QMM_F32, C, LATE>(a, s_sum)
                   : a.w_type == QMM_F16 ? norm_rows<XT, RT, QMM_F16, C, LATE>(a, s_sum)
                                         : norm_rows<XT, RT, QMM_BF16, C, LATE>(a, s_sum);
  if (odd) odd_rows(a, RT == kNoType ? XT : RT, RT == kNoType ? a.x : a.res_out, wave);
}

// One chunk per lane: up to 64 vector registers, so eight waves per SIMD if a
// wave has at most 80 scalar ones (16384 x 4096, bf16: 85 us, 91 with more).
// The same body, and no function for both, with which 16384 x 8192 took 186 us
// for 183.
template <int XT, int RT>
__global__ __launch_bounds__(1024) __attribute__((amdgpu_num_sgpr(80))) void rms_norm_q8_1_short_kernel(NormArgs a) {
  constexpr int C = 1;
  constexpr bool LATE = false;
  __shared__ float s_sum[16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // not from the thread's number, a register more
  const bool odd = a.w_type == QMM_F32   ? norm_rows<XT, RT, QMM_F32, C, LATE>(a, s_sum)
                   : a.w_type == QMM_F16 ? norm_rows<XT, RT, QMM_F16, C, LATE>(a, s_sum)
                                         : norm_rows<XT, RT, QMM_BF16, C, LATE>(a, s_sum);
  if (odd) odd_rows(a, RT == kNoType ? XT : RT, RT == kNoType ? a.x : a.res_out, wave);
}

// Rows of more than 32768 values: read again after the sum.  Scalar registers
// as above (300 x 65536, bf16: 64 us, 101 with more than 80).
__global__ __launch_bounds__(1024) __attribute__((amdgpu_num_sgpr(80)))
void rms_norm_q8_1_long_kernel(NormArgs a, int x_type, int res_type) {
  __shared__ float s_sum[16];
  const int64_t n4 = a.K / 4;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t row4 = row * n4;
    float sum = 0.0f;
    for (int64_t i = threadIdx.x; i < n4; i += 1024) {
      float4 h = load4(x_type, a.x, row4 + i);
      if (a.res) {
        const float4 r = load4(res_type, a.res, row4 + i);
        store4(res_type, a.res_out, row4 + i, make_float4(h.x + r.x, h.y + r.y, h.z + r.z, h.w + r.w));
        h = load4(res_type, a.res_out, row4 + i);  // this thread's own, as stored
      }
      sum += (h.x * h.x + h.y * h.y) + (h.z * h.z + h.w * h.w);
    }
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int k = 0; k < 16; ++k) sum += s_sum[k];
    __syncthreads();
    const float rstd = rms_scale(sum, a);
    for (int64_t i = threadIdx.x; i < n4; i += 1024) {
      const float4 h = a.res ? load4(res_type, a.res_out, row4 + i) : load4(x_type, a.x, row4 + i);
      const float4 w = load4(a.w_type, a.w, i);
      const float4 n = make_float4(h.x * rstd * (w.x + a.offset), h.y * rstd * (w.y + a.offset),
                                   h.z * rstd * (w.z + a.offset), h.w * rstd * (w.w + a.offset));
      if (a.y) store4(a.y_type, a.y, row4 + i, n);
      q8_1_block_8lanes(n, static_cast<int>(i & 7), a.xq + ((row4 + i) >> 3) * kQ8Bytes, true);
    }
    if (is_odd(rstd)) {
      __syncthreads();  // other threads wrote what this one writes again
      odd_row(a, a.res ? res_type : x_type, a.res ? a.res_out : a.x, row, threadIdx.x,
              !(sum / static_cast<float>(a.K) + a.eps < INFINITY));
    }
  }
}

template <int XT, int RT>
static void launch_norm(NormArgs a, hipStream_t st) {
  // Threads per row, by K alone: eight values each up to 4096 (1 x 4096: 3.0 us; with sixteen 3.4, but 16384 x 4096
  // 93 and 91 us), then sixteen (16384 x 8192: 186 us, with eight 191, with 32 229; all with plain loads), and 32 where a
  // workgroup is full.
  // Up to 2048 values a workgroup has several rows.
  const int chunks = a.K <= 4096 ? 1 : a.K <= 16384 ? 2 : 4;
  a.row_threads = a.K <= 512 ? 64 : a.K <= 1024 ? 128 : a.K <= 2048 ? 256
                  : static_cast<int>((a.K / (8 * chunks) + 63) / 64 * 64);
  const int threads = std::max(256, a.row_threads), rows = a.K <= 2048 ? 256 / a.row_threads : 1;
  a.row_threads = a.K <= 2048 ? a.row_threads : threads;
  const dim3 g(static_cast<unsigned>(std::min((a.T + rows - 1) / rows, kMaxGrid))), b(threads);
  if (chunks == 1) hipLaunchKernelGGL((rms_norm_q8_1_short_kernel<XT, RT>), g, b, 0, st, a);
  else if (chunks == 2 && threads <= 512) hipLaunchKernelGGL((rms_norm_q8_1_kernel<XT, RT, 2, false>), g, b, 0, st, a);
  else if (chunks == 2) hipLaunchKernelGGL((rms_norm_q8_1_kernel<XT, RT, 2, true>), g, b, 0, st, a);
  else hipLaunchKernelGGL((rms_norm_q8_1_kernel<XT, RT, 4, true>), g, b, 0, st, a);
}

template <int XT>
static void launch_norm(const NormArgs& a, int res_type, hipStream_t st) {
  if (!a.res) launch_norm<XT, kNoType>(a, st);
  else if (res_type == QMM_F32) launch_norm<XT, QMM_F32>(a, st);
  else if (res_type == QMM_F16) launch_norm<XT, QMM_F16>(a, st);
  else launch_norm<XT, QMM_BF16>(a, st);
}

// N = 16 bytes' worth of values per lane (four fp32 or eight 16-bit ones); U of
// these per thread, their loads first.
template <int TY>
__global__ __launch_bounds__(256) void q8_1_dequantize_kernel(const uint8_t* xq, void* x, int64_t n) {
  constexpr int U = 4, N = TY == QMM_F32 ? 4 : 8, kLanes = 32 / N;
  struct __attribute__((aligned(4))) Bytes { uint32_t w[N / 4]; };
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * (256 * U) + threadIdx.x; base < n;
       base += static_cast<int64_t>(gridDim.x) * (256 * U)) {
    Bytes q[U];
    uint32_t d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = min(base + u * 256, n - 1);
      const uint8_t* b = xq + i / kLanes * kQ8Bytes;
      q[u] = *reinterpret_cast<const Bytes*>(b + 4 + N * (i % kLanes));
      d[u] = ld_u16(b);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = base + u * 256;
      if (i < n) {
        const float s = h2f(d[u]);
        float f[N];
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = s * static_cast<float>(static_cast<int8_t>(q[u].w[j / 4] >> (8 * (j & 3))));
        if constexpr (TY == QMM_F32) {
          static_cast<float4*>(x)[i] = make_float4(f[0], f[1], f[2], f[3]);
        } else {
          Raw8<TY> out;
          out.set(f);
          out.store(x, i);
        }
      }
    }
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
  const NormArgs a{x, residual, residual_out, weight, static_cast<uint8_t*>(xq), y, w_type, y_type, weight_offset, eps,
                   T, K, 1024,  // set by launch_norm for rows that stay in registers
                   // its stores then leave the caches to the other data (4096 x 24576, bf16: 175 -> 143 us; 16384 x 8192:
                   // 186 -> 181); a smaller one the next kernel finds there
                   T * K >= (int64_t{128} << 20) / (res_type == QMM_F32 ? 4 : 2)};
  hipStream_t st = to_stream(stream);
  if (K > 32768)
    hipLaunchKernelGGL(rms_norm_q8_1_long_kernel, dim3(static_cast<unsigned>(std::min(T, kMaxGrid))), dim3(1024), 0, st,
                       a, x_type, res_type);
  else if (x_type == QMM_F32) launch_norm<QMM_F32>(a, res_type, st);
  else if (x_type == QMM_F16) launch_norm<QMM_F16>(a, res_type, st);
  else launch_norm<QMM_BF16>(a, res_type, st);
  return launch_status();
}

extern "C" int q8_1_dequantize(const void* xq, void* x, int x_type, int64_t T, int64_t K, void* stream) {
  if (!known_type(x_type)) return QMM_ERR_UNSUPPORTED;
  if (T < 0 || K <= 0 || (K % kQB) != 0) return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!x || !xq) return QMM_ERR_NULL;
  if (!aligned16(x) || !aligned16(xq)) return QMM_ERR_ALIGN;
  if (T > (int64_t{1} << 40) / K) return QMM_ERR_SHAPE;
  const int64_t n = T * (K / (x_type == QMM_F32 ? 4 : 8));
  const dim3 g(static_cast<unsigned>(std::min((n + 1023) / 1024, kMaxGrid))), b(256);
  hipStream_t st = to_stream(stream);
  const uint8_t* q = static_cast<const uint8_t*>(xq);
  if (x_type == QMM_F32) hipLaunchKernelGGL(q8_1_dequantize_kernel<QMM_F32>, g, b, 0, st, q, x, n);
  else if (x_type == QMM_F16) hipLaunchKernelGGL(q8_1_dequantize_kernel<QMM_F16>, g, b, 0, st, q, x, n);
  else hipLaunchKernelGGL(q8_1_dequantize_kernel<QMM_BF16>, g, b, 0, st, q, x, n);
  return launch_status();
}
