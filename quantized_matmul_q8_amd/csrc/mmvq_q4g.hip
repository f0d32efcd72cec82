// Matvec of 4-bit weights with group scales and Q8_1 activations.
//
//   y[t][m] = sum_b s[m][g(b)] * d[t][b] * (sum_i q_i a_i - z[m][g(b)] * S[t][b])
//
// over the 32-value blocks b of the row, with the block's integer sum S as
// stored in Q8_1: integer dot products, one fp32 rounding of the scales'
// product and one fma per block.
//
// A workgroup copies the T activation rows to LDS once, the bytes of every
// eight values split into the four with even and the four with odd index, so
// that the low and high halves of a weight dword meet them without further
// shuffling.  Its waves take tiles of 64/L * R weight rows: L lanes share a
// row, a lane multiplies one 32-value block (16 weight bytes) at a time, and R
// rows per lane use the activations it read from LDS.  Two batches of two
// rounds stay in flight per wave, across the ends of its tiles: 64 KB per CU
// with 16 waves.  With few rows `split` waves share a tile by parts of K.
//
// Bound by HBM at one token, 28672 x 8192, groups of 32: 24 us, 5.5 TB/s (a
// copy of 1 GiB reaches 5.1); 4096 x 11008, groups of 128 with zero points: 6.9
// us, 3.4 TB/s (the start and the end of a launch that short; mmvq_q4k reads a
// tenth more in 6.2).  28672 x 8192 takes 25, 28, 34 and 48 us at 2, 3, 5 and 8
// tokens; 57, 74, 108 and 156 VALU instructions per 2048 weights (all of the
// kernel's, counted) are 12, 15, 22 and 32 us of them.  The weights are read
// past the caches' usual order: 26.7 us otherwise at one token, where they do
// not fit the last-level cache (32000 x 4096, which does three times: 13.5 us,
// and 14.4 this way).
//
// Measured and not kept: the products on the matrix cores (16 x 16 x 64 with
// four blocks kept apart by zeros, or 4 x 4 x 4 with the weights transposed
// within quads of lanes) - 33 us from 1 to 4 tokens and 44 at 8, but slower
// than this at one to five tokens and at 4096 rows; four rounds in a batch
// (7.8 -> 9.5 us at 4096 x 11008).
#include "typed.hpp"

#include <algorithm>
#include <type_traits>

namespace qmm {

struct Q4gArgs {
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;
  const uint8_t* xq;
  float* y;
  int64_t M, tiles;
  int nblk, seg, group_blk, groups, scale_type, split;
  uint32_t magic;  // ceil(2^32 / group_blk); unused where group_blk is 1
};

constexpr uint32_t kEvenBytes = 0x06040200u, kOddBytes = 0x07050301u;

// Sum over each row of 16 lanes, in all of its lanes.
__device__ __forceinline__ float row_sum(float v) {
  v = dpp_add<0x128>(v);  // row_ror:8
  v = dpp_add<0x124>(v);
  v = dpp_add<0x122>(v);
  return dpp_add<0x121>(v);
}

// Two values summed over pairs of lane halves (or of 16-lane rows) in one
// register: lanes of the lower half (even rows) get a's sums, the others b's.
__device__ __forceinline__ float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b),
                                                  false, false);
  const unsigned x = r[0], y = r[1];  // a bit cast of a vector's element would read the vector's first
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b),
                                                  false, false);
  const unsigned x = r[0], y = r[1];  // a bit cast of a vector's element would read the vector's first
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// A copy of `per` pieces for each of T tokens by the workgroup's threads, N
// pieces of a thread in flight at once.
template <int T, int N>
struct Pieces {
  int per, all, step, lane, beg;
  uint2 v[N];

  __device__ __forceinline__ explicit Pieces(int n)
      : per(n), all(n * T), step(blockDim.x), lane(threadIdx.x & 63),
        beg(__builtin_amdgcn_readfirstlane(threadIdx.x & ~63)) {}
  __device__ __forceinline__ int place(int i, int& t) const {
    t = 0;
#pragma unroll
    for (int k = 1; k < T; ++k) t += i >= k * per ? 1 : 0;
    return i - t * per;
  }
  // fn(token, index in the token) of round i0 (uniform over the wave)
  template <class Fn>
  __device__ __forceinline__ void load(int i0, Fn fn) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (i0 + u * step < all) {
        int t;
        const int j = place(min(i0 + u * step + lane, all - 1), t);
        v[u] = fn(t, j);
      }
    }
  }
  template <class Fn>
  __device__ __forceinline__ void store(int i0, Fn fn) const {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = i0 + u * step + lane;
      if (i < all) {
        int t;
        const int j = place(i, t);
        fn(t, j, v[u]);
      }
    }
  }
};

// LDS for the activations of `seg` blocks: up to four tokens share a record per
// block, 32 bytes of values each, then (fp32 d, int32 S) each, so that one
// address and constant offsets reach all of it.  The records' sizes (padded at
// one and three tokens) let consecutive lanes read 16 bytes each without bank
// conflicts.
template <int T>
struct Layout {
  static constexpr int tokens(int g) { return T - 4 * g < 4 ? T - 4 * g : 4; }
  static constexpr int record(int g) {
    return tokens(g) == 1 ? 48 : tokens(g) == 2 ? 80 : tokens(g) == 3 ? 144 : 160;
  }
  static constexpr int kGroups = (T + 3) / 4;
  static constexpr int kBlock = T > 4 ? 160 + record(1) : record(0);  // bytes of a block in all
};

// The activations of blocks [b0, b0 + n) of T tokens in LDS.  between() runs
// after the first loads are issued and before their results are awaited:
// loads of its own come back after these.
template <int T, class Fn>
__device__ __forceinline__ void stage(const Q4gArgs& a, int b0, int n, uint8_t* lds, Fn between) {
  using Lay = Layout<T>;
  // eight values
  const auto get = [&](int t, int j) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(
        a.xq + static_cast<uint32_t>((t * a.nblk + b0 + (j >> 2)) * kQ8Bytes + 4 + 8 * (j & 3)));
    return make_uint2(q[0], q[1]);
  };
  // token t's place in block b's record
  const auto place = [&](int t, int b, int of_values, int of_factors) {
    if (T > 4 && t >= 4) return lds + a.seg * 160 + b * Lay::record(Lay::kGroups - 1) + (t - 4) * of_values +
                                (of_factors ? 32 * Lay::tokens(Lay::kGroups - 1) : 0);
    return lds + b * Lay::record(0) + t * of_values + (of_factors ? 32 * Lay::tokens(0) : 0);
  };
  const auto put = [&](int t, int j, uint2 q) {
    *reinterpret_cast<uint2*>(place(t, j >> 2, 32, 0) + 8 * (j & 3)) =
        make_uint2(__builtin_amdgcn_perm(q.y, q.x, kEvenBytes), __builtin_amdgcn_perm(q.y, q.x, kOddBytes));
  };
  // a block's scale and sum
  const auto get_ds = [&](int t, int j) {
    const uint32_t* x =
        reinterpret_cast<const uint32_t*>(a.xq + static_cast<uint32_t>((t * a.nblk + b0 + j) * kQ8Bytes));
    return make_uint2(x[0], x[9]);
  };
  const auto put_ds = [&](int t, int j, uint2 q) {
    *reinterpret_cast<uint2*>(place(t, j, 8, 1)) = make_uint2(__builtin_bit_cast(uint32_t, h2f(q.x & 0xffffu)), q.y);
  };
  constexpr int N = T > 1 ? 8 : 2;
  Pieces<T, N> x(n * 4);
  Pieces<T, (N + 3) / 4> ds(n);
  x.load(x.beg, get);
  ds.load(ds.beg, get_ds);
  between();
  x.store(x.beg, put);
  ds.store(ds.beg, put_ds);
  for (int i0 = x.beg + N * x.step; i0 < x.all; i0 += N * x.step) {
    x.load(i0, get);
    x.store(i0, put);
  }
  for (int i0 = ds.beg + (N + 3) / 4 * ds.step; i0 < ds.all; i0 += (N + 3) / 4 * ds.step) {
    ds.load(i0, get_ds);
    ds.store(i0, put_ds);
  }
}

template <int U, int R>
struct Batch {
  uint4 w[U][R];
  uint32_t s[U][R], z[U][R];
};

// All of the workgroup's LDS writes done and visible to it.  Loads from global
// memory stay in flight (a __syncthreads waits for them).
__device__ __forceinline__ void lds_barrier() { __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int T, int L, int R, bool ZEROS>
__global__ __launch_bounds__(1024) void mmvq_q4g_kernel(Q4gArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  using Lay = Layout<T>;
  constexpr int U = 2, kSub = 64 / L, kRows = kSub * R;
  const int lane = threadIdx.x & 63, li = lane % L, sub = lane / L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  // tiles [first, last) belong to the workgroup
  const int64_t first = a.tiles * blockIdx.x / gridDim.x, last = a.tiles * (blockIdx.x + 1) / gridDim.x;
  // `split` waves share a tile, each with a part of the row's rounds; such a workgroup has one tile per set of waves
  const int part = wave % a.split, slot = wave / a.split, slots = waves / a.split;
  const int zrow = (a.groups + 1) / 2;
  float acc[R * T] = {};

  // sums over the row's lanes to put(token, row of the tile, sum); the accumulators are cleared
  const auto finish = [&](auto put) {
    if constexpr (L == 64) {
      // four values end in one register: value i + {0, 2, 1, 3} in lane rows 0..3
      const int row = lane >> 4, which = (row & 1) * 2 + (row >> 1);
#pragma unroll
      for (int i = 0; i < R * T; i += 4) {
        const float v1 = i + 1 < R * T ? acc[i + 1] : 0.0f, v2 = i + 2 < R * T ? acc[i + 2] : 0.0f,
                    v3 = i + 3 < R * T ? acc[i + 3] : 0.0f;
        const float v = row_sum(fold16(fold32(acc[i], v1), fold32(v2, v3)));
        const int k = i + which;
        if ((lane & 15) == 0 && k < R * T) put(k % T, k / T, v);
      }
    } else {
#pragma unroll
      for (int k = 0; k < R * T; ++k) {
        const float v = row_sum(acc[k]);
        if (li == 0) put(k % T, (k / T) * kSub + sub, v);
      }
    }
#pragma unroll
    for (int k = 0; k < R * T; ++k) acc[k] = 0.0f;
  };

  for (int s0 = 0; s0 < a.nblk; s0 += a.seg) {
    const int n = min(a.seg, a.nblk - s0), rounds = (n + L - 1) / L;
    const int beg = rounds * part / a.split, its = rounds * (part + 1) / a.split;
    if (s0) __syncthreads();

    const auto load = [&](Batch<U, R>& B, int64_t tile, int it0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = s0 + min((it0 + u) * L + li, n - 1);
        const int g = a.group_blk == 1 ? b : static_cast<int>(__umulhi(static_cast<uint32_t>(b), a.magic));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          // with L = 64 the row is the wave's: its addresses are scalar, the lane's part a 32-bit offset
          const int64_t m = min(tile * kRows + r * kSub + (L == 64 ? 0 : sub), a.M - 1);
          const uint8_t* row = a.w + m * a.nblk * 16;
          const uint8_t* scales = static_cast<const uint8_t*>(a.scales) + m * a.groups * 2;
          B.w[u][r] = ld16_nt(row + static_cast<uint32_t>(b * 16));
          B.s[u][r] = *reinterpret_cast<const uint16_t*>(scales + static_cast<uint32_t>(g * 2));
          if constexpr (ZEROS)
            B.z[u][r] = static_cast<uint32_t>(a.zeros[m * zrow + static_cast<uint32_t>(g >> 1)]) >> (4 * (g & 1));
          else
            B.z[u][r] = 8u;
        }
      }
    };
    const auto multiply = [&](const Batch<U, R>& B, int it0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (it0 + u < its) {
          const int j = (it0 + u) * L + li, k = min(j, n - 1);
          float s[R];
          int z[R];
          uint32_t lo[R][4], hi[R][4];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float v = a.scale_type == QMM_F16 ? h2f(B.s[u][r]) : __builtin_bit_cast(float, B.s[u][r] << 16);
            s[r] = j < n ? v : 0.0f;
            z[r] = -static_cast<int>(B.z[u][r] & 15u);
            const uint32_t w[4] = {B.w[u][r].x, B.w[u][r].y, B.w[u][r].z, B.w[u][r].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              lo[r][i] = w[i] & 0x0f0f0f0fu;
              hi[r][i] = (w[i] >> 4) & 0x0f0f0f0fu;
            }
          }
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const int g = t / 4, i = t % 4;
            const uint8_t* at = lds + (g ? a.seg * 160 : 0) + k * Lay::record(g);
            const uint4 p = *reinterpret_cast<const uint4*>(at + 32 * i);
            const uint4 q = *reinterpret_cast<const uint4*>(at + 32 * i + 16);
            const uint2 ds = *reinterpret_cast<const uint2*>(at + 32 * Lay::tokens(g) + 8 * i);
            const float d = __builtin_bit_cast(float, ds.x);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              int dot = __mul24(z[r], static_cast<int>(ds.y));
              dot = dot4(lo[r][0], p.x, dot);
              dot = dot4(hi[r][0], p.y, dot);
              dot = dot4(lo[r][1], p.z, dot);
              dot = dot4(hi[r][1], p.w, dot);
              dot = dot4(lo[r][2], q.x, dot);
              dot = dot4(hi[r][2], q.y, dot);
              dot = dot4(lo[r][3], q.z, dot);
              dot = dot4(hi[r][3], q.w, dot);
              acc[r * T + t] = __builtin_fmaf(s[r] * d, static_cast<float>(dot), acc[r * T + t]);
            }
          }
        }
      }
    };
    // Batches of U rounds, two in flight: after a batch is multiplied its registers take the one after the next.  The
    // paths with and without further loads do not join again: a wait behind such a join is one for all loads.
    int64_t tile = beg < its ? first + slot : last, tile2 = tile;
    int it = beg, it2 = beg;
    const auto fetch = [&](Batch<U, R>& B) {
      // where there is no second batch its loads all go to one block
      const bool more = tile2 < last;
      load(B, more ? tile2 : last - 1, more ? it2 : rounds);
      it2 += U;
      if (it2 >= its) {
        it2 = beg;
        tile2 += slots;
      }
    };
    Batch<U, R> A, B;
    stage<T>(a, s0, n, lds, [&] {
      fetch(A);
      fetch(B);
    });
    lds_barrier();
    const auto consume = [&](const Batch<U, R>& now) {
      multiply(now, it);
      it += U;
      if (it >= its) {
        if (a.split == 1 && s0 + n == a.nblk) {
          finish([&](int k, int row, float v) {
            const int64_t m = tile * kRows + row;
            if (m < a.M) a.y[k * a.M + m] = v;
          });
        }
        it = beg;
        tile += slots;
      }
    };
    while (tile < last) {
      consume(A);
      if (tile2 >= last) {
        if (tile < last) consume(B);
        break;
      }
      fetch(A);
      consume(B);
      if (tile2 >= last) {
        if (tile < last) consume(A);
        break;
      }
      fetch(B);
    }
  }
  if (a.split > 1) {
    // the parts of each tile, added in their order
    float* parts = reinterpret_cast<float*>(lds + static_cast<size_t>(a.seg) * Lay::kBlock);
    finish([&](int k, int row, float v) { parts[(wave * T + k) * kRows + row] = v; });
    __syncthreads();
    for (int i = threadIdx.x; i < slots * T * kRows; i += blockDim.x) {
      const int w = i / (T * kRows), k = i / kRows % T, row = i % kRows;
      const int64_t tile = first + w, m = tile * kRows + row;
      float v = 0.0f;
      for (int p = 0; p < a.split; ++p) v += parts[((w * a.split + p) * T + k) * kRows + row];
      if (tile < last && m < a.M) a.y[k * a.M + m] = v;
    }
  }
}

template <int T>
static void launch(const Q4gArgs& args, int64_t M, hipStream_t st) {
  Q4gArgs a = args;
  constexpr int kLds = 160 * 1024, kParts = 16 * T * 8 * 4;
  const int cus = device_cu_count();
  // lanes per row: 64, or 16 where 64 would leave an eighth or more of them idle in the row's last round (1003 x 2272:
  // 3.4 us with 16, 4.6 with 64; 11008 x 4096: 8.1 and 6.9)
  const bool wide = ((a.nblk + 63) / 64) * 64 * 8 < a.nblk * 9;
  const int rows1 = wide ? 1 : 4;
  // two rows per lane where that still leaves every CU 16 waves' tiles (28672 x 8192: 42 us with one and 37 with two at
  // five tokens, 31 and 30 at two)
  const int R = T > 1 && M >= static_cast<int64_t>(cus) * 16 * rows1 * 2 ? 2 : 1;
  a.tiles = (M + rows1 * R - 1) / (rows1 * R);
  const int rounds = (a.nblk + (wide ? 63 : 15)) / (wide ? 64 : 16);
  // waves that share a tile: as many as leave a CU 16 waves, with a round each at least (512 x 14336, one token: 6.2 us
  // unsplit, 4.5 in eight parts; eight tokens 34 and 14, for the activations' copy has more threads too)
  a.split = 1;
  while (a.split < 16 && a.split * 2 <= rounds && a.tiles * a.split * 2 <= static_cast<int64_t>(cus) * 16) a.split *= 2;
  a.seg = std::min<int64_t>(a.nblk, (kLds - (a.split > 1 ? kParts : 0)) / Layout<T>::kBlock);
  const int waves = a.split * static_cast<int>(std::clamp<int64_t>(a.tiles / cus, 1, 16 / a.split));
  int64_t grid = (a.tiles + waves / a.split - 1) / (waves / a.split);
  // the activations are copied once per CU where they fit; in segments, and in parts, a wave has one tile
  if (a.seg == a.nblk && a.split == 1) grid = std::min<int64_t>(grid, cus);
  const dim3 g(static_cast<unsigned>(grid)), b(waves * 64);
  const size_t lds = static_cast<size_t>(a.seg) * Layout<T>::kBlock + (a.split > 1 ? kParts : 0);
  const auto go = [&](auto zeros) {
    constexpr bool Z = decltype(zeros)::value;
    constexpr int R2 = T > 1 ? 2 : 1;
    if (wide) {
      if (R == 2) hipLaunchKernelGGL((mmvq_q4g_kernel<T, 64, R2, Z>), g, b, lds, st, a);
      else hipLaunchKernelGGL((mmvq_q4g_kernel<T, 64, 1, Z>), g, b, lds, st, a);
    } else {
      if (R == 2) hipLaunchKernelGGL((mmvq_q4g_kernel<T, 16, R2, Z>), g, b, lds, st, a);
      else hipLaunchKernelGGL((mmvq_q4g_kernel<T, 16, 1, Z>), g, b, lds, st, a);
    }
  };
  if (a.zeros) go(std::true_type{});
  else go(std::false_type{});
}

}  // namespace qmm

using namespace qmm;

extern "C" int mmvq_q4g(const void* w, const void* scales, int scale_type, const void* zeros, const void* xq, float* y,
                        int64_t M, int64_t K, int64_t group, int64_t T, void* stream) {
  if (scale_type != QMM_F16 && scale_type != QMM_BF16) return QMM_ERR_UNSUPPORTED;
  if (M < 1 || M > (int64_t{1} << 26) || K < kQB || (K % kQB) != 0 || K > (int64_t{1} << 20) || group < kQB ||
      (group % kQB) != 0 || (K % group) != 0 || T < 1 || T > QMM_MMVQ_MAX_T)
    return QMM_ERR_SHAPE;
  if (!w || !scales || !xq || !y) return QMM_ERR_NULL;
  if (!aligned16(w) || !aligned16(scales) || !aligned16(zeros) || !aligned16(xq) || !aligned16(y))
    return QMM_ERR_ALIGN;
  const uint64_t gb = static_cast<uint64_t>(group / kQB);
  const Q4gArgs a{static_cast<const uint8_t*>(w), scales, static_cast<const uint8_t*>(zeros),
                  static_cast<const uint8_t*>(xq), y, M, 0, static_cast<int>(K / kQB), 0, static_cast<int>(gb),
                  static_cast<int>(K / group), scale_type, 1,
                  // exact for block numbers below 2^15: the error of b * magic is under b * group_blk < 2^32
                  static_cast<uint32_t>(((uint64_t{1} << 32) + gb - 1) / gb)};
  hipStream_t st = to_stream(stream);
  switch (T) {
    case 1: launch<1>(a, M, st); break;
    case 2: launch<2>(a, M, st); break;
    case 3: launch<3>(a, M, st); break;
    case 4: launch<4>(a, M, st); break;
    case 5: launch<5>(a, M, st); break;
    case 6: launch<6>(a, M, st); break;
    case 7: launch<7>(a, M, st); break;
    default: launch<8>(a, M, st); break;
  }
  return launch_status();
}
