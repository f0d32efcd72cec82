// Keys and values into the paged 4-bit cache, and back.
//
// Eight consecutive values of a head per lane, four lanes per block of 32, a
// head's row in D/8 lanes (rounded up to a power of two).  The key half of a
// row and its value half are the same lanes' work.
//
// A wave's rows are tokens next to each other in the list, and so are the four
// waves' of a workgroup, which goes over some heads of theirs: a cell's lines,
// of which a token has a few bytes each, are then read and written by one CU
// while they are in its caches.
//
// Reading is bound by HBM: 65536 x 8 x 128 to bf16, 353 MB: 60 us, 5.9 TB/s (with
// stores through the caches 91; with loads past them, which several lanes' share
// of a line forbids, 95).  So is appending from some ten thousand tokens on: 32768
// x 8 x 128, 176 MB, turned: 38 us, as they are 32; at 8192, 44 MB, 14.2 and 11.7,
// of which 5 are the launch and the first loads (slot, position, table, values).
// Its instructions, 20 a value, take 10 of the 14.2 and overlap.
#include "kv_q4.hpp"

#include <algorithm>

namespace qmm {

struct AppendArgs {
  const void* x[2];  // k, v
  int64_t stride[2];
  const float* rope;
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* cache;
  int64_t P, pages, page, T;
  int Hk, D, rot, row_lanes, heads, shift;  // heads of a workgroup
  bool interleaved;
};

// What a workgroup and lane work on: a token, a range of heads, and the lane's eight values.
struct Work {
  int64_t t;
  int h0, h1, j;
  __device__ __forceinline__ Work(int row_lanes, int heads, int Hk) {
    const int lane = threadIdx.x & 63, segs = (Hk + heads - 1) / heads;
    const uint32_t block = blockIdx.x / static_cast<uint32_t>(segs);
    t = static_cast<int64_t>(block) * (256 / row_lanes) + threadIdx.x / row_lanes;
    h0 = static_cast<int>(blockIdx.x - block * segs) * heads;
    h1 = min(Hk, h0 + heads);
    j = lane % row_lanes;
  }
};

// Eight of a block's values, by a quad of lanes.
struct Block8 {
  float v[8], d, m, inv;
  uint32_t dm;  // d and m as f16 bits

  // d, m and 1/d.  Quotients are the IEEE ones: with a correctly rounded
  // reciprocal of the divisor one step from the remainder rounds correctly
  // (Markstein), and so does one step of the reciprocal itself for a divisor of
  // eleven bits.
  __device__ __forceinline__ void scales() {
#pragma clang fp contract(off)
    float lo = v[0], hi = v[0], any = v[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      lo = fminf(lo, v[j]);
      hi = fmaxf(hi, v[j]);
      any += v[j];
    }
    // what is not a number or beyond the range (or sums to either) goes the long way
    if (__builtin_amdgcn_ballot_w64(!(fabsf(any) <= 32768.0f * 8.0f) || lo < -32768.0f || hi > 32768.0f)) {
      lo = INFINITY, hi = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = v[j] == v[j] ? fminf(fmaxf(v[j], -32768.0f), 32768.0f) : 0.0f;
        lo = fminf(lo, v[j]);
        hi = fmaxf(hi, v[j]);
      }
    }
    lo = fminf(lo, lane8_xchg<0xb1>(lo));
    lo = fminf(lo, lane8_xchg<0x4e>(lo)) + 0.0f;  // no minus zero
    hi = fmaxf(hi, lane8_xchg<0xb1>(hi));
    hi = fmaxf(hi, lane8_xchg<0x4e>(hi));
    constexpr float kFifteenth = 1.0f / 15.0f;
    const float span = hi - lo, q = span * kFifteenth;
    float steps = __builtin_fmaf(__builtin_fmaf(-15.0f, q, span), kFifteenth, q);
    __asm__("" : "+v"(steps));  // rounded to fp32 before f16: not one instruction that rounds once
    const uint32_t db = f2h_bits(steps), mb = f2h_bits(lo);
    d = h2f(db), m = h2f(mb);
    const float r = __builtin_amdgcn_rcpf(d);
    inv = d > 0.0f ? __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r) : 0.0f;
    dm = db | mb << 16;
  }

  // Code j into a byte of a dword: the conversion rounds to the nearest even and takes what is below 0 as that.
  __device__ __forceinline__ uint32_t code(int j, int byte, uint32_t word) const {
#pragma clang fp contract(off)
    const float p = (v[j] - m) * inv;
    return __builtin_amdgcn_cvt_pk_u8_f32(fminf(p, 15.0f), byte, word);
  }
};

template <int KT, int VT>
__global__ __launch_bounds__(256) void kv_append_q4_kernel(AppendArgs a) {
#pragma clang fp contract(off)
  const Work w(a.row_lanes, a.heads, a.Hk);
  const int lane = threadIdx.x & 63, j = w.j;
  const int64_t t = min(w.t, a.T - 1), slot = a.slots[t];
  const bool on = w.t < a.T && slot >= 0 && slot < a.pages * a.page && j < a.D / 8, turned = j < a.rot / 8;
  const int half = a.rot / 16, nb = a.D / 32, b = j >> 2, part = j & 3;
  const int tok = static_cast<int>(slot) & (kCellTokens - 1);
  const int64_t cell0 = on ? kv_cell(slot, a.page, a.shift, 0, a.Hk, a.D) : 0, head_bytes = a.page / kCellTokens * (20 * a.D);
  float cos[8], sin[8];
  if (turned) {
    const int64_t row = max(int64_t{0}, min(a.P - 1, static_cast<int64_t>(a.positions[t]))) * a.rot;
    if (a.interleaved) {
      const float4 c = load4(QMM_F32, a.rope, row / 4 + j), s = load4(QMM_F32, a.rope, (row + a.rot / 2) / 4 + j);
      cos[0] = c.x, cos[1] = c.y, cos[2] = c.z, cos[3] = c.w;
      sin[0] = s.x, sin[1] = s.y, sin[2] = s.z, sin[3] = s.w;
    } else {
      const int k = j < half ? j : j - half;
      load8(QMM_F32, a.rope, row / 8 + k, cos);
      load8(QMM_F32, a.rope, (row + a.rot / 2) / 8 + k, sin);
      if (j < half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sin[i] = -sin[i];  // of the other value of the pair
      }
    }
  }
  Raw8<KT> key, next_key;
  Raw8<VT> val, next_val;
  const auto load = [&](int h) {
    if (!on || h >= w.h1) return;
    next_key.load(a.x[0], (t * a.stride[0] + static_cast<int64_t>(h) * a.D) / 8 + j);
    next_val.load(a.x[1], (t * a.stride[1] + static_cast<int64_t>(h) * a.D) / 8 + j);
  };
  load(w.h0);
  for (int h = w.h0; h < w.h1; ++h) {
    key = next_key, val = next_val;
    load(h + 1);
    Block8 k, v;
#pragma unroll
    for (int i = 0; i < 8; ++i) k.v[i] = on ? key.get(i) : 0.0f, v.v[i] = on ? val.get(i) : 0.0f;
    if (a.rot > 0) {
      if (a.interleaved) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = k.v[2 * i], q = k.v[2 * i + 1];
            k.v[2 * i] = p * cos[i] - q * sin[i];
            k.v[2 * i + 1] = q * cos[i] + p * sin[i];
          }
        }
      } else {
        const int from = turned ? (j < half ? lane + half : lane - half) : lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl(k.v[i], from);
          if (turned) k.v[i] = k.v[i] * cos[i] + o * sin[i];
        }
      }
    }
    k.scales();
    v.scales();
    // The key's codes 0, 2, 4, 6, 1, 3, 5, 7 from the low end on.  The value's 0 to 3 and 4 to 7 as bytes: a byte of the
    // cache joins dims c and c + 16 of a block, so this lane's and those of the lane two further, half of them each.
    uint32_t k0415 = 0, k2637 = 0, v03 = 0, v47 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k0415 = k.code(4 * (i & 1) + (i >> 1), i, k0415), k2637 = k.code(4 * (i & 1) + (i >> 1) + 2, i, k2637);
      v03 = v.code(i, i, v03), v47 = v.code(4 + i, i, v47);
    }
    const uint32_t kc = k0415 | k2637 << 4;
    const uint32_t other = static_cast<uint32_t>(lane8_xchg<0x4e>(static_cast<int>(part < 2 ? v47 : v03)));
    const uint32_t vc = part < 2 ? v03 | other << 4 : other | v47 << 4;
    if (!on) continue;
    uint8_t* cell = a.cache + cell0 + h * head_bytes;
    *reinterpret_cast<uint32_t*>(cell + (b * kCellTokens + tok) * 16 + part * 4) = kc;
    const int quad = tok >> 2, c0 = (part & 1) * 8 + (part >> 1) * 4;
    uint8_t* to = cell + 10 * a.D + ((quad * 16 + c0) * nb + b) * 4 + kv_quad_byte(tok & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i * nb * 4] = static_cast<uint8_t>(vc >> (8 * i));
    if (part == 0) {
      *reinterpret_cast<uint32_t*>(cell + 8 * a.D + (b * kCellTokens + tok) * 4) = k.dm;
      uint16_t* vs = reinterpret_cast<uint16_t*>(cell + 18 * a.D + (quad * nb + b) * 16) + (tok & 3);
      vs[0] = static_cast<uint16_t>(v.dm);
      vs[4] = static_cast<uint16_t>(v.dm >> 16);
    }
  }
}

struct ReadArgs {
  const uint8_t* cache;
  const int64_t* slots;
  void* y[2];
  int64_t pages, page, T;
  int Hk, D, row_lanes, heads, shift;
  bool large;
};


// Eight f16 numbers as values of a type.  `large`: stored past the caches.
template <int TY>
__device__ __forceinline__ void store_f16(void* p, int64_t i, const h2 (&x)[4], bool large) {
  Raw8<TY> o;
  if constexpr (TY == QMM_F16) {
    o.v[0] = make_uint4(__builtin_bit_cast(uint32_t, x[0]), __builtin_bit_cast(uint32_t, x[1]),
                        __builtin_bit_cast(uint32_t, x[2]), __builtin_bit_cast(uint32_t, x[3]));
  } else {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = static_cast<float>(x[k >> 1][k & 1]);
    o.set(f);
  }
  if (large) o.store_nt(p, i);
  else o.store(p, i);
}

template <int TY>
__global__ __launch_bounds__(256) void kv_read_q4_kernel(ReadArgs a) {
  const Work w(a.row_lanes, a.heads, a.Hk);
  const int j = w.j;
  const int64_t t = min(w.t, a.T - 1), slot = a.slots[t];
  const bool on = w.t < a.T && j < a.D / 8, there = on && slot >= 0 && slot < a.pages * a.page;
  const int nb = a.D / 32, b = j >> 2, part = j & 3, tok = static_cast<int>(slot) & (kCellTokens - 1), quad = tok >> 2;
  const int c0 = (part & 1) * 8 + (part >> 1) * 4;
  const int64_t cell0 = there ? kv_cell(slot, a.page, a.shift, 0, a.Hk, a.D) : 0;
  const int64_t head_bytes = a.page / kCellTokens * (20 * a.D);
  struct Raw {
    uint32_t kw = 0, kd = 0, v[4] = {0, 0, 0, 0}, d = 0, m = 0;
  } next;
  const auto load = [&](int h) {
    if (!there || h >= w.h1) return;
    const uint8_t* cell = a.cache + cell0 + h * head_bytes;
    next.kw = *reinterpret_cast<const uint32_t*>(cell + (b * kCellTokens + tok) * 16 + part * 4);
    next.kd = *reinterpret_cast<const uint32_t*>(cell + 8 * a.D + (b * kCellTokens + tok) * 4);
    const uint8_t* from = cell + 10 * a.D + ((quad * 16 + c0) * nb + b) * 4 + kv_quad_byte(tok & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) next.v[i] = from[i * nb * 4];
    const uint8_t* vs = cell + 18 * a.D + (quad * nb + b) * 16 + (tok & 3) * 2;
    next.d = ld_u16(vs), next.m = ld_u16(vs + 8);
  };
  load(w.h0);
  for (int h = w.h0; h < w.h1; ++h) {
    const Raw now = next;
    load(h + 1);
    const uint32_t kw = now.kw, kd = now.kd, d = now.d, m = now.m;
    const uint32_t vw = now.v[0] | now.v[1] << 8 | now.v[2] << 16 | now.v[3] << 24;
    // bytes of dims c and c + 16: this lane keeps its own dims' codes and takes the rest from the lane two further
    const uint32_t low = vw & 0x0f0f0f0fu, high = (vw >> 4) & 0x0f0f0f0fu;
    const uint32_t other = static_cast<uint32_t>(lane8_xchg<0x4e>(static_cast<int>(part < 2 ? high : low)));
    if (!on) continue;
    const uint32_t v03 = part < 2 ? low : other, v47 = part < 2 ? other : high;
    // bytes of kw: codes 0 and 2, 4 and 6, 1 and 3, 5 and 7
    const uint32_t k0415 = kw & 0x0f0f0f0fu, k2637 = (kw >> 4) & 0x0f0f0f0fu;
    const uint32_t k0123 = __builtin_amdgcn_perm(k2637, k0415, 0x06040200u), k4567 = __builtin_amdgcn_perm(k2637, k0415, 0x07050301u);
    const auto values = [](uint32_t a03, uint32_t a47, uint32_t d16, uint32_t m16, h2 (&x)[4]) {
      const h2 dd = as_h2(d16 | d16 << 16), mm = as_h2(m16 | m16 << 16);
      x[0] = __builtin_elementwise_fma(codes_to_f16<false>(a03), dd, mm);
      x[1] = __builtin_elementwise_fma(codes_to_f16<true>(a03), dd, mm);
      x[2] = __builtin_elementwise_fma(codes_to_f16<false>(a47), dd, mm);
      x[3] = __builtin_elementwise_fma(codes_to_f16<true>(a47), dd, mm);
    };
    const int64_t at = (t * a.Hk + h) * (a.D / 8) + j;
    h2 x[4];
    values(k0123, k4567, kd & 0xffffu, kd >> 16, x);
    store_f16<TY>(a.y[0], at, x, a.large);
    values(v03, v47, d, m, x);
    store_f16<TY>(a.y[1], at, x, a.large);
  }
}

template <int KT>
static void launch_append(const AppendArgs& a, int v_type, dim3 g, hipStream_t st) {
  if (v_type == QMM_F32) hipLaunchKernelGGL((kv_append_q4_kernel<KT, QMM_F32>), g, dim3(256), 0, st, a);
  else if (v_type == QMM_F16) hipLaunchKernelGGL((kv_append_q4_kernel<KT, QMM_F16>), g, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((kv_append_q4_kernel<KT, QMM_BF16>), g, dim3(256), 0, st, a);
}

// Workgroups, and the heads of each: all of a token's where there are tokens enough for 1024 workgroups, else fewer.
// 8192 x 8 x 128 appended and read back: 24.5 us, with 512 workgroups 28, with 2048 27.
static dim3 kv_grid(int64_t T, int64_t Hk, int lanes, int& heads) {
  const int64_t blocks = (T + 256 / lanes - 1) / (256 / lanes);
  heads = static_cast<int>(std::max<int64_t>(1, std::min(Hk, blocks * Hk / 1024)));
  return dim3(static_cast<unsigned>(blocks * ((Hk + heads - 1) / heads)));
}

static int row_lanes_of(int64_t D) { return D == 64 ? 8 : D <= 128 ? 16 : 32; }

}  // namespace qmm

using namespace qmm;

extern "C" int kv_append_q4(const void* k, int64_t k_stride, int k_type, const void* v, int64_t v_stride, int v_type,
                            const float* rope, int64_t P, int64_t rot, int interleaved, const int32_t* positions,
                            const int64_t* slots, void* cache, int64_t pages, int64_t page, int64_t T, int64_t Hk,
                            int64_t D, void* stream) {
  if (!known_type(k_type) || !known_type(v_type)) return QMM_ERR_UNSUPPORTED;
  if (!kv_q4_shape(pages, page, Hk, D) || T < 0 || T >= kMostRows || T > 0x7fffffff / Hk) return QMM_ERR_SHAPE;
  if (!strided_rows(k_stride, Hk, D) || !strided_rows(v_stride, Hk, D)) return QMM_ERR_SHAPE;
  if (rot < 0 || rot % 16 != 0 || rot > D || (rot > 0 && (P < 1 || P > 0x7fffffff))) return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!k || !v || !slots || !cache || (rot > 0 && (!rope || !positions))) return QMM_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned_list(slots, 8) || !aligned16(cache) || !aligned16(rope) ||
      !aligned_list(positions, 4))
    return QMM_ERR_ALIGN;
  const int lanes = row_lanes_of(D);
  int heads;
  const dim3 g = kv_grid(T, Hk, lanes, heads);
  const AppendArgs a{{k, v}, {k_stride, v_stride}, rope, positions, slots, static_cast<uint8_t*>(cache), P, pages, page,
                     T, static_cast<int>(Hk), static_cast<int>(D), static_cast<int>(rot), lanes, heads, page_shift(page),
                     interleaved != 0};
  hipStream_t st = to_stream(stream);
  if (k_type == QMM_F32) launch_append<QMM_F32>(a, v_type, g, st);
  else if (k_type == QMM_F16) launch_append<QMM_F16>(a, v_type, g, st);
  else launch_append<QMM_BF16>(a, v_type, g, st);
  return launch_status();
}

extern "C" int kv_read_q4(const void* cache, int64_t pages, int64_t page, const int64_t* slots, void* k, void* v,
                          int type, int64_t T, int64_t Hk, int64_t D, void* stream) {
  if (!known_type(type)) return QMM_ERR_UNSUPPORTED;
  if (!kv_q4_shape(pages, page, Hk, D) || T < 0 || T >= kMostRows || T > 0x7fffffff / Hk) return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!cache || !slots || !k || !v) return QMM_ERR_NULL;
  if (!aligned16(cache) || !aligned_list(slots, 8) || !aligned16(k) || !aligned16(v)) return QMM_ERR_ALIGN;
  const int lanes = row_lanes_of(D);
  int heads;
  const dim3 g = kv_grid(T, Hk, lanes, heads), blk(256);
  const ReadArgs a{static_cast<const uint8_t*>(cache), slots, {k, v}, pages, page, T, static_cast<int>(Hk),
                   static_cast<int>(D), lanes, heads, page_shift(page), large_output(2 * T * Hk * D, type)};
  hipStream_t st = to_stream(stream);
  if (type == QMM_F32) hipLaunchKernelGGL(kv_read_q4_kernel<QMM_F32>, g, blk, 0, st, a);
  else if (type == QMM_F16) hipLaunchKernelGGL(kv_read_q4_kernel<QMM_F16>, g, blk, 0, st, a);
  else hipLaunchKernelGGL(kv_read_q4_kernel<QMM_BF16>, g, blk, 0, st, a);
  return launch_status();
}
