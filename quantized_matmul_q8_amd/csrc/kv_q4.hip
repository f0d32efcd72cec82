// Keys and values into the paged 4-bit cache, and back.
//
// Eight consecutive values of a head per lane, four lanes per block of 32, a
// head's row in D/8 lanes (rounded up to a power of two).  The key half of a
// row and its value half are the same lanes' work.
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
  int Hk, D, rot, row_lanes, per_wave;
  bool interleaved;
};

// The codes of a block by a quad of lanes, eight values each, packed 4 bits
// each in the order of the values; and its d and m as f16 bits.
__device__ __forceinline__ uint32_t q4_block_4lanes(const float (&x)[8], uint32_t& dm) {
#pragma clang fp contract(off)
  float v[8], lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = x[j] == x[j] ? fminf(fmaxf(x[j], -32768.0f), 32768.0f) : 0.0f;
    lo = fminf(lo, v[j]);
    hi = fmaxf(hi, v[j]);
  }
  lo = fminf(lo, lane8_xchg<0xb1>(lo));
  lo = fminf(lo, lane8_xchg<0x4e>(lo)) + 0.0f;  // no minus zero
  hi = fmaxf(hi, lane8_xchg<0xb1>(hi));
  hi = fmaxf(hi, lane8_xchg<0x4e>(hi));
  const uint32_t db = f2h_bits((hi - lo) / 15.0f), mb = f2h_bits(lo);
  const float d = h2f(db), m = h2f(mb), inv = d > 0.0f ? 1.0f / d : 0.0f;
  uint32_t codes = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float n = fminf(fmaxf(rintf((v[j] - m) * inv), 0.0f), 15.0f);
    codes |= static_cast<uint32_t>(n) << (4 * j);
  }
  dm = db | mb << 16;
  return codes;
}

// Eight codes in order -> a dword of the key layout: byte i holds codes
// {0, 4, 1, 5}[i] and the code two further.
__device__ __forceinline__ uint32_t key_dword(uint32_t c) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = (i & 1) * 4 + (i >> 1);
    w |= ((c >> (4 * n)) & 15u) << (8 * i) | ((c >> (4 * n + 8)) & 15u) << (8 * i + 4);
  }
  return w;
}

template <int KT, int VT>
__global__ __launch_bounds__(256) void kv_append_q4_kernel(AppendArgs a) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63, groups = 64 / a.row_lanes;
  const int j = lane % a.row_lanes, group = lane / a.row_lanes;
  const int units = (a.Hk + groups - 1) / groups, segs = (units + a.per_wave - 1) / a.per_wave;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t t = item / segs;
  if (t >= a.T) return;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.pages * a.page) return;
  const int u0 = static_cast<int>(item % segs) * a.per_wave, u1 = min(units, u0 + a.per_wave);
  const bool in_row = j < a.D / 8, turned = j < a.rot / 8;
  const int half = a.rot / 16, nb = a.D / 32, b = j >> 2, part = j & 3;
  const int tok = static_cast<int>(slot % kCellTokens);
  float cos[8], sin[8];
  if (turned) {
    const int64_t row = max(int64_t{0}, min(a.P - 1, static_cast<int64_t>(a.positions[t]))) * a.rot;
    if (a.interleaved) {
      const float4 c = load4(QMM_F32, a.rope, row / 4 + j), s = load4(QMM_F32, a.rope, (row + a.rot / 2) / 4 + j);
      cos[0] = c.x, cos[1] = c.y, cos[2] = c.z, cos[3] = c.w;
      sin[0] = s.x, sin[1] = s.y, sin[2] = s.z, sin[3] = s.w;
    } else {
      load8(QMM_F32, a.rope, row / 8 + j % half, cos);
      load8(QMM_F32, a.rope, (row + a.rot / 2) / 8 + j % half, sin);
    }
  }
  for (int u = u0; u < u1; ++u) {
    const int h = u * groups + group;
    const bool on = in_row && h < a.Hk;
    Raw8<KT> key;
    Raw8<VT> val;
    if (on) {
      key.load(a.x[0], (t * a.stride[0] + static_cast<int64_t>(h) * a.D) / 8 + j);
      val.load(a.x[1], (t * a.stride[1] + static_cast<int64_t>(h) * a.D) / 8 + j);
    }
    float x[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[0][i] = on ? key.get(i) : 0.0f, x[1][i] = on ? val.get(i) : 0.0f;
    if (a.rot > 0) {
      if (a.interleaved) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = x[0][2 * i], q = x[0][2 * i + 1];
            x[0][2 * i] = p * cos[i] - q * sin[i];
            x[0][2 * i + 1] = q * cos[i] + p * sin[i];
          }
        }
      } else {
        const int from = turned ? (j < half ? lane + half : lane - half) : lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl(x[0][i], from);
          if (turned) {
            const float c = x[0][i] * cos[i], s = o * sin[i];
            x[0][i] = j < half ? c - s : c + s;
          }
        }
      }
    }
    uint32_t kd, vd;
    const uint32_t kc = q4_block_4lanes(x[0], kd), vc = q4_block_4lanes(x[1], vd);
    // a byte of the values' codes joins dims c and c + 16 of a block: this lane's and those of the lane two further
    const uint32_t other = static_cast<uint32_t>(lane8_xchg<0x4e>(static_cast<int>(vc)));
    if (!on) continue;
    uint8_t* cell = a.cache + kv_cell(slot, a.page, h, a.Hk, a.D);
    *reinterpret_cast<uint32_t*>(cell + (b * kCellTokens + tok) * 16 + part * 4) = key_dword(kc);
    const uint32_t low = part < 2 ? vc : other >> 16, high = part < 2 ? other : vc >> 16;
    const int quad = tok >> 2, c0 = (part & 1) * 8 + (part >> 1) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      cell[10 * a.D + ((quad * 16 + c0 + i) * nb + b) * 4 + kv_quad_byte(tok & 3)] =
          static_cast<uint8_t>(((low >> (4 * i)) & 15u) | ((high >> (4 * i)) & 15u) << 4);
    if (part == 0) {
      *reinterpret_cast<uint32_t*>(cell + 8 * a.D + (b * kCellTokens + tok) * 4) = kd;
      uint16_t* vs = reinterpret_cast<uint16_t*>(cell + 18 * a.D + (quad * nb + b) * 16) + (tok & 3);
      vs[0] = static_cast<uint16_t>(vd);
      vs[4] = static_cast<uint16_t>(vd >> 16);
    }
  }
}

struct ReadArgs {
  const uint8_t* cache;
  const int64_t* slots;
  void* y[2];
  int64_t pages, page, T;
  int Hk, D, row_lanes;
};

// n * d + m as the f16 that it stands for, widened
__device__ __forceinline__ float q4_value(uint32_t n, uint32_t d, uint32_t m) {
  const _Float16 dh = __builtin_bit_cast(_Float16, static_cast<uint16_t>(d));
  const _Float16 mh = __builtin_bit_cast(_Float16, static_cast<uint16_t>(m));
  return static_cast<float>(__builtin_fmaf16(static_cast<_Float16>(static_cast<float>(n)), dh, mh));
}

template <int TY>
__global__ __launch_bounds__(256) void kv_read_q4_kernel(ReadArgs a) {
  const int lane = threadIdx.x & 63, groups = 64 / a.row_lanes;
  const int j = lane % a.row_lanes, group = lane / a.row_lanes;
  const int units = (a.Hk + groups - 1) / groups;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t t = item / units;
  const int h = static_cast<int>(item % units) * groups + group;
  if (t >= a.T || j >= a.D / 8 || h >= a.Hk) return;
  const int64_t slot = a.slots[t];
  const int nb = a.D / 32, b = j >> 2, part = j & 3, tok = static_cast<int>(slot & (kCellTokens - 1)), quad = tok >> 2;
  float k[8] = {}, v[8] = {};
  if (slot >= 0 && slot < a.pages * a.page) {
    const uint8_t* cell = a.cache + kv_cell(slot, a.page, h, a.Hk, a.D);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(cell + (b * kCellTokens + tok) * 16 + part * 4);
    const uint32_t dm = *reinterpret_cast<const uint32_t*>(cell + 8 * a.D + (b * kCellTokens + tok) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = (i & 1) * 4 + (i >> 1);
      k[n] = q4_value((w >> (8 * i)) & 15u, dm, dm >> 16);
      k[n + 2] = q4_value((w >> (8 * i + 4)) & 15u, dm, dm >> 16);
    }
    const uint16_t* vs = reinterpret_cast<const uint16_t*>(cell + 18 * a.D + (quad * nb + b) * 16) + (tok & 3);
    const uint32_t d = vs[0], m = vs[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = cell[10 * a.D + ((quad * 16 + (part & 1) * 8 + i) * nb + b) * 4 + kv_quad_byte(tok & 3)];
      v[i] = q4_value(part < 2 ? byte & 15u : byte >> 4, d, m);
    }
  }
  const int64_t at = (t * a.Hk + h) * (a.D / 8) + j;
  Raw8<TY> o;
  o.set(k);
  o.store(a.y[0], at);
  o.set(v);
  o.store(a.y[1], at);
}

template <int KT>
static void launch_append(const AppendArgs& a, int v_type, dim3 g, hipStream_t st) {
  if (v_type == QMM_F32) hipLaunchKernelGGL((kv_append_q4_kernel<KT, QMM_F32>), g, dim3(256), 0, st, a);
  else if (v_type == QMM_F16) hipLaunchKernelGGL((kv_append_q4_kernel<KT, QMM_F16>), g, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((kv_append_q4_kernel<KT, QMM_BF16>), g, dim3(256), 0, st, a);
}

static int row_lanes_of(int64_t D) { return D == 64 ? 8 : D <= 128 ? 16 : 32; }

}  // namespace qmm

using namespace qmm;

extern "C" int kv_append_q4(const void* k, int64_t k_stride, int k_type, const void* v, int64_t v_stride, int v_type,
                            const float* rope, int64_t P, int64_t rot, int interleaved, const int32_t* positions,
                            const int64_t* slots, void* cache, int64_t pages, int64_t page, int64_t T, int64_t Hk,
                            int64_t D, void* stream) {
  if (!known_type(k_type) || !known_type(v_type)) return QMM_ERR_UNSUPPORTED;
  if (!kv_q4_shape(pages, page, Hk, D) || T < 0 || T > 0x7fffffff / Hk) return QMM_ERR_SHAPE;
  if (!strided_rows(k_stride, Hk, D) || !strided_rows(v_stride, Hk, D)) return QMM_ERR_SHAPE;
  if (rot < 0 || rot % 16 != 0 || rot > D || (rot > 0 && (P < 1 || P > 0x7fffffff))) return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!k || !v || !slots || !cache || (rot > 0 && (!rope || !positions))) return QMM_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(slots) || !aligned16(cache) || !aligned16(rope) ||
      !aligned16(positions))
    return QMM_ERR_ALIGN;
  const int lanes = row_lanes_of(D), groups = 64 / lanes;
  const int64_t units = (Hk + groups - 1) / groups;
  const int per = static_cast<int>(std::max<int64_t>(1, std::min(units, T * units / 16384)));
  const AppendArgs a{{k, v}, {k_stride, v_stride}, rope, positions, slots, static_cast<uint8_t*>(cache), P, pages, page,
                     T, static_cast<int>(Hk), static_cast<int>(D), static_cast<int>(rot), lanes, per, interleaved != 0};
  const dim3 g(static_cast<unsigned>((T * ((units + per - 1) / per) + 3) / 4));
  hipStream_t st = to_stream(stream);
  if (k_type == QMM_F32) launch_append<QMM_F32>(a, v_type, g, st);
  else if (k_type == QMM_F16) launch_append<QMM_F16>(a, v_type, g, st);
  else launch_append<QMM_BF16>(a, v_type, g, st);
  return launch_status();
}

extern "C" int kv_read_q4(const void* cache, int64_t pages, int64_t page, const int64_t* slots, void* k, void* v,
                          int type, int64_t T, int64_t Hk, int64_t D, void* stream) {
  if (!known_type(type)) return QMM_ERR_UNSUPPORTED;
  if (!kv_q4_shape(pages, page, Hk, D) || T < 0 || T > 0x7fffffff / Hk) return QMM_ERR_SHAPE;
  if (T == 0) return QMM_OK;
  if (!cache || !slots || !k || !v) return QMM_ERR_NULL;
  if (!aligned16(cache) || !aligned16(slots) || !aligned16(k) || !aligned16(v)) return QMM_ERR_ALIGN;
  const int lanes = row_lanes_of(D), groups = 64 / lanes;
  const ReadArgs a{static_cast<const uint8_t*>(cache), slots, {k, v}, pages, page, T, static_cast<int>(Hk),
                   static_cast<int>(D), lanes};
  const dim3 g(static_cast<unsigned>((T * ((Hk + groups - 1) / groups) + 3) / 4)), blk(256);
  hipStream_t st = to_stream(stream);
  if (type == QMM_F32) hipLaunchKernelGGL(kv_read_q4_kernel<QMM_F32>, g, blk, 0, st, a);
  else if (type == QMM_F16) hipLaunchKernelGGL(kv_read_q4_kernel<QMM_F16>, g, blk, 0, st, a);
  else hipLaunchKernelGGL(kv_read_q4_kernel<QMM_BF16>, g, blk, 0, st, a);
  return launch_status();
}
