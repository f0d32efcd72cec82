// Attention over whole prompts, packed sequences.
//
//   S^T = K Q^T,  p = 2^(c (s - m)),  O^T = V^T P^T,  y = O / sum p
//
// The rows of one key head (tokens x heads of the group) are the columns of
// 32 x 32 tiles; a wave has 32 of them, a workgroup 128, which share tiles of K
// and V in LDS, copied there by the loads themselves, K two tiles ahead, V one.  S^T's
// layout leaves in each lane the terms of one query and eight keys of every
// sixteen, which is the operand that O^T takes: the terms stay in registers.
// V comes out of its rows transposed by the LDS's transposing reads.  Chunks of
// 16 bytes stand permuted within a tile's rows so that neither the reads of 32
// rows of K nor those of four rows of V meet in the LDS's banks.
//
// With the heads of a group in one tile a tile of 128 rows spans few tokens, so
// little of it lies behind the causal border, and K and V are read once for the
// group.
//
// Where all of a wave's rows see whole tiles, a tile's exponentials stand
// between the matrix instructions of the next tile's scores, in a written order.
// Few rows against many keys: the keys are split, and a second kernel joins.
//
// Bound by the matrix cores and the power they take.  6000 + 2192 tokens, 32/8
// heads of 128, bf16: 318 to 340 us, 990 to 1050 TFLOP/s, on one card of five 357
// (on one with 331 its matrix instructions alone, without copies and exponentials,
// took 256).  Its 38 spilled registers are of the last of an odd number of whole
// tiles and of masked ones, none of the steady loop.  16/4 heads of 256, 512 tokens
// behind 4096: 50 us and 8 for the join, of which 29 do not grow with the keys
// (8192 more: 60 us, 1150 TFLOP/s): the partial results of four splits, 33 MB,
// written and read, the first loads, and the masked tiles.  Half of the operands'
// LDS reads left out gains 4 %, eight waves on the same tiles 1 %.
#include "attn.hpp"

#include <algorithm>
#include <math.h>

namespace qmm {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 128;  // of a workgroup's tile: four waves of 32

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* y;
  float* part;  // [tiles][Hk][splits][128][D], then as many pairs (m, l) of rows
  int64_t q_stride, k_stride, v_stride;
  float scale;
  int window, Tq, Tk, B, Hq, Hk, group, splits, tiles, y_type;
  bool causal;
};

// An operand of eight 16-bit values, four dwords.
__device__ __forceinline__ v4u op4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) { return v4u{a, b, c, d}; }
template <bool BF16>
__device__ __forceinline__ v16f mfma32(v4u x, v4u y, v16f c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, b2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
  } else {
    typedef _Float16 f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, f2{static_cast<_Float16>(a), static_cast<_Float16>(b)});
  }
}

// c + both of a pair, in fp32.  Terms are summed as the product with the values takes them, rounded.
template <bool BF16>
__device__ __forceinline__ float add2(uint32_t pair, float c) {
  if constexpr (BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, pair), b2{static_cast<__bf16>(1.0f), static_cast<__bf16>(1.0f)}, c, false);
  } else {
    typedef _Float16 f2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f2, pair), f2{static_cast<_Float16>(1.0f), static_cast<_Float16>(1.0f)}, c, false);
  }
}

// 16 bytes per lane from off bytes into a buffer to LDS at lds + 16 * lane; zeros for what lies past the buffer's end.
// Not tracked by the compiler: see dma16.
__device__ __forceinline__ void copy16(v4u buffer, uint32_t off, uint32_t lds) {
  uint32_t saved;
  __asm__ volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds\n\t"
                   "s_mov_b32 m0, %0"
                   : "=&s"(saved)
                   : "v"(off), "s"(buffer), "s"(lds)
                   : "memory");
}

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
  return static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32))) << 32 |
         static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x)));
}

__device__ __forceinline__ float uniform(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}

constexpr int gcd16(int c) { return c % 16 == 0 ? 16 : c % 8 == 0 ? 8 : c % 4 == 0 ? 4 : c % 2 == 0 ? 2 : 1; }

// Which sequence a tile belongs to, by the waves' lanes: 64 sequences at a time.
struct Place {
  int q0, nq, k0, nk, tile;  // the sequence's first rows and counts, and the tile's number in it
  bool found;
};
__device__ __forceinline__ Place find_place(const PromptArgs& a, int n, int lane) {
  Place p{0, 0, 0, 0, 0, false};
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = min(b0 + lane, a.B - 1);
    const int q0 = max(0, min(a.Tq, a.cu_q[b])), q1 = max(q0, min(a.Tq, a.cu_q[b + 1]));
    const int k0 = max(0, min(a.Tk, a.cu_k[b])), k1 = max(k0, min(a.Tk, a.cu_k[b + 1]));  // with these, not behind them
    const int mine = b0 + lane < a.B ? ((q1 - q0) * a.group + kRows - 1) / kRows : 0;
    const int upto = wave_scan(mine);
    const uint64_t past = __builtin_amdgcn_ballot_w64(before + upto > n);
    if (past) {
      const int at = __builtin_ctzll(past);
      p.q0 = __builtin_amdgcn_readlane(q0, at);
      p.nq = __builtin_amdgcn_readlane(q1, at) - p.q0;
      // a sequence's last tiles, which see the most keys, first
      p.tile = before + __builtin_amdgcn_readlane(upto, at) - 1 - n;
      p.k0 = __builtin_amdgcn_readlane(k0, at);
      p.nk = __builtin_amdgcn_readlane(k1, at) - p.k0;
      p.found = true;
      return p;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return p;
}

template <int D, int BN, bool BF16>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void attn_prompt_kernel(PromptArgs a) {
  constexpr int C = D / 8, kRowBytes = 2 * D, kTile = BN * kRowBytes;  // chunks of a row
  constexpr int G = gcd16(C), kPeriod = 16 / G;                        // K: chunk ^ (row / kPeriod) % G
  constexpr int kVShift = C % 16 == 0 ? 0 : 1, kVMask = C % 16 == 0 ? 3 : C % 8 == 0 ? 1 : 0;  // V: chunk ^ 4 * ...
  constexpr int kCopies = BN * C / 256;                                // a wave's copies of a tile
  constexpr int kSteps = D / 16, kBlocks = D / 32, kKeys = BN / 32;
  constexpr float kSlack = 8.0f;               // a maximum is followed when it is passed by 2^8
  constexpr float kFar = 1024.0f;              // up to here `base` is off by 2^-14 at most, and alike for all terms
  constexpr int kKeyBufs = 3;
  __shared__ __attribute__((aligned(1024))) uint8_t s_k[kKeyBufs][kTile], s_v[2][kTile];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, h = lane >> 5;

  int id = blockIdx.x;
  const int kh = id % a.Hk;
  id /= a.Hk;
  const int split = id % a.splits, n = id / a.splits;
  const Place pl = find_place(a, n, lane);
  if (!pl.found) return;
  const int rows = pl.nq * a.group, row0 = pl.tile * kRows + wave * 32, before = pl.nk - pl.nq;

  // What terms of the maximum are, as an exponent of two; others are up to 2^8 times that.  In f16 those of 2^15 and, down
  // to 2^-31 of the maximum, all can be told.  In bf16 the terms of all keys sum to less than 1/2, so that no sum of them
  // times values leaves fp32 (values below 2^(-126 - lift) lose bits).
  const float lift = BF16 ? uniform(-9.0f - static_cast<float>(32 - __builtin_clz(pl.nk | 1))) : 7.0f;

  // this lane's query, and the keys it sees: lo .. at
  const int row = min(row0 + col, rows - 1), tok = row / a.group, head = kh * a.group + row % a.group;
  const int at = a.causal ? before + tok : pl.nk - 1, lo = a.window > 0 ? max(0, at - a.window + 1) : 0;
  const float mul = exponent_mul(a.scale);
  v4u q[kSteps];
  {
    // the scale's sign into the query, so that the largest product is the largest score
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(pl.q0 + tok) * a.q_stride + head * D;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, keep = vanishes(a.scale) ? 0u : ~0u;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      q[s] = *reinterpret_cast<const v4u*>(src + s * 16 + h * 8);
      q[s].x = (q[s].x ^ flip) & keep, q[s].y = (q[s].y ^ flip) & keep;
      q[s].z = (q[s].z ^ flip) & keep, q[s].w = (q[s].w ^ flip) & keep;
    }
  }
  const float slack = fminf(kSlack / mul, 3.0e38f);  // finite: the first maximum lies infinitely far above -inf

  // the bounds of the wave's rows and of the workgroup's, the same for all lanes
  const bool active = row0 < rows;
  const int wave_first = min(row0, rows - 1) / a.group, wave_last = min(row0 + 31, rows - 1) / a.group;
  const int wave_at0 = a.causal ? before + wave_first : pl.nk - 1, wave_at1 = a.causal ? before + wave_last : pl.nk - 1;
  const int wave_lo0 = a.window > 0 ? max(0, wave_at0 - a.window + 1) : 0;
  const int wave_lo1 = a.window > 0 ? max(0, wave_at1 - a.window + 1) : 0;
  const int first_tok = pl.tile * kRows / a.group, last_tok = min(pl.tile * kRows + kRows - 1, rows - 1) / a.group;
  const int all_end = max(0, (a.causal ? before + last_tok : pl.nk - 1) + 1);
  const int all_first = a.window > 0 ? max(0, before + first_tok - a.window + 1) / BN : 0;
  const int count = max(0, (all_end + BN - 1) / BN - all_first), per = (count + a.splits - 1) / a.splits;
  const int tile0 = all_first + min(count, split * per), tile1 = all_first + min(count, (split + 1) * per);

  // Copies: where each of this lane's chunks stands in a tile of the rows, and the tile as a buffer that ends with the
  // sequence's last row, so that rows behind it are zeros.
  const uint32_t k_bytes = static_cast<uint32_t>(a.k_stride) * 2, v_bytes = static_cast<uint32_t>(a.v_stride) * 2;
  uint32_t k_off[kCopies], v_off[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int at16 = (wave * kCopies + i) * 64 + lane, r = at16 / C, c = at16 % C;
    k_off[i] = r * k_bytes + static_cast<uint32_t>((c ^ ((r / kPeriod) & (G - 1))) * 16);
    v_off[i] = r * v_bytes + static_cast<uint32_t>((c ^ (4 * ((r >> kVShift) & kVMask))) * 16);
  }
  // where the next tiles to copy begin
  const int64_t first_key = pl.k0 + static_cast<int64_t>(tile0) * BN;
  uint64_t k_next = uniform(reinterpret_cast<uint64_t>(a.k) + (first_key * a.k_stride + kh * D) * 2);
  uint64_t v_next = uniform(reinterpret_cast<uint64_t>(a.v) + (first_key * a.v_stride + kh * D) * 2);
  const uint32_t k_step = BN * k_bytes, v_step = BN * v_bytes;
  const uint32_t k_lds = lds_addr(&s_k[0][0]) + wave * (kCopies * 1024), v_lds = lds_addr(&s_v[0][0]) + wave * (kCopies * 1024);
  // tile t of rows of `bytes`, which begins at `at`
  const auto tile_of = [&](uint64_t at, uint32_t bytes, int t) {
    const int left = min(BN, pl.nk - t * BN);
    return v4u{static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32) & 0xffffu,
               left > 0 ? static_cast<uint32_t>(left - 1) * bytes + kRowBytes : 0u, 0x00020000u};
  };
  // Byte offsets of the buffers of tiles t and t + 1 of keys and of the one to fill, and of tile t of values.
  uint32_t key_buf = 0, next_buf = kTile, fill_buf = 2 * kTile, value_buf = 0;
  const auto copy_k = [&](int t, uint32_t buf) {
    const v4u tile = tile_of(k_next, k_bytes, t);
    k_next += k_step;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy16(tile, k_off[i], k_lds + buf + i * 1024);
  };
  const auto copy_v = [&](int t, uint32_t buf) {
    const v4u tile = tile_of(v_next, v_bytes, t);
    v_next += v_step;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy16(tile, v_off[i], v_lds + buf + i * 1024);
  };
  if (tile0 < tile1) {
    copy_k(tile0, key_buf);
    copy_v(tile0, value_buf);
    copy_k(tile0 + 1, next_buf);
  }
  // Before a tile: its copies (and the next keys') are there for every wave, and what the other buffers held has been read,
  // so that they may be filled.  Behind the last tile they are filled with zeros.
  const auto enter = [&]() {
    wait_vmcnt<0>();
    __syncthreads();
  };
  const auto fill = [&](int t) {
    copy_k(t + 2, fill_buf);
    copy_v(t + 1, value_buf ^ kTile);
  };
  const auto leave = [&]() {
    const uint32_t k = key_buf;
    key_buf = next_buf;
    next_buf = fill_buf;
    fill_buf = k;
    value_buf ^= kTile;
  };

  // LDS addresses of this lane's operands in the first buffer.  The permutations touch bits that are clear in a row's
  // address, so an operand further on is an exclusive or away, or a sum.
  const int k_swz = (col / kPeriod) & (G - 1), i16 = lane & 15, v_row = 4 * h + (i16 >> 2);
  const uint32_t k_at = lds_addr(&s_k[0][0]) + col * kRowBytes + (h ^ k_swz) * 16;
  const uint32_t v_at = lds_addr(&s_v[0][0]) + v_row * kRowBytes + ((v_row >> kVShift) & kVMask) * 64 +
                        ((lane >> 4) & 1) * 32 + (i16 & 3) * 8;
  typedef const __attribute__((address_space(3))) v4u* lds_v4u;
  typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
  const auto k_operand = [&](uint32_t at, int kb, int s) {
    constexpr int kLow = G / 2;  // steps within which the permutation stays
    return *reinterpret_cast<lds_v4u>((at ^ (s % kLow * 32)) + (s / kLow * kLow * 32 + kb * 32 * kRowBytes));
  };
  const auto v_operand = [&](uint32_t at, int kk, int b) {
    const uint32_t off = (at ^ ((b & kVMask) * 64)) + ((b & ~kVMask) * 64 + kk * 16 * kRowBytes);
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4>(off));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4>(off + 8 * kRowBytes));
    const uint2 u = __builtin_bit_cast(uint2, x), w = __builtin_bit_cast(uint2, y);
    return op4(u.x, u.y, w.x, w.y);
  };
  // the key of register i of block kb, counted within a tile from 4 h on
  const auto key_of = [](int kb, int i) { return kb * 32 + 8 * (i >> 2) + (i & 3); };

  v16f o[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) o[b] = v16f{};
  float top = -INFINITY, base = lift, sum = 0.0f;  // what terms go by, what a scaled product takes to their exponents
  bool far = false;  // some row's exponent leaves fp32 too little behind the point: products are settled first

  const auto products = [&](v16f (&s)[kKeys], uint32_t buf) {
    const uint32_t here = k_at + buf;
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < kKeys; ++kb)
        s[kb] = mfma32<BF16>(k_operand(here, kb, st), q[st], st == 0 ? v16f{} : s[kb]);
  };
  const auto terms = [&](const v16f (&s)[kKeys], v4u (&p)[BN / 16]) {
#pragma unroll
    for (int kb = 0; kb < kKeys; ++kb) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], mul, base));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i + 1], mul, base));
        w[i / 2] = pack2<BF16>(e0, e1);
        sum = add2<BF16>(w[i / 2], sum);
      }
      p[2 * kb] = op4(w[0], w[1], w[2], w[3]);
      p[2 * kb + 1] = op4(w[4], w[5], w[6], w[7]);
    }
  };
  const auto values = [&](uint32_t v_here, const v4u (&p)[BN / 16]) {
#pragma unroll
    for (int kk = 0; kk < BN / 16; ++kk)
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) o[b] = mfma32<BF16>(v_operand(v_here, kk, b), p[kk], o[b]);
  };
  // Tiles of which some keys are not seen by some rows.  There a term of 0
  // times a value that is not finite would be NaN; products with zeros tell
  // whether there are any.
  const auto part_values = [&](uint32_t v_here, const v4u (&p)[BN / 16], int at_here, int lo_here) {
    v16f z = {};
#pragma unroll
    for (int kk = 0; kk < BN / 16; ++kk)
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) z = mfma32<BF16>(v_operand(v_here, kk, b), op4(0u, 0u, 0u, 0u), z);
    float any = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) any += z[i];
    if (__builtin_amdgcn_ballot_w64(any != any) == 0) {
      values(v_here, p);
    } else {
      // The finite values as above; then, in loops that are not unrolled, how
      // many of the others each query sees: +inf counts 1, -inf 128, NaN 16384
      // (at most 64 of each).
      constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u, kOne = BF16 ? 0x3f80u : 0x3c00u;
      const auto bad = [](uint32_t x) { return (x & kInf) == kInf; };
      const auto clean = [&](uint32_t x) { return x & ((bad(x) ? 0u : 0xffffu) | (bad(x >> 16) ? 0u : 0xffff0000u)); };
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const v4u v = v_operand(v_here, kk, b);
          o[b] = mfma32<BF16>(op4(clean(v.x), clean(v.y), clean(v.z), clean(v.w)), p[kk], o[b]);
        }
      int at_odd = at_here, lo_odd = lo_here;
      uint32_t v_odd = v_here;
      __asm__ volatile("" : "+v"(at_odd), "+v"(lo_odd), "+v"(v_odd));  // nothing of this is worked out before
#pragma unroll 1
      for (int b = 0; b < kBlocks; ++b) {
        v16f found = {};
#pragma unroll 1
        for (int kk = 0; kk < BN / 16; ++kk) {
          const v4u v = v_operand(v_odd, kk, b);
          const auto kind = [&](uint32_t x) {
            x &= 0xffffu;
            return !bad(x) ? 0u : x == kInf ? kOne : x == (kInf | 0x8000u) ? (BF16 ? 0x4300u : 0x5800u) : BF16 ? 0x4680u : 0x7400u;
          };
          const auto see = [&](int i) {
            const int j = kk * 16 + 8 * (i >> 2) + (i & 3);
            return j <= at_odd && j >= lo_odd ? kOne : 0u;
          };
          found = mfma32<BF16>(op4(kind(v.x) | kind(v.x >> 16) << 16, kind(v.y) | kind(v.y >> 16) << 16,
                                          kind(v.z) | kind(v.z >> 16) << 16, kind(v.w) | kind(v.w >> 16) << 16),
                               op4(see(0) | see(1) << 16, see(2) | see(3) << 16, see(4) | see(5) << 16,
                                          see(6) | see(7) << 16),
                               found);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = static_cast<int>(found[i]);
          const bool pos = (c & 127) != 0, neg = (c >> 7 & 127) != 0, nan = c >= 16384 || (pos && neg);
          found[i] = nan ? NAN : pos ? INFINITY : neg ? -INFINITY : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kBlocks; ++u)
          if (u == b) o[u] += found;
      }
    }
  };

  // Two products more into a maximum.
  const auto higher = [](float most, const v16f (&s)[kKeys], int n) {
    return fmaxf(fmaxf(most, s[n / 8][n % 8 * 2]), s[n / 8][n % 8 * 2 + 1]);
  };
  const auto highest = [&](const v16f (&s)[kKeys]) {
    float most = -INFINITY;
#pragma unroll
    for (int n = 0; n < kKeys * 8; ++n) most = higher(most, s, n);
    return halves_max(most);
  };
  // The maximum of new products: where it passes what all so far goes by too far, that is brought to it.
  const auto follow = [&](float most) {
    if (__builtin_amdgcn_ballot_w64(most - top > slack)) {
      most = fmaxf(most, top);
      const float zero = most == -INFINITY ? 0.0f : most, keep = __builtin_amdgcn_exp2f((top - zero) * mul);
      sum *= keep;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) o[b] *= keep;
      top = most;
      far = __builtin_amdgcn_ballot_w64(!(fabsf(zero * mul) <= kFar)) != 0;
      base = far ? lift : lift - zero * mul;
    }
  };
  // Products as `base` takes them.  A term beside the matrix instructions costs one
  // fma; its offset, rounded by itself, is a whole step of the exponent for products
  // of 2^24, so past kFar the difference is taken first.
  const auto settle = [&](v16f (&s)[kKeys]) {
    if (far) {
      const float zero = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int kb = 0; kb < kKeys; ++kb) s[kb] -= zero;
    }
  };

  // The tiles of which this wave's rows see something, and those that all of them see whole.
  const int wave0 = max(tile0, wave_lo0 / BN), wave1 = active ? min(tile1, wave_at1 < 0 ? 0 : wave_at1 / BN + 1) : 0;
  const int whole0 = max(wave0, (wave_lo1 + BN - 1) / BN), whole1 = min(wave1, wave_at0 < 0 ? 0 : (wave_at0 + 1) / BN);
  // one tile by itself
  const auto alone = [&](int t) {
    enter();
    fill(t);
    if (t >= wave0 && t < wave1) {
      const bool whole = t >= whole0 && t < whole1;
      const int at_here = at - t * BN - 4 * h, lo_here = lo - t * BN - 4 * h;
      v16f s[kKeys];
      v4u p[BN / 16];
      products(s, key_buf);
      if (!whole) {
#pragma unroll
        for (int kb = 0; kb < kKeys; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[kb][i] = key_of(kb, i) <= at_here && key_of(kb, i) >= lo_here ? s[kb][i] : -INFINITY;
      }
      follow(highest(s));
      settle(s);
      terms(s, p);
      if (whole) values(v_at + value_buf, p);
      else part_values(v_at + value_buf, p, at_here, lo_here);
    }
    leave();
  };

  int t = tile0;
  const int run0 = whole1 - whole0 >= 2 ? whole0 : tile1, run1 = whole1 - whole0 >= 2 ? whole1 : tile1;
  for (; t < run0; ++t) alone(t);
  if (t < run1) {
    v16f x[kKeys], y[kKeys];
    v4u p[BN / 16];
    // A tile's terms beside the products of the next tile's keys, then the products of the terms with the values.  The
    // order is written out: matrix instructions without a pause, their operands read five ahead, and behind each of the
    // first ones its share of the terms, two of them exponentiated and the two before packed, and now and then a copy.
    const auto step = [&](v16f (&cur)[kKeys], v16f (&next)[kKeys]) {
      settle(cur);
      const v4u k_tile = tile_of(k_next, k_bytes, t + 2), v_tile = tile_of(v_next, v_bytes, t + 1);
      k_next += k_step;
      v_next += v_step;
      constexpr int kFirst = kSteps * kKeys, kSecond = BN / 16 * kBlocks, kPairs = kKeys * 8;
      constexpr int kAheadBy = 5, kMaxIn = kSecond - 2;
      const uint32_t k_here = k_at + next_buf, v_here = v_at + value_buf;
      v4u f[kAheadBy];
      float most = -INFINITY;
      const auto operand = [&](int m) {
        return m < kFirst ? k_operand(k_here, m % kKeys, m / kKeys)
                          : v_operand(v_here, (m - kFirst) / kBlocks, (m - kFirst) % kBlocks);
      };
      float e[2][2];
      const auto raise = [&](int n) {
        const v16f& c = cur[n / 8];
        e[n & 1][0] = __builtin_amdgcn_exp2f(__builtin_fmaf(c[n % 8 * 2], mul, base));
        e[n & 1][1] = __builtin_amdgcn_exp2f(__builtin_fmaf(c[n % 8 * 2 + 1], mul, base));
      };
      const auto pack = [&](int n) {
        const uint32_t w = pack2<BF16>(e[n & 1][0], e[n & 1][1]);
        p[n / 4][n % 4] = w;
        sum = add2<BF16>(w, sum);
      };
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < kAheadBy; ++m) f[m] = operand(m);
#pragma unroll
      for (int m = 0; m < kFirst; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        next[m % kKeys] = mfma32<BF16>(f[m % kAheadBy], q[m / kKeys], m < kKeys ? v16f{} : next[m % kKeys]);
        f[m % kAheadBy] = operand(m + kAheadBy);
        static_assert(kFirst >= 4 * kCopies);
        if (m % 4 == 0 && m / 4 < kCopies) copy16(k_tile, k_off[m / 4], k_lds + fill_buf + m / 4 * 1024);
        if (m % 4 == 2 && m / 4 < kCopies) copy16(v_tile, v_off[m / 4], v_lds + (value_buf ^ kTile) + m / 4 * 1024);
#pragma unroll
        for (int n = m * kPairs / kFirst; n < (m + 1) * kPairs / kFirst; ++n) {
          raise(n);
          if (n > 0) pack(n - 1);
        }
      }
      pack(kPairs - 1);
#pragma unroll
      for (int m = 0; m < kSecond; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        o[m % kBlocks] = mfma32<BF16>(f[(kFirst + m) % kAheadBy], p[m / kBlocks], o[m % kBlocks]);
        if (m + kAheadBy < kSecond) f[(kFirst + m) % kAheadBy] = operand(kFirst + m + kAheadBy);
#pragma unroll
        for (int n = m * kPairs / kMaxIn; n < min(kPairs, (m + 1) * kPairs / kMaxIn); ++n) most = higher(most, next, n);
        if (m == kMaxIn - 1) most = halves_max(most);
      }
      __builtin_amdgcn_sched_barrier(0);
      follow(most);
    };
    enter();
    products(x, key_buf);
    follow(highest(x));
    int left = run1 - t - 1;  // steps with a next tile
    for (; left >= 2; left -= 2) {
      step(x, y);
      leave();
      enter(), ++t;
      step(y, x);
      leave();
      enter(), ++t;
    }
    if (left) {
      step(x, y);
      leave();
      enter(), ++t;
#pragma unroll
      for (int kb = 0; kb < kKeys; ++kb) x[kb] = y[kb];
    }
    fill(t);
    settle(x);
    terms(x, p);
    values(v_at + value_buf, p);
    leave();
    ++t;
  }
  for (; t < tile1; ++t) alone(t);
  wait_vmcnt<0>();

  if (!active) return;
  sum = halves_sum(sum);
  const bool mine = row0 + col < rows;
  if (a.splits > 1) {
    const int64_t slot = ((static_cast<int64_t>(n) * a.Hk + kh) * a.splits + split) * kRows + wave * 32 + col;
    float* part = a.part + slot * D;
    if (mine) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<v4f*>(part + b * 32 + 2 * i + 4 * h) = v4f{o[b][i], o[b][i + 1], o[b][i + 2], o[b][i + 3]};
      if (h == 0)
        reinterpret_cast<float2*>(a.part + static_cast<int64_t>(a.tiles) * a.Hk * a.splits * kRows * D)[slot] =
            make_float2(top, sum);
    }
  } else if (mine) {
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t out = (static_cast<int64_t>(pl.q0 + tok) * a.Hq + head) * D;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        store4(a.y_type, a.y, (out + b * 32 + 2 * i + 4 * h) / 4,
               make_float4(o[b][i] * f, o[b][i + 1] * f, o[b][i + 2] * f, o[b][i + 3] * f));
  }
}

// Joins the splits of a tile's rows, a wave per row.
__global__ __launch_bounds__(256) void attn_prompt_join_kernel(PromptArgs a, int D) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int part = blockIdx.x % (kRows / 4), kh = blockIdx.x / (kRows / 4) % a.Hk, n = blockIdx.x / (kRows / 4) / a.Hk;
  const int in_tile = part * 4 + wave;
  const int64_t slot = (static_cast<int64_t>(n) * a.Hk + kh) * a.splits * kRows + in_tile;
  const float2* ml = reinterpret_cast<const float2*>(a.part + static_cast<int64_t>(a.tiles) * a.Hk * a.splits * kRows * D);
  // every tile has its slots, whether there is such a tile or not
  Parts parts([&](int k) { return slot + k * kRows; }, a.part + min(lane * 4, D - 4), D, ml, a.splits, lane);
  const Place pl = find_place(a, n, lane);
  const int row = pl.tile * kRows + in_tile;
  if (!pl.found || row >= pl.nq * a.group) return;
  const v4f y = parts.join(exponent_mul(a.scale));
  const int64_t out = (static_cast<int64_t>(pl.q0 + row / a.group) * a.Hq + kh * a.group + row % a.group) * D;
  if (lane * 4 < D) store4(a.y_type, a.y, out / 4 + lane, make_float4(y.x, y.y, y.z, y.w));
}

// The most tiles that sequences of Tq tokens in all may have, and how many ways their keys are split.
struct PromptPlan {
  int64_t tiles, splits;
};
// A workgroup takes 1e-4 us per key and dim (0.82 us for 64 keys of 128, 0.78 for
// 32 of 256).  With s splits that is divided by s, and partial results cost 3.5 us
// for the second launch, 1.7e-6 us for each float, written and read, and 0.08 us a
// split; the best s follows.  One workgroup per CU keeps the chip busy, more only
// make more partial results.  Sequences count as of one size.  us, heads 32/8 x 128:
//                  1 split  2     4     8     16    32    this
//   512 of 512     17.4     26.7  29.0  42.5              17.5 (1)
//   512 of 4608    70.9     55.9  57.5  68.1  95.0        56.9 (2)
//   64 of 8192     115      66.5  41.2  30.4  27.4  36.7  27.0 (13)
//   16 of 32768    421      219   116   65.4  41.2  35.5  35.9 (32)
static PromptPlan prompt_plan(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t BN) {
  constexpr double kPerKey = 1e-4, kJoin = 3.5, kPerFloat = 1.7e-6, kPerSplit = 0.08;
  constexpr int64_t kCUs = 256, kMostSplits = 64;
  PromptPlan p;
  const int64_t rows = Tq * (Hq / Hk), whole = (rows + kRows - 1) / kRows;
  p.tiles = std::min(rows, whole + B);
  p.splits = 1;
  const int64_t groups = std::max<int64_t>(1, whole + (B - 1) / 2) * Hk, key_tiles = B > 0 ? (Tk / B + BN - 1) / BN : 0;
  const double alone = static_cast<double>(key_tiles * BN * D) * kPerKey;
  const double each = static_cast<double>(Tq * Hq * D) * kPerFloat + kPerSplit;
  int64_t s = std::min({static_cast<int64_t>(sqrt(alone / each)), kCUs / groups, key_tiles, kMostSplits});
  if (s < 2) return p;
  s = (key_tiles + (key_tiles + s - 1) / s - 1) / ((key_tiles + s - 1) / s);  // none without keys
  if (alone / s + kJoin + each * s < alone) p.splits = s;
  return p;
}

// With Tq * Hq below 2^30 there are then less than 2^24 workgroups, a grid's most with 256 lanes each.
constexpr int64_t kMostSequences = int64_t{1} << 23;

static bool prompt_shape(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D) {
  return B >= 0 && Tq >= 0 && Tk >= 0 && Tq < kMostTokens && Tk < kMostTokens && Hk >= 1 && Hq >= Hk && Hq <= 1024 && Hq % Hk == 0 &&
         attn_head_dim(D) && Tq < kMostTokens / Hq && B < kMostSequences / Hq;
}

// Keys of a tile.
constexpr int64_t tile_keys(int64_t D) { return D <= 128 ? 64 : 32; }

template <int D>
static void launch_prompt(const PromptArgs& a, bool bf16, dim3 g, hipStream_t st) {
  constexpr int BN = static_cast<int>(tile_keys(D));
  if (bf16) hipLaunchKernelGGL((attn_prompt_kernel<D, BN, true>), g, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((attn_prompt_kernel<D, BN, false>), g, dim3(256), 0, st, a);
}

}  // namespace qmm

using namespace qmm;

extern "C" size_t attn_prompt_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D) {
  if (!prompt_shape(B, Tq, Tk, Hq, Hk, D)) return 0;
  const PromptPlan p = prompt_plan(B, Tq, Tk, Hq, Hk, D, tile_keys(D));
  return p.splits == 1 ? 0 : static_cast<size_t>(p.tiles * Hk * p.splits * kRows * (D + 2) * 4);
}

extern "C" int attn_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, int type, const int32_t* cu_q, const int32_t* cu_k, int64_t B, float scale,
                           int causal, int64_t window, void* y, int y_type, int64_t Tq, int64_t Tk, int64_t Hq,
                           int64_t Hk, int64_t D, void* ws, size_t ws_bytes, void* stream) {
  if ((type != QMM_F16 && type != QMM_BF16) || !known_type(y_type) || (window > 0 && !causal)) return QMM_ERR_UNSUPPORTED;
  if (!prompt_shape(B, Tq, Tk, Hq, Hk, D)) return QMM_ERR_SHAPE;
  if (!strided_rows(q_stride, Hq, D) || !strided_rows(k_stride, Hk, D) || !strided_rows(v_stride, Hk, D))
    return QMM_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || window > 0x7fffffff) return QMM_ERR_SHAPE;
  if (B == 0 || Tq == 0) return QMM_OK;
  const size_t need = attn_prompt_workspace_bytes(B, Tq, Tk, Hq, Hk, D);
  if (!q || !cu_q || !cu_k || !y || (Tk > 0 && (!k || !v)) || (need > 0 && !ws)) return QMM_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned_list(cu_q, 4) || !aligned_list(cu_k, 4) ||
      !aligned16(y) || !aligned16(ws))
    return QMM_ERR_ALIGN;
  if (ws_bytes < need) return QMM_ERR_WORKSPACE;
  const PromptPlan p = prompt_plan(B, Tq, Tk, Hq, Hk, D, tile_keys(D));
  const PromptArgs a{q, k, v, cu_q, cu_k, y, static_cast<float*>(ws), q_stride, k_stride, v_stride, scale,
                     static_cast<int>(std::min(window, kMostTokens)), static_cast<int>(Tq), static_cast<int>(Tk), static_cast<int>(B),
                     static_cast<int>(Hq), static_cast<int>(Hk), static_cast<int>(Hq / Hk), static_cast<int>(p.splits),
                     static_cast<int>(p.tiles), y_type, causal != 0};
  const dim3 g(static_cast<unsigned>(p.tiles * Hk * p.splits));
  hipStream_t st = to_stream(stream);
  switch (D) {
    case 64: launch_prompt<64>(a, type == QMM_BF16, g, st); break;
    case 96: launch_prompt<96>(a, type == QMM_BF16, g, st); break;
    case 128: launch_prompt<128>(a, type == QMM_BF16, g, st); break;
    case 192: launch_prompt<192>(a, type == QMM_BF16, g, st); break;
    default: launch_prompt<256>(a, type == QMM_BF16, g, st); break;
  }
  if (p.splits > 1)
    hipLaunchKernelGGL(attn_prompt_join_kernel, dim3(static_cast<unsigned>(p.tiles * Hk * (kRows / 4))), dim3(256), 0, st,
                       a, static_cast<int>(D));
  return launch_status();
}
