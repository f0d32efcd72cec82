// Attention of a sequence's last tokens over the paged 4-bit cache.
//
//   S^T = K Q^T,  p = 2^(c (s - max s)),  O^T = V^T P^T,  y = O / sum p
//
// The query rows of one key head (new tokens x heads of the group) are the
// columns of 16 x 16 tiles.  A wave takes 32 tokens, two cells of the cache, at
// a time.  The cache's order gives each lane the codes that its place in the
// operands of v_mfma_f32_16x16x32_f16 needs, with whole loads: for K a lane has
// one key and one block (or a part of one), so one scale pair; for V one dim
// and a quad of tokens of each cell, whose scales come from a load of the whole
// cell's by row broadcasts.  The tile of S^T leaves in each lane the terms of
// one query and the same quads of tokens, which is the operand that O^T takes:
// nothing goes through LDS between the products.  Codes become f16 numbers, two
// an instruction, by the conversion of 8-bit floats (codes_to_f16), and by one fma
// the numbers that the format stands for.
//
// How the work is dealt out (the host knows no lengths):
//   short sequences  a workgroup of eight waves takes a sequence and head whole,
//                    or, where these are few, some blocks of its values
//   few of them      each is cut into as many equal parts as fill the chip
//   many             the steps of all are dealt out to a fixed number of
//                    workgroups in equal runs, found from the lengths by each,
//                    so that ragged lengths fill the chip alike
// Parts, and runs that begin or end inside a sequence, leave partial results in
// the workspace, and a second kernel joins these.
//
// Bound by HBM and, next to it, by the instructions that make numbers of codes.
// 64 sequences of 2048 to 8192 tokens, 32/8 heads of 128, 403 MB: 73 to 77 us and
// 5 for the join, 5.4 TB/s; the loads alone take 65, the instructions alone 50 (of
// about 310 a step and wave 128 make the values, as few as the format allows).
// 671 MB in sequences of one length: 114 us, 5.9 TB/s.  A short sequence is bound
// by one CU's instructions, 1 x 1000: 8.6 us.
#include "attn.hpp"
#include "kv_q4.hpp"

#include <algorithm>
#include <math.h>

namespace qmm {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 32;    // tokens of a step: two cells
constexpr float kLift = 15.0f;  // terms are 2^15 at most: f16 then keeps those down to 2^-39 of the largest

struct AttnQ4Args {
  const void* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  void* y;
  float* part;  // [slots][rows of a row block][D], then as many pairs (m, l)
  int64_t q_stride, pages, W;
  int64_t max_len;
  float scale;
  int window, B, n, Hq, Hk, group, rows, row_blocks, block_rows, cells;
  int slots;   // of partial results
  int groups;  // workgroups of equal runs; 0: parts
  int parts;   // the most of a sequence and head
  int least;   // the fewest steps of a run or part
  // a cell's page is cell * page_mul >> page_shift: right for cells below 2^31
  uint32_t page_mul, page_shift;
  bool bf16;
  int y_type;
};

// Eight codes of a dword -> the f16 numbers of bytes' low halves (0, 1), (2, 3) and high halves (0, 1), (2, 3).  (With a
// code or-ed into an f16's low bits and the offset subtracted: 13 instead of 11 instructions with the scales.)
__device__ __forceinline__ void codes(uint32_t w, h2 (&x)[4]) {
  const uint32_t low = w & 0x0f0f0f0fu, high = (w >> 4) & 0x0f0f0f0fu;
  x[0] = codes_to_f16<false>(low);
  x[1] = codes_to_f16<true>(low);
  x[2] = codes_to_f16<false>(high);
  x[3] = codes_to_f16<true>(high);
}

__device__ __forceinline__ h8 join(h2 a, h2 b, h2 c, h2 d) {
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <int K>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x150 + K, 0xf, 0xf, false));
}

// The cache is read past the device's caches: between two calls of a layer the
// other layers' caches and weights pass through these, and lines that are taken
// in push out what was written.  164 MB (8 x 16000) behind a pass over 1 GiB:
// 39 us, with ordinary loads 71; called again and again with nothing between,
// 403 MB: 79 and 85, and 82 MB, which the caches hold, 28 either way.
__device__ __forceinline__ uint32_t ld4_nt(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
}
__device__ __forceinline__ uint2 ld8_nt(const uint8_t* p) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  const v2u v = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(p));
  return make_uint2(v.x, v.y);
}

// How a head's NB blocks are dealt out: runs of four blocks (a lane has one), of two (half of one), single ones (a quarter).
template <int NB>
struct Runs {
  static constexpr int kQuads = NB / 4, kPair = (NB % 4) / 2, kOne = NB % 2, kScales = kQuads + kPair + kOne;
};

// One cell as loaded: this lane's key codes, their scales, the value codes of VB blocks, and its part of their scales.
template <int NB, int VB>
struct Cell {
  static constexpr int kVs = (4 * VB + 15) / 16;
  uint32_t k[NB], ks[Runs<NB>::kScales], v[VB], vs[kVs];

  __device__ __forceinline__ void load(const uint8_t* cell, int lane, int block) {
    constexpr int D = 32 * NB;
    const int key = lane & 15, c = lane >> 4;
#pragma unroll
    for (int r = 0; r < Runs<NB>::kQuads; ++r) {
      const uint4 x = ld16_nt(cell + r * 1024 + lane * 16);
      k[4 * r] = x.x, k[4 * r + 1] = x.y, k[4 * r + 2] = x.z, k[4 * r + 3] = x.w;
      ks[r] = ld4_nt(cell + 8 * D + r * 256 + lane * 4);
    }
    constexpr int kAt = 4 * Runs<NB>::kQuads;
    if constexpr (Runs<NB>::kPair) {
      const uint2 x = ld8_nt(cell + ((kAt + (c >> 1)) * 16 + key) * 16 + (c & 1) * 8);
      k[kAt] = x.x, k[kAt + 1] = x.y;
      ks[Runs<NB>::kQuads] = ld4_nt(cell + 8 * D + ((kAt + (c >> 1)) * 16 + key) * 4);
    }
    if constexpr (Runs<NB>::kOne) {
      k[NB - 1] = ld4_nt(cell + ((NB - 1) * 16 + key) * 16 + c * 4);
      ks[Runs<NB>::kScales - 1] = ld4_nt(cell + 8 * D + ((NB - 1) * 16 + key) * 4);
    }
    const uint8_t* values = cell + 10 * D + lane * (4 * NB) + 4 * block;
#pragma unroll
    for (int b = 0; b < VB;) {
      if constexpr (VB % 4 == 0) {
        const uint4 x = ld16_nt(values + 4 * b);
        v[b] = x.x, v[b + 1] = x.y, v[b + 2] = x.z, v[b + 3] = x.w;
        b += 4;
      } else if constexpr (VB % 2 == 0) {
        const uint2 x = ld8_nt(values + 4 * b);
        v[b] = x.x, v[b + 1] = x.y;
        b += 2;
      } else {
        v[b] = ld4_nt(values + 4 * b);
        b += 1;
      }
    }
#pragma unroll
    for (int r = 0; r < kVs; ++r) {
      const int at = 4 * block + min(r * 16 + key, 4 * VB - 1);
      vs[r] = ld4_nt(cell + 18 * D + (c * (4 * NB) + at) * 4);
    }
  }

  // The values' scales of tokens outside [lo, hi) of the cell as zeros: they may hold anything.
  __device__ __forceinline__ void clear_scales(int lane, int lo, int hi) {
#pragma unroll
    for (int r = 0; r < kVs; ++r) {
      const int t = 4 * (lane >> 4) + (lane & 1) * 2;
      vs[r] &= (t >= lo && t < hi ? 0xffffu : 0u) | (t + 1 >= lo && t + 1 < hi ? 0xffff0000u : 0u);
    }
  }

  // A operand of the products with the queries, number j.
  __device__ __forceinline__ h8 key_operand(int j) const {
    h2 x[4];
    codes(k[j], x);
    const int s = j < 4 * Runs<NB>::kQuads ? j / 4 : (Runs<NB>::kPair && j < 4 * Runs<NB>::kQuads + 2) ? Runs<NB>::kQuads
                                                                                                    : Runs<NB>::kScales - 1;
    const h2 dm = as_h2(ks[s]), d = {dm.x, dm.x}, m = {dm.y, dm.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __builtin_elementwise_fma(x[i], d, m);
    return join(x[0], x[1], x[2], x[3]);
  }

  // This cell's half of the A operands of block b's two tiles: dims c and c + 16, four tokens each.
  // The tokens of each quad come in the order 0, 2, 1, 3.
  template <int b>
  __device__ __forceinline__ void value_operands(h2 (&low)[2], h2 (&high)[2]) const {
    h2 x[4];
    codes(v[b], x);
    const uint32_t s = vs[b / 4];
    const h2 d02 = as_h2(row_bcast<b % 4 * 4>(s)), d13 = as_h2(row_bcast<b % 4 * 4 + 1>(s));
    const h2 m02 = as_h2(row_bcast<b % 4 * 4 + 2>(s)), m13 = as_h2(row_bcast<b % 4 * 4 + 3>(s));
    low[0] = __builtin_elementwise_fma(x[0], d02, m02);
    low[1] = __builtin_elementwise_fma(x[1], d13, m13);
    high[0] = __builtin_elementwise_fma(x[2], d02, m02);
    high[1] = __builtin_elementwise_fma(x[3], d13, m13);
  }

  // The values' scales as they are stored, tokens 0 and 1, then 2 and 3, in lanes next to each other -> 0 and 2, 1 and 3.
  __device__ __forceinline__ void pair_scales(int lane) {
    const uint32_t pick = (lane & 1) ? 0x03020706u : 0x05040100u;  // bytes of (other, own), own the low ones
#pragma unroll
    for (int r = 0; r < kVs; ++r) {
      const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(vs[r]), 0xb1, 0xf, 0xf, false));
      vs[r] = __builtin_amdgcn_perm(other, vs[r], pick);
    }
  }
};

// The dim at which the eight values of operand j begin in lane group c.
template <int NB>
__device__ __forceinline__ int operand_dim(int j, int c) {
  constexpr int kAt = 4 * Runs<NB>::kQuads;
  if (j < kAt) return (j / 4 * 4 + c) * 32 + j % 4 * 8;
  if (Runs<NB>::kPair && j < kAt + 2) return (kAt + (c >> 1)) * 32 + (c & 1) * 16 + (j - kAt) * 8;
  return (NB - 1) * 32 + c * 8;
}

template <int NB, int VB, int RT, int b = 0>
__device__ __forceinline__ void add_values(const Cell<NB, VB> (&cell)[2], const h8 (&p)[RT], v4f (&o)[RT][2 * VB]) {
  h2 l0[2], u0[2], l1[2], u1[2];
  cell[0].template value_operands<b>(l0, u0);
  cell[1].template value_operands<b>(l1, u1);
  const h8 low = join(l0[0], l0[1], l1[0], l1[1]), high = join(u0[0], u0[1], u1[0], u1[1]);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    o[r][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(low, p[r], o[r][2 * b], 0, 0, 0);
    o[r][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(high, p[r], o[r][2 * b + 1], 0, 0, 0);
  }
  if constexpr (b + 1 < VB) add_values<NB, VB, RT, b + 1>(cell, p, o);
}

// What a sequence and head costs besides its steps, in steps: it begins with three loads that wait for each other and ends
// with a join of the waves.  Where runs are equal without it a run over many short sequences takes the longest: 64 of 1 to
// 2000 tokens, 32/8 heads of 128: 55 us, with 3, 6, 10 and 16 more 40, 28, 26 and 26.
constexpr int kBetween = 12;

// A sequence's length, and the first key that any of its queries sees, in whole steps.
struct Extent {
  int len, floor_at, first, steps;  // at least one step, which writes the zeros of an empty sequence
};
__device__ __forceinline__ Extent extent_of(const AttnQ4Args& a, int32_t stored) {
  Extent e;
  e.len = static_cast<int>(max(int64_t{0}, min(a.max_len, static_cast<int64_t>(stored))));
  e.floor_at = a.window > 0 ? max(0, e.len - a.n - a.window + 1) : 0;
  e.first = e.floor_at / kStep * kStep;
  e.steps = max(1, (e.len - e.first + kStep - 1) / kStep);
  return e;
}

// Steps of one head and row block, summed over sequences by a wave, 64 of them at a time.
__device__ __forceinline__ int scan_steps(const AttnQ4Args& a, int b0, int lane, int& mine) {
  mine = b0 + lane < a.B ? extent_of(a, a.lens[min(b0 + lane, a.B - 1)]).steps + kBetween : 0;
  return wave_scan(mine);
}
// Of all sequences; `before`: of those before `seq`.
__device__ __forceinline__ int total_steps(const AttnQ4Args& a, int lane, int seq, int& before) {
  int total = 0, mine;
  before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int upto = scan_steps(a, b0, lane, mine);
    if (seq >= b0 && seq < b0 + 64) before = total + __builtin_amdgcn_readlane(upto - mine, seq - b0);
    total += __builtin_amdgcn_readlane(upto, 63);
  }
  return total;
}
// The sequence in which step `pos` of all heads' lies; `before`: the steps before it.
__device__ __forceinline__ int find_steps(const AttnQ4Args& a, int64_t pos, int lane, int& before) {
  const int64_t heads = static_cast<int64_t>(a.Hk) * a.row_blocks;
  before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int mine;
    const int upto = scan_steps(a, b0, lane, mine);
    const uint64_t here = __builtin_amdgcn_ballot_w64((before + upto) * heads > pos);
    if (here) {
      const int at = __builtin_ctzll(here);
      before += __builtin_amdgcn_readlane(upto - mine, at);
      return b0 + at;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return 0;
}

// In 32 bits where both numbers have no more: a quotient of 64 bits takes a hundred instructions.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(y) : x / y;
}
// The steps of a run.
__device__ __forceinline__ int64_t run_steps(const AttnQ4Args& a, int64_t total) {
  return max(static_cast<int64_t>(a.least), quotient(total + a.groups - 1, a.groups));
}

template <int VB, int kWaves>
struct AttnQ4Shared {
  float o[kWaves][16][32 * VB + 4];
  float m[kWaves][16], l[kWaves][16], mul[16];
};

// Steps `from` .. `to` of one sequence, key head and row block; `slot`: where a partial result goes, or -1 for a whole one.
struct Segment {
  int seq, kh, row_block, from, to;
  int64_t slot;
  Extent ext;
  int block = 0;  // the first of the values' blocks
};

// One segment after the other: next(s) moves s to the one behind it and tells
// whether there is one.  Its first loads begin before the results of the one
// before are joined and written.
template <int NB, int VB, int RT, int kWaves, typename Next>
__device__ __forceinline__ void attn_q4_run(const AttnQ4Args& a, AttnQ4Shared<VB, kWaves>& sh, Segment seg,
                                            const Next& next) {
  constexpr int D = 32 * NB;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, c = lane >> 4;
  const uint64_t cell_bytes = 20 * D, head_bytes = a.cells * cell_bytes, page_bytes = a.Hk * head_bytes;
  const auto page_of = [&](uint32_t cell) {
    return static_cast<uint32_t>(static_cast<uint64_t>(cell) * a.page_mul >> a.page_shift);
  };
  const auto there = [&](int page) { return static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages); };

  // one step's two cells and their page numbers
  struct Step {
    Cell<NB, VB> cell[2];
    int page[2];
  };
  // of the segment whose loads are under way
  scalar_ints pages;
  const uint8_t* head;
  uint32_t last_cell;  // nothing behind it is looked up or loaded
  const auto look_up = [&](int t, int (&page)[2]) {
#pragma unroll
    for (uint32_t u = 0; u < 2; ++u) page[u] = pages[page_of(min(static_cast<uint32_t>(t) / kCellTokens + u, last_cell))];
  };
  const auto load = [&](Step& s, int t, const int (&page)[2]) {
#pragma unroll
    for (uint32_t u = 0; u < 2; ++u) {
      const uint32_t cell = min(static_cast<uint32_t>(t) / kCellTokens + u, last_cell);
      const uint32_t pg = there(page[u]) ? page[u] : 0;
      s.cell[u].load(head + pg * page_bytes + (cell - page_of(cell) * a.cells) * static_cast<uint32_t>(cell_bytes), lane,
                     seg.block);
      s.page[u] = page[u];
    }
  };
  // Loads run one step ahead in the other buffer and look-ups two; behind the
  // end they repeat the last cell, so that every step waits for the same loads.
  const int stride = kWaves * kStep;
  int t, end;
  Step x, y;
  int page[2], ahead[2];
  v4u raw[RT][NB];  // the queries as stored
  const auto enter = [&]() {
    pages = as_scalar(a.table + static_cast<int64_t>(seg.seq) * a.W);
    head = a.cache + seg.kh * head_bytes;
    last_cell = static_cast<uint32_t>(max(0, seg.ext.len - 1)) / kCellTokens;
    end = min(seg.ext.len, seg.ext.first + seg.to * kStep);
    t = seg.ext.first + seg.from * kStep + wave * kStep;
    if (t < end) {
      look_up(t, page);
      look_up(t + stride, ahead);
      load(x, t, page);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = (seg.row_block * RT + r) * 16 + col;
      const bool on = row < a.rows;
      const int i = on ? row / a.group : a.n - 1, h = seg.kh * a.group + (on ? row % a.group : 0);
      const int64_t base = (static_cast<int64_t>(seg.seq) * a.n + i) * a.q_stride + static_cast<int64_t>(h) * D;
#pragma unroll
      for (int j = 0; j < NB; ++j)
        raw[r][j] = *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(a.q) + base + operand_dim<NB>(j, c));
    }
  };
  enter();

  for (;;) {
    const int len = seg.ext.len, floor_at = seg.ext.floor_at;

    // queries: this lane's row of each tile, its place, and what a product is multiplied with
    h8 q[RT][NB];
    float mul[RT];
    int at[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = (seg.row_block * RT + r) * 16 + col;
      at[r] = len - a.n + (row < a.rows ? row / a.group : a.n - 1);
      mul[r] = fabsf(a.scale) * kLog2e;
      if (!a.bf16) {
#pragma unroll
        for (int j = 0; j < NB; ++j) q[r][j] = __builtin_bit_cast(h8, raw[r][j]);
      } else {
        // a power of two for the row brings its largest value to 2^13: exact but for what lies 2^-27 below that; next to
        // an infinity the largest power keeps all other values finite
        float f[NB][8], top = 0.0f;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t w = raw[r][j][k >> 1];
            f[j][k] = __builtin_bit_cast(float, k & 1 ? w & 0xffff0000u : w << 16);
            top = fmaxf(top, fabsf(f[j][k]));
          }
        top = rows_max(top);
        const int e = top == 0.0f ? 0 : top < INFINITY ? __builtin_amdgcn_frexp_expf(top) - 14 : 128 - 14;
        mul[r] = __builtin_amdgcn_ldexpf(mul[r], e);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) q[r][j][k] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(f[j][k], -e));
      }
      // in the order of the keys' codes
#pragma unroll
      for (int j = 0; j < NB; ++j) q[r][j] = __builtin_shufflevector(q[r][j], q[r][j], 0, 4, 1, 5, 2, 6, 3, 7);
      // a factor above zero, so that the largest product is the largest score
      const _Float16 sign = static_cast<_Float16>(mul[r] == 0.0f ? 0.0f : a.scale < 0.0f ? -1.0f : 1.0f);
#pragma unroll
      for (int j = 0; j < NB; ++j) q[r][j] *= sign;
      mul[r] = mul[r] == 0.0f ? 1.0f : fminf(mul[r], FLT_MAX);
    }

    v4f o[RT][2 * VB];
    // the largest product so far, and this lane's part of the sum
    float top[RT], sum[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      top[r] = -INFINITY, sum[r] = 0.0f;
#pragma unroll
      for (int b = 0; b < 2 * VB; ++b) o[r][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const auto work = [&](Step& st, int t) {
      const bool there0 = there(st.page[0]), there1 = there(st.page[1]);
      // whether every query sees the whole step
      const bool whole = t + kStep <= len - a.n + 1 && t >= (a.window > 0 ? len - a.window : 0) && there0 && there1;
      v4f s[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r) s[r][0] = s[r][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const h8 k = st.cell[u].key_operand(j);
#pragma unroll
          for (int r = 0; r < RT; ++r) s[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[r][j], s[r][u], 0, 0, 0);
        }
      if (!whole) {
        const int lo = floor_at - t, hi = len - t;
        st.cell[0].clear_scales(lane, there0 ? lo : 16, hi);
        st.cell[1].clear_scales(lane, there1 ? lo - 16 : 16, hi - 16);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int j = t + (k >> 2) * kCellTokens + 4 * c + (k & 3);
            const bool seen = j <= at[r] && (a.window == 0 || j > at[r] - a.window) && (k < 4 ? there0 : there1);
            s[r][k >> 2][k & 3] = seen ? s[r][k >> 2][k & 3] : -INFINITY;
          }
      }
      st.cell[0].pair_scales(lane);
      st.cell[1].pair_scales(lane);
      h8 p[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float most = top[r];
#pragma unroll
        for (int k = 0; k < 8; ++k) most = fmaxf(most, s[r][k >> 2][k & 3]);
        most = rows_max(most);
        const float zero = most == -INFINITY ? 0.0f : most;
        if (__builtin_amdgcn_ballot_w64(most > top[r])) {
          const float keep = __builtin_amdgcn_exp2f((top[r] - zero) * mul[r]);
          sum[r] *= keep;
#pragma unroll
          for (int b = 0; b < 2 * VB; ++b) o[r][b] *= keep;
          top[r] = most;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][k >> 2][k & 3] - zero, mul[r], kLift));
          sum[r] += e;
          p[r][(k & 4) + kv_quad_byte(k & 3)] = static_cast<_Float16>(e);
        }
      }
      add_values<NB, VB, RT>(st.cell, p, o);
    };

    if (t < end) {
      // in pairs, with no way out between the two: each step then waits for its own loads alone
      const int steps = (end - t + stride - 1) / stride;
      for (int k = 1; k < steps; k += 2) {
        load(y, t + stride, ahead);
        look_up(t + 2 * stride, ahead);
        __builtin_amdgcn_sched_barrier(0);  // all of these before the work, not sunk to their use
        work(x, t);
        load(x, t + 2 * stride, ahead);
        look_up(t + 3 * stride, ahead);
        __builtin_amdgcn_sched_barrier(0);
        work(y, t + stride);
        t += 2 * stride;
      }
      if (steps & 1) work(x, t);
    }

    const Segment done = seg;
    const bool more = next(seg);
    if (more) enter();

    // join the waves, tile by tile, and write
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float l = rows_sum(sum[r]);
      if (c == 0) sh.m[wave][col] = top[r], sh.l[wave][col] = l;
      if (wave == 0 && c == 0) sh.mul[col] = mul[r];
#pragma unroll
      for (int b = 0; b < 2 * VB; ++b) *reinterpret_cast<v4f*>(&sh.o[wave][col][b * 16 + 4 * c]) = o[r][b];
      __syncthreads();
      const int row0 = (done.row_block * RT + r) * 16, rows = min(16, a.rows - row0);
      for (int x = threadIdx.x; x < rows * (8 * VB); x += 64 * kWaves) {
        const int row = x / (8 * VB), d = x % (8 * VB) * 4;
        float m = sh.m[0][row];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sh.m[w][row]);
        const float zero = m == -INFINITY ? 0.0f : m, mul = sh.mul[row];
        float total = 0.0f;
        v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f((sh.m[w][row] - zero) * mul);
          total += sh.l[w][row] * f;
          y += *reinterpret_cast<const v4f*>(&sh.o[w][row][d]) * f;
        }
        if (done.slot >= 0) {
          const int64_t at_row = done.slot * a.block_rows + r * 16 + row;
          *reinterpret_cast<v4f*>(a.part + at_row * D + d) = y;
          if (d == 0) {
            // the product of the keys with the query as it was, without its power of two
            const int e = __builtin_amdgcn_frexp_expf(mul) - __builtin_amdgcn_frexp_expf(exponent_mul(a.scale));
            reinterpret_cast<float2*>(a.part + static_cast<int64_t>(a.slots) * a.block_rows * D)[at_row] =
                make_float2(__builtin_amdgcn_ldexpf(m, e), total);
          }
        } else {
          const int i = (row0 + row) / a.group, h = done.kh * a.group + (row0 + row) % a.group;
          const int64_t out = (static_cast<int64_t>(done.seq) * a.n + i) * a.Hq + h;
          y *= total == 0.0f ? 0.0f : 1.0f / total;
          store4(a.y_type, a.y, (out * D + 32 * done.block + d) / 4, make_float4(y.x, y.y, y.z, y.w));
        }
      }
      __syncthreads();
    }
    if (!more) break;
  }
}

// One workgroup for each sequence, key head and VB blocks of the values (which vary slowest): no partial results.
template <int NB, int VB, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void attn_q4_kernel(AttnQ4Args a) {
  __shared__ AttnQ4Shared<VB, kWaves> sh;
  const unsigned items = static_cast<unsigned>(a.B) * a.Hk, item = blockIdx.x % items, part = blockIdx.x / items;
  const int kh = item % a.Hk, seq = item / a.Hk;
  const Extent e = extent_of(a, as_scalar(a.lens)[seq]);
  attn_q4_run<NB, VB, 1, kWaves>(a, sh, Segment{seq, kh, 0, 0, e.steps, -1, e, static_cast<int>(part) * VB},
                                 [](Segment&) { return false; });
}

// The parts of a sequence of so many steps.
__device__ __forceinline__ int parts_of(const AttnQ4Args& a, int steps) { return min(a.parts, (steps + a.least - 1) / a.least); }

// Equal parts of a sequence and head each.  The parts vary slowest: the first ones, which every sequence has, over all dies.
template <int NB, int RT, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void attn_q4_parts_kernel(AttnQ4Args a) {
  __shared__ AttnQ4Shared<NB, kWaves> sh;
  const unsigned heads = a.Hk * a.row_blocks, items = a.B * heads, item = blockIdx.x % items, seq = item / heads;
  const int part = blockIdx.x / items, head = item % heads;
  const Extent e = extent_of(a, as_scalar(a.lens)[seq]);
  const int parts = parts_of(a, e.steps);
  if (part >= parts) return;
  const int each = static_cast<unsigned>(e.steps) / parts, more = e.steps - each * parts;  // the first ones have one more
  const int from = part * each + min(part, more), to = from + each + (part < more ? 1 : 0);
  attn_q4_run<NB, NB, RT, kWaves>(a, sh,
                              Segment{static_cast<int>(seq), head / a.row_blocks, head % a.row_blocks, from, to,
                                      parts == 1 ? -1 : int64_t{blockIdx.x}, e},
                              [](Segment&) { return false; });
}

// Equal runs of the steps of all, and of what stands for the beginning and end of each item.
template <int NB, int RT, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void attn_q4_runs_kernel(AttnQ4Args a) {
  __shared__ AttnQ4Shared<NB, kWaves> sh;
  const int lane = threadIdx.x & 63, heads = a.Hk * a.row_blocks;
  int before;
  const int64_t total = static_cast<int64_t>(total_steps(a, lane, 0, before)) * heads, per = run_steps(a, total);
  const int64_t first = blockIdx.x * per;
  int64_t left = min(total - first, per);  // steps of the run
  if (left <= 0) return;
  int seq = find_steps(a, first, lane, before);
  Extent e = extent_of(a, as_scalar(a.lens)[seq]);
  const int64_t in = first - static_cast<int64_t>(before) * heads;
  int head = static_cast<int>(quotient(in, e.steps + kBetween));
  int from = static_cast<int>(in - static_cast<int64_t>(head) * (e.steps + kBetween));
  int64_t slot = 2 * int64_t{blockIdx.x};  // of the run's first item; then of the last one, should it not be whole
  // the run's next item with steps in it
  const auto next = [&](Segment& s) {
    while (left > 0) {
      const int to = static_cast<int>(min(static_cast<int64_t>(e.steps + kBetween), from + left)), end = min(to, e.steps);
      const bool any = from < e.steps;
      if (any) {
        const bool whole = from == 0 && end == e.steps;
        s = Segment{seq, head / a.row_blocks, head % a.row_blocks, from, end, whole ? -1 : slot, e};
      }
      left -= to - from;
      slot = 2 * int64_t{blockIdx.x} + 1;
      from = 0;
      if (left > 0 && ++head == heads) {
        head = 0;
        e = extent_of(a, as_scalar(a.lens)[++seq]);
      }
      if (any) return true;
    }
    return false;
  };
  Segment s;
  if (next(s)) attn_q4_run<NB, NB, RT, kWaves>(a, sh, s, next);
}

// Joins the partial results of one row, a wave each.
__global__ __launch_bounds__(64) void attn_q4_join_kernel(AttnQ4Args a, int D) {
  const int lane = threadIdx.x, h = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq % a.n, seq = blockIdx.x / a.Hq / a.n;
  const int row = i * a.group + h % a.group, in = row % a.block_rows, heads = a.Hk * a.row_blocks;
  const int head = h / a.group * a.row_blocks + row / a.block_rows;
  const int steps = extent_of(a, as_scalar(a.lens)[seq]).steps;
  int64_t first, second, step;  // the slots: the first, and the others' beginning and distance
  int count;
  if (a.groups == 0) {
    count = parts_of(a, steps);
    step = static_cast<int64_t>(a.B) * heads;
    first = static_cast<int64_t>(seq) * heads + head;
    second = first + step;
  } else {
    int before;
    const int64_t per = run_steps(a, static_cast<int64_t>(total_steps(a, lane, seq, before)) * heads);
    const int64_t begin = static_cast<int64_t>(before) * heads + static_cast<int64_t>(head) * (steps + kBetween);
    const int64_t g0 = quotient(begin, per), g1 = quotient(begin + steps - 1, per);
    count = static_cast<int>(g1 - g0 + 1);
    // the first run's second result, unless the run begins with it; the others' first
    first = 2 * g0 + (begin == g0 * per ? 0 : 1);
    second = 2 * (g0 + 1);
    step = 2;
  }
  if (count == 1) return;  // whole, and written
  const float2* ml = reinterpret_cast<const float2*>(a.part + static_cast<int64_t>(a.slots) * a.block_rows * D);
  const v4f y = Parts([&](int k) { return (k == 0 ? first : second + (k - 1) * step) * a.block_rows + in; },
                      a.part + min(lane * 4, D - 4), D, ml, count, lane).join(exponent_mul(a.scale));
  const int64_t out = blockIdx.x;
  if (lane * 4 < D) store4(a.y_type, a.y, (out * D + lane * 4) / 4, make_float4(y.x, y.y, y.z, y.w));
}

// How a call is cut, from the sizes that the host knows.
struct AttnQ4Plan {
  int waves, tiles, row_blocks;
  int groups, parts, least;  // all 0: whole sequences
  int64_t slots;
};

// The longest sequences that are taken whole, in tokens: one launch.  32/8 heads
// of 128, 1 x 1000: 8.6 us in a graph and 10 a call by itself; as parts 8.5 and
// 14.3; 32 x 1000: 11.8 and, as parts, 16.2 in a graph; 1 x 2000: 12.1 and 9.6.
constexpr int64_t kWhole = 1024;
// Two workgroups per CU.  With three 64 sequences of 1 to 8192 tokens take 64 us for 61, of 8192 119 for 114, and 16 x
// 4096 with 64 rows a key head 71 for 50.
constexpr int kGroups = 512;
constexpr int64_t kLeast = 8;  // steps: two a wave
// Parts: one workgroup per CU, two where a part would be longer than this, in
// steps.  32/8 heads of 128, two and one: 1 x 16000 18.5 and 14.7 us, 31 x 2000
// 20.8 and 18.5; 8 x 16000 behind a pass over 1 GiB 40 and 42.5.
constexpr int64_t kLongPart = 100;
constexpr int64_t kMostParts = 32;  // the join takes them in order: 1 x 128000 39.5 us, with 64 41.3
// Whole sequences that leave most CUs without work: one workgroup for each block
// or two of the values, all of which find the scores for themselves.  1 x 1000,
// 32/8 heads of 128: 8.6 us, in one workgroup per key head 10.2; 32/4 of 256: 12.3
// and 17.0.  With 16 waves 9.3 and (spilt) 24.6.
constexpr unsigned kFew = 256;

static AttnQ4Plan attn_q4_plan(int64_t B, int64_t n, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  AttnQ4Plan p{4, 1, 1, 0, 0, 0, 0};
  const int64_t rows = n * (Hq / Hk), most = D > 128 ? 2 : 4;
  p.tiles = static_cast<int>(rows <= 16 ? 1 : rows <= 32 ? 2 : most);
  p.row_blocks = static_cast<int>((rows + 16 * p.tiles - 1) / (16 * p.tiles));
  const int64_t items = B * Hk * p.row_blocks, steps = (max_len + kStep - 1) / kStep + 1;
  if (rows <= 16 && max_len <= kWhole) {
    p.waves = 8;
    return p;
  }
  p.least = static_cast<int>(kLeast);
  if (items >= kGroups / 2) {
    p.groups = static_cast<int>(std::min<int64_t>(kGroups, (items * steps + kLeast - 1) / kLeast));
    p.slots = 2 * p.groups;
  } else {
    const int64_t one = std::max<int64_t>(1, kGroups / 2 / std::max<int64_t>(1, items));
    const int64_t most = one * kLongPart < steps ? 2 * one : one;
    p.parts = static_cast<int>(std::min({most, (steps + kLeast - 1) / kLeast, kMostParts}));
    p.slots = p.parts == 1 ? 0 : items * p.parts;
  }
  return p;
}

template <int NB, int RT>
static void launch_split(const AttnQ4Args& a, dim3 g, hipStream_t st) {
  if (a.groups) hipLaunchKernelGGL((attn_q4_runs_kernel<NB, RT, 4>), g, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((attn_q4_parts_kernel<NB, RT, 4>), g, dim3(256), 0, st, a);
}
template <int NB>
static void launch_attn_q4(const AttnQ4Args& a, const AttnQ4Plan& p, hipStream_t st) {
  const unsigned items = static_cast<unsigned>(a.B) * a.Hk * a.row_blocks;
  const dim3 g(p.groups ? static_cast<unsigned>(p.groups) : items * p.parts);
  constexpr int VB = NB <= 4 ? 1 : 2;
  if (p.waves == 8) {
    if (items * (NB / VB) <= kFew)
      hipLaunchKernelGGL((attn_q4_kernel<NB, VB, 8>), dim3(items * (NB / VB)), dim3(512), 0, st, a);
    else
      hipLaunchKernelGGL((attn_q4_kernel<NB, NB, 8>), dim3(items), dim3(512), 0, st, a);
  } else if (p.tiles == 1) {
    launch_split<NB, 1>(a, g, st);
  } else if (p.tiles == 2 || NB > 4) {
    launch_split<NB, 2>(a, g, st);
  } else {
    launch_split<NB, NB <= 4 ? 4 : 2>(a, g, st);
  }
}

// A grid has to stay below 2^32 lanes, with up to 512 a sequence and key head.
static bool attn_q4_shape(int64_t B, int64_t n, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  return B >= 0 && n >= 1 && n <= QMM_ATTN_MAX_N && Hk >= 1 && Hq >= Hk && Hq <= 1024 && Hq % Hk == 0 &&
         attn_head_dim(D) && max_len >= 1 && max_len <= kMostTokens && B < (int64_t{1} << 23) / (n * Hq) &&
         B * ((max_len + kStep - 1) / kStep + 1 + kBetween) < (int64_t{1} << 31);
}

}  // namespace qmm

using namespace qmm;

extern "C" size_t attn_q4_workspace_bytes(int64_t B, int64_t n, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  if (!attn_q4_shape(B, n, Hq, Hk, D, max_len)) return 0;
  const AttnQ4Plan p = attn_q4_plan(B, n, Hq, Hk, D, max_len);
  return static_cast<size_t>(p.slots) * (16 * p.tiles) * (D + 2) * 4;
}

extern "C" int attn_q4(const void* q, int64_t q_stride, int type, const void* cache, int64_t pages, int64_t page,
                       const int32_t* table, int64_t W, const int32_t* lens, float scale, int64_t window, void* y,
                       int y_type, int64_t B, int64_t n, int64_t Hq, int64_t Hk, int64_t D, void* ws, size_t ws_bytes,
                       void* stream) {
  if ((type != QMM_F16 && type != QMM_BF16) || !known_type(y_type)) return QMM_ERR_UNSUPPORTED;
  if (!kv_q4_shape(pages, page, Hk, D) || W < 1 || W > kMostTokens / page) return QMM_ERR_SHAPE;
  if (!attn_q4_shape(B, n, Hq, Hk, D, W * page) || !strided_rows(q_stride, Hq, D)) return QMM_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || window > 0x7fffffff) return QMM_ERR_SHAPE;
  if (B == 0) return QMM_OK;
  const size_t need = attn_q4_workspace_bytes(B, n, Hq, Hk, D, W * page);
  if (!q || !cache || !table || !lens || !y || (need > 0 && !ws)) return QMM_ERR_NULL;
  if (!aligned16(q) || !aligned16(cache) || !aligned_list(table, 4) || !aligned_list(lens, 4) || !aligned16(y) || !aligned16(ws))
    return QMM_ERR_ALIGN;
  if (ws_bytes < need) return QMM_ERR_WORKSPACE;
  const AttnQ4Plan p = attn_q4_plan(B, n, Hq, Hk, D, W * page);
  const int cells = static_cast<int>(page / kCellTokens);
  uint32_t shift = 31;
  while ((int64_t{1} << (shift - 31)) < cells) ++shift;
  const AttnQ4Args a{q, static_cast<const uint8_t*>(cache), table, lens, y, static_cast<float*>(ws), q_stride, pages, W,
                     W * page, scale, static_cast<int>(std::min(window, kMostTokens)), static_cast<int>(B), static_cast<int>(n),
                     static_cast<int>(Hq), static_cast<int>(Hk), static_cast<int>(Hq / Hk),
                     static_cast<int>(n * (Hq / Hk)), p.row_blocks, 16 * p.tiles, cells,
                     static_cast<int>(p.slots), p.groups, p.parts, p.least,
                     static_cast<uint32_t>(((uint64_t{1} << shift) + cells - 1) / cells), shift, type == QMM_BF16, y_type};
  hipStream_t st = to_stream(stream);
  switch (D) {
    case 64: launch_attn_q4<2>(a, p, st); break;
    case 96: launch_attn_q4<3>(a, p, st); break;
    case 128: launch_attn_q4<4>(a, p, st); break;
    case 192: launch_attn_q4<6>(a, p, st); break;
    default: launch_attn_q4<8>(a, p, st); break;
  }
  if (p.slots > 0)
    hipLaunchKernelGGL(attn_q4_join_kernel, dim3(static_cast<unsigned>(B * n * Hq)), dim3(64), 0, st, a,
                       static_cast<int>(D));
  return launch_status();
}
