// fp8_core.hpp -- device code of the products over 8-bit weights: one wave's
// share of Y = X . W^T for a few rows of W, W in OCP e4m3 with one fp32 scale
// for each 128 x 128 block.
//
//   Y[t][n] = sum_b s[n / 128][b] * (sum_{c in block b} X[t][c] * W[n][c])
//
// Every value of e4m3 is a bf16 value, so codes (the weights', and those of
// e4m3 activations, which have one more scale for each 128 columns of a
// token) are widened in registers and multiplied by the bf16 matrix
// instruction: products exact, sums in fp32.  The 8-bit matrix instructions
// do not keep fp32 sums: over 128 random codes they were up to 2^-13 of
// sum |x w| off (mean 9e-6), the bf16 one 2^-22 (1.2e-8); the rate they would
// add is not what bounds a product of at most 64 tokens.  The sum of one
// 128-column block is taken on its own and enters the running fp32 sum with
// one fused multiply-add by its scale.
//
// Reading.  A tile is 16 weight rows.  One load instruction takes 8 rows x
// 128 bytes, eight lanes to a row: a compute unit takes in 116 bytes/ns of
// such loads (from L2), but 37 of the same bytes when neighbouring lanes hold
// different rows, as the matrix operand wants them.  So what is loaded goes
// through LDS -- a buffer of the wave's own, no barrier -- and is read back as
// the operand: lane l = R + 16 g holds columns 32 g .. 32 g + 31 of row R.
// Activations of more than 8 tokens, and of 5 to 8 over a long row, take the
// same way.  Within a row of the buffer the 16-byte pieces are permuted by
// exclusive or with a number of the row (swizzle128, swizzle256,
// swizzle_packed), so that the lanes of a read that are served together meet
// different banks.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kQBlock = 128;   // columns (and weight rows) that share a scale

// Token layouts of the activation operand.
//   XP4:  bf16, up to 4 tokens.  One 16-byte load per block, straight to the
//         operand's registers: matrix column 4 t + j holds token t's piece j
//         (8 of the lane group's 32 values).  Step j of the block multiplies
//         the columns that hold piece j, the others as zeros, so the four
//         columns of a token add up to its sum.
//   XP8:  bf16, up to 8 tokens, two loads: column 2 t + (j & 1).
//   XP8L: the same columns through LDS: two loads of 4 tokens x 256 bytes, not
//         of 32 bytes of a token to a lane pair.  For rows of several steps:
//         57344 x 7168, 8 tokens, 80 us with XP8, 75.5 with XP8L (2 blocks in
//         flight); 7168 x 2048, 6 tokens, all requested at once, 5.7 and 5.8;
//         gate/up of 64 tokens 2 % more.
//   XB:   bf16, NT tiles of 16 tokens, through LDS: four loads of 4 tokens x
//         256 bytes per tile.
//   X8P:  e4m3, up to 8 tokens, one load: column 2 t + i holds the lane
//         group's half i (pieces 2 i and 2 i + 1).
//   X8:   e4m3, NT tiles of 16 tokens, through LDS: two loads of 8 tokens x
//         128 bytes per tile.
// A token packed in 4 columns costs a quarter of the registers that a column
// of its own would, which is what lets a wave request all its blocks at once.
enum XKind { XP4 = 0, XP8 = 1, XB = 2, X8P = 3, X8 = 4, XP8L = 5 };

constexpr bool x_e4m3(int xk) { return xk == X8P || xk == X8; }

// kLoads: 16-byte loads per tile and block; kTokens: tokens of a tile;
// kCols: matrix columns of a token; kLds: LDS bytes of a tile.
template <int XK> struct XTraits;
template <> struct XTraits<XP4> { static constexpr int kLoads = 1, kTokens = 4, kCols = 4, kLds = 0; };
template <> struct XTraits<XP8> { static constexpr int kLoads = 2, kTokens = 8, kCols = 2, kLds = 0; };
template <> struct XTraits<XP8L> { static constexpr int kLoads = 2, kTokens = 8, kCols = 2, kLds = 2048; };
template <> struct XTraits<XB> { static constexpr int kLoads = 4, kTokens = 16, kCols = 1, kLds = 4096; };
template <> struct XTraits<X8P> { static constexpr int kLoads = 1, kTokens = 8, kCols = 2, kLds = 0; };
template <> struct XTraits<X8> { static constexpr int kLoads = 2, kTokens = 16, kCols = 1, kLds = 2048; };

// LDS of one wave: a block of its weight tiles and one token tile (tile after
// tile through the same bytes), later its sums.
template <int XK, int RT, int NT>
constexpr int fp8_wave_lds() {
  constexpr int in = RT * 2048 + XTraits<XK>::kLds, out = RT * NT * 1024;
  return in > out ? in : out;
}

// Token of this lane's matrix column within its tile.
template <int XK>
__device__ __forceinline__ int x_column_token(int lane) {
  return (lane & 15) / XTraits<XK>::kCols;
}
// Token whose values this lane requests with load i.
template <int XK>
__device__ __forceinline__ int x_load_token(int lane, int i) {
  if constexpr (XK == XB || XK == XP8L) return 4 * i + (lane >> 4);
  else if constexpr (XK == X8) return 8 * i + (lane >> 3);
  else return x_column_token<XK>(lane);
}
// Distinct tokens among a lane's loads of a tile.
template <int XK>
constexpr int x_rows() { return XTraits<XK>::kLds ? XTraits<XK>::kLoads : 1; }

// Loads go through buffer descriptors: an offset past their end (kNoLoad and
// more) reads zeros and asks nothing of memory, which is how rows, tokens and
// columns that are not there are left out without a branch.
typedef __amdgpu_buffer_rsrc_t buffer_t;
constexpr uint32_t kNoLoad = 0x80000000u;
constexpr int kNonTemporal = 2;   // cache policy: weights are read once
__device__ __forceinline__ buffer_t buffer_of(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7fffffff, 0x00020000);
}

// Where a wave reads: per lane, byte offsets from uniform bases.
template <int XK, int RT, int NT>
struct Fp8Src {
  buffer_t w[RT];           // from the tile's weight base
  uint32_t ra[RT], rb[RT];  // byte offset of row lane / 8 among the tile's rows 0-7, and among its rows 8-15, or kNoLoad
  const float* sa[RT];      // scales of the block row that holds the tile's row 0 (uniform), [blocks]
  const float* sb[RT];      // and of that of the rows of the upper lanes (row_b)
  bool row_b[RT];           // the lane's result rows take sb
  buffer_t x;               // activations
  uint32_t xo[NT][x_rows<XK>()];   // byte offset of the token row of each load, or kNoLoad
  const float* xs;          // e4m3: scales (uniform)
  uint32_t xso[NT];         // e4m3: index of the first scale of the lane's column's token
  int K;
  int lane;   // of the wave; own_lane()
};

// The lane, as a value that the compiler takes for new: what is computed from
// it (a dozen offsets) stays inside the loop over tasks, where registers are
// free, and is not carried through the routing code ahead of it.
__device__ __forceinline__ int own_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// 8 codes (two words) as 8 bf16: exact, NaN stays NaN.
__device__ __forceinline__ bf16x8 widen8(uint32_t w0, uint32_t w1) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// LDS serves a 128-bit read 16 lanes (all 64 banks) at a time, and those are
// lanes 0-3, 12-15 and 20-27, then 4-11, 16-19 and 28-31, then the same 32
// higher (measured: two lanes of one group on the same banks take longer).  As
// operand reads that is rows 0-3 and 12-15 of one lane group with rows 4-11 of
// its neighbour, whose pieces differ in bit 1 (128-byte rows, two to a round
// of the banks) or bit 2 (256-byte rows): the numbers of the former rows have
// to be a set that this bit maps onto itself.  Permuted by the row's low bits
// alone a read took 8.2 cycles, so 5.0; 1536 x 7168, 64 tokens: 13.7 -> 13.5 us.
__device__ __forceinline__ int swizzle128(int row) {
  const int r = row >> 1;
  return r ^ ((r & 2) << 1);   // of row + 8: the same with bit 2 flipped
}
__device__ __forceinline__ int swizzle256(int row) { return row ^ ((row & 4) << 1); }
__device__ __forceinline__ int swizzle_packed(int t) { return 2 * (t ^ ((t & 2) << 1)); }   // of 8 rows, pairs of pieces

// 16 rows x 128 bytes through LDS: rows lane / 8 (a) and 8 + lane / 8 (b),
// piece lane % 8, in; row lane % 16, pieces 2 g and 2 g + 1 out.  One wave's
// LDS accesses are served in order, so no wait stands between them.
__device__ __forceinline__ void rows128_store(int lane, char* lds, u32x4 a, u32x4 b) {
  const int i = (lane & ~7) | ((lane & 7) ^ swizzle128(lane >> 3));
  reinterpret_cast<u32x4*>(lds)[i] = a;
  reinterpret_cast<u32x4*>(lds)[64 + (i ^ 4)] = b;
}
__device__ __forceinline__ void rows128_load(int lane, const char* lds, u32x4& lo, u32x4& hi) {
  const int R = lane & 15, g = lane >> 4;
  const u32x4* p = reinterpret_cast<const u32x4*>(lds) + R * 8;
  lo = p[(2 * g) ^ swizzle128(R)];
  hi = p[(2 * g + 1) ^ swizzle128(R)];
}
// 16 rows x 256 bytes: row 4 i + lane / 16, piece lane % 16, in; row
// lane % 16, piece 4 g + j out.
__device__ __forceinline__ void rows256_store(int lane, char* lds, int i, u32x4 v) {
  const int t = 4 * i + (lane >> 4);
  reinterpret_cast<u32x4*>(lds)[t * 16 + ((lane & 15) ^ swizzle256(t))] = v;
}
__device__ __forceinline__ u32x4 rows256_load(int lane, const char* lds, int j) {
  const int t = lane & 15, g = lane >> 4;
  return reinterpret_cast<const u32x4*>(lds)[t * 16 + ((4 * g + j) ^ swizzle256(t))];
}

// 8 rows x 256 bytes: row 4 i + lane / 16, piece lane % 16, in; row
// (lane % 16) / 2, piece 4 g + 2 i + lane % 2 out.
__device__ __forceinline__ void packed256_store(int lane, char* lds, int i, u32x4 v) {
  const int t = 4 * i + (lane >> 4);
  reinterpret_cast<u32x4*>(lds)[t * 16 + ((lane & 15) ^ swizzle_packed(t))] = v;
}
__device__ __forceinline__ u32x4 packed256_load(int lane, const char* lds, int i) {
  const int t = (lane & 15) >> 1, g = lane >> 4;
  return reinterpret_cast<const u32x4*>(lds)[t * 16 + ((4 * g + 2 * i + (lane & 1)) ^ swizzle_packed(t))];
}

// Registers of one K block of a wave.
template <int XK, int RT, int NT>
struct Fp8Block {
  u32x4 a[RT], b[RT];
  u32x4 x[NT][XTraits<XK>::kLoads];
  float xs[NT];
};

// Request block kb; what lies past K, all of a block past the last, is zeros.
template <int XK, int RT, int NT>
__device__ __forceinline__ void fp8_load(const Fp8Src<XK, RT, NT>& s, int kb, Fp8Block<XK, RT, NT>& r) {
  const int lane = s.lane, g = lane >> 4;
  const uint32_t k0 = (uint32_t)kb * kQBlock, K = (uint32_t)s.K;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < XTraits<XK>::kLoads; ++i) {
      uint32_t c = k0;   // column of the lane's 16 bytes
      if constexpr (XK == XP4) c += 32 * g + 8 * (lane & 3);
      else if constexpr (XK == XP8) c += 32 * g + 16 * i + 8 * (lane & 1);
      else if constexpr (XK == XP8L || XK == XB) c += 8 * (lane & 15);
      else if constexpr (XK == X8P) c += 32 * g + 16 * (lane & 1);
      else c += 16 * (lane & 7);
      const uint32_t o = s.xo[nt][x_rows<XK>() > 1 ? i : 0] + (x_e4m3(XK) ? c : 2 * c);
      r.x[nt][i] = __builtin_amdgcn_raw_buffer_load_b128(s.x, c < K ? o : kNoLoad, 0, 0);
    }
    if constexpr (x_e4m3(XK)) {
      const uint32_t last = (K - 1) / kQBlock;
      r.xs[nt] = s.xs[s.xso[nt] + ((uint32_t)kb < last ? (uint32_t)kb : last)];
    }
  }
  const uint32_t c = k0 + 16 * (lane & 7);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    r.a[rt] = __builtin_amdgcn_raw_buffer_load_b128(s.w[rt], c < K ? s.ra[rt] + c : kNoLoad, 0, kNonTemporal);
    r.b[rt] = __builtin_amdgcn_raw_buffer_load_b128(s.w[rt], c < K ? s.rb[rt] + c : kNoLoad, 0, kNonTemporal);
  }
}

// acc += the block's products, each tile's by its scale sc[rt].  lds: the
// wave's buffer.
template <int XK, int RT, int NT>
__device__ __forceinline__ void fp8_block(int lane, const Fp8Block<XK, RT, NT>& r, const float (&sc)[RT], char* lds,
                                          f32x4 (&acc)[RT][NT]) {
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const f32x4 fzero = {0.f, 0.f, 0.f, 0.f};
  char* xl = lds + RT * 2048;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) rows128_store(lane, lds + rt * 2048, r.a[rt], r.b[rt]);
  // Step j's operands are made where they are used: kept apart for all four
  // steps they cost the registers of a block in flight.
  u32x4 h[NT][4];   // bf16: piece j in h[j] (packed: piece 0's, or 0 and 1's, load); e4m3: the group's halves in h[0], h[1]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if constexpr (XK == XB) {
#pragma unroll
      for (int i = 0; i < 4; ++i) rows256_store(lane, xl, i, r.x[nt][i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[nt][j] = rows256_load(lane, xl, j);
    } else if constexpr (XK == XP8L) {
#pragma unroll
      for (int i = 0; i < 2; ++i) packed256_store(lane, xl, i, r.x[nt][i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) h[nt][i] = packed256_load(lane, xl, i);
    } else if constexpr (XK == X8) {
      rows128_store(lane, xl, r.x[nt][0], r.x[nt][1]);
      rows128_load(lane, xl, h[nt][0], h[nt][1]);
    } else {
#pragma unroll
      for (int i = 0; i < XTraits<XK>::kLoads; ++i) h[nt][i] = r.x[nt][i];
    }
  }
  auto x_step = [&](int nt, int j) {
    if constexpr (x_e4m3(XK)) {
      const u32x4 v = h[nt][XK == X8 ? j >> 1 : 0];
      const bool mine = XK == X8 || (lane & 1) == (j >> 1);
      const uint32_t w0 = v[2 * (j & 1)], w1 = v[2 * (j & 1) + 1];
      return widen8(mine ? w0 : 0u, mine ? w1 : 0u);
    } else if constexpr (XK == XP4) {
      return __builtin_bit_cast(bf16x8, (lane & 3) == j ? h[nt][0] : zero);
    } else if constexpr (XK == XP8 || XK == XP8L) {
      return __builtin_bit_cast(bf16x8, (lane & 1) == (j & 1) ? h[nt][j >> 1] : zero);
    } else {
      return __builtin_bit_cast(bf16x8, h[nt][j]);
    }
  };
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    u32x4 lo, hi;
    rows128_load(lane, lds + rt * 2048, lo, hi);
    f32x4 d[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) d[nt] = fzero;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 q = j < 2 ? lo : hi;
      const bf16x8 wj = widen8(q[2 * (j & 1)], q[2 * (j & 1) + 1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) d[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wj, x_step(nt, j), d[nt], 0, 0, 0);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float f = x_e4m3(XK) ? sc[rt] * r.xs[nt] : sc[rt];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[rt][nt][i] = __builtin_fmaf(f, d[nt][i], acc[rt][nt][i]);
    }
  }
}

// Wave `wave` of `waves` over all of K: in step s it takes blocks
// (s * waves + wave) * U .. + U - 1, all U requested before any is used and
// each block's registers refilled for the next step as soon as it is.  The
// scales of a step come with one load (lanes 0.. the first block row's, lanes
// 32.. the second's) and are read out lane by lane.
template <int XK, int RT, int NT, int U>
__device__ __forceinline__ void fp8_wave(const Fp8Src<XK, RT, NT>& s, int wave, int waves, char* lds,
                                         f32x4 (&acc)[RT][NT]) {
  const int lane = s.lane;
  const int KB = (s.K + kQBlock - 1) / kQBlock;
  const int steps = (KB + waves * U - 1) / (waves * U);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[rt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
  int kb = wave * U;
  if (kb >= KB) return;   // uniform: more waves than blocks
  Fp8Block<XK, RT, NT> r[U];
  float sv[RT];
  auto load_scales = [&](int kb) {
    int i = kb + (lane & 31);
    i = i < KB ? i : KB - 1;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sv[rt] = (lane < 32 ? s.sa[rt] : s.sb[rt])[i];
  };
  auto scale_of = [&](const float (&v)[RT], int u, float (&sc)[RT]) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v[rt]), u));
      const float b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v[rt]), 32 + u));
      sc[rt] = s.row_b[rt] ? b : a;
    }
  };
  load_scales(kb);
#pragma unroll
  for (int u = 0; u < U; ++u) fp8_load<XK, RT, NT>(s, kb + u, r[u]);
  for (int st = 1; st < steps; ++st) {
    float sp[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sp[rt] = sv[rt];
    const int next = kb + waves * U;
    load_scales(next);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float sc[RT];
      scale_of(sp, u, sc);
      fp8_block<XK, RT, NT>(lane, r[u], sc, lds, acc);   // every step but the last is whole
      fp8_load<XK, RT, NT>(s, next + u, r[u]);
      __builtin_amdgcn_sched_barrier(0);   // a block's operands at a time (registers)
    }
    kb = next;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (kb + u < KB) {
      float sc[RT];
      scale_of(sv, u, sc);
      fp8_block<XK, RT, NT>(lane, r[u], sc, lds, acc);
    }
    __builtin_amdgcn_sched_barrier(0);   // a block's operands at a time (registers)
  }
  // a packed token's columns add up to its sum, left in each of them
  if constexpr (XTraits<XK>::kCols > 1) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[rt][nt][i];
          v += dpp_f32<0xB1>(v);                          // quad_perm [1,0,3,2]
          if constexpr (XTraits<XK>::kCols == 4) v += dpp_f32<0x4E>(v);  // quad_perm [2,3,0,1]
          acc[rt][nt][i] = v;
        }
  }
}

// ---- activations shared by the workgroup ---------------------------------------
//
// More than 16 tokens: a block's activations are many times a tile's weight
// bytes, so they are requested once for 64 RT weight rows.  Eight waves: four
// row groups of RT tiles, twice -- waves 0-3 and waves 4-7 take the two
// halves of the blocks, each with activations of its own in LDS, widened to
// bf16 (two buffers, one barrier a block).  Weights and activations are
// requested U blocks ahead, into registers.

constexpr int kSharedWaves = 8;

template <int RT, int NT, bool E8>
struct SharedSrc {
  static constexpr int XL = E8 ? (NT + 1) / 2 : NT;   // activation loads of a thread and block
  const uint8_t* w[RT];     // as Fp8Src
  uint32_t ra[RT], rb[RT];
  const float* sa[RT];
  const float* sb[RT];
  bool row_b[RT];
  const void* x;
  uint32_t xo[XL];          // byte offset of the token row of each load (shared_load_token)
  const float* xs;
  uint32_t xso;             // e4m3: index of the first scale of token 16 (wave % 4) + lane % 16
  int K;
};

template <bool E8>
__device__ __forceinline__ int shared_load_token(int i) {
  const int ht = threadIdx.x & 255;
  return E8 ? 32 * i + (ht >> 3) : 16 * i + (ht >> 4);
}

template <int NT> constexpr int shared_x_bytes() { return NT * 4096; }
// LDS: two activation buffers for each half, the waves' weight buffers, and
// (e4m3) two buffers of 64 token scales for each half; later the second
// half's sums.
template <int RT, int NT> constexpr int shared_lds() {
  return 4 * shared_x_bytes<NT>() + kSharedWaves * RT * 2048 + 4 * 64 * 4;
}

// Blocks [kb0, kb0 + n) of this wave's half (n may differ between the halves;
// iters >= both).  acc: the half's sums.
template <int RT, int NT, bool E8, int U>
__device__ __forceinline__ void shared_product(const SharedSrc<RT, NT, E8>& s, int kb0, int n, int iters, char* s_lds,
                                               f32x4 (&acc)[RT][NT]) {
  constexpr int XL = SharedSrc<RT, NT, E8>::XL;
  const int lane = threadIdx.x & 63, g = lane >> 4, c16 = lane & 15, ht = threadIdx.x & 255;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = wave >> 2;
  const int K = s.K, KB = (K + kQBlock - 1) / kQBlock;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const f32x4 fzero = {0.f, 0.f, 0.f, 0.f};
  char* xbuf = s_lds + half * 2 * shared_x_bytes<NT>();
  char* wbuf = s_lds + 4 * shared_x_bytes<NT>() + wave * RT * 2048;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[rt][nt] = fzero;
  u32x4 wa[U][RT], wb[U][RT], xv[U][XL];
  float sc[U][RT], xs[U];
  float* xsb = reinterpret_cast<float*>(s_lds + 4 * shared_x_bytes<NT>() + kSharedWaves * RT * 2048) + half * 128;
  auto load = [&](int i, int u) {
    int kb = kb0 + (i < n ? i : (n > 0 ? n - 1 : 0));   // past the end: the last one again, not used
    kb = kb < KB ? kb : KB - 1;
    const uint32_t k0 = (uint32_t)kb * kQBlock;
#pragma unroll
    for (int q = 0; q < XL; ++q) {
      const uint32_t c = E8 ? k0 + 16 * (ht & 7) : k0 + 8 * (ht & 15);
      const uint32_t top = (uint32_t)K - (E8 ? 16u : 8u);
      xv[u][q] = ld128(reinterpret_cast<const char*>(s.x) + (s.xo[q] + (E8 ? 1u : 2u) * (c < top ? c : top)));
    }
    uint32_t c = k0 + 16 * (lane & 7);
    c = c < (uint32_t)K - 16u ? c : (uint32_t)K - 16u;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      wa[u][rt] = ld128_stream(s.w[rt] + (s.ra[rt] + c));
      wb[u][rt] = ld128_stream(s.w[rt] + (s.rb[rt] + c));
      sc[u][rt] = (s.row_b[rt] ? s.sb[rt] : s.sa[rt])[kb];
    }
    if constexpr (E8) xs[u] = s.xs[s.xso + (uint32_t)kb];
  };
  // the half's block i into buffer i % 2: columns past K as zeros
  auto stage = [&](int i, int u) {
    char* b = xbuf + (i & 1) * shared_x_bytes<NT>();
    const int k0 = (kb0 + i) * kQBlock;
    if constexpr (E8) xsb[(i & 1) * 64 + (wave & 3) * 16 + c16] = xs[u];   // the four lanes of a token store the same value
#pragma unroll
    for (int q = 0; q < XL; ++q) {
      const int t = shared_load_token<E8>(q);
      u32x4* row = reinterpret_cast<u32x4*>(b) + t * 16;
      if constexpr (E8) {
        if (NT % 2 == 0 || t < 16 * NT) {
          const u32x4 v = k0 + 16 * (ht & 7) < K ? xv[u][q] : zero;
          row[(2 * (ht & 7)) ^ swizzle256(t & 15)] = __builtin_bit_cast(u32x4, widen8(v[0], v[1]));
          row[(2 * (ht & 7) + 1) ^ swizzle256(t & 15)] = __builtin_bit_cast(u32x4, widen8(v[2], v[3]));
        }
      } else {
        row[(ht & 15) ^ swizzle256(t & 15)] = k0 + 8 * (ht & 15) < K ? xv[u][q] : zero;
      }
    }
  };
  auto compute = [&](int i, int u) {
    const char* b = xbuf + (i & 1) * shared_x_bytes<NT>();
    const int c0 = (kb0 + i) * kQBlock + 32 * g;
    const bool tail = (kb0 + i + 1) * kQBlock > K;
    bf16x8 wv[RT][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) rows128_store(lane, wbuf + rt * 2048, wa[u][rt], wb[u][rt]);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      u32x4 lo, hi;
      rows128_load(lane, wbuf + rt * 2048, lo, hi);
      if (tail) {
        if (c0 >= K) lo = zero;
        if (c0 + 16 >= K) hi = zero;
      }
      wv[rt][0] = widen8(lo[0], lo[1]);
      wv[rt][1] = widen8(lo[2], lo[3]);
      wv[rt][2] = widen8(hi[0], hi[1]);
      wv[rt][3] = widen8(hi[2], hi[3]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const u32x4* row = reinterpret_cast<const u32x4*>(b) + (16 * nt + c16) * 16;
      f32x4 d[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) d[rt] = fzero;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 xj = __builtin_bit_cast(bf16x8, row[(4 * g + j) ^ swizzle256(c16)]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) d[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[rt][j], xj, d[rt], 0, 0, 0);
      }
      const float xf = E8 ? xsb[(i & 1) * 64 + 16 * nt + c16] : 1.f;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float f = E8 ? sc[u][rt] * xf : sc[u][rt];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[rt][nt][q] = __builtin_fmaf(f, d[rt][q], acc[rt][nt][q]);
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, u);
  stage(0, 0);
  lds_barrier();
  // iteration i: block i is multiplied, block i + 1 staged, block i + U
  // requested.  Whole groups of U iterations; the last one requests nothing
  // (a request under a condition would make every wait one for all requests).
  const int groups = (iters + U - 1) / U;
  int i = 0;
  for (int gr = 1; gr < groups; ++gr, i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      stage(i + u + 1, (u + 1) % U);
      if (i + u < n) compute(i + u, u);
      load(i + u + U, u);
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (i + u < iters) {   // uniform; 7 blocks of a half are not run as 8 (64 tokens, 7168 x 7168: 0.2 us)
      if (u + 1 < U && i + u + 1 < iters) stage(i + u + 1, u + 1);
      if (i + u < n) compute(i + u, u);
      lds_barrier();
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace moe
