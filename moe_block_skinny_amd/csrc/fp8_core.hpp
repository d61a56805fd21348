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
// 128 bytes -- a whole cache line of each, one scale block -- and a DPP row
// shift between the two loads of a tile gives every lane its operand: lane l
// = R + 16 g holds columns 32 g .. 32 g + 31 of row R.  Which K positions sit
// in which lane group is the same for both operands, so the products are
// those of the plain order.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kQBlock = 128;   // columns (and weight rows) that share a scale

// Token layouts of the activation operand.
//   XP4:  bf16, up to 4 tokens.  One 16-byte load per block: matrix column
//         4 t + j holds token t's piece j (8 of the lane group's 32 values).
//         Step j of the block multiplies the columns that hold piece j, the
//         others as zeros, so the four columns of a token add up to its sum.
//   XP8:  bf16, up to 8 tokens, two loads: column 2 t + (j & 1).
//   XB:   bf16, NT tiles of 16 tokens, four loads per tile.
//   X8P:  e4m3, up to 8 tokens, one load: column 2 t + i holds the lane
//         group's half i (pieces 2 i and 2 i + 1).
//   X8:   e4m3, NT tiles of 16 tokens, two loads per tile.
// A token packed in 4 columns costs a quarter of the registers that a column
// of its own would, which is what lets a wave request all its blocks at once.
enum XKind { XP4 = 0, XP8 = 1, XB = 2, X8P = 3, X8 = 4 };

constexpr bool x_e4m3(int xk) { return xk == X8P || xk == X8; }

template <int XK> struct XTraits;
template <> struct XTraits<XP4> { static constexpr int kLoads = 1, kTokens = 4, kCols = 4; };
template <> struct XTraits<XP8> { static constexpr int kLoads = 2, kTokens = 8, kCols = 2; };
template <> struct XTraits<XB> { static constexpr int kLoads = 4, kTokens = 16, kCols = 1; };
template <> struct XTraits<X8P> { static constexpr int kLoads = 1, kTokens = 8, kCols = 2; };
template <> struct XTraits<X8> { static constexpr int kLoads = 2, kTokens = 16, kCols = 1; };

// Token of this lane's matrix column within its tile of kTokens.
template <int XK>
__device__ __forceinline__ int x_token() {
  const int c = threadIdx.x & 15;
  return c / XTraits<XK>::kCols;
}

// Where a wave reads: per lane, byte offsets from uniform bases.
template <int RT, int NT>
struct Fp8Src {
  const uint8_t* w[RT];     // tile's weight base (uniform)
  uint32_t ra[RT], rb[RT];  // byte offset of the lane's row among rows 0-7 and 8-15 (its first column)
  const float* sa[RT];      // scales of the block row that holds the tile's row 0 (uniform), [blocks]
  const float* sb[RT];      // and of that of the rows of the upper lanes (row_b)
  bool row_b[RT];           // the lane's result rows take sb
  const void* x;            // activations (uniform)
  uint32_t xo[NT];          // byte offset of the lane's token row
  const float* xs;          // e4m3: scales (uniform)
  uint32_t xso[NT];         // e4m3: index of the lane's token's first scale
  int K;
};

// Operand of a tile from its two loads.
__device__ __forceinline__ void w_operand(u32x4 va, u32x4 vb, u32x4& lo, u32x4& hi) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // row_shr:8: lanes 8-15 of a row of 16 take vb of lane - 8; lanes 0-7 keep va
    lo[e] = (uint32_t)__builtin_amdgcn_update_dpp((int)va[e], (int)vb[e], 0x118, 0xf, 0xf, false);
    // row_shl:8: lanes 0-7 take va of lane + 8; lanes 8-15 keep vb
    hi[e] = (uint32_t)__builtin_amdgcn_update_dpp((int)vb[e], (int)va[e], 0x108, 0xf, 0xf, false);
  }
}

// 8 codes (two words) as 8 bf16: exact, NaN stays NaN.
__device__ __forceinline__ bf16x8 widen8(uint32_t w0, uint32_t w1) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Registers of one K block of a wave.
template <int XK, int RT, int NT>
struct Fp8Block {
  u32x4 a[RT], b[RT];
  u32x4 x[NT][XTraits<XK>::kLoads];
  float xs[NT];
};

// Request block kb.  A block past the last is clamped to it (and must not be
// used); in a short last block a lane past K re-reads the row's last columns.
template <int XK, int RT, int NT>
__device__ __forceinline__ void fp8_load(const Fp8Src<RT, NT>& s, int kb, Fp8Block<XK, RT, NT>& r) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int last = (s.K - 1) / kQBlock;
  const uint32_t k0 = (uint32_t)(kb < last ? kb : last) * kQBlock;
  const uint32_t K = (uint32_t)s.K;
  auto below = [](uint32_t v, uint32_t top) { return v < top ? v : top; };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const char* x = reinterpret_cast<const char*>(s.x);
    if constexpr (XK == XP4) {
      const uint32_t c = below(k0 + 32 * g + 8 * (lane & 3), K - 8);
      r.x[nt][0] = ld128(x + (s.xo[nt] + 2 * c));
    } else if constexpr (XK == XP8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t c = below(k0 + 32 * g + 16 * i + 8 * (lane & 1), K - 8);
        r.x[nt][i] = ld128(x + (s.xo[nt] + 2 * c));
      }
    } else if constexpr (XK == XB) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = below(k0 + 32 * g + 8 * j, K - 8);
        r.x[nt][j] = ld128(x + (s.xo[nt] + 2 * c));
      }
    } else if constexpr (XK == X8P) {
      const uint32_t c = below(k0 + 32 * g + 16 * (lane & 1), K - 16);
      r.x[nt][0] = ld128(x + (s.xo[nt] + c));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t c = below(k0 + 32 * g + 16 * i, K - 16);
        r.x[nt][i] = ld128(x + (s.xo[nt] + c));
      }
    }
    if constexpr (x_e4m3(XK)) r.xs[nt] = s.xs[s.xso[nt] + k0 / kQBlock];
  }
  const uint32_t c = below(k0 + 16 * (lane >> 3), K - 16);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    r.a[rt] = ld128_stream(s.w[rt] + (s.ra[rt] + c));
    r.b[rt] = ld128_stream(s.w[rt] + (s.rb[rt] + c));
  }
}

// acc += the block's products, each tile's by its scale sc[rt].
template <int XK, int RT, int NT>
__device__ __forceinline__ void fp8_block(const Fp8Block<XK, RT, NT>& r, const float (&sc)[RT], int kb, int K,
                                          f32x4 (&acc)[RT][NT]) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const f32x4 fzero = {0.f, 0.f, 0.f, 0.f};
  const bool tail = (kb + 1) * kQBlock > K;   // uniform: a short last block, zeros past K on both sides
  const int c0 = kb * kQBlock + 32 * g;
  u32x4 xv[NT][XTraits<XK>::kLoads];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < XTraits<XK>::kLoads; ++i) xv[nt][i] = r.x[nt][i];
  if (tail) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < XTraits<XK>::kLoads; ++i) {
        int c;
        if constexpr (XK == XP4) c = c0 + 8 * (lane & 3);
        else if constexpr (XK == XP8) c = c0 + 16 * i + 8 * (lane & 1);
        else if constexpr (XK == XB) c = c0 + 8 * i;
        else if constexpr (XK == X8P) c = c0 + 16 * (lane & 1);
        else c = c0 + 16 * i;
        if (c >= K) xv[nt][i] = zero;
      }
  }
  // the operand of step j
  bf16x8 xj[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (x_e4m3(XK)) {
        const u32x4 h = xv[nt][XK == X8 ? j >> 1 : 0];
        const uint32_t w0 = h[2 * (j & 1)], w1 = h[2 * (j & 1) + 1];
        const bool mine = XK == X8 || (lane & 1) == (j >> 1);
        xj[nt][j] = widen8(mine ? w0 : 0u, mine ? w1 : 0u);
      } else {
        u32x4 h;
        if constexpr (XK == XP4) h = (lane & 3) == j ? xv[nt][0] : zero;
        else if constexpr (XK == XP8) h = (lane & 1) == (j & 1) ? xv[nt][j >> 1] : zero;
        else h = xv[nt][j];
        xj[nt][j] = __builtin_bit_cast(bf16x8, h);
      }
    }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    u32x4 lo, hi;
    w_operand(r.a[rt], r.b[rt], lo, hi);
    if (tail) {
      if (c0 >= K) lo = zero;
      if (c0 + 16 >= K) hi = zero;
    }
    const bf16x8 wv[4] = {widen8(lo[0], lo[1]), widen8(lo[2], lo[3]), widen8(hi[0], hi[1]), widen8(hi[2], hi[3])};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 d = fzero;
#pragma unroll
      for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], xj[nt][j], d, 0, 0, 0);
      const float f = x_e4m3(XK) ? sc[rt] * r.xs[nt] : sc[rt];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[rt][nt][i] = __builtin_fmaf(f, d[i], acc[rt][nt][i]);
    }
  }
}

// Wave `wave` of `waves` over all of K: in step s it takes blocks
// (s * waves + wave) * U .. + U - 1, all U requested before any is used and
// each block's registers refilled for the next step as soon as it is.  The
// scales of a step come with one load (lanes 0.. the first block row's, lanes
// 32.. the second's) and are read out lane by lane.
template <int XK, int RT, int NT, int U>
__device__ __forceinline__ void fp8_wave(const Fp8Src<RT, NT>& s, int wave, int waves, f32x4 (&acc)[RT][NT]) {
  const int lane = threadIdx.x & 63;
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
      fp8_block<XK, RT, NT>(r[u], sc, kb + u, s.K, acc);   // every step but the last is whole
      fp8_load<XK, RT, NT>(s, next + u, r[u]);
    }
    kb = next;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (kb + u < KB) {
      float sc[RT];
      scale_of(sv, u, sc);
      fp8_block<XK, RT, NT>(r[u], sc, kb + u, s.K, acc);
    }
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

}  // namespace moe
