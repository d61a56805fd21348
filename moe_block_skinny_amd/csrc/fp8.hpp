// fp8.hpp -- host-side launch interface of the products over 8-bit weights
// (not part of the public API).
#pragma once

#include "internal.hpp"

namespace moe {

// n matrices [rows][cols] -> e4m3 codes of the same shape and fp32 scales,
// for each 128 columns of a row, or for each 128 x 128 block (blocks != 0).
struct QuantizeLaunch {
  int bf16, blocks;
  int n, rows, cols;
  const void* X;
  uint8_t* Q;
  float* scale;
};

// Y[t][n] = sum_c X[t][c] W[n][c] (+ R[t][n]), t < M, n < N: W [N][K] e4m3
// with Ws [N/128][K/128]; X bf16, or e4m3 with Xs [M][K/128].
struct GemmFp8Launch {
  int x_e4m3;
  const void* X;
  const float* Xs;
  const uint8_t* W;
  const float* Ws;
  const uint16_t* R;        // bf16 [M][N] or null
  void* Y;
  int y_bf16;
  int M, N, K;
  int ks_n;                 // K slices (gemm_fp8_plan); their sums and one arrival counter per row group
  float* part;
  uint32_t* counter;
};

// Shape of the product for many tokens over a long K (rt = 0: split waves take
// it): row tiles a wave, K slices, bytes of the slices' sums in the workspace
// (0: one slice).
struct GemmFp8Plan {
  int rt, ks;
  size_t part_bytes;
};
GemmFp8Plan gemm_fp8_plan(int x_e4m3, int M, int N, int K);

// The block's expert launches over 8-bit weights: ExpertLaunch with W13, W2,
// Ws13, Ws2 in e4m3 and their scales, one row of scales for each 128 gate
// rows, then for each 128 up rows: s13 [E][2][I/128][d/128], s2
// [E][d/128][I/128], ss13 [2][Is/128][d/128], ss2 [d/128][Is/128] (counts
// rounded up).  X is bf16, h two bf16 planes as ExpertLaunch has them.
struct Fp8ExpertLaunch {
  ExpertLaunch e;
  const float *s13, *s2, *ss13, *ss2;
};

// What a launch chose, for moe_last_variant.
struct Fp8Shape {
  int grid, waves, rows, tokens, slices;
};

hipError_t launch_quantize(const QuantizeLaunch& a, hipStream_t st);
hipError_t launch_gemm_fp8(const GemmFp8Launch& a, hipStream_t st, Fp8Shape* shape);
hipError_t launch_expert_up_fp8(const Fp8ExpertLaunch& a, hipStream_t st, Fp8Shape* shape);
hipError_t launch_expert_down_combine_fp8(const Fp8ExpertLaunch& a, hipStream_t st, Fp8Shape* shape);

}  // namespace moe
