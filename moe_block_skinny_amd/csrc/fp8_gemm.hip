// fp8_gemm.hip -- the 8-bit quantiser and the dense skinny product over 8-bit
// weights (fp8_core.hpp).

#include <type_traits>

#include "common.hpp"
#include "fp8.hpp"
#include "fp8_core.hpp"

namespace moe {

// ---- quantiser ---------------------------------------------------------------
//
// s = the smallest power of two with max|x| / s <= 448 over a group (128
// columns of one row, or a 128 x 128 block), q = x / s rounded to e4m3
// (nearest, ties to even).  A power of two makes x / s exact in fp32, so a
// code is rounded once, and s needs no division.  A thread takes 16
// consecutive columns (one 16-byte store of codes), 8 threads a row of a
// group.  Bound by memory: 128 matrices of 256 x 7168 bf16 in blocks, 705 MB
// read and written, 132 us (5.3 TB/s; a plain copy 4.9); 8 rows of 7168 2.8
// us, a launch's own time.

// |x| with infinities and NaN left out of the maximum.
__device__ __forceinline__ float finite_abs(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? __uint_as_float(u) : 0.f;
}

// Exponent of the group's scale: 448 = 1.75 * 2^8.  No scale is below 2^-126
// (the smallest normal number); a group of zeros has scale 1.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0u) return 0;
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}

// 16 values as loaded: 2 (bf16) or 4 (fp32) 16-byte chunks.
template <typename T> struct Chunk16 { u32x4 v[sizeof(T)]; };

template <typename T>
__device__ __forceinline__ void unpack16(const Chunk16<T>& c, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w = c.v[i >> 3][(i & 7) >> 1];
      f[i] = (i & 1) ? bf16_hi(w) : bf16_lo(w);
    } else {
      const uint32_t w = c.v[i >> 2][i & 3];
      f[i] = __uint_as_float(w);
    }
  }
}

template <typename T>
__device__ __forceinline__ Chunk16<T> load16(const T* p) {
  Chunk16<T> c;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) c.v[i] = ld128(reinterpret_cast<const u32x4*>(p) + i);
  return c;
}

__device__ __forceinline__ u32x4 codes16(const float (&f)[16], float inv) {
  u32x4 q;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[4 * w + i];
      // e4m3 has no infinity: what is not finite becomes its NaN
      s[i] = (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? __builtin_nanf("") : x * inv;
    }
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], p, true);
    q[w] = (uint32_t)p;
  }
  return q;
}

// Maximum over aligned groups of 8 lanes, left in each of them.
__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));    // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp_f32<0x4E>(v));    // quad_perm [2,3,0,1]
  return fmaxf(v, dpp_f32<0x141>(v));  // row_half_mirror: the other quad
}

constexpr int kQuantThreads = 256;

template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(QuantizeLaunch a) {
  const uint32_t KB = ((uint32_t)a.cols + kQBlock - 1) / kQBlock;   // cols may end at 2^31 - 16
  const uint32_t groups = (uint32_t)a.rows * KB;   // all matrices' rows, < 2^31
  const uint32_t stride = gridDim.x * (kQuantThreads / 8);
  const int c = threadIdx.x & 7;
  for (uint32_t g = blockIdx.x * (kQuantThreads / 8) + (threadIdx.x >> 3);; g += stride) {
    const bool in = g < groups;
    // lanes of a wave leave together: the maximum is taken across 8 of them
    if (__ballot(in) == 0ull) break;
    const uint32_t row = (in ? g : 0u) / KB, b = (in ? g : 0u) - row * KB;
    const int col = (int)b * kQBlock + 16 * c;
    const bool ok = in && col < a.cols;
    const size_t at = (size_t)row * a.cols + col;
    Chunk16<T> x = {};
    if (ok) x = load16(reinterpret_cast<const T*>(a.X) + at);
    float f[16], m = 0.f;
    unpack16(x, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(f[i]));
    const int e = scale_exponent(max8(m));
    if (ok) *reinterpret_cast<u32x4*>(a.Q + at) = codes16(f, __uint_as_float((uint32_t)(127 - e) << 23));
    if (in && c == 0) a.scale[g] = __uint_as_float((uint32_t)(127 + e) << 23);
  }
}

// One 128 x 128 block per workgroup: 8 threads a row, 4 rows a thread, all of
// them requested before the maximum is taken, so a value is read once.
template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quantize_blocks_kernel(QuantizeLaunch a) {
  constexpr int R = 4, kRows = kQuantThreads / 8;
  __shared__ float s_max[kQuantThreads / 64];
  const uint32_t KB = ((uint32_t)a.cols + kQBlock - 1) / kQBlock, RB = ((uint32_t)a.rows + kQBlock - 1) / kQBlock;
  const uint32_t bc = blockIdx.x % KB, t = blockIdx.x / KB, br = t % RB, n = t / RB;
  const int col = (int)bc * kQBlock + 16 * (threadIdx.x & 7);
  const int row0 = (int)br * kQBlock + (threadIdx.x >> 3);
  const size_t base = (size_t)n * a.rows * a.cols;
  Chunk16<T> x[R] = {};
  bool ok[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    ok[i] = col < a.cols && row0 + kRows * i < a.rows;
    if (ok[i]) x[i] = load16(reinterpret_cast<const T*>(a.X) + base + (size_t)(row0 + kRows * i) * a.cols + col);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float f[16];
    unpack16(x[i], f);
#pragma unroll
    for (int q = 0; q < 16; ++q) m = fmaxf(m, finite_abs(f[q]));
  }
  const uint32_t mw = wave_max_u32(__float_as_uint(m));   // non-negative: ordered as their bits
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = __uint_as_float(mw);
  __syncthreads();
  m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const int e = scale_exponent(m);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float f[16];
    unpack16(x[i], f);
    if (ok[i]) *reinterpret_cast<u32x4*>(a.Q + base + (size_t)(row0 + kRows * i) * a.cols + col) = codes16(f, inv);
  }
  if (threadIdx.x == 0) a.scale[blockIdx.x] = __uint_as_float((uint32_t)(127 + e) << 23);
}

hipError_t launch_quantize(const QuantizeLaunch& a0, hipStream_t st) {
  QuantizeLaunch a = a0;
  const size_t KB = ((size_t)a.cols + kQBlock - 1) / kQBlock;
  if (a.blocks) {
    const size_t g = (size_t)a.n * (((size_t)a.rows + kQBlock - 1) / kQBlock) * KB;
    if (a.bf16) launch(K_NONE, quantize_blocks_kernel<bf16_t>, dim3((unsigned)g), dim3(kQuantThreads), 0, st, a);
    else launch(K_NONE, quantize_blocks_kernel<float>, dim3((unsigned)g), dim3(kQuantThreads), 0, st, a);
  } else {
    a.rows *= a.n;
    a.n = 1;
    size_t g = ((size_t)a.rows * KB * 8 + kQuantThreads - 1) / kQuantThreads;
    if (g > 16384) g = 16384;
    if (a.bf16) launch(K_NONE, quantize_rows_kernel<bf16_t>, dim3((unsigned)g), dim3(kQuantThreads), 0, st, a);
    else launch(K_NONE, quantize_rows_kernel<float>, dim3((unsigned)g), dim3(kQuantThreads), 0, st, a);
  }
  return hipGetLastError();
}

// ---- dense skinny product ------------------------------------------------------
//
// A workgroup owns 16 RT rows of W over all of K; its waves split K by blocks
// and meet once, in LDS, in wave order (deterministic).  Bound by the bytes of
// W where there are many row groups (7168 x 7168, 5 tokens: 51.5 MB in 10.5
// us, 4.9 TB/s), else by the latency of its K steps (2304 x 7168, 8 tokens:
// 144 groups, 7.0 us; 7168 x 2048, 1 token, all of K in flight: 5.2 us); with
// 64 tokens by instruction issue (7168 x 7168, e4m3: 22.4 us, of a wave's
// cycles 17 % wait for data).

// Results of token t, rows n .. n + 3 (only those below N are there): with N a
// multiple of 4 one store, r the residual's 4 bf16 (zeros without one).
__device__ __forceinline__ u32x2 load_residual4(const GemmFp8Launch& a, int t, int n) {
  if (!a.R) return u32x2{0u, 0u};
  return *reinterpret_cast<const u32x2*>(a.R + (size_t)t * a.N + n);
}
__device__ __forceinline__ void store_rows4(const GemmFp8Launch& a, int t, int n, f32x4 v, u32x2 r) {
  const size_t o = (size_t)t * a.N + n;
  if (a.R) v += f32x4{bf16_lo(r[0]), bf16_hi(r[0]), bf16_lo(r[1]), bf16_hi(r[1])};
  if (a.y_bf16) {
    const u32x2 p = {(uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                     (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
    *reinterpret_cast<u32x2*>(reinterpret_cast<bf16_t*>(a.Y) + o) = p;
  } else {
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.Y) + o) = v;
  }
}
__device__ __forceinline__ void store_rows(const GemmFp8Launch& a, int t, int n, f32x4 v) {
  if ((a.N & 3) == 0) {
    store_rows4(a, t, n, v, load_residual4(a, t, n));
    return;
  }
  const size_t o = (size_t)t * a.N + n;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (n + q >= a.N) break;
    const float y = a.R ? v[q] + bf16_to_f32(a.R[o + q]) : v[q];
    if (a.y_bf16) reinterpret_cast<bf16_t*>(a.Y)[o + q] = f32_to_bf16(y);
    else reinterpret_cast<float*>(a.Y)[o + q] = y;
  }
}

template <int XK, int RT, int NT, int U, int MAXW>
__global__ __launch_bounds__(MAXW * 64) void gemm_fp8_kernel(GemmFp8Launch a) {
  // a wave's buffer, then its sums [RT][NT][64]
  extern __shared__ __align__(16) char s_lds[];
  constexpr int kWaveLds = fp8_wave_lds<XK, RT, NT>();
  constexpr int TOK = XTraits<XK>::kTokens, COLS = XTraits<XK>::kCols;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = (int)(blockDim.x >> 6);
  const int KB = (a.K + kQBlock - 1) / kQBlock;
  const int r0 = (int)blockIdx.x * 16 * RT;
  Fp8Src<XK, RT, NT> s;
  s.K = a.K;
  s.lane = lane;
  s.x = buffer_of(a.X);
  s.xs = a.Xs;
  const int xb = x_e4m3(XK) ? 1 : 2;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int base = r0 + 16 * rt < a.N ? r0 + 16 * rt : a.N - 1;
    const int ra = r0 + 16 * rt + (lane >> 3), rb = ra + 8;
    s.w[rt] = buffer_of(a.W + (size_t)base * a.K);
    s.ra[rt] = ra < a.N ? (uint32_t)(ra - base) * (uint32_t)a.K : kNoLoad;
    s.rb[rt] = rb < a.N ? (uint32_t)(rb - base) * (uint32_t)a.K : kNoLoad;
    s.sa[rt] = s.sb[rt] = a.Ws + (size_t)(base / kQBlock) * KB;   // a tile of 16 rows lies in one block row
    s.row_b[rt] = false;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < x_rows<XK>(); ++i) {
      const int t = nt * TOK + x_load_token<XK>(lane, i);
      s.xo[nt][i] = t < a.M ? (uint32_t)t * (uint32_t)a.K * xb : kNoLoad;
    }
    const int t = nt * TOK + x_column_token<XK>(lane);
    s.xso[nt] = (uint32_t)(t < a.M ? t : a.M - 1) * (uint32_t)KB;
  }
  f32x4 acc[RT][NT];
  fp8_wave<XK, RT, NT, U>(s, wave, waves, s_lds + wave * kWaveLds, acc);
  f32x4* mine = reinterpret_cast<f32x4*>(s_lds + wave * kWaveLds);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mine[(rt * NT + nt) * 64 + lane] = acc[rt][nt];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * NT * 64; i += (int)blockDim.x) {
    const int l = i & 63, nt = (i >> 6) % NT, rt = (i >> 6) / NT;
    const int col = l & 15;
    const int t = nt * TOK + col / COLS, n = r0 + 16 * rt + 4 * (l >> 4);
    if (col % COLS || t >= a.M || n >= a.N) continue;
    const f32x4* sum = reinterpret_cast<const f32x4*>(s_lds) + i;
    f32x4 v = sum[0];
    for (int w = 1; w < waves; ++w) v += sum[w * (kWaveLds / 16)];
    store_rows(a, t, n, v);
  }
}

// Many tokens (split_waves_win: how many): 64 RT rows of W and one of a.ks_n
// slices of K for each workgroup (shared_product).  The slices' sums meet in
// the workspace: the last workgroup of a row group to arrive adds them in slice
// order.  7168 x 7168, 64 bf16 tokens: 22.3 us, of which the start takes about
// 2.7, the blocks 12 (4.3 TB/s of W; bound by the activations' way through
// LDS), the arrival 2, the slices' sums 3.  Rows dealt evenly over all compute
// units (28 instead of 32 a wave) gained nothing: 23.0 us against 22.4.
template <int RT, int NT, bool E8, int U>
__global__ __launch_bounds__(kSharedWaves * 64) void gemm_fp8_shared_kernel(GemmFp8Launch a) {
  extern __shared__ __align__(16) char s_lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave >> 2, rg = wave & 3;
  const int KB = (a.K + kQBlock - 1) / kQBlock;
  const int tile = (int)blockIdx.x / a.ks_n, ks = (int)blockIdx.x % a.ks_n;
  const int r0 = (tile * 4 + rg) * 16 * RT;
  SharedSrc<RT, NT, E8> s;
  s.K = a.K;
  s.x = a.X;
  s.xs = a.Xs;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    // rows past N re-read the last one and are not stored
    const int base = r0 + 16 * rt < a.N ? r0 + 16 * rt : a.N - 1;
    const int ra = base + (lane >> 3), rb = ra + 8;
    s.w[rt] = a.W + (size_t)base * a.K;
    s.ra[rt] = (uint32_t)((ra < a.N ? ra : a.N - 1) - base) * (uint32_t)a.K;
    s.rb[rt] = (uint32_t)((rb < a.N ? rb : a.N - 1) - base) * (uint32_t)a.K;
    s.sa[rt] = s.sb[rt] = a.Ws + (size_t)(base / kQBlock) * KB;
    s.row_b[rt] = false;
  }
  auto token = [&](int t) { return (uint32_t)(t < a.M ? t : a.M - 1); };
#pragma unroll
  for (int i = 0; i < SharedSrc<RT, NT, E8>::XL; ++i)
    s.xo[i] = token(shared_load_token<E8>(i)) * (uint32_t)a.K * (E8 ? 1 : 2);
  s.xso = token(16 * rg + (lane & 15)) * (uint32_t)KB;
  // this slice's blocks, then the half's
  const int b0 = (int)((int64_t)KB * ks / a.ks_n), b1 = (int)((int64_t)KB * (ks + 1) / a.ks_n);
  const int iters = (b1 - b0 + 1) / 2;
  const int kb0 = b0 + half * iters, n = half ? b1 - b0 - iters : iters;
  f32x4 acc[RT][NT];
  shared_product<RT, NT, E8, U>(s, kb0, n, iters, s_lds, acc);
  // the second half's sums to the first; pieces of 16 rows x 16 tokens,
  // piece i = (row group * RT + rt) * NT + nt
  constexpr int kPieces = 4 * RT * NT;
  f32x4* sums = reinterpret_cast<f32x4*>(s_lds);   // [kPieces][64]
  f32x4* mine = sums + rg * RT * NT * 64 + lane;
  if (half == 1) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mine[(rt * NT + nt) * 64] = acc[rt][nt];
  }
  __syncthreads();
  if (half == 0) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        acc[rt][nt] += mine[(rt * NT + nt) * 64];
        mine[(rt * NT + nt) * 64] = acc[rt][nt];
      }
  }
  // the eight waves share the pieces
  constexpr int kPer = (kPieces + kSharedWaves - 1) / kSharedWaves, kSlices = 4;
  auto piece = [&](int p) { return wave + kSharedWaves * p; };
  auto token_of_piece = [&](int i) { return 16 * (i % NT) + (lane & 15); };
  auto row_of_piece = [&](int i) { return (tile * 4 * RT + i / NT) * 16 + 4 * (lane >> 4); };
  auto there = [&](int i) { return i < kPieces && token_of_piece(i) < a.M && row_of_piece(i) < a.N; };
  const bool wide = (a.N & 3) == 0;
  f32x4 v[kPer];
  u32x2 res[kPer];
  // the residual is requested ahead of what it is added to
  auto request_residual = [&] {
#pragma unroll
    for (int p = 0; p < kPer; ++p)
      res[p] = wide && there(piece(p)) ? load_residual4(a, token_of_piece(piece(p)), row_of_piece(piece(p))) : u32x2{0u, 0u};
  };
  if (a.ks_n > 1) {
    const coherent_rsrc_t prs = coherent_rsrc(a.part);
    auto off = [&](int slice, int i) { return (uint32_t)((((tile * a.ks_n + slice) * kPieces + i) * 64 + lane) * 16); };
    if (half == 0) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          st_coherent4(prs, off(ks, (rg * RT + rt) * NT + nt), __builtin_bit_cast(u32x4, acc[rt][nt]));
    }
    __shared__ int s_last;
    if (!arrive_last(a.counter + tile, (uint32_t)a.ks_n, &s_last)) return;
    // kSlices slices are requested at a time
    request_residual();
#pragma unroll
    for (int p = 0; p < kPer; ++p) v[p] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int q0 = 0; q0 < a.ks_n; q0 += kSlices) {
      u32x4 pv[kSlices][kPer];
#pragma unroll
      for (int q = 0; q < kSlices; ++q)
#pragma unroll
        for (int p = 0; p < kPer; ++p)
          pv[q][p] = ld_coherent4(prs, off(q0 + q < a.ks_n ? q0 + q : q0, piece(p) < kPieces ? piece(p) : 0));
#pragma unroll
      for (int q = 0; q < kSlices; ++q)
#pragma unroll
        for (int p = 0; p < kPer; ++p)
          if (q0 + q < a.ks_n) v[p] += __builtin_bit_cast(f32x4, pv[q][p]);
    }
  } else {
    request_residual();
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kPer; ++p) v[p] = sums[(piece(p) < kPieces ? piece(p) : 0) * 64 + lane];
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int i = piece(p);
    if (!there(i)) continue;
    if (wide) store_rows4(a, token_of_piece(i), row_of_piece(i), v[p], res[p]);
    else store_rows(a, token_of_piece(i), row_of_piece(i), v[p]);
  }
}

template <int XK, int RT, int NT, int U, int MAXW>
static void go(const GemmFp8Launch& a, hipStream_t st, Fp8Shape* shape) {
  const int KB = (a.K + kQBlock - 1) / kQBlock;
  const int steps = (KB + U * MAXW - 1) / (U * MAXW);
  const int w = (KB + U * steps - 1) / (U * steps);
  const int g = (a.N + 16 * RT - 1) / (16 * RT);
  launch(K_SKINNY, (gemm_fp8_kernel<XK, RT, NT, U, MAXW>), dim3((unsigned)g), dim3((unsigned)(64 * w)),
         (uint32_t)(w * fp8_wave_lds<XK, RT, NT>()), st, a);
  *shape = {g, w, 16 * RT, NT * XTraits<XK>::kTokens, 1};
}

// Two row tiles a wave (half the activation bytes for a weight byte) once the
// rows still make a workgroup for every other compute unit: 33 x 7168 x 2048
// 9.9 us against 11.9 with one, 64 x 4608 x 2048 11.5 against 13.8.
constexpr int kMinNForTwoTiles = 4096;

// Which kernel takes a product of more than 16 tokens.  Split waves read the
// activations for every 32 rows (16 below N = 4096), the shared kernel for
// every 64 or 128, but has a start and a meeting of about 7 us to hide, which a
// short K does not.  By the activation bytes of a column (tokens x bytes), us,
// shared against split waves:
//   one round of 32-row groups, 7168 x 7168: e4m3 17 tokens 18.2 / 13.6, 48
//     21.5 / 19.2, 64 23.2 / 23.1; bf16 17 17.4 / 14.4, 32 17.9 / 17.0, 48
//     20.9 / 25.4, 64 22.4 / 30.6; 4608 x 7168: e4m3 48 20.0 / 18.4, 64 21.4 /
//     22.2; bf16 32 15.8 / 16.2, 48 18.3 / 24.7
//   fewer rows: 2304 x 7168 e4m3 17 11.2 / 9.3, 32 11.4 / 11.8, 48 13.8 / 15.6;
//     bf16 32 11.1 / 12.9
//   more: 16384 x 7168 e4m3 17 28.4 / 23.2, 32 28.3 / 27.9, 48 31.6 / 34.5;
//     bf16 17 27.1 / 26.4, 32 26.9 / 30.5; 32768 x 4096 e4m3 32 29.2 / 32.1
//   short K: 7168 x 2048 (e4m3, 32) 11.0 / 6.6; 1001 x 1040 (bf16, 33) 8.7 / 5.1
constexpr int kSharedMinTokens = 17, kSharedMinK = 4096;
static bool split_waves_win(int x_e4m3, int M, int N) {
  const int column = M * (x_e4m3 ? 1 : 2);
  if (N >= kMinNForTwoTiles && N <= 32 * 256) return column <= 64;
  return N <= 2 * 32 * 256 && column <= 32;
}

// K slices and row tiles of the shared kernel: 64 RT rows a workgroup, and as
// many slices as put a workgroup on every compute unit, of at least four
// blocks (two a half), while the last workgroup of a row group reads at most
// kMaxPartialBytes (one or two round trips).  RT = 2 from N = 6400 on: at
// N = 7168 22.3 us against 26.0 with RT = 1, at 1536 no difference.
GemmFp8Plan gemm_fp8_plan(int x_e4m3, int M, int N, int K) {
  constexpr int kCUs = 256, kMaxPartialBytes = 128 * 1024, kMinNForTwo = 6400;
  GemmFp8Plan p = {0, 1, 0};
  if (M < kSharedMinTokens || K < kSharedMinK || split_waves_win(x_e4m3, M, N)) return p;
  const int KB = (K + kQBlock - 1) / kQBlock, nt = (M + 15) / 16;
  p.rt = N >= kMinNForTwo ? 2 : 1;
  const int rg = (N + 64 * p.rt - 1) / (64 * p.rt);
  int ks = kCUs / rg;
  const int most = kMaxPartialBytes / (64 * p.rt * 16 * nt * 4);
  if (ks > most) ks = most;
  if (ks > KB / 4) ks = KB / 4;
  if (ks < 1) ks = 1;
  p.ks = ks;
  p.part_bytes = ks > 1 ? (size_t)rg * ks * 64 * p.rt * 16 * nt * 4 : 0;
  return p;
}

template <int RT, int NT, bool E8, int U>
static void go_shared(const GemmFp8Launch& a, hipStream_t st, Fp8Shape* shape) {
  const int g = (a.N + 64 * RT - 1) / (64 * RT) * a.ks_n;
  launch(K_SKINNY, (gemm_fp8_shared_kernel<RT, NT, E8, U>), dim3((unsigned)g), dim3(kSharedWaves * 64),
         (uint32_t)shared_lds<RT, NT>(), st, a);
  *shape = {g, kSharedWaves, 64 * RT, 16 * NT, a.ks_n};
}

hipError_t launch_gemm_fp8(const GemmFp8Launch& a, hipStream_t st, Fp8Shape* shape) {
  const GemmFp8Plan p = gemm_fp8_plan(a.x_e4m3, a.M, a.N, a.K);
  const int nt = (a.M + 15) / 16;
  if (p.rt) {
    GemmFp8Launch b = a;
    b.ks_n = p.ks;
    auto pick = [&](auto E) {
      constexpr bool E8 = decltype(E)::value;
      constexpr int U = 2;   // 7168 x 7168, B = 64: 22.3 us, 24.3 at 3, 24.8 at 4 (registers); 1536 x 7168 13.5, 14.4, 13.8
      if (p.rt == 1) {
        if (nt == 2) go_shared<1, 2, false, U>(b, st, shape);   // bf16 (below)
        else if (nt == 3) go_shared<1, 3, E8, U>(b, st, shape);
        else go_shared<1, 4, E8, U>(b, st, shape);
      } else {
        if (nt == 2) go_shared<2, 2, E8, U>(b, st, shape);
        else if (nt == 3) go_shared<2, 3, E8, U>(b, st, shape);
        else go_shared<2, 4, E8, U>(b, st, shape);
      }
    };
    // up to 32 tokens of e4m3 and fewer than 6400 rows are split waves'
    if (a.x_e4m3 && p.rt == 1 && nt == 2) return hipErrorInvalidValue;
    if (a.x_e4m3) pick(std::true_type());
    else pick(std::false_type());
    return hipGetLastError();
  }
  // Blocks in flight of a wave and waves, up to 16 tokens.  More of the first
  // pays over a row of 2048 columns or more (below, it leaves three waves or
  // fewer); with 5 tokens and more, or e4m3 ones, only where every compute
  // unit has a row group (many).  Measured, us, this against the other choice:
  //   <= 4 tokens:       1 x 7168 x 7168 10.4 / 10.9, 1 x 7168 x 2048 5.0 / 5.2; 2 x 7168 x 512 3.4 / 3.45
  //   <= 8, e4m3:        5 x 7168 x 7168 11.2 / 11.5; 7 x 1536 x 4096 5.2 / 5.5, 1 x 16384 x 1024 5.4 / 5.5
  //   5 to 8:            8 x 57344 x 7168 73.7 / 76.0; 8 x 2304 x 7168 7.6 / 7.7; 8 x 7168 x 2048 5.7 / 5.8, 6 x 1024 x 1536 3.56 / 3.65
  //   9 to 16 (waves):   e4m3 16 x 7168 x 7168 13.8 / 14.5, 12 x 2304 x 7168 8.0 / 8.9; bf16 16 x 4096 x 4096 7.7 / 7.9
  const bool many = a.N >= 16 * 256, lengthy = a.K >= 2048;
  if (a.x_e4m3) {
    if (a.M <= 8 && many && lengthy) go<X8P, 1, 1, 4, 8>(a, st, shape);
    else if (a.M <= 8) go<X8P, 1, 1, 2, 8>(a, st, shape);
    else if (nt <= 1 && many) go<X8, 1, 1, 2, 4>(a, st, shape);
    else if (nt <= 1) go<X8, 1, 1, 2, 8>(a, st, shape);
    else if (a.N < kMinNForTwoTiles) {
      if (nt == 2) go<X8, 1, 2, 2, 8>(a, st, shape);
      else if (nt == 3) go<X8, 1, 3, 2, 8>(a, st, shape);
      else go<X8, 1, 4, 2, 8>(a, st, shape);
    } else {
      if (nt == 2) go<X8, 2, 2, 2, 4>(a, st, shape);
      else if (nt == 3) go<X8, 2, 3, 2, 4>(a, st, shape);
      else go<X8, 2, 4, 2, 4>(a, st, shape);
    }
  } else {
    if (a.M <= 4 && lengthy) go<XP4, 1, 1, 4, 8>(a, st, shape);
    else if (a.M <= 4) go<XP4, 1, 1, 2, 8>(a, st, shape);
    else if (a.M <= 8 && !lengthy) go<XP8, 1, 1, 2, 8>(a, st, shape);
    else if (a.M <= 8 && a.K <= 2048) go<XP8, 1, 1, 4, 8>(a, st, shape);   // all of the row in one step
    else if (a.M <= 8 && many) go<XP8L, 1, 1, 3, 8>(a, st, shape);
    else if (a.M <= 8) go<XP8L, 1, 1, 2, 8>(a, st, shape);
    else if (nt <= 1 && many) go<XB, 1, 1, 2, 4>(a, st, shape);
    else if (nt <= 1) go<XB, 1, 1, 2, 8>(a, st, shape);
    else if (a.N < kMinNForTwoTiles) {
      if (nt == 2) go<XB, 1, 2, 2, 8>(a, st, shape);
      else if (nt == 3) go<XB, 1, 3, 2, 8>(a, st, shape);
      else go<XB, 1, 4, 1, 8>(a, st, shape);
    } else {
      if (nt == 2) go<XB, 2, 2, 2, 4>(a, st, shape);
      else if (nt == 3) go<XB, 2, 3, 1, 4>(a, st, shape);
      else go<XB, 2, 4, 1, 4>(a, st, shape);
    }
  }
  return hipGetLastError();
}

}  // namespace moe
