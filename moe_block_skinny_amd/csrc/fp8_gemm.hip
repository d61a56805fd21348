// fp8_gemm.hip -- the 8-bit quantiser and the dense skinny product over 8-bit
// weights (fp8_core.hpp).

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
// group.

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
  const uint32_t KB = (uint32_t)(a.cols + kQBlock - 1) / kQBlock;
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
  const uint32_t KB = (uint32_t)(a.cols + kQBlock - 1) / kQBlock, RB = (uint32_t)(a.rows + kQBlock - 1) / kQBlock;
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
// and meet once, in LDS, in wave order (deterministic).

template <int XK, int RT, int NT, int U, int MAXW>
__global__ __launch_bounds__(MAXW * 64) void gemm_fp8_kernel(GemmFp8Launch a) {
  extern __shared__ f32x4 s_acc[];   // [waves][RT][NT][64]
  constexpr int TOK = XTraits<XK>::kTokens, COLS = XTraits<XK>::kCols;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = (int)(blockDim.x >> 6);
  const int KB = (a.K + kQBlock - 1) / kQBlock;
  const int r0 = (int)blockIdx.x * 16 * RT;
  Fp8Src<RT, NT> s;
  s.K = a.K;
  s.x = a.X;
  s.xs = a.Xs;
  const int xb = x_e4m3(XK) ? 1 : 2;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    // rows past N re-read the last one and are not stored
    const int base = r0 + 16 * rt < a.N ? r0 + 16 * rt : a.N - 1;
    const int ra = base + (lane & 7), rb = ra + 8;
    s.w[rt] = a.W + (size_t)base * a.K;
    s.ra[rt] = (uint32_t)((ra < a.N ? ra : a.N - 1) - base) * (uint32_t)a.K;
    s.rb[rt] = (uint32_t)((rb < a.N ? rb : a.N - 1) - base) * (uint32_t)a.K;
    s.sa[rt] = s.sb[rt] = a.Ws + (size_t)(base / kQBlock) * KB;   // a tile of 16 rows lies in one block row
    s.row_b[rt] = false;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    int t = nt * TOK + x_token<XK>();
    t = t < a.M ? t : a.M - 1;
    s.xo[nt] = (uint32_t)t * (uint32_t)a.K * xb;
    s.xso[nt] = (uint32_t)t * (uint32_t)KB;
  }
  f32x4 acc[RT][NT];
  fp8_wave<XK, RT, NT, U>(s, wave, waves, acc);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s_acc[((wave * RT + rt) * NT + nt) * 64 + lane] = acc[rt][nt];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * NT * 64; i += (int)blockDim.x) {
    const int l = i & 63, nt = (i >> 6) % NT, rt = (i >> 6) / NT;
    const int col = l & 15;
    const int t = nt * TOK + col / COLS, n = r0 + 16 * rt + 4 * (l >> 4);
    if (col % COLS || t >= a.M || n >= a.N) continue;
    f32x4 v = s_acc[i];
    for (int w = 1; w < waves; ++w) v += s_acc[w * RT * NT * 64 + i];
    const size_t o = (size_t)t * a.N + n;
    if ((a.N & 3) == 0) {
      if (a.R) {
        const u32x2 r = *reinterpret_cast<const u32x2*>(a.R + o);
        v += f32x4{bf16_lo(r[0]), bf16_hi(r[0]), bf16_lo(r[1]), bf16_hi(r[1])};
      }
      if (a.y_bf16) {
        const u32x2 p = {(uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                         (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
        *reinterpret_cast<u32x2*>(reinterpret_cast<bf16_t*>(a.Y) + o) = p;
      } else {
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.Y) + o) = v;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (n + q >= a.N) break;
        const float y = a.R ? v[q] + bf16_to_f32(a.R[o + q]) : v[q];
        if (a.y_bf16) reinterpret_cast<bf16_t*>(a.Y)[o + q] = f32_to_bf16(y);
        else reinterpret_cast<float*>(a.Y)[o + q] = y;
      }
    }
  }
}

template <int XK, int RT, int NT, int U, int MAXW>
static void go(const GemmFp8Launch& a, hipStream_t st, char* desc, size_t len) {
  const int KB = (a.K + kQBlock - 1) / kQBlock;
  int w = (KB + U - 1) / U;
  if (w > MAXW) w = MAXW;
  const int g = (a.N + 16 * RT - 1) / (16 * RT);
  launch(K_SKINNY, (gemm_fp8_kernel<XK, RT, NT, U, MAXW>), dim3((unsigned)g), dim3((unsigned)(64 * w)),
         (uint32_t)(w * RT * NT * 64 * sizeof(f32x4)), st, a);
  if (desc)
    snprintf(desc, len, "fp8 x=%s M=%d N=%d K=%d rows/wg=%d tokens/tile=%d waves/wg=%d grid=%d", x_e4m3(XK) ? "e4m3" : "bf16",
             a.M, a.N, a.K, 16 * RT, NT * XTraits<XK>::kTokens, w, g);
}

hipError_t launch_gemm_fp8(const GemmFp8Launch& a, hipStream_t st, char* desc, size_t len) {
  const int nt = (a.M + 15) / 16;
  if (a.x_e4m3) {
    if (a.M <= 8) go<X8P, 1, 1, 4, 16>(a, st, desc, len);
    else if (nt <= 1) go<X8, 1, 1, 4, 16>(a, st, desc, len);
    else if (nt == 2) go<X8, 2, 2, 2, 8>(a, st, desc, len);
    else if (nt == 3) go<X8, 2, 3, 2, 8>(a, st, desc, len);
    else go<X8, 2, 4, 2, 8>(a, st, desc, len);
  } else {
    if (a.M <= 4) go<XP4, 1, 1, 4, 16>(a, st, desc, len);
    else if (a.M <= 8) go<XP8, 1, 1, 4, 16>(a, st, desc, len);
    else if (nt <= 1) go<XB, 1, 1, 4, 16>(a, st, desc, len);
    else if (nt == 2) go<XB, 2, 2, 2, 8>(a, st, desc, len);
    else if (nt == 3) go<XB, 2, 3, 2, 8>(a, st, desc, len);
    else go<XB, 2, 4, 2, 8>(a, st, desc, len);
  }
  return hipGetLastError();
}

}  // namespace moe
