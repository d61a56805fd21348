// fp8_expert.hip -- routed and shared experts of the decode MoE block over
// 8-bit weights (fp8_core.hpp), and the weighted combine.
//
// The block's launches are those of the bf16 weights (expert.hip): the
// router scores in a launch of its own, or (B <= 2) in the gate/up launch;
// gate/up + SwiGLU; down + combine.  Routing, plan, h and the combine's order
// are the same functions; the expert products are these.

#include "common.hpp"
#include "expert_core.hpp"
#include "fp8.hpp"
#include "fp8_core.hpp"

namespace moe {

// Entry idx of the plan, in scalar registers: a routed expert (idx < n) or
// the shared one.
struct Fp8Entry {
  int m, I, slot0;            // tokens; expert rows; first plan slot (-1: shared, token i is token i)
  const uint8_t *W13, *W2;
  const float *s13, *s2;
};

__device__ __forceinline__ Fp8Entry fp8_entry(const Fp8ExpertLaunch& a, const PlanView& p, int n, int idx) {
  Fp8Entry v;
  const size_t DB = (size_t)(a.e.d + kQBlock - 1) / kQBlock;
  if (idx < n) {
    const size_t e = (size_t)wave_uniform(p.active[idx]);
    v.slot0 = wave_uniform(p.offs[idx]);
    v.m = wave_uniform(p.offs[idx + 1]) - v.slot0;
    v.I = a.e.I;
    const size_t IB = (size_t)(v.I + kQBlock - 1) / kQBlock;
    v.W13 = static_cast<const uint8_t*>(a.e.W13) + e * 2 * v.I * a.e.d;
    v.W2 = static_cast<const uint8_t*>(a.e.W2) + e * v.I * a.e.d;
    v.s13 = a.s13 + e * 2 * IB * DB;
    v.s2 = a.s2 + e * DB * IB;
  } else {
    v.m = a.e.B;
    v.I = a.e.Is;
    v.slot0 = -1;
    v.W13 = static_cast<const uint8_t*>(a.e.Ws13);
    v.W2 = static_cast<const uint8_t*>(a.e.Ws2);
    v.s13 = a.ss13;
    v.s2 = a.ss2;
  }
  return v;
}

// Token and slot row of the entry's i-th token.
__device__ __forceinline__ void fp8_token(const Fp8ExpertLaunch& a, const int32_t* slots, const Fp8Entry& v, int i,
                                          int& tok, int& srow) {
  if (v.slot0 >= 0) {
    srow = slots[v.slot0 + i];
    tok = srow / a.e.k;
  } else {
    tok = i;
    srow = a.e.B * a.e.k + i;
  }
}

// ---- gate/up + SwiGLU ----------------------------------------------------------
//
// A task is 8 pairs of an entry: a tile of 8 gate rows (p0 ..) and the 8 up
// rows of the same pairs.  The waves split d by blocks and meet in LDS, where
// the gate sum of a pair finds its up sum.

constexpr int kFp8Pairs = 8;
constexpr int kKeysMaxTokens = 2;
constexpr int kUpRouterWaves = 8;   // waves of a workgroup that scores router rows

template <int XK, int NT, int U>
__device__ __forceinline__ void up_fp8(const Fp8ExpertLaunch& a, const int32_t* slots, const Fp8Entry& v, int p0,
                                       f32x4* s_acc) {
  constexpr int TOK = XTraits<XK>::kTokens, COLS = XTraits<XK>::kCols;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = (int)(blockDim.x >> 6);
  const int d = a.e.d, KB = (d + kQBlock - 1) / kQBlock, IB = (v.I + kQBlock - 1) / kQBlock;
  Fp8Src<1, NT> s;
  s.K = d;
  s.x = a.e.X;
  s.xs = nullptr;
  s.w[0] = v.W13 + (size_t)p0 * d;
  s.ra[0] = (uint32_t)(lane & 7) * (uint32_t)d;   // I is a multiple of 8: no pair is past it
  s.rb[0] = (uint32_t)(v.I + (lane & 7)) * (uint32_t)d;
  s.sa[0] = v.s13 + (size_t)(p0 / kQBlock) * KB;
  s.sb[0] = v.s13 + (size_t)(IB + p0 / kQBlock) * KB;
  s.row_b[0] = lane >= 32;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int t = nt * TOK + x_token<XK>();
    int tok, sr;
    fp8_token(a, slots, v, t < v.m ? t : v.m - 1, tok, sr);
    s.xo[nt] = (uint32_t)tok * (uint32_t)d * 2;
    s.xso[nt] = 0;
  }
  f32x4 acc[1][NT];
  fp8_wave<XK, 1, NT, U>(s, wave, waves, acc);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) s_acc[(wave * NT + nt) * 64 + lane] = acc[0][nt];
  lds_barrier();
  for (int i = threadIdx.x; i < NT * 32; i += (int)blockDim.x) {
    const int l = i & 31, nt = i >> 5, col = l & 15;
    const int t = nt * TOK + col / COLS;
    if (col % COLS || t >= v.m) continue;
    f32x4 g = s_acc[nt * 64 + l], u = s_acc[nt * 64 + 32 + l];
    for (int w = 1; w < waves; ++w) {
      g += s_acc[(w * NT + nt) * 64 + l];
      u += s_acc[(w * NT + nt) * 64 + 32 + l];
    }
    f32x4 h;
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = silu(g[q]) * u[q];
    int tok, sr;
    fp8_token(a, slots, v, t, tok, sr);
    u32x2 hi, lo;
    uint32_t h0, l0, h1, l1;
    split_bf16x2(h[0], h[1], h0, l0);
    split_bf16x2(h[2], h[3], h1, l1);
    hi = u32x2{h0, h1};
    lo = u32x2{l0, l1};
    const size_t o = (size_t)sr * a.e.hld + p0 + 4 * (l >> 4);
    *reinterpret_cast<u32x2*>(h_hi(a.e) + o) = hi;
    *reinterpret_cast<u32x2*>(h_lo(a.e) + o) = lo;
  }
  lds_barrier();   // s_acc is free for the next task
}

// MAXB: the largest batch of the instantiation (4, 8 or 64).
template <int MAXB>
__device__ __forceinline__ void up_fp8_dispatch(const Fp8ExpertLaunch& a, const int32_t* slots, const Fp8Entry& v,
                                                int p0, f32x4* s_acc) {
  if constexpr (MAXB <= 4) {
    up_fp8<XP4, 1, 4>(a, slots, v, p0, s_acc);
  } else if constexpr (MAXB <= 8) {
    if (v.m <= 4) up_fp8<XP4, 1, 4>(a, slots, v, p0, s_acc);
    else up_fp8<XP8, 1, 4>(a, slots, v, p0, s_acc);
  } else {
    const int nt = (v.m + 15) / 16;
    if (v.m <= 4) up_fp8<XP4, 1, 4>(a, slots, v, p0, s_acc);
    else if (v.m <= 8) up_fp8<XP8, 1, 4>(a, slots, v, p0, s_acc);
    else if (nt <= 1) up_fp8<XB, 1, 4>(a, slots, v, p0, s_acc);
    else if (nt == 2) up_fp8<XB, 2, 2>(a, slots, v, p0, s_acc);
    else if (nt == 3) up_fp8<XB, 3, 2>(a, slots, v, p0, s_acc);
    else up_fp8<XB, 4, 2>(a, slots, v, p0, s_acc);
  }
}

template <int MAXB> struct UpFp8 {
  static constexpr int kWaves = MAXB <= 8 ? 16 : 8;   // at most; 128 or 256 registers a lane
  static constexpr int kTiles = MAXB <= 16 ? 1 : 4;
};

template <int MAXB>
__global__ __launch_bounds__(UpFp8<MAXB>::kWaves * 64) void expert_up_fp8_kernel(Fp8ExpertLaunch a) {
  constexpr int NW = UpFp8<MAXB>::kWaves;
  constexpr int kAccBytes = NW * UpFp8<MAXB>::kTiles * 64 * (int)sizeof(f32x4);
  constexpr int kScratch = MAXB > 8 && kPlanFromIdsBytes > kAccBytes ? kPlanFromIdsBytes : kAccBytes;
  __shared__ int32_t s_plan[kMaxPlanWords];
  __shared__ __align__(16) unsigned char s_scratch[kScratch];
  f32x4* s_acc = reinterpret_cast<f32x4*>(s_scratch);
  const ExpertLaunch& x = a.e;
  const int tiles_r = x.I / kFp8Pairs;
  const int tiles_s = x.Ws13 ? x.Is / kFp8Pairs : 0;
  if constexpr (MAXB <= 8) {
    // With the router rows in this launch, its first router_wgs workgroups
    // score them and leave
    if (MAXB <= 4 && x.router_wgs && (int)blockIdx.x < x.router_wgs) {
      __shared__ float s_rr[kRouterPlayedWaves * kRouterRowsInUp * 2];
      if (threadIdx.x >= kUpRouterWaves * 64) return;   // a barrier counts the waves that have not ended
      router_rows_in_up<bf16_t, kUpRouterWaves>(x, blockIdx.x, s_rr);
      return;
    }
  }
  const int G = (int)gridDim.x - x.router_wgs;
  int task = (int)blockIdx.x - x.router_wgs;
  PlanView p;
  __shared__ int s_order[MAXB > 8 ? kMaxB * kMaxK + kMaxB : 1];
  const bool here = MAXB <= 8 && (x.logits != nullptr || x.lkeys != nullptr);
  if (here) {
    if constexpr (MAXB <= 8) {
      // the shared expert's tiles need no plan: they stream while the tokens
      // are selected
      __shared__ TopkScratch s_tk[kKeysMaxTokens];   // here without ready words: at most 2 tokens, a wave each
      __shared__ int32_t s_ids[64];
      __shared__ float s_w[64];
      if (x.ready) select_own_token(x, s_tk, s_ids, s_w);
      for (; task < tiles_s; task += G) {
        const Fp8Entry v = fp8_entry(a, PlanView{}, 0, 0);
        up_fp8_dispatch<MAXB>(a, nullptr, v, task * kFp8Pairs, s_acc);
      }
      p = x.ready ? wait_token_plan(x, s_plan, s_tk, s_ids) : route_here<false, 1>(x, s_plan, s_tk, s_ids, s_w);
    }
  } else {
    p = (MAXB > 8 && x.ids_in) ? plan_from_ids(x, s_plan, s_scratch) : stage_plan(x, s_plan);
  }
  const int n = wave_uniform(p.n);
  if constexpr (MAXB > 8) {
    // entries of many tokens first
    if (threadIdx.x < 64) order_entries_by_tiles(x, p, n, s_order);
    __syncthreads();
  }
  const int total = tiles_s + n * tiles_r;
  for (; task < total; task += G) {
    const int rt = task - tiles_s;
    int idx = n, tile = task;
    if (rt >= 0) {
      idx = rt / tiles_r;
      tile = rt - idx * tiles_r;
      if (MAXB > 8) idx = wave_uniform(s_order[idx]);
    }
    const Fp8Entry v = fp8_entry(a, p, n, idx);
    up_fp8_dispatch<MAXB>(a, p.slots, v, tile * kFp8Pairs, s_acc);
  }
}

// ---- down + combine ------------------------------------------------------------
//
// A workgroup owns down_rows output rows (16 RT at most) of every entry; its
// waves claim the entries in turn (many tokens first) and leave each slot's
// outputs in an LDS tile, which is then combined in the order of combine_one.
// h is a pair of bf16 planes (hi + lo, about 16 significant bits), so a step
// of the product is two matrix instructions.

template <int RT, int KBM>
__device__ __forceinline__ void down_fp8(const Fp8ExpertLaunch& a, const int32_t* slots, const Fp8Entry& v, int r0,
                                         int r_end, float* s_y, int rows) {
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int I = v.I, IB = (I + kQBlock - 1) / kQBlock;
  const f32x4 fzero = {0.f, 0.f, 0.f, 0.f};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  u32x4 wa[RT][KBM], wb[RT][KBM];
  float sc[RT][KBM];
  // rows past the range re-read its last one (the first row of the range is uniform)
  const uint8_t* W = v.W2 + (size_t)r0 * I;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int ra = 16 * rt + (lane & 7), rb = ra + 8, last = r_end - 1 - r0;
    const uint32_t oa = (uint32_t)((ra < last ? ra : last) * I), ob = (uint32_t)((rb < last ? rb : last) * I);
    const int rs = 16 * rt + 4 * g;
#pragma unroll
    for (int kb = 0; kb < KBM; ++kb) {
      const int kc = kb < IB ? kb : IB - 1;
      uint32_t c = (uint32_t)(kc * kQBlock + 16 * (lane >> 3));
      c = c < (uint32_t)(I - 16) ? c : (uint32_t)(I - 16);
      wa[rt][kb] = ld128_stream(W + (oa + c));
      wb[rt][kb] = ld128_stream(W + (ob + c));
      sc[rt][kb] = v.s2[(uint32_t)((r0 + (rs < last ? rs : last)) / kQBlock * IB + kc)];
    }
  }
  for (int t0 = 0; t0 < v.m; t0 += 16) {
    const int t = t0 + col;
    int tok, sr;
    fp8_token(a, slots, v, t < v.m ? t : v.m - 1, tok, sr);
    const bf16_t* hh = h_hi(a.e) + (size_t)sr * a.e.hld;
    const bf16_t* hl = h_lo(a.e) + (size_t)sr * a.e.hld;
    u32x4 hv[KBM][4], lv[KBM][4];
#pragma unroll
    for (int kb = 0; kb < KBM; ++kb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = kb * kQBlock + 32 * g + 8 * j;
        const int cc = c < I - 8 ? c : I - 8;
        hv[kb][j] = ld128(hh + cc);
        lv[kb][j] = ld128(hl + cc);
        if (c >= I) hv[kb][j] = lv[kb][j] = zero;
      }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      f32x4 y = fzero;
#pragma unroll
      for (int kb = 0; kb < KBM; ++kb) {
        if (kb < IB) {
          u32x4 lo, hi;
          w_operand(wa[rt][kb], wb[rt][kb], lo, hi);
          const int c0 = kb * kQBlock + 32 * g;
          if (c0 >= I) lo = zero;
          if (c0 + 16 >= I) hi = zero;
          bf16x8 wv[4];
          wv[0] = widen8(lo[0], lo[1]);
          wv[1] = widen8(lo[2], lo[3]);
          wv[2] = widen8(hi[0], hi[1]);
          wv[3] = widen8(hi[2], hi[3]);
          f32x4 q = fzero;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], __builtin_bit_cast(bf16x8, hv[kb][j]), q, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], __builtin_bit_cast(bf16x8, lv[kb][j]), q, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(sc[rt][kb], q[i], y[i]);
        }
      }
      const int r = 16 * rt + 4 * g;
      if (t < v.m && r < rows) *reinterpret_cast<f32x4*>(s_y + (size_t)sr * rows + r) = y;
    }
  }
}

constexpr int kFp8DownWaves = 8;

template <int RT, int KBM>
__global__ __launch_bounds__(kFp8DownWaves * 64) void expert_down_combine_fp8_kernel(Fp8ExpertLaunch a) {
  __shared__ int32_t s_plan[kMaxPlanWords];
  __shared__ float s_tw[kMaxB * kMaxK];
  __shared__ int s_order[kMaxB * kMaxK + kMaxB];
  __shared__ int s_next;
  extern __shared__ f32x4 s_out[];
  float* s_y = reinterpret_cast<float*>(s_out);   // [B*k + B][rows], rows a multiple of 4
  const ExpertLaunch& x = a.e;
  const int rows = x.down_rows;
  // the router rows' keys of the gate/up launch, zero again for the next call
  if (x.lkeys) {
    const int n = x.B * x.E;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < kKeyCopies * n; i += gridDim.x * blockDim.x)
      x.lkeys[(i / n) * kKeyStride + i % n] = 0u;
  }
  for (int i = threadIdx.x; i < x.B * x.k; i += blockDim.x) s_tw[i] = x.topk_w[i];
  const PlanView p = stage_plan(x, s_plan);
  const int n = wave_uniform(p.n), ne = n + (x.Ws13 ? 1 : 0);
  const int nw = (int)(blockDim.x >> 6), wave = wave_uniform(threadIdx.x >> 6);
  if (wave == 0) {
    order_entries_by_tiles(x, p, ne, s_order);
    if ((threadIdx.x & 63) == 0) s_next = nw;
  }
  __syncthreads();
  const int r0 = (int)blockIdx.x * rows;
  const int r_end = r0 + rows < x.d ? r0 + rows : x.d;
  for (int u = wave; u < ne;) {
    const Fp8Entry v = fp8_entry(a, p, n, wave_uniform(s_order[u]));
    down_fp8<RT, KBM>(a, p.slots, v, r0, r_end, s_y, rows);
    int nx = 0;
    if ((threadIdx.x & 63) == 0) nx = atomicAdd(&s_next, 1);
    u = wave_uniform(nx);
  }
  __syncthreads();
  const int has_shared = x.Ws13 ? 1 : 0;
  for (int i = threadIdx.x; i < x.B * rows; i += blockDim.x) {
    const int t = i / rows, r = i - t * rows;
    if (r0 + r >= x.d) continue;
    const float v = combine_one(s_tw + t * x.k, x.k, has_shared,
                                [&](int j) { return s_y[(size_t)(j < x.k ? t * x.k + j : x.B * x.k + t) * rows + r]; });
    reinterpret_cast<bf16_t*>(x.out)[(size_t)t * x.d + r0 + r] = f32_to_bf16(v);
  }
}

// ---- host side -------------------------------------------------------------------

static const int kCUs = 256;

static int max_entries(const ExpertLaunch& a) {
  const int ns = a.B * a.k;
  return (ns < a.E ? ns : a.E) + (a.Ws13 ? 1 : 0);
}

// Waves of a workgroup that splits KB blocks, U at a time, in as few steps
// as maxw waves allow.
static int split_waves(int KB, int U, int maxw) {
  const int steps = (KB + U * maxw - 1) / (U * maxw);
  return (KB + U * steps - 1) / (U * steps);
}

hipError_t launch_expert_up_fp8(const Fp8ExpertLaunch& a0, hipStream_t st, char* desc, size_t len) {
  Fp8ExpertLaunch a = a0;
  const ExpertLaunch& x = a.e;
  const int KB = (x.d + kQBlock - 1) / kQBlock;
  const int ns = x.B * x.k;
  int g = (ns < x.E ? ns : x.E) * (x.I / kFp8Pairs) + (x.Ws13 ? x.Is / kFp8Pairs : 0);
  int w = split_waves(KB, 4, x.B <= 8 ? 16 : 8);
  // the router rows and the selections need their waves
  if (w < kUpRouterWaves) w = kUpRouterWaves;
  // the whole grid resident at once: no workgroup waits for one that has not started
  const int cap = kCUs * (x.B <= 8 ? 1 : 1);
  if (g > cap) g = cap;
  if (x.ready && g < x.B) g = x.B;
  const dim3 grid((unsigned)(g + x.router_wgs)), block((unsigned)(64 * w));
  if (x.B <= 4) launch(K_EXPERT_UP, expert_up_fp8_kernel<4>, grid, block, 0, st, a);
  else if (x.B <= 8) launch(K_EXPERT_UP, expert_up_fp8_kernel<8>, grid, block, 0, st, a);
  else launch(K_EXPERT_UP, expert_up_fp8_kernel<64>, grid, block, 0, st, a);
  if (desc)
    snprintf(desc, len, "fp8 up grid=%d waves/wg=%d%s%s", g, w, x.router_wgs ? " +router rows" : "",
             (x.logits || x.lkeys) ? " +top-k/plan" : "");
  return hipGetLastError();
}

hipError_t launch_expert_down_combine_fp8(const Fp8ExpertLaunch& a0, hipStream_t st, char* desc, size_t len) {
  Fp8ExpertLaunch a = a0;
  ExpertLaunch& x = a.e;
  // rows split evenly over the compute units in multiples of 4, 16 to 32 a workgroup
  int rows = 4 * ((x.d + 4 * kCUs - 1) / (4 * kCUs));
  rows = rows < 16 ? 16 : (rows > 32 ? 32 : rows);
  x.down_rows = rows;
  const int g = (x.d + rows - 1) / rows;
  int nw = max_entries(x);
  if (nw > kFp8DownWaves) nw = kFp8DownWaves;
  const size_t lds = (size_t)(x.B * x.k + x.B) * rows * sizeof(float);
  const dim3 grid((unsigned)g), block((unsigned)(64 * nw));
  const int longest = x.Ws13 && x.Is > x.I ? x.Is : x.I;
  if (rows <= 16) {
    if (longest <= kQBlock) launch(K_EXPERT_DOWN, (expert_down_combine_fp8_kernel<1, 1>), grid, block, lds, st, a);
    else launch(K_EXPERT_DOWN, (expert_down_combine_fp8_kernel<1, 2>), grid, block, lds, st, a);
  } else {
    if (longest <= kQBlock) launch(K_EXPERT_DOWN, (expert_down_combine_fp8_kernel<2, 1>), grid, block, lds, st, a);
    else launch(K_EXPERT_DOWN, (expert_down_combine_fp8_kernel<2, 2>), grid, block, lds, st, a);
  }
  if (desc) snprintf(desc, len, "fp8 down+combine grid=%d rows/wg=%d waves/wg=%d", g, rows, nw);
  return hipGetLastError();
}

}  // namespace moe
