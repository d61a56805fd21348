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
  int hbase;                  // first row of its token tiles in the tiled h
  const uint8_t *W13, *W2;
  const float *s13, *s2;
};

// s_plan: the plan's words in LDS (moe_plan_words), n: its experts.
__device__ __forceinline__ int plan_max(const Fp8ExpertLaunch& a) {
  const int ns = a.e.B * a.e.k;
  return ns < a.e.E ? ns : a.e.E;
}

__device__ __forceinline__ Fp8Entry fp8_entry(const Fp8ExpertLaunch& a, const int32_t* s_plan, int n, int idx) {
  Fp8Entry v;
  const size_t DB = (size_t)(a.e.d + kQBlock - 1) / kQBlock;
  if (idx < n) {
    const int32_t* offs = s_plan + 1 + plan_max(a);
    const size_t e = (size_t)wave_uniform(s_plan[1 + idx]);
    v.slot0 = wave_uniform(offs[idx]);
    v.hbase = ((a.e.B + 15) & ~15) + v.slot0 + 16 * idx;
    v.m = wave_uniform(offs[idx + 1]) - v.slot0;
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
    v.hbase = 0;
    v.W13 = static_cast<const uint8_t*>(a.e.Ws13);
    v.W2 = static_cast<const uint8_t*>(a.e.Ws2);
    v.s13 = a.ss13;
    v.s2 = a.ss2;
  }
  return v;
}

// Token and slot row of the entry's i-th token.
__device__ __forceinline__ void fp8_token(const Fp8ExpertLaunch& a, const int32_t* s_plan, const Fp8Entry& v, int i,
                                          int& tok, int& srow) {
  if (v.slot0 >= 0) {
    srow = s_plan[2 + 2 * plan_max(a) + v.slot0 + i];
    tok = srow / a.e.k;
  } else {
    tok = i;
    srow = a.e.B * a.e.k + i;
  }
}

// h as the down launch reads it: two bf16 planes (hi + lo, about 16
// significant bits).
//   B <= 8: slot rows [B*k + B][hld] (h_hi, h_lo); only the lanes of an
//   entry's few tokens load.
//   B > 8:  16-token tiles in operand order (a.e.ht_hi, ht_lo): tile row
//   block (hbase + 16 tt) holds, for K block kb and step j, 1 KB: lane 16 g +
//   t its 8 values -- one contiguous load per step.  From slot rows, lanes of
//   different tokens in every quad, the same loads take a compute unit 3.5
//   times as long (37 against 130 bytes/ns), and h crosses once per
//   workgroup.  An entry of up to kRowTokens tokens keeps plain rows in its
//   tile all the same: a tile's steps would bring in a cache line for every
//   16 bytes of a lone token (49.8 us for the batch-32 block, 49.9 without).
constexpr int kRowTokens = 4;
__device__ __forceinline__ uint32_t h_tile(const Fp8ExpertLaunch& a, const Fp8Entry& v, int t) {
  return (uint32_t)(v.hbase + (t & ~15)) * (uint32_t)a.e.hld;
}

// ---- gate/up + SwiGLU ----------------------------------------------------------
//
// A task is 8 RT pairs of an entry: RT tiles of 8 gate rows (p0 ..) and the 8
// up rows of the same pairs.  The waves split d by blocks and meet in LDS,
// where the gate sum of a pair finds its up sum.  At d = 7168 of 384 experts:
// 1 token 13.2 us (a chain of router rows 2.6, selection 2.8 and one task 5),
// 8 tokens 25.8 (112 MB: 4.7 of routing, then the stream), 64 tokens, I = 256,
// 47.7 (200 MB: 4.2 of plan, then 5.9 TB/s until workgroups end, from 34 on;
// the last at 46: tasks of 8 to 34 us).

constexpr int kFp8Pairs = 8;
constexpr int kKeysMaxTokens = 2;
constexpr int kUpRouterWaves = 8;   // waves of a workgroup that scores router rows
constexpr int kUpU = 2;             // blocks in flight a wave, B <= 8 (4: the same time, 25 more registers)
constexpr int kUpManyWaves = 4, kUpManyWgs = 2;   // B > 8: waves a workgroup, workgroups a compute unit (256 registers)

template <int XK, int RT, int NT, int U, bool TILED>
__device__ __forceinline__ void up_fp8(const Fp8ExpertLaunch& a, const int32_t* s_plan, const Fp8Entry& v, int p0,
                                       char* s_lds) {
  constexpr int kWaveLds = fp8_wave_lds<XK, RT, NT>();
  constexpr int TOK = XTraits<XK>::kTokens, COLS = XTraits<XK>::kCols;
  const int lane = own_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = (int)(blockDim.x >> 6);
  const int d = a.e.d, KB = (d + kQBlock - 1) / kQBlock, IB = (v.I + kQBlock - 1) / kQBlock;
  Fp8Src<XK, RT, NT> s;
  s.K = d;
  s.lane = lane;
  s.x = buffer_of(a.e.X);
  s.xs = nullptr;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    s.w[rt] = buffer_of(v.W13 + (size_t)(p0 + 8 * rt) * d);
    s.ra[rt] = (uint32_t)(lane >> 3) * (uint32_t)d;   // I is a multiple of 16: no pair is past it
    s.rb[rt] = (uint32_t)(v.I + (lane >> 3)) * (uint32_t)d;
    s.sa[rt] = v.s13 + (size_t)(p0 / kQBlock) * KB;
    s.sb[rt] = v.s13 + (size_t)(IB + p0 / kQBlock) * KB;
    s.row_b[rt] = lane >= 32;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < x_rows<XK>(); ++i) {
      const int t = nt * TOK + x_load_token<XK>(lane, i);
      int tok, sr;
      fp8_token(a, s_plan, v, t < v.m ? t : v.m - 1, tok, sr);
      s.xo[nt][i] = t < v.m ? (uint32_t)tok * (uint32_t)d * 2 : kNoLoad;
    }
    s.xso[nt] = 0;
  }
  f32x4 acc[RT][NT];
  fp8_wave<XK, RT, NT, U>(s, wave, waves, s_lds + wave * kWaveLds, acc);
  f32x4* mine = reinterpret_cast<f32x4*>(s_lds + wave * kWaveLds);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mine[(rt * NT + nt) * 64 + lane] = acc[rt][nt];
  lds_barrier();
  for (int i = threadIdx.x; i < RT * NT * 32; i += (int)blockDim.x) {
    const int l = i & 31, rt = (i >> 5) / NT, nt = (i >> 5) % NT, col = l & 15;
    const int t = nt * TOK + col / COLS;
    if (col % COLS || t >= v.m) continue;
    const f32x4* sum = reinterpret_cast<const f32x4*>(s_lds) + (i >> 5) * 64 + l;
    f32x4 g = sum[0], u = sum[32];
    for (int w = 1; w < waves; ++w) {
      g += sum[w * (kWaveLds / 16)];
      u += sum[w * (kWaveLds / 16) + 32];
    }
    f32x4 h;
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = silu(g[q]) * u[q];
    int tok, sr;
    fp8_token(a, s_plan, v, t, tok, sr);
    uint32_t h0, l0, h1, l1;
    split_bf16x2(h[0], h[1], h0, l0);
    split_bf16x2(h[2], h[3], h1, l1);
    const int i0 = p0 + 8 * rt + 4 * (l >> 4);
    if constexpr (TILED) {
      const size_t o = v.m <= kRowTokens ? (size_t)(v.hbase + t) * a.e.hld + i0 : (size_t)h_tile(a, v, t) + (i0 >> 7) * 2048 + ((i0 >> 3) & 3) * 512 + ((i0 >> 5) & 3) * 128 + (t & 15) * 8 + (i0 & 7);
      *reinterpret_cast<u32x2*>(a.e.ht_hi + o) = u32x2{h0, h1};
      *reinterpret_cast<u32x2*>(a.e.ht_lo + o) = u32x2{l0, l1};
    } else {
      const size_t o = (size_t)sr * a.e.hld + i0;
      *reinterpret_cast<u32x2*>(h_hi(a.e) + o) = u32x2{h0, h1};
      *reinterpret_cast<u32x2*>(h_lo(a.e) + o) = u32x2{l0, l1};
    }
  }
  lds_barrier();   // the buffers are free for the next task
}

// A task of 8 pairs of an entry of at most 16 tokens.  MAXB: the largest
// batch of the instantiation (4, 8 or 64).
template <int MAXB>
__device__ __forceinline__ void up_fp8_light(const Fp8ExpertLaunch& a, const int32_t* s_plan, const Fp8Entry& v, int p0,
                                             char* s_lds) {
  constexpr bool MANY = MAXB > 8;
  constexpr int U = MANY ? 4 : kUpU;
  if (MAXB <= 4 || v.m <= 4) {
    up_fp8<XP4, 1, 1, U, MANY>(a, s_plan, v, p0, s_lds);
  } else if constexpr (MAXB > 4) {
    if (!MANY || v.m <= 8) up_fp8<XP8, 1, 1, U, MANY>(a, s_plan, v, p0, s_lds);
    else if constexpr (MANY) up_fp8<XB, 1, 1, U, MANY>(a, s_plan, v, p0, s_lds);
  }
}

// A task of 16 pairs of an entry of more than 16 tokens: its activations, four
// to eight times a tile's weight bytes, are read half as often as for 8.
__device__ __forceinline__ void up_fp8_heavy(const Fp8ExpertLaunch& a, const int32_t* s_plan, const Fp8Entry& v, int p0,
                                             char* s_lds) {
  if (v.m <= 32) up_fp8<XB, 2, 2, 2, true>(a, s_plan, v, p0, s_lds);
  else if (v.m <= 48) up_fp8<XB, 2, 3, 1, true>(a, s_plan, v, p0, s_lds);
  else up_fp8<XB, 2, 4, 1, true>(a, s_plan, v, p0, s_lds);
}

// Waves of a workgroup: at most 16 of 128 registers (B <= 8), or 4 of 256.
template <int MAXB> struct UpFp8 {
  static constexpr int kWaves = MAXB <= 8 ? 16 : kUpManyWaves;
  static constexpr int kWaveLds = MAXB <= 4 ? fp8_wave_lds<XP4, 1, 1>() : MAXB <= 8 ? fp8_wave_lds<XP8, 1, 1>() : fp8_wave_lds<XB, 2, 4>();
};

template <int MAXB>
__global__ __launch_bounds__(UpFp8<MAXB>::kWaves * 64, MAXB <= 8 ? 1 : kUpManyWgs) void expert_up_fp8_kernel(Fp8ExpertLaunch a) {
  __shared__ int32_t s_plan[kMaxPlanWords];
  extern __shared__ __align__(16) char s_lds[];   // a buffer per wave; first plan_from_ids' scratch
  const ExpertLaunch& x = a.e;
  // where the tokens are selected here: without ready words at most two of
  // them, a wave each
  __shared__ TopkScratch s_tk[MAXB <= 8 ? kKeysMaxTokens : 1];
  __shared__ int32_t s_ids[64];
  __shared__ float s_w[64];
  __shared__ int s_order[MAXB > 8 ? kMaxB * kMaxK + kMaxB : 1];
  __shared__ int s_heavy[3];
  if constexpr (MAXB <= 4) {
    // With the router rows in this launch, its first router_wgs workgroups
    // score them and leave
    if ((int)blockIdx.x < x.router_wgs) {
      __shared__ float s_rr[kRouterPlayedWaves * kRouterRowsInUp * 2];
      if (threadIdx.x >= kUpRouterWaves * 64) return;   // a barrier counts the waves that have not ended
      router_rows_in_up<bf16_t, kUpRouterWaves>(x, blockIdx.x, s_rr);
      return;
    }
  }
  if constexpr (MAXB <= 8) {
    if (x.ready) select_own_token(x, s_tk, s_ids, s_w);
  }
  const int G = (int)gridDim.x - x.router_wgs, wg = (int)blockIdx.x - x.router_wgs;
  if constexpr (MAXB <= 8) {
    // Tasks of 8 pairs: the shared expert's, then the routed entries'.  Where
    // the tokens are selected here the shared tiles, which need no plan,
    // stream meanwhile (a loop of its own: one loop over both, with the
    // routing inside it, spilled 24 registers).
    const int tiles_r = x.I / kFp8Pairs, tiles_s = x.Ws13 ? x.Is / kFp8Pairs : 0;
    int task = wg;
    if (x.logits || x.lkeys) {
      for (; task < tiles_s; task += G)
        up_fp8_light<MAXB>(a, s_plan, fp8_entry(a, s_plan, -1, 0), task * kFp8Pairs, s_lds);
      if (x.ready) wait_token_plan(x, s_plan, s_tk, s_ids);
      else route_here<false, 1>(x, s_plan, s_tk, s_ids, s_w);
    } else {
      stage_plan(x, s_plan);
    }
    const int n = wave_uniform(s_plan[0]), total = tiles_s + n * tiles_r;
    for (; task < total; task += G) {
      const int idx = task < tiles_s ? n : (task - tiles_s) / tiles_r;
      const int tile = task < tiles_s ? task : task - tiles_s - idx * tiles_r;
      up_fp8_light<MAXB>(a, s_plan, fp8_entry(a, s_plan, n, idx), tile * kFp8Pairs, s_lds);
    }
  } else {
    // Heavy tasks (entries of more than 16 tokens, the shared expert's first,
    // then by falling token tiles: 16 pairs each) go one to a workgroup, then
    // the light ones (8 pairs) so that the workgroups' costs come out even:
    // measured, a task of 2, 3 or 4 token tiles takes as long as 2, 3 or 4
    // light ones.  Round r of the light tasks goes to the workgroups, last[r]
    // on, that have room for more than r of them; tiles that lie next to each
    // other are read at the same time.  (In turns, forwards and backwards,
    // the workgroups with heavy tasks ended 15 us after the others in the
    // batch-64 workload: gate/up 52.6 us.)
    const PlanView p = x.ids_in ? plan_from_ids(x, s_plan, reinterpret_cast<unsigned char*>(s_lds)) : stage_plan(x, s_plan);
    const int n = wave_uniform(s_plan[0]);
    if (threadIdx.x < 64) {
      order_entries_by_tiles(x, p, n, s_order);
      int c2 = 0, c3 = 0, c4 = 0;   // entries of at least 2, 3, 4 token tiles
      for (int e0 = 0; e0 < n; e0 += 64) {
        const int e = e0 + (int)threadIdx.x, m = e < n ? p.offs[e + 1] - p.offs[e] : 0;
        c2 += __popcll(__ballot(m > 16));
        c3 += __popcll(__ballot(m > 32));
        c4 += __popcll(__ballot(m > 48));
      }
      if (threadIdx.x == 0) {
        s_heavy[0] = c2;
        s_heavy[1] = c3;
        s_heavy[2] = c4;
      }
    }
    __syncthreads();
    const int c2 = wave_uniform(s_heavy[0]), c3 = wave_uniform(s_heavy[1]), c4 = wave_uniform(s_heavy[2]);
    const int th = x.I / (2 * kFp8Pairs), tl = x.I / kFp8Pairs;
    const int sh = x.Ws13 && x.B > 16 ? x.Is / (2 * kFp8Pairs) : 0, slt = x.Ws13 && x.B <= 16 ? x.Is / kFp8Pairs : 0;
    // heavy tasks of at least 2, 3, 4 token tiles
    const int h2 = c2 * th + sh, h3 = c3 * th + (x.B > 32 ? sh : 0), h4 = c4 * th + (x.B > 48 ? sh : 0);
    for (int task = wg; task < h2; task += G) {
      int idx = n, tile = task;
      if (task >= sh) {
        const int q = (task - sh) / th;
        idx = wave_uniform(s_order[q]);
        tile = task - sh - q * th;
      }
      up_fp8_heavy(a, s_plan, fp8_entry(a, s_plan, n, idx), tile * 2 * kFp8Pairs, s_lds);
    }
    const int light = slt + (n - c2) * tl;
    auto clip = [&](int h) { return h < G ? h : G; };   // more heavy tasks than workgroups: every one has had some
    const int g2 = h2 > G ? 0 : h2, g3 = h2 > G ? 0 : clip(h3), g4 = h2 > G ? 0 : clip(h4);
    // the fewest rounds with room for all of them
    int T = 1;
    auto room = [&](int T) {
      auto pos = [](int v) { return v > 0 ? v : 0; };
      return g4 * pos(T - 4) + (g3 - g4) * pos(T - 3) + (g2 - g3) * pos(T - 2) + (G - g2) * T;
    };
    while (room(T) < light && T < 1024) ++T;
    int base = 0;
    for (int r = 0; r < T; ++r) {
      const int first = T - 4 > r ? 0 : (T - 3 > r ? g4 : (T - 2 > r ? g3 : g2));
      const int task = base + wg - first;
      base += G - first;
      if (wg < first || task >= light) continue;
      int idx = n, tile = task;
      if (task >= slt) {
        const int q = (task - slt) / tl;
        idx = wave_uniform(s_order[c2 + q]);
        tile = task - slt - q * tl;
      }
      up_fp8_light<MAXB>(a, s_plan, fp8_entry(a, s_plan, n, idx), tile * kFp8Pairs, s_lds);
    }
  }
}

// ---- down + combine ------------------------------------------------------------
//
// A workgroup owns down_rows output rows (16 RT at most) of every entry; its
// waves claim the entries in turn (many tokens first) and leave each slot's
// outputs in an LDS tile, which is then combined in the order of combine_one.
// A wave requests the next entry's rows and scales before it multiplies
// the current one.  h is a pair of bf16 planes, so a step of the
// product is two matrix instructions.  The same workloads: 5.8, 14.7 (56 MB,
// 3.8 TB/s) and 28.0 us (102 MB, 3.7 TB/s); every compute unit reads all of h,
// which bounds it beside the rows.

template <int RT, int KBM>
struct DownRegs {
  u32x4 wa[RT][KBM], wb[RT][KBM];
  float sc[RT][KBM];
};
template <int KBM>
struct DownH {
  u32x4 hv[KBM][4], lv[KBM][4];
};

template <int RT, int KBM, bool TILED>
struct DownFp8 {
  const Fp8ExpertLaunch& a;
  const int32_t* s_plan;
  int r0, r_end, rows;
  float* s_y;
  char* lds;
  coherent_rsrc_t hi, lo;   // h planes: a lane past the entry's tokens or columns reads zeros from an offset past their end

  // token tile at t0: h operands
  __device__ __forceinline__ void load_h(const Fp8Entry& v, int t0, DownH<KBM>& h) const {
    const int lane = threadIdx.x & 63, g = lane >> 4, t = t0 + (lane & 15);
    const bool tiled = TILED && v.m > kRowTokens;   // uniform
    uint32_t base;
    if (tiled) {
      base = h_tile(a, v, t0) * 2 + lane * 16;
    } else {
      int row = v.hbase + t;
      if constexpr (!TILED) {
        int tok;
        fp8_token(a, s_plan, v, t < v.m ? t : v.m - 1, tok, row);
      }
      base = (uint32_t)row * (uint32_t)a.e.hld * 2 + 64 * g;
    }
    const uint32_t per_kb = tiled ? 4096 : 256, per_j = tiled ? 1024 : 16;
#pragma unroll
    for (int kb = 0; kb < KBM; ++kb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool ok = t < v.m && kb * kQBlock + 32 * g + 8 * j < v.I;
        const uint32_t o = ok ? base + kb * per_kb + j * per_j : kNoLoad;
        h.hv[kb][j] = __builtin_amdgcn_raw_buffer_load_b128(hi, o, 0, 0);
        h.lv[kb][j] = __builtin_amdgcn_raw_buffer_load_b128(lo, o, 0, 0);
      }
  }

  __device__ __forceinline__ void load(const Fp8Entry& v, DownRegs<RT, KBM>& r) const {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int I = v.I, IB = (I + kQBlock - 1) / kQBlock;
    // rows past the range re-read its last one
    const uint8_t* W = v.W2 + (size_t)r0 * I;
    const int last = r_end - 1 - r0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int ra = 16 * rt + (lane >> 3), rb = ra + 8, rs = 16 * rt + 4 * g;
      const uint32_t oa = (uint32_t)((ra < last ? ra : last) * I), ob = (uint32_t)((rb < last ? rb : last) * I);
#pragma unroll
      for (int kb = 0; kb < KBM; ++kb) {
        const int kc = kb < IB ? kb : IB - 1;
        uint32_t c = (uint32_t)(kc * kQBlock + 16 * (lane & 7));
        c = c < (uint32_t)(I - 16) ? c : (uint32_t)(I - 16);
        r.wa[rt][kb] = ld128_stream(W + (oa + c));
        r.wb[rt][kb] = ld128_stream(W + (ob + c));
        r.sc[rt][kb] = v.s2[(uint32_t)((r0 + (rs < last ? rs : last)) / kQBlock * IB + kc)];
      }
    }
  }

  // the entry's rows from registers to the wave's buffer
  __device__ __forceinline__ void keep(const DownRegs<RT, KBM>& r, float (&sc)[RT][KBM]) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int kb = 0; kb < KBM; ++kb) {
        rows128_store(lane, lds + (rt * KBM + kb) * 2048, r.wa[rt][kb], r.wb[rt][kb]);
        sc[rt][kb] = r.sc[rt][kb];
      }
  }

  __device__ __forceinline__ void products(const Fp8Entry& v, const float (&sc)[RT][KBM], DownH<KBM>& h) const {
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int I = v.I, IB = (I + kQBlock - 1) / kQBlock;
    const f32x4 fzero = {0.f, 0.f, 0.f, 0.f};
    const u32x4 zero = {0u, 0u, 0u, 0u};
    for (int t0 = 0;;) {
      const int t = t0 + col;
      int tok, sr;
      fp8_token(a, s_plan, v, t < v.m ? t : v.m - 1, tok, sr);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        f32x4 y = fzero;
#pragma unroll
        for (int kb = 0; kb < KBM; ++kb) {
          if (kb < IB) {
            u32x4 w0, w1;
            rows128_load(lane, lds + (rt * KBM + kb) * 2048, w0, w1);
            const int c0 = kb * kQBlock + 32 * g;
            if (c0 >= I) w0 = zero;
            if (c0 + 16 >= I) w1 = zero;
            const bf16x8 wv[4] = {widen8(w0[0], w0[1]), widen8(w0[2], w0[3]), widen8(w1[0], w1[1]), widen8(w1[2], w1[3])};
            f32x4 q = fzero;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], __builtin_bit_cast(bf16x8, h.hv[kb][j]), q, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], __builtin_bit_cast(bf16x8, h.lv[kb][j]), q, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(sc[rt][kb], q[i], y[i]);
          }
        }
        const int rr = 16 * rt + 4 * g;
        if (t < v.m && rr < rows) *reinterpret_cast<f32x4*>(s_y + (size_t)sr * rows + rr) = y;
        __builtin_amdgcn_sched_barrier(0);   // one tile's operands at a time (registers)
      }
      t0 += 16;
      if (t0 >= v.m) break;
      load_h(v, t0, h);
    }
  }
};

template <int KBM> struct DownWaves { static constexpr int kMax = KBM == 1 ? 16 : 12; };

template <int RT, int KBM, bool TILED>
__global__ __launch_bounds__(DownWaves<KBM>::kMax * 64) void expert_down_combine_fp8_kernel(Fp8ExpertLaunch a) {
  __shared__ int32_t s_plan[kMaxPlanWords];
  __shared__ float s_tw[kMaxB * kMaxK];
  __shared__ int s_order[kMaxB * kMaxK + kMaxB];
  __shared__ int s_next;
  extern __shared__ __align__(16) char s_dyn[];   // a buffer per wave, then s_y [B*k + B][rows], rows a multiple of 4
  const ExpertLaunch& x = a.e;
  const int rows = x.down_rows;
  const int nw = (int)(blockDim.x >> 6), wave = wave_uniform(threadIdx.x >> 6);
  float* s_y = reinterpret_cast<float*>(s_dyn + nw * (RT * KBM * 2048));
  // the router rows' keys of the gate/up launch, zero again for the next call
  if (x.lkeys) {
    const int n = x.B * x.E;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < kKeyCopies * n; i += gridDim.x * blockDim.x)
      x.lkeys[(i / n) * kKeyStride + i % n] = 0u;
  }
  for (int i = threadIdx.x; i < x.B * x.k; i += blockDim.x) s_tw[i] = x.topk_w[i];
  const PlanView p = stage_plan(x, s_plan);
  const int n = wave_uniform(p.n), ne = n + (x.Ws13 ? 1 : 0);
  if (wave == 0) {
    // up to 16 tokens every entry has one token tile: any order will do
    if (x.B > 16) order_entries_by_tiles(x, p, ne, s_order);
    if ((threadIdx.x & 63) == 0) s_next = nw;
  }
  __syncthreads();
  const int r0 = (int)blockIdx.x * rows;
  const int plane = (TILED ? ht_rows(x.B, x.k, x.E) : x.B * x.k + x.B) * x.hld * 2;
  const void* hh = TILED ? x.ht_hi : h_hi(x);
  const void* hl = TILED ? x.ht_lo : h_lo(x);
  const DownFp8<RT, KBM, TILED> d = {a, s_plan, r0, r0 + rows < x.d ? r0 + rows : x.d, rows, s_y,
                                     s_dyn + wave * (RT * KBM * 2048),
                                     __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(hh), 0, plane, 0x00020000),
                                     __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(hl), 0, plane, 0x00020000)};
  auto claim = [&] {
    int u = 0;
    if ((threadIdx.x & 63) == 0) u = atomicAdd(&s_next, 1);
    return wave_uniform(u);
  };
  auto entry = [&](int u) { return fp8_entry(a, s_plan, n, x.B > 16 ? wave_uniform(s_order[u]) : u); };
  if (wave < ne) {
    // The current entry's rows go to the wave's buffer as they arrive, which
    // frees their registers for the next entry's; its h is requested before
    // those, since loads return in order.
    DownRegs<RT, KBM> r;
    DownH<KBM> h;
    float sc[RT][KBM];
    Fp8Entry v = entry(wave);
    d.load(v, r);
    for (;;) {
      d.load_h(v, 0, h);
      d.keep(r, sc);
      const int u = claim();
      if (u >= ne) break;
      const Fp8Entry next = entry(u);
      d.load(next, r);
      __builtin_amdgcn_sched_barrier(0);
      d.products(v, sc, h);
      v = next;
    }
    d.products(v, sc, h);
  }
  __syncthreads();
  // four rows a thread (rows, r0 and d are multiples of 4), in combine_one's
  // order; four slots' outputs requested at a time
  const int quads = rows / 4;
  for (int i = threadIdx.x; i < x.B * quads; i += blockDim.x) {
    const int t = i / quads, r = 4 * (i - t * quads);
    if (r0 + r >= x.d) continue;
    const float* w = s_tw + t * x.k;
    auto y_of = [&](int slot) { return *reinterpret_cast<const f32x4*>(s_y + (size_t)slot * rows + r); };
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < x.k; j0 += 4) {
      f32x4 y[4];
      float wj[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = j0 + q < x.k ? j0 + q : x.k - 1;
        y[q] = y_of(t * x.k + j);
        wj[q] = w[j];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (j0 + q < x.k) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(wj[q], y[q][e], v[e]);
        }
    }
    if (x.Ws13) v += y_of(x.B * x.k + t);
    const u32x2 o = {(uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                     (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
    *reinterpret_cast<u32x2*>(reinterpret_cast<bf16_t*>(x.out) + (size_t)t * x.d + r0 + r) = o;
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

hipError_t launch_expert_up_fp8(const Fp8ExpertLaunch& a0, hipStream_t st, Fp8Shape* shape) {
  Fp8ExpertLaunch a = a0;
  const ExpertLaunch& x = a.e;
  const int KB = (x.d + kQBlock - 1) / kQBlock;
  const int ns = x.B * x.k;
  int g = (ns < x.E ? ns : x.E) * (x.I / kFp8Pairs) + (x.Ws13 ? x.Is / kFp8Pairs : 0);
  // B <= 8: as many waves to a workgroup as leave every task resident at once
  // (16 waves a compute unit): a task's bytes are then all in flight where
  // there are few tasks, and small workgroups finish evenly where there are
  // many.  Router rows and selections need four.
  int w, cap;
  if (x.B <= 8) {
    w = split_waves(KB, kUpU, g <= kCUs ? 16 : 8);
    if (w < kUpRouterWaves) w = kUpRouterWaves;
    cap = kCUs * (16 / w);
  } else {
    w = split_waves(KB, 4, kUpManyWaves);
    cap = kCUs * kUpManyWgs;
  }
  if (g > cap) g = cap;
  if (x.ready && g < x.B) g = x.B;
  const dim3 grid((unsigned)(g + x.router_wgs)), block((unsigned)(64 * w));
  auto lds = [&](int wave, int least) { return (uint32_t)(w * wave > least ? w * wave : least); };
  if (x.B <= 4) launch(K_EXPERT_UP, expert_up_fp8_kernel<4>, grid, block, lds(UpFp8<4>::kWaveLds, 0), st, a);
  else if (x.B <= 8) launch(K_EXPERT_UP, expert_up_fp8_kernel<8>, grid, block, lds(UpFp8<8>::kWaveLds, 0), st, a);
  else launch(K_EXPERT_UP, expert_up_fp8_kernel<64>, grid, block, lds(UpFp8<64>::kWaveLds, kPlanFromIdsBytes), st, a);
  *shape = {g, w, 0, 0, 0};
  return hipGetLastError();
}

template <int RT, int KBM>
static void go_down(const Fp8ExpertLaunch& a, int nw, int y_bytes, dim3 grid, hipStream_t st) {
  const dim3 block((unsigned)(64 * nw));
  const uint32_t lds = (uint32_t)(y_bytes + nw * RT * KBM * 2048);
  if (a.e.ht_hi) launch(K_EXPERT_DOWN, (expert_down_combine_fp8_kernel<RT, KBM, true>), grid, block, lds, st, a);
  else launch(K_EXPERT_DOWN, (expert_down_combine_fp8_kernel<RT, KBM, false>), grid, block, lds, st, a);
}

hipError_t launch_expert_down_combine_fp8(const Fp8ExpertLaunch& a0, hipStream_t st, Fp8Shape* shape) {
  Fp8ExpertLaunch a = a0;
  ExpertLaunch& x = a.e;
  const int longest = x.Ws13 && x.Is > x.I ? x.Is : x.I, kbm = longest <= kQBlock ? 1 : 2;
  int nw = max_entries(x);
  const int maxw = kbm == 1 ? DownWaves<1>::kMax : DownWaves<2>::kMax;
  if (nw > maxw) nw = maxw;
  // rows split evenly over the compute units in multiples of 4, 16 to 32 a
  // workgroup, and as many as fit in LDS beside the waves' buffers (160 KB,
  // of which the plan takes 17 KB)
  const int slots = x.B * x.k + x.B;
  int rows = 4 * ((x.d + 4 * kCUs - 1) / (4 * kCUs));
  rows = rows < 16 ? 16 : (rows > 32 ? 32 : rows);
  auto fits = [&](int r) { return slots * r * 4 + nw * (r > 16 ? 2 : 1) * kbm * 2048 <= 143 * 1024; };
  while (nw > 8 && !fits(rows)) --nw;
  while (rows > 4 && !fits(rows)) rows -= 4;
  x.down_rows = rows;
  const int g = (x.d + rows - 1) / rows, y = slots * rows * 4;
  if (rows <= 16) {
    if (kbm == 1) go_down<1, 1>(a, nw, y, dim3((unsigned)g), st);
    else go_down<1, 2>(a, nw, y, dim3((unsigned)g), st);
  } else {
    if (kbm == 1) go_down<2, 1>(a, nw, y, dim3((unsigned)g), st);
    else go_down<2, 2>(a, nw, y, dim3((unsigned)g), st);
  }
  *shape = {g, nw, rows, 0, 0};
  return hipGetLastError();
}

}  // namespace moe
