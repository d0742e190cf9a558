// dg_moe.hip -- a whole mixture-of-experts layer for a few tokens (decode) in
// two kernels:
//
//   moe_up_kernel    routing (top-k of the logits), and for every chosen
//                    (token, expert) pair  h = w silu(x.Wg^T) (x.Wu^T)
//   moe_down_kernel  y = residual + sum over the token's pairs of h.W2^T
//
// Bound: the chosen experts' weights, each read once (a few tokens give each
// weight a handful of operations).  So both kernels stream weights from HBM
// straight into registers with 16-byte nontemporal loads, several units
// (dg_stream.h: 16 rows x 128 K) ahead, and everything else is arranged around
// that: the activations (bf16, a few KB) are re-read through the L2 by every
// workgroup, fp8 weights are widened to bf16 in registers (exact), and the
// products run on the bf16 MFMA with the tokens of one expert as its 16
// columns -- the matrix unit has an order of magnitude to spare.
//
// The routing weight is folded into h, so the second kernel only sums; a
// workgroup of it owns 16 R output columns for all experts and tokens, which
// makes the combination over experts a private sum: no atomics, a fixed order.
//
// h is rounded to bf16 once (the MFMA's operand type; relative error 2^-9 per
// value, the size of the output's own rounding); every sum is fp32.
#include <climits>
#include <cstdint>

#include "../../include/dg.h"
#include "dg_act.h"
#include "dg_stream.h"

namespace dg {
namespace {

using namespace stream;

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kMaxTokens = 64;
constexpr int kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kMaxExperts = 512;

struct MoeParams {
  const uint16_t* x;         // bf16 [T,H]
  const float* logits;       // fp32 [T,E], or null: ids / weights are given
  int32_t* ids;              // [T,k]
  float* weights;            // [T,k]
  const uint8_t* w13;        // [E,2I,H]
  const float* s13;          // [E,2I/128,H/128] (fp8 weights)
  const uint8_t* w2;         // [E,H,I]
  const float* s2;           // [E,H/128,I/128]
  const uint16_t* residual;  // bf16 [T,H] or null
  uint16_t* y;               // bf16 [T,H]
  uint16_t* h;               // bf16 [T*k, I]: the pairs' hidden values
  int t, hid, inter, experts, top_k, scoring, renormalize;
  float scale;
};

// ---- routing tables in LDS -------------------------------------------------
// The (token, expert) pairs of the call, p = token * k + j, sorted by expert;
// a segment is a run of at most 16 NT pairs of one expert, the columns of the
// MFMA tiles that share one pass over that expert's weights.
struct Tables {
  int id[kMaxPairs];            // expert of each pair, -1: none
  float w[kMaxPairs];           // its weight
  uint16_t pair[kMaxPairs];     // sorted position -> pair
  int16_t sid[kMaxPairs];       // sorted position -> expert
  uint16_t rank[kMaxPairs];     // sorted position -> how many pairs of the expert come before
  uint16_t seg[kMaxPairs];      // segment -> its first sorted position
  int npair, nseg;
};

// Maximum over the wave, in every lane's scalar (DPP row shifts, then the two
// row broadcasts; 0 is the identity).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define DG_DPP_MAX(ctrl) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false))
  DG_DPP_MAX(0x111);
  DG_DPP_MAX(0x112);
  DG_DPP_MAX(0x114);
  DG_DPP_MAX(0x118);
  DG_DPP_MAX(0x142);
  DG_DPP_MAX(0x143);
#undef DG_DPP_MAX
  return __builtin_amdgcn_readlane(v, 63);
}

// Order-preserving key of a logit: larger float, larger key; NaN above
// everything (it reaches the token's output, as it would through a sort);
// -inf, "never this expert", 0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 0xffffffffu;
  const uint32_t b = __float_as_uint(l + 0.f);  // -0 counts as 0
  if (b == 0xff800000u) return 0;
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// Top-k of every token's logits, ties to the lowest expert: one wave per
// token, the logits in registers; each round is a maximum over the wave's
// keys and a ballot for the first lane that holds it.
__device__ __forceinline__ void route(const MoeParams& p, Tables& tb, int wave, int lane, bool publish) {
  constexpr int NI = kMaxExperts / 64;
  for (int t = wave; t < p.t; t += kWaves) {
    float l[NI];
    uint32_t key[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < p.experts ? p.logits[(int64_t)t * p.experts + e] : 0.f;
      key[i] = e < p.experts ? logit_key(l[i]) : 0;
    }
    float sum_all = 0.f;  // softmax over every expert (not renormalised)
    float top = 0.f;
    int my_id = -1;
    float my_l = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) best = max(best, key[i]);
      best = wave_max(best);
      int e = -1;
      float v = 0.f;
      if (best != 0) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint64_t m = __ballot(key[i] == best);
          if (m != 0 && e < 0) {
            const int ln = __builtin_ctzll(m);
            e = 64 * i + ln;
            v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(l[i]), ln));
            if (lane == ln) key[i] = 0;
          }
        }
      }
      if (j == 0) {
        top = v;
        if (e >= 0 && !p.renormalize && p.scoring == DG_SCORING_SOFTMAX) {
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (lane + 64 * i < p.experts) sum_all += expf(l[i] - top);
          for (int o = 32; o > 0; o >>= 1) sum_all += __shfl_xor(sum_all, o);
        }
      }
      if (lane == j) {
        my_id = e;
        my_l = v;
      }
    }
    float w = 0.f;
    if (my_id >= 0) w = p.scoring == DG_SCORING_SOFTMAX ? expf(my_l - top) : 1.f / (1.f + expf(-my_l));
    float sum = w;
    for (int o = kMaxTopK / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (p.renormalize)
      w = sum != 0.f ? w / sum : 0.f;  // sum is 0 where no expert is left (or every sigmoid underflows)
    else if (p.scoring == DG_SCORING_SOFTMAX && my_id >= 0)
      w /= sum_all;
    w *= p.scale;
    if (lane < p.top_k) {
      tb.id[t * p.top_k + lane] = my_id;
      tb.w[t * p.top_k + lane] = w;
      if (publish) {
        p.ids[t * p.top_k + lane] = my_id;
        p.weights[t * p.top_k + lane] = w;
      }
    }
  }
}

// Fills the tables.  ROUTE: from the logits (published by workgroup 0), else
// from ids / weights: ids outside [0, E) drop out, a token's repeated expert
// keeps one pair with the sum of its weights.
template <int NT, bool ROUTE>
__device__ __forceinline__ void build_tables(const MoeParams& p, Tables& tb) {
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int np = p.t * p.top_k;
  if constexpr (ROUTE) {
    route(p, tb, wave, lane, blockIdx.x == 0);
  } else {
    for (int q = tid; q < np; q += kThreads) {
      const int id = p.ids[q];
      tb.id[q] = id >= 0 && id < p.experts ? id : -1;
      tb.w[q] = p.weights[q];
    }
  }
  for (int q = np + tid; q < kMaxPairs && q < np + 4; q += kThreads) tb.id[q] = -1;  // the scan reads fours
  if (tid == 0) tb.npair = 0;
  __syncthreads();
  if constexpr (!ROUTE) {
    if (tid < p.t) {
      const int b = tid * p.top_k;
      for (int j = 1; j < p.top_k; ++j) {
        const int id = tb.id[b + j];
        if (id < 0) continue;
        for (int f = 0; f < j; ++f)
          if (tb.id[b + f] == id) {
            tb.w[b + f] += tb.w[b + j];
            tb.id[b + j] = -1;
            break;
          }
      }
    }
    __syncthreads();
  }
  // sorted position of pair q: the pairs of lower experts and the earlier
  // pairs of its own
  for (int q = tid; q < np; q += kThreads) {
    const uint32_t id = (uint32_t)tb.id[q];
    int lower = 0, same = 0;
    for (int o = 0; o < np; o += 4) {
      const int4 v = *reinterpret_cast<const int4*>(&tb.id[o]);
      const uint32_t u[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lower += u[c] < id;
        same += u[c] == id && o + c < q;
      }
    }
    if (id != 0xffffffffu) {
      const int pos = lower + same;
      tb.pair[pos] = (uint16_t)q;
      tb.sid[pos] = (int16_t)id;
      tb.rank[pos] = (uint16_t)same;
      atomicAdd(&tb.npair, 1);
    }
  }
  __syncthreads();
  if (wave == 0) {
    const int n = tb.npair;
    int base = 0;
    for (int c = 0; c < n; c += 64) {
      const int q = c + lane;
      const bool first = q < n && tb.rank[q] % (16 * NT) == 0;
      const uint64_t m = __ballot(first);
      if (first) tb.seg[base + __builtin_popcountll(m & ((1ull << lane) - 1))] = (uint16_t)q;
      base += __builtin_popcountll(m);
    }
    if (lane == 0) tb.nseg = base;
  }
  __syncthreads();
}

// The pair in MFMA column l16 of tile t of the segment that starts at sorted
// position q0, -1 if the column is empty.
__device__ __forceinline__ int column_pair(const Tables& tb, int q0, int e, int t, int l16) {
  const int q = q0 + 16 * t + l16;
  const int qc = q < kMaxPairs ? q : kMaxPairs - 1;
  return q < tb.npair && tb.sid[qc] == e ? (int)tb.pair[qc] : -1;
}

// ---- first kernel ----------------------------------------------------------
// Work item: one segment x 16 hidden columns (16 gate and the 16 matching up
// rows of its expert's w13).  The 8 waves of a workgroup take K blocks round
// robin and meet in LDS once per item.  The workgroup walks its items as one
// stream of units, D of them in flight, so the loads of the next item are
// already out while an item's sums meet.
template <bool FP8W, int NT, bool ROUTE, int D>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(const MoeParams p) {
  constexpr int WL = FP8W ? 2 : 4;
  constexpr int ES = FP8W ? 1 : 2;
  __shared__ Tables tb;
  __shared__ __attribute__((aligned(16))) v4f red[kWaves][2 * NT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  build_tables<NT, ROUTE>(p, tb);

  const int nb = p.hid >> 7, n = (nb + kWaves - 1) / kWaves;
  const int slabs = p.inter >> 4;
  const int items = (int)uniform(tb.nseg) * slabs;
  const int grid = gridDim.x;
  const int mine = items > (int)blockIdx.x ? (items - (int)blockIdx.x + grid - 1) / grid : 0;
  const int total = mine * n;
  const uint32_t row = (uint32_t)p.hid * ES;  // bytes per weight row
  const uint32_t xrow = (uint32_t)p.hid * 2;
  const uint32_t woff = (uint32_t)l16 * row + 16u * lq;

  v4i wg[D][WL], wu[D][WL], xs[D][NT][4];
  float sg[D], su[D];

  // load cursor: the item and its wave-local block
  int li = blockIdx.x, lj = 0;
  const uint8_t* gate = nullptr;
  const float* sgate = nullptr;
  uint32_t xoff[NT];
  auto enter = [&]() {  // the cursor's item
    const bool live = li < items;
    const int s = live ? li / slabs : 0;
    const int n0 = live ? (li - s * slabs) * 16 : 0;
    const int q0 = live ? tb.seg[s] : 0;
    const int e = (int)uniform(live ? tb.sid[q0] : 0);
    gate = p.w13 + ((int64_t)e * 2 * p.inter + n0) * row;
    if constexpr (FP8W) sgate = p.s13 + ((int64_t)e * 2 * (p.inter >> 7) + (n0 >> 7)) * nb;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int pr = live ? column_pair(tb, q0, e, t, l16) : -1;
      xoff[t] = pr >= 0 ? (uint32_t)(pr / p.top_k) * xrow + (FP8W ? 32u : 16u) * lq : kOut;
    }
  };
  auto load = [&](int d) {
    const int kb = wave + kWaves * lj;
    const bool live = li < items && kb < nb;
    const uint32_t wbytes = live ? 15u * row + 128u * ES : 0u;
    const auto rg = rsrc(gate + (int64_t)kb * 128 * ES, wbytes);
    const auto ru = rsrc(gate + (int64_t)p.inter * row + (int64_t)kb * 128 * ES, wbytes);
    const auto rx = rsrc(p.x + (int64_t)kb * 128, live ? (uint32_t)(p.t - 1) * xrow + 256u : 0u);
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      wg[d][i] = load16<kNt>(rg, woff + 64u * i);
      wu[d][i] = load16<kNt>(ru, woff + 64u * i);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xs[d][t][i] = load16<0>(rx, xoff[t] + (FP8W ? 128u * (i >> 1) + 16u * (i & 1) : 64u * i));
    if constexpr (FP8W) {
      const auto rs = rsrc(sgate + kb, live ? 4u : 0u);
      const auto rt = rsrc(sgate + (int64_t)(p.inter >> 7) * nb + kb, live ? 4u : 0u);
      sg[d] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, 0, 0, 0));
      su[d] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rt, 0, 0, 0));
    }
    if (++lj == n) {
      lj = 0;
      li += grid;
      enter();
    }
  };

  v4f ag[NT], au[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) ag[t] = au[t] = v4f{0.f, 0.f, 0.f, 0.f};
  enter();
#pragma unroll
  for (int d = 0; d < D; ++d) load(d);

  int ci = blockIdx.x, cj = 0;
  for (int c = 0; c < total; c += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (c + d >= total) break;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const v4f g = unit_product<FP8W>(wg[d], xs[d][t]);
        const v4f u = unit_product<FP8W>(wu[d], xs[d][t]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          ag[t][r] = FP8W ? __builtin_fmaf(sg[d], g[r], ag[t][r]) : ag[t][r] + g[r];
          au[t][r] = FP8W ? __builtin_fmaf(su[d], u[r], au[t][r]) : au[t][r] + u[r];
        }
      }
      load(d);
      if (++cj == n) {
        cj = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          red[wave][2 * t][lane] = ag[t];
          red[wave][2 * t + 1][lane] = au[t];
          ag[t] = au[t] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        __syncthreads();
        if (tid < 64 * NT) {
          const int t = wave;  // one wave per tile
          v4f g = red[0][2 * t][lane], u = red[0][2 * t + 1][lane];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) {
            g += red[w][2 * t][lane];
            u += red[w][2 * t + 1][lane];
          }
          const int s = ci / slabs, n0 = (ci - s * slabs) * 16, q0 = tb.seg[s];
          const int pr = column_pair(tb, q0, tb.sid[q0], t, l16);
          if (pr >= 0) {
            const float w = tb.w[pr];
            v4f hv;
#pragma unroll
            for (int r = 0; r < 4; ++r) hv[r] = w * (g[r] * act::sigmoid(g[r]) * u[r]);
            *reinterpret_cast<uint2*>(p.h + (int64_t)pr * p.inter + n0 + 4 * lq) = pack4(hv);
          }
        }
        __syncthreads();
        ci += grid;
      }
    }
  }
}

// ---- second kernel ---------------------------------------------------------
// A workgroup owns 16 R rows of every chosen expert's w2 (16 R output
// columns) and walks (segment, K block) units, the waves round robin.  A
// wave's sums of a segment go to its own LDS rows [token][16 R] when it
// leaves the segment, and the waves' rows meet at the end.
template <bool FP8W, int NT, int R, int D>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(const MoeParams p) {
  constexpr int WL = FP8W ? 2 : 4;
  constexpr int ES = FP8W ? 1 : 2;
  constexpr int YS = 16 * R + 4;  // floats per token in LDS
  __shared__ Tables tb;
  extern __shared__ __attribute__((aligned(16))) float yacc[];  // [waves][T][YS]
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  for (int i = tid; i < kWaves * p.t * YS / 4; i += kThreads) reinterpret_cast<v4f*>(yacc)[i] = v4f{0.f, 0.f, 0.f, 0.f};
  build_tables<NT, false>(p, tb);
  float* yw = yacc + wave * p.t * YS;

  const int nb = p.inter >> 7;
  const int nseg = (int)uniform(tb.nseg);
  const int h0 = blockIdx.x * 16 * R;
  const int units = nseg * nb;
  const int total = units > wave ? (units - wave + kWaves - 1) / kWaves : 0;
  const uint32_t row = (uint32_t)p.inter * ES;
  const uint32_t hrow = (uint32_t)p.inter * 2;
  const uint32_t woff = (uint32_t)l16 * row + 16u * lq;
  const uint32_t hbytes = (uint32_t)(p.t * p.top_k - 1) * hrow + 256u;

  v4i ws[D][R][WL], xs[D][NT][4];
  float sc[D];
  int seg_of[D], tok[D][NT];

  int ls = wave / nb, lb = wave - ls * nb;  // load cursor: segment and K block
  const uint8_t* wbase = nullptr;
  const float* sbase = nullptr;
  uint32_t hoff[NT];
  int ltok[NT];
  auto enter = [&]() {
    const bool live = ls < nseg;
    const int q0 = live ? tb.seg[ls] : 0;
    const int e = (int)uniform(live ? tb.sid[q0] : 0);
    wbase = p.w2 + ((int64_t)e * p.hid + h0) * row;
    if constexpr (FP8W) sbase = p.s2 + ((int64_t)e * (p.hid >> 7) + (h0 >> 7)) * nb;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int pr = live ? column_pair(tb, q0, e, t, l16) : -1;
      ltok[t] = pr >= 0 ? pr / p.top_k : -1;
      hoff[t] = pr >= 0 ? (uint32_t)pr * hrow + (FP8W ? 32u : 16u) * lq : kOut;
    }
  };
  auto load = [&](int d) {
    const bool live = ls < nseg;
    const auto rw = rsrc(wbase + (int64_t)lb * 128 * ES, live ? (16u * R - 1u) * row + 128u * ES : 0u);
    const auto rh = rsrc(p.h + (int64_t)lb * 128, live ? hbytes : 0u);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < WL; ++i) ws[d][r][i] = load16<kNt>(rw, woff + 16u * r * row + 64u * i);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xs[d][t][i] = load16<0>(rh, hoff[t] + (FP8W ? 128u * (i >> 1) + 16u * (i & 1) : 64u * i));
      tok[d][t] = ltok[t];
    }
    if constexpr (FP8W) {
      const auto rs = rsrc(sbase + lb, live ? 4u : 0u);
      sc[d] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, 0, 0, 0));
    }
    seg_of[d] = ls;
    lb += kWaves;
    if (lb >= nb) {
      while (lb >= nb) {
        lb -= nb;
        ++ls;
      }
      enter();
    }
  };

  v4f acc[R][NT];
  int cur = -1, ctok[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    ctok[t] = -1;
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  // (a column's lanes add to its own token's row: an empty column, whose
  // products may be NaN if a weight is, adds nothing)
  auto flush = [&]() {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (ctok[t] >= 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          v4f* a = reinterpret_cast<v4f*>(yw + ctok[t] * YS + 16 * r + 4 * lq);
          *a = *a + acc[r][t];
        }
      }
  };
  enter();
#pragma unroll
  for (int d = 0; d < D; ++d) load(d);
  for (int c = 0; c < total; c += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (c + d >= total) break;
      if (seg_of[d] != cur) {
        flush();
        cur = seg_of[d];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          ctok[t] = tok[d][t];
#pragma unroll
          for (int r = 0; r < R; ++r) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const v4f v = unit_product<FP8W>(ws[d][r], xs[d][t]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[r][t][e] = FP8W ? __builtin_fmaf(sc[d], v[e], acc[r][t][e]) : acc[r][t][e] + v[e];
        }
      load(d);
    }
  }
  flush();
  __syncthreads();
  for (int i = tid; i < p.t * 4 * R; i += kThreads) {
    const int t = i / (4 * R), c = 4 * (i - t * 4 * R);
    v4f s = *reinterpret_cast<const v4f*>(yacc + t * YS + c);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += *reinterpret_cast<const v4f*>(yacc + (w * p.t + t) * YS + c);
    const int64_t o = (int64_t)t * p.hid + h0 + c;
    if (p.residual) {
      const uint2 v = *reinterpret_cast<const uint2*>(p.residual + o);
      s += v4f{from_bf16((uint16_t)v.x), from_bf16((uint16_t)(v.x >> 16)), from_bf16((uint16_t)v.y),
               from_bf16((uint16_t)(v.y >> 16))};
    }
    *reinterpret_cast<uint2*>(p.y + o) = pack4(s);
  }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <bool FP8W, int NT>
hipError_t launch_moe(const MoeParams& p, hipStream_t stream) {
  constexpr int D = FP8W ? (NT == 1 ? 4 : 2) : 2;
  constexpr int R = 1;
  // at most min(E, pairs) experts are chosen; a segment more per full 16 NT pairs
  const long pairs = (long)p.t * p.top_k;
  const long segs = (pairs < p.experts ? pairs : p.experts) + pairs / (16 * NT);
  const long items = segs * (p.inter / 16);
  const int grid = (int)(items < 512 ? items : 512);
  if (p.logits)
    moe_up_kernel<FP8W, NT, true, D><<<grid, kThreads, 0, stream>>>(p);
  else
    moe_up_kernel<FP8W, NT, false, D><<<grid, kThreads, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = (size_t)kWaves * p.t * (16 * R + 4) * sizeof(float);
  moe_down_kernel<FP8W, NT, R, D><<<p.hid / (16 * R), kThreads, lds, stream>>>(p);
  return hipGetLastError();
}

dg_status moe(bool fp8, const void* x, const float* logits, int32_t* ids, float* weights, const void* w13,
              const float* s13, const void* w2, const float* s2, const void* residual, void* y, void* workspace,
              int tokens, int hidden, int intermediate, int num_experts, int top_k, int scoring, int renormalize,
              float scale, hipStream_t stream) {
  if (!x || !ids || !weights || !w13 || !w2 || !y || !workspace || (fp8 && (!s13 || !s2)))
    return DG_ERROR_INVALID_VALUE;
  if (tokens <= 0 || hidden <= 0 || intermediate <= 0 || num_experts <= 0 || top_k <= 0 || top_k > num_experts ||
      (scoring != DG_SCORING_SOFTMAX && scoring != DG_SCORING_SIGMOID))
    return DG_ERROR_INVALID_VALUE;
  if (tokens > kMaxTokens || top_k > kMaxTopK || num_experts > kMaxExperts || hidden % 128 != 0 ||
      intermediate % 128 != 0 || hidden > (1 << 20) || intermediate > (1 << 20))
    return DG_ERROR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(workspace, 16) || !aligned(y, 8) ||
      !aligned(residual, 8) || !aligned(logits, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(s13, 4) ||
      !aligned(s2, 4))
    return DG_ERROR_UNSUPPORTED;
  MoeParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.logits = logits;
  p.ids = ids;
  p.weights = weights;
  p.w13 = static_cast<const uint8_t*>(w13);
  p.s13 = s13;
  p.w2 = static_cast<const uint8_t*>(w2);
  p.s2 = s2;
  p.residual = static_cast<const uint16_t*>(residual);
  p.y = static_cast<uint16_t*>(y);
  p.h = static_cast<uint16_t*>(workspace);
  p.t = tokens;
  p.hid = hidden;
  p.inter = intermediate;
  p.experts = num_experts;
  p.top_k = top_k;
  p.scoring = scoring;
  p.renormalize = renormalize;
  p.scale = scale;
  (void)hipGetLastError();  // clear a stale error from unrelated work
  hipError_t e;
  if (tokens <= 16)
    e = fp8 ? launch_moe<true, 1>(p, stream) : launch_moe<false, 1>(p, stream);
  else
    e = fp8 ? launch_moe<true, 2>(p, stream) : launch_moe<false, 2>(p, stream);
  return e == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

}  // namespace
}  // namespace dg

extern "C" {

dg_status dg_moe_few_tokens_fp8(const void* x, const float* logits, int32_t* ids, float* weights, const void* w13,
                                const float* s13, const void* w2, const float* s2, const void* residual, void* y,
                                void* workspace, int tokens, int hidden, int intermediate, int num_experts, int top_k,
                                int scoring, int renormalize, float scale, hipStream_t stream) {
  return dg::moe(true, x, logits, ids, weights, w13, s13, w2, s2, residual, y, workspace, tokens, hidden,
                 intermediate, num_experts, top_k, scoring, renormalize, scale, stream);
}

dg_status dg_moe_few_tokens_bf16(const void* x, const float* logits, int32_t* ids, float* weights, const void* w13,
                                 const void* w2, const void* residual, void* y, void* workspace, int tokens,
                                 int hidden, int intermediate, int num_experts, int top_k, int scoring,
                                 int renormalize, float scale, hipStream_t stream) {
  return dg::moe(false, x, logits, ids, weights, w13, nullptr, w2, nullptr, residual, y, workspace, tokens, hidden,
                 intermediate, num_experts, top_k, scoring, renormalize, scale, stream);
}

}  // extern "C"
