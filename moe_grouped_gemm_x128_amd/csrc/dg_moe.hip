// dg_moe.hip -- a whole mixture-of-experts layer for a few tokens (decode) in
// two kernels:
//
//   moe_up_kernel    routing (top-k of the logits), and for every chosen
//                    (token, expert) pair  h = w silu(x.Wg^T) (x.Wu^T)
//   moe_down_kernel  y = residual + sum over the token's pairs of h.W2^T
//
// Bound: the chosen experts' weights, each read once (a few tokens give each
// weight a handful of operations).  So both kernels stream weights from HBM
// through a ring of LDS per wave, filled by loads of whole 128-byte lines several
// units (dg_stream.h) ahead, and everything else is arranged around that: the
// activations (bf16, a few KB) are re-read through the L2 by every workgroup,
// fp8 weights are widened to bf16 in registers (exact), and the products run on
// the bf16 MFMA with the tokens of one expert as its 16 columns -- the matrix unit
// has an order of magnitude to spare.
//
// The routing weight is folded into h, so the second kernel only sums; a
// workgroup of it owns 16 or 32 output columns for all experts and tokens, which
// makes the combination over experts a private sum: no atomics, a fixed order.
//
// h is rounded to bf16 once (the MFMA's operand type; up to 2^-8 of each value,
// the size of the output's own rounding: together 2.3e-3 to 2.6e-3 off in the norm
// without a residual, where the output's alone gives 1.67e-3); every sum is fp32.
//
// Measured, with the bytes that the counters saw: one token, 8 of 16 experts of
// 7168 x 2048 in fp8 (354 MB) 67.5 us, 5.2 TB/s; 13 tokens, 4 of 16 of 4096 x 1536 in
// bf16 (555 MB) 93 us, 6.0 TB/s; 64 tokens, 8 of 64 of 7168 x 2048 in fp8 (2.67 GB)
// 482 us, 5.5 TB/s.  Reads alone reach 7.0 TB/s, a device copy 5.2.
#include <climits>
#include <cstdint>

#include "../../include/dg.h"
#include "dg_act.h"
#include "dg_kernel.h"
#include "dg_stream.h"

namespace dg {
namespace {

using namespace stream;

constexpr int kMaxTokens = 64;
constexpr int kMaxTopK = 16;
constexpr int kMaxExperts = 512;
constexpr float kMasked = -745.f;  // below it e^l is 0 in 64 bits as well

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
// The (token, expert) pairs of the call, p = token * k + j, sorted by expert
// and token; a segment is the run of one expert's pairs: the columns of the MFMA
// tiles that share one pass over that expert's weights (at most one pair per
// token).
template <int TMAX>               // the most tokens of the call
struct Tables {
  uint64_t tokens[kMaxExperts];   // bit t: token t has the expert
  float w[TMAX * kMaxTopK];       // weight of each pair
  int16_t id[TMAX * kMaxTopK];    // its expert, -1: none
  uint16_t pair[TMAX * kMaxTopK]; // sorted position -> pair
  uint16_t base[kMaxExperts];     // expert -> its first sorted position
  uint16_t seg[kMaxExperts + 2];  // segment -> its first sorted position; the end after the last
  int16_t sid[kMaxExperts];       // segment -> expert
  int chunk_pairs[kMaxExperts / 64], chunk_segs[kMaxExperts / 64];
  int nseg, repeated;
};

// Order-preserving key of a logit: larger float, larger key; NaN above
// everything (it reaches the token's output, as it would through a sort);
// -inf, "never this expert", 0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 0xffffffffu;
  const uint32_t b = __float_as_uint(l + 0.f);  // -0 counts as 0
  if (b == 0xff800000u) return 0;
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k == 0xffffffffu ? 0x7fc00000u : (k >> 31) ? k ^ 0x80000000u : ~k);
}

// Maximum over each row of 16 lanes, in all of them (DPP rotations).
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#define DG_ROR_MAX(n) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xf, 0xf, false))
  DG_ROR_MAX(1);
  DG_ROR_MAX(2);
  DG_ROR_MAX(4);
  DG_ROR_MAX(8);
#undef DG_ROR_MAX
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#define DG_ROR_ADD(n) \
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + n, 0xf, 0xf, false))
  DG_ROR_ADD(8);
  DG_ROR_ADD(4);
  DG_ROR_ADD(2);
  DG_ROR_ADD(1);
#undef DG_ROR_ADD
  return v;
}

// Top-k of every token's logits, ties to the lowest expert: 16 lanes per
// token (four tokens per wave at a time), 16 NI >= E logits in registers.  A
// round is a maximum over the lanes and the lowest expert that holds it; lane j
// of the row keeps round j's choice.  Every workgroup does this for all tokens
// (two microseconds for 64) rather than waiting for a kernel that does it once.
template <int NI, int TMAX>
__device__ __forceinline__ void route_rows(const MoeParams& p, Tables<TMAX>& tb, bool publish) {
  const int l16 = threadIdx.x & 15;
  const int rows = (int)(blockDim.x >> 4);
  for (int t0 = 0; t0 < p.t; t0 += rows) {
    const int t = t0 + (int)(threadIdx.x >> 4);
    const bool in = t < p.t;  // (rows past the last token work on empty keys)
    uint32_t key[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = l16 + 16 * i;
      key[i] = in && e < p.experts ? logit_key(p.logits[(int64_t)t * p.experts + e]) : 0;
    }
    uint32_t top = 0, mine = 0;
    int my_id = -1;
    float all = 0.f;  // softmax over every expert (not renormalised)
    for (int j = 0; j < p.top_k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) best = max(best, key[i]);
      best = row_max(best);
      uint32_t low = 0;  // kMaxExperts - (lowest expert with the key): a maximum again
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (key[i] == best) low = max(low, (uint32_t)(kMaxExperts - (l16 + 16 * i)));
      const int e = kMaxExperts - (int)row_max(low);
      if (j == 0) {
        top = best;
        if (!p.renormalize && p.scoring == DG_SCORING_SOFTMAX) {
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (key[i] != 0) all += expf(key_logit(key[i]) - key_logit(top));
          all = row_sum(all);
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (e == l16 + 16 * i) key[i] = 0;
      if (l16 == j && best != 0) {
        my_id = e;
        mine = best;
      }
    }
    float w = 0.f;
    if (my_id >= 0) {
      const float l = key_logit(mine), most = key_logit(top);
      // Quotients of sigmoids that may all lie below fp32: from -20 down 1 + e^l is 1
      // in fp32, so they are quotients of exponentials.  (kMasked and below: a mask's
      // value, weight 0.)
      const bool small = p.renormalize && most < -20.f && most >= kMasked;
      w = small || p.scoring == DG_SCORING_SOFTMAX ? expf(l - most) : 1.f / (1.f + expf(-l));
    }
    const float sum = row_sum(w);
    if (p.renormalize)
      w = sum != 0.f ? w / sum : 0.f;  // sum is 0 where no expert is left or all are masked
    else if (p.scoring == DG_SCORING_SOFTMAX && my_id >= 0)
      w /= all;
    w *= p.scale;
    if (in && l16 < p.top_k) {
      const int q = t * p.top_k + l16;
      tb.id[q] = (int16_t)my_id;
      tb.w[q] = w;
      if (my_id >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&tb.tokens[my_id]), 1ull << t);
      if (publish) {
        p.ids[q] = my_id;
        p.weights[q] = w;
      }
    }
  }
}

// Fills the tables.  ROUTE: from the logits (published by workgroup 0), else
// from ids / weights: ids outside [0, E) drop out, a token's repeated expert
// keeps one pair with the sum of its weights.
template <bool ROUTE, int TMAX>
__device__ __forceinline__ void build_tables(const MoeParams& p, Tables<TMAX>& tb) {
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6), nthreads = blockDim.x;
  const int np = p.t * p.top_k;
  for (int e = tid; e < p.experts; e += nthreads) tb.tokens[e] = 0;
  if (tid == 0) tb.repeated = 0;
  __syncthreads();
  if constexpr (ROUTE) {
    const bool publish = blockIdx.x == 0;
    if (p.experts <= 64)
      route_rows<4>(p, tb, publish);
    else if (p.experts <= 128)
      route_rows<8>(p, tb, publish);
    else if (p.experts <= 256)
      route_rows<16>(p, tb, publish);
    else
      route_rows<32>(p, tb, publish);
  } else {
    for (int q = tid; q < np; q += nthreads) {
      const int id = p.ids[q];
      const bool ok = id >= 0 && id < p.experts;
      tb.id[q] = (int16_t)(ok ? id : -1);
      tb.w[q] = p.weights[q];
      if (ok) {
        const uint64_t bit = 1ull << (q / p.top_k);
        if (atomicOr(reinterpret_cast<unsigned long long*>(&tb.tokens[id]), bit) & bit) tb.repeated = 1;
      }
    }
  }
  __syncthreads();
  if constexpr (!ROUTE) {
    if (tb.repeated && tid < p.t) {
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
  }
  // per expert, its pairs and whether it is a segment, summed up to it: within
  // chunks of 64 experts by one wave each, then over the chunks
  const int nchunk = (p.experts + 63) >> 6, nwaves = nthreads >> 6;
  int below[kMaxExperts / 64], segs[kMaxExperts / 64];
#pragma unroll
  for (int r = 0; r < kMaxExperts / 64; ++r) {
    const int c = wave + r * nwaves;
    if (c >= nchunk) break;
    const int e = 64 * c + lane;
    const int n = e < p.experts ? __builtin_popcountll(tb.tokens[e]) : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o);
      if (lane >= o) sum += v;
    }
    const uint64_t used = __ballot(n > 0);
    below[r] = sum - n;
    segs[r] = __builtin_popcountll(used & ((1ull << lane) - 1));
    if (lane == 63) {
      tb.chunk_pairs[c] = sum;
      tb.chunk_segs[c] = __builtin_popcountll(used);
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kMaxExperts / 64; ++r) {
    const int c = wave + r * nwaves;
    if (c >= nchunk) break;
    int pairs = 0, nsegs = 0;
    for (int o = 0; o < c; ++o) {
      pairs += tb.chunk_pairs[o];
      nsegs += tb.chunk_segs[o];
    }
    const int e = 64 * c + lane;
    if (e < p.experts) {
      tb.base[e] = (uint16_t)(pairs + below[r]);
      if (tb.tokens[e]) {
        tb.seg[nsegs + segs[r]] = (uint16_t)(pairs + below[r]);
        tb.sid[nsegs + segs[r]] = (int16_t)e;
      }
    }
    if (c == nchunk - 1 && lane == 0) {
      tb.nseg = nsegs + tb.chunk_segs[c];
      tb.seg[tb.nseg] = (uint16_t)(pairs + tb.chunk_pairs[c]);
    }
  }
  __syncthreads();
  for (int q = tid; q < np; q += nthreads) {
    const int id = tb.id[q];
    if (id < 0) continue;
    const int t = q / p.top_k;
    tb.pair[tb.base[id] + __builtin_popcountll(tb.tokens[id] & ((1ull << t) - 1))] = (uint16_t)q;
  }
  __syncthreads();
}

// The pair in column c of the segment [q0, q1), -1 past its end.
template <int TMAX>
__device__ __forceinline__ int column_pair(const Tables<TMAX>& tb, int q0, int q1, int c) {
  return q0 + c < q1 ? (int)tb.pair[q0 + c] : -1;
}

// ---- first kernel ----------------------------------------------------------
// Work item: one segment x 16 hidden columns (16 gate and the 16 matching up
// rows of its expert's w13: the unit's groups A and B).  The waves of a
// workgroup take K blocks of 128 round robin and meet in LDS once per item.  A
// wave walks its items as one stream of units, so the loads of the next item
// are already out while an item's sums meet.
struct UpCursor {
  Unit u;
  const MoeParams* p;
  const Tables<kMaxTokens>* tb;
  int item, items, slabs, grid, kb, nb, waves, wave;
  int q0, q1;
  uint32_t rk;  // ceil(2^16 / k): pr / k = pr rk >> 16 for pr < 1024, k <= 16

  __device__ __forceinline__ uint32_t div_k(int pr) const { return ((uint32_t)pr * rk) >> 16; }

  __device__ __forceinline__ void seek() {  // the item and K block the cursor stands on
    u.live = item < items && wave < nb;
    if (!u.live) return;
    const int s = item / slabs, n0 = (item - s * slabs) * 16;
    q0 = (int)uniform(tb->seg[s]);
    q1 = (int)uniform(tb->seg[s + 1]);
    const int e = (int)uniform(tb->sid[s]);
    u.tiles = (q1 - q0 + 15) >> 4;
    u.wa = p->w13 + ((int64_t)e * 2 * p->inter + n0) * u.wrow;
    u.wb = u.wa + (int64_t)p->inter * u.wrow;
    if (p->s13) u.s = p->s13 + ((int64_t)e * 2 * (p->inter >> 7) + (n0 >> 7)) * nb;
    place(0);
  }
  __device__ __forceinline__ void place(int from) {  // from K block `from` of the item to kb
    const int d = kb - from;
    const int wb = p->s13 ? 128 : 256;
    u.wa += d * wb;
    u.wb += d * wb;
    u.s += d;
    u.x = reinterpret_cast<const uint8_t*>(p->x + kb * 128);
  }
  __device__ __forceinline__ void next() {
    const int from = kb;
    kb += waves;
    if (kb < nb) {
      place(from);
    } else {
      kb = wave;
      item += grid;
      seek();
    }
  }
  __device__ __forceinline__ uint32_t row(int t, int r) const {
    const int pr = column_pair(*tb, q0, q1, 16 * t + r);
    return pr >= 0 ? div_k(pr) * ((uint32_t)p->hid * 2u) : kOut;
  }
  __device__ __forceinline__ uint32_t scale(int) const { return kOut; }
};

template <int MODE, bool ROUTE, int W, int D>
__global__ __launch_bounds__(W * 64) void moe_up_kernel(const MoeParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ring_bytes(MODE, W, D)];
  __shared__ __attribute__((aligned(16))) Tables<kMaxTokens> tb;
  __shared__ __attribute__((aligned(16))) v4f red[W][2][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  build_tables<ROUTE, kMaxTokens>(p, tb);

  UpCursor c{};
  c.p = &p;
  c.tb = &tb;
  c.slabs = p.inter >> 4;
  c.items = (int)uniform(tb.nseg) * c.slabs;
  c.grid = gridDim.x;
  c.item = blockIdx.x;
  c.nb = p.hid >> 7;
  c.waves = W;
  c.wave = c.kb = wave;
  c.rk = (65536u + p.top_k - 1) / p.top_k;
  c.u.ra = c.u.rb = 16;
  c.u.wrow = (uint32_t)p.hid * (MODE == kBf16 ? 2 : 1);
  c.u.kbytes = MODE == kBf16 ? 256 : 128;
  c.u.xbytes = 256;
  c.u.xrange = (uint32_t)(p.t - 1) * (uint32_t)p.hid * 2u + 256u;
  c.u.s = p.s13;
  c.u.so[1] = (uint32_t)(p.inter >> 7) * c.nb * 4u;
  c.u.srange = c.u.so[1] + 4u;
  c.seek();
  const int mine = c.nb > wave ? (c.nb - wave + W - 1) / W : 0;  // units of an item on this wave
  Pipe<MODE, D, false, false, UpCursor> pipe;
  pipe.init(dma::lds_addr(ring) + wave * D * entry_bytes(MODE), c, lane);

  for (int item = blockIdx.x; item < c.items; item += c.grid) {
    const int s = item / c.slabs, n0 = (item - s * c.slabs) * 16;
    const int q0 = (int)uniform(tb.seg[s]), q1 = (int)uniform(tb.seg[s + 1]);
    const int tiles = (q1 - q0 + 15) >> 4;
    v4f g[kMaxTiles], u[kMaxTiles];
#pragma unroll
    for (int t = 0; t < kMaxTiles; ++t) g[t] = u[t] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < mine; ++k) pipe.template unit<kMaxTiles>(tiles, g, u);
#pragma unroll
    for (int t = 0; t < kMaxTiles; ++t) {
      if (t >= tiles) break;
      red[wave][0][lane] = g[t];
      red[wave][1][lane] = u[t];
      dma::barrier();
      if (wave == t % W) {
        v4f a = red[0][0][lane], b = red[0][1][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) {
          a += red[w][0][lane];
          b += red[w][1][lane];
        }
        const int pr = column_pair(tb, q0, q1, 16 * t + l16);
        if (pr >= 0) {
          const float w = tb.w[pr];
          v4f hv;
#pragma unroll
          for (int r = 0; r < 4; ++r) hv[r] = w * (a[r] * act::sigmoid(a[r]) * b[r]);
          *reinterpret_cast<uint2*>(p.h + (int64_t)pr * p.inter + n0 + 4 * lq) = pack4(hv);
        }
      }
      dma::barrier();
    }
  }
  dma::wait<0>();  // no load outlives the workgroup
}

// ---- second kernel ---------------------------------------------------------
// A workgroup owns 32 rows of every chosen expert's w2 (32 output columns; the
// unit's groups are 16 rows each), or 16 where 32 each would leave half of the
// CUs idle (the groups are two lines of K), and walks (segment, K block) units,
// the waves round robin.  A wave's sums of a segment go to its own LDS rows
// [token][columns] when it leaves the segment, and the waves' rows meet at the
// end.
template <int TMAX, bool SAME>
struct DownCursor {
  Unit u;
  const MoeParams* p;
  const Tables<TMAX>* tb;
  int seg, nseg, kb, nb, waves, h0;
  int q0, q1;

  __device__ __forceinline__ void seek() {
    u.live = seg < nseg;
    if (!u.live) return;
    q0 = (int)uniform(tb->seg[seg]);
    q1 = (int)uniform(tb->seg[seg + 1]);
    const int e = (int)uniform(tb->sid[seg]);
    const int wb = p->s2 && !SAME ? 128 : 256;      // bytes of K per unit
    const int xb = p->s2 && SAME ? 512 : 256;       // of the activations
    u.tiles = (q1 - q0 + 15) >> 4;
    u.wa = p->w2 + ((int64_t)e * p->hid + h0) * u.wrow + kb * wb;
    u.wb = u.wa + 16 * (int64_t)u.wrow;
    u.kbytes = (int)u.wrow - kb * wb;
    u.xbytes = 2 * p->inter - kb * xb;
    u.xrange = (uint32_t)(p->t * p->top_k - 1) * (uint32_t)p->inter * 2u + min(u.xbytes, xb);
    if (p->s2) {
      u.s = p->s2 + ((int64_t)e * (p->hid >> 7) + (h0 >> 7)) * (p->inter >> 7) + kb * (SAME ? 2 : 1);
      u.srange = SAME && u.kbytes > 128 ? 8 : 4;
    }
    u.x = reinterpret_cast<const uint8_t*>(p->h) + kb * xb;
  }
  __device__ __forceinline__ void next() {
    kb += waves;
    while (kb >= nb) {
      kb -= nb;
      ++seg;
    }
    seek();
  }
  __device__ __forceinline__ uint32_t row(int t, int r) const {
    const int pr = column_pair(*tb, q0, q1, 16 * t + r);
    return pr >= 0 ? (uint32_t)pr * ((uint32_t)p->inter * 2u) : kOut;
  }
  __device__ __forceinline__ uint32_t scale(int) const { return kOut; }
};

// TMAX: the most tokens of the call (LDS rows).
template <int MODE, int TMAX, bool SAME, int W, int D>
__global__ __launch_bounds__(W * 64) void moe_down_kernel(const MoeParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ring_bytes(MODE, W, D)];
  __shared__ __attribute__((aligned(16))) Tables<TMAX> tb;
  constexpr int R = SAME ? 16 : 32, kYStride = R + 4;  // columns; floats per token in LDS (padded against bank conflicts)
  __shared__ __attribute__((aligned(16))) float yacc[W][TMAX][kYStride];
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  for (int i = tid; i < W * TMAX * kYStride / 4; i += W * 64)
    reinterpret_cast<v4f*>(&yacc[0][0][0])[i] = v4f{0.f, 0.f, 0.f, 0.f};
  build_tables<false, TMAX>(p, tb);

  using Cursor = DownCursor<TMAX, SAME>;
  Cursor c{};
  c.p = &p;
  c.tb = &tb;
  c.nseg = (int)uniform(tb.nseg);
  c.nb = MODE == kW8A16 && SAME ? (p.inter + 255) >> 8 : p.inter >> 7;
  c.waves = W;
  c.h0 = blockIdx.x * R;
  c.seg = wave / c.nb;
  c.kb = wave - c.seg * c.nb;
  c.u.ra = c.u.rb = 16;
  c.u.wrow = (uint32_t)p.inter * (MODE == kBf16 ? 2 : 1);
  c.u.s = p.s2;
  c.u.so[1] = SAME ? 4 : 0;
  c.seek();
  Pipe<MODE, D, false, SAME, Cursor> pipe;
  pipe.init(dma::lds_addr(ring) + wave * D * entry_bytes(MODE), c, lane);

  v4f a[kMaxTiles], b[kMaxTiles];
  auto zero = [&]() {
#pragma unroll
    for (int t = 0; t < kMaxTiles; ++t) a[t] = b[t] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  // (a column's lanes add to its own token's row: an empty column, whose
  // products may be NaN if a weight is, adds nothing)
  auto flush = [&](int tiles) {
#pragma unroll
    for (int t = 0; t < kMaxTiles; ++t) {
      if (t >= tiles) break;
      const int pr = column_pair(tb, c.q0, c.q1, 16 * t + l16);
      if (pr >= 0) {
        v4f* y = reinterpret_cast<v4f*>(&yacc[wave][pr / p.top_k][4 * lq]);
        if constexpr (SAME) {
          y[0] += a[t] + b[t];
        } else {
          y[0] += a[t];
          y[4] += b[t];
        }
      }
    }
  };
  zero();
  while (c.u.live) {
    pipe.template unit<kMaxTiles>(c.u.tiles, a, b);
    if (c.kb + W >= c.nb) {  // the wave's last unit of the segment
      flush(c.u.tiles);
      zero();
    }
    c.next();
  }
  dma::wait<0>();  // no load outlives the workgroup
  __syncthreads();
  for (int i = tid; i < p.t * (R / 4); i += W * 64) {
    const int t = i / (R / 4), h = 4 * (i % (R / 4));
    v4f s = *reinterpret_cast<const v4f*>(&yacc[0][t][h]);
#pragma unroll
    for (int w = 1; w < W; ++w) s += *reinterpret_cast<const v4f*>(&yacc[w][t][h]);
    const int64_t o = (int64_t)t * p.hid + c.h0 + h;
    if (p.residual) {
      const uint2 v = *reinterpret_cast<const uint2*>(p.residual + o);
      s += v4f{from_bf16((uint16_t)v.x), from_bf16((uint16_t)(v.x >> 16)), from_bf16((uint16_t)v.y),
               from_bf16((uint16_t)(v.y >> 16))};
    }
    *reinterpret_cast<uint2*>(p.y + o) = pack4(s);
  }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int MODE>
hipError_t launch_moe(const MoeParams& p, int cus, hipStream_t stream) {
  // at most min(E, pairs) experts are chosen; one workgroup per CU (LDS)
  const long pairs = (long)p.t * p.top_k;
  const long items = (pairs < p.experts ? pairs : p.experts) * (p.inter / 16);
  const int grid = (int)(items < cus ? items : cus);
  // Waves and ring entries per wave that fit the LDS.  fp8 weights take more work
  // per byte (widening), so more waves beat deeper rings: one token on 8 experts of
  // 7168 x 2048 67.2 us with 12 waves of 2 entries, 69.9 with 8 of 4; bf16 weights
  // the other way round: 13 tokens on 4096 x 1536 94 against 97.
  constexpr int W = MODE == kW8A16 ? 12 : 8, D = MODE == kW8A16 ? 2 : 4;
  if (p.logits)
    moe_up_kernel<MODE, true, W, D><<<grid, W * 64, 0, stream>>>(p);
  else
    moe_up_kernel<MODE, false, W, D><<<grid, W * 64, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // 16 columns per workgroup where 32 would occupy at most half of the CUs
  const bool narrow = p.hid <= 16 * cus;
  if (p.t <= 16) {
    if (narrow)
      moe_down_kernel<MODE, 16, true, W, D><<<p.hid / 16, W * 64, 0, stream>>>(p);
    else
      moe_down_kernel<MODE, 16, false, W, D><<<p.hid / 32, W * 64, 0, stream>>>(p);
    return hipGetLastError();
  }
  // (the waves' sums of 64 tokens take half of the LDS: 64 tokens on 64 experts of
  // 7168 x 2048 490 us with 8 waves of 2 entries, 522 with 6 of 3, 565 with 4 of 6)
  if (narrow) {
    constexpr int WN = MODE == kW8A16 ? 10 : 8, DN = MODE == kW8A16 ? 2 : 3;
    moe_down_kernel<MODE, kMaxTokens, true, WN, DN><<<p.hid / 16, WN * 64, 0, stream>>>(p);
  } else {
    moe_down_kernel<MODE, kMaxTokens, false, 8, 2><<<p.hid / 32, 8 * 64, 0, stream>>>(p);
  }
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
  const int cus = compute_units();
  if (cus <= 0) return DG_ERROR_LAUNCH;
  const hipError_t e = fp8 ? launch_moe<kW8A16>(p, cus, stream) : launch_moe<kBf16>(p, cus, stream);
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
