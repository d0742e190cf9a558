// dg_linear_plan.h -- what the host code of the linear layers (dg_linear.hip:
// BF16 and FP8; dg_linear_int8.hip) shares: the epilogue's checks, and the
// choice of kernel, tile and K splits.
#pragma once

#include <cstdio>
#include <cstdlib>

#include "dg_linear.h"

namespace dg {
namespace linear {

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int64_t round8(int64_t n) { return (n + 7) & ~(int64_t)7; }
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

constexpr int kMaxK = 1 << 22;
constexpr int64_t kMaxLd = 1 << 22;  // a tile's 256 operand rows within 32-bit byte offsets
constexpr int64_t kMaxOutLd = 1 << 20;  // and 256 rows of up to 4 bytes an element within 31 bits

// Checks c and the epilogue's arguments and fills `e`.
inline dg_status make_epilogue(void* c, int64_t ldc, int c_type, const dg_epilogue* in, int n, Epilogue* e) {
  *e = Epilogue{};
  if (c_type != DG_TYPE_BF16 && c_type != DG_TYPE_F32) return DG_ERROR_INVALID_VALUE;
  if (ldc < n) return DG_ERROR_INVALID_VALUE;
  if (ldc > kMaxOutLd) return DG_ERROR_UNSUPPORTED;
  const int es = c_type == DG_TYPE_F32 ? 4 : 2;
  if (!aligned(c, es)) return DG_ERROR_UNSUPPORTED;
  e->out = c;
  e->ldc = ldc;
  e->out_f32 = c_type == DG_TYPE_F32;
  bool vec = aligned(c, 4 * es) && ldc % 4 == 0;
  bool vec8 = aligned(c, 16) && ldc % 8 == 0 && n % 8 == 0;
  if (in) {
    if (in->activation < DG_ACT_NONE || in->activation > DG_ACT_SILU) return DG_ERROR_INVALID_VALUE;
    e->act = in->activation;
    if (in->bias) {
      if (in->bias_type != DG_TYPE_BF16 && in->bias_type != DG_TYPE_F32) return DG_ERROR_INVALID_VALUE;
      if (!aligned(in->bias, in->bias_type == DG_TYPE_F32 ? 4 : 2)) return DG_ERROR_UNSUPPORTED;
      e->bias = in->bias;
      e->bias_f32 = in->bias_type == DG_TYPE_F32;
    }
    if (in->residual) {
      if (in->ld_residual < n) return DG_ERROR_INVALID_VALUE;
      if (!aligned(in->residual, 2) || in->ld_residual > kMaxOutLd) return DG_ERROR_UNSUPPORTED;
      e->res = static_cast<const uint16_t*>(in->residual);
      e->ldr = in->ld_residual;
      vec = vec && aligned(e->res, 8) && e->ldr % 4 == 0;
      vec8 = vec8 && aligned(e->res, 16) && e->ldr % 8 == 0;
    }
    if (in->pre) {
      if (in->ld_pre < n) return DG_ERROR_INVALID_VALUE;
      if (!aligned(in->pre, 2) || in->ld_pre > kMaxOutLd) return DG_ERROR_UNSUPPORTED;
      e->pre = static_cast<uint16_t*>(in->pre);
      e->ldp = in->ld_pre;
      vec = vec && aligned(e->pre, 8) && e->ldp % 4 == 0;
      vec8 = vec8 && aligned(e->pre, 16) && e->ldp % 8 == 0;
    }
  }
  e->vec = vec;
  e->vec8 = vec8;
  return DG_SUCCESS;
}

// The model behind the choice of tile and K splits, in microseconds:
//   passes over the workgroups x (K blocks x time per block + a fixed time and
//   one by the tile's area per item) + (split) the partials' write and read and
//   the second launch.
// Rates (TFLOP/s of the whole card on full CUs), the share of a block's time
// that a workgroup alone on a CU needs where two would share it, and the other
// constants are fitted to timings of every tile and split at 140 sizes drawn
// from 65..5000 x 64..9000, K 256..8192: the choice is 1% behind the best in
// the mean.  A workgroup alone on a CU is bound by the chain of a block (wait,
// barrier, loads issued, fragments read, MFMAs), not by bandwidth: hence the
// tiles of two groups, which halve the number of such steps (333 x 2111 x 1536:
// 11.6 us on 64x64 with two groups, 14.6 with one; 1024 x 4096 x 4096: 54.6 us
// on 128x128 against 66.6), while one group is better where two workgroups
// share a CU (517 x 1161 x 1096 backward: 18.4 us against 22.4).
constexpr double kTileRate[kNumGemmTiles] = {1280., 660., 1210., 720., 620., 880., 690., 540.};
// the same of the two products of the backward pass in one launch (42 sizes:
// 0.3% behind the best)
constexpr double kPairRate[kNumPairTiles] = {1390., 1060., 1190., 820., 600.};
constexpr double kTwoUs = 6.0;
constexpr double kAlone = 0.91, kItemUs = 2.4, kAreaUs = 2.2 / 65536;
constexpr double kSplitUs = 2.1, kPartialUs = 0.4, kPartialBytesPerUs = 5.9e6;

// time per K block and per item
struct TileTime {
  double block, item;
};
inline TileTime tile_time(int tile, double rate, int cus, bool alone) {
  const GemmTile g = kGemmTiles[tile];
  const int res = gemm_residents(tile);
  const double us = 2.0 * g.bm * g.bn * 64 * cus * res / (rate * 1e6);
  const double item = kItemUs + kAreaUs * g.bm * g.bn;
  return alone && res > 1 ? TileTime{us * kAlone, item} : TileTime{us, item * res};
}

inline bool forced_out(const GemmTile& g) {  // DG_FORCE_TILE names another tile
  const char* force = std::getenv("DG_FORCE_TILE");
  int bm, bn, wm, wn, wk;
  const int got = force && *force ? std::sscanf(force, "%dx%dx%dx%dx%d", &bm, &bn, &wm, &wn, &wk) : 0;
  return got >= 4 && !(bm == g.bm && bn == g.bn && wm == g.wm && wn == g.wn && (got == 4 || wk == g.wk));
}

inline int forced_splits() {  // DG_FORCE_SPLITS, 0: not set
  const char* e = std::getenv("DG_FORCE_SPLITS");
  return e && *e ? std::atoi(e) : 0;
}

struct Plan {
  int tile, splits, kchunk;
  double us;
};

inline Plan plan(int m, int n, int k, int cus, bool may_split) {
  const int blocks = ceil_div(k, 64);
  const int force = may_split ? forced_splits() : 0;
  Plan best{-1, 1, blocks, 1e300};
  for (int t = 0; t < kNumGemmTiles; ++t) {
    const GemmTile g = kGemmTiles[t];
    if (forced_out(g)) continue;
    const int64_t tiles = (int64_t)ceil_div(m, g.bm) * ceil_div(n, g.bn);
    const int64_t slots = (int64_t)cus * gemm_residents(t);
    for (int s = 1; s <= 16; ++s) {
      if (force && s != force) continue;
      if (s > 1 && (!may_split || blocks < s)) break;
      const int chunk = ceil_div(blocks, s);
      if (ceil_div(blocks, chunk) != s) continue;  // a split would be empty
      const double bytes = 4.0 * s * m * n;
      if (s > 1 && (bytes > 256e6 || (chunk < 4 && !force))) break;
      const double passes = (double)((tiles * s + slots - 1) / slots);
      const TileTime w = tile_time(t, kTileRate[t], cus, tiles * s <= cus);
      double us = passes * (chunk * w.block + w.item);
      if (s > 1) us += kSplitUs + kPartialUs * s + 2.0 * bytes / kPartialBytesPerUs;
      if (us < best.us) best = Plan{t, s, chunk, us};
    }
  }
  return best;
}

// Whether M <= 64 rows of BF16 go to the kernel that streams B.  Each of its
// workgroups reads all of A beside its 16 or 32 rows of B, at some 65 KB per
// microsecond: up to 16 rows B is most of it, with more rows and a long K the
// tiles with K split are faster (64 x 4096 x 7168: 18.1 us against 23.0, 48 x 2112 x
// 7168 15.0 against 19.5), with a short K slower (64 x 8192 x 1024: 9.5 against
// 8.6).  (kBesideUs: launches, which the tiles' model leaves out.)  FP8 halves
// A too: there it is the faster one for all M <= 64 (64 x 4096 x 7168 15.5 us
// against 16.0, 17 x 4096 x 7168 10.2 against 12.8).
constexpr double kRowsUs = 4.3, kRowsBytesPerUs = 65e3, kBesideUs = 2.5;

inline bool few_rows(int m, int n, int k, int cus, bool may_split) {
  if (m > kMaxFewRows) return false;
  if (m <= 16) return true;
  const double us = kRowsUs + 2.0 * k * (m + few_rows_columns(n, cus)) / kRowsBytesPerUs;
  return us <= plan(m, n, k, cus, may_split).us + kBesideUs;
}

inline void set_tiles(GemmParams& p, const GemmTile& g, int splits, int kchunk) {
  p.tiles_m = ceil_div(p.m, g.bm);
  p.tiles_n = ceil_div(p.n, g.bn);
  p.splits = splits;
  p.kchunk = kchunk;
}

}  // namespace linear
}  // namespace dg
