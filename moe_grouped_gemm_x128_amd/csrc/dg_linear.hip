// dg_linear.hip -- host side of the linear layer (include/dg.h): argument
// checks, the choice of kernel and tile, launches.  Validation runs before any
// HIP call.
#include "dg_linear.h"

#include <cstdio>
#include <cstdlib>

namespace dg {
namespace {

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t round8(int64_t n) { return (n + 7) & ~(int64_t)7; }
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

constexpr int kMaxK = 1 << 22;
constexpr int64_t kMaxLd = 1 << 22;  // a tile's 256 operand rows within 32-bit byte offsets
constexpr int64_t kMaxOutLd = 1 << 20;  // and 256 rows of up to 4 bytes an element within 31 bits

// Checks c and the epilogue's arguments and fills `e`.
dg_status make_epilogue(void* c, int64_t ldc, int c_type, const dg_epilogue* in, int n, Epilogue* e) {
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
TileTime tile_time(int tile, double rate, int cus, bool alone) {
  const GemmTile g = kGemmTiles[tile];
  const int res = gemm_residents(tile);
  const double us = 2.0 * g.bm * g.bn * 64 * cus * res / (rate * 1e6);
  const double item = kItemUs + kAreaUs * g.bm * g.bn;
  return alone && res > 1 ? TileTime{us * kAlone, item} : TileTime{us, item * res};
}

bool forced_out(const GemmTile& g) {  // DG_FORCE_TILE names another tile
  const char* force = std::getenv("DG_FORCE_TILE");
  int bm, bn, wm, wn, wk;
  const int got = force && *force ? std::sscanf(force, "%dx%dx%dx%dx%d", &bm, &bn, &wm, &wn, &wk) : 0;
  return got >= 4 && !(bm == g.bm && bn == g.bn && wm == g.wm && wn == g.wn && (got == 4 || wk == g.wk));
}

int forced_splits() {  // DG_FORCE_SPLITS, 0: not set
  const char* e = std::getenv("DG_FORCE_SPLITS");
  return e && *e ? std::atoi(e) : 0;
}

struct Plan {
  int tile, splits, kchunk;
  double us;
};

Plan plan(int m, int n, int k, int cus, bool may_split) {
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

bool few_rows(int m, int n, int k, int cus, bool may_split) {
  if (m > kMaxFewRows) return false;
  if (m <= 16) return true;
  const double us = kRowsUs + 2.0 * k * (m + few_rows_columns(n, cus)) / kRowsBytesPerUs;
  return us <= plan(m, n, k, cus, may_split).us + kBesideUs;
}

// da and db in one launch: the tile, and how many of its workgroups da gets.
struct PairPlan {
  int tile, first, grid;
  double us;
};

PairPlan plan_pair(const GemmParams& nn, const GemmParams& tn, int cus) {
  PairPlan best{-1, 0, 0, 1e300};
  for (int t = 0; t < kNumPairTiles; ++t) {
    const GemmTile g = kGemmTiles[t];
    if (forced_out(g)) continue;
    const int64_t ta = (int64_t)ceil_div(nn.m, g.bm) * ceil_div(nn.n, g.bn);
    const int64_t tb = (int64_t)ceil_div(tn.m, g.bm) * ceil_div(tn.n, g.bn);
    if (ta > (1 << 24) || tb > (1 << 24)) continue;
    const int64_t slots = (int64_t)(cus > 16 ? cus / 8 * 8 : 16) * gemm_residents(t);
    const int ka = ceil_div(nn.k, 64), kb = ceil_div(tn.k, 64);
    const TileTime w = tile_time(t, kPairRate[t], cus, ta + tb <= cus);
    for (int passes = 1; passes <= 16; ++passes) {  // of da's workgroups
      const int64_t first = (ceil_div(ta, passes) + 7) / 8 * 8;
      if (first >= slots) continue;
      int64_t rest = slots - first;
      if (rest > tb) rest = (tb + 7) / 8 * 8;
      const double a = (double)((ta + first - 1) / first) * (ka * w.block + w.item);
      const double b = (double)((tb + rest - 1) / rest) * (kb * w.block + w.item);
      const double us = a > b ? a : b;
      if (us < best.us) best = PairPlan{t, (int)first, (int)(first + rest), us};
    }
  }
  return best;
}

void set_tiles(GemmParams& p, const GemmTile& g, int splits, int kchunk) {
  p.tiles_m = ceil_div(p.m, g.bm);
  p.tiles_n = ceil_div(p.n, g.bn);
  p.splits = splits;
  p.kchunk = kchunk;
}

// One tile GEMM with its epilogue (arguments checked).
dg_status gemm(int layout, GemmParams& p, int cus, bool may_split, hipStream_t stream) {
  for (int attempt = 0; attempt < 2; ++attempt) {
    const Plan c = plan(p.m, p.n, p.k, cus, may_split && attempt == 0);
    if (c.tile < 0) return DG_ERROR_UNSUPPORTED;
    const GemmTile g = kGemmTiles[c.tile];
    set_tiles(p, g, c.splits, c.kchunk);
    const int64_t items = (int64_t)p.tiles_m * p.tiles_n * c.splits;
    if (items > (1 << 30)) return DG_ERROR_UNSUPPORTED;
    // a multiple of 8 workgroups: the ids of a workgroup stay on its XCD's run
    const int64_t slots = (int64_t)(cus > 8 ? cus / 8 * 8 : 8) * gemm_residents(c.tile);
    const int grid = (int)(items < slots ? (items + 7) / 8 * 8 : slots);
    if (std::getenv("DG_LOG"))
      std::fprintf(stderr, "[dg] linear layout=%d m=%d n=%d k=%d -> tile %dx%d wk=%d splits=%d grid=%d\n", layout, p.m, p.n,
                   p.k, g.bm, g.bn, g.wk, c.splits, grid);
    if (c.splits == 1) return launch_gemm(layout, c.tile, p, grid, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
    p.ws_stride = (int64_t)p.m * p.n;
    SplitBuffer ws = split_buffer(stream, (size_t)(4 * c.splits * p.ws_stride));
    if (!ws.ptr) {
      (void)hipGetLastError();
      continue;  // no buffer to be had: the same product without a split
    }
    p.ws = static_cast<float*>(ws.ptr);
    const bool ok = launch_gemm(layout, c.tile, p, grid, stream) == hipSuccess &&
                    launch_splitk_linear(p.epi, p.ws, p.ws_stride, p.splits, p.m, p.n, stream) == hipSuccess;
    const bool freed = return_split_buffer(ws, stream);
    return ok && freed ? DG_SUCCESS : DG_ERROR_LAUNCH;
  }
  return DG_ERROR_LAUNCH;
}

bool bad_operand(const void* p, int64_t ld, int cols) { return ld < cols || !p; }
bool unfit_operand(const void* p, int64_t ld) { return !aligned(p, 16) || ld % 8 != 0 || ld > kMaxLd; }

// Rows of dc that one workgroup of the activation's backward pass takes: 64
// (the bias partials are then 1/32 of the traffic) where that gives the card
// work, else 16 (517 x 1161: 24 us with 45 workgroups of 64 rows).
int dact_rows(int m, int n) { return (int64_t)ceil_div(m, 64) * ceil_div(n, 256) >= 512 ? 64 : 16; }

// workspace of the backward pass: dpre bf16 [m, ldp], then the bias partials
int64_t dpre_bytes(int m, int n) { return (2 * (int64_t)m * round8(n) + 15) & ~(int64_t)15; }

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_gemm_bf16_nt_epilogue(const void* a, int64_t lda, const void* b, int64_t ldb, void* c, int64_t ldc,
                                   int c_type, const dg_epilogue* epi, int m, int n, int k, hipStream_t stream) {
  if (!a || !b || !c || m <= 0 || n <= 0 || k <= 0) return DG_ERROR_INVALID_VALUE;
  if (bad_operand(a, lda, k) || bad_operand(b, ldb, k)) return DG_ERROR_INVALID_VALUE;
  Epilogue e;
  const dg_status st = make_epilogue(c, ldc, c_type, epi, n, &e);
  if (st != DG_SUCCESS) return st;
  if (k % 8 != 0 || k > kMaxK || unfit_operand(a, lda) || unfit_operand(b, ldb)) return DG_ERROR_UNSUPPORTED;
  const int cus = compute_units();
  if (cus <= 0) return DG_ERROR_LAUNCH;
  (void)hipGetLastError();  // clear a stale error from unrelated work
  const char* force = std::getenv("DG_FORCE_TILE");
  const bool may_split = !is_capturing(stream);
  if (!(force && *force) && few_rows(m, n, k, cus, may_split)) {
    RowsParams p{};
    p.a = static_cast<const uint8_t*>(a);
    p.b = static_cast<const uint8_t*>(b);
    p.lda = 2 * lda;
    p.ldb = 2 * ldb;
    p.m = m;
    p.n = n;
    p.k = k;
    p.epi = e;
    return launch_linear_rows(false, p, cus, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
  }
  GemmParams p{};
  p.a = static_cast<const uint8_t*>(a);
  p.b = static_cast<const uint8_t*>(b);
  p.lda = 2 * lda;
  p.ldb = 2 * ldb;
  p.m = m;
  p.n = n;
  p.k = k;
  p.epi = e;
  return gemm(kNT, p, cus, may_split, stream);
}

dg_status dg_gemm_fp8_nt_epilogue(const void* a, const float* sa, const void* b, const float* sb, void* c, int64_t ldc,
                                  int c_type, const dg_epilogue* epi, int m, int n, int k, hipStream_t stream) {
  if (!a || !sa || !b || !sb || !c || m <= 0 || n <= 0 || k <= 0) return DG_ERROR_INVALID_VALUE;
  Epilogue e;
  const dg_status st = make_epilogue(c, ldc, c_type, epi, n, &e);
  if (st != DG_SUCCESS) return st;
  if (k % 128 != 0 || k > kMaxK || !aligned(a, 16) || !aligned(b, 16) || !aligned(sa, 4) || !aligned(sb, 4))
    return DG_ERROR_UNSUPPORTED;
  const char* force = std::getenv("DG_FORCE_TILE");
  if (m <= kMaxFewRows && !(force && *force)) {
    const int cus = compute_units();
    if (cus <= 0) return DG_ERROR_LAUNCH;
    (void)hipGetLastError();
    RowsParams p{};
    p.a = static_cast<const uint8_t*>(a);
    p.b = static_cast<const uint8_t*>(b);
    p.sa = sa;
    p.sb = sb;
    p.lda = p.ldb = k;
    p.m = m;
    p.n = n;
    p.k = k;
    p.epi = e;
    return launch_linear_rows(true, p, cus, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
  }
  return linear_fp8(a, sa, b, sb, e, m, n, k, stream);
}

dg_status dg_gemm_bf16_nt_epilogue_backward_workspace(int m, int n, int64_t* bytes) {
  if (!bytes || m <= 0 || n <= 0) return DG_ERROR_INVALID_VALUE;
  *bytes = dpre_bytes(m, n) + 4 * (int64_t)ceil_div(m, dact_rows(m, n)) * n;
  return DG_SUCCESS;
}

dg_status dg_gemm_bf16_nt_epilogue_backward(const void* dc, int64_t lddc, const void* a, int64_t lda, const void* b,
                                            int64_t ldb, const void* pre, int64_t ld_pre, int activation, void* da,
                                            int64_t ldda, void* db, int64_t lddb, float* dbias, void* workspace, int m,
                                            int n, int k, hipStream_t stream) {
  if (!dc || m <= 0 || n <= 0 || k <= 0 || lddc < n) return DG_ERROR_INVALID_VALUE;
  if (activation < DG_ACT_NONE || activation > DG_ACT_SILU) return DG_ERROR_INVALID_VALUE;
  const bool act = activation != DG_ACT_NONE;
  if (act && (!pre || ld_pre < n)) return DG_ERROR_INVALID_VALUE;
  if ((da && (bad_operand(b, ldb, k) || ldda < k)) || (db && (bad_operand(a, lda, k) || lddb < k)) || !workspace)
    return DG_ERROR_INVALID_VALUE;
  if (k % 8 != 0 || k > kMaxK || n > kMaxK || m > kMaxK || !aligned(dc, 2) || (act && !aligned(pre, 2)) ||
      !aligned(workspace, 16) || (da && (unfit_operand(b, ldb) || !aligned(da, 2))) ||
      (db && (unfit_operand(a, lda) || !aligned(db, 2))) || !aligned(dbias, 4))
    return DG_ERROR_UNSUPPORTED;
  GemmParams nn{}, tn{};  // da, db
  if (da) {
    const dg_status st = make_epilogue(da, ldda, DG_TYPE_BF16, nullptr, k, &nn.epi);
    if (st != DG_SUCCESS) return st;
  }
  if (db) {
    const dg_status st = make_epilogue(db, lddb, DG_TYPE_BF16, nullptr, k, &tn.epi);
    if (st != DG_SUCCESS) return st;
  }
  const int cus = compute_units();
  if (cus <= 0) return DG_ERROR_LAUNCH;
  (void)hipGetLastError();
  // without an activation dpre is dc: it is read in place where its rows fit
  // the products' loads (16-byte rows, whole chunks of 8)
  const bool in_place = !act && n % 8 == 0 && lddc % 8 == 0 && aligned(dc, 16) && lddc <= kMaxLd;
  const int64_t ldp = in_place ? lddc : round8(n);
  uint16_t* dpre = in_place ? nullptr : static_cast<uint16_t*>(workspace);
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dpre_bytes(m, n));
  if ((dpre && (da || db)) || dbias) {
    DactParams d{};
    d.dc = static_cast<const uint16_t*>(dc);
    d.pre = act ? static_cast<const uint16_t*>(pre) : nullptr;
    d.dpre = da || db ? dpre : nullptr;
    d.partial = dbias ? partial : nullptr;
    d.lddc = lddc;
    d.ldpre = ld_pre;
    d.ldp = round8(n);
    d.m = m;
    d.n = n;
    d.rows = dact_rows(m, n);
    d.act = activation;
    d.vec = aligned(dc, 16) && lddc % 8 == 0 && (!act || (aligned(pre, 16) && ld_pre % 8 == 0));
    if (launch_dact(d, stream) != hipSuccess) return DG_ERROR_LAUNCH;
  }
  const int chunks = ceil_div(m, dact_rows(m, n));  // of the bias partials
  const uint8_t* g = in_place ? static_cast<const uint8_t*>(dc) : reinterpret_cast<const uint8_t*>(dpre);
  if (da) {
    nn.a = g;
    nn.lda = 2 * ldp;
    nn.b = static_cast<const uint8_t*>(b);
    nn.ldb = 2 * ldb;
    nn.wb = k;
    nn.m = m;
    nn.n = k;
    nn.k = n;
  }
  if (db) {
    tn.a = g;
    tn.lda = 2 * ldp;
    tn.wa = (int)round8(n);
    tn.b = static_cast<const uint8_t*>(a);
    tn.ldb = 2 * lda;
    tn.wb = k;
    tn.m = n;
    tn.n = k;
    tn.k = m;
  }
  const bool may_split = !is_capturing(stream);
  // (the pair's products are not split)
  if (da && db && nn.epi.vec8 && tn.epi.vec8 && !(may_split && forced_splits() > 1)) {
    const PairPlan c = plan_pair(nn, tn, cus);
    const Plan ca = plan(nn.m, nn.n, nn.k, cus, may_split), cb = plan(tn.m, tn.n, tn.k, cus, may_split);
    // Two launches where splitting K gains more than sharing the card does:
    // 45 x 6920 x 2520 37 us against 47.  (kTwoUs: what the second launch and the
    // transposed operands cost beyond the model; 517 x 1161 x 1096 is 18 us in
    // one launch and 27 in two, where the model sees 17 and 17.)
    if (c.tile >= 0 && c.us <= ca.us + cb.us + kTwoUs) {
      const GemmTile tile = kGemmTiles[c.tile];
      set_tiles(nn, tile, 1, ceil_div(nn.k, 64));
      set_tiles(tn, tile, 1, ceil_div(tn.k, 64));
      if (std::getenv("DG_LOG"))
        std::fprintf(stderr, "[dg] linear backward m=%d n=%d k=%d -> tile %dx%d first=%d grid=%d\n", m, n, k, tile.bm,
                     tile.bn, c.first, c.grid);
      return launch_gemm_pair(c.tile, nn, tn, c.first, c.grid, partial, dbias, chunks, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
    }
  }
  if (dbias && launch_bias_sum(partial, dbias, chunks, n, stream) != hipSuccess) return DG_ERROR_LAUNCH;
  if (da) {
    const dg_status r = gemm(kNN, nn, cus, may_split, stream);
    if (r != DG_SUCCESS) return r;
  }
  if (db) return gemm(kTN, tn, cus, may_split, stream);
  return DG_SUCCESS;
}

}  // extern "C"
