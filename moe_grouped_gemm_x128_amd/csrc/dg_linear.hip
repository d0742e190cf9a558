// dg_linear.hip -- host side of the linear layer (include/dg.h): argument
// checks, the choice of kernel and tile, launches.  Validation runs before any
// HIP call.
#include "dg_linear_plan.h"

namespace dg {
namespace {

using namespace linear;

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
using namespace dg::linear;

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
