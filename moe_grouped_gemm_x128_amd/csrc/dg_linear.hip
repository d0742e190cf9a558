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
constexpr int64_t kMaxLd = 1 << 23;  // a tile's 256 operand rows within 32-bit byte offsets

// Checks c and the epilogue's arguments and fills `e`.
dg_status make_epilogue(void* c, int64_t ldc, int c_type, const dg_epilogue* in, int n, Epilogue* e) {
  *e = Epilogue{};
  if (c_type != DG_TYPE_BF16 && c_type != DG_TYPE_F32) return DG_ERROR_INVALID_VALUE;
  if (ldc < n) return DG_ERROR_INVALID_VALUE;
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
      if (!aligned(in->residual, 2)) return DG_ERROR_UNSUPPORTED;
      e->res = static_cast<const uint16_t*>(in->residual);
      e->ldr = in->ld_residual;
      vec = vec && aligned(e->res, 8) && e->ldr % 4 == 0;
      vec8 = vec8 && aligned(e->res, 16) && e->ldr % 8 == 0;
    }
    if (in->pre) {
      if (in->ld_pre < n) return DG_ERROR_INVALID_VALUE;
      if (!aligned(in->pre, 2)) return DG_ERROR_UNSUPPORTED;
      e->pre = static_cast<uint16_t*>(in->pre);
      e->ldp = in->ld_pre;
      vec = vec && aligned(e->pre, 8) && e->ldp % 4 == 0;
      vec8 = vec8 && aligned(e->pre, 16) && e->ldp % 8 == 0;
    }
  }
  e->vec = vec;
  // 32-bit byte offsets over a tile's 256 rows
  e->vec8 = vec8 && ldc <= kMaxLd / 4 && e->ldr <= kMaxLd / 4 && e->ldp <= kMaxLd / 4;
  return DG_SUCCESS;
}

// Tile and K splits of a tile GEMM: the least modelled time
//   passes over the CUs x (K blocks x time per block + fixed time per item)
//   + (split) the partials' write, their read and the second launch.
// Times per block from the rate a tile reaches on full CUs.
struct Plan {
  int tile, splits, kchunk;
};

Plan plan(int layout, int m, int n, int k, int cus, bool may_split) {
  // TFLOP/s of the whole card when every CU works on this tile
  static const double rate[kNumGemmTiles] = {1350., 1150., 1080., 850., 600.};
  const int blocks = ceil_div(k, 64);
  const char* force = std::getenv("DG_FORCE_TILE");
  const char* fsplit = std::getenv("DG_FORCE_SPLITS");
  Plan best{-1, 1, blocks};
  double best_us = 1e300;
  for (int t = 0; t < kNumGemmTiles; ++t) {
    const GemmTile g = kGemmTiles[t];
    if (force && *force) {
      int bm, bn, wm, wn;
      if (std::sscanf(force, "%dx%dx%dx%d", &bm, &bn, &wm, &wn) == 4 &&
          !(bm == g.bm && bn == g.bn && wm == g.wm && wn == g.wn))
        continue;
    }
    const double tiles = (double)ceil_div(m, g.bm) * ceil_div(n, g.bn);
    const int res = gemm_residents(t);
    const double block_us = 2.0 * g.bm * g.bn * 64 * cus * res / (rate[t] * 1e6);
    for (int s = 1; s <= 16; ++s) {
      if (fsplit && *fsplit && may_split && s != std::atoi(fsplit)) continue;
      if (s > 1 && (!may_split || blocks < s)) break;
      const int chunk = ceil_div(blocks, s);
      if (ceil_div(blocks, chunk) != s) continue;  // a split would be empty
      const double bytes = 4.0 * s * m * n;
      if (s > 1 && (bytes > 256e6 || (chunk < 4 && !(fsplit && *fsplit)))) break;
      const double passes = (double)ceil_div((int64_t)(tiles * s), (int64_t)cus * res);
      double us = passes * (chunk * block_us + 3.0 * res);
      if (s > 1) us += 4.0 + 2.0 * bytes / 4e6;
      if (us < best_us) {
        best_us = us;
        best = Plan{t, s, chunk};
      }
    }
  }
  return best;
}

// One tile GEMM with its epilogue (arguments checked).
dg_status gemm(int layout, GemmParams& p, int cus, hipStream_t stream) {
  const bool may_split = !is_capturing(stream);
  for (int attempt = 0; attempt < 2; ++attempt) {
    const Plan c = plan(layout, p.m, p.n, p.k, cus, may_split && attempt == 0);
    if (c.tile < 0) return DG_ERROR_UNSUPPORTED;
    const GemmTile g = kGemmTiles[c.tile];
    p.tiles_m = ceil_div(p.m, g.bm);
    p.tiles_n = ceil_div(p.n, g.bn);
    p.splits = c.splits;
    p.kchunk = c.kchunk;
    const int64_t items = (int64_t)p.tiles_m * p.tiles_n * c.splits;
    if (items > (1 << 30)) return DG_ERROR_UNSUPPORTED;
    // a multiple of 8 workgroups: the ids of a workgroup stay on its XCD's run
    const int64_t slots = (int64_t)(cus > 8 ? cus / 8 * 8 : 8) * gemm_residents(c.tile);
    const int grid = (int)(items < slots ? (items + 7) / 8 * 8 : slots);
    if (std::getenv("DG_LOG"))
      std::fprintf(stderr, "[dg] linear layout=%d m=%d n=%d k=%d -> tile %dx%d splits=%d grid=%d\n", layout, p.m, p.n,
                   p.k, g.bm, g.bn, c.splits, grid);
    if (c.splits == 1) return launch_gemm(layout, c.tile, p, grid, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
    p.ws_stride = (int64_t)p.m * p.n;
    bool owned = false;
    void* ws = split_workspace(stream, (size_t)(4 * c.splits * p.ws_stride), &owned);
    if (!ws) {
      (void)hipGetLastError();
      continue;  // no buffer to be had: the same product without a split
    }
    p.ws = static_cast<float*>(ws);
    const bool ok = launch_gemm(layout, c.tile, p, grid, stream) == hipSuccess &&
                    launch_splitk_linear(p.epi, p.ws, p.ws_stride, p.splits, p.m, p.n, stream) == hipSuccess;
    const bool freed = !owned || hipFreeAsync(ws, stream) == hipSuccess;
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
  if (m <= kMaxFewRows && !(force && *force)) {
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
  return gemm(kNT, p, cus, stream);
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
    if (dbias && launch_bias_sum(partial, dbias, ceil_div(m, d.rows), n, stream) != hipSuccess)
      return DG_ERROR_LAUNCH;
  }
  const uint8_t* g = in_place ? static_cast<const uint8_t*>(dc) : reinterpret_cast<const uint8_t*>(dpre);
  if (da) {
    GemmParams p{};
    p.a = g;
    p.lda = 2 * ldp;
    p.b = static_cast<const uint8_t*>(b);
    p.ldb = 2 * ldb;
    p.wb = k;
    p.m = m;
    p.n = k;
    p.k = n;
    const dg_status st = make_epilogue(da, ldda, DG_TYPE_BF16, nullptr, k, &p.epi);
    if (st != DG_SUCCESS) return st;
    const dg_status r = gemm(kNN, p, cus, stream);
    if (r != DG_SUCCESS) return r;
  }
  if (db) {
    GemmParams p{};
    p.a = g;
    p.lda = 2 * ldp;
    p.wa = (int)round8(n);
    p.b = static_cast<const uint8_t*>(a);
    p.ldb = 2 * lda;
    p.wb = k;
    p.m = n;
    p.n = k;
    p.k = m;
    const dg_status st = make_epilogue(db, lddb, DG_TYPE_BF16, nullptr, k, &p.epi);
    if (st != DG_SUCCESS) return st;
    return gemm(kTN, p, cus, stream);
  }
  return DG_SUCCESS;
}

}  // extern "C"
