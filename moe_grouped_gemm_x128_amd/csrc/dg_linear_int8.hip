// dg_linear_int8.hip -- host side of the INT8 linear layer and its quantiser
// (include/dg.h): argument checks, the choice of kernel and tile, launches.
// Validation runs before any HIP call.
//
// The kernels move INT8 operands as the BF16 ones of half the K (the same bytes
// per block, two matrix instructions' worth of values in the time of one), so
// the choice of tile and K splits is the BF16 layer's at K / 2.
#include "dg_linear_plan.h"

using namespace dg;
using namespace dg::linear;

extern "C" {

dg_status dg_gemm_int8_nt_epilogue(const void* a, int64_t lda, const float* sa, const void* b, int64_t ldb,
                                   const float* sb, void* c, int64_t ldc, int c_type, const dg_epilogue* epi, int m,
                                   int n, int k, hipStream_t stream) {
  if (!a || !sa || !b || !sb || !c || m <= 0 || n <= 0 || k <= 0 || lda < k || ldb < k) return DG_ERROR_INVALID_VALUE;
  Epilogue e;
  const dg_status st = make_epilogue(c, ldc, c_type, epi, n, &e);
  if (st != DG_SUCCESS) return st;
  // 2^14 K < 2^31: the largest sum, of K products -128 * -128, fits int32
  if (k % 16 != 0 || k >= 1 << 17 || !aligned(a, 16) || !aligned(b, 16) || lda % 16 != 0 || ldb % 16 != 0 ||
      lda > kMaxLd || ldb > kMaxLd || !aligned(sa, 4) || !aligned(sb, 4))
    return DG_ERROR_UNSUPPORTED;
  const int cus = compute_units();
  if (cus <= 0) return DG_ERROR_LAUNCH;
  (void)hipGetLastError();  // clear a stale error from unrelated work
  const char* force = std::getenv("DG_FORCE_TILE");
  const bool may_split = !is_capturing(stream);
  if (!(force && *force) && few_rows(m, n, k / 2, cus, may_split)) {
    RowsParams p{};
    p.a = static_cast<const uint8_t*>(a);
    p.b = static_cast<const uint8_t*>(b);
    p.sa = sa;
    p.sb = sb;
    p.lda = lda;
    p.ldb = ldb;
    p.m = m;
    p.n = n;
    p.k = k / 2;
    p.epi = e;
    return launch_linear_rows_int8(p, cus, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
  }
  GemmParams p{};
  p.a = static_cast<const uint8_t*>(a);
  p.b = static_cast<const uint8_t*>(b);
  p.lda = lda;
  p.ldb = ldb;
  p.m = m;
  p.n = n;
  p.k = k / 2;
  p.epi = e;
  for (int attempt = 0; attempt < 2; ++attempt) {
    const Plan t = plan(p.m, p.n, p.k, cus, may_split && attempt == 0);
    if (t.tile < 0) return DG_ERROR_UNSUPPORTED;
    const GemmTile g = kGemmTiles[t.tile];
    set_tiles(p, g, t.splits, t.kchunk);
    const int64_t items = (int64_t)p.tiles_m * p.tiles_n * t.splits;
    if (items > (1 << 30)) return DG_ERROR_UNSUPPORTED;
    // a multiple of 8 workgroups: the ids of a workgroup stay on its XCD's run
    const int64_t slots = (int64_t)(cus > 8 ? cus / 8 * 8 : 8) * gemm_residents(t.tile);
    const int grid = (int)(items < slots ? (items + 7) / 8 * 8 : slots);
    if (std::getenv("DG_LOG"))
      std::fprintf(stderr, "[dg] linear int8 m=%d n=%d k=%d -> tile %dx%d wk=%d splits=%d grid=%d\n", m, n, k, g.bm,
                   g.bn, g.wk, t.splits, grid);
    if (t.splits == 1) return launch_gemm_int8(t.tile, p, sa, sb, grid, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
    p.ws_stride = (int64_t)p.m * p.n;
    SplitBuffer ws = split_buffer(stream, (size_t)(4 * t.splits * p.ws_stride));
    if (!ws.ptr) {
      (void)hipGetLastError();
      continue;  // no buffer to be had: the same product without a split
    }
    p.ws = static_cast<float*>(ws.ptr);
    const bool ok = launch_gemm_int8(t.tile, p, sa, sb, grid, stream) == hipSuccess &&
                    launch_splitk_int8(p, sa, sb, stream) == hipSuccess;
    const bool freed = return_split_buffer(ws, stream);
    return ok && freed ? DG_SUCCESS : DG_ERROR_LAUNCH;
  }
  return DG_ERROR_LAUNCH;
}

dg_status dg_quantize_int8_rows(const void* x, int64_t ld_x, int x_type, void* q, float* s, int m, int k,
                                hipStream_t stream) {
  if (!x || !q || !s || m <= 0 || k <= 0 || ld_x < k || (x_type != DG_TYPE_BF16 && x_type != DG_TYPE_F32))
    return DG_ERROR_INVALID_VALUE;
  const bool f32 = x_type == DG_TYPE_F32;
  if (!aligned(x, f32 ? 4 : 2) || !aligned(s, 4) || ld_x > ((int64_t)1 << 40) || k > 1 << 30)
    return DG_ERROR_UNSUPPORTED;
  (void)hipGetLastError();
  return launch_quantize_int8(x, f32, ld_x, static_cast<int8_t*>(q), s, m, k, stream) == hipSuccess ? DG_SUCCESS
                                                                                                    : DG_ERROR_LAUNCH;
}

}  // extern "C"
