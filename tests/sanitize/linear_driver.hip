// linear_driver.hip -- the linear layer's and the few-token MoE layer's host
// code (tests/test_host_linear.py): every plan that sizes from one row to
// thousands get, held against what the kernels assume, and accepted and refused
// calls.
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include "recording_stubs.h"

namespace {

int bad = 0;
long launches = 0;
#define CHECK(c)                                                              \
  do {                                                                        \
    if (!(c)) {                                                               \
      if (bad++ < 20) fprintf(stderr, "line %d: %s (%s)\n", __LINE__, #c, at); \
    }                                                                         \
  } while (0)
char at[128];

int up(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

void check_gemm(const dg::GemmParams& p, const dg::GemmTile& t, int grid) {
  const int blocks = up(p.k, 64);
  CHECK(p.tiles_m == up(p.m, t.bm) && p.tiles_n == up(p.n, t.bn));
  CHECK(p.splits >= 1 && p.kchunk >= 1 && up(blocks, p.kchunk) == p.splits);  // no empty split, none missing
  CHECK(grid > 0 && grid % 8 == 0);
  CHECK((int64_t)p.tiles_m * p.tiles_n * p.splits <= (1 << 30));
  CHECK(p.splits == 1 || (p.ws && p.ws_stride == (int64_t)p.m * p.n && p.ws_stride * 4 * p.splits <= 256000000));
  // 32-bit byte offsets: a tile's rows of either operand, and of every output
  CHECK(255 * p.lda + 128 < (1ll << 31) && 255 * p.ldb + 128 < (1ll << 31));
  CHECK((255 * p.epi.ldc + p.n) * 4 < (1ll << 31));
}

}  // namespace

void rec::seen_gemm(int, int tile, const dg::GemmParams& p, int grid) {
  ++launches;
  CHECK(tile >= 0 && tile < dg::kNumGemmTiles);
  check_gemm(p, dg::kGemmTiles[tile], grid);
}
void rec::seen_pair(int tile, const dg::GemmParams& nn, const dg::GemmParams& tn, int first, int grid, int chunks) {
  ++launches;
  CHECK(tile >= 0 && tile < dg::kNumPairTiles);
  CHECK(first > 0 && first % 8 == 0 && grid > first);
  check_gemm(nn, dg::kGemmTiles[tile], first);
  check_gemm(tn, dg::kGemmTiles[tile], grid - first);
  CHECK(nn.splits == 1 && tn.splits == 1 && nn.epi.vec8 && tn.epi.vec8);
  CHECK(nn.k == tn.m && nn.m == tn.k && nn.n == tn.n && chunks > 0);
}
void rec::seen_rows(const dg::RowsParams& p) {
  ++launches;
  CHECK(p.m <= dg::kMaxFewRows && (int64_t)(p.m - 1) * p.lda + 2ll * p.k < (1ll << 31));
}
void rec::seen_dact(const dg::DactParams& p) {
  CHECK(p.rows > 0 && p.rows % 8 == 0 && (p.dpre || p.partial) && p.ldp >= p.n && p.ldp % 8 == 0);
  CHECK(up(p.m, p.rows) <= 65536);  // the grid's y
}
void rec::seen_fp8(int kind, const dg::TileShape& s, const dg::Params& p, int grid) {
  ++launches;
  CHECK(dg::has_instance(kind, s) && p.tiles_m == up(p.m, s.bm) && p.tiles_n == up(p.n, s.bn));
  CHECK(grid > 0 && up(p.kbs, p.kchunk) == p.splits && (p.splits == 1 || p.ws));
}

int main() {
  void* const P = reinterpret_cast<void*>(uintptr_t(0x10000));
  float* const F = static_cast<float*>(P);
  const int ms[] = {1, 2, 16, 17, 40, 64, 65, 130, 517, 2048, 4096, 70000, 1 << 22};
  const int ns[] = {1, 8, 64, 141, 1024, 4097, 7168, 1 << 20};
  const int ks[] = {8, 64, 136, 1096, 2048, 7168, 1 << 22};
  for (int cus : {256, 64, 8, 1}) {
    rec::g_cus = cus;
    for (int m : ms)
      for (int n : ns)
        for (int k : ks) {
          snprintf(at, sizeof at, "cus=%d m=%d n=%d k=%d", cus, m, n, k);
          dg_epilogue e{};
          e.activation = (m + n) % 5;
          e.bias = P;
          if (n % 2) e.residual = P, e.ld_residual = n;
          for (int type : {DG_TYPE_BF16, DG_TYPE_F32})
            CHECK(dg_gemm_bf16_nt_epilogue(P, k, P, k, P, n, type, &e, m, n, k, nullptr) == DG_SUCCESS);
          const int k8 = (k + 127) / 128 * 128;
          const dg_status s = dg_gemm_fp8_nt_epilogue(P, F, P, F, P, n, (m + k) % 2, &e, m, n, k8, nullptr);
          CHECK(s == DG_SUCCESS || (s == DG_ERROR_UNSUPPORTED && (int64_t)m * n > (1ll << 36)));
          if (k > (1 << 20)) continue;  // (the gradients' rows)
          int64_t need = 0;
          CHECK(dg_gemm_bf16_nt_epilogue_backward_workspace(m, n, &need) == DG_SUCCESS && need >= 2ll * m * n);
          const int parts = (m + n + k / 8) % 4;  // all three, or two of them
          CHECK(dg_gemm_bf16_nt_epilogue_backward(P, n, P, k, P, k, P, n, (m + n) % 5, parts == 1 ? nullptr : P, k,
                                                  parts == 2 ? nullptr : P, k, parts == 3 ? nullptr : F, P, m, n, k,
                                                  nullptr) == DG_SUCCESS);
        }
    for (int t : {1, 16, 17, 64})
      for (int h : {128, 4096, 4224, 1 << 20})
        for (int i : {128, 1408, 1 << 20})
          for (int e : {1, 64, 512}) {
            snprintf(at, sizeof at, "cus=%d t=%d h=%d i=%d e=%d", cus, t, h, i, e);
            const int k = e < 16 ? e : 16;
            int32_t* ids = static_cast<int32_t*>(P);
            rec::g_grids.clear();
            CHECK(dg_moe_few_tokens_fp8(P, F, ids, F, P, F, P, F, P, P, P, t, h, i, e, k, 0, 1, 1.f, nullptr) == DG_SUCCESS);
            CHECK(dg_moe_few_tokens_bf16(P, nullptr, ids, F, P, P, nullptr, P, P, t, h, i, e, k, 1, 0, 1.f, nullptr) ==
                  DG_SUCCESS);
            CHECK(rec::g_grids.size() == 4);
            for (int g : rec::g_grids) CHECK(g > 0 && g <= (1 << 16));
            CHECK(dg_moe_few_tokens_fp8(P, F, ids, F, P, F, P, F, P, P, P, t, h, i, e, e + 1, 0, 1, 1.f, nullptr) ==
                  DG_ERROR_INVALID_VALUE);
          }
  }
  // refused calls reach no launch
  snprintf(at, sizeof at, "refusals");
  const long before = launches;
  const int64_t far = (1ll << 20) + 8;
  CHECK(dg_gemm_bf16_nt_epilogue(P, LLONG_MAX & ~7ll, P, 64, P, 64, 0, nullptr, 8, 64, 64, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(dg_gemm_bf16_nt_epilogue(P, 64, P, 64, P, LLONG_MAX, 0, nullptr, 8, 64, 64, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(dg_gemm_bf16_nt_epilogue(P, 64, P, 64, P, 64, 0, nullptr, 8, 64, INT_MAX & ~7, nullptr) == DG_ERROR_INVALID_VALUE);
  CHECK(dg_gemm_bf16_nt_epilogue_backward(P, 64, P, 64, P, 64, P, 64, 1, P, far, P, 64, F, P, 8, 64, 64, nullptr) ==
        DG_ERROR_UNSUPPORTED);
  CHECK(dg_gemm_bf16_nt_epilogue_backward(P, 64, P, 64, P, 64, P, 64, 1, P, 64, P, far, F, P, 8, 64, 64, nullptr) ==
        DG_ERROR_UNSUPPORTED);
  CHECK(launches == before);
  CHECK(launches > 2000);
  printf("launches=%ld bad=%d\n", launches, bad);
  return bad != 0;
}
