// rows_driver.hip -- the host code of the norm, the sorted tokens and the INT8
// layer (tests/test_host_rows.py): launches and plans that sizes from one to the
// largest get, held against what the kernels assume, and refused calls.
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
char at[160];

int up(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// The kernels launched by name since the last call: how many, and of the last
// one that it has threads and fewer than 2^32 of them.
size_t launched() {
  const size_t n = rec::g_grids.size();
  for (int g : rec::g_grids) CHECK(g > 0);
  if (n) {
    const uint64_t groups = (uint64_t)rec_grid.x * rec_grid.y * rec_grid.z;
    CHECK(rec_block.x % 64 == 0 && rec_block.x <= 1024 && groups * rec_block.x < (1ull << 32));
  }
  rec::g_grids.clear();
  return n;
}

}  // namespace

void rec::seen_gemm(int, int, const dg::GemmParams&, int) { CHECK(false); }
void rec::seen_pair(int, const dg::GemmParams&, const dg::GemmParams&, int, int, int) { CHECK(false); }
void rec::seen_rows(const dg::RowsParams&) { CHECK(false); }
void rec::seen_dact(const dg::DactParams&) { CHECK(false); }
void rec::seen_fp8(int, const dg::TileShape&, const dg::Params&, int) { CHECK(false); }

namespace dg {
hipError_t launch_linear_rows_int8(const RowsParams& p, int, hipStream_t) {
  ++launches;
  CHECK(p.m <= kMaxFewRows && (int64_t)(p.m - 1) * p.lda + 2ll * p.k < (1ll << 31) && p.k % 8 == 0 && p.sa && p.sb);
  return hipSuccess;
}
hipError_t launch_gemm_int8(int tile, const GemmParams& p, const float* sa, const float* sb, int grid, hipStream_t) {
  ++launches;
  CHECK(tile >= 0 && tile < kNumGemmTiles && sa && sb && grid > 0 && grid % 8 == 0);
  const GemmTile& t = kGemmTiles[tile];
  CHECK(p.tiles_m == up(p.m, t.bm) && p.tiles_n == up(p.n, t.bn) && p.k % 8 == 0);
  CHECK(p.splits >= 1 && p.kchunk >= 1 && up(up(p.k, 64), p.kchunk) == p.splits);
  CHECK((int64_t)p.tiles_m * p.tiles_n * p.splits <= (1 << 30));
  CHECK(p.splits == 1 || (p.ws && p.ws_stride == (int64_t)p.m * p.n && p.ws_stride * 4 * p.splits <= 256000000));
  CHECK(255 * p.lda + 128 < (1ll << 31) && 255 * p.ldb + 128 < (1ll << 31) && (255 * p.epi.ldc + p.n) * 4 < (1ll << 31));
  return hipSuccess;
}
hipError_t launch_splitk_int8(const GemmParams& p, const float*, const float*, hipStream_t) {
  CHECK(p.splits > 1);
  return hipSuccess;
}
hipError_t launch_quantize_int8(const void*, bool, int64_t, int8_t*, float*, int, int, hipStream_t) { return hipSuccess; }
}  // namespace dg

int main() {
  void* const P = reinterpret_cast<void*>(uintptr_t(0x10000));
  void* const Q = reinterpret_cast<void*>(uintptr_t(0x7000000000));  // far from P
  float* const F = static_cast<float*>(P);
  int32_t* const I = static_cast<int32_t*>(P);
  // INT8 layer
  for (int cus : {256, 64, 8, 1}) {
    rec::g_cus = cus;
    for (int m : {1, 16, 17, 64, 65, 130, 517, 4096, 70000, 1 << 22})
      for (int n : {1, 8, 141, 1024, 7168, 1 << 20})
        for (int k : {16, 64, 272, 2048, 7168, (1 << 17) - 16}) {
          snprintf(at, sizeof at, "int8 cus=%d m=%d n=%d k=%d", cus, m, n, k);
          dg_epilogue e{};
          e.activation = (m + n) % 5;
          e.bias = P;
          if (n % 2) e.residual = P, e.ld_residual = n;
          for (int type : {DG_TYPE_BF16, DG_TYPE_F32})
            CHECK(dg_gemm_int8_nt_epilogue(P, k, F, P, k, F, P, n, type, &e, m, n, k, nullptr) == DG_SUCCESS);
        }
  }
  CHECK(launches > 1000);
  // norm
  for (int t : {1, 2, 511, 512, 768, 769, 5000, 1 << 21, (1 << 21) + 1, INT_MAX})
    for (int h : {1, 8, 64, 100, 512, 2048, 2111, 4096, 4100, 8192, 8200, 16383, 16384}) {
      snprintf(at, sizeof at, "norm t=%d h=%d", t, h);
      dg_norm in{};
      in.x = P;
      in.ld_x = h;
      in.eps = 1e-6f;
      CHECK(dg_rmsnorm_bf16(&in, P, h, t, h, nullptr) == DG_SUCCESS && launched() == 1);
      CHECK(dg_rmsnorm_quantize_int8(&in, P, F, t, h, nullptr) == DG_SUCCESS && launched() == 1);
      const dg_status s = dg_rmsnorm_quantize_fp8_1x128(&in, P, F, t, h, nullptr);
      CHECK(s == (h % 128 ? DG_ERROR_UNSUPPORTED : DG_SUCCESS) && launched() == (h % 128 ? 0u : 1u));
      int64_t need = -1;
      CHECK(dg_rmsnorm_bf16_backward_workspace(t, h, &need) == DG_SUCCESS && need >= 0);
      void* ws = need ? P : nullptr;
      auto backward = [&](void* dx, float* dw) {
        return dg_rmsnorm_bf16_backward(P, h, P, h, nullptr, 0, F, nullptr, 0, dx, h, dw, ws, t, h, nullptr);
      };
      CHECK(backward(Q, F) == DG_SUCCESS && launched() == (need ? 2u : 1u));
      CHECK(backward(P, F) == DG_SUCCESS && launched() == 2);  // dx over its inputs: dw apart
      CHECK(backward(Q, nullptr) == DG_SUCCESS && launched() == 1);
      CHECK(backward(nullptr, F) == DG_SUCCESS && launched() == (need ? 2u : 1u));
      CHECK(backward(nullptr, nullptr) == DG_SUCCESS && launched() == 0);
    }
  // sorted tokens
  for (int t : {1, 64, 1024, 1025, 2048, 2049, 70000, 1 << 19, 1 << 23})
    for (int k : {1, 8, 16})
      for (int e : {1, 7, 256, 1024}) {
        snprintf(at, sizeof at, "sort t=%d k=%d e=%d", t, k, e);
        int64_t need = -1;
        const dg_status s = dg_moe_sort_workspace(t, k, e, &need);
        const bool fits = (int64_t)t * k <= (1 << 23);
        CHECK(s == (fits ? DG_SUCCESS : DG_ERROR_UNSUPPORTED));
        if (!fits) continue;
        CHECK(need >= 0 && need <= 256 * 4 * (int64_t)e);
        const size_t n = need ? 2 : 1;
        CHECK(dg_moe_sort_contiguous(I, I, I, nullptr, need ? P : nullptr, t, k, e, 1 << 20, nullptr) == DG_SUCCESS && launched() == n);
        CHECK(dg_moe_sort_masked(I, I, I, need ? P : nullptr, t, k, e, 128, nullptr) == DG_SUCCESS && launched() == n);
        if (need) CHECK(dg_moe_sort_masked(I, I, I, nullptr, t, k, e, 128, nullptr) == DG_ERROR_INVALID_VALUE && launched() == 0);
        for (int h : {128, 7168, 1 << 20})
          for (int64_t m : {(int64_t)128, (int64_t)1 << 24, (int64_t)INT_MAX / 128 * 128}) {
            snprintf(at, sizeof at, "rows t=%d k=%d h=%d m=%lld", t, k, h, (long long)m);
            CHECK(dg_moe_dispatch_bf16(P, h, I, I, P, t, k, h, m, nullptr) == DG_SUCCESS && launched() == 1);
            CHECK(dg_moe_dispatch_fp8(P, F, I, nullptr, P, F, t, k, h, m, nullptr) == DG_SUCCESS && launched() == 1);
            CHECK(dg_moe_dispatch_fp8_ue8m0(P, I, I, I, P, I, t, k, h, m, nullptr) == DG_SUCCESS && launched() == 1);
            CHECK(dg_moe_combine_bf16(P, I, F, P, h, P, h, t, k, h, m, nullptr) == DG_SUCCESS && launched() == 1);
            CHECK(dg_moe_combine_bf16_backward(P, h, P, I, F, I, P, F, t, k, h, m, nullptr) == DG_SUCCESS && launched() == 1);
          }
      }
  // refused calls reach no launch
  snprintf(at, sizeof at, "refusals");
  const long before = launches;
  CHECK(dg_gemm_int8_nt_epilogue(P, LLONG_MAX & ~15ll, F, P, 64, F, P, 64, 0, nullptr, 8, 64, 64, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(dg_gemm_int8_nt_epilogue(P, 64, F, P, 64, F, P, LLONG_MAX, 0, nullptr, 8, 64, 64, nullptr) == DG_ERROR_UNSUPPORTED);
  dg_norm in{};
  in.x = P;
  in.ld_x = LLONG_MAX;
  CHECK(dg_rmsnorm_bf16(&in, P, 64, 8, 64, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(dg_rmsnorm_bf16_backward(P, LLONG_MAX, P, 64, nullptr, 0, F, nullptr, 0, P, 64, F, P, 8, 64, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(dg_moe_sort_masked(I, I, I, P, INT_MAX, 16, 4, 8, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(dg_moe_dispatch_bf16(P, LLONG_MAX & ~7ll, I, I, P, 8, 2, 64, 128, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(dg_moe_combine_bf16(P, I, F, P, 64, P, LLONG_MAX & ~7ll, 8, 2, 64, 128, nullptr) == DG_ERROR_UNSUPPORTED);
  CHECK(launches == before && launched() == 0);
  printf("launches=%ld bad=%d\n", launches, bad);
  return bad != 0;
}
