// dg_linear_rows.hip -- the linear layer for few rows (M <= 64: decode steps,
// router logits): C = act(A.B^T + bias) + residual, bound by reading B once.
//
// A workgroup owns 16 R columns of C and all rows; its 8 waves take K blocks
// round robin and meet once in LDS.  B streams into registers with 16-byte
// nontemporal loads, D units ahead (dg_stream.h); A (at most 64 rows) is
// re-read through the L2 by every workgroup.  No second kernel and no
// workspace: the split over K is inside the workgroup.
#include "dg_linear.h"
#include "dg_stream.h"

namespace dg {
namespace {

using namespace stream;

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;

template <bool FP8, int NT, int R, int D>
__global__ __launch_bounds__(kThreads) void linear_rows_kernel(const RowsParams p) {
  constexpr int WL = FP8 ? 2 : 4;        // 16-byte pieces of a lane per unit, of both operands
  constexpr int BB = FP8 ? 128 : 256;    // bytes of a K block
  __shared__ __attribute__((aligned(16))) v4f red[kWaves][R * NT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int nb = (p.k + 127) >> 7;
  const int n = (nb + kWaves - 1) / kWaves;  // units per wave
  const int n0 = blockIdx.x * 16 * R;
  const int rows = min(16 * R, p.n - n0);
  const uint32_t kbytes = (uint32_t)p.k * (FP8 ? 1 : 2);
  const uint32_t ldb = (uint32_t)p.ldb, lda = (uint32_t)p.lda;
  const uint8_t* b0 = p.b + (int64_t)n0 * p.ldb;
  const uint32_t boff = (uint32_t)l16 * ldb + 16u * lq, aoff = (uint32_t)l16 * lda + 16u * lq;

  v4i ws[D][R][WL], xs[D][NT][WL];
  float sb[D], sa[D][NT];
  int lj = 0;
  auto load = [&](int d) {
    const int kb = wave + kWaves * lj;
    const bool live = kb < nb;
    const uint32_t koff = live ? (uint32_t)kb * BB : 0u;
    // rows past the operands' last one end the range; K past the row's end
    // (BF16 only: FP8 has whole blocks) is left out lane by lane
    const auto rb = rsrc(b0 + koff, live ? (uint32_t)(rows - 1) * ldb + kbytes - koff : 0u);
    const auto ra = rsrc(p.a + koff, live ? (uint32_t)(p.m - 1) * lda + kbytes - koff : 0u);
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const bool in = FP8 || koff + 64u * i + 16u * lq < kbytes;
#pragma unroll
      for (int r = 0; r < R; ++r)
        ws[d][r][i] = load16<kNt>(rb, in ? boff + 16u * r * ldb + 64u * i : kOut);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xs[d][t][i] = load16<0>(ra, in ? aoff + 16u * t * lda + 64u * i : kOut);
    }
    if constexpr (FP8) {
      const auto rs = rsrc(p.sb + (int64_t)(n0 >> 7) * nb + kb, live ? 4u : 0u);
      sb[d] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, 0, 0, 0));
      const auto rt = rsrc(p.sa + kb, live ? ((uint32_t)(p.m - 1) * nb + 1) * 4u : 0u);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        sa[d][t] = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(rt, (uint32_t)(16 * t + l16) * nb * 4u, 0, 0));
    }
    ++lj;
  };

  v4f acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int d = 0; d < D; ++d) load(d);
  for (int c = 0; c < n; c += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (c + d >= n) break;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (FP8) {
            const v8i w = v8i{ws[d][r][0][0], ws[d][r][0][1], ws[d][r][0][2], ws[d][r][0][3],
                              ws[d][r][1][0], ws[d][r][1][1], ws[d][r][1][2], ws[d][r][1][3]};
            const v8i x = v8i{xs[d][t][0][0], xs[d][t][0][1], xs[d][t][0][2], xs[d][t][0][3],
                              xs[d][t][1][0], xs[d][t][1][1], xs[d][t][1][2], xs[d][t][1][3]};
            const v4f q = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0,
                                                                           0, 0);
            const float s = sa[d][t] * sb[d];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][t][e] = __builtin_fmaf(s, q[e], acc[r][t][e]);
          } else {
#pragma unroll
            for (int i = 0; i < WL; ++i)
              acc[r][t] = mfma_bf16(__builtin_bit_cast(v8bf, ws[d][r][i]), __builtin_bit_cast(v8bf, xs[d][t][i]),
                                    acc[r][t]);
          }
        }
      load(d);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[wave][r * NT + t][lane] = acc[r][t];
  __syncthreads();
  for (int s = wave; s < R * NT; s += kWaves) {
    v4f v = red[0][s][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[w][s][lane];
    const int m = 16 * (s % NT) + l16, c = n0 + 16 * (s / NT) + 4 * lq;
    if (m < p.m && c < p.n) {
      v += epi::bias4(p.epi, c, p.n);
      epi::finish4(p.epi, m, c, p.n, v);
    }
  }
}

template <bool FP8, int NT, int R, int D>
hipError_t launch(const RowsParams& p, hipStream_t stream) {
  linear_rows_kernel<FP8, NT, R, D><<<(p.n + 16 * R - 1) / (16 * R), kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_rows(bool fp8, const RowsParams& p, int, hipStream_t stream) {
  if (fp8) {
    if (p.m <= 16) return launch<true, 1, 1, 4>(p, stream);
    if (p.m <= 32) return launch<true, 2, 1, 4>(p, stream);
    return launch<true, 4, 1, 3>(p, stream);
  }
  if (p.m <= 16) return launch<false, 1, 1, 4>(p, stream);
  if (p.m <= 32) return launch<false, 2, 1, 3>(p, stream);
  return launch<false, 4, 1, 2>(p, stream);
}

}  // namespace dg
