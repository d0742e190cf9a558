// dg_linear_gemm.hip -- the linear layer's BF16 kernels: the tiles of
// dg_linear_tile.h (the forward product, and the two products of the backward
// pass), the activation's backward pass and the bias gradient.
#include <cstddef>

#include "dg_linear_tile.h"

namespace dg {
namespace {

using namespace tile;

// dbias of columns 64 b .. 64 b + 63: a workgroup's first four waves sum a
// quarter of the chunks each.
__device__ __forceinline__ void bias_sum(const float* partial, float* dbias, int chunks, int n, int b,
                                         float (*sum)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = b * 64 + lane, per = (chunks + 3) / 4;
  float v = 0.f;
  if (wave < 4 && c < n) {
#pragma unroll 8
    for (int k = wave * per; k < min(chunks, (wave + 1) * per); ++k) v += partial[(int64_t)k * n + c];
  }
  if (wave < 4) sum[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < n) dbias[c] = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
}

template <int BM, int BN, int WM, int WN, int WK, int S, bool TA, bool TB, bool LINES>
__global__ __launch_bounds__(WM * WN * WK * 64) void linear_gemm_kernel(const GemmParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds<BM, BN, WM, WN, WK, S>];
  run_items<BM, BN, WM, WN, WK, S, TA, TB, LINES, 0>(p, blockIdx.x, gridDim.x, smem);
}

// The two products of the backward pass in one launch: workgroups below
// `first` compute da (NN), the others db (TN).  Small ones overlap whole
// (517 x 1161 x 1096: 27 us against 33 in two launches), large ones fill the
// card's last pass together.
// The workgroups past the products' sum the bias partials (bias_sum).
struct PairParams {
  GemmParams nn, tn;
  int first, grid;
  const float* partial;
  float* dbias;
  int chunks;
};
template <int BM, int BN, int WM, int WN, int WK, int S>
__global__ __launch_bounds__(WM * WN * WK * 64) void linear_gemm_pair_kernel(const PairParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds<BM, BN, WM, WN, WK, S>];
  if ((int)blockIdx.x < p.first)
    run_items<BM, BN, WM, WN, WK, S, false, true, true, offsetof(PairParams, nn)>(p.nn, blockIdx.x, p.first, smem);
  else if ((int)blockIdx.x < p.grid)
    run_items<BM, BN, WM, WN, WK, S, true, true, true, offsetof(PairParams, tn)>(p.tn, blockIdx.x - p.first,
                                                                             p.grid - p.first, smem);
  else
    bias_sum(p.partial, p.dbias, p.chunks, p.tn.m, blockIdx.x - p.grid, reinterpret_cast<float(*)[64]>(smem));
}

template <int TILE, bool TA, bool TB>
hipError_t launch_tile(const GemmParams& p, int grid, hipStream_t stream) {
  constexpr GemmTile t = kGemmTiles[TILE];
  if (p.splits == 1 && p.epi.vec8)
    linear_gemm_kernel<t.bm, t.bn, t.wm, t.wn, t.wk, t.stages, TA, TB, true><<<grid, gemm_threads(t), 0, stream>>>(p);
  else
    linear_gemm_kernel<t.bm, t.bn, t.wm, t.wn, t.wk, t.stages, TA, TB, false><<<grid, gemm_threads(t), 0, stream>>>(p);
  return hipGetLastError();
}

template <int TILE>
hipError_t launch_layout(int layout, const GemmParams& p, int grid, hipStream_t stream) {
  if (layout == kNT) return launch_tile<TILE, false, false>(p, grid, stream);
  if (layout == kNN) return launch_tile<TILE, false, true>(p, grid, stream);
  return launch_tile<TILE, true, true>(p, grid, stream);
}

template <int TILE>
hipError_t launch_both(const PairParams& p, hipStream_t stream) {
  constexpr GemmTile t = kGemmTiles[TILE];
  const int grid = p.grid + (p.dbias ? (p.tn.m + 63) / 64 : 0);
  linear_gemm_pair_kernel<t.bm, t.bn, t.wm, t.wn, t.wk, t.stages><<<grid, gemm_threads(t), 0, stream>>>(p);
  return hipGetLastError();
}

// ---- the activation's backward pass and the bias gradient ----
// A workgroup takes 256 columns x p.rows rows.  Bound by HBM: dc and pre read,
// dpre written, once (4096 x 7168: 34 us, 5.2 TB/s).  dpre is rounded to bf16, the
// MFMA's operand type: da and db are 2.35e-3 off in the norm, where their own
// rounding alone gives 1.66e-3; the bias gradient sums the unrounded values.
//
// Rows on 16-byte boundaries: 32 lanes of 8 columns by 8 rows in flight; the
// column sums of the 8 row lanes meet in LDS.
__global__ __launch_bounds__(256) void dact_kernel(const DactParams p) {
  __shared__ float sum[8][256];
  const int lx = threadIdx.x & 31, ly = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + lx * 8, r0 = blockIdx.y * p.rows;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.f;
  if (c < p.ldp) {
#pragma unroll 2
    for (int r = r0 + ly; r < min(p.m, r0 + p.rows); r += 8) {
      float d[8], x[8];
      const uint16_t* dc = p.dc + (int64_t)r * p.lddc + c;
      const uint16_t* pr = p.pre ? p.pre + (int64_t)r * p.ldpre + c : nullptr;
      if (c + 7 < p.n) {
        const uint4 v = *reinterpret_cast<const uint4*>(dc);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[2 * e] = epi::from_bf16(w[e] & 0xffffu);
          d[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
        if (pr) {
          const uint4 u = *reinterpret_cast<const uint4*>(pr);
          const uint32_t y[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[2 * e] = epi::from_bf16(y[e] & 0xffffu);
            x[2 * e + 1] = __uint_as_float(y[e] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] = c + e < p.n ? epi::from_bf16(dc[e]) : 0.f;
          x[e] = pr && c + e < p.n ? epi::from_bf16(pr[e]) : 0.f;
        }
      }
      if (pr) act::times_grad<8>(d, x, p.act);
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += d[e];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = (uint32_t)epi::to_bf16(d[2 * e]) | ((uint32_t)epi::to_bf16(d[2 * e + 1]) << 16);
      if (p.dpre)  // (the padding columns are zeros: 0 times a finite derivative)
        *reinterpret_cast<uint4*>(p.dpre + (int64_t)r * p.ldp + c) = uint4{o[0], o[1], o[2], o[3]};
    }
  }
  if (p.partial) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[ly][lx * 8 + e] = s[e];
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col < p.n) {
      float v = 0.f;
#pragma unroll
      for (int y = 0; y < 8; ++y) v += sum[y][threadIdx.x];
      p.partial[(int64_t)blockIdx.y * p.n + col] = v;
    }
  }
}

// Other rows: one column per lane (2-byte accesses that cover whole runs), 16
// rows in flight (517 x 1161: 5 us; columns 32 apart by one lane, each behind its
// own branch, 13).  Rows may lie any distance apart: their starts are 64-bit and
// uniform, a lane's column is 32-bit.  Lanes and rows past the end read the last
// column and row again, so that no load has a branch, and drop what they get.
__global__ __launch_bounds__(256) void dact_columns_kernel(const DactParams p) {
  const int c = blockIdx.x * 256 + threadIdx.x, r0 = blockIdx.y * p.rows;
  const int rows = min(p.rows, p.m - r0);
  const bool in = c < p.n;
  const uint32_t at = 2u * (uint32_t)min(c, p.n - 1);  // bytes into a row
  auto value = [&](const uint16_t* base, int64_t ld, int r) {
    const uint8_t* row = reinterpret_cast<const uint8_t*>(base + (int64_t)(r0 + min(r, rows - 1)) * ld);
    return epi::from_bf16(*reinterpret_cast<const uint16_t*>(row + at));
  };
  float s = 0.f;
  for (int r = 0; r < rows; r += 16) {
    float d[16], x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) d[e] = value(p.dc, p.lddc, r + e);
    if (p.pre) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = value(p.pre, p.ldpre, r + e);
      act::times_grad<16>(d, x, p.act);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (!in || r + e >= rows) d[e] = 0.f;
      s += d[e];
      if (p.dpre && c < p.ldp && r + e < rows) p.dpre[(int64_t)(r0 + r + e) * p.ldp + c] = epi::to_bf16(d[e]);
    }
  }
  if (p.partial && in) p.partial[(int64_t)blockIdx.y * p.n + c] = s;
}

__global__ __launch_bounds__(256) void bias_sum_kernel(const float* partial, float* dbias, int chunks, int n) {
  __shared__ float sum[4][64];
  bias_sum(partial, dbias, chunks, n, blockIdx.x, sum);
}

}  // namespace

hipError_t launch_gemm(int layout, int tile, const GemmParams& p, int grid, hipStream_t stream) {
  switch (tile) {
    case 0: return launch_layout<0>(layout, p, grid, stream);
    case 1: return launch_layout<1>(layout, p, grid, stream);
    case 2: return launch_layout<2>(layout, p, grid, stream);
    case 3: return launch_layout<3>(layout, p, grid, stream);
    case 4: return launch_layout<4>(layout, p, grid, stream);
    case 5: return launch_layout<5>(layout, p, grid, stream);
    case 6: return launch_layout<6>(layout, p, grid, stream);
    case 7: return launch_layout<7>(layout, p, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_gemm_pair(int tile, const GemmParams& nn, const GemmParams& tn, int first, int grid,
                            const float* partial, float* dbias, int chunks, hipStream_t stream) {
  const PairParams p{nn, tn, first, grid, partial, dbias, chunks};
  switch (tile) {
    case 0: return launch_both<0>(p, stream);
    case 1: return launch_both<1>(p, stream);
    case 2: return launch_both<2>(p, stream);
    case 3: return launch_both<3>(p, stream);
    case 4: return launch_both<4>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_dact(const DactParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.ldp + 255) / 256), (unsigned)((p.m + p.rows - 1) / p.rows));
  if (p.vec)
    dact_kernel<<<grid, 256, 0, stream>>>(p);
  else
    dact_columns_kernel<<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_bias_sum(const float* partial, float* dbias, int chunks, int n, hipStream_t stream) {
  bias_sum_kernel<<<(n + 63) / 64, 256, 0, stream>>>(partial, dbias, chunks, n);
  return hipGetLastError();
}

}  // namespace dg
