// dg_linear.h -- what the linear layer's host code (dg_linear.hip) and its
// kernels (dg_linear_rows.hip: few rows; dg_linear_gemm.hip: tiles) share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_epilogue.h"
#include "dg_kernel.h"

namespace dg {

// Few rows (M <= 64): BF16 or FP8 operands, K contiguous in both.
constexpr int kMaxFewRows = 64;
struct RowsParams {
  const uint8_t* a;  // [M, K], rows lda bytes apart
  const uint8_t* b;  // [N, K], rows ldb bytes apart
  const float* sa;   // FP8: [M, K/128]
  const float* sb;   // FP8: [ceil(N/128), K/128]
  int64_t lda, ldb;
  int m, n, k;       // k in values
  Epilogue epi;
};
// Columns of C per workgroup: 16 where 32 would occupy at most half of the CUs
constexpr int few_rows_columns(int n, int num_cus) { return n <= 16 * num_cus ? 16 : 32; }
hipError_t launch_linear_rows(bool fp8, const RowsParams& p, int num_cus, hipStream_t stream);
// INT8: k counts pairs of values (the bytes of as many bf16 ones), sa [M], sb [N]
hipError_t launch_linear_rows_int8(const RowsParams& p, int num_cus, hipStream_t stream);

// Tiles, BF16: C[m, n] = sum_k A(m, k) B(n, k).  An operand is stored with K
// contiguous ([rows, K]) or, "transposed", with K as the row index ([K, rows]).
struct GemmParams {
  const uint8_t* a;
  const uint8_t* b;
  int64_t lda, ldb;  // bytes between rows of the stored operand
  int wa, wb;        // a transposed operand's stored width: its row count rounded up to 8
  int m, n, k;
  int tiles_m, tiles_n;
  int splits, kchunk;  // K blocks of 64 per split
  float* ws;           // fp32 partials [splits][m][n] (splits > 1)
  int64_t ws_stride;
  Epilogue epi;
};
enum GemmLayout : int { kNT = 0, kNN = 1, kTN = 2 };  // A, B stored: [m,k] [n,k]; [m,k] [k,n]; [k,m] [k,n]

struct GemmTile {
  int bm, bn, wm, wn, wk, stages;  // wk groups of wm x wn waves, each every wk-th block of K
};
constexpr int gemm_threads(const GemmTile& t) { return t.wm * t.wn * t.wk * 64; }
constexpr GemmTile kGemmTiles[] = {
    {256, 256, 2, 4, 1, 2}, {256, 128, 4, 2, 1, 3}, {128, 128, 2, 2, 1, 2}, {64, 128, 2, 2, 1, 3},
    {64, 64, 2, 2, 1, 4},   {128, 128, 2, 2, 2, 2}, {64, 128, 2, 2, 2, 3},  {64, 64, 2, 2, 2, 3}};
constexpr int kNumGemmTiles = 8, kNumPairTiles = 5;  // the first kNumPairTiles in launch_gemm_pair too
// workgroups of a tile that share a CU (LDS)
constexpr int gemm_residents(int tile) { return tile >= 2 && tile <= 4 ? 2 : 1; }
hipError_t launch_gemm(int layout, int tile, const GemmParams& p, int grid, hipStream_t stream);

// INT8, both operands with K contiguous (launch_gemm's kNT): p.k counts pairs of values, p.ws holds int32 partials,
// and launch_splitk_int8 turns those into C.
hipError_t launch_gemm_int8(int tile, const GemmParams& p, const float* sa, const float* sb, int grid,
                            hipStream_t stream);
hipError_t launch_splitk_int8(const GemmParams& p, const float* sa, const float* sb, hipStream_t stream);

// Rows of x [m, k] as INT8 with a scale each.
hipError_t launch_quantize_int8(const void* x, bool f32, int64_t ldx, int8_t* q, float* s, int m, int k,
                                hipStream_t stream);

// An NN and a TN product (neither split, both with Epilogue::vec8) in one launch: `first` workgroups (a multiple of 8) on
// the first, the rest on the second; and the bias sum of launch_bias_sum (dbias
// null: none).
hipError_t launch_gemm_pair(int tile, const GemmParams& nn, const GemmParams& tn, int first, int grid,
                            const float* partial, float* dbias, int chunks, hipStream_t stream);

// dpre = dc * act'(pre) as bf16 [m, ldp] (columns n .. ldp - 1 zero), unless
// dpre is null, and the column sums of the unrounded dpre in chunks of `rows`
// rows, partial [ceil(m / rows)][n], unless partial is null.
struct DactParams {
  const uint16_t* dc;
  const uint16_t* pre;  // null: no activation
  uint16_t* dpre;
  float* partial;
  int64_t lddc, ldpre, ldp;
  int rows;             // a multiple of 8
  int m, n, act, vec;   // vec: rows of dc and pre start on 16-byte boundaries
};
hipError_t launch_dact(const DactParams& p, hipStream_t stream);
// dbias[c] = sum over chunks of partial[chunk][c], in order
hipError_t launch_bias_sum(const float* partial, float* dbias, int chunks, int n, hipStream_t stream);

}  // namespace dg
