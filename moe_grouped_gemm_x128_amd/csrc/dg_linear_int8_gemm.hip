// dg_linear_int8_gemm.hip -- the INT8 linear layer's kernels: the tiles of
// dg_linear_tile.h, the sum of K splits, and the quantiser of rows.
#include "dg_fp8_codec.h"
#include "dg_linear_tile.h"

namespace dg {
namespace {

using namespace tile;

template <int BM, int BN, int WM, int WN, int WK, int S, bool LINES>
__global__ __launch_bounds__(WM * WN * WK * 64) void linear_int8_kernel(const GemmParams p, const Scales s) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds<BM, BN, WM, WN, WK, S>];
  run_items<BM, BN, WM, WN, WK, S, false, false, LINES, 0, true>(p, blockIdx.x, gridDim.x, smem, s);
}

template <int TILE>
hipError_t launch_tile(const GemmParams& p, const Scales& s, int grid, hipStream_t stream) {
  constexpr GemmTile t = kGemmTiles[TILE];
  if (p.splits == 1 && p.epi.vec8)
    linear_int8_kernel<t.bm, t.bn, t.wm, t.wn, t.wk, t.stages, true><<<grid, gemm_threads(t), 0, stream>>>(p, s);
  else
    linear_int8_kernel<t.bm, t.bn, t.wm, t.wn, t.wk, t.stages, false><<<grid, gemm_threads(t), 0, stream>>>(p, s);
  return hipGetLastError();
}

// The K splits' int32 partials summed (exact, so in any order), scaled and
// through the epilogue: four columns per thread.
__global__ __launch_bounds__(256) void splitk_int8_kernel(const GemmParams p, const Scales s, int vec) {
  const int nq = (p.n + 3) / 4;
  const int64_t items = (int64_t)p.m * nq;
  const int* ws = reinterpret_cast<const int*>(p.ws);
  for (int64_t it = blockIdx.x * 256LL + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
    const int64_t row = it / nq;
    const int c = (int)(it - row * nq) * 4;
    const int* w = ws + row * p.n + c;
    const v4f bias = epi::bias4(p.epi, c, p.n);
    const float sa = s.sa[row];
    v4f sb;
#pragma unroll
    for (int r = 0; r < 4; ++r) sb[r] = s.sb[min(c + r, p.n - 1)];
    v4i sum = v4i{0, 0, 0, 0};
    if (vec && c + 3 < p.n) {
#pragma unroll 8
      for (int k = 0; k < p.splits; ++k) sum += *reinterpret_cast<const v4i*>(w + k * p.ws_stride);
    } else {
#pragma unroll 4
      for (int k = 0; k < p.splits; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (c + r < p.n) sum[r] += w[k * p.ws_stride + r];
    }
    v4f v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = (float)sum[r] * sb[r] * sa;
    epi::finish4(p.epi, row, c, p.n, v + bias);
  }
}

// Rows as INT8: s = amax / 127 (1 for a row of zeros), codes the nearest whole
// numbers to x / s, ties to even.  L lanes take a row and read it twice, the second
// time from the caches (a row of up to 128 K values is at most 512 KB).  Short rows
// are bound by the chain to a row's largest value, so they have fewer lanes and
// go several to a workgroup: 16 lanes up to 1 KB (bf16, us with 16, 64, 256: 131072 x
// 128 14, 34, 97; 32768 x 512 12, 15, 31), 64 up to 4 KB where rows are many (16384
// x 1024 13, 12, 20; 16384 x 2048 27, 23, 26), 256 beyond (7168 x 4096 37, 23, 20).
template <bool F32>
__device__ __forceinline__ float value(const void* x, int64_t i) {
  if constexpr (F32)
    return static_cast<const float*>(x)[i];
  else
    return epi::from_bf16(static_cast<const uint16_t*>(x)[i]);
}
template <bool F32>
__device__ __forceinline__ void value4(const void* x, int64_t i, float* f) {
  if constexpr (F32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + i);
    f[0] = epi::from_bf16(v.x);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = epi::from_bf16(v.y);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}
__device__ __forceinline__ int code(float x, const codec::GroupRecip& g) {
  return (int)__builtin_rintf(fminf(fmaxf(x * g.k * g.r, -127.f), 127.f));
}

template <bool F32, bool VEC, int L>
__global__ __launch_bounds__(256) void quantize_int8_kernel(const void* x, int64_t ldx, int8_t* q, float* s, int m, int k) {
  __shared__ float part[2][4];
  const int tid = threadIdx.x, own = tid % L;
  int turn = 0;
  for (int64_t row = blockIdx.x * (256LL / L) + tid / L; row < m; row += gridDim.x * (256LL / L), turn ^= 1) {
    const int64_t at = row * ldx;
    float most = 0.f;
    bool nan = false;
    if constexpr (VEC) {
#pragma unroll 4
      for (int c = own * 4; c < k; c += L * 4) {
        float f[4];
        value4<F32>(x, at + c, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          most = fmaxf(most, fabsf(f[e]));
          nan |= f[e] != f[e];
        }
      }
    } else {
#pragma unroll 4
      for (int c = own; c < k; c += L) {
        const float f = value<F32>(x, at + c);
        most = fmaxf(most, fabsf(f));
        nan |= f != f;
      }
    }
    most = nan ? __builtin_inff() : most;
#pragma unroll
    for (int d = (L < 64 ? L : 64) / 2; d > 0; d /= 2) most = fmaxf(most, __shfl_xor(most, d, 64));
    if constexpr (L > 64) {
      if ((tid & 63) == 0) part[turn][tid >> 6] = most;
      __syncthreads();
      most = fmaxf(fmaxf(part[turn][0], part[turn][1]), fmaxf(part[turn][2], part[turn][3]));
    }
    const float scale = most == 0.f ? 1.f : most / 127.f;
    const codec::GroupRecip g = codec::group_recip(scale);
    // (a row with a NaN or an infinity: a NaN scale)
    if (own == 0) s[row] = most < __builtin_inff() ? scale : __builtin_nanf("");
    int8_t* out = q + row * k;
    if constexpr (VEC) {
#pragma unroll 4
      for (int c = own * 4; c < k; c += L * 4) {
        float f[4];
        value4<F32>(x, at + c, f);
        *reinterpret_cast<uint32_t*>(out + c) = (uint32_t)(code(f[0], g) & 0xff) | ((uint32_t)(code(f[1], g) & 0xff) << 8) |
                                                ((uint32_t)(code(f[2], g) & 0xff) << 16) | ((uint32_t)code(f[3], g) << 24);
      }
    } else {
#pragma unroll 4
      for (int c = own; c < k; c += L) out[c] = (int8_t)code(value<F32>(x, at + c), g);
    }
  }
}

template <bool F32, bool VEC>
hipError_t launch_quantize(const void* x, int64_t ldx, int8_t* q, float* s, int m, int k, hipStream_t stream) {
  const int64_t bytes = (int64_t)k * (F32 ? 4 : 2);
  const int lanes = bytes <= 1024 ? 16 : bytes <= 4096 && m >= 1024 ? 64 : 256;
  const int64_t groups = ((int64_t)m * lanes + 255) / 256;
  const int grid = (int)(groups < (1 << 20) ? groups : 1 << 20);
  if (lanes == 16)
    quantize_int8_kernel<F32, VEC, 16><<<grid, 256, 0, stream>>>(x, ldx, q, s, m, k);
  else if (lanes == 64)
    quantize_int8_kernel<F32, VEC, 64><<<grid, 256, 0, stream>>>(x, ldx, q, s, m, k);
  else
    quantize_int8_kernel<F32, VEC, 256><<<grid, 256, 0, stream>>>(x, ldx, q, s, m, k);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_int8(int tile, const GemmParams& p, const float* sa, const float* sb, int grid,
                            hipStream_t stream) {
  const Scales s{sa, sb};
  switch (tile) {
    case 0: return launch_tile<0>(p, s, grid, stream);
    case 1: return launch_tile<1>(p, s, grid, stream);
    case 2: return launch_tile<2>(p, s, grid, stream);
    case 3: return launch_tile<3>(p, s, grid, stream);
    case 4: return launch_tile<4>(p, s, grid, stream);
    case 5: return launch_tile<5>(p, s, grid, stream);
    case 6: return launch_tile<6>(p, s, grid, stream);
    case 7: return launch_tile<7>(p, s, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_splitk_int8(const GemmParams& p, const float* sa, const float* sb, hipStream_t stream) {
  const int64_t blocks = ((int64_t)p.m * ((p.n + 3) / 4) + 255) / 256;
  splitk_int8_kernel<<<(int)(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(p, Scales{sa, sb}, p.n % 4 == 0 ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_quantize_int8(const void* x, bool f32, int64_t ldx, int8_t* q, float* s, int m, int k,
                                hipStream_t stream) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(x);
  const bool vec = k % 4 == 0 && (m == 1 || ldx % 4 == 0) && at % (f32 ? 16 : 8) == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0;
  if (f32)
    return vec ? launch_quantize<true, true>(x, ldx, q, s, m, k, stream) : launch_quantize<true, false>(x, ldx, q, s, m, k, stream);
  return vec ? launch_quantize<false, true>(x, ldx, q, s, m, k, stream) : launch_quantize<false, false>(x, ldx, q, s, m, k, stream);
}

}  // namespace dg
