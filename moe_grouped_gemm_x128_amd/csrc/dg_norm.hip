// dg_norm.hip -- root-mean-square norm of rows with the residual's addition
// (include/dg.h): output in bf16, FP8 with 1x128 scales or INT8 with a scale per
// row; and its backward pass.
//
//     z = x + residual,  r = 1 / sqrt(mean(z^2) + eps),  y = z r w
//
// A workgroup of W waves owns a row and keeps it in registers: a thread holds 8
// consecutive columns of each of I pieces of the row, so x and the residual are
// read once and z, y are written once, and one barrier separates them.  Rows may
// start anywhere: 16-byte accesses need no alignment here, and cost what aligned
// ones do but for a line more per wave (3000 x 7783: 58 us, 89 with one column per
// lane); only a row's last thread, where H is no multiple of 8, stores its values
// in pieces of 4, 2 and 1 (kTail; kernels of their own, since the branch alone costs
// the others 3%).  A short row (heads: H <= 512) belongs to L lanes of a wave
// instead, several rows to a wave, without LDS or barrier (131072 rows of 128:
// 34 us with a wave each, 13 so).  INT8's scale needs the row's largest |y| too:
// max |z w| is met at the same barrier as sum z^2 and multiplied by r after it
// (where that leaves fp32's range, max |y| is met at a barrier of its own).
//
// Bound by HBM: 4096 x 7168 with a residual into FP8 is 206 MB in 43.7 us, 4.7
// TB/s, where a copy reaches 5.1.  The 300 vector instructions of 16 values are a
// third of that, so they count: 8192 x 7168 into FP8 took 43.8 us with a square
// root and a division per thread and two factors per value, 38.7 without.
#include "dg_bf16.h"
#include "dg_fp8_codec.h"
#include "dg_kernel.h"

namespace dg {
namespace {

using bf16::from_bf16;
using bf16::to_bf16;

enum Out : int { kBf16 = 0, kFp8 = 1, kFp8Ue8m0 = 2, kInt8 = 3 };

constexpr int kMaxHidden = 16384;  // what 16 waves hold in two pieces
constexpr int64_t kMaxLd = (int64_t)1 << 40;

struct NormParams {
  const uint16_t* x;
  const uint16_t* res;  // or null
  const void* w;        // or null
  uint16_t* sum;        // or null
  float* rstd;          // or null
  void* y;              // bf16, FP8 or INT8
  void* s;              // scales
  int64_t ldx, ldr, lds, ldy;
  int t, h, w_f32;
  float eps, inv_h;
};

// ---- a thread's 8 consecutive values ----
// `left` values from p to the row's end.  Where those are fewer than 8 (there are
// h & 7, the same for every row: kTail) the last 8 of the row are loaded, and the
// first ones shifted out when they are used: one load for every lane, and no wait
// between a row's loads (333 x 2111 4.8 -> 4.6 us, backward of 2048 x 1161 13.6 -> 12.5).
// The values in front may be another lane's, which may be storing them: they are
// dropped.  kShort: h < 8, a lane per row, value by value.
enum Tail : int { kNone = 0, kTail = 1, kShort = 2 };
struct Raw {
  uint4 v;
};

template <int TAIL>
__device__ __forceinline__ Raw load(const uint16_t* p, int left, int h) {
  Raw r{uint4{0, 0, 0, 0}};
  if constexpr (TAIL == kShort) {
    uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < h) o[e / 2] |= (uint32_t)p[e] << (e % 2 * 16);
    r.v = uint4{o[0], o[1], o[2], o[3]};
  } else {
    __builtin_memcpy(&r.v, TAIL ? p + min(left - 8, 0) : p, 16);  // (one load, whatever the address)
  }
  return r;
}
template <int TAIL>
__device__ __forceinline__ void widen(const Raw& r, float* f, int left, int h) {
  uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
  if (TAIL == kTail && left < 8) {
    const int out = 8 - (h & 7);
    if (out & 4) w[0] = w[2], w[1] = w[3], w[2] = w[3] = 0;
    if (out & 2) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = 0;
    if (out & 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_alignbit(e < 3 ? w[e + 1] : 0u, w[e], 16);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = from_bf16(w[e]);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
template <int TAIL>
__device__ __forceinline__ void store(uint16_t* p, const float* f, int left, int h) {
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = (uint32_t)to_bf16(f[2 * e]) | ((uint32_t)to_bf16(f[2 * e + 1]) << 16);
  if (!TAIL || left >= 8) {
    __builtin_memcpy(p, o, 16);
  } else {
    if (h & 4) __builtin_memcpy(p, o, 8);
    const uint32_t two = h & 4 ? o[2] : o[0];
    if (h & 2) __builtin_memcpy(p + (h & 4), &two, 4);
    const uint32_t one = h & 4 ? (h & 2 ? o[3] : o[2]) : (h & 2 ? o[1] : o[0]);
    if (h & 1) p[h & 6] = (uint16_t)one;
  }
}
// The weight's values from column c on.
template <int TAIL>
__device__ __forceinline__ void load_weight(const void* w, int f32, int c, int h, float* f) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.f;
  } else if (f32) {
    const float* p = static_cast<const float*>(w) + c;
    if (!TAIL || h - c >= 8) {
      __builtin_memcpy(f, p, 32);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = c + e < h ? p[e] : 0.f;
    }
  } else {
    widen<TAIL>(load<TAIL>(static_cast<const uint16_t*>(w) + c, h - c, h), f, h - c, h);
  }
}

// ---- reductions ----
// v combined with the value `n` lanes round in the lane's row of 16.
template <int N>
__device__ __forceinline__ float round16(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float max16(float v) {  // over a row of 16 lanes, in all of them
  v = fmaxf(v, round16<8>(v));
  v = fmaxf(v, round16<4>(v));
  v = fmaxf(v, round16<2>(v));
  return fmaxf(v, round16<1>(v));
}
// The same over the L lanes of a row (0: over the wave).
template <int L>
__device__ __forceinline__ float max_row(float v) {
  v = max16(v);
  if constexpr (L != 16) v = fmaxf(v, __shfl_xor(v, 16, 64));
  if constexpr (L == 64 || L == 0) v = fmaxf(v, __shfl_xor(v, 32, 64));
  return v;
}
template <int L>
__device__ __forceinline__ float sum_row(float v) {
  v += round16<8>(v);
  v += round16<4>(v);
  v += round16<2>(v);
  v += round16<1>(v);
  if constexpr (L != 16) v += __shfl_xor(v, 16, 64);
  if constexpr (L == 64 || L == 0) v += __shfl_xor(v, 32, 64);
  return v;
}

// 1 / sqrt(v) by the root unit, within 2^-22 (a square root and a division are 25
// instructions in every lane).  Small v is raised by 2^64 first: the unit does
// without subnormal operands.
__device__ __forceinline__ float inverse_root(float v) {
  const bool small = v < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v);
  return small ? r * 0x1p32f : r;
}

// ---- scales ----
// FP8: amax / 448 as a product and 1 / s by the reciprocal unit: y / s is within
// 2^-21 of exact, and 2 instructions instead of two divisions' forty (every lane
// of a group computes them).  |y| <= amax and a subnormal s is rounded up, so no
// code needs a clamp.  A scale below 2^-60 is raised by 2^64, y alike, so that the
// reciprocal stays finite.
struct Factor {
  float s, k, r;
  __device__ __forceinline__ void scale(float* y) const {  // 8 values by 1 / s
    if (k != 1.f) {  // (rare)
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= k;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= r;
  }
};
__device__ __forceinline__ Factor fp8_factor(float amax) {
  float s = amax == 0.f ? 1.f : amax * (1.f / codec::kE4m3Max);
  if (s < 0x1p-126f) s += 0x1p-149f;  // (never below amax / 448: it was rounded by half of that)
  const float k = s < 0x1p-60f ? 0x1p64f : 1.f;
  return Factor{s, k, __builtin_amdgcn_rcpf(s * k)};
}
// INT8's, dg_quantize_int8_rows' rule: s = RN(amax / 127) and r = RN(1 / s), each the
// product or the unit and one residual, which is exact (checked for every amax and
// every mantissa of s; the product alone misses one scale in twenty, the unit one
// reciprocal in nine; 4096 x 7168 with a residual 44.3 us without the residuals, 44.7
// with them).
__device__ __forceinline__ Factor int8_factor(float amax) {
  constexpr float kInv = 1.f / 127.f;
  const bool small = amax < 0x1p-42f;  // (residuals and the reciprocal stay normal)
  const float k = small ? 0x1p64f : 1.f, a = amax * k;
  float d = a * kInv;
  d = __builtin_fmaf(__builtin_fmaf(-d, 127.f, a), kInv, d);
  float s = small ? d * 0x1p-64f : d;
  if (s < 0x1p-126f) {  // (zero, or rounded up)
    s = a == 0.f ? 1.f : s + 0x1p-149f;
    d = s * k;
  }
  const float r = __builtin_amdgcn_rcpf(d);
  return Factor{s, k, __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r)};
}
// codec::ue8m0_code, the least E with 2^(E - 127) >= RN(amax / 448), read off amax's
// fields: amax / 448 is amax / (1.75 2^8).  (The one value whose subnormal quotient is
// rounded down to a power is 0x4600001.  Checked for every finite amax.)  And 2^(127 - E).
__device__ __forceinline__ uint32_t power_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0) return 127;
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u && b != 0x4600001u ? 1 : 0);
  return (uint32_t)max(e, 0);
}
__device__ __forceinline__ float inverse_power(uint32_t e) {
  return __uint_as_float(e >= 254 ? 0x400000u : (254u - e) << 23);
}

// L: lanes per row, 0: a workgroup per row.
template <int OUT, int I, int L, int TAIL>
__global__ __launch_bounds__(I == 2 ? 1024 : 512) void norm_kernel(const NormParams p) {
  __shared__ float part[2][2][16];
  __shared__ float most_y[OUT == kInt8 ? 2 : 1][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int lanes = L ? L : blockDim.x, own = L ? tid % (L ? L : 1) : tid;  // of the row; this thread among them
  const int rows = L ? blockDim.x / (L ? L : 1) : 1;
  int turn = 0;  // (two sets of sums: a wave writes its next row's while others still read this one's)
  for (int64_t row = (int64_t)blockIdx.x * rows + (L ? tid / (L ? L : 1) : 0); row < p.t;
       row += (int64_t)gridDim.x * rows, turn ^= 1) {
    const uint16_t* x = p.x + row * p.ldx;
    const uint16_t* res = p.res ? p.res + row * p.ldr : nullptr;
    Raw xr[I], rr[I];
    float w[I][8], z[I][8];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (i * lanes + own) * 8;
      if (c < p.h) {
        xr[i] = load<TAIL>(x + c, p.h - c, p.h);
        if (res) rr[i] = load<TAIL>(res + c, p.h - c, p.h);
        load_weight<TAIL>(p.w, p.w_f32, c, p.h, w[i]);
      }
    }
    float ss = 0.f, most = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (i * lanes + own) * 8;
      if (c < p.h) {
        widen<TAIL>(xr[i], z[i], p.h - c, p.h);
        if (res) {
          float f[8];
          widen<TAIL>(rr[i], f, p.h - c, p.h);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[i][e] += f[e];
        }
        if (p.sum) store<TAIL>(p.sum + row * p.lds + c, z[i], p.h - c, p.h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = __builtin_fmaf(z[i][e], z[i][e], ss);
          if constexpr (OUT == kInt8) most = fmaxf(most, fabsf(z[i][e] * w[i][e]));
        }
      }
    }
    ss = sum_row<L>(ss);
    if constexpr (OUT == kInt8) most = max_row<L>(most);
    if (L == 0 && waves > 1) {
      if (lane == 0) {
        part[turn][0][wave] = ss;
        if constexpr (OUT == kInt8) part[turn][1][wave] = most;
      }
      __syncthreads();
      ss = part[turn][0][0];
      for (int k = 1; k < waves; ++k) ss += part[turn][0][k];
      if constexpr (OUT == kInt8) {
        most = part[turn][1][0];
        for (int k = 1; k < waves; ++k) most = fmaxf(most, part[turn][1][k]);
      }
    }
    float r = inverse_root(__builtin_fmaf(ss, p.inv_h, p.eps));
    // a row with a NaN, whose sum of squares is not finite, or of zeros without an
    // eps: NaN in y, or NaN scales, so that what is computed from its codes is NaN too
    const bool bad = !(ss < __builtin_inff()) || r == __builtin_inff();
    if (p.rstd && own == 0) p.rstd[row] = r;
    if (OUT == kBf16 && bad) r = __builtin_nanf("");  // (r = 0 would give zeros)
    Factor f{};
    float last = r;  // INT8: y = z w last
    if constexpr (OUT == kInt8) {
      // the largest |z w| times r is the largest |(z w) r|: rounding keeps the order
      float amax = most * r;
      // z w so small or large that fp32 does not hold it to full precision (or a
      // row of zeros), though y may be in range: the largest |y| itself
      if (!(most > 0x1p-100f && most < 0x1p120f)) {
        amax = 0.f;
        last = 1.f;
#pragma unroll
        for (int i = 0; i < I; ++i)
          if ((i * lanes + own) * 8 < p.h)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              z[i][e] = z[i][e] * r * w[i][e];
              w[i][e] = 1.f;
              amax = fmaxf(amax, fabsf(z[i][e]));
            }
        amax = max_row<L>(amax);
        if (L == 0 && waves > 1) {
          if (lane == 0) most_y[turn][wave] = amax;
          __syncthreads();
          for (int k = 0; k < waves; ++k) amax = fmaxf(amax, most_y[turn][k]);
        }
      }
      f = int8_factor(amax);
      if (own == 0) static_cast<float*>(p.s)[row] = bad ? __builtin_nanf("") : f.s;
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (i * lanes + own) * 8;
      const bool in = c < p.h;
      float y[8];
      // (opaque: the compiler would keep z w from above beside z and w, 16 more registers)
      if constexpr (OUT == kInt8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) asm("" : "+v"(w[i][e]));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = !in ? 0.f : OUT == kInt8 ? z[i][e] * w[i][e] * last : z[i][e] * r * w[i][e];
      if constexpr (OUT == kBf16) {
        if (in) store<TAIL>(static_cast<uint16_t*>(p.y) + row * p.ldy + c, y, p.h - c, p.h);
      } else if constexpr (OUT == kInt8) {
        int q[8];
        f.scale(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = (int)__builtin_rintf(y[e]);
        int8_t* out = static_cast<int8_t*>(p.y) + row * p.h + c;
        if (TAIL ? c + 8 <= p.h : in) {
          uint32_t o[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            o[e] = (uint32_t)(q[4 * e] & 0xff) | ((uint32_t)(q[4 * e + 1] & 0xff) << 8) |
                   ((uint32_t)(q[4 * e + 2] & 0xff) << 16) | ((uint32_t)q[4 * e + 3] << 24);
          __builtin_memcpy(out, o, 8);
        } else if (TAIL && in) {
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (c + e < p.h) out[e] = (int8_t)q[e];
        }
      } else {
        // a group of 128 columns is 16 lanes
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
        m = max16(m);
        uint32_t code = 0;
        if constexpr (OUT == kFp8Ue8m0) {
          code = power_of(m);
          const float k = inverse_power(code);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= k;
        } else {
          f = fp8_factor(m);
          f.scale(y);
        }
        if (in) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.h + c) =
              uint2{codec::encode4(y[0], y[1], y[2], y[3]), codec::encode4(y[4], y[5], y[6], y[7])};
          if ((lane & 15) == 0) {
            const int group = c >> 7, groups = p.h >> 7;
            if constexpr (OUT == kFp8Ue8m0) {
              const int bytes = (groups + 3) / 4 * 4;
              uint8_t* at = static_cast<uint8_t*>(p.s) + row * bytes;
              at[group] = bad ? 255 : (uint8_t)code;
              if (group == groups - 1)
                for (int k = groups; k < bytes; ++k) at[k] = 0;
            } else {
              static_cast<float*>(p.s)[row * groups + group] = bad ? __builtin_nanf("") : f.s;
            }
          }
        }
      }
    }
  }
}

// ---- backward ----
//     g = w dy,  dz = r g - z r^3 / H sum(g z) + dsum,  dw = sum over rows of dy z r
// A workgroup walks rows blockIdx.x, + gridDim.x, ...; a thread owns the same
// columns of each, so dw is a sum in its registers, written once to
// partial[workgroup] and summed in workgroup order by a second kernel (no
// atomics: the same inputs give the same bits).
//
// Few rows: dw needs nothing of the rows' sums (r is given), so workgroups of
// their own sum its columns, beside those of the rows and in the same launch,
// reading dy and z again from the caches: no partials, no second kernel.
struct BackwardParams {
  const uint16_t* dy;
  const uint16_t* x;
  const uint16_t* dsum;  // or null
  const void* w;         // or null
  const float* rstd;
  uint16_t* dx;          // or null
  float* partial;        // or null
  float* dw;             // few rows: or null
  int64_t lddy, ldx, ldds, lddx;
  int t, h, w_f32;
  int columns;           // few rows: workgroups that sum columns of dw, the first ones
};

// Few rows: dw's columns are summed beside the rows.  A tile's rows are read by
// one workgroup, so the time grows with them, and dy and z are read twice, while the
// partials' way pays a second launch and their traffic.  GPU time, us, beside : by
// partials, at rows of
//             512         768         1024        1280        1536
//     264  3.6 : 6.3   3.9 : 6.4   4.5 : 6.4   4.6 : 6.4   5.5 : 6.5
//    1161  5.3 : 8.5   6.8 : 9.2   8.3 : 9.7   9.4 : 10.7 10.5 : 11.2
//    2111  6.6 : 10.6  7.9 : 11.2  9.4 : 12.2 10.5 : 12.8 11.6 : 13.6
//    4096  7.1 : 12.1  9.1 : 12.9 11.2 : 13.6 13.2 : 13.9 15.4 : 13.9
//    7168 10.6 : 16.2 14.1 : 15.8 18.1 : 16.6 21.4 : 18.1 24.9 : 19.9
//   10240 15.6 : 14.9 21.1 : 16.9 26.4 : 19.6 31.4 : 21.5 38.1 : 27.0
constexpr int kFewRows = 1536;
constexpr int64_t kFewValues = 11 << 19;
bool few(int t, int h) { return t <= kFewRows && (int64_t)t * h <= kFewValues; }

// dw's columns c0 .. c0 + 31: a wave takes 16 rows at a time (64 columns and 8 rows:
// 517 x 1161 8.4 us for 6.0).  Where H is no multiple of 32 the last tile starts
// early and some columns are summed twice, to the same bits: a tail's code for
// one workgroup cost 517 x 1161 a microsecond, mostly to fetch it.
constexpr int kTileColumns = 32;
template <int TAIL>
__device__ __forceinline__ void sum_columns(const BackwardParams& p, int c0, float (*part)[kTileColumns]) {
  constexpr int LPR = kTileColumns / 8, RPW = 64 / LPR;
  constexpr int U = 6;  // 8 waves have 768 rows in flight at once
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int c = c0 + (lane % LPR) * 8, n = p.h - c;  // (n <= 0: none)
  const int step = waves * RPW;
  float dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.f;
  if (n > 0) {
    for (int r0 = wave * RPW + lane / LPR; r0 < p.t; r0 += step * U) {
      Raw x[U], d[U];
      float r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r0 + u * step;
        x[u] = d[u] = Raw{uint4{0, 0, 0, 0}};
        r[u] = 0.f;
        if (row < p.t) {
          x[u] = load<TAIL>(p.x + row * p.ldx + c, n, p.h);
          d[u] = load<TAIL>(p.dy + row * p.lddy + c, n, p.h);
          r[u] = p.rstd[row];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float z[8], g[8];
        widen<TAIL>(x[u], z, n, p.h);
        widen<TAIL>(d[u], g, n, p.h);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = __builtin_fmaf(g[e], z[e] * r[u], dw[e]);
      }
    }
  }
#pragma unroll
  for (int m = LPR; m < 64; m *= 2)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] += __shfl_xor(dw[e], m, 64);
  if (lane < LPR) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[wave][lane * 8 + e] = dw[e];
  }
  __syncthreads();
  if (tid < kTileColumns && c0 + tid < p.h) {
    float v = part[0][tid];
    for (int w = 1; w < waves; ++w) v += part[w][tid];
    p.dw[c0 + tid] = v;
  }
}

template <int I, int L, int TAIL>
__global__ __launch_bounds__(I == 2 ? 1024 : 512) void norm_backward_kernel(const BackwardParams p) {
  __shared__ float part[2][16];
  __shared__ float columns[16][kTileColumns];
  __shared__ float together[L ? 512 : 1][8];  // dw of the rows' lanes
  if ((int)blockIdx.x < p.columns) {
    if (L == 16 && p.h < kTileColumns)
      sum_columns<TAIL>(p, 0, columns);
    else
      sum_columns<kNone>(p, min((int)blockIdx.x * kTileColumns, p.h - kTileColumns), columns);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int group = blockIdx.x - p.columns, groups = gridDim.x - p.columns;
  const int lanes = L ? L : blockDim.x, own = L ? tid % (L ? L : 1) : tid;  // of the row; this thread among them
  const int rows = L ? blockDim.x / (L ? L : 1) : 1;
  float w[I][8], dw[I][8];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (i * lanes + own) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    if (c < p.h) load_weight<TAIL>(p.w, p.w_f32, c, p.h, w[i]);
  }
  int turn = 0;
  for (int64_t row = (int64_t)group * rows + (L ? tid / (L ? L : 1) : 0); row < p.t;
       row += (int64_t)groups * rows, turn ^= 1) {
    float z[I][8], d[I][8];
    Raw xr[I], dr[I], ds[I];
    const float r = p.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (i * lanes + own) * 8;
      if (c < p.h) {
        xr[i] = load<TAIL>(p.x + row * p.ldx + c, p.h - c, p.h);
        dr[i] = load<TAIL>(p.dy + row * p.lddy + c, p.h - c, p.h);
        if (p.dsum) ds[i] = load<TAIL>(p.dsum + row * p.ldds + c, p.h - c, p.h);
      }
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (i * lanes + own) * 8;
      if (c < p.h) {
        widen<TAIL>(xr[i], z[i], p.h - c, p.h);
        widen<TAIL>(dr[i], d[i], p.h - c, p.h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = z[i][e] * r;
          dw[i][e] = __builtin_fmaf(d[i][e], n, dw[i][e]);
          d[i][e] *= w[i][e];
          z[i][e] = n;
          dot = __builtin_fmaf(d[i][e], n, dot);
        }
      }
    }
    if (!p.dx) continue;  // (for dw alone; uniform over the workgroup)
    dot = sum_row<L>(dot);
    if (L == 0 && waves > 1) {
      // (two sets: a wave writes its next row's while others still read this one's)
      if (lane == 0) part[turn][wave] = dot;
      __syncthreads();
      dot = part[turn][0];
      for (int k = 1; k < waves; ++k) dot += part[turn][k];
    }
    const float mean = dot / (float)p.h;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (i * lanes + own) * 8;
      if (c < p.h) {
        float o[8], f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = r * __builtin_fmaf(-z[i][e], mean, d[i][e]);
        if (p.dsum) {
          widen<TAIL>(ds[i], f, p.h - c, p.h);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += f[e];
        }
        store<TAIL>(p.dx + row * p.lddx + c, o, p.h - c, p.h);
      }
    }
  }
  if (L && p.partial) {
    // the workgroup's rows, in order
    if constexpr (L != 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) together[tid][e] = dw[0][e];
      __syncthreads();
      if (tid < p.h) {
        float v = 0.f;
        for (int g = 0; g < rows; ++g) v += together[g * L + tid / 8][tid % 8];
        p.partial[(int64_t)group * p.h + tid] = v;
      }
    }
  } else if (p.partial) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (i * lanes + own) * 8;
      if (c < p.h) {
        float* q = p.partial + (int64_t)group * p.h + c;
        if (!TAIL || c + 8 <= p.h) {
          __builtin_memcpy(q, dw[i], 32);
        } else {
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (c + e < p.h) q[e] = dw[i][e];
        }
      }
    }
  }
}

// dw of columns C b .. C b + C - 1: 1024 / C slices of the partials, summed in order.
template <int C>
__global__ __launch_bounds__(1024) void norm_weight_sum_kernel(const float* partial, float* dw, int parts, int h) {
  constexpr int kSlices = 1024 / C;
  __shared__ float sum[kSlices][C];
  const int x = threadIdx.x % C, slice = threadIdx.x / C;
  const int c = blockIdx.x * C + x, per = (parts + kSlices - 1) / kSlices;
  float v = 0.f;
  if (c < h) {
#pragma unroll 16
    for (int k = slice * per; k < min(parts, (slice + 1) * per); ++k) v += partial[(int64_t)k * h + c];
  }
  sum[slice][x] = v;
  __syncthreads();
  if (slice == 0 && c < h) {
    v = sum[0][x];
#pragma unroll
    for (int k = 1; k < kSlices; ++k) v += sum[k][x];
    dw[c] = v;
  }
}

// ---- host ----
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Lanes per row (L), or pieces per thread (I) and waves (W) of a row of h columns.
// Two pieces keep twice as much in flight as one (8192 x 7168 into INT8: 101 us with
// one, 85 with two) and let up to 16 waves hold any row; four in 8 waves are
// slower (8192 x 12288 into FP8: 205 us with four, 130 with two; backward 166 and 151).
struct Shape {
  int pieces, waves, lanes;
};
Shape shape_of(int h) {
  if (h <= 512) return Shape{1, 4, h <= 128 ? 16 : h <= 256 ? 32 : 64};
  const int units = ceil_div(h, 512);  // columns of a wave's piece
  const int pieces = units <= 8 ? 1 : 2;
  return Shape{pieces, ceil_div(units, pieces), 0};
}

// (a launch holds fewer than 2^32 threads: more rows than that go several to a workgroup)
constexpr int kMostGroups = 1 << 21;

template <int OUT, int I, int L>
hipError_t launch_norm(const NormParams& p, int waves, hipStream_t stream) {
  const int groups = ceil_div(p.t, L ? 64 * waves / (L ? L : 1) : 1);
  const int grid = groups < kMostGroups ? groups : kMostGroups;
  constexpr bool kAny = OUT == kBf16 || OUT == kInt8;  // (FP8's rows are whole groups of 128)
  if (kAny && L == 16 && p.h < 8)
    norm_kernel<OUT, I, L, kAny && L == 16 ? kShort : kNone><<<grid, 64 * waves, 0, stream>>>(p);
  else if (kAny && p.h % 8)
    norm_kernel<OUT, I, L, kAny ? kTail : kNone><<<grid, 64 * waves, 0, stream>>>(p);
  else
    norm_kernel<OUT, I, L, kNone><<<grid, 64 * waves, 0, stream>>>(p);
  return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const NormParams& p, hipStream_t stream) {
  const Shape s = shape_of(p.h);
  if (s.lanes == 16) return launch_norm<OUT, 1, 16>(p, s.waves, stream);
  if (s.lanes == 32) return launch_norm<OUT, 1, 32>(p, s.waves, stream);
  if (s.lanes == 64) return launch_norm<OUT, 1, 64>(p, s.waves, stream);
  if (s.pieces == 1) return launch_norm<OUT, 1, 0>(p, s.waves, stream);
  return launch_norm<OUT, 2, 0>(p, s.waves, stream);
}

template <int I, int L>
hipError_t launch_backward(const BackwardParams& p, int grid, int waves, hipStream_t stream) {
  if (L == 16 && p.h < 8)
    norm_backward_kernel<I, L, L == 16 ? kShort : kNone><<<grid, 64 * waves, 0, stream>>>(p);
  else if (p.h % 8)
    norm_backward_kernel<I, L, kTail><<<grid, 64 * waves, 0, stream>>>(p);
  else
    norm_backward_kernel<I, L, kNone><<<grid, 64 * waves, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_rows(const BackwardParams& p, const Shape& s, int grid, hipStream_t stream) {
  if (s.lanes == 16) return launch_backward<1, 16>(p, grid, 8, stream);
  if (s.lanes == 32) return launch_backward<1, 32>(p, grid, 8, stream);
  if (s.lanes == 64) return launch_backward<1, 64>(p, grid, 8, stream);
  if (s.pieces == 1) return launch_backward<1, 0>(p, grid, s.waves, stream);
  return launch_backward<2, 0>(p, grid, s.waves, stream);
}

bool bad_weight(const void* w, int type) { return w && type != DG_TYPE_BF16 && type != DG_TYPE_F32; }
bool unfit_weight(const void* w, int type) { return w && !aligned(w, type == DG_TYPE_F32 ? 4 : 2); }
bool unfit_rows(const void* p, int64_t ld) { return !aligned(p, 2) || ld > kMaxLd; }

// Checks `in` and fills `p`.
dg_status make_norm(const dg_norm* in, int t, int h, NormParams* p) {
  if (!in || !in->x || t <= 0 || h <= 0 || in->ld_x < h || !(in->eps >= 0.f) || in->eps > 3.4e38f)
    return DG_ERROR_INVALID_VALUE;
  if ((in->residual && in->ld_residual < h) || (in->sum && in->ld_sum < h) || bad_weight(in->weight, in->weight_type))
    return DG_ERROR_INVALID_VALUE;
  if (h > kMaxHidden || unfit_rows(in->x, in->ld_x) || (in->residual && unfit_rows(in->residual, in->ld_residual)) ||
      (in->sum && unfit_rows(in->sum, in->ld_sum)) || unfit_weight(in->weight, in->weight_type) || !aligned(in->rstd, 4))
    return DG_ERROR_UNSUPPORTED;
  *p = NormParams{};
  p->x = static_cast<const uint16_t*>(in->x);
  p->res = static_cast<const uint16_t*>(in->residual);
  p->w = in->weight;
  p->w_f32 = in->weight_type == DG_TYPE_F32;
  p->sum = static_cast<uint16_t*>(in->sum);
  p->rstd = in->rstd;
  p->ldx = in->ld_x;
  p->ldr = in->ld_residual;
  p->lds = in->ld_sum;
  p->t = t;
  p->h = h;
  p->eps = in->eps;
  p->inv_h = 1.f / (float)h;
  return DG_SUCCESS;
}

dg_status fp8(const dg_norm* in, void* q, void* s, int t, int h, bool ue8m0, hipStream_t stream) {
  NormParams p;
  const dg_status st = make_norm(in, t, h, &p);
  if (st != DG_SUCCESS) return st;
  if (!q || !s) return DG_ERROR_INVALID_VALUE;
  if (h % 128 != 0 || !aligned(q, 8) || !aligned(s, 4)) return DG_ERROR_UNSUPPORTED;
  p.y = q;
  p.s = s;
  (void)hipGetLastError();  // clear a stale error from unrelated work
  const hipError_t e = ue8m0 ? launch_out<kFp8Ue8m0>(p, stream) : launch_out<kFp8>(p, stream);
  return e == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

// Workgroups of the backward pass.  Each keeps a partial dw of h values, 4 bytes
// written and read again.  As many for each of 256 CUs as give it some 16 waves, and
// no more than it holds at once, since all should end together (two pieces: 2 of 5
// to 8 waves; 8192 x 7168: 90 us with 512, 123 with 585; 16384 x 4096: 99 with 512, 108
// with 768; 16384 x 1024: 39 with 512, 24 with 2048), and above 512 only where each
// still has 8 rows (4096 x 1024: 16 with 2048, 14.6 with 512).
int backward_parts(int t, int h) {
  const Shape s = shape_of(h);
  int each = 2;  // workgroups for a CU
  if (!s.lanes) each = s.waves > 8 ? 1 : s.pieces > 1 ? 2 : 16 / s.waves;
  while (each > 2 && t < 8 * 256 * each) --each;
  return t < 256 * each ? t : 256 * each;
}

// Whether the memory of two matrices' rows may meet.
bool overlap(const void* a, int64_t lda, const void* b, int64_t ldb, int t, int h) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + 2 * ((uintptr_t)(t - 1) * ldb + h) && b0 < a0 + 2 * ((uintptr_t)(t - 1) * lda + h);
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_rmsnorm_bf16(const dg_norm* in, void* y, int64_t ld_y, int tokens, int hidden, hipStream_t stream) {
  NormParams p;
  const dg_status st = make_norm(in, tokens, hidden, &p);
  if (st != DG_SUCCESS) return st;
  if (!y || ld_y < hidden) return DG_ERROR_INVALID_VALUE;
  if (unfit_rows(y, ld_y)) return DG_ERROR_UNSUPPORTED;
  p.y = y;
  p.ldy = ld_y;
  (void)hipGetLastError();
  return launch_out<kBf16>(p, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_rmsnorm_quantize_fp8_1x128(const dg_norm* in, void* q, float* s, int tokens, int hidden,
                                        hipStream_t stream) {
  return fp8(in, q, s, tokens, hidden, false, stream);
}

dg_status dg_rmsnorm_quantize_fp8_1x128_ue8m0(const dg_norm* in, void* q, int32_t* s, int tokens, int hidden,
                                              hipStream_t stream) {
  return fp8(in, q, s, tokens, hidden, true, stream);
}

dg_status dg_rmsnorm_quantize_int8(const dg_norm* in, void* q, float* s, int tokens, int hidden, hipStream_t stream) {
  NormParams p;
  const dg_status st = make_norm(in, tokens, hidden, &p);
  if (st != DG_SUCCESS) return st;
  if (!q || !s) return DG_ERROR_INVALID_VALUE;
  if (!aligned(s, 4)) return DG_ERROR_UNSUPPORTED;
  p.y = q;
  p.s = s;
  (void)hipGetLastError();
  return launch_out<kInt8>(p, stream) == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_rmsnorm_bf16_backward_workspace(int tokens, int hidden, int64_t* bytes) {
  if (!bytes || tokens <= 0 || hidden <= 0) return DG_ERROR_INVALID_VALUE;
  *bytes = few(tokens, hidden) ? 0 : 4 * (int64_t)backward_parts(tokens, hidden) * hidden;
  return DG_SUCCESS;
}

dg_status dg_rmsnorm_bf16_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, const void* weight,
                                   int weight_type, const float* rstd, const void* dsum, int64_t ld_dsum, void* dx,
                                   int64_t ld_dx, float* dweight, void* workspace, int tokens, int hidden,
                                   hipStream_t stream) {
  const int t = tokens, h = hidden;
  if (!dy || !x || !rstd || t <= 0 || h <= 0 || ld_dy < h || ld_x < h || (dx && ld_dx < h) ||
      (dx && dsum && ld_dsum < h) || bad_weight(weight, weight_type) ||
      (dweight && !few(t, h) && !workspace))
    return DG_ERROR_INVALID_VALUE;
  const bool beside = dweight && few(t, h);
  const bool with_dsum = dx && dsum;
  if (h > kMaxHidden || unfit_rows(dy, ld_dy) || unfit_rows(x, ld_x) || (dx && unfit_rows(dx, ld_dx)) ||
      (with_dsum && unfit_rows(dsum, ld_dsum)) || unfit_weight(weight, weight_type) || !aligned(rstd, 4) ||
      !aligned(dweight, 4) || (dweight && !beside && !aligned(workspace, 16)))
    return DG_ERROR_UNSUPPORTED;
  if (!dx && !dweight) return DG_SUCCESS;
  BackwardParams p{};
  p.dy = static_cast<const uint16_t*>(dy);
  p.x = static_cast<const uint16_t*>(x);
  p.dsum = with_dsum ? static_cast<const uint16_t*>(dsum) : nullptr;
  p.w = weight;
  p.w_f32 = weight_type == DG_TYPE_F32;
  p.rstd = rstd;
  p.dx = static_cast<uint16_t*>(dx);
  p.partial = dweight && !beside ? static_cast<float*>(workspace) : nullptr;
  p.dw = beside ? dweight : nullptr;
  p.lddy = ld_dy;
  p.ldx = ld_x;
  p.ldds = ld_dsum;
  p.lddx = ld_dx;
  p.t = t;
  p.h = h;
  Shape s = shape_of(h);
  const int parts = backward_parts(t, h);
  int grid = parts;
  (void)hipGetLastError();
  if (beside) {
    const int columns = ceil_div(h, kTileColumns);
    p.columns = columns;
    if (s.waves < 8) s.waves = 8;  // (the rows' workgroups too, where they share the launch)
    const int rows = !dx ? 0 : s.lanes ? ceil_div(t, 512 / s.lanes) : t;
    grid = columns + rows;
    if (dx && (overlap(dx, ld_dx, dy, ld_dy, t, h) || overlap(dx, ld_dx, x, ld_x, t, h))) {
      // dx over what dw's columns are summed from: those first, in a launch of their own
      if (launch_rows(p, s, columns, stream) != hipSuccess) return DG_ERROR_LAUNCH;
      p.columns = 0;
      grid = rows;
    }
  }
  if (launch_rows(p, s, grid, stream) != hipSuccess) return DG_ERROR_LAUNCH;
  if (p.partial) {
    // (many partials are a long chain for a column: more slices; few: whole lines. In
    // all, with 64 columns and 16: 16384 x 1024, 2048 partials, 31.5 us and 29.9; 1024 x
    // 4096, 512 partials, 13.3 and 14.6)
    if (parts > 512)
      norm_weight_sum_kernel<16><<<ceil_div(h, 16), 1024, 0, stream>>>(p.partial, dweight, parts, h);
    else
      norm_weight_sum_kernel<64><<<ceil_div(h, 64), 1024, 0, stream>>>(p.partial, dweight, parts, h);
    if (hipGetLastError() != hipSuccess) return DG_ERROR_LAUNCH;
  }
  return DG_SUCCESS;
}

}  // extern "C"
