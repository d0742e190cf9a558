// dg_stream.h -- device helpers of the weight-streaming kernels (few rows
// against a large weight matrix): wave-uniform buffer resources, streaming
// loads into registers, and the operand fragments of one "unit".
//
// A unit is 16 weight rows x 128 values along K, multiplied by up to 16
// activation rows (one MFMA tile).  Lane l holds bytes [64 i + 16 (l / 16),
// + 16) of weight row l % 16 and the same k of activation row l % 16: which k
// a lane holds does not matter to the product as long as both operands agree,
// and this assignment makes every load 16 bytes per lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {
namespace stream {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr uint32_t kOut = 0x80000000u;  // a lane offset past every resource's range: reads zero, touches no memory
constexpr int kNt = 2;                  // cache policy: nontemporal (data read once)

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Raw buffer resource over [base, base + bytes); bytes must be wave-uniform.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  const uint64_t u = (uint64_t)uniform((uint32_t)b) | ((uint64_t)uniform((uint32_t)(b >> 32)) << 32);
  return __builtin_amdgcn_make_buffer_rsrc((void*)u, (short)0, (int)uniform(bytes), 0x00020000);
}

template <int AUX>
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, AUX));
}

// 8 fp8 (e4m3) bytes as 8 bf16 values (exact: every e4m3 value is a bf16 value).
__device__ __forceinline__ v8bf fp8_to_bf16(int lo, int hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ v4f mfma_bf16(const v8bf& w, const v8bf& x, const v4f& acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, acc, 0, 0, 0);
}

// The product of one unit with one activation tile, from a zero accumulator.
// Weights in fp8: w[0..1], 16 values each; in bf16: w[0..3], 8 values each.
// x[0..3]: 8 bf16 values each.
template <bool FP8W>
__device__ __forceinline__ v4f unit_product(const v4i* w, const v4i* x) {
  v4f p = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (FP8W) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      p = mfma_bf16(fp8_to_bf16(w[i][0], w[i][1]), __builtin_bit_cast(v8bf, x[2 * i]), p);
      p = mfma_bf16(fp8_to_bf16(w[i][2], w[i][3]), __builtin_bit_cast(v8bf, x[2 * i + 1]), p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p = mfma_bf16(__builtin_bit_cast(v8bf, w[i]), __builtin_bit_cast(v8bf, x[i]), p);
  }
  return p;
}

__device__ __forceinline__ uint16_t to_bf16(float x) {
  const __bf16 h = (__bf16)x;  // round to nearest even
  return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ float from_bf16(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ uint2 pack4(const v4f& v) {
  return uint2{(uint32_t)to_bf16(v[0]) | ((uint32_t)to_bf16(v[1]) << 16),
               (uint32_t)to_bf16(v[2]) | ((uint32_t)to_bf16(v[3]) << 16)};
}

}  // namespace stream
}  // namespace dg
