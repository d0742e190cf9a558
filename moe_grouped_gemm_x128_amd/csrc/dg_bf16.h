// dg_bf16.h -- conversions between fp32, bf16 and fp8 (e4m3) values in
// registers (device code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {
namespace bf16 {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint16_t to_bf16(float x) {
  const __bf16 h = (__bf16)x;  // round to nearest even
  return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ float from_bf16(uint32_t h) { return __uint_as_float(h << 16); }  // (bits above the 16th drop)

__device__ __forceinline__ uint2 pack4(const v4f& v) {
  return uint2{(uint32_t)to_bf16(v[0]) | ((uint32_t)to_bf16(v[1]) << 16),
               (uint32_t)to_bf16(v[2]) | ((uint32_t)to_bf16(v[3]) << 16)};
}
__device__ __forceinline__ v4f unpack4(const uint2& v) {
  return v4f{from_bf16(v.x & 0xffffu), __uint_as_float(v.x & 0xffff0000u), from_bf16(v.y & 0xffffu),
             __uint_as_float(v.y & 0xffff0000u)};
}

// 8 fp8 (e4m3) bytes as 8 bf16 values (exact: every e4m3 value is a bf16 value).
__device__ __forceinline__ v8bf fp8_to_bf16(int lo, int hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

}  // namespace bf16
}  // namespace dg
