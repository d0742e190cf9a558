// dg_epilogue.h -- the linear layer's epilogue: what it needs (host and
// device), and its device code for four consecutive outputs of one row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dg.h"

namespace dg {

struct Epilogue {
  const void* bias;     // [N] fp32 or bf16, or null
  const uint16_t* res;  // bf16, row stride ldr elements, or null
  uint16_t* pre;        // bf16, row stride ldp elements, or null
  void* out;            // bf16 or fp32, row stride ldc elements
  int64_t ldr, ldp, ldc;
  int bias_f32, out_f32, act;
  int vec;              // 1: rows of out, pre and res start on 4-element boundaries (8 or 16 bytes)
  int vec8;             // 1: the same for 8 elements (16 bytes of bf16), and N is a multiple of 8
};

}  // namespace dg

#if defined(__HIPCC__)
#include "dg_act.h"

namespace dg {
namespace epi {

typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint16_t to_bf16(float x) {
  const __bf16 h = (__bf16)x;  // round to nearest even
  return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ float from_bf16(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint2 pack4(const v4f& v) {
  return uint2{(uint32_t)to_bf16(v[0]) | ((uint32_t)to_bf16(v[1]) << 16),
               (uint32_t)to_bf16(v[2]) | ((uint32_t)to_bf16(v[3]) << 16)};
}
__device__ __forceinline__ v4f unpack4(const uint2& v) {
  return v4f{from_bf16(v.x & 0xffffu), __uint_as_float(v.x & 0xffff0000u), from_bf16(v.y & 0xffffu),
             __uint_as_float(v.y & 0xffff0000u)};
}

// The bias of columns n .. n + 3 (0 past the last column or without a bias).
__device__ __forceinline__ v4f bias4(const Epilogue& e, int n, int cols) {
  v4f b = v4f{0.f, 0.f, 0.f, 0.f};
  if (e.bias) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < cols)
        b[r] = e.bias_f32 ? static_cast<const float*>(e.bias)[n + r]
                          : from_bf16(static_cast<const uint16_t*>(e.bias)[n + r]);
  }
  return b;
}

// Row `m`, columns n .. n + 3 (those below `cols`): v = the product plus
// bias.  Stores pre, applies the activation, adds the residual, stores out.
__device__ __forceinline__ void finish4(const Epilogue& e, int64_t m, int n, int cols, v4f v) {
  const bool whole = e.vec && n + 3 < cols;
  if (e.pre) {
    uint16_t* q = e.pre + m * e.ldp + n;
    if (whole) {
      *reinterpret_cast<uint2*>(q) = pack4(v);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < cols) q[r] = to_bf16(v[r]);
    }
  }
  if (e.act != DG_ACT_NONE) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = act::apply(v[r], e.act);
  }
  if (e.res) {
    const uint16_t* q = e.res + m * e.ldr + n;
    if (whole) {
      v += unpack4(*reinterpret_cast<const uint2*>(q));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < cols) v[r] += from_bf16(q[r]);
    }
  }
  if (e.out_f32) {
    float* q = static_cast<float*>(e.out) + m * e.ldc + n;
    if (whole) {
      *reinterpret_cast<v4f*>(q) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < cols) q[r] = v[r];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(e.out) + m * e.ldc + n;
    if (whole) {
      *reinterpret_cast<uint2*>(q) = pack4(v);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < cols) q[r] = to_bf16(v[r]);
    }
  }
}

}  // namespace epi
}  // namespace dg
#endif
