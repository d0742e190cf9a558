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
#include "dg_bf16.h"

namespace dg {
namespace epi {

using bf16::from_bf16;
using bf16::pack4;
using bf16::to_bf16;
using bf16::unpack4;
using bf16::v4f;

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
  act::apply<4>(v, e.act);
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

// ---- a wave's tile in whole lines ----
// Eight consecutive outputs of one row, for rows that start on 16-byte
// boundaries (Epilogue::vec8) and 32-bit byte offsets from the tile's first
// row.  `v` is the product, `bias` its columns' bias, `res` the residual's 16
// bytes.  Offsets past the resources' range drop the stores, so every wave
// issues the same number of them.
struct Rows {
  __amdgpu_buffer_rsrc_t out, pre, res;
};
typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i pack8(const float* v) {
  v4i o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = (int)((uint32_t)to_bf16(v[2 * e]) | ((uint32_t)to_bf16(v[2 * e + 1]) << 16));
  return o;
}

// The resources of a tile's rows m0 .. m0 + rows - 1 (rows of n columns).
__device__ __forceinline__ Rows rows_of(const Epilogue& e, int64_t m0, int rows, int n) {
  auto make = [&](const void* p, int64_t ld, int es) {
    const uint8_t* b = static_cast<const uint8_t*>(p) + m0 * ld * es;
    return __builtin_amdgcn_make_buffer_rsrc((void*)b, (short)0, p ? (int)(((rows - 1) * ld + n) * es) : 0, 0x00020000);
  };
  return Rows{make(e.out, e.ldc, e.out_f32 ? 4 : 2), make(e.pre, e.ldp, 2), make(e.res, e.ldr, 2)};
}

__device__ __forceinline__ v4i residual8(const Epilogue& e, const Rows& r, int m, int n, bool in) {
  const uint32_t off = in ? ((uint32_t)m * (uint32_t)e.ldr + (uint32_t)n) * 2u : 0x80000000u;
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r.res, off, 0, 0));
}

// The sums alone, as bf16.
__device__ __forceinline__ void store8(const Epilogue& e, const Rows& r, int m, int n, bool in, const float* v) {
  const uint32_t off = in ? ((uint32_t)m * (uint32_t)e.ldc + (uint32_t)n) * 2u : 0x80000000u;
  __builtin_amdgcn_raw_buffer_store_b128(pack8(v), r.out, off, 0, 0);
}

__device__ __forceinline__ void finish8(const Epilogue& e, const Rows& r, int m, int n, bool in, float* v,
                                        const float* bias, const v4i& res) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += bias[i];
  if (e.pre) {
    const uint32_t off = in ? ((uint32_t)m * (uint32_t)e.ldp + (uint32_t)n) * 2u : 0x80000000u;
    __builtin_amdgcn_raw_buffer_store_b128(pack8(v), r.pre, off, 0, 0);
  }
  act::apply<8>(v, e.act);
  if (e.res) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] += from_bf16((uint32_t)res[i] & 0xffffu);
      v[2 * i + 1] += __uint_as_float((uint32_t)res[i] & 0xffff0000u);
    }
  }
  if (e.out_f32) {
    const uint32_t off = in ? ((uint32_t)m * (uint32_t)e.ldc + (uint32_t)n) * 4u : 0x80000000u;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __builtin_amdgcn_raw_buffer_store_b128(
          __builtin_bit_cast(v4i, v4f{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]}), r.out, off + 16u * h, 0, 0);
  } else {
    const uint32_t off = in ? ((uint32_t)m * (uint32_t)e.ldc + (uint32_t)n) * 2u : 0x80000000u;
    __builtin_amdgcn_raw_buffer_store_b128(pack8(v), r.out, off, 0, 0);
  }
}

}  // namespace epi
}  // namespace dg
#endif
