// dg_stream.h -- the weight-streaming pipeline of the kernels that multiply
// few rows by large weights (the linear layer for few rows, the few-token MoE
// layer), all bound by reading the weights once.
//
// A wave works alone on a stream of units: two groups A and B of 16 weight rows,
// or the same 16 rows at consecutive lines of K (SAME), and up to 4 tiles of 16
// activation rows.  A unit is 256 bytes of K of the weights; with fp8 weights,
// bf16 activations and groups of different rows 128.  The wave has a private ring of D
// entries in LDS, filled by loads straight to LDS and drained in order, so no
// barrier separates loads from use: an entry is complete when at most the loads
// of the D - 1 younger entries are in flight.  Every entry has the same number
// of loads:
//   weight entry: one 128-byte line of K of each group's 16 rows (4 KB);
//   activation entry: two lines of K of one tile's 16 rows (4 KB);
//   with scales, a 4-byte load of them in either (the lanes that have one).
// Each load instruction covers 8 rows x one whole 128-byte line.  Loading the
// same bytes in the MFMA's own lane order (16 rows x 64 bytes, straight to
// registers) runs at 30 GB/s per CU from the L2 instead of 74 and streams HBM at
// 5.7 instead of 7.0 TB/s: sixteen half lines per 16 lanes keep the address path
// busy four times as long.  In LDS the 16-byte chunk c of row r sits at c ^ swz(r)
// (applied on the global side), so the fragment reads meet no bank twice.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_bf16.h"
#include "dg_dma.h"

namespace dg {
namespace stream {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
using bf16::fp8_to_bf16;
using bf16::from_bf16;
using bf16::pack4;
using bf16::to_bf16;
using bf16::v4f;
using bf16::v8bf;

constexpr uint32_t kOut = 0x80000000u;  // a lane offset past every resource's range: reads zero, touches no memory
constexpr int kMaxTiles = 4;

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

__device__ __forceinline__ v4f mfma_bf16(const v4i& w, const v4i& x, const v4f& acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), acc, 0, 0,
                                                 0);
}
// One block of 128 FP8 products.  The FP8 matrix instructions (this one and the
// 16x16x32 form alike) keep 16 bits or so of a block's sum: 1.5e-5 off in the
// norm, measured, some 2e-5 of the products' sizes for one sum, where bf16's on
// the same values are 1e-8 off.  That is below a bf16 result's own rounding
// unless the products cancel; where the result is fp32 (EXACT) the codes
// are converted, exactly, and multiplied as bf16 (64 x 4096 x 7168: 14.6 us
// against 13.9).
template <bool EXACT>
__device__ __forceinline__ v4f mfma_fp8(const v4i& w0, const v4i& w1, const v4i& x0, const v4i& x1) {
  if constexpr (EXACT) {
    v4f p = v4f{0.f, 0.f, 0.f, 0.f};
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(w0[0], w0[1]), fp8_to_bf16(x0[0], x0[1]), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(w0[2], w0[3]), fp8_to_bf16(x0[2], x0[3]), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(w1[0], w1[1]), fp8_to_bf16(x1[0], x1[1]), p, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(w1[2], w1[3]), fp8_to_bf16(x1[2], x1[3]), p, 0, 0, 0);
  }
  const v8i w = v8i{w0[0], w0[1], w0[2], w0[3], w1[0], w1[1], w1[2], w1[3]};
  const v8i x = v8i{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Operand types: bf16 by bf16; fp8 weights with bf16 activations; fp8 by fp8.
enum Mode : int { kBf16 = 0, kW8A16 = 1, kFp8 = 2 };

constexpr int entry_bytes(int mode) { return 4096 + (mode == kBf16 ? 0 : mode == kW8A16 ? 16 : 128); }
constexpr int ring_bytes(int mode, int waves, int depth) { return waves * depth * entry_bytes(mode); }

// The unit a cursor stands on, as wave-uniform values; Cursor adds
//   uint32_t row(int tile, int r): this lane's byte offset of activation row r
//     of a tile from `x`, or kOut;
//   uint32_t scale(int tile): fp8 by fp8: the lane's byte offset into `xs`;
//   void next(): the following unit (or !live).
struct Unit {
  bool live;
  int tiles;            // activation tiles
  const uint8_t* wa;    // group A's first row at the unit's K
  const uint8_t* wb;
  int ra, rb;           // rows of A and B that exist
  uint32_t wrow;        // bytes between weight rows
  const uint8_t* x;     // the activations at the unit's K
  uint32_t xrange;      // bytes from x to the end of the last activation row's unit
  int kbytes;           // bytes of K left in a weight row from here (lines past them read nothing)
  int xbytes;           // the same of an activation row
  const float* s;       // scales: group g's for the first line of K at byte so[g]; kFp8: the second line's after it
  uint32_t so[2], srange;
  const float* xs;      // kFp8: activation scales at the unit's K
  uint32_t xsrange;
};

// PARTIAL: rows and lines may be cut (the linear layer); otherwise every unit
// has 16 rows in both groups and whole lines.  EXACT: see mfma_fp8.
template <int MODE, int D, bool PARTIAL, bool SAME, class Cursor, bool EXACT = false>
struct Pipe {
  static constexpr int kEntry = entry_bytes(MODE);
  static constexpr int kLoads = MODE == kBf16 ? 4 : 5;
  static constexpr int WE = SAME || MODE == kW8A16 ? 1 : 2;  // weight entries per unit
  static constexpr int XE = SAME && MODE == kW8A16 ? 2 : 1;  // activation entries per tile
  static_assert((D - 1) * kLoads < 64, "vmcnt range");

  uint32_t ring;       // LDS address
  Cursor ic;           // the unit being loaded
  int phase = 0;       // its next entry
  int islot = 0, cslot = 0;
  int lane, lrow;      // the lane's row (of 8) in a load
  uint32_t xc[2], wv[2];  // its chunk's byte in a line, and its offset in the weights, for the two loads of 16 rows
  uint32_t o[4];       // LDS offsets of chunks lq, lq + 4, 2 lq, 2 lq + 1 of row l16

  __device__ __forceinline__ void init(uint32_t lds, const Cursor& c, int lane_) {
    ring = lds;
    ic = c;
    lane = lane_;
    lrow = lane >> 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      xc[j] = (uint32_t)(((lane & 7) ^ swz(8 * j + lrow)) << 4);
      wv[j] = (uint32_t)(8 * j + lrow) * ic.u.wrow + xc[j];
    }
    const int l16 = lane & 15, lq = lane >> 4, s = swz(l16);
    o[0] = (uint32_t)(l16 * 128 + ((lq ^ s) << 4));
    o[1] = (uint32_t)(l16 * 128 + (((lq + 4) ^ s) << 4));
    o[2] = (uint32_t)(l16 * 128 + (((2 * lq) ^ s) << 4));
    o[3] = (uint32_t)(l16 * 128 + (((2 * lq + 1) ^ s) << 4));
#pragma unroll
    for (int d = 0; d < D; ++d) issue();
  }

  // The loads of the next entry, into the ring's next slot.
  __device__ __forceinline__ void issue() {
    const uint32_t lds = uniform(ring + islot * kEntry);
    islot = islot + 1 == D ? 0 : islot + 1;
    const Unit& u = ic.u;
    if (phase < WE || !u.live) {
      // one line of K of 16 rows of A and 16 of B, or two lines of A's
      const int koff = !SAME && u.live ? 128 * phase : 0;
      const int left = u.live ? (PARTIAL || SAME ? u.kbytes - koff : 128) : 0;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int rows = PARTIAL ? (g && !SAME ? u.rb : u.ra) : 16;
        const int lg = SAME ? left - 128 * g : left;
        const dma::v4i r = dma::resource(SAME ? u.wa + 128 * g : (g ? u.wb : u.wa) + koff,
                                         lg > 0 && rows > 0 ? (uint32_t)(rows - 1) * u.wrow + min(lg, 128) : 0u);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          dma::load16_nt(lds + (2 * g + j) * 1024, r, !PARTIAL || (int)xc[j] < lg ? wv[j] : kOut);
      }
      if constexpr (MODE != kBf16) {
        // lane 0: A's scale, lane 1: B's
        const uint32_t so = (lane ? u.so[1] : u.so[0]) + (MODE == kFp8 && !SAME ? 4u * phase : 0u);
        const dma::v4i r = dma::resource(u.s, left > 0 ? u.srange : 0u);
        if (lane < 2) dma::load4(lds + 4096, r, so);
      }
    } else {
      const int t = (phase - WE) / XE;
      const int kx = 256 * ((phase - WE) % XE);
      const uint32_t off[2] = {ic.row(t, lrow), ic.row(t, 8 + lrow)};
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        const int at = kx + 128 * l;  // byte of the unit's K
        const bool part = PARTIAL || SAME;
        const dma::v4i r = dma::resource(u.x + at, !part || (int)u.xrange > at ? u.xrange - at : 0u);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          dma::load16(lds + (2 * l + j) * 1024, r, !part || at + (int)xc[j] < u.xbytes ? off[j] + xc[j] : kOut);
      }
      if constexpr (MODE != kBf16) {
        if constexpr (MODE == kFp8) {
          const dma::v4i r = dma::resource(u.xs, u.xsrange);
          const uint32_t so = ic.scale(t);
          if (lane < 32) dma::load4(lds + 4096, r, so);
        } else {
          const dma::v4i r = dma::resource(u.x, 0u);  // none: reads nothing
          if (lane < 2) dma::load4(lds + 4096, r, 0u);
        }
      }
    }
    if (u.live && ++phase == WE + XE * u.tiles) {
      phase = 0;
      ic.next();
    }
  }

  typedef __attribute__((address_space(3))) const v4i* lv;
  typedef __attribute__((address_space(3))) const float* lf;

  // The next entry to use, landed: `held` entries before it are still unreleased.
  template <int HELD>
  __device__ __forceinline__ uint32_t arrive() {
    static_assert(HELD < D, "the ring holds the unit's entries");
    const uint32_t lds = ring + cslot * kEntry;
    cslot = cslot + 1 == D ? 0 : cslot + 1;
    dma::wait<(D - 1 - HELD) * kLoads>();
    return lds;
  }
  // The LDS reads of N entries are done: their slots are loaded anew.
  template <int N>
  __device__ __forceinline__ void release() {
    dma::lds_done();
#pragma unroll
    for (int i = 0; i < N; ++i) issue();
  }

  // One unit of `tiles` tiles into the sums of A and B (tile t's lanes: column
  // l16, rows 4 lq .. 4 lq + 3 of the group; SAME: two parts of one sum).  The
  // last weight entry and the first activation entry are read together: one
  // LDS latency for both.
  template <int NT>
  __device__ __forceinline__ void unit(int tiles, v4f* a, v4f* b) {
    v4i w[2][WE][2];  // [group][entry][chunk lq, lq + 4]
    float s[2][WE];
#pragma unroll
    for (int e = 0; e < WE; ++e) {
      const uint32_t lds = arrive<0>();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int j = 0; j < 2; ++j) w[g][e][j] = *(lv)(uintptr_t)(lds + 2048 * g + o[j]);
        s[g][e] = MODE != kBf16 ? *(lf)(uintptr_t)(lds + 4096 + 4 * g) : 1.f;
      }
      if (e + 1 < WE) release<1>();
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t > 0 && t >= tiles) break;
#pragma unroll
      for (int xe = 0; xe < XE; ++xe) {
        const bool held = t == 0 && xe == 0;  // with the weights
        const uint32_t lds = held ? arrive<1>() : arrive<0>();
        v4i x[2][2];
        float xs[2];
#pragma unroll
        for (int l = 0; l < 2; ++l) {
#pragma unroll
          for (int j = 0; j < 2; ++j) x[l][j] = *(lv)(uintptr_t)(lds + 2048 * l + o[(MODE == kW8A16 ? 2 : 0) + j]);
          xs[l] = MODE == kFp8 ? *(lf)(uintptr_t)(lds + 4096 + 4 * (16 * l + (lane & 15))) : 1.f;
        }
        if (held) release<2>(); else release<1>();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          v4f& acc = g ? b[t] : a[t];
          if constexpr (MODE == kBf16) {
            // group g by every line of the unit, or (SAME) its own
#pragma unroll
            for (int l = 0; l < 2; ++l)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (!SAME || l == g) acc = mfma_bf16(w[g][SAME ? 0 : l][j], x[l][j], acc);
          } else if constexpr (MODE == kW8A16) {
            if (SAME && xe != g) continue;
            v4f p = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              p = mfma_bf16(__builtin_bit_cast(v4i, fp8_to_bf16(w[g][0][j][0], w[g][0][j][1])), x[j][0], p);
              p = mfma_bf16(__builtin_bit_cast(v4i, fp8_to_bf16(w[g][0][j][2], w[g][0][j][3])), x[j][1], p);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(s[g][0], p[r], acc[r]);
          } else {
#pragma unroll
            for (int l = 0; l < 2; ++l) {
              if (SAME && l != g) continue;
              const int e = SAME ? 0 : l;
              const v4f p = mfma_fp8<EXACT>(w[g][e][0], w[g][e][1], x[l][0], x[l][1]);
              const float f = s[g][e] * xs[l];
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(f, p[r], acc[r]);
            }
          }
        }
      }
    }
  }
};

}  // namespace stream
}  // namespace dg
