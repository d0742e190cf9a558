// recording_stubs.h -- test infrastructure for the host code of the GEMMs and
// the linear layer on a machine without a GPU: the HIP runtime calls that it
// makes and the library's kernel launches, replaced by functions that write
// down what they were asked to do.  Addresses are made up and never read.
#pragma once

#include <stdint.h>
#include <unistd.h>

#include <mutex>
#include <vector>

#include "../../moe_grouped_gemm_x128_amd/csrc/dg_linear.h"

namespace rec {

enum What { ALLOC, FREE, SPLIT_GEMM, REDUCE };
struct Op {
  What what;
  uintptr_t stream;
  const void* ptr;
};

inline std::mutex g_mutex;
inline std::vector<Op> g_ops;
inline uintptr_t g_next = 0x100000000;  // the next made-up device address
inline int g_cus = 256;
inline int g_pause_us = 0;  // inside a launch: time for another thread to come between

inline void note(What w, hipStream_t s, const void* p) {
  std::lock_guard<std::mutex> l(g_mutex);
  g_ops.push_back(Op{w, reinterpret_cast<uintptr_t>(s), p});
}
inline void pause() {
  if (g_pause_us) usleep(g_pause_us);
}

// What a driver checks of the launches: it defines these.
void seen_gemm(int layout, int tile, const dg::GemmParams& p, int grid);
void seen_pair(int tile, const dg::GemmParams& nn, const dg::GemmParams& tn, int first, int grid, int chunks);
void seen_rows(const dg::RowsParams& p);
void seen_dact(const dg::DactParams& p);
void seen_fp8(int kind, const dg::TileShape& s, const dg::Params& p, int grid);
inline std::vector<int> g_grids;  // of the kernels launched by name (hipLaunchKernel)

}  // namespace rec

extern "C" {
// (kernel<<<grid, block>>>: push, then the kernel's host function pops and launches)
static thread_local dim3 rec_grid, rec_block;
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
  rec_grid = grid;
  rec_block = block;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = rec_grid;
  *block = rec_block;
  *shared = 0;
  *stream = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3, void**, size_t, hipStream_t) {
  rec::g_grids.push_back((int)(grid.x * grid.y * grid.z));
  return hipSuccess;
}
hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = rec::g_cus;
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipMemPoolCreate(hipMemPool_t* pool, const hipMemPoolProps*) {
  *pool = reinterpret_cast<hipMemPool_t>(uintptr_t(0x1000));
  return hipSuccess;
}
hipError_t hipMemPoolSetAttribute(hipMemPool_t, hipMemPoolAttr, void*) { return hipSuccess; }
hipError_t hipMallocFromPoolAsync(void** p, size_t bytes, hipMemPool_t, hipStream_t s) {
  {
    std::lock_guard<std::mutex> l(rec::g_mutex);
    *p = reinterpret_cast<void*>(rec::g_next);
    rec::g_next += (bytes + 4095) / 4096 * 4096 + 4096;
  }
  rec::note(rec::ALLOC, s, *p);
  return hipSuccess;
}
hipError_t hipFreeAsync(void* p, hipStream_t s) {
  rec::note(rec::FREE, s, p);
  return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* c) {
  *c = hipStreamCaptureStatusNone;
  return hipSuccess;
}
}

namespace dg {

hipError_t launch(int kind, const TileShape& shape, const Params& p, int grid, hipStream_t s) {
  rec::pause();
  rec::seen_fp8(kind, shape, p, grid);
  if (p.splits > 1) rec::note(rec::SPLIT_GEMM, s, p.ws);
  return hipSuccess;
}
hipError_t launch_splitk_reduce(int, const Params& p, hipStream_t s) {
  rec::pause();
  rec::note(rec::REDUCE, s, p.ws);
  return hipSuccess;
}
hipError_t launch_splitk_linear(const Epilogue&, const float* ws, int64_t, int, int, int, hipStream_t s) {
  rec::pause();
  rec::note(rec::REDUCE, s, ws);
  return hipSuccess;
}
hipError_t launch_gemm(int layout, int tile, const GemmParams& p, int grid, hipStream_t s) {
  rec::pause();
  rec::seen_gemm(layout, tile, p, grid);
  if (p.splits > 1) rec::note(rec::SPLIT_GEMM, s, p.ws);
  return hipSuccess;
}
hipError_t launch_gemm_pair(int tile, const GemmParams& nn, const GemmParams& tn, int first, int grid, const float*,
                            float*, int chunks, hipStream_t) {
  rec::seen_pair(tile, nn, tn, first, grid, chunks);
  return hipSuccess;
}
hipError_t launch_linear_rows(bool, const RowsParams& p, int, hipStream_t) {
  rec::seen_rows(p);
  return hipSuccess;
}
hipError_t launch_dact(const DactParams& p, hipStream_t) {
  rec::seen_dact(p);
  return hipSuccess;
}
hipError_t launch_bias_sum(const float*, float*, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_swiglu_quantize(const uint16_t*, uint8_t*, float*, int, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize(int, const float*, uint8_t*, float*, int, int, int, hipStream_t) { return hipSuccess; }

}  // namespace dg
