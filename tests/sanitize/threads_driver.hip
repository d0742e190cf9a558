// threads_driver.hip -- split-K calls on one stream from several host threads
// (tests/test_host_threads.py): in the order in which work reaches a stream,
// every split product is followed by its own reduction, and no buffer is given
// back between the two or used after it was.
#include <stdio.h>

#include <atomic>
#include <map>
#include <set>
#include <thread>

#include "recording_stubs.h"

void rec::seen_gemm(int, int, const dg::GemmParams&, int) {}
void rec::seen_pair(int, const dg::GemmParams&, const dg::GemmParams&, int, int, int) {}
void rec::seen_rows(const dg::RowsParams&) {}
void rec::seen_dact(const dg::DactParams&) {}
void rec::seen_fp8(int, const dg::TileShape&, const dg::Params&, int) {}

namespace {

void* const P = reinterpret_cast<void*>(uintptr_t(0x10000));
std::atomic<int> failed_calls{0};

// One thread's calls: forward and backward products of the linear layer and FP8
// products whose K is split, their partials growing from call to call.
void calls(hipStream_t stream, int turn) {
  for (int i = 0; i < 6; ++i) {
    const int n = 256 + 64 * ((i + turn) % 5);
    int bad = 0;
    switch ((i + turn) % 3) {
      case 0:
        bad = dg_gemm_bf16_nt_epilogue(P, 8192, P, 8192, P, n, DG_TYPE_BF16, nullptr, 80 + 16 * i, n, 8192, stream);
        break;
      case 1:
        bad = dg_gemm_bf16_nt_epilogue_backward(P, 16 * n, P, 6000, P, 6000, nullptr, 0, DG_ACT_NONE, P, 6000, nullptr, 0,
                                                nullptr, P, 45, 16 * n, 6000, stream);
        break;
      default:
        bad = dg_gemm_fp8_nt(P, static_cast<const float*>(P), P, static_cast<const float*>(P), P, 64, n, 16384, stream);
    }
    if (bad) ++failed_calls;
  }
}

}  // namespace

int main() {
  int bad = 0;
  rec::g_pause_us = 20;
  for (int round = 0; round < 30; ++round) {  // (at most 64 streams keep a buffer)
    const hipStream_t stream = reinterpret_cast<hipStream_t>(uintptr_t(0x5000 + 16 * round));
    std::thread t[4];
    for (int k = 0; k < 4; ++k) t[k] = std::thread(calls, stream, k);
    for (auto& x : t) x.join();
  }
  struct State {
    const void* product = nullptr;  // its partials wait for their reduction
  };
  std::map<uintptr_t, State> streams;
  std::set<const void*> live;
  int products = 0;
  for (const rec::Op& o : rec::g_ops) {
    State& s = streams[o.stream];
    const char* what = nullptr;
    switch (o.what) {
      case rec::ALLOC: live.insert(o.ptr); break;
      case rec::FREE:
        if (!live.erase(o.ptr)) what = "a buffer given back twice";
        if (s.product == o.ptr) what = "a buffer given back between a product and its reduction";
        break;
      case rec::SPLIT_GEMM:
        ++products;
        if (!live.count(o.ptr)) what = "a product into a buffer that was given back";
        if (s.product) what = "a product before the last one's reduction";
        s.product = o.ptr;
        break;
      case rec::REDUCE:
        if (s.product != o.ptr) what = "a reduction of another product's partials";
        s.product = nullptr;
        break;
    }
    if (what && bad++ < 5) fprintf(stderr, "stream %zx: %s\n", (size_t)o.stream, what);
  }
  if (products < 300) {
    fprintf(stderr, "only %d split products\n", products);
    ++bad;
  }
  bad += failed_calls;
  printf("products=%d bad=%d\n", products, bad);
  return bad != 0;
}
