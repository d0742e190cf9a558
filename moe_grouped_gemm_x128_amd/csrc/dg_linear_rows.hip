// dg_linear_rows.hip -- the linear layer for few rows (M <= 64: decode steps,
// router logits): C = act(A.B^T + bias) + residual, bound by reading B once.
//
// A workgroup owns 32 columns of C (the stream's groups are 16 rows of B each)
// and all rows of A; its waves take units of 256 bytes of K round robin
// (dg_stream.h) and meet once in LDS.  Where 32 columns each would leave half of
// the CUs idle it owns 16 (the groups are two lines of K of the same rows): more
// CUs load, though each loads A once more.  No second kernel and no
// workspace: the split over K is inside the workgroup.
#include "dg_linear.h"
#include "dg_stream.h"

namespace dg {
namespace {

using namespace stream;

// A workgroup's columns n0 .. n0 + 31, K units `kb`, kb + W, ...
struct RowsCursor {
  Unit u;
  const uint8_t* b;   // row n0 of B
  const RowsParams* p;
  int kb, nb, waves, fp8;

  __device__ __forceinline__ void place() {
    u.live = kb < nb;
    if (!u.live) return;
    u.kbytes = u.xbytes = p->k * (fp8 ? 1 : 2) - 256 * kb;
    u.wa = b + (int64_t)256 * kb;
    u.wb = u.wa + 16 * p->ldb;
    u.x = p->a + (int64_t)256 * kb;
    u.xrange = (uint32_t)((p->m - 1) * p->lda) + (uint32_t)min(u.xbytes, 256);
    if (fp8) {
      // (the unit's second line of 128 may lie past the row's last block: its
      // operand bytes and its scales then read zero)
      u.s = p->sb + 2 * kb;
      u.srange = u.kbytes > 128 ? 8 : 4;
      u.xs = p->sa + 2 * kb;
      u.xsrange = (uint32_t)((p->m - 1) * (p->k >> 7)) * 4u + (u.kbytes > 128 ? 8u : 4u);
    }
  }
  __device__ __forceinline__ void next() {
    kb += waves;
    place();
  }
  __device__ __forceinline__ uint32_t row(int t, int r) const {
    const int m = 16 * t + r;
    return m < p->m ? (uint32_t)m * (uint32_t)p->lda : kOut;
  }
  __device__ __forceinline__ uint32_t scale(int t) const {
    const int lane = threadIdx.x & 63, m = 16 * t + (lane & 15);
    return m < p->m && (lane < 16 || u.kbytes > 128) ? ((uint32_t)m * (uint32_t)(p->k >> 7) + (uint32_t)(lane >> 4)) * 4u : kOut;
  }
};

template <int MODE, int NT, bool SAME, bool EXACT, int W, int D>
__global__ __launch_bounds__(W * 64) void linear_rows_kernel(const RowsParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ring_bytes(MODE, W, D)];
  // the waves' sums meet where the ring was
  constexpr int G = SAME ? 1 : 2;  // groups of 16 columns
  static_assert(ring_bytes(MODE, W, D) >= W * G * NT * 1024, "the sums fit the ring");
  v4f(*red)[G * NT][64] = reinterpret_cast<v4f(*)[G * NT][64]>(ring);
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16 * G;

  RowsCursor c{};
  c.p = &p;
  c.fp8 = MODE == kFp8;
  c.b = p.b + (int64_t)n0 * p.ldb;
  c.nb = (p.k * (MODE == kFp8 ? 1 : 2) + 255) >> 8;
  c.waves = W;
  c.kb = wave;
  c.u.tiles = NT;
  c.u.ra = min(16, p.n - n0);
  c.u.rb = min(16, p.n - n0 - 16);
  c.u.so[1] = SAME ? 4 : 0;
  c.u.wrow = (uint32_t)p.ldb;
  RowsParams q = p;
  if constexpr (MODE == kFp8) {
    q.sb = p.sb + (int64_t)(n0 >> 7) * (p.k >> 7);  // the workgroup's columns lie in one block of 128
    c.p = &q;
  }
  c.place();
  const int mine = c.nb > wave ? (c.nb - wave + W - 1) / W : 0;
  // what the epilogue reads, asked for before the stream: its latency is hidden
  const int em = 16 * (wave / G) + l16, en = n0 + 16 * (wave % G) + 4 * lq;  // wave's first group of sums
  const bool mine_out = wave < G * NT && em < p.m && en < p.n;
  v4f bias = v4f{0.f, 0.f, 0.f, 0.f};
  if (mine_out) bias = epi::bias4(p.epi, en, p.n);
  Pipe<MODE, D, true, SAME, RowsCursor, EXACT> pipe;
  pipe.init(dma::lds_addr(ring) + wave * D * entry_bytes(MODE), c, lane);
  v4f a[NT], b[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) a[t] = b[t] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < mine; ++k) pipe.template unit<NT>(NT, a, b);
  dma::wait<0>();   // no load lands in the ring any more
  dma::barrier();   // on any wave
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if constexpr (SAME) {
      red[wave][t][lane] = a[t] + b[t];
    } else {
      red[wave][2 * t][lane] = a[t];
      red[wave][2 * t + 1][lane] = b[t];
    }
  }
  __syncthreads();
  static_assert(G * NT <= W, "one group of sums per wave");
  if (mine_out) {
    v4f v = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w][wave][lane];
    epi::finish4(p.epi, em, en, p.n, v + bias);
  }
}

// Waves and ring entries per wave: 12 of 2 (64 x 4096 x 7168 in FP8 15.2 us against
// 15.5 with 8 of 4, 32 x 8192 x 1024 in BF16 7.0 against 7.4), but where a wave's sums and
// operands need more registers than 12 waves leave it.
template <int MODE, int NT, bool SAME, bool EXACT>
hipError_t launch_columns(const RowsParams& p, hipStream_t stream) {
  constexpr bool wide = MODE == kFp8 && NT == 4 && (EXACT || !SAME);
  constexpr int W = wide ? 8 : 12, D = wide ? 4 : 2, C = SAME ? 16 : 32;
  linear_rows_kernel<MODE, NT, SAME, EXACT, W, D><<<(p.n + C - 1) / C, W * 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <int MODE, int NT, bool EXACT>
hipError_t launch(const RowsParams& p, int cus, hipStream_t stream) {
  if (few_rows_columns(p.n, cus) == 16) return launch_columns<MODE, NT, true, EXACT>(p, stream);
  return launch_columns<MODE, NT, false, EXACT>(p, stream);
}

template <int MODE, bool EXACT>
hipError_t launch_mode(const RowsParams& p, int cus, hipStream_t stream) {
  if (p.m <= 16) return launch<MODE, 1, EXACT>(p, cus, stream);
  if (p.m <= 32) return launch<MODE, 2, EXACT>(p, cus, stream);
  return launch<MODE, 4, EXACT>(p, cus, stream);
}

}  // namespace

hipError_t launch_linear_rows(bool fp8, const RowsParams& p, int num_cus, hipStream_t stream) {
  if (!fp8) return launch_mode<kBf16, false>(p, num_cus, stream);
  return p.epi.out_f32 ? launch_mode<kFp8, true>(p, num_cus, stream) : launch_mode<kFp8, false>(p, num_cus, stream);
}

}  // namespace dg
