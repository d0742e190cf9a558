// dg_moe_rows.hip -- tokens sorted by expert and back (include/dg.h): the rows
// of the grouped layouts that the tokens' experts take, the copies of the tokens
// there, the weighted sum back, and its gradients.
//
// A slot (t, j) is token t's j-th expert; slots are numbered t * top_k + j.  All
// of it is moving rows, bound by HBM; sums are fp32 in the order of a token's
// slots, and nothing is added by atomics whose order could change a result.
#include "dg_bf16.h"
#include "dg_kernel.h"

namespace dg {
namespace {

using bf16::from_bf16;
using bf16::to_bf16;

constexpr int kMaxTopK = 16;
constexpr int kMaxExperts = 1024;
constexpr int kSegment = 128;         // rows that an expert's segment is a multiple of
constexpr int kMaxSlots = 1 << 23;
constexpr int kMaxHidden = 1 << 20;

// ---- sort: the row of every slot ----
// Stable counting sort.  Slots go in chunks, a workgroup each; a wave owns a run
// of its chunk, 64 slots a round.  Lanes of a wave with the same expert find each
// other by ballots over the bits of the expert's number, so a slot's rank is the
// count of its expert in the chunks before, the waves before, the wave's rounds
// before and the lanes before -- slots of an expert keep their order, whatever
// runs first.  What bounds it is the chain of those steps, not their work: chunks
// are one round long where there are few, and up to kCountedHere slots every
// workgroup counts all of them itself, instead of a launch before it (2048 x 8
// slots, 64 experts: 9.8 us with that launch and two rounds).
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kMaxChunks = 256;
constexpr int kCountedHere = 16384;

struct SortParams {
  const int32_t* ids;
  int32_t* m_indices;  // contiguous layout
  int32_t* rows;
  int32_t* counts;     // rows of each expert, or null
  int32_t* hist;       // [chunks][experts], counted by sort_count_kernel, or null: counted here
  int slots, experts, chunk, chunks;
  int limit;           // contiguous: M_total; masked: M_max
};

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const SortParams p) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * p.chunk, end = min(p.slots, first + p.chunk);
  for (int s = first + threadIdx.x; s < end; s += kSortThreads) {
    const int e = p.ids[s];
    if ((uint32_t)e < (uint32_t)p.experts) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) p.hist[(int64_t)blockIdx.x * p.experts + e] = count[e];
}

// The wave's LDS accesses before come before those after (lanes of a wave run
// in step, and its LDS accesses are done in order: this is for the compiler).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The lanes of the wave whose `e` equals this lane's (bits: of the largest e).
__device__ __forceinline__ uint64_t same_lanes(int e, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((e >> b) & 1);
    m &= (e >> b) & 1 ? set : ~set;
  }
  return m;
}

// ONE: a wave's run is one round.
template <bool MASKED, bool ONE>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const SortParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t before[kSortWaves][kMaxExperts];  // of an expert, in the waves before (and rounds done)
  __shared__ int base[kMaxExperts];                      // row of the chunk's first slot of an expert
  __shared__ int first_row[kMaxExperts], total[kMaxExperts];
  __shared__ int part[2][kSortThreads];
  __shared__ int wave_sum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = p.experts, bits = 32 - __builtin_clz(E);  // (E itself stands for "no expert")
  const int c0 = blockIdx.x * p.chunk, c1 = min(p.slots, c0 + p.chunk);
  const int run = ONE ? 64 : ((p.chunk + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int w0 = c0 + wave * run, w1 = min(c1, w0 + run);
  auto expert = [&](int s) {
    const int id = s < w1 ? p.ids[s] : -1;
    return (uint32_t)id < (uint32_t)E ? id : E;
  };
  int mine = ONE ? expert(w0 + lane) : 0;
  for (int i = tid; i < kSortWaves * (kMaxExperts / 2); i += kSortThreads)
    if ((i % (kMaxExperts / 2)) * 2 < E) reinterpret_cast<uint32_t*>(before)[i] = 0;
  part[0][tid] = part[1][tid] = 0;
  __syncthreads();
  // counts per wave
  uint64_t same = ONE ? same_lanes(mine, bits) : 0;
  if constexpr (ONE) {
    if (mine < E && (same & ((1ull << lane) - 1)) == 0) before[wave][mine] = (uint16_t)__popcll(same);
  } else {
    for (int s = w0; s < w1; s += 64) {
      const int e = expert(s + lane);
      const uint64_t m = same_lanes(e, bits);
      if (e < E && (m & ((1ull << lane) - 1)) == 0) before[wave][e] += (uint16_t)__popcll(m);
      wave_sync();
    }
  }
  // counts of all chunks, and of those before this one
  int per = 1;  // threads per expert, a power of two
  if (p.chunks > 1) {
    if (p.hist) {
      while (per * 2 * E <= kSortThreads) per *= 2;
      const int e = tid / per, k = tid % per;
      int a = 0, b = 0;
      if (e < E) {
#pragma unroll 8
        for (int c = k; c < p.chunks; c += per) {
          const int n = p.hist[(int64_t)c * E + e];
          a += n;
          b += c < (int)blockIdx.x ? n : 0;
        }
      }
      part[0][tid] = a;
      part[1][tid] = b;
    } else {
#pragma unroll 4
      for (int s = tid; s < p.slots; s += kSortThreads) {
        const int id = p.ids[s];
        if ((uint32_t)id < (uint32_t)E) {
          atomicAdd(&part[0][id], 1);
          if (s < c0) atomicAdd(&part[1][id], 1);
        }
      }
    }
  }
  __syncthreads();
  int earlier = 0, all = 0;  // of expert `tid`
  if (tid < E) {
    int n[kSortWaves], sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) n[w] = before[w][tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      before[w][tid] = (uint16_t)sum;
      sum += n[w];
    }
    all = sum;
    if (p.chunks > 1) {
      all = 0;
      for (int k = 0; k < per; ++k) {
        all += part[0][tid * per + k];
        earlier += part[1][tid * per + k];
      }
    }
  }
  // the experts' first rows
  int start;
  if constexpr (MASKED) {
    start = tid < E ? tid * p.limit : 0;
  } else {
    const int padded = tid < E ? (all + kSegment - 1) / kSegment * kSegment : 0;
    int v = padded;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int u = __shfl_up(v, d, 64);
      if (lane >= d) v += u;
    }
    if (lane == 63) wave_sum[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += wave_sum[w];
    start = v - padded;
  }
  if (tid < E) {
    base[tid] = start + earlier;
    first_row[tid] = start;
    total[tid] = all;
    if (p.counts && blockIdx.x == 0)
      p.counts[tid] = MASKED ? min(all, p.limit) : max(0, min(all, p.limit - start));
  }
  __syncthreads();
  // rows of the slots
  auto place = [&](int s, int e, uint64_t m) {
    const int lower = __popcll(m & ((1ull << lane) - 1));
    int row = -1;
    if (e < E) {
      row = base[e] + before[wave][e] + lower;
      if (MASKED ? row >= first_row[e] + p.limit : row >= p.limit) row = -1;
    }
    if constexpr (!ONE) {
      wave_sync();  // (every lane has read its count)
      if (e < E && lower == 0) before[wave][e] += (uint16_t)__popcll(m);
      wave_sync();
    }
    if (s < w1) p.rows[s] = row;
  };
  if constexpr (ONE) {
    place(w0 + lane, mine, same);
  } else {
    for (int s = w0; s < w1; s += 64) {
      const int e = expert(s + lane);
      place(s + lane, e, same_lanes(e, bits));
    }
  }
  if constexpr (!MASKED) {
    // the experts of the rows, a wave per block of 128: the last expert that
    // starts at or before the block is the only one that can have rows in it
    for (int64_t r0 = ((int64_t)blockIdx.x * kSortWaves + wave) * kSegment; r0 < p.limit;
         r0 += (int64_t)p.chunks * kSortWaves * kSegment) {
      int lo = 0, hi = E;  // first_row[lo] <= r0, and first_row[hi] > r0 or hi == E
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first_row[mid] <= r0)
          lo = mid;
        else
          hi = mid;
      }
      const int64_t end = first_row[lo] + total[lo], r = r0 + 2 * lane;
      p.m_indices[r] = r < end ? lo : -1;
      p.m_indices[r + 1] = r + 1 < end ? lo : -1;
    }
  }
}

// ---- 16 bytes per lane ----
// Rows that are gathered are read once, with the nontemporal cache policy (the
// gradients of 4096 x 8 rows of 8 KB: 179 -> 168 us).  Rows that are scattered
// are written with it from 256 MB on, the size of the last cache, which
// would keep none of them for the GEMM that reads them (470 MB: 108 -> 88 us, with
// that GEMM 753 -> 729); fewer are left in the caches (59 MB, with the GEMM: 184 us,
// 197 with the policy).
typedef unsigned v4u __attribute__((ext_vector_type(4)));
constexpr int64_t kLastCache = 256 << 20;

__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }
__device__ __forceinline__ uint4 load16_once(const void* p) {
  const v4u v = __builtin_nontemporal_load(static_cast<const v4u*>(p));
  return uint4{v[0], v[1], v[2], v[3]};
}
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, const uint4& v) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, static_cast<v4u*>(p));
  else
    *static_cast<uint4*>(p) = v;
}

// ---- rows without a token in the segments' last blocks: zeros ----
// (a segment starts on a block of 128 with at least one row: a block whose first
// row is taken belongs to a segment, and its rows of -1 are the padding)
constexpr int kPadRows = 32;  // rows of a block per workgroup
template <bool STREAM>
__device__ void zero_padding(const int32_t* m_indices, int group, int groups, int64_t m, uint8_t* a, int64_t row_bytes,
                             uint8_t* sa, int scale_bytes) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int64_t r0 = (int64_t)group * kPadRows; r0 < m; r0 += (int64_t)groups * kPadRows) {  // (m is a multiple of 128)
    if (m_indices[r0 / kSegment * kSegment] < 0) continue;
    for (int64_t r = r0 + wave; r < r0 + kPadRows; r += waves) {
      if (m_indices[r] >= 0) continue;
      for (int64_t b = lane * 16; b < row_bytes; b += 1024) store16<STREAM>(a + r * row_bytes + b, uint4{0, 0, 0, 0});
      for (int b = lane * 4; b < scale_bytes; b += 256) *reinterpret_cast<uint32_t*>(sa + r * scale_bytes + b) = 0;
    }
  }
}

// ---- dispatch: a[row of slot] = x[token] ----
// A wave takes one KB of a token's row into registers and writes it to each of
// its slots' rows: x is read once.  (Two, four and eight KB per wave are 3 to 6%
// slower at 8192 tokens of 7 KB to 8 rows each, and leave CUs idle at few tokens.)
struct DispatchParams {
  const uint8_t* x;
  const uint8_t* s;   // scales, or null
  const int32_t* rows;
  const int32_t* m_indices;  // or null: padding rows stay as they are
  uint8_t* a;
  uint8_t* sa;
  int64_t ldx, m;     // bytes between x's rows; rows of a
  int tokens, top_k, row_bytes, scale_bytes, pieces, copies;  // pieces: waves per token; copies: workgroups that copy
};

template <bool STREAM>
__global__ __launch_bounds__(256) void dispatch_kernel(const DispatchParams p) {
  if ((int)blockIdx.x >= p.copies) {
    zero_padding<STREAM>(p.m_indices, blockIdx.x - p.copies, gridDim.x - p.copies, p.m, p.a, p.row_bytes, p.sa, p.scale_bytes);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t items = (int64_t)p.tokens * p.pieces;
  for (int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); item < items;
       item += (int64_t)p.copies * 4) {
    const int64_t token = item / p.pieces;
    const int piece = (int)(item - token * p.pieces);
    const uint8_t* x = p.x + token * p.ldx;
    const int at = piece * 1024 + lane * 16;
    const bool in = at < p.row_bytes;
    // (the rows of the token's slots, one per lane)
    const int32_t own = lane < p.top_k ? p.rows[token * p.top_k + lane] : -1;
    uint4 v{0, 0, 0, 0};
    if (in) v = load16(x + at);
    // the first piece's wave moves the scales too, 256 bytes at a time
    const uint8_t* s = p.s + token * p.scale_bytes + lane * 4;
    const int scales = piece == 0 ? p.scale_bytes - lane * 4 : 0;  // bytes from this lane's word on
    uint32_t first = 0;
    if (scales > 0) first = *reinterpret_cast<const uint32_t*>(s);
    for (int j = 0; j < p.top_k; ++j) {
      const int64_t row = __builtin_amdgcn_readlane(own, j);
      if (row < 0 || row >= p.m) continue;
      if (in) store16<STREAM>(p.a + row * p.row_bytes + at, v);
      uint8_t* sa = p.sa + row * p.scale_bytes + lane * 4;
      if (scales > 0) *reinterpret_cast<uint32_t*>(sa) = first;
      for (int b = 256; b < scales; b += 256) *reinterpret_cast<uint32_t*>(sa + b) = *reinterpret_cast<const uint32_t*>(s + b);
    }
  }
}

// ---- combine: y[t] = residual[t] + sum_j w[t, j] o[row of slot (t, j)] ----
// A wave takes 512 columns of a token, 8 per lane.
__device__ __forceinline__ void widen8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = from_bf16(w[e]);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = (uint32_t)to_bf16(f[2 * e]) | ((uint32_t)to_bf16(f[2 * e + 1]) << 16);
  return uint4{o[0], o[1], o[2], o[3]};
}

struct CombineParams {
  const uint16_t* o;
  const int32_t* rows;
  const float* weights;  // or null: ones
  const uint16_t* res;   // or null
  uint16_t* y;
  int64_t ldr, ldy, m;
  int tokens, top_k, h, pieces;
};

__device__ __forceinline__ void combine_piece(const CombineParams& p, int64_t token, int c, int lane) {
  const bool in = c < p.h;
  const int64_t slot = token * p.top_k + lane;
  int own = -1;
  float weight = 0.f;
  if (lane < p.top_k) {
    own = p.rows[slot];
    if (own >= p.m) own = -1;
    weight = p.weights ? p.weights[slot] : 1.f;
  }
  float y[8];
  uint4 r{0, 0, 0, 0};
  if (p.res && in) r = load16(p.res + token * p.ldr + c);
  widen8(r, y);
  for (int j0 = 0; j0 < p.top_k; j0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = __builtin_amdgcn_readlane(own, (j0 + j) & 63);
      v[j] = uint4{0, 0, 0, 0};
      if (row >= 0 && in) v[j] = load16_once(p.o + (int64_t)row * p.h + c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (a slot without a row adds nothing, whatever its weight)
      if (__builtin_amdgcn_readlane(own, (j0 + j) & 63) < 0) continue;
      const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), (j0 + j) & 63));
      float f[8];
      widen8(v[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(w, f[e], y[e]);
    }
  }
  if (in) store16<false>(p.y + token * p.ldy + c, pack8(y));
}

__global__ __launch_bounds__(256) void combine_kernel(const CombineParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t items = (int64_t)p.tokens * p.pieces;
  for (int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); item < items;
       item += (int64_t)gridDim.x * 4)
    combine_piece(p, item / p.pieces, (int)(item % p.pieces) * 512 + lane * 8, lane);
}
// ---- combine's backward pass ----
//     do[row of (t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], o[row of (t, j)]>
// A workgroup takes a token: dy is read once, and the products of its waves'
// columns meet in LDS.
struct CombineBackwardParams {
  const uint16_t* dy;
  const uint16_t* o;     // read if dweights
  const int32_t* rows;
  const float* weights;  // or null: ones
  const int32_t* m_indices;  // or null: padding rows of do stay as they are
  uint16_t* dout;        // or null
  float* dweights;       // or null
  int64_t lddy, m;
  int tokens, top_k, h, copies;  // copies: workgroups that take tokens
};

template <int K, bool STREAM>
__global__ __launch_bounds__(512) void combine_backward_kernel(const CombineBackwardParams p) {
  __shared__ float part[2][8][kMaxTopK];
  if ((int)blockIdx.x >= p.copies) {
    zero_padding<STREAM>(p.m_indices, blockIdx.x - p.copies, gridDim.x - p.copies, p.m, reinterpret_cast<uint8_t*>(p.dout),
                 2 * (int64_t)p.h, nullptr, 0);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  int turn = 0;  // (two sets of sums: a wave writes its next token's while others still read this one's)
  for (int64_t token = blockIdx.x; token < p.tokens; token += p.copies, turn ^= 1) {
    int own = -1;
    float weight = 1.f;
    if (lane < p.top_k) {
      own = p.rows[token * p.top_k + lane];
      if (own >= p.m) own = -1;
      if (p.weights) weight = p.weights[token * p.top_k + lane];
    }
    float dot[K], w[K];
    int row[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      dot[j] = 0.f;
      row[j] = __builtin_amdgcn_readlane(own, j);
      w[j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
    }
    for (int c = tid * 8; c < p.h; c += blockDim.x * 8) {
      float d[8];
      widen8(load16(p.dy + token * p.lddy + c), d);
#pragma unroll
      for (int j0 = 0; j0 < K; j0 += 8) {
        uint4 v[8];
        if (p.dweights) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] = uint4{0, 0, 0, 0};
            if (row[j0 + j] >= 0) v[j] = load16_once(p.o + (int64_t)row[j0 + j] * p.h + c);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (row[j0 + j] < 0) continue;
          if (p.dweights) {
            float f[8];
            widen8(v[j], f);
            // (8 products on their own, then one addition: a chain of H / 4096 + 7, not of 8 H / 4096)
            float piece = d[0] * f[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) piece = __builtin_fmaf(d[e], f[e], piece);
            dot[j0 + j] += piece;
          }
          if (p.dout) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = w[j0 + j] * d[e];
            store16<STREAM>(p.dout + (int64_t)row[j0 + j] * p.h + c, pack8(f));
          }
        }
      }
    }
    if (!p.dweights) continue;  // (uniform over the workgroup)
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j >= p.top_k) break;
      float v = dot[j];
#pragma unroll
      for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d, 64);
      if (lane == 0) part[turn][wave][j] = v;
    }
    __syncthreads();
    if (tid < p.top_k) {
      float v = part[turn][0][tid];
      for (int w = 1; w < waves; ++w) v += part[turn][w][tid];
      p.dweights[token * p.top_k + tid] = v;
    }
  }
}

// ---- host ----
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

void chunks_of(int slots, int* chunk, int* chunks) {
  const int even = ceil_div(slots, kMaxChunks);
  *chunk = even > kSortThreads ? even : kSortThreads;  // at least a round of every wave
  *chunks = ceil_div(slots, *chunk);
}

// Sizes of a routing (0: fine).
dg_status bad_routing(int tokens, int top_k, int experts) {
  if (tokens <= 0 || top_k <= 0 || experts <= 0) return DG_ERROR_INVALID_VALUE;
  if (top_k > kMaxTopK || experts > kMaxExperts || (int64_t)tokens * top_k > kMaxSlots) return DG_ERROR_UNSUPPORTED;
  return DG_SUCCESS;
}

dg_status sort(SortParams p, int tokens, int top_k, bool masked, void* workspace, hipStream_t stream) {
  p.slots = tokens * top_k;
  chunks_of(p.slots, &p.chunk, &p.chunks);
  p.hist = p.slots > kCountedHere ? static_cast<int32_t*>(workspace) : nullptr;
  (void)hipGetLastError();  // clear a stale error from unrelated work
  if (p.hist) {
    sort_count_kernel<<<p.chunks, kSortThreads, 0, stream>>>(p);
    if (hipGetLastError() != hipSuccess) return DG_ERROR_LAUNCH;
  }
  if (p.chunk == kSortThreads)
    masked ? sort_place_kernel<true, true><<<p.chunks, kSortThreads, 0, stream>>>(p)
           : sort_place_kernel<false, true><<<p.chunks, kSortThreads, 0, stream>>>(p);
  else
    masked ? sort_place_kernel<true, false><<<p.chunks, kSortThreads, 0, stream>>>(p)
           : sort_place_kernel<false, false><<<p.chunks, kSortThreads, 0, stream>>>(p);
  return hipGetLastError() == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

// The checks that the calls on rows share.
dg_status bad_rows(const int32_t* rows, int tokens, int top_k, int hidden, int64_t m) {
  if (!rows || tokens <= 0 || top_k <= 0 || hidden <= 0 || m <= 0) return DG_ERROR_INVALID_VALUE;
  if (top_k > kMaxTopK || (int64_t)tokens * top_k > kMaxSlots || hidden > kMaxHidden || m > INT32_MAX || !aligned(rows, 4))
    return DG_ERROR_UNSUPPORTED;
  return DG_SUCCESS;
}

// Workgroups for n pieces of work: one each up to kMostGroups, then several each
// (a launch holds fewer than 2^32 threads).
constexpr int kMostGroups = 1 << 21;
int groups_of(int64_t n) { return n < kMostGroups ? (int)n : kMostGroups; }
int pad_groups(const int32_t* m_indices, int64_t m) { return m_indices ? groups_of(m / kPadRows) : 0; }

// Bytes that the slots' rows are at most.
int64_t written(int tokens, int top_k, int64_t m, int64_t row_bytes) {
  const int64_t slots = (int64_t)tokens * top_k;
  return (slots < m ? slots : m) * row_bytes;
}

dg_status dispatch(DispatchParams p, hipStream_t stream) {
  p.pieces = ceil_div(p.row_bytes, 1024);
  p.copies = groups_of(((int64_t)p.tokens * p.pieces + 3) / 4);
  const int grid = p.copies + pad_groups(p.m_indices, p.m);
  (void)hipGetLastError();
  if (written(p.tokens, p.top_k, p.m, p.row_bytes) >= kLastCache)
    dispatch_kernel<true><<<grid, 256, 0, stream>>>(p);
  else
    dispatch_kernel<false><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError() == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dispatch_fp8(const void* x, const void* s, const int32_t* rows, const int32_t* m_indices, void* a, void* sa,
                       int tokens, int top_k, int hidden, int64_t m, int scale_bytes, hipStream_t stream) {
  if (!x || !s || !a || !sa) return DG_ERROR_INVALID_VALUE;
  const dg_status st = bad_rows(rows, tokens, top_k, hidden, m);
  if (st != DG_SUCCESS) return st;
  if (hidden % 128 != 0 || !aligned(x, 16) || !aligned(a, 16) || !aligned(s, 4) || !aligned(sa, 4) || !aligned(m_indices, 4) ||
      (m_indices && m % kSegment != 0))
    return DG_ERROR_UNSUPPORTED;
  DispatchParams p{};
  p.x = static_cast<const uint8_t*>(x);
  p.s = static_cast<const uint8_t*>(s);
  p.rows = rows;
  p.m_indices = m_indices;
  p.a = static_cast<uint8_t*>(a);
  p.sa = static_cast<uint8_t*>(sa);
  p.ldx = hidden;
  p.m = m;
  p.tokens = tokens;
  p.top_k = top_k;
  p.row_bytes = hidden;
  p.scale_bytes = scale_bytes;
  return dispatch(p, stream);
}

// bf16 rows of `ld` elements that start on 16-byte boundaries
bool unfit_rows(const void* p, int64_t ld, int tokens) {
  return !aligned(p, 16) || (tokens > 1 && ld % 8 != 0) || ld > ((int64_t)1 << 40);
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_moe_sort_workspace(int tokens, int top_k, int num_experts, int64_t* bytes) {
  if (!bytes) return DG_ERROR_INVALID_VALUE;
  const dg_status st = bad_routing(tokens, top_k, num_experts);
  if (st != DG_SUCCESS) return st;
  int chunk, chunks;
  chunks_of(tokens * top_k, &chunk, &chunks);
  *bytes = tokens * top_k > kCountedHere ? 4 * (int64_t)chunks * num_experts : 0;
  return DG_SUCCESS;
}

dg_status dg_moe_sort_contiguous(const int32_t* ids, int32_t* m_indices, int32_t* rows, int32_t* counts,
                                 void* workspace, int tokens, int top_k, int num_experts, int m_total,
                                 hipStream_t stream) {
  if (!ids || !m_indices || !rows || m_total <= 0) return DG_ERROR_INVALID_VALUE;
  int64_t need;
  const dg_status st = dg_moe_sort_workspace(tokens, top_k, num_experts, &need);
  if (st != DG_SUCCESS) return st;
  if (need && !workspace) return DG_ERROR_INVALID_VALUE;
  if (m_total % kSegment != 0 || !aligned(ids, 4) || !aligned(m_indices, 4) || !aligned(rows, 4) || !aligned(counts, 4) ||
      (need && !aligned(workspace, 4)))
    return DG_ERROR_UNSUPPORTED;
  SortParams p{};
  p.ids = ids;
  p.m_indices = m_indices;
  p.rows = rows;
  p.counts = counts;
  p.experts = num_experts;
  p.limit = m_total;
  return sort(p, tokens, top_k, false, workspace, stream);
}

dg_status dg_moe_sort_masked(const int32_t* ids, int32_t* masked_m, int32_t* rows, void* workspace, int tokens,
                             int top_k, int num_experts, int m_max, hipStream_t stream) {
  if (!ids || !masked_m || !rows || m_max <= 0) return DG_ERROR_INVALID_VALUE;
  int64_t need;
  const dg_status st = dg_moe_sort_workspace(tokens, top_k, num_experts, &need);
  if (st != DG_SUCCESS) return st;
  if (need && !workspace) return DG_ERROR_INVALID_VALUE;
  // (a slot past M_max is numbered before it drops out: E M_max + slots in 32 bits)
  if ((int64_t)num_experts * m_max + (int64_t)tokens * top_k > INT32_MAX || !aligned(ids, 4) || !aligned(masked_m, 4) ||
      !aligned(rows, 4) || (need && !aligned(workspace, 4)))
    return DG_ERROR_UNSUPPORTED;
  SortParams p{};
  p.ids = ids;
  p.rows = rows;
  p.counts = masked_m;
  p.experts = num_experts;
  p.limit = m_max;
  return sort(p, tokens, top_k, true, workspace, stream);
}

dg_status dg_moe_dispatch_bf16(const void* x, int64_t ld_x, const int32_t* rows, const int32_t* m_indices, void* a,
                               int tokens, int top_k, int hidden, int64_t m, hipStream_t stream) {
  if (!x || !a || ld_x < hidden) return DG_ERROR_INVALID_VALUE;
  const dg_status st = bad_rows(rows, tokens, top_k, hidden, m);
  if (st != DG_SUCCESS) return st;
  if (hidden % 8 != 0 || unfit_rows(x, ld_x, tokens) || !aligned(a, 16) || !aligned(m_indices, 4) ||
      (m_indices && m % kSegment != 0))
    return DG_ERROR_UNSUPPORTED;
  DispatchParams p{};
  p.x = static_cast<const uint8_t*>(x);
  p.rows = rows;
  p.m_indices = m_indices;
  p.a = static_cast<uint8_t*>(a);
  p.ldx = 2 * ld_x;
  p.m = m;
  p.tokens = tokens;
  p.top_k = top_k;
  p.row_bytes = 2 * hidden;
  return dispatch(p, stream);
}

dg_status dg_moe_dispatch_fp8(const void* x, const float* s, const int32_t* rows, const int32_t* m_indices, void* a,
                              float* sa, int tokens, int top_k, int hidden, int64_t m, hipStream_t stream) {
  return dispatch_fp8(x, s, rows, m_indices, a, sa, tokens, top_k, hidden, m, hidden / 128 * 4, stream);
}

dg_status dg_moe_dispatch_fp8_ue8m0(const void* x, const int32_t* s, const int32_t* rows, const int32_t* m_indices,
                                    void* a, int32_t* sa, int tokens, int top_k, int hidden, int64_t m,
                                    hipStream_t stream) {
  return dispatch_fp8(x, s, rows, m_indices, a, sa, tokens, top_k, hidden, m, (int)(((int64_t)hidden + 511) / 512 * 4),
                      stream);
}

dg_status dg_moe_combine_bf16(const void* o, const int32_t* rows, const float* weights, const void* residual,
                              int64_t ld_residual, void* y, int64_t ld_y, int tokens, int top_k, int hidden, int64_t m,
                              hipStream_t stream) {
  if (!o || !y || ld_y < hidden || (residual && ld_residual < hidden)) return DG_ERROR_INVALID_VALUE;
  const dg_status st = bad_rows(rows, tokens, top_k, hidden, m);
  if (st != DG_SUCCESS) return st;
  if (hidden % 8 != 0 || !aligned(o, 16) || unfit_rows(y, ld_y, tokens) ||
      (residual && unfit_rows(residual, ld_residual, tokens)) || !aligned(weights, 4))
    return DG_ERROR_UNSUPPORTED;
  CombineParams p{};
  p.o = static_cast<const uint16_t*>(o);
  p.rows = rows;
  p.weights = weights;
  p.res = static_cast<const uint16_t*>(residual);
  p.y = static_cast<uint16_t*>(y);
  p.ldr = ld_residual;
  p.ldy = ld_y;
  p.m = m;
  p.tokens = tokens;
  p.top_k = top_k;
  p.h = hidden;
  p.pieces = ceil_div(hidden, 512);
  (void)hipGetLastError();
  combine_kernel<<<groups_of(((int64_t)tokens * p.pieces + 3) / 4), 256, 0, stream>>>(p);
  return hipGetLastError() == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

dg_status dg_moe_combine_bf16_backward(const void* dy, int64_t ld_dy, const void* o, const int32_t* rows,
                                       const float* weights, const int32_t* m_indices, void* dout, float* dweights,
                                       int tokens, int top_k, int hidden, int64_t m, hipStream_t stream) {
  if (!dy || ld_dy < hidden || (dweights && !o)) return DG_ERROR_INVALID_VALUE;
  const dg_status st = bad_rows(rows, tokens, top_k, hidden, m);
  if (st != DG_SUCCESS) return st;
  if (hidden % 8 != 0 || unfit_rows(dy, ld_dy, tokens) || (dweights && !aligned(o, 16)) || !aligned(dout, 16) ||
      !aligned(weights, 4) || !aligned(dweights, 4) || !aligned(m_indices, 4) || (m_indices && m % kSegment != 0))
    return DG_ERROR_UNSUPPORTED;
  if (!dout && !dweights) return DG_SUCCESS;
  CombineBackwardParams p{};
  p.dy = static_cast<const uint16_t*>(dy);
  p.o = static_cast<const uint16_t*>(o);
  p.rows = rows;
  p.weights = weights;
  p.m_indices = dout ? m_indices : nullptr;
  p.dout = static_cast<uint16_t*>(dout);
  p.dweights = dweights;
  p.lddy = ld_dy;
  p.m = m;
  p.tokens = tokens;
  p.top_k = top_k;
  p.h = hidden;
  const int waves = ceil_div(hidden, 512) < 8 ? ceil_div(hidden, 512) : 8;
  p.copies = groups_of(tokens);
  const int grid = p.copies + pad_groups(p.m_indices, m);
  (void)hipGetLastError();
  const bool many = dout && written(tokens, top_k, m, 2 * (int64_t)hidden) >= kLastCache;
  if (top_k <= 8)
    many ? combine_backward_kernel<8, true><<<grid, 64 * waves, 0, stream>>>(p)
         : combine_backward_kernel<8, false><<<grid, 64 * waves, 0, stream>>>(p);
  else
    many ? combine_backward_kernel<16, true><<<grid, 64 * waves, 0, stream>>>(p)
         : combine_backward_kernel<16, false><<<grid, 64 * waves, 0, stream>>>(p);
  return hipGetLastError() == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH;
}

}  // extern "C"
