// dg_linear_tile.h -- GEMM tiles of the linear layer (device code): the forward
// product (NT) with its epilogue, in BF16 and INT8, and the two products of the
// BF16 backward pass, which read an operand with K as its row index (NN, TN)
// where it lies -- no transposed copy is made.
//
// A workgroup owns a BM x BN tile; K goes in blocks of 64 values through a ring
// of S LDS stages filled by loads straight to LDS.  It has WK groups of WM x WN
// waves, each with every WK-th block of K and a share of a stage; their sums meet
// in LDS, where each group takes FM / WK fragment rows of every wave's tile.
// Stored layouts of a block in LDS:
//   K contiguous: [row][64 k], 128-byte rows, 16-byte chunk c of row r at
//     position c ^ swz(r); a fragment is one 16-byte read per lane;
//   transposed:   [k][BX columns], 32-byte unit u of row k at u ^ hsw(k); a
//     fragment is two transposing LDS reads (ds_read_b64_tr_b16: 16 lanes read
//     4 k x 16 columns and each gets the 4 k of its column).
// Both swizzles are applied on the global side of the load (the lane that lands
// on a position fetches the chunk that belongs there) and spread the 64 lanes
// of a fragment read over all banks.
//
// Per block a wave multiplies two halves of 32 k.  The fragments of the next
// half are read between the current half's MFMAs; the one barrier of a block
// sits between the halves, where the last reads of a block's stage and the
// arrival of the next block meet, so MFMAs are queued on both sides of it.
//
// The MFMA takes B rows first and A rows second: a lane holds 4 consecutive
// columns of one row of C.
//
// INT8: a fragment's 16 bytes are 16 values where BF16's are 8, and the INT8
// instruction multiplies twice as many of them in the same time, so everything
// that moves bytes is the BF16 product's of half the K (GemmParams::k counts
// pairs of values); the sums are int32, exact, and become fp32 times the row's
// and the column's scale on their way into the epilogue.
#pragma once

#include <type_traits>

#include "dg_dma.h"
#include "dg_linear.h"

namespace dg {
namespace tile {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kGroupM = 8;  // tile rows per raster group
constexpr uint32_t kOut = 0x80000000u;

__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
// transposed: RB bytes per k (128: 4 units of 32 bytes, and k's parity moves by
// half the banks; 256 and more: 8 units or more, every k starts on bank 0)
template <int RB>
__device__ __forceinline__ int hsw(int k) {
  return RB == 128 ? ((k >> 1) & 1) | (((k >> 3) & 1) << 1) : (k & 3) | (((k >> 3) & 1) << 2);
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ v4f mfma(const v8bf& b, const v8bf& a, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}
__device__ __forceinline__ v4i mfma(const v8bf& b, const v8bf& a, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, b), __builtin_bit_cast(v4i, a), c, 0, 0, 0);
}

// INT8's scales, of A's rows and B's.
struct Scales {
  const float* sa;
  const float* sb;
};

// One operand's share of the tile: BX rows of C (or columns), stored K
// contiguous (TR = false) or transposed.  PAIRS: a half's fragments are chunks
// 2 lq + s instead of lq + 4 s (any order of K that both operands share): no
// bank conflicts, against 22% of the cycles in SQ_LDS_BANK_CONFLICT (INT8; with
// the loads spread 1 to 3% faster).
template <int BX, int WX, int NW, bool TR, bool PAIRS>
struct Operand {
  static constexpr int kBytes = BX * 128;                    // LDS bytes per stage
  static constexpr int kPieces = BX / 8;                     // 1 KB loads per stage
  static constexpr int kQ = kPieces / NW;                    // per wave
  static constexpr int WTX = BX / WX, F = WTX / 16;          // fragments per wave
  static constexpr int RB = BX * 2;                          // transposed: bytes per LDS row
  static constexpr int CPR = BX / 8, RP = 64 / CPR;          // chunks per row, rows per load
  static_assert(kPieces % NW == 0, "the same loads on every wave");
  static_assert(TR ? (NW * RP) % 16 == 0 && BX % 64 == 0 : (NW * 8) % 16 == 0, "swizzle fixed per lane");

  // global side
  uint32_t voff, step;  // this lane's offset in its first piece, bytes between a wave's pieces
  int chunk;            // K contiguous: the lane's 8-value chunk of a block
  // LDS side
  uint32_t off[TR ? F : 2];

  __device__ __forceinline__ void init(int64_t ld, int wave, int lane, int wx) {
    if constexpr (!TR) {
      const int r0 = wave * 8 + (lane >> 3);
      chunk = (lane & 7) ^ swz(r0);
      voff = (uint32_t)r0 * (uint32_t)ld + (uint32_t)chunk * 16u;
      step = (uint32_t)(NW * 8) * (uint32_t)ld;
    } else {
      const int k0 = wave * RP + lane / CPR;
      const int pc = lane % CPR;
      chunk = 0;
      voff = (uint32_t)k0 * (uint32_t)ld + (uint32_t)(((((pc >> 1) ^ hsw<RB>(k0)) << 1) | (pc & 1)) * 16);
      step = (uint32_t)(NW * RP) * (uint32_t)ld;
    }
    const int l16 = lane & 15, lq = lane >> 4;
    if constexpr (!TR) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        off[s] = (uint32_t)((wx * WTX + l16) * 128 + (((PAIRS ? 2 * lq + s : 4 * s + lq) ^ swz(l16)) << 4));
    } else {
      const int h = hsw<RB>(8 * lq + (l16 >> 2));  // the same for all rows that this lane addresses
#pragma unroll
      for (int i = 0; i < F; ++i)
        off[i] = (uint32_t)((8 * lq + (l16 >> 2)) * RB + (((wx * F + i) ^ h) << 5) + ((l16 & 3) << 3));
    }
  }

  // The loads of one block: `left` K values from the block's start to the end
  // of the item (<= 0: nothing is read), `base` the operand at the block's start
  // and the tile's first row, `rows` the tile's rows that exist (TR: stored
  // columns from the tile's first one).  K contiguous: rows are padded with
  // zeros to a multiple of 8 values where K is not one (dpre).
  __device__ __forceinline__ void issue(const uint8_t* base, int64_t ld, int rows, int left, uint32_t lds,
                                        int wave) const {
    const int kv = min(left, 64);
    const bool live = left > 0 && rows > 0;
    const uint32_t bytes = !live ? 0u
                           : TR  ? (uint32_t)(kv - 1) * (uint32_t)ld + 2u * rows
                                 : (uint32_t)(min(rows, BX) - 1) * (uint32_t)ld + 2u * ((kv + 7) & ~7);
    const v4i r = dma::resource(base, bytes);
    const uint32_t v = TR || 8 * chunk < kv ? voff : kOut;
#pragma unroll
    for (int q = 0; q < kQ; ++q) dma::load16(lds + (wave + NW * q) * 1024, r, v + q * step);
  }

  // The same (K contiguous) to be issued one by one.
  struct Block {
    v4i r;
    uint32_t v, lds;
  };
  __device__ __forceinline__ Block block(const uint8_t* base, int64_t ld, int rows, int left, uint32_t lds,
                                         int wave) const {
    const int kv = min(left, 64);
    const uint32_t bytes =
        left > 0 && rows > 0 ? (uint32_t)(min(rows, BX) - 1) * (uint32_t)ld + 2u * ((kv + 7) & ~7) : 0u;
    return Block{dma::resource(base, bytes), 8 * chunk < kv ? voff : kOut, lds + wave * 1024};
  }
  __device__ __forceinline__ void load(const Block& b, int q) const {
    dma::load16(b.lds + NW * q * 1024, b.r, b.v + q * step);
  }

  // Fragment i of half s from the stage at LDS address `lds`.
  __device__ __forceinline__ v8bf frag(uint32_t lds, int i, int s) const {
    // (constant parts added to a pointer: they go into the instruction's offset)
    typedef __attribute__((address_space(3))) uint8_t* lp;
    if constexpr (!TR) {
      const lp at = (lp)(uintptr_t)(lds + off[s]);
      return __builtin_bit_cast(v8bf, *(__attribute__((address_space(3))) const v4i*)(at + i * 2048));
    } else {
      typedef __attribute__((address_space(3))) v4s* lt;
      const lp at = (lp)(uintptr_t)(lds + off[i]);
      const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lt)(at + s * 32 * RB)));
      const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lt)(at + (s * 32 + 4) * RB)));
      return __builtin_bit_cast(v8bf, v4i{lo[0], lo[1], hi[0], hi[1]});
    }
  }
};

// LDS of a workgroup: the ring, and the epilogue's rows where they are its own.
template <int BM, int BN, int WM, int WN, int WK, int S>
constexpr int kLds = WK * (S * (BM + BN) * 128 + (S == 2 && WK == 1 ? WM * WN * 16 * (BN / WN) * 4 : 0));

// The items of one product that workgroup `wg` of `nwg` computes.  `p` is the
// kernel's argument at byte ARG; INT8: with `scales`.  LINES: K is not split and every row of the
// output, pre and residual is whole 16-byte pieces (a form of its own: the two
// epilogues in one kernel cost the K loop some 45 registers).
template <int BM, int BN, int WM, int WN, int WK, int S, bool TA, bool TB, bool LINES, int ARG, bool INT8 = false>
__device__ __forceinline__ void run_items(const GemmParams& p, int wg, int nwg, uint8_t* smem,
                                          const Scales& scales = Scales{}) {
  using Acc = std::conditional_t<INT8, v4i, v4f>;
  constexpr int NW = WM * WN;  // waves of a group
  using OpA = Operand<BM, WM, NW, TA, INT8>;
  using OpB = Operand<BN, WN, NW, TB, INT8>;
  constexpr int FM = OpA::F, FN = OpB::F;
  constexpr int PART = OpA::kBytes + OpB::kBytes;  // a group's share of a stage
  constexpr int STAGE = WK * PART;
  constexpr int FR = FM / WK;  // fragment rows of C that a group finishes
  static_assert(FM % WK == 0, "whole fragment rows per group");
  constexpr int LOADS = OpA::kQ + OpB::kQ;  // per wave and block
  // whole-line epilogue: 16 rows of a wave at a time, fp32, the 16-byte chunk c
  // of row r at c ^ r
  constexpr int RS = OpB::WTX * 4, RC = RS / 16;                        // bytes and chunks per row
  constexpr int LPR = OpB::WTX / 8, RPR = 64 / LPR, ROUNDS = 16 / RPR;  // lanes per row, rows per round
  constexpr int kStores = FR * ROUNDS;                                   // 16-byte bf16 stores of a wave
  constexpr bool kOwnRows = S == 2 && WK == 1;
  constexpr int kBehind = kOwnRows ? S - 1 : S - 2;  // blocks of the next item loaded before the stores
  // LDS that a wave's sums pass through, and (WK > 1) its rows that others finish
  constexpr int kRows = 16 * RS, kGiven = (FM - FR) * FN * 1024;
  static_assert(kOwnRows || (kRows <= PART / NW && kGiven <= PART / NW), "a wave's rows fit its share of the slot");
  static_assert((S - 2) * LOADS + 2 * kStores < 64, "vmcnt range");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = (int)uniform((tid >> 6) % NW), wk = WK == 1 ? 0 : (int)uniform((tid >> 6) / NW);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = dma::lds_addr(smem) + wk * PART;
  OpA oa;
  OpB ob;
  oa.init(p.lda, wave, lane, wm);
  ob.init(p.ldb, wave, lane, wn);

  // ---- work items: (tile, K split); each XCD walks a contiguous run ----
  const int items = p.tiles_m * p.tiles_n * p.splits;
  const int per_xcd = (items + 7) >> 3;
  struct Item {
    bool live;
    int m0, n0, split, k0, k1;
  };
  auto decode = [&](int t) -> Item {
    Item x{false, 0, 0, 0, 0, 0};
    const int L = (t & 7) * per_xcd + (t >> 3);
    if (t >= per_xcd * 8 || L >= items) return x;
    const int tile = L / p.splits;
    x.split = L - tile * p.splits;
    const int group = kGroupM * p.tiles_n;
    const int gid = tile / group;
    const int gm = min(p.tiles_m - gid * kGroupM, kGroupM);
    const int r = tile - gid * group;
    x.m0 = (gid * kGroupM + r % gm) * BM;
    x.n0 = (r / gm) * BN;
    x.k0 = x.split * p.kchunk * 64;
    x.k1 = min(p.k, x.k0 + p.kchunk * 64);
    x.live = true;
    return x;
  };
  // (an id that maps past the items is followed by live ones of other XCDs'
  // runs: a workgroup's own ids t, t + nwg, ... with nwg a multiple of 8
  // stay on one XCD's run and end together)
  auto next = [&](int& t) {
    Item x = decode(t);
    while (!x.live && t < per_xcd * 8) {
      t += nwg;
      x = decode(t);
    }
    t += nwg;
    return x;
  };

  // ---- the stream of K blocks over the workgroup's items ----
  int lt = wg;
  Item li{};
  const uint8_t *pa = nullptr, *pb = nullptr;
  int left = 0;
  auto enter = [&]() {
    li = next(lt);
    left = li.live ? li.k1 - li.k0 : 0;
    const int64_t k0 = li.k0 + 64 * wk;  // (past the item's end: read by no load)
    pa = p.a + (TA ? k0 * p.lda + 2 * li.m0 : (int64_t)li.m0 * p.lda + 2 * k0);
    pb = p.b + (TB ? k0 * p.ldb + 2 * li.n0 : (int64_t)li.n0 * p.ldb + 2 * k0);
  };
  auto advance = [&]() {
    left -= 64 * WK;
    if (left <= 0) {
      if (li.live) enter();
    } else {
      pa += WK * (TA ? 64 * p.lda : 128);
      pb += WK * (TB ? 64 * p.ldb : 128);
    }
  };
  auto issue = [&](int slot) {
    const uint32_t st = uniform(lds0 + slot * STAGE);
    oa.issue(pa, p.lda, (TA ? p.wa : p.m) - li.m0, left - 64 * wk, st, wave);
    ob.issue(pb, p.ldb, (TB ? p.wb : p.n) - li.n0, left - 64 * wk, st + OpA::kBytes, wave);
    advance();
  };

  int ct = wg;
  Item cur = next(ct);
  if (!cur.live) return;
  enter();
#pragma unroll
  for (int s = 0; s < S; ++s) issue(s);
  dma::wait<(S - 1) * LOADS>();
  dma::barrier();

  int q = 0;       // ring slot of the current block
  int stores = 0;  // the previous item's stores per kStores, 0: not counted
  while (cur.live) {
    const int nkb = (cur.k1 - cur.k0 + 64 * WK - 1) / (64 * WK);
    Acc acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    // Fragments of half a block: B's twice (the half being multiplied and the
    // next), A's once -- a row's fragment is read anew for the next half as soon
    // as its MFMAs are issued.
    v8bf fa[FM], fb[2][FN];
    auto read_b = [&](int set, int slot, int s) {
#pragma unroll
      for (int i = 0; i < FN; ++i) fb[set][i] = ob.frag(lds0 + slot * STAGE + OpA::kBytes, i, s);
    };
    // INT8: the fences keep a fragment's read right behind the last product that
    // needs the old one (left to itself the compiler gathers the reads where
    // their registers spill, or moves them behind the barrier), and the next
    // block's loads go out one row of products apart instead of all at once
    // behind the barrier.  (4096 x 7168 x 4096: 138 us without either, 136 with
    // the fences, 128 with both.)
    typename OpA::Block next_a;
    typename OpB::Block next_b;
    auto multiply = [&](int set, int slot, int s, bool spread = false) {
      if constexpr (!INT8) read_b(set ^ 1, slot, s);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
#pragma unroll
        for (int i = 0; i < FN; ++i) acc[i][j] = mfma(fb[set][i], fa[j], acc[i][j]);
        if constexpr (INT8) __builtin_amdgcn_sched_barrier(0);
        fa[j] = oa.frag(lds0 + slot * STAGE, j, s);
        if constexpr (INT8) {
#pragma unroll
          for (int i = j * FN / FM; i < (j + 1) * FN / FM; ++i)
            fb[set ^ 1][i] = ob.frag(lds0 + slot * STAGE + OpA::kBytes, i, s);
          __builtin_amdgcn_sched_barrier(0);
          if (spread) {
#pragma unroll
            for (int l = j * LOADS / FM; l < (j + 1) * LOADS / FM; ++l) {
              if (l < OpA::kQ)
                oa.load(next_a, l);
              else
                ob.load(next_b, l - OpA::kQ);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    };
    read_b(0, q, 0);
#pragma unroll
    for (int j = 0; j < FM; ++j) fa[j] = oa.frag(lds0 + q * STAGE, j, 0);
    // (the epilogue passes the sums through LDS: through rows of its own where
    // the ring has two stages, else through the ring slot of the item's last
    // block, which is loaded anew only after it)
    int last = q;  // the slot of the block multiplied last
#pragma unroll 1
    for (int kb = 0; kb < nkb; ++kb) {
      multiply(0, q, 1);
      // this wave has read the block's stage (the barrier waits for its LDS
      // reads) and its share of the next block has landed (the previous item's
      // stores are younger than the blocks that were loaded before them)
      if (kb < kBehind && stores == 1)
        dma::wait<(S - 2) * LOADS + kStores>();
      else if (kb < kBehind && stores == 2)
        dma::wait<(S - 2) * LOADS + 2 * kStores>();
      else
        dma::wait<(S - 2) * LOADS>();
      dma::barrier();
      constexpr bool kSpread = INT8 && kOwnRows;
      if constexpr (kSpread) {
        const uint32_t st = uniform(lds0 + q * STAGE);
        next_a = oa.block(pa, p.lda, p.m - li.m0, left - 64 * wk, st, wave);
        next_b = ob.block(pb, p.ldb, p.n - li.n0, left - 64 * wk, st + OpA::kBytes, wave);
      } else {
        if (kOwnRows || kb + 1 < nkb) issue(q);
      }
      const int done = q;
      q = q + 1 == S ? 0 : q + 1;
      // (after the item's last block this reads the next item's first fragments,
      // which are read again behind the epilogue: one form of the loop's body)
      multiply(1, q, 0, kSpread);
      if constexpr (kSpread) advance();
      last = done;
    }

    // ---- epilogue ----
    // (the lane's indices made anew, opaque to the compiler: it would otherwise
    // keep offsets made from them in registers through the K loop)
    uint32_t lane_again = threadIdx.x & 63;
    asm volatile("" : "+v"(lane_again));
    const int lane = (int)lane_again, l16 = lane & 15, lq = lane >> 4;
    // (and its parameters read anew from the kernel's arguments, for the same reason)
    typedef const __attribute__((address_space(4))) GemmParams* Args;
    Args args = (Args)((const __attribute__((address_space(4))) uint8_t*)__builtin_amdgcn_kernarg_segment_ptr() + ARG);
    asm volatile("" : "+s"(args));
    Epilogue ep;
    __builtin_memcpy(&ep, (const Epilogue*)&args->epi, sizeof(ep));
    // 16 rows at a time: the wave's sums go to LDS as the MFMA leaves them and
    // come back as rows, 8 consecutive columns per lane
    {
      typedef __attribute__((address_space(3))) v4f* lp;
      const uint32_t so = kOwnRows ? lds0 + S * STAGE + wave * kRows : lds0 + last * STAGE + wave * (PART / NW);
      const int j_first = wk * FR;  // the group's own fragment rows
      if constexpr (WK > 1) {
        // the groups' sums of one half of K each meet: a wave hands out the rows
        // that others finish, in order, and adds what it gets in the groups' order
        typedef __attribute__((address_space(3))) Acc* la;
        const uint32_t given = so;
#pragma unroll
        for (int j = 0; j < FM; ++j)
          if (j / FR != wk) {
            const int x = j - (j / FR > wk ? FR : 0);
#pragma unroll
            for (int i = 0; i < FN; ++i)
              *(la)(uintptr_t)(given + (x * FN + i) * 1024 + lane * 16) = acc[i][j];
          }
        dma::lds_done();
        dma::barrier();
#pragma unroll
        for (int j = 0; j < FM; ++j)
          if (j / FR == wk) {
#pragma unroll
            for (int i = 0; i < FN; ++i) {
              Acc sum = Acc{0, 0, 0, 0};
#pragma unroll
              for (int h = 0; h < WK; ++h) {
                const uint32_t from = given + (h - wk) * PART + ((j - (j / FR > h ? FR : 0)) * FN + i) * 1024 + lane * 16;
                if (h == wk)
                  sum += acc[i][j];
                else
                  sum += *(la)(uintptr_t)from;
              }
              acc[i][j] = sum;
            }
          }
        dma::barrier();  // before the rows below take their place
      }
      const int m0w = wm * OpA::WTX, n = cur.n0 + wn * OpB::WTX + 8 * (lane % LPR);
      const int rows = min(BM, p.m - cur.m0);
      const epi::Rows er = epi::rows_of(ep, cur.m0, rows, p.n);
      // residual rows are loaded kAhead rows of fragments before their use: a
      // load waits for the stores before it
      constexpr int kAhead = FR < 4 ? FR : 4;
      // fragment row j = STEP x + FIRST of the sums, into LDS (the loops over x
      // below are not unrolled: one copy of the epilogue's code per STEP rows; the
      // row is picked by an opaque bit, since the compiler makes "jc == j" an
      // access by index, which would put the sums in scratch memory)
      // INT8: the scales of this lane's rows and columns
      v4f sb[INT8 ? FN : 1];
      float sa[INT8 ? FM : 1];
      const bool raw = INT8 && !LINES && p.splits > 1;  // partial sums stay whole numbers: bits that no fp32 operation touches
      if constexpr (INT8) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sb[i][e] = scales.sb[min(cur.n0 + wn * OpB::WTX + 16 * i + 4 * lq + e, p.n - 1)];
#pragma unroll
        for (int j = 0; j < FM; ++j) sa[j] = scales.sa[min(cur.m0 + m0w + 16 * j + l16, p.m - 1)];
      }
      auto put = [&](int j, int first, int step) {
        uint32_t bit = 1u << j;
        asm("" : "+s"(bit));
#pragma unroll
        for (int jc = first; jc < FM; jc += step)
          if (bit >> jc & 1) {
#pragma unroll
            for (int i = 0; i < FN; ++i) {
              v4f v;
              if constexpr (INT8) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  v[e] = raw ? __int_as_float(acc[i][jc][e]) : (float)acc[i][jc][e] * sb[i][e] * sa[jc];
              } else {
                v = acc[i][jc];
              }
              *(lp)(uintptr_t)(so + l16 * RS + (((4 * i + lq) ^ (l16 & (RC - 1))) << 4)) = v;
            }
          }
        dma::lds_done();
      };
      if constexpr (LINES) {
        float bias[8];
        const v4f b0 = epi::bias4(ep, n, p.n), b1 = epi::bias4(ep, n + 4, p.n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bias[e] = b0[e];
          bias[4 + e] = b1[e];
        }
        epi::v4i res[kAhead][ROUNDS];
        auto load_res = [&](int j, epi::v4i* to) {
#pragma unroll
          for (int h = 0; h < ROUNDS; ++h) {
            const int m = m0w + 16 * j + RPR * h + lane / LPR;
            to[h] = epi::residual8(ep, er, m, n, j < j_first + FR && m < rows && n < p.n);
          }
        };
        constexpr bool kPlain = TB;  // the backward pass's products: nothing but the sums, in bf16
        if (!kPlain && ep.res) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j) load_res(j_first + j, res[j]);
        }
#pragma unroll 1
        for (int jo = j_first; jo < j_first + FR; jo += kAhead) {
#pragma unroll
          for (int ji = 0; ji < kAhead; ++ji) {
            const int j = jo + ji;
            put(j, ji, kAhead);
            float v[ROUNDS][8];
#pragma unroll
            for (int h = 0; h < ROUNDS; ++h) {
              const int r = RPR * h + lane / LPR;
              const uint32_t a = so + r * RS, c = 2 * (lane % LPR), x = r & (RC - 1);
              const v4f lo = *(lp)(uintptr_t)(a + ((c ^ x) << 4)), hi = *(lp)(uintptr_t)(a + (((c + 1) ^ x) << 4));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[h][e] = lo[e];
                v[h][4 + e] = hi[e];
              }
            }
            dma::lds_done();  // before the next rows take their place
            epi::v4i rs[ROUNDS];
#pragma unroll
            for (int h = 0; h < ROUNDS; ++h) rs[h] = res[ji][h];
            if (!kPlain && ep.res) load_res(j + kAhead, res[ji]);
#pragma unroll
            for (int h = 0; h < ROUNDS; ++h) {
              const int m = m0w + 16 * j + RPR * h + lane / LPR;
              if constexpr (kPlain)
                epi::store8(ep, er, m, n, m < rows && n < p.n, v[h]);
              else
                epi::finish8(ep, er, m, n, m < rows && n < p.n, v[h], bias, rs[h]);
            }
          }
        }
      } else {
        // Rows that do not start on 16-byte boundaries, and partial sums: one
        // column per lane, so that an instruction still covers whole rows' runs
        // (8 columns per lane in 2-byte pieces would touch every line 8 times)
        constexpr int NV = 16 * OpB::WTX / 64, RPV = 64 / OpB::WTX;  // values per lane and 16 rows; rows per value
        const int col = lane % OpB::WTX, nc = cur.n0 + wn * OpB::WTX + col;
        const bool whole = p.splits == 1, with_res = whole && ep.res;
        const float bias = whole && ep.bias && nc < p.n
                               ? (ep.bias_f32 ? static_cast<const float*>(ep.bias)[nc]
                                              : epi::from_bf16(static_cast<const uint16_t*>(ep.bias)[nc]))
                               : 0.f;
        const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(p.ws + cur.split * p.ws_stride + (int64_t)cur.m0 * p.n), (short)0, whole ? 0 : rows * p.n * 4,
            0x00020000);
        // byte offset of value e of fragment row j in rows of ld elements of es
        // bytes (from an opaque copy of the lane's place: the compiler would
        // otherwise keep every value's offset in every tensor across the rows)
        auto at = [&](int j, int e, int64_t ld, int es) -> uint32_t {
          uint32_t place = (uint32_t)lane;
          asm("" : "+v"(place));
          const int m = m0w + 16 * j + RPV * e + (int)(place / OpB::WTX);
          const int c = cur.n0 + wn * OpB::WTX + (int)(place % OpB::WTX);
          return m < rows && c < p.n ? ((uint32_t)m * (uint32_t)ld + (uint32_t)c) * es : kOut;
        };
        uint16_t res[NV];
        auto load_col = [&](int j) {
#pragma unroll
          for (int e = 0; e < NV; ++e)
            res[e] = __builtin_amdgcn_raw_buffer_load_b16(er.res, j < j_first + FR ? at(j, e, ep.ldr, 2) : kOut, 0, 0);
        };
        if (with_res) load_col(j_first);
#pragma unroll 1
        for (int j = j_first; j < j_first + FR; ++j) {
          put(j, 0, 1);
          float v[NV];
#pragma unroll
          for (int e = 0; e < NV; ++e) {
            typedef __attribute__((address_space(3))) const float* lf;
            const int row = e * RPV + lane / OpB::WTX;
            const float got =
                *(lf)(uintptr_t)(so + row * RS + (((col >> 2) ^ (row & (RC - 1))) << 4) + ((col & 3) << 2));
            v[e] = raw ? got : got + bias;
          }
          dma::lds_done();
          if (!whole) {
#pragma unroll
            for (int e = 0; e < NV; ++e)
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), part, at(j, e, p.n, 4), 0, 0);
            continue;
          }
          if (ep.pre) {
#pragma unroll
            for (int e = 0; e < NV; ++e)
              __builtin_amdgcn_raw_buffer_store_b16(epi::to_bf16(v[e]), er.pre, at(j, e, ep.ldp, 2), 0, 0);
          }
          act::apply<NV>(v, ep.act);
          if (with_res) {
#pragma unroll
            for (int e = 0; e < NV; ++e) v[e] += epi::from_bf16(res[e]);
            load_col(j + 1);
          }
          if (ep.out_f32) {
#pragma unroll
            for (int e = 0; e < NV; ++e)
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), er.out, at(j, e, ep.ldc, 4), 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < NV; ++e)
              __builtin_amdgcn_raw_buffer_store_b16(epi::to_bf16(v[e]), er.out, at(j, e, ep.ldc, 2), 0, 0);
          }
        }
      }
      if constexpr (!kOwnRows) {
        dma::barrier();  // every wave is done with the slot
        issue(last);
      }
      const int per = !LINES ? 0 : (ep.out_f32 ? 2 : 1) + (ep.pre ? 1 : 0);
      stores = per <= 2 ? per : 0;
    }
    cur = next(ct);
  }
  dma::wait<0>();  // no load outlives the workgroup
}

}  // namespace tile
}  // namespace dg
