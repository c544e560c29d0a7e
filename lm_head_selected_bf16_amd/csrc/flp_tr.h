// Products of 16-bit operands of which one or both lie with K along their rows' stride (a weight
// [K][N], tokens [K][M]): such an operand is staged as it lies and turned while it is read from
// LDS (ds_read_b64_tr_b16), so no transposed copy is written.
//
// ds_read_b64_tr_b16: of 16 lanes, lane i gives the address of four elements of row i / 4 and
// gets the four rows' elements of column i.  Two such reads fill a fragment of 8 K values: lane
// (i, g) of a wave holds column i at K = 8 g + 0..7, the order of a fragment read whole from a
// row-major operand.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flp_engine.h"
#include "flp_launch.h"

namespace flp {
namespace {  // every file has its own copies of the kernels it launches

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// The read.  `restrict` gives it an alias scope: without one the compiler takes it to read what any
// load to LDS in flight writes, and waits for all of those first (the ring does its own waiting;
// products half again as long).
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ u32x2 read_turned(lds_char* __restrict p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4_t*)p));
}

// K rows of 64 per stage (two MFMA steps of 32), as in the engine.
constexpr int kTrRows = 64;

// An operand of ROWS rows with K contiguous: the engine's tile and fragments.
template <int ROWS, int NW, int NF>
struct PlainOp {
  using Tile = DTile<ROWS, NW>;
  static constexpr int kChunks = ROWS * 8;  // 16-byte LDS chunks per stage
  static constexpr int kReads = NF;         // LDS reads of a step
  static constexpr int count(int w) { return Tile::count(w); }
  Tile tile;
  const char* base;
  int at;
  // base: first row of the tile at the first K; ld: bytes from row to row; first: the wave's row
  __device__ __forceinline__ void init(const char* base_, int64_t ld, int64_t rows_valid, int lane,
                                       int first) {  // at its first stage
    base = base_;
    tile.init(ld, 128, rows_valid, lane);
    const int i = lane & 15, g = lane >> 4;
    at = (first + i) * 8 + (g ^ ((i >> 1) & 7));
  }
  __device__ __forceinline__ void issue(u32x4* lds, int wave) {
    tile.issue(base, 0, false, lds, wave);
    base += 128;
  }
  template <int STEP>
  __device__ __forceinline__ void read(u32x4 (&f)[NF], const u32x4* lds) const {
    const u32x4* p = lds + (STEP ? at ^ 4 : at);
#pragma unroll
    for (int n = 0; n < NF; ++n) f[n] = p[n * 128];
  }
};

// An operand of COLS columns with its K along the rows: a stage is 64 rows of COLS elements.  An
// LDS row is 16 (8) blocks of 16 elements, the last ones unused where COLS has fewer; block b of
// row k sits at place b ^ s(k).  A read touches the rows 8 g + 4 h + 0..3 of the four groups g of
// lanes, which s spreads over all places (over eight of them: any two neighbouring groups), so
// that no two use a bank at the same time (s(k) = k mod 16, which repeats from group to group
// but one: 2 more cycles a read and a third of the loop's time).
// PAIR: two matrices under each other, the second from row `split` on, `rows` rows each.
template <int COLS, int NW, int NF, bool PAIR>
struct TurnedOp {
  static constexpr int kBlocks = COLS / 16, kPlaces = kBlocks > 8 ? 16 : 8;
  static constexpr int kPitch = kPlaces * 32;  // bytes
  static constexpr int kChunks = kTrRows * kPitch / 16;
  static constexpr int kInsts = kTrRows * kPitch / 1024, kPer = kInsts / NW;
  static constexpr int kReads = 2 * NF;
  static constexpr uint32_t kNowhere = 0x70000000u;  // an offset past every resource: zeros
  static_assert(COLS % 16 == 0 && kBlocks <= 16 && kInsts % NW == 0, "whole instructions per wave");
  static constexpr int count(int) { return kPer; }
  static __device__ __forceinline__ int swizzle(int k) {
    return (kPlaces == 16 ? (k >> 1) & 12 : ((k >> 1) ^ (k >> 2)) & 4) | (k & 3);
  }

  // The stages are issued in order, each call moving on by one.
  const char *next, *second_;  // at the tile's first column
  int64_t step;                // bytes from stage to stage
  int ld, rows_left, stages_left, rows;  // rows_left: of this matrix; stages_left: before the second
  int64_t off;
  uint32_t o[kPer];            // the lane's offsets within a stage
  int at[2][NF];               // bytes
  // base: column 0 of the matrix; ld: bytes from row to row; col0: the tile's first column of
  // `cols`; first: the first row; wave_block: the wave's first block of 16 columns in the tile
  __device__ __forceinline__ void init(const char* base, const char* second, int64_t split,
                                       int64_t rows_, int64_t ld_, int64_t col0, int64_t cols,
                                       int64_t first, int lane, int wave, int wave_block) {
    off = col0 * 2;
    ld = int(ld_);
    step = ld_ * kTrRows;
    rows = int(rows_);
    second_ = second + off;
    const bool past = PAIR && first >= split;
    const int64_t k = past ? first - split : first;
    next = (past ? second : base) + off + k * ld_;
    rows_left = int(rows_ - k);
    stages_left = past || !PAIR ? 0 : int((split - first) / kTrRows);
    stages_left = __builtin_amdgcn_readfirstlane(stages_left);
    rows_left = __builtin_amdgcn_readfirstlane(rows_left);
    const int64_t left = (cols - col0 + 15) / 16;
    const int blocks = left < kBlocks ? int(left) : kBlocks;
    constexpr int kLanes = kPitch / 16;  // of a row
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int row = (wave * kPer + j) * (1024 / kPitch) + lane / kLanes;
      const int b = ((lane % kLanes) >> 1) ^ swizzle(row);
      o[j] = b < blocks ? uint32_t(row) * uint32_t(ld) + uint32_t(b * 32 + (lane & 1) * 16) : kNowhere;
    }
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 8 * g + 4 * h + (i >> 2);
#pragma unroll
      for (int n = 0; n < NF; ++n)
        at[h][n] = k * kPitch + ((wave_block + n) ^ swizzle(k)) * 32 + (i & 3) * 8;
    }
  }
  // The next 64 rows: those past the matrix's end are past the resource, and read as zeros.
  __device__ __forceinline__ void issue(u32x4* lds, int wave) {
    const int here = min(max(rows_left, 0), kTrRows);  // no branch: the loop stays one block
    const int records = __builtin_amdgcn_readfirstlane(max(here * ld - int(off), 0));
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)next, (short)0, records, 0x00020000);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(lds + (wave * kPer + j) * 64), 16, int(o[j]),
          0, 0, 0);
    next += step;
    rows_left -= kTrRows;
    if constexpr (PAIR) {
      stages_left -= 1;
      const bool turn = stages_left == 0;
      next = turn ? second_ : next;
      rows_left = turn ? rows : rows_left;
    }
  }
  template <int STEP>
  __device__ __forceinline__ void read(u32x4 (&f)[NF], const u32x4* lds) const {
    lds_char* p = (lds_char*)lds;
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      const u32x2 x = read_turned(p + at[0][n] + STEP * 32 * kPitch);
      const u32x2 y = read_turned(p + at[1][n] + STEP * 32 * kPitch);
      f[n] = u32x4{x.x, x.y, y.x, y.y};
    }
  }
};

// acc = A . B^T over nst stages: the engine's ring of three buffers of A and two of
// B (Engine::split), over operands of either kind.
template <class E, class OpA, class OpB, int NA, int NB, int NW>
struct TrRing {
  static constexpr size_t kLds = (3 * size_t(OpA::kChunks) + 2 * size_t(OpB::kChunks)) * 16;
  struct Frag {
    u32x4 a[NA], b[NB];
  };
  __device__ __forceinline__ static void mmas(f32x4_t (&acc)[NA][NB], const Frag& f) {
#pragma unroll
    for (int m = 0; m < NA; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n) mma64<E>(acc[m][n], f.b[n], f.a[m]);
  }
  __device__ __forceinline__ static void interleave() {
    constexpr int kR = OpA::kReads + OpB::kReads, kM = NA * NB;
    constexpr int kStep = kM / kR > 0 ? kM / kR : 1;
    constexpr int kPairs = kR < kM / kStep ? kR : kM / kStep;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, kStep, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    if constexpr (kM > kStep * kPairs) __builtin_amdgcn_sched_group_barrier(0x008, kM - kStep * kPairs, 0);
    if constexpr (kR > kPairs) __builtin_amdgcn_sched_group_barrier(0x100, kR - kPairs, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
  static constexpr int mix_of(int w, int ka, int kb) { return ka * OpA::count(w) + kb * OpB::count(w); }
  static constexpr int mix_end(int w, int ka, int kb) {
    return w + 1 < NW && mix_of(w + 1, ka, kb) == mix_of(w, ka, kb) ? mix_end(w + 1, ka, kb) : w;
  }
  // Until at most KA stages of this wave's A loads and KB of its B loads are outstanding.
  template <int KA, int KB, int W = 0>
  __device__ __forceinline__ static void wait(int wave) {
    constexpr int kLast = mix_end(W, KA, KB);
    if constexpr (kLast + 1 < NW) {
      if (wave <= kLast) {
        wait_own<mix_of(W, KA, KB)>();
        return;
      }
      wait<KA, KB, kLast + 1>(wave);
    } else {
      wait_own<mix_of(W, KA, KB)>();
    }
  }
  __device__ __forceinline__ static void run(f32x4_t (&acc)[NA][NB], OpA& a, OpB& b, int nst,
                                             u32x4* smem, int wave) {
    u32x4* const sa = smem;
    u32x4* const sb = smem + 3 * OpA::kChunks;
    auto issue_a = [&](int buf) { a.issue(sa + buf * OpA::kChunks, wave); };
    auto issue_b = [&](int buf) { b.issue(sb + buf * OpB::kChunks, wave); };
    issue_a(0);
    issue_b(0);
    if (nst > 1) {
      issue_a(1);
      issue_b(1);
    }
    if (nst > 2) {
      issue_a(2);
      wait<2, 1>(wave);
    } else if (nst > 1) {
      wait<1, 1>(wave);
    } else {
      wait_own<0>();
    }
    barrier_only();
    Frag f0, f1;
    a.template read<0>(f0.a, sa);
    b.template read<0>(f0.b, sb);
    int ca = 0, cb = 0;
    auto stage = [&](auto mode) {
      // 0: barrier + B(t + 2) + A(t + 3), 1: barrier + B(t + 2), 2: barrier, 3: none
      constexpr int kMode = decltype(mode)::value;
      const int na = ca == 2 ? 0 : ca + 1, nb = cb ^ 1;
      a.template read<1>(f1.a, sa + ca * OpA::kChunks);
      b.template read<1>(f1.b, sb + cb * OpB::kChunks);
      mmas(acc, f0);
      interleave();
      if constexpr (kMode <= 1)
        wait<1, 0>(wave);
      else if constexpr (kMode == 2)
        wait_own<0>();
      if constexpr (kMode <= 2) barrier_only();
      if constexpr (kMode <= 1) issue_b(cb);
      if constexpr (kMode == 0) issue_a(ca);
      if constexpr (kMode <= 2) {
        a.template read<0>(f0.a, sa + na * OpA::kChunks);
        b.template read<0>(f0.b, sb + nb * OpB::kChunks);
      }
      mmas(acc, f1);
      interleave();
      ca = na;
      cb = nb;
    };
    int t = 0;
    for (; t + 3 < nst; ++t) stage(Mode<0>{});
    if (t + 2 < nst) {
      stage(Mode<1>{});
      ++t;
    }
    if (t + 1 < nst) stage(Mode<2>{});
    stage(Mode<3>{});
  }
};

}  // namespace
}  // namespace flp
