// The MFMA engine: tiles of C = A B^T fed by direct global -> LDS loads, and what its epilogues
// share.  Included by the kernels of the head (flp_kernels.hip) and of the gated projection
// (flp_gated.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace flp {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kStageBytes = 64;   // bytes of K per operand row per pipeline stage
constexpr int kGroupM = 8;        // row tiles per scheduling group

struct BF16 {
  static constexpr int kSize = 2;
};
struct F16 {
  static constexpr int kSize = 2;
};
struct F32 {
  static constexpr int kSize = 4;
};

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Both halves of a 16-lane (32-lane) exchange: every lane gets the values of lanes
// l and l ^ 16 (l ^ 32), lower row first (v_permlane16_swap / v_permlane32_swap, a
// VALU move).  A commutative combine of the two equals the xor-butterfly step.
__device__ __forceinline__ f32x2_t pair16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f32x2_t{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ f32x2_t pair32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f32x2_t{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// x of lane l ^ m.  For m = 1 and 2 a DPP quad permutation ([1, 0, 3, 2] and
// [2, 3, 0, 1]) and for m = 8 a rotation by 8 within the 16-lane row do it as a
// VALU move; other distances go through ds_bpermute.
__device__ __forceinline__ float lane_xor(float x, int m) {
  const int b = __float_as_int(x);
  if (m == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0xB1, 0xF, 0xF, true));
  if (m == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x4E, 0xF, 0xF, true));
  if (m == 8) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x128, 0xF, 0xF, true));
  return __shfl_xor(x, m);
}

// 64 bytes of K per lane quad: one bf16 16x16x32 MFMA, or four fp32 16x16x4
// MFMAs over the same 16 bytes per lane (K index 4g + t in instruction t).
template <class E>
__device__ __forceinline__ void mma64(f32x4_t& c, const u32x4& a, const u32x4& b);

template <>
__device__ __forceinline__ void mma64<BF16>(f32x4_t& c, const u32x4& a, const u32x4& b) {
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                               __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

template <>
__device__ __forceinline__ void mma64<F16>(f32x4_t& c, const u32x4& a, const u32x4& b) {
  c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                              __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <>
__device__ __forceinline__ void mma64<F32>(f32x4_t& c, const u32x4& a, const u32x4& b) {
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
}

// Bits of a 16-bit element type, rounded to nearest even.  gfx950 converts fp32
// to bf16 in hardware (v_cvt_pk_bf16_f32, round to nearest even, denormals kept:
// bit for bit the rounding (u + 0x7FFF + ((u >> 16) & 1)) >> 16 of the fp32 bits
// for every finite value).
template <class E>
__device__ __forceinline__ uint32_t bits16(float f);
template <>
__device__ __forceinline__ uint32_t bits16<BF16>(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
template <>
__device__ __forceinline__ uint32_t bits16<F16>(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}
template <class E>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return bits16<E>(lo) | (bits16<E>(hi) << 16);
}
template <>
__device__ __forceinline__ uint32_t pack2<BF16>(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Store four consecutive fp32 values as the element type.
template <class E>
__device__ __forceinline__ void store4(void* base, int64_t idx, const f32x4_t& v) {
  static_assert(E::kSize == 2, "16-bit element types");
  u32x2 w;
  w.x = pack2<E>(v.x, v.y);
  w.y = pack2<E>(v.z, v.w);
  *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(base) + idx) = w;
}

template <>
__device__ __forceinline__ void store4<F32>(void* base, int64_t idx, const f32x4_t& v) {
  *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(base) + idx) = v;
}

// K-blocked layout of the backward GEMM operands (dz, dz^T, W^T, hidden^T):
// element (r, k) of a matrix with `rows` rows sits at ((k / KB) * rows + r) * KB
// + k % KB, KB = 128 bytes of K.  One 128-byte pipeline stage of a GEMM tile is
// then a contiguous block of tile rows x 128 bytes.
template <int KB>
__device__ __forceinline__ int64_t kblk(int64_t r, int64_t k, int64_t rows) {
  return ((k / KB) * rows + r) * KB + (k % KB);
}

// Workgroup id -> (row tile, column tile).  Workgroups are dispatched
// round-robin over the 8 XCDs, so ids are first regrouped so that each XCD
// receives a contiguous run of logical tiles (sharing its L2), then the run is
// walked in groups of GM row tiles, row tile fastest, so that the workgroups
// resident at one time share both operand tiles.  Logits tiles use GM = 8
// (8 row tiles x 4 vocabulary tiles per XCD at a time; 4 and 16 measured slower);
// the backward GEMMs use GM = 1, the 12 column tiles of one row tile in turn
// (measured best of 1, 2, 4, 8 and 16 with their split LDS ring).
template <int GM = kGroupM>
__device__ __forceinline__ void tile_of(int bid, int nbm, int nbn, int& tm, int& tn) {
  const int total = nbm * nbn;
  const int per = total >> 3;
  int lin = bid;
  if (bid < per * 8) lin = (bid & 7) * per + (bid >> 3);
  const int width = GM * nbn;
  const int grp = lin / width;
  const int first = grp * GM;
  const int gm = min(nbm - first, GM);
  const int in = lin - grp * width;
  tm = first + in % gm;
  tn = in / gm;
}

// ---- direct global -> LDS staging of one operand tile --------------------------------------
//
// A pipeline stage holds 128 bytes of K per operand row (two 64-byte MFMA steps),
// so that every load covers whole 128-byte cache lines.  In LDS a row is 8
// 16-byte chunks; logical chunk c of row r sits at position c ^ ((r >> 1) & 7),
// which puts the 16 rows of a fragment read on 16 distinct bank groups.  One wave
// instruction fills 64 consecutive LDS chunks (lane l -> chunk base + l): it
// covers rows 8 inst + l / 8 at positions l % 8.  Rows past the end of the
// operand read a clamped (valid) row whose results are never used; in a last,
// half stage (64 bytes of K left) the upper four chunks repeat the lower four.
template <int ROWS, int NW>
struct DTile {
  static constexpr int kInsts = ROWS / 8;
  static constexpr int kPer = (kInsts + NW - 1) / NW;
  // Wave w issues instructions w*kPer .. min(kInsts, (w+1)*kPer) - 1, so the last
  // waves may issue fewer: count(w) per stage.
  static constexpr int count(int w) {
    return kInsts - w * kPer <= 0 ? 0 : (kInsts - w * kPer > kPer ? kPer : kInsts - w * kPer);
  }
  static_assert(ROWS % 16 == 0, "tile rows must be a multiple of 16");
  int q;                // row within the instruction's 8 rows
  int c0, c1;           // logical chunk loaded by this lane for even / odd instructions
  int64_t ld, ks, rows_valid;  // row stride, stage stride (bytes), rows that exist
  bool full;            // every row of the tile is valid: no clamping

  __device__ __forceinline__ void init(int64_t ld_, int64_t ks_, int64_t rows_valid_, int lane) {
    ld = ld_;
    ks = ks_;
    rows_valid = rows_valid_;
    full = rows_valid_ >= ROWS;
    q = lane >> 3;
    c0 = (lane & 7) ^ (q >> 1);
    c1 = c0 ^ 4;
  }
  __device__ __forceinline__ void issue(const char* base, int stage, bool half, u32x4* lds,
                                        int wave) const {
    // A raw buffer resource based at the stage keeps the per-lane part a 32-bit
    // offset that does not change from stage to stage.
    const char* sb = base + int64_t(stage) * ks;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)sb, (short)0, 0x7FFFFFFF, 0x00020000);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int inst = wave * kPer + j;
      if (kInsts % NW == 0 || inst < kInsts) {
        int c = (inst & 1) ? c1 : c0;
        c = half ? (c & 3) : c;
        int64_t r = int64_t(inst) * 8 + q;
        if (!full) r = r < rows_valid ? r : rows_valid - 1;
        const uint32_t off = uint32_t(r * ld) + uint32_t(c * 16);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void*)(lds + inst * 64), 16, int(off), 0, 0, 0);
      }
    }
  }
};

// Wait until at most N of this wave's vector-memory loads are outstanding and its
// LDS reads have completed, then barrier the workgroup.  The direct loads
// complete in issue order.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_own() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

// ---- the MFMA engine -------------------------------------------------------------------------
//
// A ring of NS LDS buffers of one 128-byte stage each (two for the large tiles);
// stage t lives in buffer t % NS and holds the MFMA steps 2t (chunks 0-3) and
// 2t + 1 (chunks 4-7).  Every MFMA step multiplies fragments read from LDS during
// the previous step.  The workgroup synchronises once per stage, between its two
// steps: stage t + 1 must have landed (its loads were issued NS - 1 stages
// earlier) and every wave must be done reading stage t, whose buffer then receives
// the loads of stage t + NS.  Small tiles do little work per stage, so they use a
// deeper ring to keep enough loads in flight.
// What a peeled pipeline stage does at its barrier (a compile-time tag).
template <int M>
using Mode = std::integral_constant<int, M>;

template <class E, int BM, int BN, int WM, int WN, int NS = 2, int NSA = NS>
struct Engine {
  using TileA = DTile<BM, WM * WN>;
  static constexpr int NW = WM * WN;
  static constexpr int NT = 64 * NW;
  static constexpr int RW = BM / WM;
  static constexpr int CW = BN / WN;
  static constexpr int WMB = RW / 16;
  static constexpr int WNB = CW / 16;
  static constexpr int kSlots = (BM + BN) * 8;  // 16-byte LDS chunks per stage
  // NSA buffers of the A operand, NS of B (NSA = NS: one ring of both).
  static constexpr size_t kLds = (size_t(NSA) * BM + size_t(NS) * BN) * 128;
  static_assert(NS >= 2, "at least two LDS stages");
  static_assert(NSA == NS || (NS == 2 && NSA == 3), "A ring one deeper than B: 3 and 2 buffers");
  static_assert(RW % 16 == 0 && CW % 16 == 0, "wave tile must be a multiple of 16");

  struct Frag {
    u32x4 a[WMB], b[WNB];
  };

  // Fragments of one MFMA step from the buffer at `st`: per-lane base chunks fa,
  // fb; the 16-row blocks are immediate offsets (128 chunks apart).
  __device__ __forceinline__ static void read(Frag& f, const u32x4* st, int fa, int fb) {
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb) f.a[mb] = st[fa + mb * 128];
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) f.b[nb] = st[BM * 8 + fb + nb * 128];
  }

  // The same with the A and B fragments in separate buffers.
  __device__ __forceinline__ static void read2(Frag& f, const u32x4* sa, const u32x4* sb, int fa,
                                               int fb) {
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb) f.a[mb] = sa[fa + mb * 128];
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) f.b[nb] = sb[fb + nb * 128];
  }

  __device__ __forceinline__ static void mmas(f32x4_t (&acc)[WMB][WNB], const Frag& f) {
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb) mma64<E>(acc[mb][nb], f.b[nb], f.a[mb]);
  }

  // Keep the reads of the next step spread among the MFMAs of this one, starting
  // with MFMAs: the wait for this step's fragments then precedes every new read
  // (LDS reads complete in order, so a read issued first would be waited for too).
  __device__ __forceinline__ static void interleave() {
    constexpr int kR = WMB + WNB, kM = WMB * WNB * (E::kSize == 2 ? 1 : 4);
    constexpr int kStep = kM / kR > 0 ? kM / kR : 1;
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, kStep, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    if constexpr (kM > kStep * kR) __builtin_amdgcn_sched_group_barrier(0x008, kM - kStep * kR, 0);
    __builtin_amdgcn_sched_barrier(0);
  }

  // acc (+)= A[rows, K] . B[rows, K]^T over kbytes of K (a multiple of 64; ODD when
  // kbytes / 64 is odd).  a and b point at the first row of the tile; rows past
  // *_rows_valid are clamped.
  template <bool ODD>
  __device__ __forceinline__ static void run(f32x4_t (&acc)[WMB][WNB], const char* a, int64_t lda,
                                             int64_t a_rows_valid, const char* b, int64_t ldb,
                                             int64_t b_rows_valid, int64_t kbytes, u32x4* smem) {
    run<ODD>(acc, a, lda, 128, a_rows_valid, b, ldb, 128, b_rows_valid, kbytes, smem);
  }
  // The same with explicit stage strides (bytes from one 128-byte K stage of a row
  // to the next): 128 for row-major operands, rows x 128 for K-blocked ones.
  template <bool ODD>
  __device__ __forceinline__ static void run(f32x4_t (&acc)[WMB][WNB], const char* a, int64_t lda,
                                             int64_t a_ks, int64_t a_rows_valid, const char* b,
                                             int64_t ldb, int64_t b_ks, int64_t b_rows_valid,
                                             int64_t kbytes, u32x4* smem) {
    walk<ODD, DTile<BN, NW>>(acc, a, lda, a_ks, a_rows_valid, b, ldb, b_ks, b_rows_valid, kbytes,
                             smem);
  }
  // The same with a B operand of another kind, TB, which issues as many loads per wave; `more`
  // is for its init.
  template <bool ODD, class TB, class... More>
  __device__ __forceinline__ static void walk(f32x4_t (&acc)[WMB][WNB], const char* a, int64_t lda,
                                              int64_t a_ks, int64_t a_rows_valid, const char* b,
                                              int64_t ldb, int64_t b_ks, int64_t b_rows_valid,
                                              int64_t kbytes, u32x4* smem, More... more) {
    const int tid = threadIdx.x, lane = tid & 63;
    // Wave-uniform, so that the LDS destinations of the direct loads (M0) are scalar.
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM, i = lane & 15, g = lane >> 4;
    const int nsteps = int(kbytes / kStageBytes);
    const int nst = (nsteps + 1) / 2;
    TileA ta;
    TB tb;
    ta.init(lda, a_ks, a_rows_valid, lane);
    tb.init(ldb, b_ks, b_rows_valid, lane, more...);
    // Chunk of the even step for this lane; the odd step's is pos ^ 4.
    const int pos = g ^ ((i >> 1) & 7);
    const int fa = (wm * RW + i) * 8 + pos;
    const int fb = (wn * CW + i) * 8 + pos;
    auto issue = [&](int t) {
      u32x4* dst = smem + (t % NS) * kSlots;
      const bool half = ODD && t == nst - 1;
      ta.issue(a, t, half, dst, wave);
      tb.issue(b, t, half, dst + BM * 8, wave);
    };
    if constexpr (NSA != NS) {
      static_assert(!ODD, "the split ring serves the GEMMs, whose K is whole 128-byte stages");
      split(acc, nst, ta, tb, a, b, fa, fb, smem, wave);
      return;
    } else if constexpr (NS > 2) {
      deep<ODD>(acc, nst, issue, fa, fb, smem, wave);
      return;
    }
    issue(0);
    if (nst > 1) {
      issue(1);
      wait_stages<1>(wave);
      barrier_only();
    } else {
      wait_barrier<0>();
    }
    Frag f0, f1;
    read(f0, smem, fa, fb);
    // Stage t: step 2t from f0 (read one step earlier) while reading step 2t + 1
    // into f1; synchronise; step 2t + 1 from f1 while reading step 2t + 2 into
    // f0.  After the last stage the other buffer still holds consumed data that
    // no load overwrites any more; reading it (unused) keeps the body free of
    // branches around the fragment reads.
    //
    // The stages that issue loads run in a loop of their own whose body has no
    // branches (one block the scheduler orders as a whole); the last two stages
    // (barrier only, then neither barrier nor loads) are peeled off.
    auto stage = [&](int t, auto mode) {
      constexpr int kMode = decltype(mode)::value;  // 0: barrier + loads, 1: barrier, 2: none
      read(f1, smem + (t & 1) * kSlots, fa ^ 4, fb ^ 4);
      mmas(acc, f0);
      interleave();
      if constexpr (kMode <= 1) wait_barrier<0>();
      if constexpr (kMode == 0) issue(t + 2);
      read(f0, smem + ((t + 1) & 1) * kSlots, fa, fb);
      mmas(acc, f1);
      interleave();
    };
    for (int t = 0; t + 2 < nst; ++t) stage(t, Mode<0>{});
    if (nst >= 2) stage(nst - 2, Mode<1>{});
    if (!ODD) stage(nst - 1, Mode<2>{});
    if constexpr (ODD) mmas(acc, f0);
  }

  // The ring of NS > 2 stages: the first NS stages are issued up front; at the
  // barrier of stage t, stages t + 2 .. t + NS - 1 may still be in flight (every
  // stage issues the same number of loads per wave, a half stage included), and
  // near the end of the K walk everything is waited for.  Waves may issue
  // different numbers of loads per stage (the instructions of a tile are split
  // over the waves in runs of kPer), so each wave waits on its own count: a
  // wave-uniform branch picks the immediate, and every wave then reaches the one
  // barrier.
  static_assert(NS == 2 || (NS - 1) * (TileA::kPer + DTile<BN, NW>::kPer) <= 63,
                "the loads in flight must fit the vmcnt counter");
  static constexpr int loads_of(int w) { return TileA::count(w) + DTile<BN, NW>::count(w); }
  // Last wave of the run of waves from w on that issue as many loads as wave w.
  static constexpr int run_end(int w) {
    return w + 1 < NW && loads_of(w + 1) == loads_of(w) ? run_end(w + 1) : w;
  }
  template <int Stages, int W = 0>
  __device__ __forceinline__ static void wait_stages(int wave) {
    constexpr int Last = run_end(W);
    if constexpr (Last + 1 < NW) {
      if (wave <= Last) {
        wait_own<Stages * loads_of(W)>();
        return;
      }
      wait_stages<Stages, Last + 1>(wave);
    } else {
      wait_own<Stages * loads_of(W)>();
    }
  }
  // Per-wave wait until at most KA stages of its A loads and KB stages of its B
  // loads are outstanding.
  static constexpr int mix_of(int w, int ka, int kb) {
    return ka * TileA::count(w) + kb * DTile<BN, NW>::count(w);
  }
  static constexpr int mix_end(int w, int ka, int kb) {
    return w + 1 < NW && mix_of(w + 1, ka, kb) == mix_of(w, ka, kb) ? mix_end(w + 1, ka, kb) : w;
  }
  template <int KA, int KB, int W = 0>
  __device__ __forceinline__ static void wait_mix(int wave) {
    constexpr int Last = mix_end(W, KA, KB);
    if constexpr (Last + 1 < NW) {
      if (wave <= Last) {
        wait_own<mix_of(W, KA, KB)>();
        return;
      }
      wait_mix<KA, KB, Last + 1>(wave);
    } else {
      wait_own<mix_of(W, KA, KB)>();
    }
  }

  // The split ring: three buffers of the A operand, two of B.  The GEMMs stream
  // their A operand (dz, dz^T) from HBM once, while B (W^T, hidden^T) is shared by
  // many workgroups through the caches, so the A loads get two stages of time to
  // land and the B loads one.  At the barrier of stage t the buffers of stage t
  // are free and receive B(t + 2), then A(t + 3), in that order: the direct loads
  // complete in issue order, so waiting until only this wave's A(t + 2) loads may
  // be outstanding (issued at the previous barrier, after B(t + 1)) guarantees
  // that all of stage t + 1 has landed.
  template <class TA, class TB>
  __device__ __forceinline__ static void split(f32x4_t (&acc)[WMB][WNB], int nst, const TA& ta,
                                               const TB& tb, const char* a, const char* b, int fa,
                                               int fb, u32x4* smem, int wave) {
    u32x4* const sa = smem;
    u32x4* const sb = smem + NSA * BM * 8;
    auto issue_a = [&](int t, int buf) { ta.issue(a, t, false, sa + buf * BM * 8, wave); };
    auto issue_b = [&](int t, int buf) { tb.issue(b, t, false, sb + buf * BN * 8, wave); };
    issue_a(0, 0);
    issue_b(0, 0);
    if (nst > 1) {
      issue_a(1, 1);
      issue_b(1, 1);
    }
    if (nst > 2) {
      issue_a(2, 2);
      wait_mix<2, 1>(wave);  // A(1), B(1), A(2) may be in flight
    } else if (nst > 1) {
      wait_mix<1, 1>(wave);
    } else {
      wait_own<0>();
    }
    barrier_only();
    Frag f0, f1;
    read2(f0, sa, sb, fa, fb);
    int ca = 0, cb = 0;  // buffers of stage t
    // As in the two-stage ring, the stages that issue both loads run in a loop
    // without branches, and the last three stages are peeled off.
    auto stage = [&](int t, auto mode) {
      // 0: barrier + B(t + 2) + A(t + 3), 1: barrier + B(t + 2), 2: barrier, 3: none
      constexpr int kMode = decltype(mode)::value;
      const int na = ca == 2 ? 0 : ca + 1, nb = cb ^ 1;
      read2(f1, sa + ca * BM * 8, sb + cb * BN * 8, fa ^ 4, fb ^ 4);
      mmas(acc, f0);
      interleave();
      if constexpr (kMode <= 1)
        wait_mix<1, 0>(wave);  // only A(t + 2) may be in flight
      else if constexpr (kMode == 2)
        wait_own<0>();
      if constexpr (kMode <= 2) barrier_only();
      if constexpr (kMode <= 1) issue_b(t + 2, cb);
      if constexpr (kMode == 0) issue_a(t + 3, ca);
      read2(f0, sa + na * BM * 8, sb + nb * BN * 8, fa, fb);
      mmas(acc, f1);
      interleave();
      ca = na;
      cb = nb;
    };
    int t = 0;
    for (; t + 3 < nst; ++t) stage(t, Mode<0>{});
    if (t + 2 < nst) stage(t++, Mode<1>{});
    if (t + 1 < nst) stage(t++, Mode<2>{});
    stage(t, Mode<3>{});
  }

  template <bool ODD, class Issue>
  __device__ __forceinline__ static void deep(f32x4_t (&acc)[WMB][WNB], int nst, Issue& issue,
                                              int fa, int fb, u32x4* smem, int wave) {
    for (int t = 0; t < NS && t < nst; ++t) issue(t);
    if (nst >= NS) {
      wait_stages<NS - 1>(wave);
      barrier_only();
    } else {
      wait_barrier<0>();
    }
    Frag f0, f1;
    read(f0, smem, fa, fb);
    int cur = 0;  // buffer of stage t
    // 0: wait + barrier + loads of stage t + NS, 1: wait + barrier, 2: wait for all
    // + barrier, 3: none; the load-issuing stages again form a loop of their own.
    auto stage = [&](int t, auto mode) {
      constexpr int kMode = decltype(mode)::value;
      const int nxt = cur + 1 == NS ? 0 : cur + 1;
      read(f1, smem + cur * kSlots, fa ^ 4, fb ^ 4);
      mmas(acc, f0);
      interleave();
      if constexpr (kMode <= 1) {
        wait_stages<NS - 2>(wave);
        barrier_only();
      } else if constexpr (kMode == 2) {
        wait_barrier<0>();
      }
      if constexpr (kMode == 0) issue(t + NS);
      read(f0, smem + nxt * kSlots, fa, fb);
      mmas(acc, f1);
      interleave();
      cur = nxt;
    };
    int t = 0;
    for (; t + NS < nst; ++t) stage(t, Mode<0>{});
    if (t + NS - 1 < nst) stage(t++, Mode<1>{});
    for (; t + 1 < nst; ++t) stage(t, Mode<2>{});
    if (!ODD) stage(t, Mode<3>{});
    if constexpr (ODD) mmas(acc, f0);
  }
};

}  // namespace flp
