// Products of K-blocked operands on the MFMA engine, for the backwards of the head
// (flp_kernels.hip) and of the gated projection (flp_gated.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "flp_engine.h"
#include "flp_launch.h"

namespace flp {
namespace {  // every file has its own copies of the kernels it launches

// ---- GEMMs of the backward ----------------------------------------------------------------
//
// C[M x N] (+)= sum_k A[m][k] B[n][k], both operands in the K-blocked layout.
//   d_hidden: M = tokens, N = D, K = V (padded); A = dz, B = W^T.
//   d_weight: M = V, N = D, K = tokens (padded); A = dz^T, B = hidden^T.
// LOAD: start from the fp32 accumulator p.acc; STORE: 0 = element type to p.out,
// 1 = fp32 to p.acc, 2 = the fp32 sums of K slab blockIdx.y to p.acc[blockIdx.y].
// SCALED: the result is multiplied by *p.scale before it is rounded to p.out.
// TWO: two results under each other in A's rows: row m is row m of p.out, from p.split on row
// m - p.split of p.out2, each with p.rows_each rows (past those A's rows are padding) or null.
template <class E, int BM, int BN, int WM, int WN, bool LOAD, int STORE, int NS = 2, int NSA = NS,
          bool SCALED = false, bool TWO = false>
__global__ __launch_bounds__(64 * WM * WN) void k_gemm(GemmArgs p) {
  using Eng = Engine<E, BM, BN, WM, WN, NS, NSA>;
  constexpr int RW = Eng::RW, CW = Eng::CW, WMB = Eng::WMB, WNB = Eng::WNB;
  extern __shared__ u32x4 smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % WM, wn = wave / WM, i = lane & 15, g = lane >> 4;
  const int nbm = int((p.M + BM - 1) / BM), nbn = int((p.N + BN - 1) / BN);
  int tm, tn;
  tile_of<1>(blockIdx.x, nbm, nbn, tm, tn);
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;
  const int64_t nl = n0 + wn * CW + 4 * g;
  int64_t k0 = 0, kn = p.K;
  if constexpr (STORE == 2) {
    k0 = int64_t(blockIdx.y) * p.k_slab;
    kn = min(p.k_slab, p.K - k0);
  }
  const int64_t st0 = k0 * E::kSize / 128;  // first 128-byte K stage

  f32x4_t acc[WMB][WNB];
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    const int64_t m = m0 + wm * RW + mb * 16 + i;
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) {
      f32x4_t x = {0.f, 0.f, 0.f, 0.f};
      if (LOAD && m < p.M && nl + nb * 16 < p.N)
        x = *reinterpret_cast<const f32x4_t*>(p.acc + m * p.N + nl + nb * 16);
      acc[mb][nb] = x;
    }
  }
  Eng::template run<false>(acc,
                           reinterpret_cast<const char*>(p.a) + m0 * p.lda_b + st0 * p.a_ks,
                           p.lda_b, p.a_ks, p.M - m0,
                           reinterpret_cast<const char*>(p.b) + n0 * p.ldb_b + st0 * p.b_ks,
                           p.ldb_b, p.b_ks, p.N - n0, kn * E::kSize, smem);
  if constexpr (SCALED) {
    static_assert(STORE == 0, "only the rounded result is scaled");
    const float scale = *p.scale;
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb) acc[mb][nb] *= scale;
  }

  if constexpr (STORE == 0 && E::kSize == 2) {
    // 16-bit output: the tile is staged in the operand ring (rows of BN values plus 16
    // bytes) and written as 16-byte chunks of whole output rows.  The output is
    // 16-byte aligned, its row stride (D elements) a multiple of 32 and N = D a
    // multiple of 8, so every chunk lies inside one row.
    constexpr int kRowB = BN * 2 + 16;
    constexpr int kCh = BN * 2 / 16;  // 16-byte chunks per tile row
    static_assert(size_t(BM) * kRowB <= Eng::kLds, "the staged tile fits the operand ring");
    char* lds = reinterpret_cast<char*>(smem);
    __syncthreads();  // every wave is done reading the operand ring
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb) {
        const int rl = wm * RW + mb * 16 + i;
        const int cl = wn * CW + nb * 16 + 4 * g;
        u32x2 w;
        w.x = pack2<E>(acc[mb][nb][0], acc[mb][nb][1]);
        w.y = pack2<E>(acc[mb][nb][2], acc[mb][nb][3]);
        *reinterpret_cast<u32x2*>(lds + rl * kRowB + cl * 2) = w;
      }
    __syncthreads();
    for (int idx = tid; idx < BM * kCh; idx += Eng::NT) {
      const int rl = idx / kCh, ch = idx - rl * kCh;
      const int64_t m = m0 + rl, n = n0 + ch * 8;
      if constexpr (TWO) {
        const bool second = m >= p.split;
        const int64_t mo = second ? m - p.split : m;
        uint16_t* const out = reinterpret_cast<uint16_t*>(second ? p.out2 : p.out);
        if (mo < p.rows_each && n < p.N && out != nullptr)
          *reinterpret_cast<u32x4*>(out + mo * p.ldo + n) =
              *reinterpret_cast<const u32x4*>(lds + rl * kRowB + ch * 16);
      } else if (m < p.M && n < p.N) {
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.out) + m * p.ldo + n) =
            *reinterpret_cast<const u32x4*>(lds + rl * kRowB + ch * 16);
      }
    }
    return;
  }

#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    const int64_t m = m0 + wm * RW + mb * 16 + i;
    if (m >= p.M) continue;
    if constexpr (TWO) {
      static_assert(STORE == 0, "two results are rounded ones");
      const bool second = m >= p.split;
      const int64_t mo = second ? m - p.split : m;
      void* const out = second ? p.out2 : p.out;
      if (mo >= p.rows_each || out == nullptr) continue;
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
        if (nl + nb * 16 < p.N) store4<E>(out, mo * p.ldo + nl + nb * 16, acc[mb][nb]);
      continue;
    }
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) {
      if (nl + nb * 16 >= p.N) continue;
      if (STORE >= 1)
        *reinterpret_cast<f32x4_t*>(p.acc + ((STORE == 2 ? int64_t(blockIdx.y) * p.M : 0) + m) * p.N +
                                    nl + nb * 16) = acc[mb][nb];
      else
        store4<E>(p.out, m * p.ldo + nl + nb * 16, acc[mb][nb]);
    }
  }
}

// d_hidden in vocabulary slabs (the cross entropy's backward of up to kSlabRows rows): the
// slabs' fp32 sums side by side, then added in ascending order and rounded once.
template <class E>
__global__ __launch_bounds__(256) void k_slab_fold(GemmArgs p, int slabs) {
  const int64_t n = p.M * p.N;  // a multiple of 32
  const float scale = p.scale != nullptr ? *p.scale : 1.0f;
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < n;
       i += int64_t(gridDim.x) * 1024) {
    f32x4_t s = *reinterpret_cast<const f32x4_t*>(p.acc + i);
    for (int k = 1; k < slabs; ++k) s += *reinterpret_cast<const f32x4_t*>(p.acc + k * n + i);
    store4<E>(p.out, i, s * scale);
  }
}

template <class E, int BM, int BN, int WM, int WN, bool LOAD, int STORE, int NS = 2, int NSA = NS,
          bool SCALED = false, bool TWO = false>
hipError_t gemm_cfg(const GemmArgs& a, hipStream_t s) {
  using Eng = Engine<E, BM, BN, WM, WN, NS, NSA>;
  static std::atomic<int> ready[kMaxDevices];
  const hipError_t e = prepare(k_gemm<E, BM, BN, WM, WN, LOAD, STORE, NS, NSA, SCALED, TWO>, Eng::kLds, ready);
  if (e != hipSuccess) return e;
  const int64_t blocks = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  const unsigned slabs = STORE == 2 ? unsigned((a.K + a.k_slab - 1) / a.k_slab) : 1u;
  hipLaunchKernelGGL((k_gemm<E, BM, BN, WM, WN, LOAD, STORE, NS, NSA, SCALED, TWO>),
                     dim3(unsigned(blocks), slabs), dim3(Eng::NT), Eng::kLds, s, a);
  return hipGetLastError();
}

// A-operand ring depth of the 256 x 224 backward GEMM tiles (B keeps two buffers):
// the split ring of Engine::split (d_hidden and d_weight 2 % faster than one ring of
// two stages, same bits).
constexpr int kGemmNSA = 3;

}  // namespace
}  // namespace flp
