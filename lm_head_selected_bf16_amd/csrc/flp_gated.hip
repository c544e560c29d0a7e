// The gated projection of a feed-forward block, forward and backward:
//
//   z = x Wg^T,  u = x Wu^T,  out = act(z) u
//   dz = grad u act'(z),  du = grad act(z)
//   d_x = dz Wg + du Wu,  d_Wg = dz^T x,  d_Wu = du^T x
//
// Forward: one pass of the MFMA engine whose B operand interleaves the two weights, so that
// a lane holds z and u of the same elements and the epilogue needs nothing else.  For the
// backward it keeps a = act(z) and b = u act'(z), so that no third product is needed:
// dz = grad b, du = grad a.  Beside 16-bit types they are kept in 24 bits (fp32 without its
// last 8): kept in 16, their roundings make the gradients' error 3.1e-3 where the rounding of
// dz, du and the result alone gives 2.4e-3.
//
// Backward: dz and du side by side, once K-blocked by columns (the A operand of d_x, against
// [Wg; Wu]^T) and once by tokens (that of the weight gradients, against x^T), and two
// products.  Their rounding to the element type is what the matrix instructions take.
//
// Bound by the matrix instructions for many rows, by reading the weights for few.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "flp_chunk.h"
#include "flp_engine.h"
#include "flp_gemm.h"
#include "flp_launch.h"

namespace flp {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + exp(-v)); no cancellation on either side.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

// The factor f(z) of act(z) = z f(z): the logistic function (silu), the normal distribution's
// (gelu), or the logistic one of its odd cubic approximation (gelu_tanh: 0.5 (1 + tanh v) is
// the logistic function of 2 v).
constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;
template <int ACT>
__device__ __forceinline__ float act_factor(float z) {
  if (ACT == FLP_ACT_GELU) return 0.5f * erfcf(-0.70710678118654752f * z);
  if (ACT == FLP_ACT_GELU_TANH) return sigmoid(kTanhA * z * fmaf(kTanhB * z, z, 1.0f));
  return sigmoid(z);
}
// act'(z) from the factor.
template <int ACT>
__device__ __forceinline__ float act_slope(float z, float f) {
  if (ACT == FLP_ACT_GELU)
    return fmaf(z * 0.39894228040143268f, fast_exp2(-0.5f * kLog2e * z * z), f);
  if (ACT == FLP_ACT_GELU_TANH)
    return fmaf(z * f * (1.0f - f), kTanhA * fmaf(3.0f * kTanhB * z, z, 1.0f), f);
  return f * fmaf(z, 1.0f - f, 1.0f);
}

// What the forward keeps of four consecutive columns of a row: a and b, 12 bytes each (the upper
// halves of their fp32 values, then the next bytes) or, in fp32, 16.
template <class E>
struct Kept {
  static constexpr int kBytes = E::kSize == 2 ? 24 : 32;
  // to 24 bits, to nearest; an infinity or NaN only loses bits that do not make it
  __device__ __forceinline__ static uint32_t round24(float v) {
    const uint32_t b = __float_as_uint(v);
    return (b & 0x7F800000u) == 0x7F800000u ? b : b + 0x80u;
  }
  struct Packed {
    uint32_t h0, h1, lo;
  };
  __device__ __forceinline__ static Packed pack(const f32x4_t& v) {
    const uint32_t b0 = round24(v.x), b1 = round24(v.y), b2 = round24(v.z), b3 = round24(v.w);
    return {(b0 >> 16) | (b1 & 0xFFFF0000u), (b2 >> 16) | (b3 & 0xFFFF0000u),
            ((b0 >> 8) & 0xFFu) | (b1 & 0xFF00u) | ((b2 << 8) & 0xFF0000u) |
                ((b3 << 16) & 0xFF000000u)};
  }
  __device__ __forceinline__ static void store(char* p, const f32x4_t& a, const f32x4_t& b) {
    typedef u32x4 loose16 __attribute__((aligned(8)));
    if constexpr (E::kSize == 2) {
      const Packed u = pack(a), v = pack(b);
      *reinterpret_cast<loose16*>(p) = u32x4{u.h0, u.h1, v.h0, v.h1};
      *reinterpret_cast<u32x2*>(p + 16) = u32x2{u.lo, v.lo};
    } else {
      reinterpret_cast<f32x4_t*>(p)[0] = a;
      reinterpret_cast<f32x4_t*>(p)[1] = b;
    }
  }
  __device__ __forceinline__ static void unpack(uint32_t h0, uint32_t h1, uint32_t lo, float* v) {
    v[0] = __uint_as_float((h0 << 16) | ((lo << 8) & 0xFF00u));
    v[1] = __uint_as_float((h0 & 0xFFFF0000u) | (lo & 0xFF00u));
    v[2] = __uint_as_float((h1 << 16) | ((lo >> 8) & 0xFF00u));
    v[3] = __uint_as_float((h1 & 0xFFFF0000u) | ((lo >> 16) & 0xFF00u));
  }
  // Eight columns: a and b (p a multiple of eight columns: 16-byte aligned).
  __device__ __forceinline__ static void load8(const char* p, float (&a)[8], float (&b)[8]) {
    const u32x4* q = reinterpret_cast<const u32x4*>(p);
    if constexpr (E::kSize == 2) {
      const u32x4 w0 = q[0], w1 = q[1], w2 = q[2];
      unpack(w0.x, w0.y, w1.x, a);
      unpack(w0.z, w0.w, w1.y, b);
      unpack(w1.z, w1.w, w2.z, a + 4);
      unpack(w2.x, w2.y, w2.w, b + 4);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[4 * h + e] = __uint_as_float(q[2 * h][e]);
          b[4 * h + e] = __uint_as_float(q[2 * h + 1][e]);
        }
    }
  }
};

// The B operand of a forward tile of BN rows, CW for each column of waves: of a wave's rows the
// first half are rows of Wg, the second the same rows of Wu.
template <int BN, int NW, int CW>
struct PairTile {
  using Plain = DTile<BN, NW>;
  static constexpr int kHalf = CW / 2;
  static_assert(kHalf % 8 == 0, "an instruction loads eight rows of one weight");
  const char* up;  // first row of the tile in Wu (the base that issue gets is Wg's)
  int q, c0, c1;
  int64_t ld, ks, rows_valid;
  bool full;

  __device__ __forceinline__ void init(int64_t ld_, int64_t ks_, int64_t rows_valid_, int lane,
                                       const char* up_) {
    up = up_;
    ld = ld_;
    ks = ks_;
    rows_valid = rows_valid_;
    full = rows_valid_ >= BN / 2;
    q = lane >> 3;
    c0 = (lane & 7) ^ (q >> 1);
    c1 = c0 ^ 4;
  }
  __device__ __forceinline__ void issue(const char* base, int stage, bool half, u32x4* lds,
                                        int wave) const {
    const int64_t at = int64_t(stage) * ks;
#pragma unroll
    for (int j = 0; j < Plain::kPer; ++j) {
      const int inst = wave * Plain::kPer + j;
      if (Plain::kInsts % NW == 0 || inst < Plain::kInsts) {
        const int first = inst * 8, in = first % CW;
        const char* sb = (in < kHalf ? base : up) + at;
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void*)sb, (short)0, 0x7FFFFFFF, 0x00020000);
        int c = (inst & 1) ? c1 : c0;
        c = half ? (c & 3) : c;
        int64_t r = first / CW * kHalf + in % kHalf + q;
        if (!full) r = r < rows_valid ? r : rows_valid - 1;
        const uint32_t off = uint32_t(r * ld) + uint32_t(c * 16);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void*)(lds + inst * 64), 16, int(off), 0, 0, 0);
      }
    }
  }
};

// Four consecutive values to an address that only fits the element, n of them valid.
template <class E>
__device__ __forceinline__ void store_loose4(void* base, int64_t idx, const f32x4_t& v, int64_t n) {
  if constexpr (E::kSize == 2) {
    typedef u32x2 loose2 __attribute__((aligned(2)));
    uint16_t* p = static_cast<uint16_t*>(base) + idx;
    if (n >= 4) {
      *reinterpret_cast<loose2*>(p) = u32x2{pack2<E>(v.x, v.y), pack2<E>(v.z, v.w)};
    } else {
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < n) p[r] = uint16_t(bits16<E>(v[r]));
    }
  } else {
    typedef f32x4_t loose4 __attribute__((aligned(4)));
    float* p = static_cast<float*>(base) + idx;
    if (n >= 4) {
      *reinterpret_cast<loose4*>(p) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < n) p[r] = v[r];
    }
  }
}

template <class E, int BM, int BN, int WM, int WN, int NS, bool ODD, int ACT>
__global__ __launch_bounds__(64 * WM * WN) void k_gated_fwd(GatedFwdArgs p) {
  using Eng = Engine<E, BM, BN, WM, WN, NS>;
  constexpr int RW = Eng::RW, CW = Eng::CW, WMB = Eng::WMB, WNB = Eng::WNB, kHalf = CW / 2;
  static_assert(WNB % 2 == 0, "a wave holds z and u of the same columns");
  extern __shared__ u32x4 smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM, i = lane & 15, g = lane >> 4;
  constexpr int kCols = BN / 2;
  const int nbm = int((p.N + BM - 1) / BM), nbn = int((p.F + kCols - 1) / kCols);
  int tm, tn;
  tile_of(blockIdx.x, nbm, nbn, tm, tn);
  const int64_t row0 = int64_t(tm) * BM, col0 = int64_t(tn) * kCols;
  const int64_t kbytes = p.D * E::kSize;
  f32x4_t acc[WMB][WNB];
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Eng::template walk<ODD, PairTile<BN, Eng::NW, CW>>(
      acc, static_cast<const char*>(p.x) + row0 * kbytes, kbytes, 128, p.N - row0,
      static_cast<const char*>(p.w_gate) + col0 * kbytes, kbytes, 128, p.F - col0, kbytes, smem,
      static_cast<const char*>(p.w_up) + col0 * kbytes);
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    const int64_t row = row0 + wm * RW + mb * 16 + i;
    if (row >= p.N) continue;
#pragma unroll
    for (int nb = 0; nb < WNB / 2; ++nb) {
      const int64_t col = col0 + wn * kHalf + nb * 16 + 4 * g;
      if (col >= p.F) continue;
      const f32x4_t z = acc[mb][nb], u = acc[mb][nb + WNB / 2];
      f32x4_t a, b;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float f = act_factor<ACT>(z[r]);
        a[r] = z[r] * f;
        b[r] = u[r] * act_slope<ACT>(z[r], f);
      }
      if (p.saved != nullptr)  // rows of a multiple of 64 columns
        Kept<E>::store(static_cast<char*>(p.saved) +
                           (row * p.ld_saved + col) / 4 * Kept<E>::kBytes,
                       a, b);
      store_loose4<E>(p.out, row * p.F + col, a * u, p.F - col);
    }
  }
}

// ---- dz and du, for both products -------------------------------------------------------------
//
// A workgroup takes 64 tokens x 64 columns: whole rows in, and out of LDS the same tile by
// columns (dz: the K of d_x) and by tokens (dzT), each a contiguous K-blocked piece.  The K
// positions of 16-bit operands take the order of launch_transpose, whose results they meet:
// position 32 b + 8 g + 4 h + r holds column (token) 32 b + 16 h + 4 g + r.
// Columns past F and tokens past N are zeros.
template <class E>
struct Elem;
template <>
struct Elem<BF16> {
  using T = __bf16;
};
template <>
struct Elem<F16> {
  using T = _Float16;
};
template <>
struct Elem<F32> {
  using T = float;
};

template <class E>
__global__ __launch_bounds__(256) void k_gated_dz(GatedDzArgs p) {
  using T = typename Elem<E>::T;
  constexpr bool k16 = E::kSize == 2;
  constexpr int kPitch = k16 ? 33 : 65;  // words of a tile row
  __shared__ uint32_t tile[2][64][kPitch];
  const int64_t r0 = int64_t(blockIdx.y) * 64, c0 = int64_t(blockIdx.x) * 64;
  const int t = threadIdx.x;
  {
    const int rl = t >> 2, seg = (t & 3) * 16;
    const int64_t row = r0 + rl;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int cl = seg + half * 8;
      const int64_t n = row < p.N ? p.F - (c0 + cl) : 0;
      Chunk<T> gr;
      gr.load(static_cast<const T*>(p.grad) + row * p.F + c0 + cl, n);
      float a[kChunk], b[kChunk], dz[kChunk], du[kChunk];
      if (n > 0)
        Kept<E>::load8(static_cast<const char*>(p.saved) +
                           (row * p.ld_saved + c0 + cl) / 4 * Kept<E>::kBytes,
                       a, b);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        const float g = float(T(gr.v[e]));
        dz[e] = e < n ? g * b[e] : 0.f;
        du[e] = e < n ? g * a[e] : 0.f;
      }
      if constexpr (k16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          tile[0][rl][cl / 2 + e] = pack2<E>(dz[2 * e], dz[2 * e + 1]);
          tile[1][rl][cl / 2 + e] = pack2<E>(du[2 * e], du[2 * e + 1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          tile[0][rl][cl + e] = __float_as_uint(dz[e]);
          tile[1][rl][cl + e] = __float_as_uint(du[e]);
        }
      }
    }
  }
  __syncthreads();
  const int64_t rows_t = 2 * p.ld_saved;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int64_t k0 = c0 + m * p.ld_saved;  // column of [dz | du], row of its transpose
    if constexpr (k16) {
      uint16_t* const dz = static_cast<uint16_t*>(p.dz);
      uint16_t* const dzT = static_cast<uint16_t*>(p.dzT);
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        const int rl = (t >> 3) + 32 * pass, j = t & 7;
        const int from = 32 * (j >> 2) + 4 * (j & 3);
        if (dz != nullptr && r0 + rl < p.N) {
          const uint32_t* w = tile[m][rl] + from / 2;
          *reinterpret_cast<u32x4*>(dz + kblk<64>(r0 + rl, k0 + 8 * j, p.N)) =
              u32x4{w[0], w[1], w[8], w[9]};
        }
        if (dzT != nullptr) {
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            h[k] = (tile[m][from + 16 * (k >> 2) + (k & 3)][rl >> 1] >> (16 * (rl & 1))) & 0xFFFFu;
          *reinterpret_cast<u32x4*>(dzT + kblk<64>(k0 + rl, r0 + 8 * j, rows_t)) =
              u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                    h[6] | (h[7] << 16)};
        }
      }
    } else {
      uint32_t* const dz = static_cast<uint32_t*>(p.dz);
      uint32_t* const dzT = static_cast<uint32_t*>(p.dzT);
#pragma unroll
      for (int pass = 0; pass < 16; ++pass) {
        const int a = (t >> 6) + 4 * pass, b = t & 63;
        if (dz != nullptr && r0 + a < p.N) dz[kblk<32>(r0 + a, k0 + b, p.N)] = tile[m][a][b];
        if (dzT != nullptr) dzT[kblk<32>(k0 + a, r0 + b, rows_t)] = tile[m][b][a];
      }
    }
  }
}

// ---- launchers ----------------------------------------------------------------------------------

template <class F>
hipError_t by_act(flp_activation act, F f) {
  if (act == FLP_ACT_GELU) return f(std::integral_constant<int, FLP_ACT_GELU>{});
  if (act == FLP_ACT_GELU_TANH) return f(std::integral_constant<int, FLP_ACT_GELU_TANH>{});
  return f(std::integral_constant<int, FLP_ACT_SILU>{});
}

template <class E, int BM, int BN, int WM, int WN, int NS, bool ODD>
hipError_t fwd_cfg(const GatedFwdArgs& a, hipStream_t s) {
  using Eng = Engine<E, BM, BN, WM, WN, NS>;
  return by_act(a.act, [&](auto act) {
    constexpr int kAct = decltype(act)::value;
    static std::atomic<int> ready[kMaxDevices];
    const hipError_t e = prepare(k_gated_fwd<E, BM, BN, WM, WN, NS, ODD, kAct>, Eng::kLds, ready);
    if (e != hipSuccess) return e;
    const int64_t blocks = ((a.N + BM - 1) / BM) * ((a.F + BN / 2 - 1) / (BN / 2));
    hipLaunchKernelGGL((k_gated_fwd<E, BM, BN, WM, WN, NS, ODD, kAct>), dim3(unsigned(blocks)),
                       dim3(Eng::NT), Eng::kLds, s, a);
    return hipGetLastError();
  });
}

template <class E, bool ODD>
hipError_t fwd_rows(const GatedFwdArgs& a, hipStream_t s) {
  auto fills = [&](int64_t bm, int64_t cols) {
    return (a.N + bm - 1) / bm * ((a.F + cols - 1) / cols) >= 160;
  };
  if (a.N > 128 && fills(256, 128)) return fwd_cfg<E, 256, 256, 4, 2, 2, ODD>(a, s);
  if (a.N > 64 && fills(128, 64)) return fwd_cfg<E, 128, 128, 2, 2, 3, ODD>(a, s);
  if (a.N > 32) return fwd_cfg<E, 64, 64, 2, 2, 4, ODD>(a, s);
  return fwd_cfg<E, 32, 64, 2, 2, 4, ODD>(a, s);
}

template <class E>
hipError_t fwd_all(const GatedFwdArgs& a, hipStream_t s) {
  const bool odd = (a.D * E::kSize / kStageBytes) % 2 == 1;
  return odd ? fwd_rows<E, true>(a, s) : fwd_rows<E, false>(a, s);
}

template <class E>
hipError_t dz_all(const GatedDzArgs& a, hipStream_t s) {
  const dim3 grid(unsigned(a.ld_saved / 64), unsigned((a.N + 63) / 64));
  hipLaunchKernelGGL(k_gated_dz<E>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---- products of the backward -----------------------------------------------------------------
//
// The largest tile that gives most compute units a workgroup.  A chain over K is the same in
// every tile, so the tile does not change the bits.

template <class E>
hipError_t dw_all(const GemmArgs& a, hipStream_t s) {
  constexpr bool k16 = E::kSize == 2;
  auto fills = [&](int64_t bm, int64_t bn) {
    return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn) >= 160;
  };
  if constexpr (k16) {
    if (fills(256, 224)) return gemm_cfg<E, 256, 224, 4, 2, false, 0, 2, kGemmNSA, false, true>(a, s);
  }
  if (fills(128, 128)) return gemm_cfg<E, 128, 128, 2, 2, false, 0, k16 ? 3 : 2, k16 ? 3 : 2, false, true>(a, s);
  if (fills(64, 64)) return gemm_cfg<E, 64, 64, 2, 2, false, 0, 4, 4, false, true>(a, s);
  return gemm_cfg<E, 64, 32, 4, 1, false, 0, 8, 8, false, true>(a, s);
}

template <class E>
hipError_t dx_all(const GemmArgs& a, hipStream_t s) {
  constexpr bool k16 = E::kSize == 2;
  if (a.k_slab == 0) {
    if constexpr (k16) return gemm_cfg<E, 256, 224, 4, 2, false, 0, 2, kGemmNSA>(a, s);
    return gemm_cfg<E, 128, 128, 2, 2, false, 0>(a, s);
  }
  const int64_t slabs = (a.K + a.k_slab - 1) / a.k_slab;
  auto fills = [&](int64_t bm, int64_t bn) {
    return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn) * slabs >= 160;
  };
  hipError_t e;
  if (k16 && a.M > 128 && fills(256, 224))
    e = gemm_cfg<E, 256, k16 ? 224 : 128, 4, 2, false, 2, 2, k16 ? kGemmNSA : 2>(a, s);
  else if (a.M > 64 && fills(128, 128))
    e = gemm_cfg<E, 128, 128, 2, 2, false, 2, k16 ? 3 : 2>(a, s);
  else if (a.M > 32 && fills(64, 64))
    e = gemm_cfg<E, 64, 64, 2, 2, false, 2, 4>(a, s);
  else
    e = gemm_cfg<E, 64, 32, 4, 1, false, 2, 8>(a, s);
  if (e != hipSuccess) return e;
  const int64_t n = a.M * a.N;
  hipLaunchKernelGGL(k_slab_fold<E>, dim3(unsigned(std::min<int64_t>((n + 1023) / 1024, 4096))),
                     dim3(256), 0, s, a, int(slabs));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_dx(flp_dtype x, const GemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DHIDDEN, s);
  if (x == FLP_BF16) return dx_all<BF16>(a, s);
  return x == FLP_F16 ? dx_all<F16>(a, s) : dx_all<F32>(a, s);
}

hipError_t launch_gated_dw(flp_dtype x, const GemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DWEIGHT, s);
  if (x == FLP_BF16) return dw_all<BF16>(a, s);
  return x == FLP_F16 ? dw_all<F16>(a, s) : dw_all<F32>(a, s);
}

hipError_t launch_gated_forward(flp_dtype x, const GatedFwdArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_GATED, s);
  if (x == FLP_BF16) return fwd_all<BF16>(a, s);
  return x == FLP_F16 ? fwd_all<F16>(a, s) : fwd_all<F32>(a, s);
}

hipError_t launch_gated_dz(flp_dtype x, const GatedDzArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_GATED, s);
  if (x == FLP_BF16) return dz_all<BF16>(a, s);
  return x == FLP_F16 ? dz_all<F16>(a, s) : dz_all<F32>(a, s);
}

}  // namespace flp
