// gfx950 (CDNA4) kernels of the fused linear selected-token log-probability.
//
// Forward ("Fused Linear LogP" docs page, sections "Backends" and "Reference
// Semantics"): each workgroup computes one [BM x 256] tile of scaled logits
// z = (h W^T + b) / T with bf16 (or fp32) MFMA and fp32 accumulation, folds
// the tile into a per-row (max, sum of exp) pair and picks up the target
// logit; a merge kernel folds the pairs of all vocabulary tiles into lse and
// logp.  The [N, V] logits never reach HBM.
//
// Backward (PR #234, "Implementation details"; PR #555 summary): per row
// chunk, a dlogits kernel recomputes the same logit tiles and writes
// dz = G (onehot - exp(z - lse)) / T row-major and transposed; two GEMMs give
// d_hidden = dz W and d_weight (+)= dz^T hidden, each with one fixed ascending
// K order; d_bias partials are folded in ascending row-tile order.  No atomics.
//
// One MFMA engine serves all four contractions.  Every operand is stored
// K-contiguous (W is transposed once per backward for d_hidden; hidden per
// chunk for d_weight) and streamed by direct global->LDS loads
// (buffer_load_dwordx4 ... lds, no register staging, whole 128-byte lines) into two
// LDS stages of 128 bytes of K per row.  Waves form a WM x WN grid; each wave
// owns a (BM/WM) x (BN/WN) block of 16 x 16 MFMA tiles with fp32 accumulators,
// and double-buffers its operand fragments across the two 64-byte halves of a
// stage.
//
// Register layout: every MFMA is issued as mfma(A = N-side fragment,
// B = M-side fragment), so lane l holds output row (l % 16) of a 16-row block
// and four consecutive output columns 4 (l / 16) + 0..3 of a 16-column block.
// Both fragments are 16 bytes of K read from LDS at (row l % 16, chunk l / 16).
//
// Batch invariance: every logit has the same MFMA chain over K (ascending
// 64-byte steps, same instruction, same lane placement of K) and every
// per-row reduction over a 256-column vocabulary tile uses one fixed tree
// defined by column positions only: in-lane over the 4 columns x 8 column
// blocks a lane holds of each 128-column half, across the four 16-lane groups
// by xor-butterfly (16, then 32), then half 0 + half 1.  No per-row arithmetic
// depends on N, the row tile or the row's position.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include <math.h>

#include "flp_engine.h"
#include "flp_gemm.h"
#include "flp_launch.h"

namespace flp {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTileCols = 256;    // vocabulary tile of the logits kernels
constexpr int kHalfCols = 128;    // columns per wave column in the logits kernels
// The exponent z log2 e - M log2 e as one FMA is off by the rounding of M log2 e.  Beyond
// this size the forward takes the difference z - M first, which is exact for the entries
// that matter (tiles masked with -1e30 or the lowest fp32 value would otherwise overflow the
// exponential), and the cross entropy's backward z - lse with what lse's own rounding left
// out.
constexpr float kHugeLogit = 1e4f;

__device__ __forceinline__ int64_t load_target(const void* t, int t64, int64_t i) {
  return t64 ? reinterpret_cast<const int64_t*>(t)[i] : int64_t(reinterpret_cast<const int32_t*>(t)[i]);
}

// ---- forward: logits tile -> per-row (max, sum of exp) partial + target logit -------------
//
// Workgroup = WM x 2 waves; wave (wm, wn) owns rows [wm*RW, wm*RW + RW) and the 128
// vocabulary columns [wn*128, wn*128 + 128) of the BM x 256 tile.
template <class E, int BM, int WM, int NS = 2>
using LogitEngine = Engine<E, BM, kTileCols, WM, 2, NS>;

// Where a wave's accumulators of a logit tile are kept: every store and load is one
// contiguous KB, and the tile comes back to the lanes it left.
template <int WMB, int WNB>
__device__ __forceinline__ f32x4_t* kept_tile(float* logits, int64_t tile, int waves, int wave,
                                              int lane) {
  return reinterpret_cast<f32x4_t*>(logits) + ((tile * waves + wave) * (WMB * WNB)) * 64 + lane;
}

// The fixed per-row tree over the 32 values one lane holds of a wave's 128 columns.
template <int WNB>
__device__ __forceinline__ float lane_sum(const float (&e)[WNB][4]) {
  static_assert(WNB == 8, "the reduction tree is defined for 8 column blocks per wave");
  float s[WNB];
#pragma unroll
  for (int nb = 0; nb < WNB; ++nb) s[nb] = (e[nb][0] + e[nb][1]) + (e[nb][2] + e[nb][3]);
  return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// LOSS (the cross entropy's forward) adds, when p.zsum is given, the tile's sum of logits
// per row (times p.zunit, a power of two at most 1 / V, so that columns masked with the
// lowest fp32 value cannot overflow it).
// SAVE keeps the products h W^T of the tile in p.logits, in the order of the lanes'
// accumulators (kept_tile), for the dlogits kernel of the same row chunk.  16384 x 2688 x
// 131072 bf16 on MI355X: this kernel 8.7 -> 9.8 ms, k_dz 9.4 -> 3.1 ms (17.2 GB read and
// written, 5.5 TB/s).  It pays where the product costs more than 8 bytes per logit: from
// D of about 1024 on in bf16 (4096 x 1024 x 50257: 2112 and 2104 us a step), in fp32 from
// about 100 on.
template <class E, int BM, int WM, bool ODD, int NS = 2, bool LOSS = false, bool SAVE = false>
__global__ __launch_bounds__(128 * WM) void k_fwd(FwdArgs p) {
  using Eng = LogitEngine<E, BM, WM, NS>;
  constexpr int RW = Eng::RW, WMB = Eng::WMB, WNB = Eng::WNB, NT = Eng::NT;
  extern __shared__ u32x4 smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: tile tests become scalar
  const int wm = wave % WM, wn = wave / WM, i = lane & 15, g = lane >> 4;
  const int nbm = int((p.N + BM - 1) / BM);
  const int nbn = int((p.V + kTileCols - 1) / kTileCols);
  int tm, tn;
  tile_of(blockIdx.x, nbm, nbn, tm, tn);
  const int64_t row0 = int64_t(tm) * BM, col0 = int64_t(tn) * kTileCols;
  const int64_t kbytes = p.D * E::kSize;

  f32x4_t acc[WMB][WNB];
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Eng::template run<ODD>(acc, reinterpret_cast<const char*>(p.hidden) + row0 * kbytes, kbytes, p.N - row0,
           reinterpret_cast<const char*>(p.weight) + col0 * kbytes, kbytes, p.V - col0, kbytes,
           smem);
  if constexpr (SAVE) {
    f32x4_t* keep = kept_tile<WMB, WNB>(p.logits, int64_t(tm) * nbn + tn, 2 * WM, wave, lane);
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
        __builtin_nontemporal_store(acc[mb][nb], keep + (mb * WNB + nb) * 64);
  }
  // Waves still reading their last fragments after the last stage barrier may read
  // either buffer (buffer 0 when the stage count is odd): LDS is reused below.
  __syncthreads();

  // [2][BM] row max of y = h W^T + b per wave column, [2][BM] row sums, [BM] row max of z
  // (LOSS: and [2][BM] row sums of logits)
  static_assert(7 * BM * sizeof(float) <= Eng::kLds, "the row reductions fit the operand ring");
  float* red = reinterpret_cast<float*>(smem);
  const int64_t cw = col0 + wn * kHalfCols;
  // Columns of this wave at or past lim are vocabulary padding (lim < 128 only in
  // the last vocabulary tile).
  const int lim = int(p.V - cw < kHalfCols ? p.V - cw : kHalfCols);
  float bcol[WNB][4];
#pragma unroll
  for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
    for (int r = 0; r < 4; ++r) bcol[nb][r] = 0.f;
  if (p.bias != nullptr) {
    const float* bw = p.bias + cw + 4 * g;
    if (lim == kHalfCols) {  // wave-uniform: every column of the wave exists
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) bcol[nb][r] = bw[nb * 16 + r];
    } else {
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (nb * 16 + 4 * g + r < lim) bcol[nb][r] = bw[nb * 16 + r];
    }
  }

  // The logits are z = y / T with y = h W^T + b; the accumulators become y and 1/T
  // enters through the exp argument's FMA.
  // The row max of z is the row max of y times 1/T, bit for bit: rounding is
  // monotone, so max_j fl(y_j / T) = fl(max_j(y_j) / T).
  float invT[WMB];
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    const int rl = wm * RW + mb * 16 + i;
    const int64_t row = row0 + rl;
    invT[mb] = (p.temperature != nullptr && row < p.N) ? 1.0f / p.temperature[row] : 1.0f;
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[mb][nb][r] += bcol[nb][r];
    if constexpr (LOSS) {
      if (p.zsum != nullptr) {
        float zs = 0.f;
#pragma unroll
        for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (lim == kHalfCols || nb * 16 + 4 * g + r < lim)
              zs = fmaf(acc[mb][nb][r], p.zunit, zs);
        f32x2_t q = pair16(zs);
        zs = q.x + q.y;
        q = pair32(zs);
        if (g == 0) red[5 * BM + wn * BM + rl] = q.x + q.y;
      }
    }
    if (lim < kHalfCols) {  // the last vocabulary tile: padding columns drop out
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (nb * 16 + 4 * g + r >= lim) acc[mb][nb][r] = -INFINITY;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) mx = fmaxf(mx, acc[mb][nb][r]);
    f32x2_t q = pair16(mx);
    mx = fmaxf(q.x, q.y);
    q = pair32(mx);
    mx = fmaxf(q.x, q.y);
    if (g == 0) red[wn * BM + rl] = mx;
  }
  __syncthreads();
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    const int rl = wm * RW + mb * 16 + i;
    const int64_t row = row0 + rl;
    const float M = fmaxf(red[rl], red[BM + rl]) * invT[mb];  // row max of z
    // Without a finite logit or +inf in the tile's row, M is -inf and the exponents are taken
    // as they are: entries of -inf then add 0 and NaN entries make the tile's sum NaN.
    const float base = M == -INFINITY ? 0.f : M;
    const float Ml = base * kLog2e;
    const float k = invT[mb] * kLog2e;
    if (wn == 0 && g == 0) red[4 * BM + rl] = M;
    // exp(z - M) = 2^(y (log2 e / T) - M log2 e): one FMA per logit
    float e[WNB][4];
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) e[nb][r] = fast_exp2(fmaf(acc[mb][nb][r], k, -Ml));
    if (fabsf(M) > kHugeLogit) {
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          e[nb][r] = fast_exp2((acc[mb][nb][r] * invT[mb] - base) * kLog2e);
    }
    float s = lane_sum<WNB>(e);
    f32x2_t q = pair16(s);
    s = q.x + q.y;
    q = pair32(s);
    s = q.x + q.y;
    if (g == 0) red[2 * BM + wn * BM + rl] = s;
    if (row < p.N) {
      const int64_t t = load_target(p.targets, p.t64, row) - p.t_off;
      const int64_t rel = t - cw;
      if (t >= 0 && t < p.V && rel >= 0 && rel < kHalfCols && int((rel & 15) >> 2) == g) {
        const int tnb = int(rel >> 4), tr = int(rel & 3);
        float yt = 0.f;
#pragma unroll
        for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) yt = (nb == tnb && r == tr) ? acc[mb][nb][r] : yt;
        p.zt[row] = yt * invT[mb];
      }
    }
  }
  __syncthreads();
  for (int rl = tid; rl < BM; rl += NT) {
    const int64_t row = row0 + rl;
    if (row < p.N) {
      const float M = red[4 * BM + rl];
      const float S = red[2 * BM + rl] + red[3 * BM + rl];
      p.part[int64_t(tn) * p.N + row] = make_float2(M, S);
      if constexpr (LOSS) {
        if (p.zsum != nullptr)
          p.zsum[int64_t(tn) * p.N + row] = red[5 * BM + rl] + red[6 * BM + rl];
      }
    }
  }
}

// ---- merge: per-tile pairs -> lse, logp ------------------------------------------------------
//
// The row max M is the largest tile max (exact in any order).  The sum
// S = sum_t s_t 2^((m_t - M) log2 e) runs over 256 leaves: leaf j adds the tiles
// [j L, j L + L) (L = ceil(n_vt / 256)) in ascending order, and the leaves are
// added by a complete binary tree (pairs, pairs of pairs, ...).  Both depend on the
// vocabulary only, so a row gets the same bits whatever the batch and whichever
// of the two workgroup shapes below merges it: R = 1 row per workgroup (one leaf
// per thread, for small batches) or R = 8 rows (eight leaves per thread).  The tree
// levels inside a wave are xor butterflies over the lanes of one row (addition is
// commutative, so both partners hold the same bits), the last two levels combine
// the four waves.  LL = tiles per leaf when they fit in registers (1 or 2), else 0:
// the tiles are then read twice (max, then sum).
constexpr int kMergeLeaves = 256;
constexpr int64_t kMergeRowMax = 2048;  // batches up to this size: one row per workgroup

// A tile of nothing but -inf has the sum 0; one of -inf and NaN has the sum NaN, which has to
// reach the row's.
__device__ __forceinline__ float merge_term(float2 q, float M) {
  return q.x == -INFINITY ? q.y : q.y * fast_exp2((q.x - M) * kLog2e);
}

//
// LOSS (the cross entropy): the tiles' sums of logits (p.zsum, if any) are added over
// the same leaves and tree, and the row's loss is written instead of logp:
//   loss = (1 - s) (lse - z_t) + s (lse - mean z) + c lse^2,  0 for an ignored target.
template <int R, int LL, bool LOSS = false>
__global__ __launch_bounds__(256) void k_merge(MergeArgs p) {
  constexpr int P = kMergeLeaves / (256 / R);  // leaves per thread
  __shared__ float sm[4][R], ss[4][R], sz[4][R];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rl = tid % R, c = tid / R;  // row in the workgroup, thread of the row
  const int64_t row = int64_t(blockIdx.x) * R + rl;
  const bool live = row < p.N;
  const int64_t L = (p.n_vt + kMergeLeaves - 1) / kMergeLeaves;
  const int64_t v0 = int64_t(c) * P * L, v1 = min(p.n_vt, v0 + P * L);
  const bool fin = c == 0 && live;
  int64_t t = -1;
  float zt = 0.f;
  if (fin) {
    t = load_target(p.targets, p.t64, row);
    zt = p.zt[row];
  }
  auto tile = [&](int64_t v) {
    return (live && v < v1) ? p.part[v * p.N + row] : make_float2(-INFINITY, 0.f);
  };
  float2 q[LL > 0 ? P * LL : 1];
  float m = -INFINITY;
  if constexpr (LL > 0) {
#pragma unroll
    for (int u = 0; u < P * LL; ++u) q[u] = tile(v0 + u);
#pragma unroll
    for (int u = 0; u < P * LL; ++u) m = fmaxf(m, q[u].x);
  } else {
    for (int64_t v = v0; v < v1; ++v) m = fmaxf(m, tile(v).x);
  }
#pragma unroll
  for (int k = R; k < 64; k <<= 1) m = fmaxf(m, lane_xor(m, k));
  if (lane < R) sm[wave][rl] = m;
  __syncthreads();
  const float M = fmaxf(fmaxf(sm[0][rl], sm[1][rl]), fmaxf(sm[2][rl], sm[3][rl]));
  float l[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if constexpr (LL > 0) {
      l[k] = merge_term(q[k * LL], M);
#pragma unroll
      for (int j = 1; j < LL; ++j) l[k] += merge_term(q[k * LL + j], M);
    } else {
      l[k] = 0.f;
      for (int64_t v = v0 + k * L; v < v0 + (k + 1) * L; ++v) l[k] += merge_term(tile(v), M);
    }
  }
  float sum;
  if constexpr (P == 8)
    sum = ((l[0] + l[1]) + (l[2] + l[3])) + ((l[4] + l[5]) + (l[6] + l[7]));
  else
    sum = l[0];
#pragma unroll
  for (int k = R; k < 64; k <<= 1) sum += lane_xor(sum, k);
  if (lane < R) ss[wave][rl] = sum;
  if constexpr (LOSS) {
    if (p.zsum != nullptr) {  // uniform over the launch
      float z[P];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        z[k] = 0.f;
        for (int64_t v = v0 + k * L; v < v0 + (k + 1) * L; ++v)
          z[k] += (live && v < v1) ? p.zsum[v * p.N + row] : 0.f;
      }
      float zs;
      if constexpr (P == 8)
        zs = ((z[0] + z[1]) + (z[2] + z[3])) + ((z[4] + z[5]) + (z[6] + z[7]));
      else
        zs = z[0];
#pragma unroll
      for (int k = R; k < 64; k <<= 1) zs += lane_xor(zs, k);
      if (lane < R) sz[wave][rl] = zs;
    }
  }
  __syncthreads();
  if (fin) {
    const float S = (ss[0][rl] + ss[1][rl]) + (ss[2][rl] + ss[3][rl]);
    const float ls = logf(S);
    const bool valid = t >= 0 && t < p.V;
    if constexpr (LOSS) {
      float loss = 0.f;
      if (valid) {
        const float lse = M + ls;
        loss = ls - (zt - M);
        if (p.zsum != nullptr) {
          const float zs = (sz[0][rl] + sz[1][rl]) + (sz[2][rl] + sz[3][rl]);
          loss = fmaf(1.0f - p.smoothing, loss, p.smoothing * (lse - zs * p.zmean));
        }
        if (p.z_loss != 0.f) loss = fmaf(p.z_loss * lse, lse, loss);
      }
      p.loss[row] = loss;
    } else {
      p.logp[row] = valid ? (zt - M) - ls : 0.0f;
    }
    if (p.lse != nullptr) p.lse[row] = M + ls;
    // what that sum's rounding left out (exact: |M| >= |ls| wherever it matters)
    if (p.lse_rest != nullptr) p.lse_rest[row] = ls - ((M + ls) - M);
  }
}

__global__ __launch_bounds__(256) void k_fill(float* dst, int64_t n, float value) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) dst[i] = value;
}

// ---- the operator on materialised logits ----------------------------------------------------
//
// One wave per row, four rows per workgroup.  Lane l owns the 16-byte chunks
// l, l + 64, l + 128, ... of its row and keeps an online (max, sum of exp) over
// them in chunk order; the 64 lane pairs are then combined by a xor butterfly
// whose combine step is symmetric, so every lane ends with the same bits.  The
// row is read once with streaming loads, four chunks per lane in flight.
// Where a maximum is -inf the exponents are taken as they are: entries of -inf add 0
// (a lane may hold nothing else) and NaN entries make the sum NaN.

template <class E>
__device__ __forceinline__ void unpack8(const u32x4& v, float (&x)[8]);
template <>
__device__ __forceinline__ void unpack8<BF16>(const u32x4& v, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(v[k] << 16);
    x[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void unpack8<F16>(const u32x4& v, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = float(__builtin_bit_cast(_Float16, uint16_t(v[k] & 0xFFFFu)));
    x[2 * k + 1] = float(__builtin_bit_cast(_Float16, uint16_t(v[k] >> 16)));
  }
}

template <class E>
__device__ __forceinline__ float load_elem(const void* base, int64_t i);
template <>
__device__ __forceinline__ float load_elem<BF16>(const void* base, int64_t i) {
  return __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(base)[i]) << 16);
}
template <>
__device__ __forceinline__ float load_elem<F16>(const void* base, int64_t i) {
  return float(reinterpret_cast<const _Float16*>(base)[i]);
}
template <>
__device__ __forceinline__ float load_elem<F32>(const void* base, int64_t i) {
  return reinterpret_cast<const float*>(base)[i];
}

template <class E>
__global__ __launch_bounds__(256) void k_logits_fwd(LogitsArgs p) {
  constexpr int EPC = 16 / E::kSize;  // elements per 16-byte chunk
  constexpr int kBatch = 4;
  const int lane = threadIdx.x & 63;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= p.N) return;
  if (p.mask != nullptr && p.mask[row] == 0) {  // a row left out by an indexed call
    if (lane == 0) {
      p.logp[row] = 0.0f;
      if (p.lse_out != nullptr) p.lse_out[row] = 0.0f;
    }
    return;
  }
  const int64_t nch = p.V / EPC;
  const u32x4* src =
      reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p.logits) + row * p.V * E::kSize);
  float M = -INFINITY, S = 0.f;
  for (int64_t c0 = lane; c0 < nch; c0 += 64 * kBatch) {
    u32x4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (c0 + u * 64 < nch) v[u] = __builtin_nontemporal_load(src + c0 + u * 64);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (c0 + u * 64 >= nch) break;
      float x[EPC];
      if constexpr (E::kSize == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(v[u][k]);
      } else {
        unpack8<E>(v[u], x);
      }
      float cm = x[0];
#pragma unroll
      for (int k = 1; k < EPC; ++k) cm = fmaxf(cm, x[k]);
      const float Mn = fmaxf(M, cm);
      const float base = Mn == -INFINITY ? 0.f : Mn;
      float e = 0.f;
#pragma unroll
      for (int k = 0; k < EPC; ++k) e += fast_exp2((x[k] - base) * kLog2e);
      S = S * fast_exp2((M - base) * kLog2e) + e;
      M = Mn;
    }
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const float Mo = __shfl_xor(M, off), So = __shfl_xor(S, off);
    const float Mn = fmaxf(M, Mo);
    const float base = Mn == -INFINITY ? 0.f : Mn;
    const float a = S * fast_exp2((M - base) * kLog2e);
    const float b = So * fast_exp2((Mo - base) * kLog2e);
    S = a + b;
    M = Mn;
  }
  if (lane != 0) return;
  const float ls = logf(S);
  const int64_t t = load_target(p.targets, p.t64, row);
  const bool valid = t >= 0 && t < p.V;
  const float zt = valid ? load_elem<E>(p.logits, row * p.V + t) : 0.f;
  p.logp[row] = valid ? (zt - M) - ls : 0.0f;
  if (p.lse_out != nullptr) p.lse_out[row] = M + ls;
}

template <class E>
__global__ __launch_bounds__(256) void k_logits_bwd(LogitsArgs p) {
  constexpr int EPC = 16 / E::kSize;
  constexpr int kBatch = 4;
  const int lane = threadIdx.x & 63;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= p.N) return;
  const int64_t nch = p.V / EPC;
  const u32x4* src =
      reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p.logits) + row * p.V * E::kSize);
  u32x4* dst = reinterpret_cast<u32x4*>(reinterpret_cast<char*>(p.d_logits) + row * p.V * E::kSize);
  if (p.mask != nullptr && p.mask[row] == 0) {  // a row left out by an indexed call: zero gradient
    const u32x4 z = {0u, 0u, 0u, 0u};
    for (int64_t c = lane; c < nch; c += 64) __builtin_nontemporal_store(z, dst + c);
    return;
  }
  const int64_t t = load_target(p.targets, p.t64, row);
  const bool valid = t >= 0 && t < p.V;
  const float G = valid ? p.grad_out[row] : 0.f;
  const float L = p.lse[row];
  for (int64_t c0 = lane; c0 < nch; c0 += 64 * kBatch) {
    u32x4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (c0 + u * 64 < nch) v[u] = __builtin_nontemporal_load(src + c0 + u * 64);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t c = c0 + u * 64;
      if (c >= nch) break;
      float x[EPC], d[EPC];
      if constexpr (E::kSize == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(v[u][k]);
      } else {
        unpack8<E>(v[u], x);
      }
#pragma unroll
      for (int k = 0; k < EPC; ++k) {
        const float pr = fast_exp2((x[k] - L) * kLog2e);
        const float oh = (c * EPC + k == t) ? 1.0f : 0.0f;
        d[k] = valid ? G * (oh - pr) : 0.0f;
      }
      u32x4 w;
      if constexpr (E::kSize == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(d[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack2<E>(d[2 * k], d[2 * k + 1]);
      }
      __builtin_nontemporal_store(w, dst + c);
    }
  }
}

// ---- dlogits: recompute the logit tile, dz = G (onehot - p) / T, d_bias partials ------------
//
// dz is written token-major (the A operand of d_hidden = dz W) and transposed (the
// A operand of d_weight = dz^T hidden), both in the K-blocked layout of the GEMM
// operands.  16-bit inputs write them straight from the registers, every wave
// store instruction one contiguous 1 KB run (8 rows x one 128-byte K block).
//
// dz is rounded once to the inputs' type there (fp32 inputs: not at all), since the
// products' matrix instructions take both operands in one type: with fp32 dz they would run
// at an eighth of the rate (library products on MI355X: 154 TFLOP/s, bf16 1185) and twice
// as much would be written and read.  d_bias adds the unrounded entries.
//
// K order.  Within every 32-wide block of K, the 16-bit backward GEMMs take their K
// positions in the order
//   K position 32 b + 8 g + 4 h + r  <->  index 32 b + 16 h + 4 g + r
// (g, r = 0..3; h = 0, 1) of the vocabulary (d_hidden) or token (d_weight)
// dimension: the order in which a lane of the logit tile holds its values, so that
// each lane's eight values of two adjacent 16-column blocks form one 16-byte chunk
// of K.  The transposes of W and of hidden (k_transpose16) apply the same order, so
// every product pairs the same dz, W and hidden entries as in the natural order.

// LOSS (the cross entropy's backward): dz = c p + onehot o + u with the per-row factors
// p.grad_out (c), p.onehot (o) and p.uniform (u); no temperature.
// KEPT: the tile's products come from p.logits, where the chunk's forward left them, and
// are not recomputed; everything after them is the same code, so dz has the same bits.
template <class E, int BM, int WM, bool ODD, bool LOSS = false, bool KEPT = false,
          int BN = kTileCols>
__global__ __launch_bounds__(128 * WM) void k_dz(DzArgs p) {
  using Eng = Engine<E, BM, BN, WM, 2>;
  constexpr int kHalf = BN / 2;  // columns of a wave
  constexpr int RW = Eng::RW, WMB = Eng::WMB, WNB = Eng::WNB, NT = Eng::NT;
  constexpr bool kDirect = E::kSize == 2;  // 16-bit: stores straight from the registers
  static_assert(!kDirect || (BM == kTileCols && BN == kTileCols && WM == 4),
                "the 16-bit store path is laid out for the 256 x 256 tile with 4 x 2 waves");
  extern __shared__ u32x4 smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: tile tests become scalar
  const int wm = wave % WM, wn = wave / WM, i = lane & 15, g = lane >> 4;
  const int nbm = int((p.rows + BM - 1) / BM);
  const int nbn = int(p.ldz / BN);  // the vocabulary padded to whole 256-column tiles
  int tm, tn;
  tile_of(blockIdx.x, nbm, nbn, tm, tn);
  const int64_t row0 = int64_t(tm) * BM, col0 = int64_t(tn) * BN;
  const int64_t kbytes = p.D * E::kSize;

  f32x4_t acc[WMB][WNB];
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if constexpr (KEPT) {
    const f32x4_t* keep = kept_tile<WMB, WNB>(p.logits, int64_t(tm) * nbn + tn, 2 * WM, wave, lane);
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
        acc[mb][nb] = __builtin_nontemporal_load(keep + (mb * WNB + nb) * 64);
  } else if (BN == kTileCols || col0 < p.V) {
    Eng::template run<ODD>(acc, reinterpret_cast<const char*>(p.hidden) + row0 * kbytes, kbytes,
                           p.rows - row0, reinterpret_cast<const char*>(p.weight) + col0 * kbytes,
                           kbytes, p.V - col0, kbytes, smem);
  }

  const int64_t cw = col0 + wn * kHalf;
  // Columns of this wave at or past lim are vocabulary padding (lim < 128 only in
  // the last vocabulary tile).
  const int lim = int(p.V - cw < kHalf ? p.V - cw : kHalf);
  f32x4_t csum[WNB];
  // The per-row inputs of the wave's rows and the bias are all loaded before the
  // first of them is used (rows past the batch read the last row, whose values are
  // then not used), so the epilogue waits for one memory round trip, not one per
  // input and row block.  The branches are wave-uniform and outside the row loops.
  auto rowc = [&](int mb) {
    const int64_t row = row0 + wm * RW + mb * 16 + i;
    return row < p.rows ? row : p.rows - 1;
  };
  float rtemp[WMB], rgrad[WMB], rlse[WMB];
  int64_t rt64[WMB];
  int32_t rt32[WMB];
  if (p.t64) {
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb) {
      rt64[mb] = reinterpret_cast<const int64_t*>(p.targets)[rowc(mb)];
      rt32[mb] = 0;
    }
  } else {
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb) {
      rt32[mb] = reinterpret_cast<const int32_t*>(p.targets)[rowc(mb)];
      rt64[mb] = 0;
    }
  }
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    rgrad[mb] = p.grad_out[rowc(mb)];
    rlse[mb] = p.lse[rowc(mb)];
    rtemp[mb] = 1.0f;
  }
  float ronehot[WMB], runif[WMB], rrest[WMB];  // LOSS only
  if constexpr (LOSS) {
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb) {
      ronehot[mb] = p.onehot[rowc(mb)];
      runif[mb] = p.uniform[rowc(mb)];
      rrest[mb] = p.lse_rest[rowc(mb)];
    }
  } else if (p.temperature != nullptr) {
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb) rtemp[mb] = p.temperature[rowc(mb)];
  }
  float bcol[WNB][4];
#pragma unroll
  for (int nb = 0; nb < WNB; ++nb) {
    csum[nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r) bcol[nb][r] = 0.f;
  }
  if (p.bias != nullptr) {
    const float* bw = p.bias + cw + 4 * g;
    if (lim == kHalf) {  // wave-uniform: every column of the wave exists
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) bcol[nb][r] = bw[nb * 16 + r];
    } else {
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (nb * 16 + 4 * g + r < lim) bcol[nb][r] = bw[nb * 16 + r];
    }
  }
  // Nothing computed from the per-row inputs may move above this point (it would
  // wait for them in front of the bias loads).
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb)
    asm volatile("" : "+v"(rt32[mb]), "+v"(rt64[mb]), "+v"(rtemp[mb]), "+v"(rgrad[mb]), "+v"(rlse[mb]));
  // Per row block: k = log2(e) / T, L log2(e), G = grad / T (0 for an ignored target)
  // and the target's column within the wave (-1: not among its columns, -2: ignored).
  float rk[WMB], rl[WMB], rg[WMB];
  int rtc[WMB];
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    const int64_t row = row0 + wm * RW + mb * 16 + i;
    const bool rv = row < p.rows;
    const float invT = (p.temperature != nullptr && rv) ? 1.0f / rtemp[mb] : 1.0f;
    const int64_t t = !rv ? -1 : p.t64 ? rt64[mb] : int64_t(rt32[mb]);
    const bool valid = t >= 0 && t < p.V;
    rg[mb] = valid ? rgrad[mb] * invT : 0.f;
    rl[mb] = (rv ? rlse[mb] : 0.f) * (LOSS ? 1.0f : kLog2e);
    rk[mb] = invT * kLog2e;
    const int64_t trel = t - cw;
    rtc[mb] = !valid ? -2 : (trel >= 0 && trel < kHalf) ? int(trel) : -1;
  }
  {
    // dz = G (onehot - exp(z - lse)) / T, kept in the accumulator registers, with
    // z = y / T, y = h W^T + b: the accumulators become y, and
    // exp(z - lse) = 2^(y (log2 e / T) - lse log2 e) is one FMA and one exp2 per logit.
#pragma unroll
    for (int mb = 0; mb < WMB; ++mb) {
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[mb][nb][r] += bcol[nb][r];
      const int64_t row = row0 + wm * RW + mb * 16 + i;
      const float G = rg[mb], k = rk[mb], Ll = rl[mb];
      const bool valid = rtc[mb] != -2;
      const int tcol = rtc[mb] >= 0 ? rtc[mb] : -1;
      // Every kept logit is G (0 - p) = (-G) p (bit for bit, except that a p that
      // underflows to 0 gives a zero of the other sign); the target's entry,
      // G (1 - p), is taken from the row's logit before the tile is overwritten.
      // Few rows of a wave have their target among its 128 columns, so that part
      // runs under a branch most waves skip.
      float vt = 0.f;
      if (LOSS) {
        // The softmax in place of the logits, then one FMA per entry.
        const float L = rl[mb];
        if (fabsf(L) > kHugeLogit) {
#pragma unroll
          for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[mb][nb][r] = fast_exp2(((acc[mb][nb][r] - L) - rrest[mb]) * kLog2e);
        } else {
          const float Lk = L * kLog2e;
#pragma unroll
          for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[mb][nb][r] = fast_exp2(fmaf(acc[mb][nb][r], kLog2e, -Lk));
        }
        const float o = ronehot[mb] + runif[mb];
        if (tcol >= 0) {
#pragma unroll
          for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (nb * 16 + 4 * g + r == tcol) vt = fmaf(G, acc[mb][nb][r], o);
        }
      } else if (tcol >= 0) {
        float yt = 0.f;
#pragma unroll
        for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (nb * 16 + 4 * g + r == tcol) yt = acc[mb][nb][r];
        vt = G * (1.0f - fast_exp2(fmaf(yt, k, -Ll)));
      }
      const float nG = -G;
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[mb][nb][r] = LOSS ? fmaf(G, acc[mb][nb][r], runif[mb])
                                : nG * fast_exp2(fmaf(acc[mb][nb][r], k, -Ll));
      if (tcol >= 0) {
#pragma unroll
        for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (nb * 16 + 4 * g + r == tcol) acc[mb][nb][r] = vt;
      }
      // Rows with an ignored target and the vocabulary padding get zeros (+0).
      if (!valid) {
#pragma unroll
        for (int nb = 0; nb < WNB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      if (lim < kHalf) {  // wave-uniform: the last vocabulary tile only
#pragma unroll
        for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (nb * 16 + 4 * g + r >= lim) acc[mb][nb][r] = 0.f;
      }
#pragma unroll
      for (int nb = 0; nb < WNB; ++nb) {
        const f32x4_t d = acc[mb][nb];
        csum[nb] += d;
        if constexpr (!kDirect) {
          constexpr int KB = 128 / E::kSize;
          const int64_t c = cw + nb * 16 + 4 * g;
          if (p.dz != nullptr) store4<E>(p.dz, kblk<KB>(row, c, p.ldt), d);
          if (p.dzT != nullptr) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int64_t at = kblk<KB>(c + r, row, p.ldz);
              if constexpr (E::kSize == 4)
                reinterpret_cast<float*>(p.dzT)[at] = d[r];
              else
                reinterpret_cast<uint16_t*>(p.dzT)[at] = uint16_t(bits16<E>(d[r]));
            }
          }
        }
      }
    }
  }
  if constexpr (kDirect) {
    // Lane (i, g) holds, for row block mb and the column blocks 2 c, 2 c + 1 of its
    // wave, token i at the vocabulary columns 32 c + 16 h + 4 g + r: in the K order
    // above, chunk g of the 32-wide step c of that token (16 bytes).
    //
    // dz^T: an MFMA multiplies such a chunk by a 0/1 matrix selecting 16 of its 32
    // columns (column 16 e + n for output column n), which lays the 16 x 16 block out
    // column-wise: lane (n, g) gets column 16 e + n at tokens 4 g + r.  A 16-bit value
    // times 1 plus zeros is exact in fp32, so these are the same bits.  The row blocks
    // 2 q and 2 q + 1 together give the tokens 32 q + 16 h + 4 g + r of one column:
    // chunk g of its 32-wide token step q.
    //
    // Stores.  A 128-byte K block is two such steps.  Lane i < 8 holds chunk g of
    // step 0 (X) for row i, lane i + 8 the same for row i + 8; their step-1 chunks
    // (Y) are swapped between the two lanes (lane i ^ 8, a DPP row rotation), after
    // which one store covers rows 0..7 (lanes i < 8: X at chunk g, lanes i >= 8: the
    // partner's Y at chunk 4 + g) and another rows 8..15: 8 rows x 128 bytes each.
    constexpr uint32_t kOne = std::is_same<E, F16>::value ? 0x3C00u : 0x3F80u;  // 1.0
    // The selection B operand: lane (n, g) supplies rows 8 g .. 8 g + 7 of column n,
    // and column n selects K slot 8 (n >> 2) + 4 e + (n & 3).
    u32x4 sel[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int jj = g == (i >> 2) ? 4 * e + (i & 3) : -1;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        sel[e][w] = (jj == 2 * w ? kOne : 0u) | (jj == 2 * w + 1 ? kOne << 16 : 0u);
    }
    const bool lo = i < 8;
    // Element offsets, within one 16-row block and one 128-byte K block, of this
    // lane's 16 bytes in the store of rows 0..7 (o0) and of rows 8..15 (o1).
    const int o0 = (i & 7) * 64 + (lo ? g : 4 + g) * 8;
    const int o1 = o0 + 8 * 64 + (lo ? 32 : -32);
    // The swap is a DPP row rotation by 8 whose bank mask writes only the lanes that
    // take the partner's value (banks 2 and 3 = lanes 8..15 for the first store,
    // banks 0 and 1 for the second); the other lanes keep x.
    auto store_pair = [&](uint16_t* base, const u32x4& x, const u32x4& y) {
      u32x4 s0, s1;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        s0[w] = uint32_t(__builtin_amdgcn_update_dpp(int(x[w]), int(y[w]), 0x128, 0xF, 0xC, false));
        s1[w] = uint32_t(__builtin_amdgcn_update_dpp(int(x[w]), int(y[w]), 0x128, 0xF, 0x3, false));
      }
      __builtin_nontemporal_store(s0, reinterpret_cast<u32x4*>(base + o0));
      __builtin_nontemporal_store(s1, reinterpret_cast<u32x4*>(base + o1));
    };
    uint16_t* const dz = reinterpret_cast<uint16_t*>(p.dz);
    uint16_t* const dzT = reinterpret_cast<uint16_t*>(p.dzT);
    const int64_t tw = row0 + wm * RW;  // first token of this wave's rows (a multiple of 64)
#pragma unroll
    for (int b = 0; b < WNB / 4; ++b) {  // the two 128-byte K blocks of the wave's 128 columns
      u32x4 f[WMB][2];
#pragma unroll
      for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int nb = 4 * b + 2 * cc;
          f[mb][cc].x = pack2<E>(acc[mb][nb][0], acc[mb][nb][1]);
          f[mb][cc].y = pack2<E>(acc[mb][nb][2], acc[mb][nb][3]);
          f[mb][cc].z = pack2<E>(acc[mb][nb + 1][0], acc[mb][nb + 1][1]);
          f[mb][cc].w = pack2<E>(acc[mb][nb + 1][2], acc[mb][nb + 1][3]);
        }
      if (dz != nullptr) {
        const int64_t kb = (cw + 64 * b) / 64;  // K block of columns cw + 64 b .. + 63
#pragma unroll
        for (int mb = 0; mb < WMB; ++mb)
          store_pair(dz + (kb * p.ldt + tw + mb * 16) * 64, f[mb][0], f[mb][1]);
      }
      if (dzT != nullptr) {
#pragma unroll
        for (int cc = 0; cc < 2; ++cc)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            u32x4 t[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              f32x4_t u0 = {0.f, 0.f, 0.f, 0.f}, u1 = {0.f, 0.f, 0.f, 0.f};
              mma64<E>(u0, f[2 * q][cc], sel[e]);
              mma64<E>(u1, f[2 * q + 1][cc], sel[e]);
              t[q] = u32x4{pack2<E>(u0[0], u0[1]), pack2<E>(u0[2], u0[3]), pack2<E>(u1[0], u1[1]),
                           pack2<E>(u1[2], u1[3])};
            }
            // rows: vocabulary columns cw + 64 b + 32 cc + 16 e + 0..15; K block: the
            // wave's 64 tokens
            const int64_t vrow = cw + 64 * b + 32 * cc + 16 * e;
            store_pair(dzT + ((tw / 64) * p.ldz + vrow) * 64, t[0], t[1]);
          }
      }
    }
  }
  if (p.dbias_part == nullptr) return;
  // Column sums over the tile's rows: in-lane over row blocks, then over the 16
  // lanes holding the other rows, then ascending over row waves.  The 16-lane step
  // is a reduce-scatter: a lane holds 32 column values (j = 4 nb + r); at the step
  // over lane bit m it keeps the half of its values that bit selects and adds the
  // partner's copy of that half, so after the four steps lane i holds the finished
  // sums of columns j = 2i and 2i + 1 (30 exchanges instead of 128).  With fewer values
  // than lanes (a narrow tile) the last steps add the one value left in both partners.
  constexpr int kVals = 4 * WNB, kLeft = kVals > 16 ? kVals / 16 : 1;
  static_assert((WNB & (WNB - 1)) == 0, "the column reduction halves the values per lane");
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);  // [WM][BN]
  {
    float v[kVals];
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * nb + r] = csum[nb][r];
#pragma unroll
    for (int h = kVals / 2, m = 8; m >= 1; h >>= 1, m >>= 1) {
      if (h == 0) {
        v[0] += lane_xor(v[0], m);
        continue;
      }
      const bool up = (i & m) != 0;
#pragma unroll
      for (int k = 0; k < h; ++k) {
        const float send = up ? v[k] : v[k + h];
        const float keep = up ? v[k + h] : v[k];
        v[k] = keep + lane_xor(send, m);
      }
    }
#pragma unroll
    for (int e = 0; e < kLeft; ++e) {
      const int j = kVals >= 16 ? kLeft * i + e : i * kVals / 16;
      red[wm * BN + wn * kHalf + (j >> 2) * 16 + 4 * g + (j & 3)] = v[e];
    }
  }
  __syncthreads();
  for (int c = tid; c < BN; c += NT) {
    float s = red[c];
#pragma unroll
    for (int w = 1; w < WM; ++w) s += red[w * BN + c];
    if (LOSS && p.d_bias != nullptr) {  // the only row tile: finished, as k_dbias_fold would
      if (col0 + c < p.V) p.d_bias[col0 + c] = (0.0f + s) * (p.bias_scale ? *p.bias_scale : 1.0f);
    } else {
      p.dbias_part[int64_t(tm) * p.ldz + col0 + c] = s;
    }
  }
}

// Whether a row's target lies in [0, V).
struct LiveRows {
  const void* targets;
  int t64;
  int64_t V;
  __device__ __forceinline__ bool operator()(int64_t r) const {
    const int64_t t = load_target(targets, t64, r);
    return t >= 0 && t < V;
  }
};

// A second matrix of the same width in the same launch (W beside a chunk's hidden rows): the
// workgroups past the first one's rows_pad take its rows, none of which are checked.
struct PlainRows {
  const void* src;
  int64_t rows, rows_pad;
  void* dst;
  template <class T>
  __device__ __forceinline__ bool take(int64_t& r0, const T* __restrict__& s, int64_t& n,
                                       int64_t& pad, T* __restrict__& d) const {
    const int64_t first = (pad + 63) / 64 * 64;
    if (r0 < first) return true;
    r0 -= first;
    s = static_cast<const T*>(src);
    n = rows;
    pad = rows_pad;
    d = static_cast<T*>(dst);
    return false;
  }
};

// ---- tiled transpose ---------------------------------------------------------------------------
// dst = src^T in the K-blocked layout (dst has `cols` rows and K = rows_pad);
// entries r in [rows, rows_pad) are written as zeros.
// LIVE: source rows whose target is outside [0, V) count as zeros, whatever they hold (a
// padded row's infinities and NaN must not reach a product with its zero gradients).
template <class T, bool LIVE = false>
__global__ __launch_bounds__(256) void k_transpose(const T* __restrict__ src, int64_t rows,
                                                   int64_t rows_pad, int64_t cols, int64_t ld_src,
                                                   T* __restrict__ dst, LiveRows live,
                                                   PlainRows also) {
  __shared__ T tile[64][65];
  int64_t r0 = int64_t(blockIdx.y) * 64;
  const int64_t c0 = int64_t(blockIdx.x) * 64;
  bool check = true;
  if constexpr (LIVE) check = also.take(r0, src, rows, rows_pad, dst);
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
  for (int u = 0; u < 16; ++u) {  // sixteen loads in flight
    const int k = ty + 4 * u;
    const int64_t r = r0 + k, c = c0 + tx;
    bool in = r < rows && c < cols;
    if constexpr (LIVE) in = in && (!check || live(r));
    tile[k][tx] = in ? src[r * ld_src + c] : T(0);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int k = ty + 4 * u;
    const int64_t c = c0 + k, r = r0 + tx;
    if (r < rows_pad && c < cols) dst[kblk<128 / sizeof(T)>(c, r, cols)] = tile[tx][k];
  }
}

// The same for 16-bit elements with 16-byte global accesses on both sides: a
// 64 x 64 tile is read as 8 16-byte chunks per source row and written as 8
// 16-byte chunks per destination row (one 128-byte K block).  Requires
// 16-byte aligned source rows and rows_pad a multiple of 64.  The destination's K
// positions take the fragment-major order of the 16-bit backward GEMMs: K
// position 32 b + 8 g + 4 h + r holds source row 32 b + 16 h + 4 g + r.
template <bool LIVE = false>
__global__ __launch_bounds__(256) void k_transpose16(const uint16_t* __restrict__ src, int64_t rows,
                                                     int64_t rows_pad, int64_t cols, int64_t ld_src,
                                                     uint16_t* __restrict__ dst, LiveRows live,
                                                     PlainRows also) {
  __shared__ uint32_t tile[64][33];  // [row][column pair], 132-byte rows
  int64_t r0 = int64_t(blockIdx.y) * 64;
  const int64_t c0 = int64_t(blockIdx.x) * 64;
  bool check = true;
  if constexpr (LIVE) check = also.take(r0, src, rows, rows_pad, dst);
  const int t = threadIdx.x, j = t & 7, q = t >> 3;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int rl = q + 32 * p;
    const int64_t r = r0 + rl, c = c0 + 8 * j;
    u32x4 v = {0u, 0u, 0u, 0u};
    bool in = r < rows && c < cols;
    if constexpr (LIVE) in = in && (!check || live(r));
    if (in) v = *reinterpret_cast<const u32x4*>(src + r * ld_src + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[rl][4 * j + e] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int cl = q + 32 * p;
    const int64_t c = c0 + cl, r = r0 + 8 * j;
    // K positions 8 j + k of the tile: block j >> 2, g = j & 3, h = k >> 2, r = k & 3.
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int src = 32 * (j >> 2) + 16 * (k >> 2) + 4 * (j & 3) + (k & 3);
      h[k] = (tile[src][cl >> 1] >> (16 * (cl & 1))) & 0xFFFFu;
    }
    const u32x4 w = {h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                     h[6] | (h[7] << 16)};
    if (c < cols && r < rows_pad) *reinterpret_cast<u32x4*>(dst + kblk<64>(c, r, cols)) = w;
  }
}

// ---- d_bias: ascending fold of the per-row-tile partials --------------------------------------
__global__ __launch_bounds__(256) void k_dbias_fold(const float* part, int64_t n_parts, int64_t ldz,
                                                    int64_t V, float* d_bias, int init,
                                                    const float* scale) {
  const int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (v >= V) return;
  // scale: a power of two that the finished sums are multiplied by (exact both ways)
  const float f = scale != nullptr ? *scale : 1.0f;
  float s = init ? 0.0f : d_bias[v] / f;
  for (int64_t r = 0; r < n_parts; ++r) s += part[r * ldz + v];
  d_bias[v] = s * f;
}

// ---- launch helpers ----------------------------------------------------------------------------

template <class E, int BM, int WM, bool ODD, bool LOSS, int NS = 2>
hipError_t fwd_cfg(const FwdArgs& a, hipStream_t s) {
  using Eng = LogitEngine<E, BM, WM, NS>;
  static std::atomic<int> ready[kMaxDevices];
  const hipError_t e = prepare(k_fwd<E, BM, WM, ODD, NS, LOSS>, Eng::kLds, ready);
  if (e != hipSuccess) return e;
  const int64_t blocks = ((a.N + BM - 1) / BM) * ((a.V + kTileCols - 1) / kTileCols);
  hipLaunchKernelGGL((k_fwd<E, BM, WM, ODD, NS, LOSS>), dim3(unsigned(blocks)), dim3(Eng::NT),
                     Eng::kLds, s, a);
  return hipGetLastError();
}

// The loss's forward over 256-row tiles that keeps the products.
template <class E, bool ODD>
hipError_t fwd_keep(const FwdArgs& a, hipStream_t s) {
  using Eng = LogitEngine<E, int(kDzRowTile), 4, 2>;
  static std::atomic<int> ready[kMaxDevices];
  const hipError_t e = prepare(k_fwd<E, int(kDzRowTile), 4, ODD, 2, true, true>, Eng::kLds, ready);
  if (e != hipSuccess) return e;
  const int64_t blocks = ((a.N + kDzRowTile - 1) / kDzRowTile) * ((a.V + kTileCols - 1) / kTileCols);
  hipLaunchKernelGGL((k_fwd<E, int(kDzRowTile), 4, ODD, 2, true, true>), dim3(unsigned(blocks)),
                     dim3(Eng::NT), Eng::kLds, s, a);
  return hipGetLastError();
}

template <class E>
hipError_t dz_kept(const DzArgs& a, hipStream_t s) {
  // LDS for the sums over rows only
  const int64_t blocks = ((a.rows + kDzRowTile - 1) / kDzRowTile) * ((a.V + kTileCols - 1) / kTileCols);
  hipLaunchKernelGGL((k_dz<E, int(kDzRowTile), 4, false, true, true>), dim3(unsigned(blocks)),
                     dim3(512), 4 * kTileCols * sizeof(float), s, a);
  return hipGetLastError();
}

// Number of 64-byte K stages of a logits tile is odd (D * element size / 64).
template <class E>
bool odd_stages(int64_t D) {
  return ((D * E::kSize) / kStageBytes) % 2 == 1;
}

template <class E, bool ODD, bool LOSS>
hipError_t fwd_rows(const FwdArgs& a, hipStream_t s) {
  const int64_t vt = (a.V + kTileCols - 1) / kTileCols;
  if (a.N <= 32) {
    // Over at most 256 vocabulary tiles (a vocabulary shard) the few workgroups each
    // wait out a load latency per stage with two stages, so they keep three in flight
    // (four LDS stages, 147 KB).  Over the full vocabulary the 2-stage tiles, two
    // workgroups per compute unit, stream W faster.
    if (vt <= 256) return fwd_cfg<E, 32, 2, ODD, LOSS, 4>(a, s);
    return fwd_cfg<E, 32, 2, ODD, LOSS>(a, s);
  }
  // The largest tile that gives most compute units a workgroup: larger tiles read less of
  // hidden and W per product, and every tile gives a row the same bits.  On MI355X:
  // 64 x 256 x 4096 fp32 24 -> 16 us, 128 x 1024 x 16384 fp32 132 -> 48 and bf16 27 -> 16,
  // 1000 x 1024 x 8192 fp32 244 -> 143; 64 x 1024 x 50257 fp32 in 32-row tiles 93, in
  // 64-row tiles 81.
  auto fills = [&](int64_t bm) { return (a.N + bm - 1) / bm * vt >= 160; };
  if (a.N > 128 && fills(256)) return fwd_cfg<E, 256, 4, ODD, LOSS>(a, s);
  if (a.N > 64 && fills(128)) return fwd_cfg<E, 128, 2, ODD, LOSS>(a, s);
  if (fills(64)) return fwd_cfg<E, 64, 2, ODD, LOSS>(a, s);
  return fwd_cfg<E, 32, 2, ODD, LOSS, 4>(a, s);
}

template <class E, bool LOSS = false>
hipError_t fwd_dispatch(const FwdArgs& a, hipStream_t s) {
  return odd_stages<E>(a.D) ? fwd_rows<E, true, LOSS>(a, s) : fwd_rows<E, false, LOSS>(a, s);
}

template <class E, int BM, int WM, bool ODD, bool LOSS, int BN = kTileCols>
hipError_t dz_cfg(const DzArgs& a, hipStream_t s) {
  using Eng = Engine<E, BM, BN, WM, 2>;
  constexpr size_t lds = Eng::kLds;
  static std::atomic<int> ready[kMaxDevices];
  const hipError_t e = prepare(k_dz<E, BM, WM, ODD, LOSS, false, BN>, lds, ready);
  if (e != hipSuccess) return e;
  const int64_t blocks = ((a.rows + BM - 1) / BM) * (a.ldz / BN);
  hipLaunchKernelGGL((k_dz<E, BM, WM, ODD, LOSS, false, BN>), dim3(unsigned(blocks)), dim3(Eng::NT),
                     lds, s, a);
  return hipGetLastError();
}

// fp32 products are slow enough that idle compute units cost more than narrow tiles' extra
// reads, so few fp32 rows take tiles of 64 or 128 rows by 32 columns, and more of them
// 256 rows by 32, 64 or 256 columns, the widest that give every compute unit a workgroup.
// A row wave keeps the 64 rows it has in the 256 x 256 tile, so the sums over rows have the
// same order and every output the same bits.  On MI355X, 256 columns and here: 64 x 256 x
// 4096 49 -> 12 us, 128 x 1024 x 50257 161 -> 135, 256 x 256 x 4096 76 -> 19, 1000 x 1024 x
// 8192 252 -> 145; 1000 x 512 x 16384 156 in 256 columns, 158 in 64, 170 in 32.
template <class E, bool ODD, bool LOSS>
hipError_t dz_rows(const DzArgs& a, hipStream_t s) {
  if constexpr (E::kSize == 4) {
    if (a.rows <= 64) return dz_cfg<E, 64, 1, ODD, LOSS, 32>(a, s);
    if (a.rows <= 128) return dz_cfg<E, 128, 2, ODD, LOSS, 32>(a, s);
    const int64_t per_col = (a.rows + kDzRowTile - 1) / kDzRowTile * a.ldz;
    if (per_col < 256 * 64) return dz_cfg<E, int(kDzRowTile), 4, ODD, LOSS, 32>(a, s);
    if (per_col < 256 * kTileCols) return dz_cfg<E, int(kDzRowTile), 4, ODD, LOSS, 64>(a, s);
  }
  return dz_cfg<E, int(kDzRowTile), 4, ODD, LOSS>(a, s);
}

template <class E, bool LOSS>
hipError_t dz_dispatch(const DzArgs& a, hipStream_t s) {
  return odd_stages<E>(a.D) ? dz_rows<E, true, LOSS>(a, s) : dz_rows<E, false, LOSS>(a, s);
}

// The per-element MFMA chain does not depend on the tile shape, so the GEMM
// variants may use different tiles and still give the same bits.
//
// The largest tile whose slabs give every compute unit a workgroup: larger tiles read
// less of dz and W^T per product (1000 x 2688 x 131072 bf16 on MI355X: 256 x 224 tiles
// 609 us, 128 x 128 tiles 1020 us).  The tile does not change the bits.
template <class E>
hipError_t dx_slabs(const GemmArgs& a, hipStream_t s) {
  constexpr bool k16 = E::kSize == 2;
  const int64_t slabs = (a.K + a.k_slab - 1) / a.k_slab;
  auto fills = [&](int64_t bm, int64_t bn) {
    return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn) * slabs >= 256;
  };
  hipError_t e;
  if (k16 && a.M > 128 && fills(256, 224))
    e = gemm_cfg<E, 256, k16 ? 224 : 128, 4, 2, false, 2, 2, k16 ? kGemmNSA : 2>(a, s);
  else if (a.M > 64 && fills(128, 128))
    e = gemm_cfg<E, 128, 128, 2, 2, false, 2, k16 ? 3 : 2>(a, s);
  else if (a.M > 128)
    e = gemm_cfg<E, 128, 64, 2, 2, false, 2, 4>(a, s);
  else if (a.M <= 64 && fills(64, 128))
    e = gemm_cfg<E, 64, 128, 2, 2, false, 2, 3>(a, s);
  else if (fills(64, 32))
    e = gemm_cfg<E, 64, 32, 4, 1, false, 2, 8>(a, s);
  else
    e = gemm_cfg<E, 64, 16, 4, 1, false, 2, 8>(a, s);
  if (e != hipSuccess) return e;
  const int64_t n = a.M * a.N;
  hipLaunchKernelGGL(k_slab_fold<E>, dim3(unsigned(std::min<int64_t>((n + 1023) / 1024, 4096))),
                     dim3(256), 0, s, a, int((a.K + a.k_slab - 1) / a.k_slab));
  return hipGetLastError();
}

// d_hidden walks the whole vocabulary for every tile and cannot split K without
// changing the bits, so a batch of few rows has few tiles: there the tiles shrink
// (more workgroups stream W^T side by side) and the LDS ring deepens.  Thresholds
// measured on the 16-bit training shape (D = 2688, V = 131072): 64 x 16 tiles are
// fastest up to 64 rows, 64 x 32 up to 128, 128 x 64 up to 512, 128 x 128 up to
// 1024, and the 256 x 224 tile from 2048 rows on.
template <class E, bool SCALED = false>
hipError_t dx_tiles16(const GemmArgs& a, hipStream_t s) {
  if (a.k_slab > 0) return dx_slabs<E>(a, s);
  if (a.M <= 64) return gemm_cfg<E, 64, 16, 4, 1, false, 0, 8, 8, SCALED>(a, s);
  if (a.M <= 128) return gemm_cfg<E, 64, 32, 4, 1, false, 0, 8, 8, SCALED>(a, s);
  if (a.M <= 512) return gemm_cfg<E, 128, 64, 2, 2, false, 0, 4, 4, SCALED>(a, s);
  if (a.M <= 1024) return gemm_cfg<E, 128, 128, 2, 2, false, 0, 3, 3, SCALED>(a, s);
  return gemm_cfg<E, 256, 224, 4, 2, false, 0, 2, kGemmNSA, SCALED>(a, s);
}
template <class E>
hipError_t dx_dispatch(const GemmArgs& a, hipStream_t s);
template <>
hipError_t dx_dispatch<BF16>(const GemmArgs& a, hipStream_t s) {
  return dx_tiles16<BF16>(a, s);
}
template <>
hipError_t dx_dispatch<F16>(const GemmArgs& a, hipStream_t s) {
  if (a.scale != nullptr) return dx_tiles16<F16, true>(a, s);
  return dx_tiles16<F16>(a, s);
}
template <>
hipError_t dx_dispatch<F32>(const GemmArgs& a, hipStream_t s) {
  if (a.k_slab > 0) return dx_slabs<F32>(a, s);
  // as for 16 bits: smaller tiles and a deeper ring where there are few rows (64 rows over
  // D = 256, V = 4096 on MI355X: 241 -> 28 us)
  if (a.M <= 64) return gemm_cfg<F32, 64, 16, 4, 1, false, 0, 8>(a, s);
  if (a.M <= 128) return gemm_cfg<F32, 64, 32, 4, 1, false, 0, 8>(a, s);
  if (a.M <= 512) return gemm_cfg<F32, 128, 64, 2, 2, false, 0, 4>(a, s);
  return gemm_cfg<F32, 128, 128, 2, 2, false, 0>(a, s);
}

template <class E>
hipError_t dw_dispatch(const GemmArgs& a, hipStream_t s);
template <>
hipError_t dw_dispatch<BF16>(const GemmArgs& a, hipStream_t s) {
  if (a.load_acc) {
    if (a.store_acc) return gemm_cfg<BF16, 256, 224, 4, 2, true, 1, 2, kGemmNSA>(a, s);
    return gemm_cfg<BF16, 256, 224, 4, 2, true, 0, 2, kGemmNSA>(a, s);
  }
  if (a.store_acc) return gemm_cfg<BF16, 256, 224, 4, 2, false, 1, 2, kGemmNSA>(a, s);
  return gemm_cfg<BF16, 256, 224, 4, 2, false, 0, 2, kGemmNSA>(a, s);
}
template <>
hipError_t dw_dispatch<F16>(const GemmArgs& a, hipStream_t s) {
  if (a.scale != nullptr && !a.store_acc) {  // the rounded result only
    if (a.load_acc) return gemm_cfg<F16, 256, 224, 4, 2, true, 0, 2, kGemmNSA, true>(a, s);
    return gemm_cfg<F16, 256, 224, 4, 2, false, 0, 2, kGemmNSA, true>(a, s);
  }
  if (a.load_acc) {
    if (a.store_acc) return gemm_cfg<F16, 256, 224, 4, 2, true, 1, 2, kGemmNSA>(a, s);
    return gemm_cfg<F16, 256, 224, 4, 2, true, 0, 2, kGemmNSA>(a, s);
  }
  if (a.store_acc) return gemm_cfg<F16, 256, 224, 4, 2, false, 1, 2, kGemmNSA>(a, s);
  return gemm_cfg<F16, 256, 224, 4, 2, false, 0, 2, kGemmNSA>(a, s);
}
template <>
hipError_t dw_dispatch<F32>(const GemmArgs& a, hipStream_t s) {
  if (a.load_acc) {
    if (a.store_acc) return gemm_cfg<F32, 128, 128, 2, 2, true, 1>(a, s);
    return gemm_cfg<F32, 128, 128, 2, 2, true, 0>(a, s);
  }
  if (a.store_acc) return gemm_cfg<F32, 128, 128, 2, 2, false, 1>(a, s);
  return gemm_cfg<F32, 128, 128, 2, 2, false, 0>(a, s);
}

}  // namespace

hipError_t launch_loss_forward(flp_dtype x, const FwdArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_FORWARD, s);
  if (a.logits != nullptr) {  // bf16 and fp32
    if (x == FLP_BF16)
      return odd_stages<BF16>(a.D) ? fwd_keep<BF16, true>(a, s) : fwd_keep<BF16, false>(a, s);
    return odd_stages<F32>(a.D) ? fwd_keep<F32, true>(a, s) : fwd_keep<F32, false>(a, s);
  }
  if (x == FLP_BF16) return fwd_dispatch<BF16, true>(a, s);
  if (x == FLP_F16) return fwd_dispatch<F16, true>(a, s);
  return fwd_dispatch<F32, true>(a, s);
}

hipError_t launch_forward(flp_dtype x, const FwdArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_FORWARD, s);
  if (x == FLP_BF16) return fwd_dispatch<BF16>(a, s);
  if (x == FLP_F16) return fwd_dispatch<F16>(a, s);
  return fwd_dispatch<F32>(a, s);
}

template <int R, bool LOSS>
void merge_rows(const MergeArgs& a, hipStream_t s) {
  const dim3 grid(unsigned((a.N + R - 1) / R));
  const int64_t L = (a.n_vt + kMergeLeaves - 1) / kMergeLeaves;
  if (L == 1)
    hipLaunchKernelGGL((k_merge<R, 1, LOSS>), grid, dim3(256), 0, s, a);
  else if (L == 2)
    hipLaunchKernelGGL((k_merge<R, 2, LOSS>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_merge<R, 0, LOSS>), grid, dim3(256), 0, s, a);
}

template <bool LOSS>
hipError_t merge_all(const MergeArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_MERGE, s);
  // One row per workgroup while that still gives a few workgroups per compute unit.
  if (a.N <= kMergeRowMax)
    merge_rows<1, LOSS>(a, s);
  else
    merge_rows<8, LOSS>(a, s);
  return hipGetLastError();
}

hipError_t launch_merge(const MergeArgs& a, hipStream_t s) { return merge_all<false>(a, s); }
hipError_t launch_loss_merge(const MergeArgs& a, hipStream_t s) { return merge_all<true>(a, s); }

hipError_t launch_fill(float* dst, int64_t n, float value, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_fill, dim3(unsigned((n + 255) / 256)), dim3(256), 0, s, dst, n, value);
  return hipGetLastError();
}

hipError_t launch_logits_forward(flp_dtype x, const LogitsArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_LOGITS_FORWARD, s);
  const dim3 grid(unsigned((a.N + 3) / 4));
  if (x == FLP_BF16)
    hipLaunchKernelGGL(k_logits_fwd<BF16>, grid, dim3(256), 0, s, a);
  else if (x == FLP_F16)
    hipLaunchKernelGGL(k_logits_fwd<F16>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_logits_fwd<F32>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_logits_backward(flp_dtype x, const LogitsArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_LOGITS_BACKWARD, s);
  const dim3 grid(unsigned((a.N + 3) / 4));
  if (x == FLP_BF16)
    hipLaunchKernelGGL(k_logits_bwd<BF16>, grid, dim3(256), 0, s, a);
  else if (x == FLP_F16)
    hipLaunchKernelGGL(k_logits_bwd<F16>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_logits_bwd<F32>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_dz(flp_dtype x, const DzArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DLOGITS, s);
  const bool loss = a.onehot != nullptr;
  if (a.logits != nullptr) return x == FLP_BF16 ? dz_kept<BF16>(a, s) : dz_kept<F32>(a, s);
  if (x == FLP_BF16) return loss ? dz_dispatch<BF16, true>(a, s) : dz_dispatch<BF16, false>(a, s);
  if (x == FLP_F16) return loss ? dz_dispatch<F16, true>(a, s) : dz_dispatch<F16, false>(a, s);
  return loss ? dz_dispatch<F32, true>(a, s) : dz_dispatch<F32, false>(a, s);
}

hipError_t launch_dx(flp_dtype x, const GemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DHIDDEN, s);
  if (x == FLP_BF16) return dx_dispatch<BF16>(a, s);
  if (x == FLP_F16) return dx_dispatch<F16>(a, s);
  return dx_dispatch<F32>(a, s);
}

hipError_t launch_dw(flp_dtype x, const GemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DWEIGHT, s);
  if (x == FLP_BF16) return dw_dispatch<BF16>(a, s);
  if (x == FLP_F16) return dw_dispatch<F16>(a, s);
  return dw_dispatch<F32>(a, s);
}

hipError_t launch_transpose(flp_dtype x, const void* src, int64_t rows, int64_t rows_pad, int64_t cols,
                            int64_t ld_src, void* dst, hipStream_t s) {
  ProfScope ps(FLP_K_TRANSPOSE, s);
  const dim3 grid(unsigned((cols + 63) / 64), unsigned((rows_pad + 63) / 64));
  if (x != FLP_F32)
    hipLaunchKernelGGL(k_transpose16<>, grid, dim3(256), 0, s, static_cast<const uint16_t*>(src),
                       rows, rows_pad, cols, ld_src, static_cast<uint16_t*>(dst), LiveRows{},
                       PlainRows{});
  else
    hipLaunchKernelGGL(k_transpose<float>, grid, dim3(256), 0, s, static_cast<const float*>(src),
                       rows, rows_pad, cols, ld_src, static_cast<float*>(dst), LiveRows{},
                       PlainRows{});
  return hipGetLastError();
}

hipError_t launch_transpose_live(flp_dtype x, const void* src, int64_t rows, int64_t rows_pad,
                                 int64_t cols, const void* targets, bool t64, int64_t V, void* dst,
                                 const void* weight, int64_t weight_pad, void* weight_dst,
                                 hipStream_t s) {
  ProfScope ps(FLP_K_TRANSPOSE, s);
  const PlainRows also{weight, V, weight_pad, weight_dst};
  const int64_t blocks = (rows_pad + 63) / 64 + (weight != nullptr ? (weight_pad + 63) / 64 : 0);
  const dim3 grid(unsigned((cols + 63) / 64), unsigned(blocks));
  const LiveRows live{targets, t64 ? 1 : 0, V};
  if (x != FLP_F32)
    hipLaunchKernelGGL(k_transpose16<true>, grid, dim3(256), 0, s,
                       static_cast<const uint16_t*>(src), rows, rows_pad, cols, cols,
                       static_cast<uint16_t*>(dst), live, also);
  else
    hipLaunchKernelGGL((k_transpose<float, true>), grid, dim3(256), 0, s,
                       static_cast<const float*>(src), rows, rows_pad, cols, cols,
                       static_cast<float*>(dst), live, also);
  return hipGetLastError();
}

hipError_t launch_dbias_fold(const float* part, int64_t n_parts, int64_t ldz, int64_t V,
                             float* d_bias, int init, const float* scale, hipStream_t s) {
  ProfScope ps(FLP_K_DBIAS, s);
  hipLaunchKernelGGL(k_dbias_fold, dim3(unsigned((V + 255) / 256)), dim3(256), 0, s, part, n_parts,
                     ldz, V, d_bias, init, scale);
  return hipGetLastError();
}

const char* kernel_ids() {
  return "engine: direct global->LDS (buffer_load_dwordx4 lds, whole lines), 2 LDS stages x 128 B of K "
         "(3-8 for the small dX tiles), "
         "mfma_f32_16x16x32_bf16 | 16x16x32_f16 | 16x16x4f32; k_fwd<BM 32/64/128 x BN 256 2x2 waves (BM 32: 4 stages where few workgroups fit), "
         "BM 256 4x2 waves>; k_merge<1 or 8 rows; 256 leaves, fixed tree>; k_dz<BM 256 x BN 256, 4x2 waves; fp32: BM 64, 128 x BN 32, BM 256 x BN 32, 64>; "
         "k_gemm dX, dW<256x224, 4x2 waves, K-blocked operands; dX for <= 1024 rows: 64x16, "
         "64x32, 128x64, 128x128>; k_transpose (K-blocked); "
         "k_dbias_fold; k_fill; k_logits_fwd, k_logits_bwd<one wave per row>; "
         "rows: k_mark, k_compact, k_gather, k_scatter_rows, k_scatter_hidden; "
         "cross entropy: k_fwd, k_merge, k_dz with loss terms, k_loss_sum, k_loss_grad, k_gemm dX "
         "over vocabulary slabs and k_slab_fold (<= 8192 rows); "
         "embedding: k_embed_fwd (scaled), radix sort (k_sort_hist, k_sort_scatter; 9-bit digits; <= 4096 tokens: k_sort_rank; "
         "zero riders), k_embed_runs<32-position groups>, k_embed_rows; k_dropout; layer norm: "
         "k_norm_fwd_row, k_norm_bwd_row<one or four waves per row>, k_norm_fold; wide rows: "
         "k_norm_fwd, k_norm_dx, k_norm_params; "
         "blocks: k_gated_fwd<256x256 8 waves, 128x128, 64x64, 32x64; both weights interleaved>, "
         "k_gated_dz, k_gated_gemm<256x224, 128x128; ds_read_b64_tr_b16>, k_gated_fold; fp32: "
         "k_gated_dz32, k_gemm, k_slab_fold; k_rms_fwd, k_rms_bwd<one to eight waves per row>, "
         "k_rms_fold; k_adamw<8 or 32 bits; 2048-element tiles>";
}

}  // namespace flp
