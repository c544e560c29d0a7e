// Untied embedding lookup and its deterministic grad_weight ("Feat/nemotron h
// lm head logprob cuda", PR #555 summary bullets: an untied embedding lookup
// whose grad_weight is a sorted-segment deterministic reduction; its Known
// issues note that the pages' version accumulates repeated ids in BF16 and
// misses FP64 parity, so here every segment accumulates in fp32 and rounds
// once).
//
//   out[i]      = s E[ids[i]]               (a zero row for ids outside [0, V))
//   d_E[v]      = s (sum over tokens i with ids[i] == v of grad[i], in ascending i)
//
// with s = 1 for the plain lookup.
//
// The backward sorts the (id, token) pairs by id with a stable LSD radix sort
// (9-bit digits, blocks of 256 keys; ranks inside a block come from an in-order
// count, so the sort is deterministic; up to 4096 tokens are placed by counting in one
// launch instead).  The sorted list is then cut into fixed
// groups of 32 positions, one workgroup each, so a frequent id does not serialise
// on one wave: inside a group every run of equal ids is summed in fp32 in token
// order; a segment that spans several groups adds its per-group pieces in group
// order.  Every order is fixed by the sorted list: the output is bitwise
// reproducible.
//
// Writing d_E is most of the work, and most of its rows are zeros (ids that do not
// occur).  The sort's scatter passes occupy few compute units and wait on latency, so
// each of them carries extra "rider" workgroups that clear a share of d_E; the rows of
// ids that occur are written after the last of them.  N = 16384, D = 2688, V = 131072
// bf16 on MI355X: 174 us for 793 MB in six launches (riders that spared the occurring
// rows, behind a pass that marked them: 190 us in eleven).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "flp_launch.h"

namespace flp {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kSortBlock = int(kEmbSortBlock);  // keys per block of a radix pass (one per thread)

__device__ __forceinline__ int64_t load_id(const void* ids, bool i64, int64_t i) {
  return i64 ? reinterpret_cast<const int64_t*>(ids)[i]
             : int64_t(reinterpret_cast<const int32_t*>(ids)[i]);
}

// One 16-byte chunk times `scale`, rounded once per element.
template <class T>
__device__ __forceinline__ u32x4 scale_chunk(u32x4 v, float scale) {
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
  vec x = __builtin_bit_cast(vec, v);
#pragma unroll
  for (int k = 0; k < int(16 / sizeof(T)); ++k) x[k] = T(float(x[k]) * scale);
  return __builtin_bit_cast(u32x4, x);
}

// One wave per token row, four rows per workgroup: 16-byte chunks, copied as they are
// (T = void) or multiplied by `scale`.  A launch holds fewer than 2^32 threads, so past
// 2^25 rows a wave takes several.
template <class T>
__global__ __launch_bounds__(256) void k_embed_fwd(const u32x4* __restrict__ weight,
                                                   const void* __restrict__ ids, int i64,
                                                   int64_t N, int64_t V, int64_t row_vec,
                                                   float scale, u32x4* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  for (int64_t i = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); i < N;
       i += int64_t(gridDim.x) * 4) {
    const int64_t v = load_id(ids, i64 != 0, i);
    u32x4* dst = out + i * row_vec;
    if (v >= 0 && v < V) {
      const u32x4* src = weight + v * row_vec;
      for (int64_t c = lane; c < row_vec; c += 64) {
        if constexpr (std::is_void<T>::value)
          dst[c] = src[c];
        else
          dst[c] = scale_chunk<T>(src[c], scale);
      }
    } else {
      const u32x4 z = {0u, 0u, 0u, 0u};
      for (int64_t c = lane; c < row_vec; c += 64) dst[c] = z;
    }
  }
}

// A share of d_E to be cleared by workgroups appended to another kernel's grid: the
// 16-byte chunks [c0, c1), `per` per workgroup.  One store per thread is fastest (352 MB
// on MI355X: 50 us beside a sort pass; 4 stores per thread 55, 16 stores 64); only a share
// beyond 16 GB takes more, since a launch holds fewer than 2^32 threads.
struct ZeroRider {
  u32x4* dW;
  int64_t c0, c1, per;
  ZeroRider(void* d_weight, int64_t first, int64_t last)
      : dW(static_cast<u32x4*>(d_weight)), c0(first), c1(last),
        per(256 * (1 + (last - first) / (int64_t(1) << 30))) {}
  int64_t blocks() const { return (c1 - c0 + per - 1) / per; }
};

__device__ __forceinline__ void ride(const ZeroRider& z, int64_t r) {
  const int64_t c1 = min(z.c1, z.c0 + (r + 1) * z.per);
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int64_t c = z.c0 + r * z.per + threadIdx.x; c < c1; c += 256)
    __builtin_nontemporal_store(zero, z.dW + c);
}

// Sort keys: the id, or V for an id outside [0, V) (those sort last and are
// dropped); values: the token index.  The first pass reads them from the ids.
constexpr int kDigitBits = int(kEmbDigitBits), kDigits = 1 << kDigitBits;
struct SortArgs {
  const void* ids;
  int i64;
  int64_t V;
  const uint32_t* keys;  // [n], or null in the first pass
  const int32_t* vals;
  int64_t n;
  int shift;
  int64_t n_blocks, ld;  // ld: n_blocks rounded up to 4
  int32_t* hist;         // [kDigits][ld]
  __device__ __forceinline__ uint32_t key(int64_t i) const {
    if (keys != nullptr) return keys[i];
    const int64_t v = load_id(ids, i64 != 0, i);
    return (v >= 0 && v < V) ? uint32_t(v) : uint32_t(V);
  }
};

// Per-block digit counts, stored digit-major: hist[d * ld + b].
__global__ __launch_bounds__(256) void k_sort_hist(SortArgs p) {
  const int64_t b = blockIdx.x;
  __shared__ int32_t cnt[kDigits];
  const int t = threadIdx.x;
  for (int d = t; d < kDigits; d += 256) cnt[d] = 0;
  __syncthreads();
  const int64_t i = b * kSortBlock + t;
  if (i < p.n) atomicAdd(&cnt[(p.key(i) >> p.shift) & (kDigits - 1)], 1);
  __syncthreads();
  for (int d = t; d < kDigits; d += 256) p.hist[d * p.ld + b] = cnt[d];
}

// Stable scatter of one radix pass.  A block holds 256 consecutive keys.  Its
// offset for digit d is the count of all keys with a smaller digit plus the
// count of keys with digit d in earlier blocks (each thread sums its digits'
// counts, then an exclusive scan over the digit totals in LDS); a key's
// place adds the number of keys before it in the block with the same digit.
__global__ __launch_bounds__(256) void k_sort_scatter(SortArgs p, uint32_t* __restrict__ kout,
                                                      int32_t* __restrict__ vout, ZeroRider z) {
  const int64_t b = blockIdx.x;
  if (b >= p.n_blocks) {
    ride(z, b - p.n_blocks);
    return;
  }
  typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
  __shared__ int32_t tot[kDigits];
  __shared__ int32_t run[kDigits];
  __shared__ int32_t dig[256];
  const int t = threadIdx.x;
  constexpr int kPer = kDigits / 256;
  int32_t before[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    before[e] = 0;
    int32_t all = 0;
    const int32_t* h = p.hist + int64_t(t + 256 * e) * p.ld;
    for (int64_t q0 = 0; q0 < p.n_blocks; q0 += 32) {  // eight 16-byte loads in flight
      i32x4 c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        c[u] = q0 + 4 * u < p.n_blocks ? *reinterpret_cast<const i32x4*>(h + q0 + 4 * u)
                                       : i32x4{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t q = q0 + 4 * u + k;
          const int32_t x = q < p.n_blocks ? c[u][k] : 0;  // the padding is not written
          before[e] += q < b ? x : 0;
          all += x;
        }
    }
    tot[t + 256 * e] = all;
  }
  __syncthreads();
  if (t < 64) {  // exclusive scan of the digit totals by one wave
    constexpr int kLane = kDigits / 64;
    int32_t x[kLane], sum = 0;
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      x[k] = tot[kLane * t + k];
      sum += x[k];
    }
    int32_t inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int32_t y = __shfl_up(inc, off);
      if (t >= off) inc += y;
    }
    int32_t at = inc - sum;
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      run[kLane * t + k] = at;
      at += x[k];
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kPer; ++e) run[t + 256 * e] += before[e];
  const int64_t i = b * kSortBlock + t;
  const bool valid = i < p.n;
  const uint32_t key = valid ? p.key(i) : 0u;
  const int d = valid ? int((key >> p.shift) & (kDigits - 1)) : -1;
  dig[t] = d;
  __syncthreads();
  int r = 0;
  for (int u = 0; u < t; ++u) r += (dig[u] == d) ? 1 : 0;
  if (valid) {
    const int32_t pos = run[d] + r;
    kout[pos] = key;
    vout[pos] = p.keys != nullptr ? p.vals[i] : int32_t(i);
  }
}

// Few tokens: the whole stable sort in one launch.  A key's place is the number of keys
// before it, counted over all of them in LDS, so nothing waits for another launch.  A
// workgroup places 64 keys, one per lane; each of its waves counts a quarter of the keys
// (four per read, the same for every lane).  On MI355X, the gradient with the radix passes
// and here: 1501 x 520 of 5003 55 and 43 us, 4096 x 2688 of 131072 153 and 145, 8192 x 520
// 56 and 65.
constexpr int64_t kRankMax = 4096;
__global__ __launch_bounds__(256) void k_sort_rank(SortArgs p, uint32_t* __restrict__ kout,
                                                   int32_t* __restrict__ vout, ZeroRider z) {
  const int64_t b = blockIdx.x, blocks = (p.n + 63) / 64;
  if (b >= blocks) {
    ride(z, b - blocks);
    return;
  }
  __shared__ u32x4 keys4[kRankMax / 4];
  __shared__ int32_t part[4][64];
  uint32_t* key = reinterpret_cast<uint32_t*>(keys4);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int n = int(p.n), n4 = (n + 3) / 4;
  for (int i0 = 0; i0 < 4 * n4; i0 += 8 * 256) {  // eight loads in flight
    uint32_t k[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) k[u] = p.key(min(i0 + u * 256 + t, n - 1));
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * 256 + t;
      if (i < 4 * n4) key[i] = i < n ? k[u] : ~0u;  // past every key
    }
  }
  __syncthreads();
  const int lo4 = int(b) * 16, i = int(b) * 64 + lane;  // lo4: this workgroup's keys
  const uint32_t k = key[min(i, n - 1)];
  // the wave's quarter, and the parts of it before, among and after the workgroup's keys
  const int q0 = n4 * wave / 4, q1 = n4 * (wave + 1) / 4;
  const int a1 = max(q0, min(q1, lo4)), a2 = max(q0, min(q1, lo4 + 16));
  int32_t at = 0;
#pragma unroll 4
  for (int q = q0; q < a1; ++q) {
    const u32x4 v = keys4[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) at += v[e] <= k ? 1 : 0;
  }
  for (int q = a1; q < a2; ++q) {
    const u32x4 v = keys4[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) at += (v[e] < k || (v[e] == k && 4 * q + e < i)) ? 1 : 0;
  }
#pragma unroll 4
  for (int q = a2; q < q1; ++q) {
    const u32x4 v = keys4[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) at += v[e] < k ? 1 : 0;
  }
  part[wave][lane] = at;
  __syncthreads();
  if (wave == 0 && i < n) {
    at = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    kout[at] = k;
    vout[at] = i;
  }
}

template <int SIZE>
__device__ __forceinline__ void unpack_chunk(const u32x4& v, float* x, bool f16);

template <>
__device__ __forceinline__ void unpack_chunk<2>(const u32x4& v, float* x, bool f16) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (f16) {
      x[2 * k] = float(__builtin_bit_cast(_Float16, uint16_t(v[k] & 0xFFFFu)));
      x[2 * k + 1] = float(__builtin_bit_cast(_Float16, uint16_t(v[k] >> 16)));
    } else {
      x[2 * k] = __uint_as_float(v[k] << 16);
      x[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
    }
  }
}

template <>
__device__ __forceinline__ void unpack_chunk<4>(const u32x4& v, float* x, bool) {
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(v[k]);
}

__device__ __forceinline__ uint32_t round_bf16(float f) {  // round to nearest even
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7F800000u) == 0x7F800000u) return (u >> 16) | ((u & 0xFFFFu) ? 0x40u : 0u);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

__device__ __forceinline__ uint32_t round_16(float f, bool f16) {
  return f16 ? uint32_t(__builtin_bit_cast(uint16_t, _Float16(f))) : round_bf16(f);
}

template <int XS, bool OUT_F32>
__device__ __forceinline__ void store_chunk(const float* sum, float scale, void* dW, int64_t v,
                                            int64_t row_vec, int64_t c, bool f16) {
  constexpr int EPC = 16 / XS;
  float acc[EPC];  // the finished fp32 sum times `scale` (1: the same bits), rounded below
#pragma unroll
  for (int k = 0; k < EPC; ++k) acc[k] = sum[k] * scale;
  if constexpr (OUT_F32) {
    float* out = static_cast<float*>(dW) + (v * row_vec + c) * EPC;
#pragma unroll
    for (int k = 0; k < EPC; k += 4) {
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(acc[k + j]);
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(out + k));
    }
  } else {
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = round_16(acc[2 * k], f16) | (round_16(acc[2 * k + 1], f16) << 16);
    __builtin_nontemporal_store(w, static_cast<u32x4*>(dW) + v * row_vec + c);
  }
}

// Pass A: one workgroup per group of kSegGroup consecutive sorted positions.  The
// group is cut into runs of equal id; each run is summed in fp32 in sorted
// (= ascending token) order.  A run that is its id's whole segment is written to
// d_W at once; a run that starts at the group's first position goes to the
// group's head slot, any other run that reaches past the group to its tail slot
// (a group holds at most one of each).  Each thread owns one 16-byte chunk of a row.
constexpr int kSegGroup = int(kEmbSegGroup);

template <int XS, bool OUT_F32>
__device__ __forceinline__ void finish_run(const float* acc, float scale, int64_t j, int a, bool whole,
                                           uint32_t k, float* head, float* tail, void* dW,
                                           int64_t row_vec, int64_t c, bool f16) {
  constexpr int EPC = 16 / XS;
  if (whole) {
    store_chunk<XS, OUT_F32>(acc, scale, dW, int64_t(k), row_vec, c, f16);
  } else {
    float* slot = (a == 0 ? head : tail) + (j * row_vec + c) * EPC;
#pragma unroll
    for (int q = 0; q < EPC; q += 4) {
      u32x4 w;
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = __float_as_uint(acc[q + u]);
      *reinterpret_cast<u32x4*>(slot + q) = w;
    }
  }
}

// Threads per workgroup of the two passes below, one 16-byte chunk of the row each (128
// of them fill a 336-chunk row's workgroups better than 256: 61 -> 46 us).
constexpr int kColThreads = 128;

template <int XS, bool OUT_F32>
__global__ __launch_bounds__(kColThreads) void k_embed_runs(const u32x4* __restrict__ grad, int f16,
                                                    const uint32_t* __restrict__ keys,
                                                    const int32_t* __restrict__ tok, int64_t N,
                                                    int64_t V, int64_t row_vec,
                                                    float* __restrict__ head,
                                                    float* __restrict__ tail, void* __restrict__ dW,
                                                    float scale) {
  constexpr int EPC = 16 / XS;
  __shared__ uint32_t skey[kSegGroup];
  __shared__ int32_t stok[kSegGroup];
  __shared__ uint8_t whole[kSegGroup];  // the run ending before position p is its whole segment
  const int64_t j = blockIdx.x;
  const int64_t s0 = j * kSegGroup;
  const int n = int((N - s0) < kSegGroup ? (N - s0) : kSegGroup);
  if (threadIdx.x < kSegGroup) {
    // positions past the batch and dropped ids read as key V (never summed)
    const bool in = int(threadIdx.x) < n;
    const uint32_t k = in ? keys[s0 + threadIdx.x] : uint32_t(V);
    const bool live = in && int64_t(k) < V;
    skey[threadIdx.x] = k;
    stok[threadIdx.x] = live ? tok[s0 + threadIdx.x] : -1;
    // a run inside the group is the whole segment iff neither neighbour of the group has
    // its id (a dropped id's key V is never a live one)
    const uint32_t prev = s0 > 0 ? keys[s0 - 1] : uint32_t(V);
    const uint32_t next = s0 + kSegGroup < N ? keys[s0 + kSegGroup] : uint32_t(V);
    whole[threadIdx.x] = uint8_t(live && k != prev && k != next);
  }
  __syncthreads();
  // summed positions: the prefix of the group with ids in [0, V) (dropped ids sort last)
  int m = 0;
  while (m < n && int64_t(skey[m]) < V) ++m;
  for (int64_t c = int64_t(blockIdx.y) * kColThreads + threadIdx.x; c < row_vec;
       c += int64_t(gridDim.y) * kColThreads) {
    // every row of the group in flight at once, then the runs in order
    u32x4 x4[kSegGroup];
#pragma unroll
    for (int p = 0; p < kSegGroup; ++p) {
      const int32_t t = stok[p];
      x4[p] = grad[int64_t(t < 0 ? 0 : t) * row_vec + c];
    }
    float acc[EPC];
#pragma unroll
    for (int q = 0; q < EPC; ++q) acc[q] = 0.0f;
    int a = 0;
#pragma unroll
    for (int p = 0; p < kSegGroup; ++p) {
      if (p < m) {
        if (p > a && skey[p] != skey[p - 1]) {
          finish_run<XS, OUT_F32>(acc, scale, j, a, whole[a] != 0, skey[p - 1], head, tail, dW,
                                  row_vec, c, f16 != 0);
#pragma unroll
          for (int q = 0; q < EPC; ++q) acc[q] = 0.0f;
          a = p;
        }
        float x[EPC];
        unpack_chunk<XS>(x4[p], x, f16 != 0);
#pragma unroll
        for (int q = 0; q < EPC; ++q) acc[q] += x[q];
      }
    }
    if (m > a)  // the group's last run
      finish_run<XS, OUT_F32>(acc, scale, j, a, whole[a] != 0, skey[a], head, tail, dW, row_vec, c,
                              f16 != 0);
  }
}

// Pass B: an id whose segment spans several groups adds its pieces in group
// order (the first group's head or tail slot, then the head slots of the
// following groups); an id inside one group was written by pass A.  One workgroup
// per group: the group in which a spanning segment begins combines it, eight pieces
// in flight.
template <int XS, bool OUT_F32>
__global__ __launch_bounds__(kColThreads) void k_embed_rows(const uint32_t* __restrict__ keys, int64_t N,
                                                    int64_t V, int64_t row_vec,
                                                    const float* __restrict__ head,
                                                    const float* __restrict__ tail, int f16,
                                                    float scale, void* __restrict__ dW) {
  constexpr int EPC = 16 / XS;
  __shared__ int32_t count;
  const int t = threadIdx.x;
  const int64_t g0 = blockIdx.x, s0 = g0 * kSegGroup;
  if (s0 + kSegGroup >= N) return;  // nothing follows the last group
  const uint32_t k = keys[s0 + kSegGroup - 1];
  if (int64_t(k) >= V || keys[s0 + kSegGroup] != k) return;
  const bool from_start = keys[s0] == k;
  if (from_start && s0 > 0 && keys[s0 - 1] == k) return;  // began in an earlier group
  // Groups after g0 whose first position has the id: all up to the first that has not.
  int64_t g1 = g0;
  for (;;) {
    if (t == 0) count = kColThreads;
    __syncthreads();
    const int64_t s = (g1 + 1 + t) * kSegGroup;
    if (s >= N || keys[s] != k) atomicMin(&count, t);
    __syncthreads();
    const int n = count;
    g1 += n;
    if (n < kColThreads) break;
    __syncthreads();
  }
  const float* first = from_start ? head : tail;
  for (int64_t c = int64_t(blockIdx.y) * kColThreads + t; c < row_vec;
       c += int64_t(gridDim.y) * kColThreads) {
    float acc[EPC];
    const float* f = first + (g0 * row_vec + c) * EPC;
#pragma unroll
    for (int q = 0; q < EPC; ++q) acc[q] = f[q];
    int64_t g = g0 + 1;
    for (; g + 8 <= g1 + 1; g += 8) {  // eight pieces in flight, added in group order
      float x[8][EPC];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float* h = head + ((g + u) * row_vec + c) * EPC;
#pragma unroll
        for (int q = 0; q < EPC; ++q) x[u][q] = h[q];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int q = 0; q < EPC; ++q) acc[q] += x[u][q];
    }
    for (; g <= g1; ++g) {
      const float* h = head + (g * row_vec + c) * EPC;
#pragma unroll
      for (int q = 0; q < EPC; ++q) acc[q] += h[q];
    }
    store_chunk<XS, OUT_F32>(acc, scale, dW, int64_t(k), row_vec, c, f16 != 0);
  }
}

}  // namespace

int embed_sort_passes(int64_t V) {
  int bits = 0;
  while ((uint64_t(V) >> bits) != 0) ++bits;  // keys run up to V (the dropped-id key)
  return (bits + kDigitBits - 1) / kDigitBits;
}

hipError_t launch_embedding_forward(flp_dtype x, const void* weight, const void* ids, bool i64,
                                    int64_t N, int64_t D, int64_t V, float scale, void* out,
                                    hipStream_t s) {
  ProfScope ps(FLP_K_EMBEDDING, s);
  const int64_t row_vec = D * int64_t(dtype_size(x)) / 16;
  auto launch = [&](auto kernel) {
    const int64_t grid = std::min<int64_t>((N + 3) / 4, 1 << 23);
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(256), 0, s,
                       static_cast<const u32x4*>(weight), ids, int(i64), N, V, row_vec, scale,
                       static_cast<u32x4*>(out));
  };
  if (scale == 1.0f)
    launch(k_embed_fwd<void>);
  else if (x == FLP_BF16)
    launch(k_embed_fwd<__bf16>);
  else if (x == FLP_F16)
    launch(k_embed_fwd<_Float16>);
  else
    launch(k_embed_fwd<float>);
  return hipGetLastError();
}

hipError_t launch_embedding_backward(const EmbedBwdArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_EMBEDDING, s);
  const int64_t N = a.N, V = a.V;
  SortArgs p{};
  p.ids = a.ids;
  p.i64 = int(a.i64);
  p.V = V;
  p.n = N;
  p.n_blocks = (N + kSortBlock - 1) / kSortBlock;
  p.ld = (p.n_blocks + 3) / 4 * 4;
  p.hist = a.hist;
  const int passes = N <= kRankMax ? 1 : embed_sort_passes(V);
  const int64_t chunks = V * (a.D * int64_t(dtype_size(a.dw)) / 16);
  for (int k = 0; k < passes; ++k) {
    const int src = k & 1, dst = src ^ 1;
    p.keys = k == 0 ? nullptr : a.keys[src];
    p.vals = a.vals[src];
    p.shift = kDigitBits * k;
    if (N > kRankMax)
      hipLaunchKernelGGL(k_sort_hist, dim3(unsigned(p.n_blocks)), dim3(256), 0, s, p);
    const ZeroRider z(a.d_weight, chunks / passes * k,
                      k + 1 == passes ? chunks : chunks / passes * (k + 1));
    const int64_t blocks = N > kRankMax ? p.n_blocks : (N + 63) / 64;
    hipLaunchKernelGGL(N > kRankMax ? k_sort_scatter : k_sort_rank,
                       dim3(unsigned(blocks + z.blocks())), dim3(256), 0, s, p, a.keys[dst],
                       a.vals[dst], z);
  }
  const int fin = passes & 1;
  const int64_t row_vec = a.D * int64_t(dtype_size(a.x)) / 16;
  const dim3 groups(unsigned((N + kSegGroup - 1) / kSegGroup),
                    unsigned(std::min<int64_t>((row_vec + kColThreads - 1) / kColThreads, 65535)));
  const int f16 = a.x == FLP_F16 ? 1 : 0;
  const u32x4* g = static_cast<const u32x4*>(a.grad);
  auto sums = [&](auto runs, auto rows) {
    hipLaunchKernelGGL(runs, groups, dim3(kColThreads), 0, s, g, f16, a.keys[fin], a.vals[fin], N, V,
                       row_vec, a.head, a.tail, a.d_weight, a.scale);
    hipLaunchKernelGGL(rows, groups, dim3(kColThreads), 0, s, a.keys[fin], N, V, row_vec, a.head, a.tail,
                       f16, a.scale, a.d_weight);
  };
  if (a.x == FLP_F32)
    sums(k_embed_runs<4, true>, k_embed_rows<4, true>);
  else if (a.dw == FLP_F32)
    sums(k_embed_runs<2, true>, k_embed_rows<2, true>);
  else
    sums(k_embed_runs<2, false>, k_embed_rows<2, false>);
  return hipGetLastError();
}

}  // namespace flp
