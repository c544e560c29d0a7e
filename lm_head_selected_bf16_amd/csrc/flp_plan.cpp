// Workspace layouts and fail-closed argument validation for the C ABI.
// Pure host arithmetic: no HIP call, no pointer is ever dereferenced, so every
// gate can be exercised on a machine without a GPU.
#include "flp_plan.h"

#include <algorithm>
#include <cmath>
#include <limits>
#include <new>
#include <vector>

namespace flp {

namespace {

// Vocabulary slabs of d_hidden for few rows: up to 16 of at least 2048 columns.  bf16 on
// MI355X, 1000 rows over 1344 x 50257: one walk 443 us, 4 slabs 250, 8 slabs 208, 16 slabs
// 183 (24 of them 210: more sums to add); 64 rows over 992 x 20000: 55, 23, 23, 24.  fp32,
// whose products take longer than the sums: at least 1024 columns (64 x 256 x 4096: slabs of
// 2048 20 us, 1024 15, 512 12; 4096 x 512 x 8192: 269, 277, 300).
constexpr int64_t kMaxSlabs = 16, kMinSlab = 2048, kMinSlabF32 = 1024;


constexpr int64_t kMaxIndex = std::numeric_limits<int64_t>::max() / 16;

bool mul_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxIndex / a; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
  uintptr_t lo = 0, hi = 0;
  bool live() const { return hi > lo; }
};

Span span(const void* p, size_t bytes) {
  Span s;
  if (p != nullptr && bytes > 0) {
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + bytes;
  }
  return s;
}

bool overlap(const Span& a, const Span& b) {
  return a.live() && b.live() && a.lo < b.hi && b.lo < a.hi;
}

// Every output span must be disjoint from every input span and from every other
// output span.
bool any_alias(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

// An empty batch writes only d_weight and d_bias, as zeros (sums over no rows).
flp_status validate_empty_sums(int64_t D, int64_t V, size_t xs, const void* weight,
                               const float* bias, const void* d_weight, flp_dtype dw,
                               const float* d_bias) {
  if (!aligned(d_weight, 16) || !aligned(d_bias, 4)) return FLP_MISALIGNED;
  const Span ins[] = {span(weight, size_t(V) * D * xs), span(bias, size_t(V) * 4)};
  const Span outs[] = {span(d_weight, size_t(V) * D * dtype_size(dw)), span(d_bias, size_t(V) * 4)};
  return any_alias(outs, 2, ins, 2) ? FLP_INVALID_ARGUMENT : FLP_OK;
}

flp_status check_dims(int64_t N, int64_t D, int64_t V, flp_dtype x, flp_dtype t) {
  if (N < 0 || D < 1 || V < 1) return FLP_INVALID_ARGUMENT;
  if (x != FLP_BF16 && x != FLP_F16 && x != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if (t != FLP_I64 && t != FLP_I32) return FLP_UNSUPPORTED_DTYPE;
  if (D % 32 != 0) return FLP_UNSUPPORTED_SHAPE;
  // The logit-tile kernels address the rows of a hidden / weight tile through a
  // buffer resource with 32-bit offsets (row r of at most 256 at r * D * size,
  // plus the chunk within the 128-byte stage): every such offset must stay below
  // the resource's 2^31 - 1 records.
  if (D > kMaxIndex / 256 || D * int64_t(dtype_size(x)) * 256 >= (int64_t(1) << 31))
    return FLP_UNSUPPORTED_SHAPE;
  const int64_t rows = std::max<int64_t>(round_up(std::max<int64_t>(N, 1), kRowQuantum), 1);
  const int64_t ldz = round_up(V, kVocabTile);
  if (!mul_ok(rows, D) || !mul_ok(ldz, D) || !mul_ok(rows, ldz) ||
      !mul_ok(ceil_div(V, kVocabTile), rows))
    return FLP_UNSUPPORTED_SHAPE;
  // Grid limits: row tiles x vocab tiles and the output tiles of the GEMMs.
  if (ceil_div(rows, 16) * ceil_div(V, kVocabTile) > (int64_t(1) << 31) - 1) return FLP_UNSUPPORTED_SHAPE;
  return FLP_OK;
}

}  // namespace

FwdLayout fwd_layout(int64_t N, int64_t /*D*/, int64_t V) {
  FwdLayout L;
  L.n_vt = ceil_div(V, kVocabTile);
  L.part_off = 0;
  L.zt_off = align_up(size_t(L.n_vt) * size_t(N) * 8);
  L.total = L.zt_off + align_up(size_t(N) * 4);
  return L;
}

BwdLayout bwd_layout_for_chunk(int64_t N, int64_t D, int64_t V, flp_dtype x, flp_dtype dw,
                               int64_t chunk, bool need_dh, bool need_dw, bool need_db) {
  BwdLayout L;
  const int64_t full = round_up(std::max<int64_t>(N, 1), kRowQuantum);
  chunk = std::min(round_up(std::max<int64_t>(chunk, 1), kRowQuantum), full);
  const size_t xs = dtype_size(x);
  L.chunk = chunk;
  L.n_chunks = ceil_div(std::max<int64_t>(N, 1), chunk);
  L.ldz = round_up(V, kVocabTile);
  L.ldt = chunk;
  size_t off = 0;
  L.dz_off = off;
  if (need_dh) off += align_up(size_t(chunk) * size_t(L.ldz) * xs);
  L.wt_off = off;  // W^T [D][ldz], zero-padded past V
  if (need_dh) off += align_up(size_t(D) * size_t(L.ldz) * xs);
  L.dzt_off = off;
  if (need_dw) off += align_up(size_t(L.ldz) * size_t(chunk) * xs);
  L.ht_off = off;
  if (need_dw) off += align_up(size_t(D) * size_t(chunk) * xs);
  L.dbp_off = off;
  if (need_db) off += align_up(size_t(chunk / kDzRowTile) * size_t(L.ldz) * 4);
  L.acc_off = off;
  L.use_acc = need_dw && dw != FLP_F32 && L.n_chunks > 1;
  if (L.use_acc) off += align_up(size_t(V) * size_t(D) * 4);
  L.total = std::max<size_t>(off, kAlign);
  return L;
}

namespace {

// Row quanta of a chunk, rounded down to a whole number of d_hidden waves when that is
// possible.
int64_t whole_waves(int64_t nq, int64_t D, flp_dtype x) {
  const bool f32 = x == FLP_F32;
  const int64_t tm = f32 ? kGemmTile32 : kGemmTileM16, tn = f32 ? kGemmTile32 : kGemmTileN16;
  const int64_t ct = ceil_div(D, tn);
  int64_t a = ct, b = kNumCUs;  // gcd
  while (b != 0) {
    const int64_t r = a % b;
    a = b;
    b = r;
  }
  const int64_t wave_rows = (kNumCUs / a) * tm;
  if (wave_rows % kRowQuantum != 0) return nq;
  const int64_t wq = wave_rows / kRowQuantum;
  return nq >= wq ? nq / wq * wq : nq;
}

}  // namespace

BwdLayout bwd_layout_for_bytes(int64_t N, int64_t D, int64_t V, flp_dtype x, flp_dtype dw,
                               size_t bytes, bool need_dh, bool need_dw, bool need_db) {
  const int64_t full = round_up(std::max<int64_t>(N, 1), kRowQuantum);
  BwdLayout L = bwd_layout_for_chunk(N, D, V, x, dw, full, need_dh, need_dw, need_db);
  if (L.total <= bytes) return L;
  // Several chunks: the fp32 accumulator (if any) plus per-chunk buffers.
  const size_t ldz = size_t(round_up(V, kVocabTile));
  const size_t xs = dtype_size(x);
  const size_t q = size_t(kRowQuantum);
  const size_t per_quantum = (need_dh ? q * ldz * xs : 0) + (need_dw ? q * (ldz + size_t(D)) * xs : 0) +
                             (need_db ? (q / size_t(kDzRowTile)) * ldz * 4 : 0);
  const size_t fixed = ((need_dw && dw != FLP_F32) ? align_up(size_t(V) * size_t(D) * 4) : 0) +
                       (need_dh ? align_up(size_t(D) * ldz * xs) : 0);
  // The layout of nq quanta takes fixed + nq * per_quantum bytes plus alignment
  // padding, so this nq is an upper bound; step down to the first that fits.
  int64_t nq = 0;
  if (per_quantum > 0 && bytes > fixed) nq = int64_t((bytes - fixed) / per_quantum);
  nq = std::min<int64_t>(nq, full / kRowQuantum);
  if (need_dh) nq = whole_waves(nq, D, x);
  for (; nq >= 1; --nq) {
    L = bwd_layout_for_chunk(N, D, V, x, dw, nq * kRowQuantum, need_dh, need_dw, need_db);
    if (L.total <= bytes) return L;
  }
  L = BwdLayout();
  return L;
}

SelLayout sel_layout(int64_t N, int64_t n_rows) {
  SelLayout L;
  L.cap = std::max<int64_t>(std::min(n_rows, N), 0);
  size_t off = 0;
  L.mask_off = off;
  off += align_up(size_t(std::max<int64_t>(N, 0)));
  L.pos_off = off;
  off += align_up(size_t(std::max<int64_t>(N, 0)) * 4);
  L.sel_off = off;
  off += align_up(size_t(L.cap) * 4);
  L.total = std::max<size_t>(off, kAlign);
  return L;
}

IdxLayout idx_layout(int64_t N, int64_t D, int64_t n_rows, flp_dtype x, bool backward,
                     bool need_dh) {
  IdxLayout L;
  L.sel = sel_layout(N, n_rows);
  const size_t c = size_t(L.sel.cap);
  const size_t row_bytes = size_t(D) * dtype_size(x);
  size_t off = L.sel.total;
  L.h_off = off;
  off += align_up(c * row_bytes);
  L.t_off = off;
  off += align_up(c * 8);
  L.temp_off = off;
  off += align_up(c * 4);
  if (backward) {
    L.g_off = off;
    off += align_up(c * 4);
    L.lse_in_off = off;
    off += align_up(c * 4);
    L.dh_off = off;
    if (need_dh) off += align_up(c * row_bytes);
  } else {
    L.logp_off = off;
    off += align_up(c * 4);
    L.lse_off = off;
    off += align_up(c * 4);
  }
  L.dense_off = off;
  return L;
}

EmbLayout emb_layout(int64_t N, int64_t D, int64_t V) {
  EmbLayout L;
  const size_t n = size_t(std::max<int64_t>(N, 0));
  L.n_blocks = ceil_div(std::max<int64_t>(N, 1), kEmbSortBlock);
  size_t off = 0;
  for (int k = 0; k < 2; ++k) {
    L.keys_off[k] = off;
    off += align_up(n * 4);
    L.vals_off[k] = off;
    off += align_up(n * 4);
  }
  L.hist_off = off;
  // The documented size counts two words per id beside the digit counts of 256 digits; the
  // 512 digits' counts may take more than those.
  const size_t hist = (size_t(1) << kEmbDigitBits) * size_t(round_up(L.n_blocks, 4)) * 4;
  off += std::max(align_up(hist), align_up(size_t(256) * size_t(L.n_blocks) * 4) +
                                      2 * align_up(size_t(V) * 4));
  const size_t groups = size_t(ceil_div(std::max<int64_t>(N, 1), kEmbSegGroup));
  L.head_off = off;
  off += align_up(groups * size_t(D) * 4);
  L.tail_off = off;
  off += align_up(groups * size_t(D) * 4);
  L.total = off;
  return L;
}

flp_status validate_rows(int64_t N, const void* rows, flp_dtype r, int64_t n_rows) {
  if (N < 0 || n_rows < 0) return FLP_INVALID_ARGUMENT;
  if (r != FLP_I64 && r != FLP_I32) return FLP_UNSUPPORTED_DTYPE;
  if (N > kMaxIndexedRows || n_rows > kMaxIndex / 8) return FLP_UNSUPPORTED_SHAPE;
  if (n_rows > 0 && rows == nullptr) return FLP_INVALID_ARGUMENT;
  if (!aligned(rows, dtype_size(r))) return FLP_MISALIGNED;
  return FLP_OK;
}

namespace {
// The forward's gates.  own_scratch: the workspace is the library's own fixed
// array (the allocation-free entry point), which cannot overlap a caller's
// buffer, so only its size is checked.
flp_status forward_gates(int64_t N, int64_t D, int64_t V, flp_dtype x, const void* hidden,
                         const void* weight, const float* bias, const void* targets, flp_dtype t,
                         const float* temperature, const float* out_logp, const float* out_lse,
                         const void* workspace, size_t workspace_bytes, bool own_scratch) {
  flp_status st = check_dims(N, D, V, x, t);
  if (st != FLP_OK) return st;
  if (N == 0) return FLP_OK;
  if (!hidden || !weight || !targets || !out_logp || (!own_scratch && !workspace))
    return FLP_INVALID_ARGUMENT;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || (!own_scratch && !aligned(workspace, 16)) ||
      !aligned(bias, 4) || !aligned(temperature, 4) || !aligned(out_logp, 4) ||
      !aligned(out_lse, 4) || !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const size_t xs = dtype_size(x);
  const Span ins[] = {span(hidden, size_t(N) * D * xs), span(weight, size_t(V) * D * xs),
                      span(bias, size_t(V) * 4), span(targets, size_t(N) * dtype_size(t)),
                      span(temperature, size_t(N) * 4)};
  const Span outs[] = {span(out_logp, size_t(N) * 4), span(out_lse, size_t(N) * 4),
                       own_scratch ? Span() : span(workspace, workspace_bytes)};
  if (any_alias(outs, 3, ins, 5)) return FLP_INVALID_ARGUMENT;
  if (workspace_bytes < fwd_layout(N, D, V).total) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}
}  // namespace

flp_status validate_forward(int64_t N, int64_t D, int64_t V, flp_dtype x, const void* hidden,
                            const void* weight, const float* bias, const void* targets,
                            flp_dtype t, const float* temperature, const float* out_logp,
                            const float* out_lse, const void* workspace,
                            size_t workspace_bytes) {
  return forward_gates(N, D, V, x, hidden, weight, bias, targets, t, temperature, out_logp,
                       out_lse, workspace, workspace_bytes, false);
}

flp_status validate_forward_noalloc(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                    const void* hidden, const void* weight, const float* bias,
                                    const void* targets, flp_dtype t, const float* temperature,
                                    const float* out_logp, const float* out_lse,
                                    size_t scratch_bytes) {
  return forward_gates(N, D, V, x, hidden, weight, bias, targets, t, temperature, out_logp,
                       out_lse, nullptr, scratch_bytes, true);
}

flp_status validate_forward_partial(int64_t N, int64_t D, int64_t V_local, int64_t vocab_start,
                                    int64_t V_total, flp_dtype x, const void* hidden,
                                    const void* weight, const float* bias, const void* targets,
                                    flp_dtype t, const float* temperature, const void* partial,
                                    const float* zt) {
  flp_status st = check_dims(N, D, V_local, x, t);
  if (st != FLP_OK) return st;
  if (vocab_start < 0 || V_total < 1 || vocab_start > V_total - V_local) return FLP_INVALID_ARGUMENT;
  // Shard boundaries on vocabulary-tile boundaries keep every tile, and so every
  // partial, identical to the unsharded one.
  if (vocab_start % kVocabTile != 0) return FLP_UNSUPPORTED_SHAPE;
  if (V_local % kVocabTile != 0 && vocab_start + V_local != V_total) return FLP_UNSUPPORTED_SHAPE;
  if (N == 0) return FLP_OK;
  if (!hidden || !weight || !targets || !partial || !zt) return FLP_INVALID_ARGUMENT;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(partial, 16) || !aligned(zt, 4) ||
      !aligned(bias, 4) || !aligned(temperature, 4) || !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const size_t xs = dtype_size(x);
  const Span ins[] = {span(hidden, size_t(N) * D * xs), span(weight, size_t(V_local) * D * xs),
                      span(bias, size_t(V_local) * 4), span(targets, size_t(N) * dtype_size(t)),
                      span(temperature, size_t(N) * 4)};
  const Span outs[] = {span(partial, size_t(ceil_div(V_local, kVocabTile)) * size_t(N) * 8),
                       span(zt, size_t(N) * 4)};
  if (any_alias(outs, 2, ins, 5)) return FLP_INVALID_ARGUMENT;
  return FLP_OK;
}

flp_status validate_merge(int64_t N, int64_t V_total, const void* partials, const float* zt,
                          const void* targets, flp_dtype t, const float* out_logp,
                          const float* out_lse) {
  if (N < 0 || V_total < 1) return FLP_INVALID_ARGUMENT;
  if (t != FLP_I64 && t != FLP_I32) return FLP_UNSUPPORTED_DTYPE;
  const int64_t n_vt = ceil_div(V_total, kVocabTile);
  if (!mul_ok(n_vt, std::max<int64_t>(N, 1)) || !mul_ok(n_vt * std::max<int64_t>(N, 1), 8))
    return FLP_UNSUPPORTED_SHAPE;
  if (N == 0) return FLP_OK;
  if (!partials || !zt || !targets || !out_logp) return FLP_INVALID_ARGUMENT;
  if (!aligned(partials, 16) || !aligned(zt, 4) || !aligned(out_logp, 4) || !aligned(out_lse, 4) ||
      !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const Span ins[] = {span(partials, size_t(n_vt) * size_t(N) * 8), span(zt, size_t(N) * 4),
                      span(targets, size_t(N) * dtype_size(t))};
  const Span outs[] = {span(out_logp, size_t(N) * 4), span(out_lse, size_t(N) * 4)};
  if (any_alias(outs, 2, ins, 3)) return FLP_INVALID_ARGUMENT;
  return FLP_OK;
}

namespace {

flp_status check_logits_dims(int64_t N, int64_t V, flp_dtype x, flp_dtype t) {
  if (N < 0 || V < 1) return FLP_INVALID_ARGUMENT;
  if (x != FLP_BF16 && x != FLP_F16 && x != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if (t != FLP_I64 && t != FLP_I32) return FLP_UNSUPPORTED_DTYPE;
  // Rows are streamed in 16-byte chunks.
  if ((V * int64_t(dtype_size(x))) % 16 != 0) return FLP_UNSUPPORTED_SHAPE;
  const int64_t n = std::max<int64_t>(N, 1);
  if (!mul_ok(n, V) || !mul_ok(n * V, 8) || ceil_div(n, 4) > (int64_t(1) << 31) - 1)
    return FLP_UNSUPPORTED_SHAPE;
  return FLP_OK;
}

}  // namespace

flp_status validate_logits_forward(int64_t N, int64_t V, flp_dtype x, const void* logits,
                                   const void* targets, flp_dtype t, const float* out_logp,
                                   const float* out_lse) {
  flp_status st = check_logits_dims(N, V, x, t);
  if (st != FLP_OK || N == 0) return st;
  if (!logits || !targets || !out_logp) return FLP_INVALID_ARGUMENT;
  if (!aligned(logits, 16) || !aligned(out_logp, 4) || !aligned(out_lse, 4) ||
      !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const Span ins[] = {span(logits, size_t(N) * size_t(V) * dtype_size(x)),
                      span(targets, size_t(N) * dtype_size(t))};
  const Span outs[] = {span(out_logp, size_t(N) * 4), span(out_lse, size_t(N) * 4)};
  if (any_alias(outs, 2, ins, 2)) return FLP_INVALID_ARGUMENT;
  return FLP_OK;
}

flp_status validate_logits_backward(int64_t N, int64_t V, flp_dtype x, const float* grad_out,
                                    const float* lse, const void* logits, const void* targets,
                                    flp_dtype t, const void* d_logits) {
  flp_status st = check_logits_dims(N, V, x, t);
  if (st != FLP_OK || N == 0) return st;
  if (!grad_out || !lse || !logits || !targets || !d_logits) return FLP_INVALID_ARGUMENT;
  if (!aligned(logits, 16) || !aligned(d_logits, 16) || !aligned(grad_out, 4) ||
      !aligned(lse, 4) || !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const Span ins[] = {span(grad_out, size_t(N) * 4), span(lse, size_t(N) * 4),
                      span(logits, size_t(N) * size_t(V) * dtype_size(x)),
                      span(targets, size_t(N) * dtype_size(t))};
  const Span outs[] = {span(d_logits, size_t(N) * size_t(V) * dtype_size(x))};
  if (any_alias(outs, 1, ins, 4)) return FLP_INVALID_ARGUMENT;
  return FLP_OK;
}

flp_status validate_backward(int64_t N, int64_t D, int64_t V, flp_dtype x, const float* grad_out,
                             const float* lse, const void* hidden, const void* weight,
                             const float* bias, const void* targets, flp_dtype t,
                             const float* temperature, const void* d_hidden,
                             const void* d_weight, flp_dtype dw, const float* d_bias,
                             const void* workspace, size_t workspace_bytes) {
  flp_status st = check_dims(N, D, V, x, t);
  if (st != FLP_OK) return st;
  if (dw != x && dw != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if (N == 0) return validate_empty_sums(D, V, dtype_size(x), weight, bias, d_weight, dw, d_bias);
  if (!grad_out || !lse || !hidden || !weight || !targets) return FLP_INVALID_ARGUMENT;
  if (!d_hidden && !d_weight && !d_bias) return FLP_OK;
  if (!workspace) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x);
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(workspace, 16) ||
      !aligned(grad_out, 4) || !aligned(lse, 4) || !aligned(bias, 4) ||
      !aligned(temperature, 4) || !aligned(targets, dtype_size(t)) ||
      !aligned(d_hidden, 16) || !aligned(d_weight, 16) || !aligned(d_bias, 4))
    return FLP_MISALIGNED;
  const Span ins[] = {span(grad_out, size_t(N) * 4), span(lse, size_t(N) * 4),
                      span(hidden, size_t(N) * D * xs), span(weight, size_t(V) * D * xs),
                      span(bias, size_t(V) * 4), span(targets, size_t(N) * dtype_size(t)),
                      span(temperature, size_t(N) * 4)};
  const Span outs[] = {span(d_hidden, size_t(N) * D * xs),
                       span(d_weight, size_t(V) * D * dtype_size(dw)),
                       span(d_bias, size_t(V) * 4), span(workspace, workspace_bytes)};
  if (any_alias(outs, 4, ins, 7)) return FLP_INVALID_ARGUMENT;
  const BwdLayout L = bwd_layout_for_bytes(N, D, V, x, dw, workspace_bytes, d_hidden != nullptr,
                                           d_weight != nullptr, d_bias != nullptr);
  if (L.chunk == 0) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

flp_status validate_forward_indexed(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                    const void* hidden, const void* weight, const float* bias,
                                    const void* targets, flp_dtype t, const float* temperature,
                                    const void* rows, flp_dtype r, int64_t n_rows,
                                    const float* out_logp, const float* out_lse,
                                    const void* workspace, size_t workspace_bytes) {
  flp_status st = check_dims(N, D, V, x, t);
  if (st != FLP_OK) return st;
  if ((st = validate_rows(N, rows, r, n_rows)) != FLP_OK) return st;
  if (N == 0) return FLP_OK;
  if (!hidden || !weight || !targets || !out_logp || !workspace) return FLP_INVALID_ARGUMENT;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(workspace, 16) ||
      !aligned(bias, 4) || !aligned(temperature, 4) || !aligned(out_logp, 4) ||
      !aligned(out_lse, 4) || !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const size_t xs = dtype_size(x);
  const Span ins[] = {span(hidden, size_t(N) * D * xs), span(weight, size_t(V) * D * xs),
                      span(bias, size_t(V) * 4), span(targets, size_t(N) * dtype_size(t)),
                      span(temperature, size_t(N) * 4), span(rows, size_t(n_rows) * dtype_size(r))};
  const Span outs[] = {span(out_logp, size_t(N) * 4), span(out_lse, size_t(N) * 4),
                       span(workspace, workspace_bytes)};
  if (any_alias(outs, 3, ins, 6)) return FLP_INVALID_ARGUMENT;
  const IdxLayout L = idx_layout(N, D, n_rows, x, false, false);
  const size_t need = L.dense_off + (L.sel.cap > 0 ? fwd_layout(L.sel.cap, D, V).total : 0);
  if (workspace_bytes < need) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

flp_status validate_backward_indexed(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                     const float* grad_out, const float* lse, const void* hidden,
                                     const void* weight, const float* bias, const void* targets,
                                     flp_dtype t, const float* temperature, const void* rows,
                                     flp_dtype r, int64_t n_rows, const void* d_hidden,
                                     const void* d_weight, flp_dtype dw, const float* d_bias,
                                     const void* workspace, size_t workspace_bytes) {
  flp_status st = check_dims(N, D, V, x, t);
  if (st != FLP_OK) return st;
  if (dw != x && dw != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if ((st = validate_rows(N, rows, r, n_rows)) != FLP_OK) return st;
  if (N == 0) return validate_empty_sums(D, V, dtype_size(x), weight, bias, d_weight, dw, d_bias);
  if (!grad_out || !lse || !hidden || !weight || !targets) return FLP_INVALID_ARGUMENT;
  if (!d_hidden && !d_weight && !d_bias) return FLP_OK;
  if (!workspace) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x);
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(workspace, 16) ||
      !aligned(grad_out, 4) || !aligned(lse, 4) || !aligned(bias, 4) ||
      !aligned(temperature, 4) || !aligned(targets, dtype_size(t)) ||
      !aligned(d_hidden, 16) || !aligned(d_weight, 16) || !aligned(d_bias, 4))
    return FLP_MISALIGNED;
  const Span ins[] = {span(grad_out, size_t(N) * 4), span(lse, size_t(N) * 4),
                      span(hidden, size_t(N) * D * xs), span(weight, size_t(V) * D * xs),
                      span(bias, size_t(V) * 4), span(targets, size_t(N) * dtype_size(t)),
                      span(temperature, size_t(N) * 4), span(rows, size_t(n_rows) * dtype_size(r))};
  const Span outs[] = {span(d_hidden, size_t(N) * D * xs),
                       span(d_weight, size_t(V) * D * dtype_size(dw)),
                       span(d_bias, size_t(V) * 4), span(workspace, workspace_bytes)};
  if (any_alias(outs, 4, ins, 8)) return FLP_INVALID_ARGUMENT;
  const IdxLayout L = idx_layout(N, D, n_rows, x, true, d_hidden != nullptr);
  if (workspace_bytes < L.dense_off) return FLP_WORKSPACE_TOO_SMALL;
  if (L.sel.cap > 0 &&
      bwd_layout_for_bytes(L.sel.cap, D, V, x, dw, workspace_bytes - L.dense_off,
                           d_hidden != nullptr, d_weight != nullptr, d_bias != nullptr)
              .chunk == 0)
    return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

flp_status validate_logits_indexed(int64_t N, int64_t V, flp_dtype x, bool backward,
                                   const float* grad_out, const float* lse, const void* logits,
                                   const void* targets, flp_dtype t, const void* rows,
                                   flp_dtype r, int64_t n_rows, const void* out_a,
                                   const void* out_b, const void* workspace,
                                   size_t workspace_bytes) {
  flp_status st = check_logits_dims(N, V, x, t);
  if (st != FLP_OK) return st;
  if ((st = validate_rows(N, rows, r, n_rows)) != FLP_OK) return st;
  if (N == 0) return FLP_OK;
  if (!logits || !targets || !out_a || !workspace) return FLP_INVALID_ARGUMENT;
  if (backward && (!grad_out || !lse)) return FLP_INVALID_ARGUMENT;
  const size_t row_out = backward ? size_t(V) * dtype_size(x) : 4;
  if (!aligned(logits, 16) || !aligned(out_a, backward ? 16 : 4) || !aligned(out_b, 4) ||
      !aligned(grad_out, 4) || !aligned(lse, 4) || !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const Span ins[] = {span(logits, size_t(N) * size_t(V) * dtype_size(x)),
                      span(targets, size_t(N) * dtype_size(t)), span(grad_out, size_t(N) * 4),
                      span(lse, size_t(N) * 4), span(rows, size_t(n_rows) * dtype_size(r))};
  const Span outs[] = {span(out_a, size_t(N) * row_out), span(out_b, size_t(N) * 4),
                       span(workspace, workspace_bytes)};
  if (any_alias(outs, 3, ins, 5)) return FLP_INVALID_ARGUMENT;
  if (workspace_bytes < align_up(size_t(N))) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

namespace {

flp_status check_embedding_dims(int64_t N, int64_t D, int64_t V, flp_dtype x, flp_dtype id) {
  if (N < 0 || D < 1 || V < 1) return FLP_INVALID_ARGUMENT;
  if (x != FLP_BF16 && x != FLP_F16 && x != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if (id != FLP_I64 && id != FLP_I32) return FLP_UNSUPPORTED_DTYPE;
  // rows move in 16-byte chunks; token indices, sort keys (ids and the dropped-id
  // key V) and segment bounds are 32-bit
  if ((D * int64_t(dtype_size(x))) % 16 != 0) return FLP_UNSUPPORTED_SHAPE;
  if (N > kMaxIndexedRows || V > kMaxIndexedRows - 1) return FLP_UNSUPPORTED_SHAPE;
  if (!mul_ok(std::max<int64_t>(N, 1), D) || !mul_ok(V, D) || !mul_ok(V * D, 8))
    return FLP_UNSUPPORTED_SHAPE;
  return FLP_OK;
}

}  // namespace

flp_status validate_embedding_forward(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                      const void* weight, const void* ids, flp_dtype id,
                                      const void* out) {
  flp_status st = check_embedding_dims(N, D, V, x, id);
  if (st != FLP_OK || N == 0) return st;
  if (!weight || !ids || !out) return FLP_INVALID_ARGUMENT;
  if (!aligned(weight, 16) || !aligned(out, 16) || !aligned(ids, dtype_size(id)))
    return FLP_MISALIGNED;
  const size_t xs = dtype_size(x);
  const Span ins[] = {span(weight, size_t(V) * D * xs), span(ids, size_t(N) * dtype_size(id))};
  const Span outs[] = {span(out, size_t(N) * D * xs)};
  if (any_alias(outs, 1, ins, 2)) return FLP_INVALID_ARGUMENT;
  return FLP_OK;
}

flp_status validate_embedding_backward(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                       const void* grad, const void* ids, flp_dtype id,
                                       const void* d_weight, flp_dtype dw, const void* workspace,
                                       size_t workspace_bytes) {
  flp_status st = check_embedding_dims(N, D, V, x, id);
  if (st != FLP_OK) return st;
  if (dw != x && dw != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  // 128 threads per group of 32 positions, and a launch holds fewer than 2^32
  if (N >= (int64_t(1) << 30)) return FLP_UNSUPPORTED_SHAPE;
  if (!d_weight) return FLP_INVALID_ARGUMENT;
  if (N == 0) return validate_empty_sums(D, V, dtype_size(x), nullptr, nullptr, d_weight, dw, nullptr);
  if (!grad || !ids || !workspace) return FLP_INVALID_ARGUMENT;
  if (!aligned(grad, 16) || !aligned(d_weight, 16) || !aligned(workspace, 16) ||
      !aligned(ids, dtype_size(id)))
    return FLP_MISALIGNED;
  const size_t xs = dtype_size(x);
  const Span ins[] = {span(grad, size_t(N) * D * xs), span(ids, size_t(N) * dtype_size(id))};
  const Span outs[] = {span(d_weight, size_t(V) * D * dtype_size(dw)),
                       span(workspace, workspace_bytes)};
  if (any_alias(outs, 2, ins, 2)) return FLP_INVALID_ARGUMENT;
  if (workspace_bytes < emb_layout(N, D, V).total) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

LossFwdLayout loss_fwd_layout(int64_t N, int64_t D, int64_t V) {
  LossFwdLayout L;
  L.fwd = fwd_layout(N, D, V);
  L.rows_off = L.fwd.total;
  L.zsum_off = L.rows_off + align_up(size_t(N) * 4);
  L.total = L.zsum_off + align_up(size_t(L.fwd.n_vt) * size_t(N) * 4);
  return L;
}

float loss_zunit(int64_t V) {
  float u = 1.0f;
  for (int64_t v = 1; v < V; v *= 2) u *= 0.5f;
  return u;
}

LossGradLayout loss_grad_layout(int64_t N, int64_t D, int64_t V, flp_dtype x) {
  LossGradLayout L;
  const size_t row = align_up(size_t(N) * 4);
  L.onehot_off = row;
  L.uniform_off = 2 * row;
  L.unscale_off = 3 * row;
  L.slab_off = L.unscale_off + kAlign;
  L.total = L.slab_off;
  const int64_t ldz = round_up(V, kVocabTile);
  const int64_t slabs = std::min<int64_t>(kMaxSlabs, ldz / (x == FLP_F32 ? kMinSlabF32 : kMinSlab));
  if (N <= kSlabRows && slabs > 1) {
    L.k_slab = round_up(ceil_div(ldz, slabs), kVocabTile);
    L.total += align_up(size_t(ceil_div(ldz, L.k_slab)) * size_t(N) * size_t(D) * 4);
  }
  return L;
}

namespace {

flp_status check_loss_terms(double label_smoothing, double z_loss, flp_reduction reduction) {
  if (!(label_smoothing >= 0.0 && label_smoothing <= 1.0)) return FLP_INVALID_ARGUMENT;
  if (!(z_loss >= 0.0 && z_loss <= double(std::numeric_limits<float>::max())))
    return FLP_INVALID_ARGUMENT;
  if (reduction != FLP_REDUCE_NONE && reduction != FLP_REDUCE_SUM && reduction != FLP_REDUCE_MEAN)
    return FLP_INVALID_ARGUMENT;
  return FLP_OK;
}

}  // namespace

flp_status validate_cross_entropy_forward(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                          const void* hidden, const void* weight,
                                          const float* bias, const void* targets, flp_dtype t,
                                          double label_smoothing, double z_loss,
                                          flp_reduction reduction, const float* out_loss,
                                          const float* out_stats, const void* workspace,
                                          size_t workspace_bytes) {
  flp_status st = check_dims(N, D, V, x, t);
  if (st != FLP_OK) return st;
  if ((st = check_loss_terms(label_smoothing, z_loss, reduction)) != FLP_OK) return st;
  const bool rows = reduction == FLP_REDUCE_NONE;
  if (N == 0) {
    if (!rows && !out_loss) return FLP_INVALID_ARGUMENT;
    return aligned(out_loss, 4) ? FLP_OK : FLP_MISALIGNED;
  }
  if (!hidden || !weight || !targets || !out_loss || !workspace) return FLP_INVALID_ARGUMENT;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(workspace, 16) ||
      !aligned(bias, 4) || !aligned(out_loss, 4) || !aligned(out_stats, 4) ||
      !aligned(targets, dtype_size(t)))
    return FLP_MISALIGNED;
  const size_t xs = dtype_size(x);
  const Span ins[] = {span(hidden, size_t(N) * D * xs), span(weight, size_t(V) * D * xs),
                      span(bias, size_t(V) * 4), span(targets, size_t(N) * dtype_size(t))};
  const Span outs[] = {span(out_loss, rows ? size_t(N) * 4 : 4), span(out_stats, size_t(N) * 8),
                       span(workspace, workspace_bytes)};
  if (any_alias(outs, 3, ins, 4)) return FLP_INVALID_ARGUMENT;
  if (workspace_bytes < loss_fwd_layout(N, D, V).total) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

flp_status validate_cross_entropy_backward(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                           const float* grad_out, const float* stats,
                                           const void* hidden, const void* weight,
                                           const float* bias, const void* targets, flp_dtype t,
                                           double label_smoothing, double z_loss,
                                           flp_reduction reduction, const void* d_hidden,
                                           const void* d_weight, const float* d_bias,
                                           const void* workspace, size_t workspace_bytes) {
  flp_status st = check_dims(N, D, V, x, t);
  if (st != FLP_OK) return st;
  if ((st = check_loss_terms(label_smoothing, z_loss, reduction)) != FLP_OK) return st;
  if (N == 0) return validate_empty_sums(D, V, dtype_size(x), weight, bias, d_weight, x, d_bias);
  if (!grad_out || !stats || !hidden || !weight || !targets) return FLP_INVALID_ARGUMENT;
  if (!d_hidden && !d_weight && !d_bias) return FLP_OK;
  if (!workspace) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x);
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(workspace, 16) ||
      !aligned(grad_out, 4) || !aligned(stats, 4) || !aligned(bias, 4) ||
      !aligned(targets, dtype_size(t)) || !aligned(d_hidden, 16) || !aligned(d_weight, 16) ||
      !aligned(d_bias, 4))
    return FLP_MISALIGNED;
  const size_t g = reduction == FLP_REDUCE_NONE ? size_t(N) * 4 : 4;
  const Span ins[] = {span(grad_out, g), span(stats, size_t(N) * 8),
                      span(hidden, size_t(N) * D * xs), span(weight, size_t(V) * D * xs),
                      span(bias, size_t(V) * 4), span(targets, size_t(N) * dtype_size(t))};
  const Span outs[] = {span(d_hidden, size_t(N) * D * xs), span(d_weight, size_t(V) * D * xs),
                       span(d_bias, size_t(V) * 4), span(workspace, workspace_bytes)};
  if (any_alias(outs, 4, ins, 6)) return FLP_INVALID_ARGUMENT;
  const size_t front = loss_grad_layout(N, D, V, x).total;
  if (workspace_bytes < front) return FLP_WORKSPACE_TOO_SMALL;
  const BwdLayout L = bwd_layout_for_bytes(N, D, V, x, x, workspace_bytes - front,
                                           d_hidden != nullptr, d_weight != nullptr,
                                           d_bias != nullptr);
  return L.chunk == 0 ? FLP_WORKSPACE_TOO_SMALL : FLP_OK;
}

LossAllLayout loss_all_layout(int64_t N, int64_t D, int64_t V, flp_dtype x, int64_t chunk,
                              bool need_dh, bool need_dw, bool need_db) {
  LossAllLayout L;
  L.grad = loss_grad_layout(N, D, V, x);
  L.bwd = bwd_layout_for_chunk(N, D, V, x, x, chunk, need_dh, need_dw, need_db);
  const size_t rows = size_t(L.bwd.chunk), n_vt = size_t(L.bwd.ldz / kVocabTile);
  size_t off = L.grad.total;
  L.inv_off = off;
  off += kAlign;
  L.rows_off = off;
  off += align_up(size_t(N) * 4);
  L.lse_off = off;
  off += align_up(size_t(N) * 8);
  L.part_off = off;
  off += align_up(n_vt * rows * 8);
  L.zt_off = off;
  off += align_up(rows * 4);
  L.zsum_off = off;
  off += align_up(n_vt * rows * 4);
  L.logits_off = off;
  off += rows * size_t(L.bwd.ldz) * 4;
  L.bwd_off = off;
  L.total = off + L.bwd.total;
  return L;
}

LossAllLayout loss_all_layout_for_bytes(int64_t N, int64_t D, int64_t V, flp_dtype x, size_t bytes,
                                        bool need_dh, bool need_dw, bool need_db) {
  const int64_t full = ceil_div(std::max<int64_t>(N, 1), kRowQuantum);
  auto at = [&](int64_t nq) {
    return loss_all_layout(N, D, V, x, nq * kRowQuantum, need_dh, need_dw, need_db);
  };
  LossAllLayout L = at(full);
  if (L.total <= bytes) return L;
  int64_t lo = 0, hi = full - 1;  // the most quanta that fit: the size grows with them
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (at(mid).total <= bytes)
      lo = mid;
    else
      hi = mid - 1;
  }
  if (need_dh && lo > 0) lo = whole_waves(lo, D, x);
  if (lo < 1) return LossAllLayout();
  return at(lo);
}

flp_status validate_cross_entropy_gradients(int64_t N, int64_t D, int64_t V, flp_dtype x,
                                            const void* hidden, const void* weight,
                                            const float* bias, const void* targets, flp_dtype t,
                                            double label_smoothing, double z_loss,
                                            flp_reduction reduction, const float* out_loss,
                                            const float* out_stats, const void* d_hidden,
                                            const void* d_weight, const float* d_bias,
                                            const void* workspace, size_t workspace_bytes) {
  flp_status st = check_dims(N, D, V, x, t);
  if (st != FLP_OK) return st;
  if (x == FLP_F16) return FLP_UNSUPPORTED_DTYPE;
  if ((st = check_loss_terms(label_smoothing, z_loss, reduction)) != FLP_OK) return st;
  if (reduction == FLP_REDUCE_NONE || !out_loss) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x);
  if (N > 0 && (!hidden || !weight || !targets || !workspace)) return FLP_INVALID_ARGUMENT;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(workspace, 16) ||
      !aligned(bias, 4) || !aligned(targets, dtype_size(t)) || !aligned(out_loss, 4) ||
      !aligned(out_stats, 4) || !aligned(d_hidden, 16) || !aligned(d_weight, 16) ||
      !aligned(d_bias, 4))
    return FLP_MISALIGNED;
  const Span ins[] = {span(hidden, size_t(N) * D * xs), span(weight, size_t(V) * D * xs),
                      span(bias, size_t(V) * 4), span(targets, size_t(N) * dtype_size(t))};
  const Span outs[] = {span(out_loss, 4), span(out_stats, size_t(N) * 8),
                       span(d_hidden, size_t(N) * D * xs), span(d_weight, size_t(V) * D * xs),
                       span(d_bias, size_t(V) * 4),
                       span(N > 0 ? workspace : nullptr, workspace_bytes)};
  if (any_alias(outs, 6, ins, 4)) return FLP_INVALID_ARGUMENT;
  if (N == 0) return FLP_OK;
  const LossAllLayout L = loss_all_layout_for_bytes(N, D, V, x, workspace_bytes,
                                                    d_hidden != nullptr, d_weight != nullptr,
                                                    d_bias != nullptr);
  return L.bwd.chunk == 0 ? FLP_WORKSPACE_TOO_SMALL : FLP_OK;
}

flp_status validate_scale_inplace(int64_t n, flp_dtype x_dtype, const void* x,
                                  const float* factor) {
  if (n < 0) return FLP_INVALID_ARGUMENT;
  if (x_dtype != FLP_BF16 && x_dtype != FLP_F16 && x_dtype != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if (!mul_ok(n, 4)) return FLP_UNSUPPORTED_SHAPE;
  if (n == 0) return FLP_OK;
  if (!x || !factor) return FLP_INVALID_ARGUMENT;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(factor, 4)) return FLP_MISALIGNED;
  const Span ins[] = {span(factor, 4)};
  const Span outs[] = {span(x, size_t(n) * dtype_size(x_dtype))};
  return any_alias(outs, 1, ins, 1) ? FLP_INVALID_ARGUMENT : FLP_OK;
}

NormLayout norm_layout(int64_t N, int64_t D) {
  NormLayout L;
  L.slab_rows = std::max(kNormMinRows, ceil_div(N, kNormSlabs));
  L.slabs = ceil_div(N, L.slab_rows);
  L.total = align_up(size_t(L.slabs) * 2 * size_t(D) * 4);
  return L;
}

namespace {

flp_status check_norm_dims(int64_t N, int64_t D, flp_dtype x, flp_dtype w) {
  if (N < 0 || D < 1) return FLP_INVALID_ARGUMENT;
  if (x != FLP_BF16 && x != FLP_F16 && x != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if (w != x && w != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  // the column kernels take 16 columns per 256-thread workgroup, and a launch holds fewer
  // than 2^32 threads
  if (D >= (int64_t(1) << 27) || !mul_ok(std::max<int64_t>(N, 1), D)) return FLP_UNSUPPORTED_SHAPE;
  return FLP_OK;
}

}  // namespace

flp_status validate_layer_norm_forward(int64_t N, int64_t D, flp_dtype x_dtype, const void* x,
                                       flp_dtype w_dtype, const void* weight, const void* bias,
                                       double eps, const void* out, const float* mean,
                                       const float* rstd) {
  flp_status st = check_norm_dims(N, D, x_dtype, w_dtype);
  if (st != FLP_OK) return st;
  if (!(eps >= 0.0) || eps > double(std::numeric_limits<float>::max())) return FLP_INVALID_ARGUMENT;
  if (N == 0) return FLP_OK;
  if (!x || !out) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x_dtype), ws = dtype_size(w_dtype);
  if (!aligned(x, xs) || !aligned(out, xs) || !aligned(weight, ws) || !aligned(bias, ws) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return FLP_MISALIGNED;
  const Span ins[] = {span(x, size_t(N) * D * xs), span(weight, size_t(D) * ws),
                      span(bias, size_t(D) * ws)};
  const Span outs[] = {span(out, size_t(N) * D * xs), span(mean, size_t(N) * 4),
                       span(rstd, size_t(N) * 4)};
  return any_alias(outs, 3, ins, 3) ? FLP_INVALID_ARGUMENT : FLP_OK;
}

flp_status validate_layer_norm_backward(int64_t N, int64_t D, flp_dtype x_dtype, const void* grad,
                                        const void* x, flp_dtype w_dtype, const void* weight,
                                        const float* mean, const float* rstd, const void* d_x,
                                        const void* d_weight, const void* d_bias,
                                        const void* workspace, size_t workspace_bytes) {
  flp_status st = check_norm_dims(N, D, x_dtype, w_dtype);
  if (st != FLP_OK) return st;
  const size_t xs = dtype_size(x_dtype), ws = dtype_size(w_dtype);
  const bool params = d_weight != nullptr || d_bias != nullptr;
  if (!d_x && !params) return FLP_OK;
  if (N > 0 && (!grad || !x || !mean || !rstd || (params && !workspace)))
    return FLP_INVALID_ARGUMENT;
  if (!aligned(grad, xs) || !aligned(x, xs) || !aligned(d_x, xs) || !aligned(weight, ws) ||
      !aligned(d_weight, ws) || !aligned(d_bias, ws) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(workspace, 16))
    return FLP_MISALIGNED;
  const Span ins[] = {span(grad, size_t(N) * D * xs), span(x, size_t(N) * D * xs),
                      span(weight, size_t(D) * ws), span(mean, size_t(N) * 4),
                      span(rstd, size_t(N) * 4)};
  const Span outs[] = {span(d_x, size_t(N) * D * xs), span(d_weight, size_t(D) * ws),
                       span(d_bias, size_t(D) * ws),
                       span(params && N > 0 ? workspace : nullptr, workspace_bytes)};
  if (any_alias(outs, 4, ins, 5)) return FLP_INVALID_ARGUMENT;
  if (params && N > 0 && workspace_bytes < norm_layout(N, D).total) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

flp_status validate_dropout(int64_t n, flp_dtype x_dtype, const void* x, double p,
                            const int64_t* rng, const void* out) {
  if (n < 0 || !(p >= 0.0 && p <= 1.0)) return FLP_INVALID_ARGUMENT;
  if (x_dtype != FLP_BF16 && x_dtype != FLP_F16 && x_dtype != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
  if (!mul_ok(n, 4)) return FLP_UNSUPPORTED_SHAPE;
  if (n == 0) return FLP_OK;
  if (!x || !rng || !out) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x_dtype);
  if (!aligned(x, xs) || !aligned(out, xs) || !aligned(rng, 8)) return FLP_MISALIGNED;
  const Span ins[] = {span(x, size_t(n) * xs), span(rng, 16)};
  const Span outs[] = {span(out, size_t(n) * xs)};
  return any_alias(outs, 1, ins, 2) ? FLP_INVALID_ARGUMENT : FLP_OK;
}

GatedLayout gated_layout(int64_t N, int64_t D, int64_t F, flp_dtype x, bool need_dx,
                         bool need_dw) {
  GatedLayout L;
  const size_t xs = dtype_size(x);
  const bool wide = x == FLP_F32;
  L.fp = round_up(F, kGatedPad);
  L.np = round_up(N, kGatedPad);
  const int64_t K = 2 * L.fp;
  size_t at = 0;
  auto take = [&](size_t& off, size_t bytes) {
    off = at;
    at += align_up(bytes);
  };
  auto slab_of = [&](int64_t k, int64_t slabs) {  // of at least 256
    slabs = std::min({slabs, kGatedSlabs, k / 256});
    return slabs > 1 ? round_up(ceil_div(k, slabs), 128) : 0;
  };
  if (need_dx || !wide) take(L.dz_off, size_t(K) * N * xs);
  if (x == FLP_F16) {
    const int64_t across = ceil_div(L.fp, 256);
    L.parts = int(across * std::min(std::max<int64_t>(kGatedParts / across, 1), ceil_div(N, 16)));
    take(L.top_off, size_t(L.parts + 1) * 4);
  }
  if (wide && need_dx) take(L.wt_off, size_t(K) * D * xs);
  if (wide && need_dw) {
    take(L.dzt_off, size_t(K) * L.np * xs);
    take(L.xt_off, size_t(D) * L.np * xs);
  }
  size_t acc = 0;
  if (need_dx) {
    // what the smallest batch of the class needs to fill the chip, and no less than the class's own
    int64_t least = 1, own = kGatedSlabs;
    for (const GatedRows& c : kGatedRows)
      if (N > c.above) least = c.above + 1, own = c.slabs;
    L.dx_slab = slab_of(K, std::max(own, std::min(kGatedSlabs, ceil_div(kGatedTiles * 128 * 128, least * D))));
    if (L.dx_slab > 0) acc = size_t(ceil_div(K, L.dx_slab)) * N * D * 4;
  }
  if (need_dw && !wide) {
    L.dw_slab = slab_of(L.np, kGatedTiles / std::max<int64_t>(ceil_div(K, 128) * ceil_div(D, 128), 1));
    if (L.dw_slab > 0) acc = std::max(acc, size_t(ceil_div(L.np, L.dw_slab)) * K * D * 4);
  }
  take(L.acc_off, acc);
  L.total = at;
  return L;
}

namespace {

flp_status check_gated(int64_t N, int64_t D, int64_t F, flp_dtype x, flp_activation act) {
  const flp_status st = check_dims(N, D, F, x, FLP_I64);  // F stands where the vocabulary does
  if (st != FLP_OK) return st;
  if (act != FLP_ACT_SILU && act != FLP_ACT_GELU && act != FLP_ACT_GELU_TANH)
    return FLP_INVALID_ARGUMENT;
  // 256 rows of dz (of 2 F elements) stay below 2^31 bytes, and a launch holds fewer than 2^32
  // threads (256 for 64 x 64 elements of dz, the weights and x).  N: the interface's own limit; the
  // launches would hold more.
  if (N > int64_t(65535) * 64 || F > int64_t(32767) * 64) return FLP_UNSUPPORTED_SHAPE;
  const int64_t nt = ceil_div(N, 64), nc = ceil_div(F, 64), nd = ceil_div(D, 64);
  if (nc * nt + 2 * nc * nd + nt * nd >= (int64_t(1) << 24)) return FLP_UNSUPPORTED_SHAPE;
  return FLP_OK;
}

}  // namespace

flp_status validate_gated_forward(int64_t N, int64_t D, int64_t F, flp_dtype x_dtype, const void* x,
                                  const void* w_gate, const void* w_up, flp_activation act,
                                  const void* out, const void* saved) {
  const flp_status st = check_gated(N, D, F, x_dtype, act);
  if (st != FLP_OK || N == 0) return st;
  if (!x || !w_gate || !w_up || !out) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x_dtype);
  if (!aligned(x, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(out, xs) ||
      !aligned(saved, 16))
    return FLP_MISALIGNED;
  const Span ins[] = {span(x, size_t(N) * D * xs), span(w_gate, size_t(F) * D * xs),
                      span(w_up, size_t(F) * D * xs)};
  const Span outs[] = {span(out, size_t(N) * F * xs),
                       span(saved, gated_saved_bytes(N, F, x_dtype))};
  return any_alias(outs, 2, ins, 3) ? FLP_INVALID_ARGUMENT : FLP_OK;
}

flp_status validate_gated_backward(int64_t N, int64_t D, int64_t F, flp_dtype x_dtype,
                                   const void* grad, const void* saved, const void* x,
                                   const void* w_gate, const void* w_up, flp_activation act,
                                   const void* d_x, const void* d_w_gate, const void* d_w_up,
                                   const void* workspace, size_t workspace_bytes) {
  const flp_status st = check_gated(N, D, F, x_dtype, act);
  if (st != FLP_OK) return st;
  const bool dw = d_w_gate || d_w_up;
  if (!d_x && !dw) return FLP_OK;
  if (N > 0 && (!grad || !saved || !workspace)) return FLP_INVALID_ARGUMENT;
  if (N > 0 && ((d_x && (!w_gate || !w_up)) || (dw && !x))) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x_dtype);
  if (!aligned(grad, xs) || !aligned(saved, 16) || !aligned(x, 16) || !aligned(w_gate, 16) ||
      !aligned(w_up, 16) || !aligned(d_x, 16) || !aligned(d_w_gate, 16) || !aligned(d_w_up, 16) ||
      !aligned(workspace, 16))
    return FLP_MISALIGNED;
  const size_t weight = size_t(F) * D * xs, rows = size_t(N) * D * xs;
  const Span ins[] = {span(grad, size_t(N) * F * xs),
                      span(saved, gated_saved_bytes(N, F, x_dtype)),
                      span(x, rows), span(w_gate, weight), span(w_up, weight)};
  const Span outs[] = {span(d_x, rows), span(d_w_gate, weight), span(d_w_up, weight),
                       span(N > 0 ? workspace : nullptr, workspace_bytes)};
  if (any_alias(outs, 4, ins, 5)) return FLP_INVALID_ARGUMENT;
  if (N > 0 && workspace_bytes < gated_layout(N, D, F, x_dtype, d_x != nullptr, dw).total)
    return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

RmsLayout rms_layout(int64_t N, int64_t D, int64_t gate_rows) {
  RmsLayout L;
  L.gates = gate_rows > 1 && gate_rows == N;
  const int64_t parts = gate_rows > 1 && !L.gates ? gate_rows : 1;
  L.rows_per_gate = N / parts;
  L.slab_rows = std::min(std::max(kNormMinRows, ceil_div(N, kNormSlabs)),
                         std::max<int64_t>(L.rows_per_gate, 1));
  L.slabs_per_gate = ceil_div(L.rows_per_gate, L.slab_rows);
  L.slabs = L.slabs_per_gate * parts;
  L.total = align_up(size_t(L.slabs) * 2 * size_t(D) * 4);
  return L;
}

namespace {

flp_status check_rms(int64_t N, int64_t D, flp_dtype x_dtype, flp_dtype w_dtype, const void* y,
                     bool post, const void* post_weight, int64_t gate_rows, const void* gate,
                     double scale) {
  const flp_status st = check_norm_dims(N, D, x_dtype, w_dtype);
  if (st != FLP_OK) return st;
  if (gate_rows < 0 || !(std::fabs(scale) <= double(std::numeric_limits<float>::max())))
    return FLP_INVALID_ARGUMENT;
  if (D > kRmsMaxWidth) return FLP_UNSUPPORTED_SHAPE;
  if (N >= (int64_t(1) << 31)) return FLP_UNSUPPORTED_SHAPE;
  // the backward's workgroups of 512 threads, one for each of a gate row's rows at least, stay
  // below 2^32 threads in a launch
  if (N > gate_rows && gate_rows > kRmsMaxGates) return FLP_UNSUPPORTED_SHAPE;
  if (N > 0) {
    if (gate_rows > 0 && N % gate_rows != 0) return FLP_INVALID_ARGUMENT;
    if ((gate != nullptr) != (gate_rows > 0)) return FLP_INVALID_ARGUMENT;
    if (!y && (post || gate)) return FLP_INVALID_ARGUMENT;
  }
  return post_weight && !post ? FLP_INVALID_ARGUMENT : FLP_OK;
}

}  // namespace

flp_status validate_rms_forward(int64_t N, int64_t D, flp_dtype x_dtype, const void* x,
                                const void* y, flp_dtype w_dtype, const void* weight, bool post,
                                const void* post_weight, int64_t gate_rows, const void* gate,
                                double scale, double eps, const void* out_r, const void* out_n,
                                const float* rstd, const float* post_rstd) {
  flp_status st = check_rms(N, D, x_dtype, w_dtype, y, post, post_weight, gate_rows, gate, scale);
  if (st != FLP_OK) return st;
  if (!(eps >= 0.0) || eps > double(std::numeric_limits<float>::max())) return FLP_INVALID_ARGUMENT;
  if (N == 0) return FLP_OK;
  if (!x || !out_n || (y != nullptr) != (out_r != nullptr)) return FLP_INVALID_ARGUMENT;
  const size_t xs = dtype_size(x_dtype), ws = dtype_size(w_dtype);
  if (!aligned(x, xs) || !aligned(y, xs) || !aligned(out_r, xs) || !aligned(out_n, xs) ||
      !aligned(weight, ws) || !aligned(post_weight, ws) || !aligned(gate, ws) ||
      !aligned(rstd, 4) || !aligned(post_rstd, 4))
    return FLP_MISALIGNED;
  const size_t rows = size_t(N) * D * xs;
  const Span ins[] = {span(x, rows), span(y, rows), span(weight, size_t(D) * ws),
                      span(post_weight, size_t(D) * ws), span(gate, size_t(gate_rows) * D * ws)};
  const Span outs[] = {span(out_r, rows), span(out_n, rows), span(rstd, size_t(N) * 4),
                       span(post_rstd, size_t(N) * 4)};
  return any_alias(outs, 4, ins, 5) ? FLP_INVALID_ARGUMENT : FLP_OK;
}

flp_status validate_rms_backward(int64_t N, int64_t D, flp_dtype x_dtype, const void* grad_r,
                                 const void* grad_n, const void* x, const void* y,
                                 flp_dtype w_dtype, const void* weight, bool post,
                                 const void* post_weight, int64_t gate_rows, const void* gate,
                                 double scale, const float* rstd, const float* post_rstd,
                                 const void* d_x, const void* d_y, const void* d_weight,
                                 const void* d_post_weight, const void* d_gate,
                                 const void* workspace, size_t workspace_bytes) {
  flp_status st = check_rms(N, D, x_dtype, w_dtype, y, post, post_weight, gate_rows, gate, scale);
  if (st != FLP_OK) return st;
  const size_t xs = dtype_size(x_dtype), ws = dtype_size(w_dtype);
  const RmsLayout L = rms_layout(N, D, gate_rows);
  const bool sums = d_weight || d_post_weight || (d_gate && !L.gates);
  if (!d_x && !d_y && !sums && !d_gate) return FLP_OK;
  if (N > 0 && ((!grad_r && !grad_n) || !x || !rstd || (post && !post_rstd) || (sums && !workspace)))
    return FLP_INVALID_ARGUMENT;
  if (N > 0 && ((!y && (d_y || grad_r)) || (!gate && d_gate) || (!post && d_post_weight)))
    return FLP_INVALID_ARGUMENT;
  if (!aligned(grad_r, xs) || !aligned(grad_n, xs) || !aligned(x, xs) || !aligned(y, xs) ||
      !aligned(d_x, xs) || !aligned(d_y, xs) || !aligned(weight, ws) || !aligned(post_weight, ws) ||
      !aligned(gate, ws) || !aligned(d_weight, ws) || !aligned(d_post_weight, ws) ||
      !aligned(d_gate, ws) || !aligned(rstd, 4) || !aligned(post_rstd, 4) || !aligned(workspace, 16))
    return FLP_MISALIGNED;
  const size_t rows = size_t(N) * D * xs, one = size_t(D) * ws, gates = size_t(gate_rows) * one;
  const Span ins[] = {span(grad_r, rows),      span(grad_n, rows),
                      span(x, rows),           span(y, rows),
                      span(weight, one),       span(post_weight, one),
                      span(gate, gates),       span(rstd, size_t(N) * 4),
                      span(post_rstd, size_t(N) * 4)};
  const Span outs[] = {span(d_x, rows),          span(d_y, rows),
                       span(d_weight, one),      span(d_post_weight, one),
                       span(d_gate, gates),      span(sums && N > 0 ? workspace : nullptr,
                                                      workspace_bytes)};
  if (any_alias(outs, 6, ins, 9)) return FLP_INVALID_ARGUMENT;
  if (sums && N > 0 && workspace_bytes < L.total) return FLP_WORKSPACE_TOO_SMALL;
  return FLP_OK;
}

namespace {

// Whether an output span overlaps an input or another output, by a sweep over all of them (a
// step has thousands).
struct Range {
  uintptr_t lo, hi;
  bool out;
};
bool any_alias(std::vector<Range>& all) {
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t any = 0, outs = 0;  // the furthest ends so far
  for (const Range& r : all) {
    if (r.lo < outs || (r.out && r.lo < any)) return true;
    any = std::max(any, r.hi);
    if (r.out) outs = std::max(outs, r.hi);
  }
  return false;
}

}  // namespace

flp_status validate_adamw_step(int64_t n_tensors, const flp_adamw_tensor* tensors, int state_bits,
                               int64_t step, const int64_t* step_on_device, double lr,
                               const float* lr_on_device, double beta1, double beta2, double eps,
                               const float* grad_scale) {
  const double most = double(std::numeric_limits<float>::max());
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return FLP_INVALID_ARGUMENT;
  if (state_bits != 8 && state_bits != 32) return FLP_UNSUPPORTED_DTYPE;
  if (!step_on_device && step < 1) return FLP_INVALID_ARGUMENT;
  if (!lr_on_device && !(std::fabs(lr) <= most)) return FLP_INVALID_ARGUMENT;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return FLP_INVALID_ARGUMENT;
  if (!(eps >= 0.0 && eps <= most)) return FLP_INVALID_ARGUMENT;
  // the kernel multiplies by a reciprocal, infinite below: an element without moments would be 0 inf
  if (eps > 0.0 && eps < double(std::numeric_limits<float>::min())) return FLP_INVALID_ARGUMENT;
  if (!aligned(step_on_device, 8) || !aligned(lr_on_device, 4) || !aligned(grad_scale, 4))
    return FLP_MISALIGNED;
  const bool eight = state_bits == 8;
  try {
    std::vector<Range> all;
    all.reserve(size_t(n_tensors) * 7 + 3);
    auto add = [&](const void* p, int64_t bytes, bool out) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      if (p != nullptr) all.push_back({lo, lo + size_t(bytes), out});
    };
    add(step_on_device, 8, false);
    add(lr_on_device, 4, false);
    add(grad_scale, 4, false);
    for (int64_t k = 0; k < n_tensors; ++k) {
      const flp_adamw_tensor& t = tensors[k];
      const flp_dtype p = t.p_dtype, g = t.g_dtype;
      if (t.n < 0 || !(std::fabs(t.weight_decay) <= most)) return FLP_INVALID_ARGUMENT;
      if (p != FLP_BF16 && p != FLP_F16 && p != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
      if (g != p && g != FLP_F32) return FLP_UNSUPPORTED_DTYPE;
      if (!mul_ok(t.n, 4)) return FLP_UNSUPPORTED_SHAPE;
      if (t.n == 0) continue;
      if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return FLP_INVALID_ARGUMENT;
      if (eight && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return FLP_INVALID_ARGUMENT;
      const size_t ps = dtype_size(p), gs = dtype_size(g), ss = eight ? 1 : 4;
      if (!aligned(t.param, ps) || !aligned(t.grad, gs) || !aligned(t.exp_avg, ss) ||
          !aligned(t.exp_avg_sq, ss) || !aligned(t.master, 4) ||
          (eight && (!aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))))
        return FLP_MISALIGNED;
      add(t.param, t.n * int64_t(ps), true);
      add(t.grad, t.n * int64_t(gs), false);
      add(t.exp_avg, t.n * int64_t(ss), true);
      add(t.exp_avg_sq, t.n * int64_t(ss), true);
      add(t.master, t.n * 4, true);
      if (eight) {
        add(t.exp_avg_scale, ceil_div(t.n, kAdamBlock) * 4, true);
        add(t.exp_avg_sq_scale, ceil_div(t.n, kAdamBlock) * 4, true);
      }
    }
    return any_alias(all) ? FLP_INVALID_ARGUMENT : FLP_OK;
  } catch (const std::bad_alloc&) {
    return FLP_HIP_ERROR;
  }
}

}  // namespace flp
