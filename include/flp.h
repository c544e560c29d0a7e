/*
 * flp.h -- C ABI of the fused linear selected-token log-probability library
 * for AMD MI355X (gfx950).
 *
 * For token rows i = 0..N-1, vocabulary columns v = 0..V-1:
 *
 *   z_iv   = (hidden_i . W_v + b_v) / T_i            scaled logits (never stored)
 *   lse_i  = log sum_v exp(z_iv)
 *   logp_i = z_i[t_i] - lse_i     if 0 <= t_i < V, else exactly 0
 *
 * The operation is the one of the "Fused Linear LogP" docs page (section
 * "Reference Semantics": linear layer, log_softmax, gather at the target;
 * section "Tensor Contract": shapes, dtypes, float32 output
 * z[target] - logsumexp(z)).  The optional per-row temperature and the
 * fail-closed gates follow the "Feat/nemotron h lm head logprob cuda" page
 * (PR #555, summary bullets); the temperature divides the biased logits.
 * Out-of-range targets give logp = 0 and zero gradient (PR #234 inline
 * review; PR #547 page, section "What", indexed semantics).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers on the current HIP device,
 *     row-major and densely packed, owned by the caller.  The library
 *     allocates no device memory and keeps no state besides a once-
 *     initialised per-device property cache (and, only while the optional
 *     kernel timing below is enabled, a pool of HIP events); the calls are
 *     re-entrant.
 *   - Work is enqueued on `stream` (a hipStream_t, or NULL for the default
 *     stream) and the call returns at once (the measurement probes at the end
 *     are the one exception).  Outputs are valid once the stream has
 *     synchronised; device faults surface there.
 *   - Inputs are read-only.  Outputs are overwritten, never accumulated.
 *     No output may overlap any input or another output (checked from the
 *     address ranges; FLP_INVALID_ARGUMENT otherwise).
 *   - Every argument is validated before anything is enqueued.  On any
 *     non-OK status nothing has been enqueued and no output was touched.
 *     There is no fallback path: an unsupported case is an error.
 *   - N = 0 enqueues nothing, except that the backward calls still write
 *     d_weight and d_bias (when given) as zeros: they are sums over the
 *     rows, and a sum over no rows is zero.
 *   - Results are deterministic and batch-invariant: logp, lse and each row
 *     of d_hidden are bitwise the same whatever the other rows are, whatever
 *     N is and wherever the row sits; d_weight and d_bias are bitwise the
 *     same from run to run and for any backward workspace size.
 */
#ifndef FLP_H_
#define FLP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum flp_status {
  FLP_OK = 0,
  FLP_INVALID_ARGUMENT = 1,      /* null required pointer, N < 0, V < 1, D < 1, overlap */
  FLP_UNSUPPORTED_DTYPE = 2,     /* a dtype outside the lists below */
  FLP_UNSUPPORTED_SHAPE = 3,     /* D % 32 != 0, 256 * D * element size >= 2^31 (32-bit row
                                    offsets inside a 256-row tile), or a size beyond the
                                    64-bit index range */
  FLP_MISALIGNED = 4,            /* hidden/weight/workspace not 16-byte aligned, others not
                                    aligned to their element size */
  FLP_WORKSPACE_TOO_SMALL = 5,   /* workspace_bytes below the *_workspace_bytes minimum */
  FLP_UNSUPPORTED_DEVICE = 6,    /* current device is not gfx950 */
  FLP_HIP_ERROR = 7              /* a HIP runtime call or kernel launch failed */
} flp_status;

typedef enum flp_dtype {
  FLP_BF16 = 0,   /* bfloat16, 2 bytes */
  FLP_F32 = 1,    /* IEEE binary32 */
  FLP_I64 = 2,    /* int64 target ids */
  FLP_I32 = 3,    /* int32 target ids */
  FLP_F16 = 4     /* IEEE binary16 */
} flp_dtype;

/*
 * Forward workspace in bytes for (N, D, V): per-row, per-vocabulary-tile
 * partial (max, sum-of-exp) pairs and the target logits.  16-byte aligned.
 * These are the per-row softmax statistics of each vocabulary slab that the
 * "Fused Linear LogP" docs page folds instead of materialising the logits
 * (intro and "Tensor Parallel Vocab Shards": per-slab partials combined in a
 * fixed order); the caller provides the memory so that the library allocates
 * nothing.  Returns 0 for N < 0, D < 1 or V < 1.
 */
size_t flp_forward_workspace_bytes(int64_t N, int64_t D, int64_t V);

/*
 * Forward: out_logp[i] and (optionally) out_lse[i] for every row.
 *
 *   x_dtype      FLP_BF16, FLP_F16 or FLP_F32: element type of hidden and weight
 *                (the docs page's Tensor Contract lists bf16 / fp16 / fp32).
 *   hidden       [N, D] x_dtype, 16-byte aligned.
 *   weight       [V, D] x_dtype, 16-byte aligned.
 *   bias         [V] float32, or NULL for no bias.  Entries of -infinity or of a large
 *                negative value (-1e30, the lowest float32) mask their columns.
 *   targets      [N] ids of t_dtype (FLP_I64 or FLP_I32); any value is legal,
 *                an id outside [0, V) marks the row as ignored (logp = 0).
 *   temperature  [N] float32 (> 0, finite; not checked), or NULL for T = 1.
 *   out_logp     [N] float32.
 *   out_lse      [N] float32 log-sum-exp of the scaled logits, or NULL
 *                (rollout).  logp is bitwise the same either way.
 *   workspace    >= flp_forward_workspace_bytes(N, D, V) bytes, 16-byte
 *                aligned; scratch, contents undefined after the call.
 *   stream       hipStream_t to enqueue on.
 *
 * Requirements: D % 32 == 0, V >= 1, N >= 0.
 */
flp_status flp_forward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                       const void* hidden, const void* weight, const float* bias,
                       const void* targets, flp_dtype t_dtype,
                       const float* temperature,
                       float* out_logp, float* out_lse,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Largest forward workspace (flp_forward_workspace_bytes) that the
 * allocation-free forward serves: the size of its fixed per-device scratch
 * array, 33 MiB (at V = 131072, batches of up to 8439 rows).
 */
#define FLP_FORWARD_NOALLOC_MAX_BYTES ((size_t)33 << 20)

/*
 * Allocation-free forward, for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  The same computation as flp_forward, with the same bits, but the
 * workspace is a fixed array of FLP_FORWARD_NOALLOC_MAX_BYTES that the library
 * holds on every device it runs on (from the first call on that device until
 * the process ends); the caller passes only inputs and outputs.  The call
 * allocates nothing: no hipMalloc, no hipFree, no allocating library routine
 * (keep the optional kernel timing below off, since it creates HIP events).
 *
 * Arguments, gates and statuses as for flp_forward, plus FLP_WORKSPACE_TOO_SMALL
 * when flp_forward_workspace_bytes(N, D, V) exceeds FLP_FORWARD_NOALLOC_MAX_BYTES.
 * All calls on one device share its array: calls that overlap in time on one
 * device (two streams, two threads) race and must be serialised by the caller.
 */
flp_status flp_forward_noalloc(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                               const void* hidden, const void* weight, const float* bias,
                               const void* targets, flp_dtype t_dtype,
                               const float* temperature, float* out_logp, float* out_lse,
                               void* stream);

/*
 * Vocabulary shards ("Fused Linear LogP" docs page, "Tensor Parallel Vocab
 * Shards"): a rank that holds rows [vocab_start, vocab_start + V_local) of the
 * weight computes the per-tile partials of its slice; the partials of all
 * shards, concatenated in ascending vocabulary order, are folded by flp_merge
 * exactly as flp_forward folds its own, so the result is bitwise that of the
 * unsharded call.
 *
 * Bytes of the partial block of a shard of V_local rows: ceil(V_local / 256)
 * slabs x N (max, sum-of-exp) float pairs, slab-major ([slab][N] float2).
 */
size_t flp_forward_partial_bytes(int64_t N, int64_t V_local);

/*
 * Partial forward over one vocabulary shard.
 *
 *   weight       [V_local, D] x_dtype: rows vocab_start .. vocab_start + V_local - 1
 *                of the full weight.
 *   bias         [V_local] float32 slice of the full bias, or NULL.
 *   targets      [N] global ids (as for flp_forward).
 *   hidden, x_dtype, t_dtype, temperature: as for flp_forward.
 *   partial      flp_forward_partial_bytes(N, V_local) bytes, 16-byte aligned:
 *                the shard's [slab][N] (max, sum-of-exp) pairs.
 *   zt           [N] float32: the scaled target logit for rows whose target is
 *                in this shard, 0.0 for every other row, so that the shards' zt
 *                add up exactly to the full target logits.
 *
 * Requirements: vocab_start % 256 == 0; V_local % 256 == 0 unless the shard
 * ends the vocabulary (vocab_start + V_local == V_total); D % 32 == 0.
 */
flp_status flp_forward_partial(int64_t N, int64_t D, int64_t V_local, int64_t vocab_start,
                               int64_t V_total, flp_dtype x_dtype, const void* hidden,
                               const void* weight, const float* bias, const void* targets,
                               flp_dtype t_dtype, const float* temperature, void* partial,
                               float* zt, void* stream);

/*
 * Merge of the partials of all shards of a V_total vocabulary.
 *
 *   partials     [ceil(V_total / 256)][N] (max, sum-of-exp) float pairs: the
 *                shards' partial blocks concatenated in ascending vocabulary
 *                order; 16-byte aligned.
 *   zt           [N] float32: the sum of the shards' zt.
 *   targets      [N] global ids of t_dtype.
 *   out_logp     [N] float32; out_lse [N] float32 or NULL (as for flp_forward).
 */
flp_status flp_merge(int64_t N, int64_t V_total, const void* partials, const float* zt,
                     const void* targets, flp_dtype t_dtype, float* out_logp, float* out_lse,
                     void* stream);

/*
 * The sibling operator on materialised logits ("Fused LogP": the docs page's
 * intro contrasts it with the linear op; PR #234 "Summary" and "Implementation
 * details", PR #547 "What"): the same lse, selected log-probability and dlogits
 * definitions applied to given logits, with no projection, bias or temperature.
 *
 *   logits       [N, V] x_dtype (FLP_BF16, FLP_F16 or FLP_F32), row-major,
 *                16-byte aligned; V * element size must be a multiple of 16.
 *   targets      [N] ids of t_dtype; an id outside [0, V) gives logp = 0 and a
 *                zero gradient row.
 *   out_logp     [N] float32; out_lse [N] float32 or NULL.
 *
 * One wave per row streams the row once (online max / sum of exp per lane in
 * chunk order, then a fixed butterfly across the wave): a row's results do not
 * depend on the other rows.
 */
flp_status flp_logits_forward(int64_t N, int64_t V, flp_dtype x_dtype, const void* logits,
                              const void* targets, flp_dtype t_dtype, float* out_logp,
                              float* out_lse, void* stream);

/*
 *   d_logits[i, v] = G_i (onehot(t_i)_v - exp(logits[i, v] - lse_i)),
 *   G_i = grad_out[i] for in-range targets, else 0.
 *
 *   grad_out     [N] float32;  lse [N] float32 from flp_logits_forward.
 *   d_logits     [N, V] x_dtype (RNE from fp32), 16-byte aligned; must not
 *                overlap the inputs.
 */
flp_status flp_logits_backward(int64_t N, int64_t V, flp_dtype x_dtype, const float* grad_out,
                               const float* lse, const void* logits, const void* targets,
                               flp_dtype t_dtype, void* d_logits, void* stream);

/*
 * Backward workspace in bytes: the dlogits tile buffers the backward keeps
 * between its recompute and its two GEMMs ("Fused Linear LogP" docs page,
 * intro: tiled dlogits workspaces), the transposed operands, the d_bias
 * partials and, when the rows run in several chunks, the fp32 d_weight
 * accumulator that makes the chunking bit-neutral (PR #555 summary bullets:
 * chunked deterministic backward).  chunk_rows = 0 asks for the minimum (row
 * chunks of 256, or one chunk of the whole batch when that needs less because a
 * single chunk needs no fp32 d_W accumulator); a positive chunk_rows asks for the size that lets the
 * backward process that many rows per chunk (rounded up to a multiple of
 * 256, capped at N rounded up).  Any workspace at least the minimum is
 * accepted; a larger one gives larger chunks and the same bits.
 */
size_t flp_backward_workspace_bytes(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                    flp_dtype dw_dtype, int64_t chunk_rows);

/*
 * Rows per chunk that flp_backward uses with `workspace_bytes` of workspace
 * when the outputs flagged by need_* (0 or 1) are requested: a multiple of 256,
 * at most N rounded up to 256, or 0 when the workspace is below the minimum.
 * Pure host arithmetic (no device needed); the chunking never changes the bits.
 */
int64_t flp_backward_chunk_rows(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                flp_dtype dw_dtype, size_t workspace_bytes, int need_d_hidden,
                                int need_d_weight, int need_d_bias);

/*
 * Backward of L = sum_i grad_out[i] * logp[i]:
 *
 *   dz_iv     = G_i (onehot(t_i)_v - exp(z_iv - lse_i)) / T_i,
 *               G_i = grad_out[i] if 0 <= t_i < V else 0
 *   d_hidden  = dz W          [N, D] in x_dtype (RNE from fp32 accumulation)
 *   d_weight  = dz^T hidden   [V, D] in dw_dtype (fp32 accumulation over the
 *                              tokens in ascending order, one final rounding)
 *   d_bias    = sum_i dz_i    [V] float32
 *
 * (PR #234, "Implementation details": grad_out * (one_hot - softmax) from the
 * saved statistics; PR #555 summary: chunked deterministic backward whose
 * chunking is bit-neutral.)
 *
 *   grad_out     [N] float32.
 *   lse          [N] float32 as written by flp_forward for the same inputs.
 *   hidden, weight, bias, targets, t_dtype, temperature: as in flp_forward.
 *   d_hidden     [N, D] x_dtype, or NULL to skip.
 *   d_weight     [V, D] dw_dtype (x_dtype or FLP_F32), or NULL to skip.
 *   d_bias       [V] float32, or NULL to skip (allowed with bias == NULL).
 *   workspace    >= flp_backward_workspace_bytes(N, D, V, x_dtype, dw_dtype, 0).
 */
flp_status flp_backward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                        const float* grad_out, const float* lse,
                        const void* hidden, const void* weight, const float* bias,
                        const void* targets, flp_dtype t_dtype,
                        const float* temperature,
                        void* d_hidden, void* d_weight, flp_dtype dw_dtype,
                        float* d_bias,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Indexed (row-subset) variants (PR #547 "What", indexed semantics; PR #234
 * "Implementation details": rows left out by an indexed call get exactly zero
 * gradients).  A list of row ids selects which rows of the batch are computed:
 *
 *   rows         [n_rows] ids of r_dtype (FLP_I64 or FLP_I32), any order; may be
 *                NULL when n_rows == 0.  An id listed more than once selects its
 *                row once; an id outside [0, N) is ignored.
 *
 * Outputs keep the full row shape.  A selected row gets exactly the bits the
 * dense call gives it; every other row gets logp = 0, lse = 0 and zero
 * gradient rows.  d_weight and d_bias sum over the selected rows only.  The
 * linear variants gather the selected rows into the workspace (ascending row
 * order), run the dense kernels on them and scatter the results back, so their
 * cost scales with min(n_rows, N), not N.  No host synchronisation: the number
 * of distinct selected rows stays on the device, and the capacity min(n_rows, N)
 * sizes the work.  Row ids must be below 2^31.
 *
 * Workspace sizes depend on n_rows; flp_backward_indexed_workspace_bytes's
 * chunk_rows has the meaning it has for flp_backward_workspace_bytes, applied
 * to the selected rows.
 */
size_t flp_forward_indexed_workspace_bytes(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                           int64_t n_rows);
flp_status flp_forward_indexed(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                               const void* hidden, const void* weight, const float* bias,
                               const void* targets, flp_dtype t_dtype, const float* temperature,
                               const void* rows, flp_dtype r_dtype, int64_t n_rows,
                               float* out_logp, float* out_lse, void* workspace,
                               size_t workspace_bytes, void* stream);
size_t flp_backward_indexed_workspace_bytes(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                            flp_dtype dw_dtype, int64_t n_rows,
                                            int64_t chunk_rows);
/* lse: [N] as written by flp_forward_indexed (or flp_forward) for the same
 * inputs; only the selected rows are read. */
flp_status flp_backward_indexed(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                const float* grad_out, const float* lse, const void* hidden,
                                const void* weight, const float* bias, const void* targets,
                                flp_dtype t_dtype, const float* temperature, const void* rows,
                                flp_dtype r_dtype, int64_t n_rows, void* d_hidden,
                                void* d_weight, flp_dtype dw_dtype, float* d_bias,
                                void* workspace, size_t workspace_bytes, void* stream);

/* The operator on materialised logits, indexed: the workspace holds one byte
 * per row (the selection mask). */
size_t flp_logits_indexed_workspace_bytes(int64_t N);
flp_status flp_logits_forward_indexed(int64_t N, int64_t V, flp_dtype x_dtype,
                                      const void* logits, const void* targets, flp_dtype t_dtype,
                                      const void* rows, flp_dtype r_dtype, int64_t n_rows,
                                      float* out_logp, float* out_lse, void* workspace,
                                      size_t workspace_bytes, void* stream);
flp_status flp_logits_backward_indexed(int64_t N, int64_t V, flp_dtype x_dtype,
                                       const float* grad_out, const float* lse,
                                       const void* logits, const void* targets,
                                       flp_dtype t_dtype, const void* rows, flp_dtype r_dtype,
                                       int64_t n_rows, void* d_logits, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * Untied embedding lookup ("Feat/nemotron h lm head logprob cuda", PR #555
 * summary bullets: the untied embedding lookup of the same model row, with a
 * sorted-segment deterministic grad_weight; its Known issues: the pages'
 * version accumulates repeated ids in BF16 and misses FP64 parity, so here each
 * segment accumulates in fp32 and is rounded once).
 *
 *   out[i]    = weight[ids[i]]                        [N, D] x_dtype
 *   d_weight  = sum over i with ids[i] == v of grad[i], summed in ascending i
 *
 *   x_dtype   FLP_BF16, FLP_F16 or FLP_F32 (weight, out, grad); D * element
 *             size must be a multiple of 16.
 *   ids       [N] of id_dtype (FLP_I64 or FLP_I32).  An id outside [0, V)
 *             reads as a zero row and contributes no gradient.
 *   d_weight  [V, D] of dw_dtype (x_dtype or FLP_F32); every row is written
 *             (zero for ids that do not occur).
 *   workspace >= flp_embedding_backward_workspace_bytes(N, D, V): radix-sort
 *             buffers, per-id segment bounds and fp32 pieces of segments that
 *             span several 32-position groups of the sorted list.
 *
 * The backward sorts (id, token) pairs with a stable radix sort and sums each
 * id's segment in fp32 in a fixed order (token order inside each group of 32
 * sorted positions, groups in ascending order): d_weight is bitwise
 * reproducible.  N < 2^31 (2^30 in the backward),
 * V < 2^31 - 1.
 */
flp_status flp_embedding_forward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                 const void* weight, const void* ids, flp_dtype id_dtype,
                                 void* out, void* stream);
size_t flp_embedding_backward_workspace_bytes(int64_t N, int64_t D, int64_t V);
flp_status flp_embedding_backward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                  const void* grad, const void* ids, flp_dtype id_dtype,
                                  void* d_weight, flp_dtype dw_dtype, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * The lookup with a scaling factor, as models that multiply their embedding by
 * sqrt(D) use it: out[i] = scale * weight[ids[i]] (each product rounded once to
 * x_dtype), and d_weight = scale * (the sum above), the fp32 sum times scale rounded
 * once.  scale: any finite value.  Everything else as for the two calls above, whose
 * results scale = 1 gives bit for bit; the backward's workspace is
 * flp_embedding_backward_workspace_bytes(N, D, V).
 */
flp_status flp_embedding_scaled_forward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                        const void* weight, const void* ids, flp_dtype id_dtype,
                                        float scale, void* out, void* stream);
flp_status flp_embedding_scaled_backward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                         const void* grad, const void* ids, flp_dtype id_dtype,
                                         float scale, void* d_weight, flp_dtype dw_dtype,
                                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Dropout between the embedding and the head, with a mask that is never stored:
 *
 *   out[e] = x[e] / (1 - q) where u[e] >= 65536 q, else 0;   q = round(65536 p) / 65536
 *
 * u[e] is the 16-bit piece e % 8 (low halves first) of the 128 bits that the ten-round
 * 4 x 32 counter-based generator of Salmon et al. (2011) gives for the key rng[0] and
 * the counter (e / 8, rng[1]).  The mask depends on e, p and rng only: the backward is
 * the same call on the gradient, with the same p and rng.  A dropped element is 0
 * whatever x[e] is (infinite or NaN included).
 *
 *   n         elements; x and out are [n] x_dtype (FLP_BF16, FLP_F16 or FLP_F32),
 *             aligned to their element size.
 *   p         probability of dropping, 0 <= p <= 1 (rounded to a multiple of 2^-16;
 *             1 drops everything).
 *   rng       two int64 on the device: seed and offset, any values (read as unsigned).
 *             Calls with different offsets draw independent masks; since they are
 *             read on the device, a captured call draws a new mask when the caller
 *             changes them between replays.
 */
flp_status flp_dropout(int64_t n, flp_dtype x_dtype, const void* x, double p, const int64_t* rng,
                       void* out, void* stream);

/*
 * Softmax cross entropy of the projected rows, z_iv = hidden_i . W_v + b_v: the training
 * loss whose per-token part is -logp of flp_forward, with label smoothing s and a squared
 * log-partition term c (the logits are not kept; flp_cross_entropy_gradients holds those
 * of one row chunk in its workspace):
 *
 *   loss_i = (1 - s) (lse_i - z_i[t_i]) + s (lse_i - mean_v z_iv) + c lse_i^2
 *
 * for rows whose target lies in [0, V); the others (padding) have loss 0 exactly, take
 * part in no sum or count and get zero gradients, whatever their hidden row holds.
 *
 *   label_smoothing  0 <= s <= 1.   z_loss  c >= 0, finite.
 *   reduction    FLP_REDUCE_NONE: out_loss [N]; FLP_REDUCE_SUM: out_loss [1], the sum;
 *                FLP_REDUCE_MEAN: out_loss [1], the sum over the number of counted rows
 *                (0 when there are none).
 *   out_loss     float32.
 *   out_stats    [2, N] float32, or NULL: lse, and the part of it that its rounding left
 *                out (0 unless lse is large); the backward reads both.
 *   workspace    >= flp_cross_entropy_forward_workspace_bytes(N, D, V), 16-byte aligned.
 *   N = 0 writes 0 to a reduced loss.
 *   Everything else as for flp_forward.
 *
 * A vocabulary entry masked through the bias (-infinity, or the lowest float32) has
 * probability 0; with label smoothing an entry of -infinity makes the loss infinite, as
 * its definition does.  A NaN logit makes the loss and lse of its row NaN (unless the row
 * is padding).  The rows' losses and lse do not depend on the other rows; the
 * reductions add the rows in an order fixed by N.
 */
typedef enum flp_reduction {
  FLP_REDUCE_NONE = 0,
  FLP_REDUCE_SUM = 1,
  FLP_REDUCE_MEAN = 2
} flp_reduction;

size_t flp_cross_entropy_forward_workspace_bytes(int64_t N, int64_t D, int64_t V);
flp_status flp_cross_entropy_forward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                     const void* hidden, const void* weight, const float* bias,
                                     const void* targets, flp_dtype t_dtype,
                                     double label_smoothing, double z_loss,
                                     flp_reduction reduction, float* out_loss, float* out_stats,
                                     void* workspace, size_t workspace_bytes, void* stream);
/*
 *   dz_iv    = g_i ((1 + 2 c lse_i) exp(z_iv - lse_i) - (1 - s) onehot(t_i)_v - s / V)
 *   d_hidden = dz W,  d_weight = dz^T hidden,  d_bias = sum_i dz_i
 *
 * g_i is grad_out[i] (FLP_REDUCE_NONE), grad_out[0] (FLP_REDUCE_SUM) or grad_out[0] over
 * the number of counted rows (FLP_REDUCE_MEAN), 0 for rows that are not counted.
 *
 *   stats      [2, N] as written by the forward for the same inputs.
 *   d_hidden [N, D], d_weight [V, D] x_dtype, d_bias [V] float32: each may be NULL.
 *   workspace  >= flp_cross_entropy_backward_workspace_bytes(N, D, V, x_dtype, 0);
 *              chunk_rows as for flp_backward_workspace_bytes.
 *
 * For FLP_F16, dz is held times a power of two that brings its largest row factor to
 * 2^10, taken back when the fp32 sums are rounded: small gradients (a mean over many
 * rows) do not underflow on the way.
 *
 * For 16-bit types dz is rounded to x_dtype between its fp32 epilogue and the two
 * products, whose matrix instructions take operands of that type (as flp_backward does);
 * d_bias adds the unrounded entries.  The error this adds to d_hidden and d_weight is that
 * of one more rounding of their size.
 *
 * Batches of up to 8192 rows sum d_hidden over slabs of the vocabulary, larger ones in
 * one walk: a row's d_hidden is bitwise the same among batches of one kind, and differs
 * between the two by the order of that fp32 sum.
 */
size_t flp_cross_entropy_backward_workspace_bytes(int64_t N, int64_t D, int64_t V,
                                                  flp_dtype x_dtype, int64_t chunk_rows);
flp_status flp_cross_entropy_backward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                      const float* grad_out, const float* stats,
                                      const void* hidden, const void* weight, const float* bias,
                                      const void* targets, flp_dtype t_dtype,
                                      double label_smoothing, double z_loss,
                                      flp_reduction reduction, void* d_hidden, void* d_weight,
                                      float* d_bias, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Loss and gradients of a training step in one call, for an upstream gradient of 1
 * (reduction FLP_REDUCE_SUM or FLP_REDUCE_MEAN; FLP_BF16 or FLP_F32).  Row chunk by row
 * chunk, the forward leaves its fp32 logits in the workspace and dz is made from them
 * instead of from a second product, so a step takes three products of the size of the
 * logits where forward and backward calls take four.  out_loss, out_stats and the
 * gradients have the bits of those two calls with grad_out = 1.
 *
 *   out_loss   [1].  out_stats [2, N] or NULL.  d_hidden, d_weight, d_bias as for
 *              flp_cross_entropy_backward, each may be NULL.
 *   workspace  >= flp_cross_entropy_gradients_workspace_bytes(N, D, V, x_dtype, 0);
 *              chunk_rows as for flp_backward_workspace_bytes.  A chunk of all rows takes
 *              about 8 (FLP_BF16) or 12 (FLP_F32) bytes per logit.
 *   N = 0 writes zeros to out_loss, d_weight and d_bias.
 */
size_t flp_cross_entropy_gradients_workspace_bytes(int64_t N, int64_t D, int64_t V,
                                                   flp_dtype x_dtype, int64_t chunk_rows);
flp_status flp_cross_entropy_gradients(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype,
                                       const void* hidden, const void* weight, const float* bias,
                                       const void* targets, flp_dtype t_dtype,
                                       double label_smoothing, double z_loss,
                                       flp_reduction reduction, float* out_loss, float* out_stats,
                                       void* d_hidden, void* d_weight, float* d_bias,
                                       void* workspace, size_t workspace_bytes, void* stream);
/*
 * x[e] *= *factor in place (one rounding), for gradients made with an upstream gradient
 * of 1.  x: [n] x_dtype, aligned to its element size; factor: one float32 on the device.
 * A factor of exactly 1 leaves x alone and costs a launch.
 */
flp_status flp_scale_inplace(int64_t n, flp_dtype x_dtype, void* x, const float* factor,
                             void* stream);

/*
 * Layer norm of the rows x[i, :], as it stands in front of the head:
 *
 *   mean_i = sum_d x_id / D,   rstd_i = 1 / sqrt(sum_d (x_id - mean_i)^2 / D + eps)
 *   out    = (x - mean) rstd weight + bias
 *
 *   x, out    [N, D] x_dtype (FLP_BF16, FLP_F16 or FLP_F32).  Any D >= 1 (below 2^27):
 *             rows need no alignment beyond their element size.
 *   weight, bias  [D] of w_dtype (x_dtype or FLP_F32), each may be NULL (1 and 0).
 *   eps       >= 0, finite.  A constant row with eps = 0 has no norm (NaN).  The sums are
 *             fp32: a row whose squared deviations add up to more than fp32 holds (3.4e38)
 *             has rstd 0, one whose squares all vanish (below 2^-150) counts as constant.
 *   out_mean, out_rstd  [N] float32, or NULL; the backward reads both.
 *
 * fp32 arithmetic, one rounding per output element; a row's results do not depend on
 * the other rows.
 */
flp_status flp_layer_norm_forward(int64_t N, int64_t D, flp_dtype x_dtype, const void* x,
                                  flp_dtype w_dtype, const void* weight, const void* bias,
                                  double eps, void* out, float* out_mean, float* out_rstd,
                                  void* stream);
/*
 *   d_x       = rstd (g - mean_d(g) - xhat mean_d(g xhat)),  g = grad_out * weight
 *   d_weight  = sum_i grad_out_i xhat_i,   d_bias = sum_i grad_out_i
 *
 *   grad_out, d_x       [N, D] x_dtype.  d_weight, d_bias [D] w_dtype.  d_x, d_weight
 *             and d_bias may each be NULL to skip it.
 *   mean, rstd  [N] as written by the forward for the same x and eps.
 *   workspace >= flp_layer_norm_backward_workspace_bytes(N, D) bytes, 16-byte aligned:
 *             partial sums of d_weight and d_bias (not needed, and not touched, when
 *             both are NULL).
 *
 * The sums over rows are fp32 in a fixed order and rounded once; N = 0 writes zeros to
 * d_weight and d_bias.
 */
size_t flp_layer_norm_backward_workspace_bytes(int64_t N, int64_t D);
flp_status flp_layer_norm_backward(int64_t N, int64_t D, flp_dtype x_dtype, const void* grad_out,
                                   const void* x, flp_dtype w_dtype, const void* weight,
                                   const float* mean, const float* rstd, void* d_x,
                                   void* d_weight, void* d_bias, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * The first half of a gated feed-forward block: both projections, the activation and the
 * product in one kernel:
 *
 *   z = x w_gate^T,   u = x w_up^T,   out = act(z) u
 *
 *   activation   FLP_ACT_SILU       z / (1 + exp(-z))
 *                FLP_ACT_GELU       z Phi(z), Phi the normal distribution function
 *                FLP_ACT_GELU_TANH  0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
 *   x            [N, D] x_dtype (FLP_BF16, FLP_F16 or FLP_F32), 16-byte aligned.
 *   w_gate, w_up [F, D] x_dtype, each 16-byte aligned (they may be the halves of one [2 F, D]).
 *   out          [N, F] x_dtype, aligned to its element size; made in fp32 from the fp32 sums
 *                and rounded once.
 *   saved        flp_gated_linear_saved_bytes(N, F, x_dtype) bytes, 16-byte aligned: act(z)
 *                and u act'(z) for the backward, in 24 bits each (fp32: 32) and a layout of
 *                their own; or NULL.
 *
 * Requirements: D % 32 == 0 (and the size limits of flp_forward), 1 <= F <= 64 * 32767,
 * N <= 64 * 65535, N F + 2 D F + N D below about 2^36.
 */
typedef enum flp_activation {
  FLP_ACT_SILU = 0,
  FLP_ACT_GELU = 1,
  FLP_ACT_GELU_TANH = 2
} flp_activation;

size_t flp_gated_linear_saved_bytes(int64_t N, int64_t F, flp_dtype x_dtype);
flp_status flp_gated_linear_forward(int64_t N, int64_t D, int64_t F, flp_dtype x_dtype,
                                    const void* x, const void* w_gate, const void* w_up,
                                    flp_activation activation, void* out, void* saved,
                                    void* stream);
/*
 *   dz  = grad_out u act'(z),   du = grad_out act(z)
 *   d_x = dz w_gate + du w_up,   d_w_gate = dz^T x,   d_w_up = du^T x
 *
 *   grad_out   [N, F] x_dtype, aligned to its element size.
 *   saved      as written by the forward for the same inputs, activation among them: it holds
 *              act(z) and u act'(z), so that activation is checked here, but not used again.
 *   d_x [N, D], d_w_gate, d_w_up [F, D] x_dtype, 16-byte aligned: each may be NULL to skip it.
 *   workspace  >= flp_gated_linear_backward_workspace_bytes(N, D, F, x_dtype, d_x wanted, a
 *              weight gradient wanted), 16-byte aligned: dz and du (2 N F elements; fp32: also
 *              transposed, with the weights and x), and fp32 sums over slabs of small products.
 *
 * For 16-bit types dz and du are rounded to x_dtype on the way, whose matrix instructions take
 * operands of that type; the products' sums are fp32 and rounded once.  FLP_F16: where the
 * largest finite magnitude in dz and du is below 1, or 2^15 or more, they are held times the power
 * of two that takes it to about 2^10, and the sums times its inverse, so that they keep their
 * bits.  The sums run in an order fixed by the sizes; d_x of a row is bitwise the same among batches
 * of up to 512 rows, and among those of more, up to 1024, 2048, 8192 and beyond (FLP_F16: of those
 * with the same power of two).  N = 0 writes zeros to d_w_gate and d_w_up.
 */
size_t flp_gated_linear_backward_workspace_bytes(int64_t N, int64_t D, int64_t F,
                                                 flp_dtype x_dtype, int need_d_x,
                                                 int need_d_weights);
flp_status flp_gated_linear_backward(int64_t N, int64_t D, int64_t F, flp_dtype x_dtype,
                                     const void* grad_out, const void* saved, const void* x,
                                     const void* w_gate, const void* w_up,
                                     flp_activation activation, void* d_x, void* d_w_gate,
                                     void* d_w_up, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * Root mean square norm of the rows x[i, :]:
 *
 *   rstd_i = 1 / sqrt(sum_d x_id^2 / D + eps),   out = x rstd weight
 *
 *   x, out    [N, D] x_dtype (FLP_BF16, FLP_F16 or FLP_F32), 1 <= D <= 16384, N < 2^31: rows
 *             need no alignment beyond their element size.
 *   weight    [D] of w_dtype (x_dtype or FLP_F32), or NULL for 1.
 *   eps       >= 0, finite.  A row of zeros with eps = 0 has no norm (NaN).  Rows of any size
 *             have their norm, as long as fp32 holds rstd.
 *   out_rstd  [N] float32, or NULL; the backward reads it.
 *
 * fp32 arithmetic, one rounding per output element; a row's results do not depend on the
 * other rows.
 *
 * Backward:  g = grad_out weight,  d_x = rstd (g - xhat mean_d(g xhat)),
 *            d_weight = sum_i grad_out_i xhat_i,   xhat = x rstd
 *
 *   d_x, d_weight   may each be NULL.  workspace as for flp_residual_rms_norm_backward, with
 *   gate_rows = 0.
 */
flp_status flp_rms_norm_forward(int64_t N, int64_t D, flp_dtype x_dtype, const void* x,
                                flp_dtype w_dtype, const void* weight, double eps, void* out,
                                float* out_rstd, void* stream);
flp_status flp_rms_norm_backward(int64_t N, int64_t D, flp_dtype x_dtype, const void* grad_out,
                                 const void* x, flp_dtype w_dtype, const void* weight,
                                 const float* rstd, void* d_x, void* d_weight, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * What stands between two blocks of a model: the residual stream x takes in the block's
 * output y, and the next block's (or the head's) norm is made in the same pass:
 *
 *   p = y rstd(y) post_weight  (post_norm nonzero)   or  p = y
 *   r = x + scale gate p,      n = r rstd(r) weight
 *
 * with the norm and the rounding of flp_rms_norm_forward (n is made from r before its
 * rounding).
 *
 *   x, y, out_r, out_n   [N, D] x_dtype.  y = NULL (with post_norm = 0, no gate, out_r = NULL)
 *                is flp_rms_norm_forward.
 *   weight, post_weight  [D] of w_dtype, each may be NULL for 1 (post_weight only with
 *                post_norm).
 *   gate         [gate_rows, D] of w_dtype, N a multiple of gate_rows: row i takes gate row
 *                i / (N / gate_rows).  One row is a gate per channel, one per sequence a
 *                modulation, N rows a gate per element; others than N at most 2^22.  NULL with
 *                gate_rows = 0 for 1.
 *   scale        finite.
 *   out_rstd, out_post_rstd  [N] float32, or NULL; the backward reads them (the second with
 *                post_norm only).
 */
flp_status flp_residual_rms_norm_forward(int64_t N, int64_t D, flp_dtype x_dtype, const void* x,
                                         const void* y, flp_dtype w_dtype, const void* weight,
                                         int post_norm, const void* post_weight,
                                         int64_t gate_rows, const void* gate, double scale,
                                         double eps, void* out_r, void* out_n, float* out_rstd,
                                         float* out_post_rstd, void* stream);
/*
 *   gw  = grad_n weight,   d_x = grad_r + rstd (gw - rhat mean_d(gw rhat)),   rhat = r rstd
 *   d_weight = sum_i grad_n rhat,   d_gate = sum over a gate's rows of scale d_x p
 *   g   = scale gate d_x post_weight,   d_post_weight = sum_i scale gate d_x yhat
 *   d_y = rstd_y (g - yhat mean_d(g yhat)),   yhat = y rstd_y;   without post_norm d_y = g
 *
 *   grad_r, grad_n  [N, D] x_dtype; one of them may be NULL (zero).
 *   rstd, post_rstd as written by the forward for the same inputs.
 *   d_x, d_y [N, D] x_dtype, d_weight, d_post_weight [D], d_gate [gate_rows, D] w_dtype: each
 *                may be NULL to skip it.
 *   workspace >= flp_residual_rms_norm_backward_workspace_bytes(N, D, gate_rows), 16-byte
 *                aligned: partial sums over rows (not needed, and not touched, when d_weight,
 *                d_post_weight and a d_gate of fewer than N rows are all NULL).
 *
 * The sums over rows are fp32 in a fixed order and rounded once; N = 0 writes zeros to them.
 */
size_t flp_residual_rms_norm_backward_workspace_bytes(int64_t N, int64_t D, int64_t gate_rows);
flp_status flp_residual_rms_norm_backward(
    int64_t N, int64_t D, flp_dtype x_dtype, const void* grad_r, const void* grad_n, const void* x,
    const void* y, flp_dtype w_dtype, const void* weight, int post_norm, const void* post_weight,
    int64_t gate_rows, const void* gate, double scale, const float* rstd, const float* post_rstd,
    void* d_x, void* d_y, void* d_weight, void* d_post_weight, void* d_gate, void* workspace,
    size_t workspace_bytes, void* stream);

/*
 * One AdamW step over many tensors at once, with decoupled weight decay:
 *
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t)  m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * in fp32, element by element; param, the states and the master copy are updated in place.
 *
 *   tensors      n_tensors descriptors in HOST memory, read during the call.  Their types may
 *                differ from tensor to tensor; a tensor with n = 0 is left alone.
 *   p_dtype      FLP_BF16, FLP_F16 or FLP_F32.  g_dtype: the same, or FLP_F32.
 *   master       [n] float32 copy of the parameters that the step updates, param then being
 *                its rounding; or NULL: param is updated and rounded itself.
 *   state_bits   32: exp_avg and exp_avg_sq are [n] float32, m and v.
 *                8: they are [n] bytes, e4m3 codes of m and of the ROOT of v in units of a
 *                scale per 256 consecutive elements, exp_avg_scale and exp_avg_sq_scale
 *                [ceil(n / 256)] float32 (the block's largest magnitude, at least 2^-100,
 *                over 448).  The step itself uses m and v before they are rounded.  Codes are
 *                rounded to nearest where beta1 <= 0.9 and beta2 <= 0.95 (but for an m that fades
 *                to 0 through the last five codes).  With longer windows
 *                a step moves a state by far less than half a code, and nearest rounding would
 *                hold it still: they are rounded up or down by a threshold that depends on the
 *                step's number and the element's index alone, to within one code and right on
 *                average over the steps (so the number has to count on from step to step).  A
 *                positive root rounds to no less than the smallest positive code.  A gradient that is
 *                not finite reaches its own element's parameter and states, and in 8 bits an
 *                infinite one makes all of its block's states NaN (one whose square alone passes
 *                fp32, those in exp_avg_sq).
 *   step         number t of this step, from 1; or step_on_device, one int64 that the kernel
 *                reads (below 1 counts as 1), so that a captured call takes part in every
 *                replay's own step.  The caller counts.
 *   lr           or lr_on_device, one float32.   grad_scale: one float32 on the device, or
 *                NULL for 1 (a clipping factor, or what takes a loss scale back).
 *   beta1, beta2 in [0, 1).   eps: 0, or at least 2^-126 (fp32's least normal value).
 *
 * param, states, scales and master copies of all tensors must be distinct memory; gradients
 * may repeat.  Alignment: each pointer to its element size.  An element's result does not
 * depend on the other tensors of the call.
 */
typedef struct flp_adamw_tensor {
  void* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;      /* state_bits 8 */
  float* exp_avg_sq_scale;   /* state_bits 8 */
  float* master;             /* or NULL */
  int64_t n;
  double weight_decay;
  flp_dtype p_dtype;
  flp_dtype g_dtype;
} flp_adamw_tensor;

flp_status flp_adamw_step(int64_t n_tensors, const flp_adamw_tensor* tensors, int state_bits,
                          int64_t step, const int64_t* step_on_device, double lr,
                          const float* lr_on_device, double beta1, double beta2, double eps,
                          const float* grad_scale, void* stream);

/*
 * Measurement probes (not part of the operator): the achievable dense bf16
 * MFMA rate and the shader clock it runs at, and the achievable streaming-read
 * bandwidth, so that figures can be quoted against measured peaks as well as
 * nominal ones.  Unlike every other call these synchronise `stream` and return
 * their results in host memory.
 *
 *   scratch        device buffer of >= flp_probe_scratch_bytes() bytes, 16-byte
 *                  aligned; contents undefined afterwards.
 *   flp_probe_mfma 2048 workgroups x 4 waves each run `iters` x 128
 *                  v_mfma_f32_16x16x32_bf16 on register operands (random bf16
 *                  values with |x| in [2^-7, 2), or zeros when zero_operands is
 *                  nonzero), timed by HIP events after one untimed launch;
 *                  *out_tflops = flops / time; *out_clock_ghz = median over
 *                  workgroups of shader-clock cycles / real-time ticks during
 *                  the loop x the real-time clock rate.  1 <= iters <= 10^6.
 *   flp_probe_read reads `bytes` (a multiple of 16, 16-byte aligned) of
 *                  `buffer` five times with streaming loads after one untimed
 *                  pass; *out_gbs = bytes read / time.
 */
size_t flp_probe_scratch_bytes(void);
flp_status flp_probe_mfma(int zero_operands, int64_t iters, void* scratch, size_t scratch_bytes,
                          double* out_tflops, double* out_clock_ghz, void* stream);
flp_status flp_probe_read(const void* buffer, size_t bytes, void* scratch, size_t scratch_bytes,
                          double* out_gbs, void* stream);

/*
 * Optional per-kernel timing with HIP events, for benchmarks.  While enabled,
 * every kernel the library enqueues is bracketed by two events recorded on
 * the same stream; flp_profile_read synchronises those events and returns, per
 * kernel kind, the summed duration in milliseconds and the launch count since
 * the previous read (then clears them).  Enabling it adds two event records
 * per kernel and nothing else; results are unaffected.  Process-wide, guarded
 * by a mutex.
 */
typedef enum flp_kernel_kind {
  FLP_K_FORWARD = 0,    /* logits tile + per-tile (max, sum of exp) + target logit */
  FLP_K_MERGE = 1,      /* fixed-tree merge of the tile partials -> lse, logp */
  FLP_K_DLOGITS = 2,    /* logits tile recompute -> dz, dz^T, d_bias partials */
  FLP_K_TRANSPOSE = 3,  /* W -> W^T, hidden chunk -> hidden^T (K-blocked) */
  FLP_K_DHIDDEN = 4,    /* d_hidden = dz W */
  FLP_K_DWEIGHT = 5,    /* d_weight (+)= dz^T hidden */
  FLP_K_DBIAS = 6,      /* ascending fold of the d_bias partials */
  FLP_K_LOGITS_FORWARD = 7,   /* flp_logits_forward */
  FLP_K_LOGITS_BACKWARD = 8,  /* flp_logits_backward */
  FLP_K_ROWS = 9,       /* indexed variants: row selection, gather, scatter */
  FLP_K_EMBEDDING = 10, /* flp_embedding_forward / flp_embedding_backward */
  FLP_K_DROPOUT = 11,   /* flp_dropout */
  FLP_K_LAYER_NORM = 12, /* flp_layer_norm_forward / flp_layer_norm_backward */
  FLP_K_LOSS = 13,      /* flp_cross_entropy_*: row losses, their sum, gradient factors */
  FLP_K_ADAMW = 14,     /* flp_adamw_step */
  FLP_K_RMS_NORM = 15,  /* flp_rms_norm_*, flp_residual_rms_norm_* */
  FLP_K_GATED = 16,     /* flp_gated_linear_*, besides its products in the backward */
  FLP_K_COUNT = 17
} flp_kernel_kind;

void flp_profile_enable(int on);
/* ms[k] and count[k] for k < min(n, FLP_K_COUNT); returns FLP_HIP_ERROR if an
 * event query fails. */
flp_status flp_profile_read(double* ms, int64_t* count, int n);

/*
 * Static text for a status code.  Every unsupported case is reported as an
 * error, never served by another path: the fail-closed gates of PR #555
 * (summary bullets and "Acceptance checks").  Unknown codes give
 * "FLP_UNKNOWN_STATUS".  The string is owned by the library.
 */
const char* flp_status_string(flp_status status);

/*
 * Build provenance: library version, target architecture, git revision and the
 * kernel ids and tile shapes, plus "fallback=none" (this library has no
 * fallback path).  PR #555 (summary bullets, "Acceptance checks") records which
 * backend and kernels produced a result and that no fallback ran; this string
 * is that record for this library.  Static storage owned by the library.
 */
const char* flp_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* FLP_H_ */
