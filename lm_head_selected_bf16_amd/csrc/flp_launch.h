// Kernel argument blocks and launchers (implemented in flp_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>

#include "flp_plan.h"

namespace flp {

// The current device is a gfx950 (cached per device): FLP_OK, else
// FLP_UNSUPPORTED_DEVICE (or FLP_HIP_ERROR when the device cannot be queried).
flp_status check_device();
// Enqueue the forward (logit tiles, then the ascending merge) on `s` with its
// workspace at `workspace`, laid out as fwd_layout(N, D, V).  The arguments
// have been validated.
flp_status enqueue_forward(int64_t N, int64_t D, int64_t V, flp_dtype x_dtype, const void* hidden,
                           const void* weight, const float* bias, const void* targets,
                           flp_dtype t_dtype, const float* temperature, float* out_logp,
                           float* out_lse, void* workspace, hipStream_t s);

// Dynamic LDS above 64 KiB must be opted into per kernel and device.  Each launch
// site keeps a per-device record of having done so; two threads that race on the
// first launch both set the same attribute.
constexpr int kMaxDevices = 64;
template <class K>
hipError_t prepare(K kernel, size_t lds, std::atomic<int> (&ready)[kMaxDevices]) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool tracked = dev >= 0 && dev < kMaxDevices;
  if (tracked && ready[dev].load(std::memory_order_acquire) != 0) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
  if (e == hipSuccess && tracked) ready[dev].store(1, std::memory_order_release);
  return e;
}

struct FwdArgs {
  const void* hidden;
  const void* weight;
  const float* bias;
  const void* targets;
  int t64;
  const float* temperature;
  int64_t N, D, V;
  int64_t t_off;    // vocabulary id of weight row 0 (0 unless a shard)
  float2* part;     // [n_vt][N]
  float* zt;        // [N]
  float* zsum = nullptr;  // cross entropy: [n_vt][N] sums of logits times zunit, or null
  float zunit = 0.f;
  float* logits = nullptr;  // cross entropy: keep the products (256-row tiles), or null
};
struct MergeArgs {
  const float2* part;
  const float* zt;
  const void* targets;
  int t64;
  int64_t N, V, n_vt;
  float* logp;
  float* lse;       // may be null
  float* lse_rest = nullptr;  // [N] the part of lse that its rounding lost, may be null
  // cross entropy (launch_loss_merge, which writes loss and not logp)
  const float* zsum = nullptr;  // [n_vt][N] sums of logits, or null without smoothing
  float zmean = 0.f;            // factor of their sum that gives the row's mean
  float smoothing = 0.f, z_loss = 0.f;
  float* loss = nullptr;        // [N]
};
struct DzArgs {
  const void* hidden;   // chunk start
  const void* weight;
  const float* bias;
  const void* targets;  // chunk start
  int t64;
  const float* temperature;  // chunk start or null
  const float* grad_out;     // chunk start
  const float* lse;          // chunk start
  int64_t rows, D, V, ldz, ldt;  // ldz: vocabulary padded; ldt: rows allocated in the chunk
  void* dz;                  // [ldt rows][ldz] K-blocked, or null when d_hidden is not needed
  void* dzT;                 // [ldz rows][ldt] K-blocked, or null when d_weight is not needed
  float* dbias_part;         // [rows_alloc / kDzRowTile][ldz] or null
  // cross entropy (null otherwise; grad_out then holds the softmax's factor): chunk start
  const float* onehot = nullptr;   // the target entry's added term
  const float* uniform = nullptr;  // every entry's added term
  const float* lse_rest = nullptr;
  float* d_bias = nullptr;         // set: the batch is one row tile, whose sums are d_bias itself
  const float* bias_scale = nullptr;  // what they are multiplied by, or null
  float* logits = nullptr;         // products kept by the forward, or null to recompute
};
struct LogitsArgs {
  const void* logits;        // [N][V]
  const void* targets;
  int t64;
  int64_t N, V;
  const float* grad_out;     // backward only
  const float* lse;          // backward only
  float* logp;               // forward only
  float* lse_out;            // forward only, may be null
  void* d_logits;            // backward only
  const uint8_t* mask;       // [N] selected rows (indexed variants) or null for all rows
};
struct GatherArgs {
  const int32_t* sel;        // [cap] selected row ids, -1 for padding entries
  const void* hidden;        // [N][D]
  int64_t row_bytes;         // D * element size (a multiple of 16)
  const void* targets;
  int t64;
  const float* temperature;  // may be null
  const float* grad_out;     // may be null
  const float* lse;          // may be null
  void* h_c;                 // [cap][D]
  int64_t* t_c;              // [cap]
  float* temp_c;             // [cap] or null
  float* g_c;                // [cap] or null
  float* lse_c;              // [cap] or null
};
struct GemmArgs {
  const void* a;   // M-side operand
  const void* b;   // N-side operand
  int64_t lda_b, ldb_b;  // row strides in bytes (128 in the K-blocked layout)
  int64_t a_ks, b_ks;    // bytes from one 128-byte K stage to the next (rows x 128)
  int64_t M, N, K;
  void* out;             // output (x dtype or fp32)
  int64_t ldo;           // elements
  float* acc;            // fp32 accumulator [M][N] (dW) or null
  int load_acc;          // continue from acc
  int store_acc;         // store fp32 to acc (else store to out in x dtype)
  const float* scale = nullptr;  // fp16: factor of the rounded result, or null for 1
  int64_t k_slab = 0;    // d_hidden: > 0 sums K in slabs of this length, held in acc [slabs][M][N]
};

hipError_t launch_forward(flp_dtype x, const FwdArgs& a, hipStream_t s);
hipError_t launch_loss_forward(flp_dtype x, const FwdArgs& a, hipStream_t s);
hipError_t launch_merge(const MergeArgs& a, hipStream_t s);
hipError_t launch_loss_merge(const MergeArgs& a, hipStream_t s);
hipError_t launch_fill(float* dst, int64_t n, float value, hipStream_t s);
hipError_t launch_logits_forward(flp_dtype x, const LogitsArgs& a, hipStream_t s);
hipError_t launch_logits_backward(flp_dtype x, const LogitsArgs& a, hipStream_t s);
hipError_t launch_dz(flp_dtype x, const DzArgs& a, hipStream_t s);
hipError_t launch_dx(flp_dtype x, const GemmArgs& a, hipStream_t s);
hipError_t launch_dw(flp_dtype x, const GemmArgs& a, hipStream_t s);
// dst = src^T for src [rows][cols] (row stride ld_src elements), written K-blocked
// with cols rows and K = rows_pad; K entries in [rows, rows_pad) are zero-filled.
hipError_t launch_transpose(flp_dtype x, const void* src, int64_t rows, int64_t rows_pad, int64_t cols,
                            int64_t ld_src, void* dst, hipStream_t s);
// The same for hidden rows (row stride cols): rows whose target is outside [0, V) read as
// zeros.  In the same launch, unless null: weight [V][cols], padded to weight_pad.
hipError_t launch_transpose_live(flp_dtype x, const void* src, int64_t rows, int64_t rows_pad,
                                 int64_t cols, const void* targets, bool t64, int64_t V, void* dst,
                                 const void* weight, int64_t weight_pad, void* weight_dst,
                                 hipStream_t s);
hipError_t launch_dbias_fold(const float* part, int64_t n_parts, int64_t ldz, int64_t V,
                             float* d_bias, int init, const float* scale, hipStream_t s);
const char* kernel_ids();

// Row selection for the indexed variants (flp_rows.hip).  launch_zero clears
// bytes / 4 words.  launch_select builds the mask; with pos != null it also
// compacts it into pos / sel.
hipError_t launch_zero(void* dst, size_t bytes, hipStream_t s);
hipError_t launch_select(const void* rows, bool r64, int64_t n_rows, int64_t N, uint8_t* mask,
                         int32_t* pos, int32_t* sel, int64_t cap, hipStream_t s);
hipError_t launch_gather(const GatherArgs& a, int64_t cap, hipStream_t s);
hipError_t launch_scatter_rows(const int32_t* pos, int64_t N, const float* logp_c,
                               const float* lse_c, float* logp, float* lse, hipStream_t s);
hipError_t launch_scatter_hidden(const int32_t* pos, int64_t N, const void* dh_c, size_t row_bytes,
                                 void* dh, hipStream_t s);

// Untied embedding lookup and its sorted-segment grad_weight (flp_embed.hip).
struct EmbedBwdArgs {
  flp_dtype x;               // dtype of grad (and of the embedding)
  flp_dtype dw;              // x or FLP_F32
  const void* grad;          // [N][D]
  const void* ids;           // [N]
  bool i64;
  int64_t N, D, V;
  uint32_t* keys[2];         // [N] radix-sort ping-pong buffers
  int32_t* vals[2];          // [N]
  int32_t* hist;             // [2^kEmbDigitBits][ceil(N / kEmbSortBlock) rounded up to 4]
  float* head;               // [ceil(N / kEmbSegGroup)][D] fp32 pieces of segments that span groups
  float* tail;               // same shape
  void* d_weight;            // [V][D] dw
  float scale;               // factor of the summed gradient rows
};
int embed_sort_passes(int64_t V);
hipError_t launch_embedding_forward(flp_dtype x, const void* weight, const void* ids, bool i64,
                                    int64_t N, int64_t D, int64_t V, float scale, void* out,
                                    hipStream_t s);
hipError_t launch_embedding_backward(const EmbedBwdArgs& a, hipStream_t s);

// Layer norm (flp_norm.hip).
struct NormFwdArgs {
  int64_t N, D;
  const void* x;             // [N][D]
  const void* weight;        // [D] or null
  const void* bias;          // [D] or null
  bool wide;                 // the parameters are fp32 (set by the launcher)
  float eps;
  void* out;                 // [N][D]
  float* mean;               // [N] or null
  float* rstd;               // [N] or null
};
struct NormBwdArgs {
  int64_t N, D;
  const void* grad;          // [N][D]
  const void* x;             // [N][D]
  const void* weight;        // [D] or null
  bool wide;                 // the parameters are fp32 (set by the launcher)
  const float* mean;         // [N]
  const float* rstd;         // [N]
  void* d_x;                 // [N][D] or null
  void* d_weight;            // [D] or null
  void* d_bias;              // [D] or null
  int64_t slabs, slab_rows;  // rows are summed in slabs of slab_rows
  float* part;               // [slabs][2][D] partial d_weight and d_bias, or null for neither
};
hipError_t launch_layer_norm_forward(flp_dtype x, flp_dtype w, const NormFwdArgs& a,
                                     hipStream_t s);
hipError_t launch_layer_norm_backward(flp_dtype x, flp_dtype w, const NormBwdArgs& a,
                                      hipStream_t s);

// Dropout (flp_dropout.hip): elements whose 16 random bits are below `drop` become 0.
hipError_t launch_dropout(flp_dtype x_dtype, int64_t n, const void* x, const uint64_t* rng,
                          uint32_t drop, float scale, void* out, hipStream_t s);

// Row kernels of the cross entropy (flp_loss.hip).
struct LossSumArgs {         // forward: the sum or mean of the rows' losses
  int64_t N, V;
  const void* targets;
  int t64;
  const float* rows;         // [N] per-row losses
  int mean;
  float* loss;               // [1]
};
struct LossGradArgs {        // backward: the per-row factors of the logit gradient
  int64_t N, V;
  const void* targets;
  int t64;
  const float* grad_out;     // [N], or [1] for a reduced loss, or null for 1
  const float* inv;          // [1] 1 / rows of the mean, or null to count them here
  const float* lse;          // [N]
  float smoothing, z_loss;
  int reduction;             // flp_reduction
  int rescale;               // bring the largest factor to [2^10, 2^11) (fp16)
  float* softmax;            // [N] factor of the softmax
  float* onehot;             // [N] term of the target entry
  float* uniform;            // [N] term of every entry
  float* unscale;            // [1] factor that takes the scaling back
  const float* lse_rest;     // [N]
  int64_t k_slab;            // vocabulary slab of d_hidden, 0 for none
  float* slab_sums;          // [slabs][N][D]
};
hipError_t launch_loss_sum(const LossSumArgs& a, hipStream_t s);
hipError_t launch_loss_grad(const LossGradArgs& a, hipStream_t s);
// *inv = 1 / the number of targets in [0, V) (1 if there are none).
hipError_t launch_loss_count(int64_t N, int64_t V, const void* targets, bool t64, float* inv,
                             hipStream_t s);
// x *= *factor in place (n elements); nothing is touched when the factor is 1.
hipError_t launch_scale(flp_dtype x_dtype, int64_t n, void* x, const float* factor, hipStream_t s);

// Measurement probes (flp_probe.hip); they synchronise the stream.
size_t probe_scratch_bytes();
hipError_t probe_mfma(int zero, int64_t iters, void* scratch, hipStream_t s, double* tflops,
                      double* clock_ghz);
hipError_t probe_read(const void* buf, size_t bytes, void* scratch, hipStream_t s, double* gbs);

// Event brackets around each launch while profiling is enabled (flp_api.cpp).
struct ProfScope {
  ProfScope(int kind, hipStream_t s);
  ~ProfScope();
  int kind;
  hipStream_t stream;
  hipEvent_t a = nullptr;
};

}  // namespace flp
