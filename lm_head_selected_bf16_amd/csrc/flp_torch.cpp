// Autograd nodes of the operators around a model's body (embedding lookup, dropout, layer
// norm, linear cross entropy), over the C ABI.
//
// They allocate outputs and workspaces with torch and pass addresses on, as torch_ops.py does
// for the other operators; the checks of a call's arguments are made there, before it comes
// here.  Autograd runs a backward on a thread of its own, which has to take over the Python
// interpreter for a node written in Python and then runs it from cold caches: a layer norm of
// 37 x 1003, forward and backward, took 118 us on the host that way and takes 74 here.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/extension.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <optional>
#include <stdexcept>
#include <string>
#include <vector>

#include "flp.h"

namespace {

using torch::autograd::AutogradContext;
using torch::autograd::Function;
using torch::autograd::variable_list;
using OptTensor = std::optional<at::Tensor>;

// The entry points of the loaded library.
struct Api {
  decltype(&::flp_embedding_scaled_forward) embedding_forward;
  decltype(&::flp_embedding_scaled_backward) embedding_backward;
  decltype(&::flp_embedding_backward_workspace_bytes) embedding_backward_bytes;
  decltype(&::flp_dropout) dropout;
  decltype(&::flp_layer_norm_forward) norm_forward;
  decltype(&::flp_layer_norm_backward) norm_backward;
  decltype(&::flp_layer_norm_backward_workspace_bytes) norm_backward_bytes;
  decltype(&::flp_cross_entropy_forward) loss_forward;
  decltype(&::flp_cross_entropy_forward_workspace_bytes) loss_forward_bytes;
  decltype(&::flp_cross_entropy_backward) loss_backward;
  decltype(&::flp_cross_entropy_backward_workspace_bytes) loss_backward_bytes;
  decltype(&::flp_adamw_step) adamw_step;
  decltype(&::flp_gated_linear_saved_bytes) gated_saved_bytes;
  decltype(&::flp_gated_linear_forward) gated_forward;
  decltype(&::flp_gated_linear_backward) gated_backward;
  decltype(&::flp_gated_linear_backward_workspace_bytes) gated_backward_bytes;
  decltype(&::flp_residual_rms_norm_forward) rms_forward;
  decltype(&::flp_residual_rms_norm_backward) rms_backward;
  decltype(&::flp_residual_rms_norm_backward_workspace_bytes) rms_backward_bytes;
};
Api api;

void bind(const std::map<std::string, uintptr_t>& at) {
  auto take = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(at.at(name));
  };
  take(api.embedding_forward, "flp_embedding_scaled_forward");
  take(api.embedding_backward, "flp_embedding_scaled_backward");
  take(api.embedding_backward_bytes, "flp_embedding_backward_workspace_bytes");
  take(api.dropout, "flp_dropout");
  take(api.norm_forward, "flp_layer_norm_forward");
  take(api.norm_backward, "flp_layer_norm_backward");
  take(api.norm_backward_bytes, "flp_layer_norm_backward_workspace_bytes");
  take(api.loss_forward, "flp_cross_entropy_forward");
  take(api.loss_forward_bytes, "flp_cross_entropy_forward_workspace_bytes");
  take(api.loss_backward, "flp_cross_entropy_backward");
  take(api.loss_backward_bytes, "flp_cross_entropy_backward_workspace_bytes");
  take(api.adamw_step, "flp_adamw_step");
  take(api.gated_saved_bytes, "flp_gated_linear_saved_bytes");
  take(api.gated_forward, "flp_gated_linear_forward");
  take(api.gated_backward, "flp_gated_linear_backward");
  take(api.gated_backward_bytes, "flp_gated_linear_backward_workspace_bytes");
  take(api.rms_forward, "flp_residual_rms_norm_forward");
  take(api.rms_backward, "flp_residual_rms_norm_backward");
  take(api.rms_backward_bytes, "flp_residual_rms_norm_backward_workspace_bytes");
}

// A non-OK status: FlpError in Python, as a Python exception from here on.  A backward runs in
// autograd's engine, which hands those on as they are and any other but torch's own as
// RuntimeError.
void check(const char* fn, flp_status st) {
  if (st == FLP_OK) return;
  py::gil_scoped_acquire interpreter;
  py::object cls = py::module_::import("lm_head_selected_bf16_amd._abi").attr("FlpError");
  PyErr_SetObject(cls.ptr(), cls(fn, int(st)).ptr());
  python_error e;
  e.persist();
  throw e;
}

flp_dtype code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return FLP_BF16;
    case at::kHalf: return FLP_F16;
    case at::kFloat: return FLP_F32;
    case at::kLong: return FLP_I64;
    case at::kInt: return FLP_I32;
    default: TORCH_CHECK_TYPE(false, "unsupported dtype");
  }
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* fptr(const at::Tensor& t) { return static_cast<float*>(ptr(t)); }

at::Tensor bytes(size_t n, const at::Tensor& like) {
  return at::empty({int64_t(n > 16 ? n : 16)}, like.options().dtype(at::kByte));
}

// The same, halved as often as needed and at least `least`, as the device has room for.
at::Tensor bytes(size_t n, size_t least, const at::Tensor& like) {
  while (n > least) {
    try {
      return bytes(n, like);
    } catch (const c10::OutOfMemoryError&) {
      n = n / 2 > least ? n / 2 : least;
    }
  }
  return bytes(n, like);
}

// A leaf's data may have been exchanged between the forward and the backward.
void same(bool ok) { TORCH_CHECK_VALUE(ok, "an input of the forward has changed since then"); }
bool dense(const at::Tensor& t) { return t.is_cuda() && t.is_contiguous(); }

// The upstream gradient as the library takes it.  contiguous() returns a dense view at any
// offset of its storage (what the backward of a concatenation hands on) as it is.
at::Tensor aligned16(const at::Tensor& t) {
  at::Tensor c = t.contiguous();
  return reinterpret_cast<uintptr_t>(ptr(c)) % 16 == 0 ? c : c.clone();
}

// The gradients cannot be differentiated again: where a graph of the backward is asked for, the
// backward of what is derived from one that depends on something to be differentiated raises.
// (Without the node such a gradient would pass for a constant.)
struct FirstOrder : Function<FirstOrder> {
  static at::Tensor forward(AutogradContext*, const at::Tensor& t) { return at::alias(t); }
  static variable_list backward(AutogradContext*, variable_list) {
    throw std::runtime_error(
        "trying to differentiate twice a function that is marked with once_differentiable: what "
        "its backward computes does not require grad");
  }
};

at::Tensor first_order(const at::Tensor& t) {
  return FirstOrder::apply(t.detach().requires_grad_(true));
}

// t, which depends on `from`.
template <class... Ts>
at::Tensor first_order(const at::Tensor& t, const Ts&... from) {
  const bool graph = at::GradMode::is_enabled() && t.defined() &&
                     ((from.defined() && from.requires_grad()) || ...);
  return graph ? first_order(t) : t;
}

// Every backward runs on the stream of its forward, which autograd makes current for it;
// `stream` is that stream's handle.

struct EmbeddingNode : Function<EmbeddingNode> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& weight, const at::Tensor& ids,
                            double scale, int64_t stream) {
    const int64_t V = weight.size(0), D = weight.size(1);
    auto shape = ids.sizes().vec();
    shape.push_back(D);
    at::Tensor out = at::empty(shape, weight.options());
    check("flp_embedding_scaled_forward",
          api.embedding_forward(ids.numel(), D, V, code(weight), ptr(weight), ptr(ids), code(ids),
                                scale, ptr(out), reinterpret_cast<void*>(stream)));
    ctx->save_for_backward({ids});
    ctx->saved_data["V"] = V;
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["stream"] = stream;
    ctx->saved_data["N"] = ids.numel();
    return out;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const at::Tensor ids = ctx->get_saved_variables()[0];
    const int64_t N = ctx->saved_data["N"].toInt(), V = ctx->saved_data["V"].toInt();
    same(dense(ids) && ids.numel() == N && ids.device() == grads[0].device());
    const at::Tensor g = aligned16(grads[0]);
    const int64_t D = g.size(-1);
    at::Tensor dw = at::empty({V, D}, g.options());
    const size_t size = api.embedding_backward_bytes(N, D, V);
    const at::Tensor ws = bytes(size, g);
    check("flp_embedding_scaled_backward",
          api.embedding_backward(N, D, V, code(g), ptr(g), ptr(ids), code(ids),
                                 ctx->saved_data["scale"].toDouble(), ptr(dw), code(g), ptr(ws),
                                 size_t(ws.numel()),
                                 reinterpret_cast<void*>(ctx->saved_data["stream"].toInt())));
    return {first_order(dw, grads[0]), at::Tensor(), at::Tensor(), at::Tensor()};
  }
};

struct DropoutNode : Function<DropoutNode> {
  static at::Tensor run(const at::Tensor& x, double p, const at::Tensor& rng, int64_t stream) {
    at::Tensor out = at::empty_like(x);
    check("flp_dropout", api.dropout(x.numel(), code(x), ptr(x), p,
                                     static_cast<const int64_t*>(ptr(rng)), ptr(out),
                                     reinterpret_cast<void*>(stream)));
    return out;
  }
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, double p,
                            const at::Tensor& rng, int64_t stream) {
    ctx->save_for_backward({rng});
    ctx->saved_data["p"] = p;
    ctx->saved_data["stream"] = stream;
    return run(x, p, rng, stream);
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const at::Tensor rng = ctx->get_saved_variables()[0];
    same(dense(rng) && rng.scalar_type() == at::kLong && rng.numel() == 2 &&
         rng.device() == grads[0].device());
    const at::Tensor dx = run(grads[0].contiguous(), ctx->saved_data["p"].toDouble(), rng,
                              ctx->saved_data["stream"].toInt());
    return {first_order(dx, grads[0]), at::Tensor(), at::Tensor(), at::Tensor()};
  }
};

struct LayerNormNode : Function<LayerNormNode> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, const OptTensor& weight,
                            const OptTensor& bias, double eps, int64_t stream) {
    const int64_t D = x.size(-1), N = x.numel() / D;
    const at::Tensor w = weight.value_or(at::Tensor()), b = bias.value_or(at::Tensor());
    const at::Tensor& typed = w.defined() ? w : b.defined() ? b : x;
    at::Tensor out = at::empty_like(x);
    const at::Tensor stats = at::empty({2, N}, x.options().dtype(at::kFloat));
    check("flp_layer_norm_forward",
          api.norm_forward(N, D, code(x), ptr(x), code(typed), ptr(w), ptr(b), eps, ptr(out),
                           fptr(stats), fptr(stats) + N, reinterpret_cast<void*>(stream)));
    ctx->save_for_backward({x, w, stats});
    ctx->saved_data["type"] = int64_t(typed.scalar_type());
    ctx->saved_data["bias"] = b.defined();
    ctx->saved_data["stream"] = stream;
    return out;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const at::Tensor &x = saved[0], &w = saved[1], &stats = saved[2];
    const auto type = at::ScalarType(ctx->saved_data["type"].toInt());
    const bool has_bias = ctx->saved_data["bias"].toBool();
    same(dense(x) && x.sizes() == grads[0].sizes() && x.scalar_type() == grads[0].scalar_type() &&
         x.device() == grads[0].device());
    const int64_t D = x.size(-1), N = x.numel() / D;
    same(!w.defined() || (dense(w) && w.dim() == 1 && w.size(0) == D && w.scalar_type() == type &&
                          w.device() == x.device()));
    const at::Tensor g = grads[0].contiguous();
    // the inputs that are tensors have edges, in order
    const bool need_x = ctx->needs_input_grad(0);
    const bool need_w = w.defined() && ctx->needs_input_grad(1);
    const bool need_b = has_bias && ctx->needs_input_grad(w.defined() ? 2 : 1);
    const auto opts = x.options().dtype(type);
    at::Tensor dx, dw, db, ws;
    size_t size = 0;
    if (need_x) dx = at::empty_like(x);
    if (need_w) dw = at::empty({D}, opts);
    if (need_b) db = at::empty({D}, opts);
    if (need_w || need_b) {
      ws = bytes(api.norm_backward_bytes(N, D), x);
      size = size_t(ws.numel());
    }
    const flp_dtype wd = type == at::kBFloat16 ? FLP_BF16 : type == at::kHalf ? FLP_F16 : FLP_F32;
    check("flp_layer_norm_backward",
          api.norm_backward(N, D, code(x), ptr(g), ptr(x), wd, ptr(w), fptr(stats),
                            fptr(stats) + N, ptr(dx), ptr(dw), ptr(db), ptr(ws), size,
                            reinterpret_cast<void*>(ctx->saved_data["stream"].toInt())));
    return {first_order(dx, grads[0], x, w), first_order(dw, grads[0], x),
            first_order(db, grads[0]), at::Tensor(), at::Tensor()};
  }
};

struct CrossEntropyNode : Function<CrossEntropyNode> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& hidden,
                            const at::Tensor& weight, const at::Tensor& targets,
                            const OptTensor& bias, double smoothing, double z_loss,
                            int64_t reduction, int64_t most_workspace, int64_t stream) {
    const int64_t N = targets.numel(), V = weight.size(0), D = weight.size(1);
    const at::Tensor b = bias.value_or(at::Tensor());
    const auto f32 = hidden.options().dtype(at::kFloat);
    at::Tensor loss = reduction == FLP_REDUCE_NONE ? at::empty(targets.sizes(), f32)
                                                   : at::empty({}, f32);
    const at::Tensor stats = at::empty({2, N}, f32);
    const at::Tensor ws = bytes(api.loss_forward_bytes(N, D, V), hidden);
    check("flp_cross_entropy_forward",
          api.loss_forward(N, D, V, code(hidden), ptr(hidden), ptr(weight), fptr(b), ptr(targets),
                           code(targets), smoothing, z_loss, flp_reduction(reduction), fptr(loss),
                           fptr(stats), ptr(ws), size_t(ws.numel()),
                           reinterpret_cast<void*>(stream)));
    ctx->save_for_backward({hidden, weight, targets, b, stats});
    ctx->saved_data["smoothing"] = smoothing;
    ctx->saved_data["z_loss"] = z_loss;
    ctx->saved_data["reduction"] = reduction;
    ctx->saved_data["most"] = most_workspace;
    ctx->saved_data["stream"] = stream;
    ctx->saved_data["V"] = V;
    return loss;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const at::Tensor &hidden = saved[0], &weight = saved[1], &targets = saved[2], &b = saved[3],
                     &stats = saved[4];
    const int64_t V = ctx->saved_data["V"].toInt(), N = stats.size(1);
    same(dense(hidden) && dense(weight) && dense(targets) && targets.numel() == N &&
         weight.dim() == 2 && weight.size(0) == V && hidden.dim() >= 1 &&
         hidden.size(-1) == weight.size(1) && hidden.numel() == N * weight.size(1) &&
         hidden.scalar_type() == weight.scalar_type() && hidden.device() == weight.device() &&
         hidden.device() == targets.device() && hidden.device() == grads[0].device() &&
         (!b.defined() || (dense(b) && b.scalar_type() == at::kFloat && b.numel() == V &&
                           b.device() == hidden.device())));
    const int64_t D = weight.size(1);
    const at::Tensor g = grads[0].contiguous();
    at::Tensor dh, dw, db;
    if (ctx->needs_input_grad(0)) dh = at::empty_like(hidden);
    if (ctx->needs_input_grad(1)) dw = at::empty_like(weight);
    if (b.defined() && ctx->needs_input_grad(3)) db = at::empty_like(b);
    // a smaller workspace runs more row chunks, with the same bits
    const size_t whole = api.loss_backward_bytes(N, D, V, code(hidden), N > 1 ? N : 1);
    const size_t least = api.loss_backward_bytes(N, D, V, code(hidden), 0);
    const size_t most = std::max(least, size_t(ctx->saved_data["most"].toInt()));
    const at::Tensor ws = bytes(std::min(whole, most), least, hidden);
    check("flp_cross_entropy_backward",
          api.loss_backward(N, D, V, code(hidden), fptr(g), fptr(stats), ptr(hidden), ptr(weight),
                            fptr(b), ptr(targets), code(targets),
                            ctx->saved_data["smoothing"].toDouble(),
                            ctx->saved_data["z_loss"].toDouble(),
                            flp_reduction(ctx->saved_data["reduction"].toInt()), ptr(dh), ptr(dw),
                            fptr(db), ptr(ws), size_t(ws.numel()),
                            reinterpret_cast<void*>(ctx->saved_data["stream"].toInt())));
    variable_list out(9);
    out[0] = first_order(dh, grads[0], hidden, weight, b);
    out[1] = first_order(dw, grads[0], hidden, weight, b);
    out[3] = first_order(db, grads[0], hidden, weight, b);
    return out;
  }
};

struct GatedLinearNode : Function<GatedLinearNode> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, const at::Tensor& w_gate,
                            const at::Tensor& w_up, int64_t act, int64_t stream) {
    const int64_t F = w_gate.size(0), D = w_gate.size(1), N = x.numel() / D;
    auto shape = x.sizes().vec();
    shape.back() = F;
    at::Tensor out = at::empty(shape, x.options());
    const at::Tensor saved = bytes(api.gated_saved_bytes(N, F, code(x)), x);
    check("flp_gated_linear_forward",
          api.gated_forward(N, D, F, code(x), ptr(x), ptr(w_gate), ptr(w_up), flp_activation(act),
                            ptr(out), ptr(saved), reinterpret_cast<void*>(stream)));
    ctx->save_for_backward({x, w_gate, w_up, saved});
    ctx->saved_data["act"] = act;
    ctx->saved_data["stream"] = stream;
    ctx->saved_data["F"] = F;
    return out;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const at::Tensor &x = saved[0], &wg = saved[1], &wu = saved[2];
    const int64_t F = ctx->saved_data["F"].toInt();
    const at::Tensor g = grads[0].contiguous();
    const int64_t N = g.numel() / F;
    same(dense(x) && dense(wg) && dense(wu) && wg.dim() == 2 && wg.size(0) == F &&
         wu.sizes() == wg.sizes() && x.dim() >= 1 && x.size(-1) == wg.size(1) &&
         x.numel() == N * wg.size(1) && x.scalar_type() == g.scalar_type() &&
         wg.scalar_type() == g.scalar_type() && wu.scalar_type() == g.scalar_type() &&
         x.device() == g.device() && wg.device() == g.device() && wu.device() == g.device());
    const int64_t D = wg.size(1);
    at::Tensor dx, dwg, dwu;
    if (ctx->needs_input_grad(0)) dx = at::empty_like(x);
    if (ctx->needs_input_grad(1)) dwg = at::empty_like(wg);
    if (ctx->needs_input_grad(2)) dwu = at::empty_like(wu);
    const at::Tensor ws = bytes(api.gated_backward_bytes(N, D, F, code(x), dx.defined(),
                                                         dwg.defined() || dwu.defined()),
                                x);
    check("flp_gated_linear_backward",
          api.gated_backward(N, D, F, code(x), ptr(g), ptr(saved[3]), ptr(x), ptr(wg), ptr(wu),
                             flp_activation(ctx->saved_data["act"].toInt()), ptr(dx), ptr(dwg),
                             ptr(dwu), ptr(ws), size_t(ws.numel()),
                             reinterpret_cast<void*>(ctx->saved_data["stream"].toInt())));
    return {first_order(dx, grads[0], x, wg, wu), first_order(dwg, grads[0], x, wg, wu),
            first_order(dwu, grads[0], x, wg, wu), at::Tensor(), at::Tensor()};
  }
};

// The norms around a block: {r, n}, or {n} without y.
struct RmsNormNode : Function<RmsNormNode> {
  static variable_list forward(AutogradContext* ctx, const at::Tensor& x, const OptTensor& y,
                               const OptTensor& weight, const OptTensor& post_weight,
                               const OptTensor& gate, bool post, double scale, double eps,
                               int64_t stream) {
    const int64_t D = x.size(-1), N = x.numel() / D;
    const at::Tensor b = y.value_or(at::Tensor()), w = weight.value_or(at::Tensor()),
                     pw = post_weight.value_or(at::Tensor()), g = gate.value_or(at::Tensor());
    const at::Tensor& typed = w.defined() ? w : pw.defined() ? pw : g.defined() ? g : x;
    const int64_t gates = g.defined() ? g.numel() / D : 0;
    at::Tensor r, n = at::empty_like(x);
    if (b.defined()) r = at::empty_like(x);
    const at::Tensor stats = at::empty({post ? 2 : 1, N}, x.options().dtype(at::kFloat));
    check("flp_residual_rms_norm_forward",
          api.rms_forward(N, D, code(x), ptr(x), ptr(b), code(typed), ptr(w), post, ptr(pw), gates,
                          ptr(g), scale, eps, ptr(r), ptr(n), fptr(stats),
                          post ? fptr(stats) + N : nullptr, reinterpret_cast<void*>(stream)));
    ctx->save_for_backward({x, b, w, pw, g, stats});
    ctx->saved_data["type"] = int64_t(typed.scalar_type());
    ctx->saved_data["post"] = post;
    ctx->saved_data["gates"] = gates;
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["stream"] = stream;
    ctx->set_materialize_grads(false);
    if (b.defined()) return {r, n};
    return {n};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const at::Tensor &x = saved[0], &y = saved[1], &w = saved[2], &pw = saved[3], &gate = saved[4],
                     &stats = saved[5];
    const auto type = at::ScalarType(ctx->saved_data["type"].toInt());
    const bool post = ctx->saved_data["post"].toBool();
    const int64_t gates = ctx->saved_data["gates"].toInt(), N = stats.size(1);
    variable_list out(9);
    const at::Tensor gr = y.defined() ? grads[0] : at::Tensor();
    const at::Tensor gn = y.defined() ? grads[1] : grads[0];
    if (!gr.defined() && !gn.defined()) return out;
    const at::Tensor& up = gn.defined() ? gn : gr;
    auto rows = [&](const at::Tensor& t) {
      return !t.defined() || (dense(t) && t.sizes() == up.sizes() && t.device() == up.device() &&
                              t.scalar_type() == up.scalar_type());
    };
    same(rows(x) && rows(y) && x.dim() >= 1 && x.numel() == N * x.size(-1));
    const int64_t D = x.size(-1);
    auto param = [&](const at::Tensor& t, int64_t n) {
      return !t.defined() || (dense(t) && t.numel() == n * D && t.scalar_type() == type &&
                              t.device() == x.device());
    };
    same(param(w, 1) && param(pw, 1) && param(gate, gates));
    const at::Tensor cr = gr.defined() ? gr.contiguous() : gr;
    const at::Tensor cn = gn.defined() ? gn.contiguous() : gn;
    // the inputs that are tensors have edges, in order
    size_t edge = 0;
    auto needs = [&](const at::Tensor& t) {
      return t.defined() && ctx->needs_input_grad(edge++);
    };
    at::Tensor dx, dy, dw, dpw, dg, ws;
    if (needs(x)) dx = at::empty_like(x);
    if (needs(y)) dy = at::empty_like(y);
    if (needs(w)) dw = at::empty_like(w);
    if (needs(pw)) dpw = at::empty_like(pw);
    if (needs(gate)) dg = at::empty_like(gate);
    size_t size = 0;
    if (dw.defined() || dpw.defined() || dg.defined()) {
      ws = bytes(api.rms_backward_bytes(N, D, gates), x);
      size = size_t(ws.numel());
    }
    const flp_dtype wd = type == at::kBFloat16 ? FLP_BF16 : type == at::kHalf ? FLP_F16 : FLP_F32;
    check("flp_residual_rms_norm_backward",
          api.rms_backward(N, D, code(x), ptr(cr), ptr(cn), ptr(x), ptr(y), wd, ptr(w), post,
                           ptr(pw), gates, ptr(gate), ctx->saved_data["scale"].toDouble(),
                           fptr(stats), post ? fptr(stats) + N : nullptr, ptr(dx), ptr(dy),
                           ptr(dw), ptr(dpw), ptr(dg), ptr(ws), size,
                           reinterpret_cast<void*>(ctx->saved_data["stream"].toInt())));
    auto once = [&](const at::Tensor& t) {
      return first_order(t, gr, gn, x, y, w, pw, gate);
    };
    out[0] = once(dx);
    out[1] = once(dy);
    out[2] = once(dw);
    out[3] = once(dpw);
    out[4] = once(dg);
    return out;
  }
};

// ---- AdamW ----
//
// No autograd node, but lists of tensors: with its arguments checked in Python, a step over 300
// tensors would take several ms on the host.

// A list or tuple of tensors or None, as Python holds it (a copy into a vector costs 60 ns for each).
class List {
 public:
  explicit List(py::handle from, const char* what)
      : held_(py::reinterpret_steal<py::object>(PySequence_Fast(from.ptr(), what))) {
    if (!held_) throw py::error_already_set();
  }
  size_t size() const { return size_t(PySequence_Fast_GET_SIZE(held_.ptr())); }
  const at::Tensor* at(size_t k) const {
    PyObject* const o = PySequence_Fast_GET_ITEM(held_.ptr(), Py_ssize_t(k));
    if (o == Py_None) return nullptr;
    TORCH_CHECK_TYPE(THPVariable_Check(o), "expected a tensor, got ", Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
  }
  const at::Tensor& need(size_t k) const {
    const at::Tensor* const t = at(k);
    TORCH_CHECK_TYPE(t != nullptr, "expected a tensor, got None");
    return *t;
  }

 private:
  py::object held_;
};

// decay: a number, or one for each parameter.
void adamw_step(py::handle params_, py::handle grads_, py::handle exp_avg_, py::handle exp_avg_sq_,
                py::handle exp_avg_scale_, py::handle exp_avg_sq_scale_, py::handle master_,
                py::handle decay_, int64_t step, const OptTensor& step_on_device, double lr,
                const OptTensor& lr_on_device, double beta1, double beta2, double eps,
                const OptTensor& grad_scale, int64_t stream) {
  auto list = [](py::handle h) {
    return h.is_none() ? std::optional<List>() : std::optional<List>(List(h, "expected a list of tensors"));
  };
  const List params(params_, "expected a list of parameters"), grads(grads_, "expected a list of gradients"),
      exp_avg(exp_avg_, "expected a list of states"), exp_avg_sq(exp_avg_sq_, "expected a list of states");
  const auto exp_avg_scale = list(exp_avg_scale_), exp_avg_sq_scale = list(exp_avg_sq_scale_),
             master = list(master_);
  const bool one_decay = PyFloat_Check(decay_.ptr()) || PyLong_Check(decay_.ptr());
  std::vector<double> decay;
  if (one_decay)
    decay.push_back(decay_.cast<double>());
  else
    decay = decay_.cast<std::vector<double>>();
  const size_t count = params.size();
  const bool eight = exp_avg_scale.has_value();
  TORCH_CHECK_VALUE(grads.size() == count && exp_avg.size() == count &&
                        exp_avg_sq.size() == count && (one_decay || decay.size() == count) &&
                        (!master || master->size() == count),
                    "there must be as many gradients, states, master copies and weight decays as "
                    "parameters");
  TORCH_CHECK_VALUE(eight == exp_avg_sq_scale.has_value() &&
                        (!eight || (exp_avg_scale->size() == count &&
                                    exp_avg_sq_scale->size() == count)),
                    "states in 8 bits need a scale tensor for each parameter's exp_avg and "
                    "exp_avg_sq");
  if (count == 0) return;
  const at::Device device = params.need(0).device();
  auto here = [&](const at::Tensor& t, const char* what) {
    TORCH_CHECK_VALUE(t.layout() == at::kStrided && t.is_cuda() && t.is_contiguous() &&
                          t.device() == device,
                      what, " must be contiguous GPU tensors on one device");
  };
  auto scalar = [&](const OptTensor& t, at::ScalarType type, const char* what) -> void* {
    if (!t) return nullptr;
    here(*t, what);
    TORCH_CHECK_VALUE(t->scalar_type() == type && t->numel() == 1, what, " must be one ", type,
                      " element");
    return t->data_ptr();
  };
  const at::ScalarType held = eight ? at::kFloat8_e4m3fn : at::kFloat;
  std::vector<flp_adamw_tensor> table;
  table.reserve(count);
  std::vector<const at::Tensor*> written;
  written.reserve(count * 5);
  for (size_t k = 0; k < count; ++k) {
    const at::Tensor* const grad = grads.at(k);
    if (grad == nullptr) continue;
    const at::Tensor &p = params.need(k), &g = *grad;
    const int64_t n = p.numel();
    here(p, "parameters");
    here(g, "gradients");
    TORCH_CHECK_TYPE(p.scalar_type() == at::kBFloat16 || p.scalar_type() == at::kHalf ||
                         p.scalar_type() == at::kFloat,
                     "parameters must be bfloat16, float16 or float32");
    TORCH_CHECK_TYPE(g.scalar_type() == p.scalar_type() || g.scalar_type() == at::kFloat,
                     "a gradient must have its parameter's dtype or float32");
    TORCH_CHECK_VALUE(g.sizes() == p.sizes(), "a gradient must have its parameter's shape");
    flp_adamw_tensor t{};
    t.param = ptr(p);
    t.grad = ptr(g);
    t.n = n;
    t.weight_decay = decay[one_decay ? 0 : k];
    t.p_dtype = code(p);
    t.g_dtype = code(g);
    written.push_back(&p);
    auto state = [&](const at::Tensor& s) {
      here(s, "states");
      TORCH_CHECK_TYPE(s.scalar_type() == held, "states must be ", held,
                       eight ? " where they have scales" : " where they have no scales");
      TORCH_CHECK_VALUE(s.numel() == n, "a state must have as many elements as its parameter");
      written.push_back(&s);
      return ptr(s);
    };
    auto scale = [&](const at::Tensor& s) {
      here(s, "scales");
      TORCH_CHECK_VALUE(s.scalar_type() == at::kFloat && s.numel() == (n + 255) / 256,
                        "scales must be float32, one for each 256 elements of the parameter");
      written.push_back(&s);
      return fptr(s);
    };
    t.exp_avg = state(exp_avg.need(k));
    t.exp_avg_sq = state(exp_avg_sq.need(k));
    if (eight) {
      t.exp_avg_scale = scale(exp_avg_scale->need(k));
      t.exp_avg_sq_scale = scale(exp_avg_sq_scale->need(k));
    }
    if (master && master->at(k) != nullptr) {
      const at::Tensor& w = master->need(k);
      here(w, "master copies");
      TORCH_CHECK_VALUE(w.scalar_type() == at::kFloat && w.numel() == n,
                        "a master copy must be float32 with its parameter's elements");
      written.push_back(&w);
      t.master = fptr(w);
    }
    table.push_back(t);
  }
  const auto* at_step = static_cast<const int64_t*>(scalar(step_on_device, at::kLong, "step"));
  const auto* at_lr = static_cast<const float*>(scalar(lr_on_device, at::kFloat, "lr"));
  const auto* at_scale = static_cast<const float*>(scalar(grad_scale, at::kFloat, "grad_scale"));
  check("flp_adamw_step",
        api.adamw_step(int64_t(table.size()), table.data(), eight ? 8 : 32, step, at_step, lr, at_lr,
                       beta1, beta2, eps, at_scale, reinterpret_cast<void*>(stream)));
  // what was saved for a backward has changed
  for (const at::Tensor* t : written)
    if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

}  // namespace

PYBIND11_MODULE(_flp_torch, m) {
  m.doc() = "Autograd nodes over libflp.so.";
  py::register_exception_translator([](std::exception_ptr p) {  // out of a forward
    try {
      if (p) std::rethrow_exception(p);
    } catch (python_error& e) {
      e.restore();
    }
  });
  m.def("bind", &bind);
  m.def("first_order", [](const at::Tensor& t) { return first_order(t); });
  m.def("embedding", [](const at::Tensor& weight, const at::Tensor& ids, double scale,
                        int64_t stream) { return EmbeddingNode::apply(weight, ids, scale, stream); });
  m.def("dropout", [](const at::Tensor& x, double p, const at::Tensor& rng, int64_t stream) {
    return DropoutNode::apply(x, p, rng, stream);
  });
  m.def("layer_norm", [](const at::Tensor& x, const OptTensor& weight, const OptTensor& bias,
                         double eps, int64_t stream) {
    return LayerNormNode::apply(x, weight, bias, eps, stream);
  });
  m.def("gated_linear", [](const at::Tensor& x, const at::Tensor& w_gate, const at::Tensor& w_up,
                           int64_t act, int64_t stream) {
    return GatedLinearNode::apply(x, w_gate, w_up, act, stream);
  });
  m.def("rms_norm", [](const at::Tensor& x, const OptTensor& y, const OptTensor& weight,
                       const OptTensor& post_weight, const OptTensor& gate, bool post,
                       double scale, double eps, int64_t stream) {
    return RmsNormNode::apply(x, y, weight, post_weight, gate, post, scale, eps, stream);
  });
  m.def("adamw_step", &adamw_step);
  m.def("cross_entropy",
        [](const at::Tensor& hidden, const at::Tensor& weight, const at::Tensor& targets,
           const OptTensor& bias, double smoothing, double z_loss, int64_t reduction,
           int64_t most_workspace, int64_t stream) {
          return CrossEntropyNode::apply(hidden, weight, targets, bias, smoothing, z_loss,
                                         reduction, most_workspace, stream);
        });
}
