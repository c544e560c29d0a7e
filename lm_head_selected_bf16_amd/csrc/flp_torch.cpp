// Autograd nodes of the operators around a model's body (embedding lookup, dropout, layer
// norm, linear cross entropy), over the C ABI.
//
// They allocate outputs and workspaces with torch and pass addresses on, as torch_ops.py does
// for the other operators; the checks of a call's arguments are made there, before it comes
// here.  Autograd runs a backward on a thread of its own, which has to take over the Python
// interpreter for a node written in Python and then runs it from cold caches: a layer norm of
// 37 x 1003, forward and backward, took 118 us on the host that way and takes 74 here.
#include <torch/csrc/Exceptions.h>
#include <torch/extension.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <optional>
#include <stdexcept>
#include <string>

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
  m.def("cross_entropy",
        [](const at::Tensor& hidden, const at::Tensor& weight, const at::Tensor& targets,
           const OptTensor& bias, double smoothing, double z_loss, int64_t reduction,
           int64_t most_workspace, int64_t stream) {
          return CrossEntropyNode::apply(hidden, weight, targets, bias, smoothing, z_loss,
                                         reduction, most_workspace, stream);
        });
}
