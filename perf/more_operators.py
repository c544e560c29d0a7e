"""Workloads of the operators of a model's blocks between its embedding and its head, and of the
step that trains them:

    gated     out = act(x @ w_gate^T) * (x @ w_up^T), the first half of a gated feed-forward
              block, and its gradients
    norm      the norms around a block: r = x + scale * gate * norm(y) and n = norm(r), root
              mean square norms, and their gradients
    adamw     one AdamW step over all tensors of a model, states in 32 bits or in 8

Every case can be run in two ways on the same inputs: in elementary torch operations in
32 bits (``own = False``), and through this package's entry points (``own = True``).
``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}

# The width and batch of the training workload of bench.py, and 8/3 of the width.
_D, _N, _F = 2688, 16384, 7168


def listed():
    return [
        # one token of one sequence: the weights are all there is to read
        dict(name="gated_token", op="gated", N=1, D=_D, F=_F, dtype="bf16", act="silu", grad=False),
        # a small fp32 model's step, nothing a multiple of the tiles
        dict(name="gated_small_fp32", op="gated", N=201, D=288, F=771, dtype="fp32", act="silu",
             grad=True),
        # a ragged fp16 batch, an odd inner width
        dict(name="gated_ragged_fp16", op="gated", N=1000, D=1344, F=3587, dtype="fp16",
             act="gelu", grad=True),
        # one training step of a block as wide as the headline head
        dict(name="gated_train", op="gated", N=_N, D=_D, F=_F, dtype="bf16", act="silu",
             grad=True),
        # behind a block of one decoding step of a small serving batch
        dict(name="norm_decode", op="norm", N=32, D=_D, dtype="bf16", wdtype="bf16", groups=0,
             block=True, post=False, grad=False),
        # in front of the first block of a small fp32 model: no block's output yet
        dict(name="norm_first_fp32", op="norm", N=513, D=777, dtype="fp32", wdtype="fp32",
             groups=0, block=False, post=False, grad=True),
        # 17 sequences of 241 tokens with a gate each, fp32 parameters over fp16 rows that
        # start off the 16-byte grid
        dict(name="norm_odd_fp16", op="norm", N=4097, D=1345, dtype="fp16", wdtype="fp32",
             groups=17, block=True, post=True, grad=True),
        # one training step: a norm on both sides of the block and a learned gate per channel
        dict(name="norm_train", op="norm", N=_N, D=_D, dtype="bf16", wdtype="bf16", groups=1,
             block=True, post=True, grad=True),
        # a tiny fp32 model: thirty tensors, most of them far below one tile
        dict(name="adamw_small_fp32", op="adamw", layers=6, D=97, F=259, V=501, dtype="fp32",
             gdtype="fp32", bits=32, master=False),
        # fine-tuning a small fp16 model with 8-bit states
        dict(name="adamw_fp16_8bit", op="adamw", layers=8, D=520, F=1387, V=5003, dtype="fp16",
             gdtype="fp32", bits=8, master=True),
        # a bfloat16 model with fp32 master weights and states
        dict(name="adamw_bf16_master", op="adamw", layers=6, D=_D, F=_F, V=0, dtype="bf16",
             gdtype="bf16", bits=32, master=True),
        # the same with 8-bit states and the headline head's matrix among the tensors
        dict(name="adamw_head_8bit", op="adamw", layers=4, D=_D, F=_F, V=131072, dtype="bf16",
             gdtype="bf16", bits=8, master=False),
    ]


def _log_size(rng, lo, hi):
    """A size whose logarithm is uniform between those of lo and hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "norm", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "gated":
        while True:
            case = dict(op=op, N=_log_size(rng, 1, 16384), D=32 * _log_size(rng, 2, 128),
                        F=_log_size(rng, 100, 14336), dtype=dtype,
                        act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                        grad=rng.random() < 0.7)
            # fp32 products run at a small fraction of the 16-bit rate
            cost = case["N"] * case["D"] * case["F"] * (16 if dtype == "fp32" else 1)
            if cost <= _N * _D * _F:
                return case
    if op == "norm":
        groups = rng.choice([0, 0, 1, 1, _log_size(rng, 2, 64)])
        each = max(1, groups)
        block = rng.random() < 0.8
        return dict(op=op, N=each * max(1, _log_size(rng, 1, 16384) // each),
                    D=_log_size(rng, 32, 2688), dtype=dtype, wdtype=rng.choice([dtype, "fp32"]),
                    groups=groups if block else 0, block=block,
                    post=block and rng.random() < 0.5, grad=rng.random() < 0.7)
    return dict(op=op, layers=rng.randint(1, 8), D=_log_size(rng, 32, 2688),
                F=_log_size(rng, 64, 4096), V=rng.choice([0, _log_size(rng, 100, 50257)]),
                dtype=dtype, gdtype=rng.choice([dtype, "fp32"]), bits=rng.choice([8, 32]),
                master=dtype != "fp32" and rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------------

_EPS = 1e-6                                          # of the norms
_LR, _BETAS, _ADAM_EPS, _DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.1
_SCALE = 0.7                                         # of the residual branch
_GROUP = 256                                         # elements that share a scale in 8 bits
_TOP, _LEAST = 448.0, 2.0 ** -9                      # largest and smallest positive 8-bit values
_FLOOR = 2.0 ** -100                                 # a block's largest value counts as at least this


def _shapes(case):
    """The model's tensors: the matrices, then the vectors, which do not decay."""
    D, F, V, n = case["D"], case["F"], case["V"], case["layers"]
    matrices = ([(V, D)] if V else []) + [(F, D), (F, D), (D, F)] * n
    return matrices, [(D,), (D,)] * n + [(D,)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = dict(case=case)
    if case["op"] == "gated":
        N, D, F = case["N"], case["D"], case["F"]
        s["x"] = normal(N, D)
        s["w_gate"] = normal(F, D, std=1 / math.sqrt(D))
        s["w_up"] = normal(F, D, std=1 / math.sqrt(D))
        if case["grad"]:
            s["grad_out"] = normal(N, F)
    elif case["op"] == "norm":
        N, D = case["N"], case["D"]
        wd = _DTYPES[case["wdtype"]]
        # rows of different size, as a residual stream has them
        size = torch.rand(N, 1, generator=g, device="cuda") * 4 + 0.5
        s["x"] = (torch.randn(N, D, generator=g, device="cuda") * size).to(dt)
        s["weight"] = normal(D, std=0.1, mean=1.0, dtype=wd)
        if case["block"]:
            s["y"] = (torch.randn(N, D, generator=g, device="cuda") * (size * 0.3 + 0.1)).to(dt)
            s["post_weight"] = normal(D, std=0.1, mean=1.0, dtype=wd) if case["post"] else None
            s["gate"] = None
            if case["groups"]:
                s["gate"] = normal(case["groups"], D, std=0.2, mean=0.5, dtype=wd)
        if case["grad"]:
            s["grad_n"] = normal(N, D)
            if case["block"]:
                s["grad_r"] = normal(N, D)
    else:
        # Every kind of tensor in one buffer, each tensor from a multiple of _GROUP elements on.
        matrices, vectors = _shapes(case)
        at, spans = 0, []
        for k, shape in enumerate(matrices + vectors):
            spans.append((at, math.prod(shape), shape))
            at += -(-spans[-1][1] // _GROUP) * _GROUP
            if k + 1 == len(matrices):
                s["decays"] = at
        def used(flat):
            for a, n, _ in spans:
                flat[a + n:a + -(-n // _GROUP) * _GROUP] = 0
            return flat
        p = used(torch.randn(at, generator=g, device="cuda").mul_(0.02))
        s["param"] = p.to(dt)
        s["master"] = p.to(dt).float().add_(p, alpha=2.0 ** -12) if case["master"] else None
        # gradients of very different size from tensor to tensor and within one
        size = torch.exp(torch.randn(at // _GROUP, 1, generator=g, device="cuda") * 1.5 - 5)
        draw_ = lambda: used((torch.randn(at // _GROUP, _GROUP, generator=g, device="cuda")  # noqa: E731
                              * size).view(-1))
        s["grad"] = draw_().to(_DTYPES[case["gdtype"]])
        m, v = draw_().mul_(0.3), draw_().square_().mul_(0.5)
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _to8(m)
            s["v"], s["v_scale"] = _to8(v.sqrt_(), divisor=True)
        else:
            s["m"], s["v"] = m, v
        s["step"] = 1000 + int(seed) % 7
        # the tensors as a training program holds them
        kinds = ["param", "grad", "m", "v"] + (["master"] if case["master"] else [])
        s["tensors"] = {k: [s[k][a:a + n].view(shape) for a, n, shape in spans] for k in kinds}
        if case["bits"] == 8:
            for k in ("m_scale", "v_scale"):
                s["tensors"][k] = [s[k][a // _GROUP:-(-(a + n) // _GROUP)] for a, n, _ in spans]
        s["decay"] = [_DECAY] * len(matrices) + [0.0] * len(vectors)
    # what a training program holds as parameters and activations to differentiate by
    if case.get("grad"):
        for k in ("x", "y", "w_gate", "w_up", "weight", "post_weight", "gate"):
            if s.get(k) is not None:
                s[k].requires_grad_(True)
    return s


# ---- the plain form: elementary operations in 32 bits, one rounding at the end ------------------

def _erf_part(z):
    """The normal distribution's integral up to z."""
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _plain_act(act, z):
    """act(z) and its derivative."""
    if act == "silu":
        f = torch.sigmoid(z)
        return z * f, f * (1.0 + z * (1.0 - f))
    if act == "gelu":
        f = _erf_part(z)
        return z * f, f + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), (0.5 * (1.0 + t)
                                 + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z))


def _plain_gated(s):
    dt = s["x"].dtype
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    z, u = x @ wg.t(), x @ wu.t()
    a, da = _plain_act(s["case"]["act"], z)
    out = (a * u).to(dt)
    if "grad_out" not in s:
        return out
    g = s["grad_out"].float()
    dz, du = g * u * da, g * a
    return (out, (dz @ wg + du @ wu).to(dt), (dz.t() @ x).to(dt), (du.t() @ x).to(dt))


def _plain_norm(s):
    case, dt = s["case"], s["x"].dtype
    N, D = s["x"].shape
    w = s["weight"].float()
    r = s["x"].float()
    if case["block"]:
        y = s["y"].float()
        hat = y
        if case["post"]:
            rstd_y = torch.rsqrt((y * y).mean(dim=1, keepdim=True) + _EPS)
            hat = y * rstd_y
            wp = s["post_weight"].float()
            p = hat * wp
        else:
            p = y
        gate = None
        if s["gate"] is not None:
            gate = s["gate"].float().repeat_interleave(N // s["gate"].shape[0], dim=0)
            p = p * gate
        r = r + _SCALE * p
    rstd = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + _EPS)
    rhat = r * rstd
    n = (rhat * w).to(dt)
    outs = (r.to(dt), n) if case["block"] else (n,)
    if not case["grad"]:
        return outs
    gn = s["grad_n"].float()
    gw = gn * w
    dr = rstd * (gw - rhat * (gw * rhat).mean(dim=1, keepdim=True))
    outs = outs + ((gn * rhat).sum(dim=0).to(s["weight"].dtype),)
    if not case["block"]:
        return outs + (dr.to(dt),)
    dr = dr + s["grad_r"].float()
    dp = _SCALE * dr                            # by gate * p
    if gate is not None:
        d_gate = dp * (hat * wp if case["post"] else y)
        d_gate = d_gate.view(s["gate"].shape[0], -1, D).sum(dim=1).to(s["gate"].dtype)
        dp = dp * gate
    dy = dp
    if case["post"]:
        gy = dp * wp
        dy = rstd_y * (gy - hat * (gy * hat).mean(dim=1, keepdim=True))
        outs = outs + ((dp * hat).sum(dim=0).to(s["post_weight"].dtype),)
    if gate is not None:
        outs = outs + (d_gate,)
    return outs + (dr.to(dt), dy.to(dt))


def _to8(x, divisor=False):
    """x in 8 bits with a scale per _GROUP elements.  Of what is divided by (the roots of second
    moments), no positive value becomes 0."""
    b = x.view(-1, _GROUP)
    top = b.abs().amax(dim=1, keepdim=True).clamp_(min=_FLOOR)
    q = b * (_TOP / top)
    if divisor:
        q = torch.where(b > 0, q.clamp(min=_LEAST), q)
    return q.to(torch.float8_e4m3fn).view(-1), (top * (1.0 / _TOP)).view(-1)


def _from8(q, scale):
    return (q.view(-1, _GROUP).float() * scale[:, None]).view(-1)


def _plain_adamw(s):
    case, t = s["case"], s["step"]
    s["step"] += 1
    (b1, b2), eight = _BETAS, case["bits"] == 8
    g = s["grad"].float()
    m = _from8(s["m"], s["m_scale"]) if eight else s["m"]
    v = _from8(s["v"], s["v_scale"]).square() if eight else s["v"]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * (g * g)
    root = v.sqrt()
    p = (s["master"] if case["master"] else s["param"]).float()
    k = s["decays"]
    p = torch.cat([p[:k] * (1.0 - _LR * _DECAY), p[k:]])
    p = p - _LR / (1.0 - b1 ** t) * (m / (root / math.sqrt(1.0 - b2 ** t) + _ADAM_EPS))
    s["param"].copy_(p)
    if case["master"]:
        s["master"].copy_(p)
    if eight:
        q, scale = _to8(m)
        s["m"].copy_(q), s["m_scale"].copy_(scale)
        q, scale = _to8(root, divisor=True)
        s["v"].copy_(q), s["v_scale"].copy_(scale)
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("param", "master", "m", "m_scale", "v", "v_scale")
            if s.get(k) is not None}


# ---- this package's entry points -----------------------------------------------------------------

def _own(s):
    import lm_head_selected_bf16_amd as flp
    case = s["case"]
    if case["op"] == "gated":
        out = flp.gated_linear(s["x"], s["w_gate"], s["w_up"], activation=case["act"])
        if not case["grad"]:
            return out
        return (out,) + torch.autograd.grad(out, [s["x"], s["w_gate"], s["w_up"]], s["grad_out"])
    if case["op"] == "norm" and not case["block"]:
        n = flp.rms_norm(s["x"], s["weight"], eps=_EPS)
        if not case["grad"]:
            return (n,)
        dx, dw = torch.autograd.grad(n, [s["x"], s["weight"]], s["grad_n"])
        return n, dw, dx
    if case["op"] == "norm":
        r, n = flp.residual_rms_norm(s["x"], s["y"], s["weight"], post_weight=s["post_weight"],
                                     gate=s["gate"], scale=_SCALE, eps=_EPS)
        if not case["grad"]:
            return r, n
        leaves = [s[k] for k in ("weight", "post_weight", "gate", "x", "y") if s[k] is not None]
        return (r, n) + torch.autograd.grad([r, n], leaves, [s["grad_r"], s["grad_n"]])
    t = s["tensors"]
    state = flp.AdamWState(t["m"], t["v"], t.get("m_scale"), t.get("v_scale"), t.get("master"))
    flp.adamw_step(t["param"], t["grad"], state, s["step"], _LR, betas=_BETAS, eps=_ADAM_EPS,
                   weight_decay=s["decay"])
    s["step"] += 1
    return _adamw_outputs(s)


def run(state):
    if own:
        return _own(state)
    plain = {"gated": _plain_gated, "norm": _plain_norm, "adamw": _plain_adamw}
    with torch.no_grad():
        return plain[state["case"]["op"]](state)


def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"] == "gated":
        N, D, F = case["N"], case["D"], case["F"]
        b, f = (N * D + 2 * F * D + N * F) * e, 4 * N * D * F
        if case["grad"]:
            b += (N * F + N * D + 2 * F * D) * e
            f += 8 * N * D * F
        return {"bytes": b, "flops": f}
    if case["op"] == "norm":
        N, D, we = case["N"], case["D"], _SIZE[case["wdtype"]]
        params = (1 + (1 if case["post"] else 0) + case["groups"]) * D * we
        rows = 4 if case["block"] else 2
        b, f = rows * N * D * e + params, 3 * rows * N * D
        if case["grad"]:
            b += rows * N * D * e + params
            f += 7 * rows * N * D
        return {"bytes": b, "flops": f}
    matrices, vectors = _shapes(case)
    n = sum(math.prod(shape) for shape in matrices + vectors)
    state = 2 * (1 + 4 / _GROUP) if case["bits"] == 8 else 8
    # param, master and states are read and written, the gradient is read; a parameter beside
    # its master is written only
    b = n * (_SIZE[case["gdtype"]] + 2 * state + (e + 8 if case["master"] else 2 * e))
    return {"bytes": int(b), "flops": 16 * n}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _exact_gated(case, s):
    import torch.nn.functional as nnf
    x, wg, wu = (s[k].detach().double().requires_grad_(case["grad"])
                 for k in ("x", "w_gate", "w_up"))
    z = x @ wg.T
    if case["act"] == "silu":
        a = nnf.silu(z)
    else:
        a = nnf.gelu(z, approximate="tanh" if case["act"] == "gelu_tanh" else "none")
    out = a * (x @ wu.T)
    if not case["grad"]:
        return out
    return (out.detach(),) + torch.autograd.grad(out, [x, wg, wu], s["grad_out"].double())


def _exact_norm(case, s):
    def rms(v, weight):
        return v / torch.sqrt(v.square().sum(dim=-1, keepdim=True) / v.shape[-1] + _EPS) * weight

    names = [k for k in ("weight", "post_weight", "gate", "x", "y") if s.get(k) is not None]
    d = {k: s[k].detach().double().requires_grad_(case["grad"]) for k in names}
    if not case["block"]:
        n = rms(d["x"], d["weight"])
        if not case["grad"]:
            return (n,)
        return (n.detach(),) + torch.autograd.grad(n, [d["weight"], d["x"]], s["grad_n"].double())
    b = rms(d["y"], d["post_weight"]) if case["post"] else d["y"]
    if case["groups"]:
        b = (b.view(case["groups"], -1, case["D"]) * d["gate"][:, None, :]).view_as(b)
    r = d["x"] + b * _SCALE
    n = rms(r, d["weight"])
    if not case["grad"]:
        return r, n
    grads = torch.autograd.grad([r, n], [d[k] for k in names],
                                [s["grad_r"].double(), s["grad_n"].double()])
    return (r.detach(), n.detach()) + grads


def _exact_adamw(case, s):
    (b1, b2), t = _BETAS, s["step"]

    def held(name):
        x = s[name].double()
        if case["bits"] == 32:
            return x
        return x * s[name + "_scale"].double().repeat_interleave(_GROUP)

    def in8(x):
        top = x.view(-1, _GROUP).abs().amax(dim=1).clamp(min=_FLOOR)
        q = x / top.repeat_interleave(_GROUP) * _TOP
        return q.float().to(torch.float8_e4m3fn).double(), top / _TOP

    g = s["grad"].double()
    m = held("m") * b1 + g * (1 - b1)
    v = held("v")
    v = (v * v if case["bits"] == 8 else v) * b2 + g * g * (1 - b2)
    p = (s["master"] if case["master"] else s["param"]).double()
    p[:s["decays"]] *= 1 - _LR * _DECAY
    root = torch.sqrt(v)
    p -= _LR * (m / (1 - b1 ** t)) / (root / math.sqrt(1 - b2 ** t) + _ADAM_EPS)
    out = {"param": p}
    if case["master"]:
        out["master"] = p
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    (out["m"], out["m_scale"]), (code, out["v_scale"]) = in8(m), in8(root)
    out["v"] = torch.where((root > 0) & (code < _LEAST), _LEAST, code)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "norm": _exact_norm, "adamw": _exact_adamw}[case["op"]](case, s)
