"""Workloads of the operators around a language model's head and embedding:

    embedding       out = scale * weight[ids], d_weight by sorted tokens
    dropout         out = x * keep / (1 - p), keep recomputed from a counter-based generator
    layer_norm      normalisation over the last dimension, with d_weight and d_bias
    cross_entropy   softmax cross entropy of hidden @ weight^T + bias with label smoothing
                    and a squared log-partition term, and its gradients

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

# The head and embedding of the training workload of bench.py.
_D, _V, _N = 2688, 131072, 16384


def listed():
    return [
        # the token embedding of one decoding step of a small serving batch
        dict(name="embedding_decode", op="embedding", N=32, D=_D, V=_V, dtype="bf16", grad=False),
        # fine-tuning a small vocabulary in fp32, an odd number of tokens
        dict(name="embedding_small_fp32", op="embedding", N=1501, D=520, V=5003, dtype="fp32",
             grad=True),
        # the embedding of one training step: lookup and the gradient of the whole table
        dict(name="embedding_train", op="embedding", N=_N, D=_D, V=_V, dtype="bf16", grad=True),
        # dropout of a short fp32 sequence with an odd number of elements
        dict(name="dropout_small_fp32", op="dropout", N=37, D=1003, dtype="fp32", p=0.25),
        # dropout of the hidden states of one training step, forward and backward
        dict(name="dropout_train", op="dropout", N=_N, D=_D, dtype="bf16", p=0.1),
        # the final norm of one decoding step
        dict(name="norm_decode", op="layer_norm", N=32, D=_D, dtype="bf16", wdtype="bf16",
             grad=False),
        # an odd width whose rows start off the 16-byte grid, fp32 parameters over fp16 rows
        dict(name="norm_odd_fp16", op="layer_norm", N=4097, D=1345, dtype="fp16", wdtype="fp32",
             grad=True),
        # the final norm of one training step, with both parameter gradients
        dict(name="norm_train", op="layer_norm", N=_N, D=_D, dtype="bf16", wdtype="bf16",
             grad=True),
        # a tiny fp32 model, every term of the loss
        dict(name="loss_tiny_fp32", op="cross_entropy", N=64, D=256, V=4096, dtype="fp32",
             smoothing=0.1, z_loss=1e-4, bias=True, reduction="mean", ignored=0.06, grad=True),
        # a ragged fp16 batch of padded sequences over a vocabulary of no round size
        dict(name="loss_ragged_fp16", op="cross_entropy", N=1000, D=1344, V=50257, dtype="fp16",
             smoothing=0.0, z_loss=1e-4, bias=False, reduction="sum", ignored=0.2, grad=True),
        # evaluation: the loss of every token, no gradient
        dict(name="loss_eval", op="cross_entropy", N=2048, D=_D, V=_V, dtype="bf16",
             smoothing=0.0, z_loss=0.0, bias=False, reduction="none", ignored=0.05, grad=False),
        # the loss and every gradient of one training step of the headline head
        dict(name="loss_train", op="cross_entropy", N=_N, D=_D, V=_V, dtype="bf16",
             smoothing=0.05, z_loss=1e-4, bias=True, reduction="mean", ignored=0.02, grad=True),
    ]


def _log_size(rng, lo, hi):
    """A size whose logarithm is uniform between those of lo and hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embedding", "dropout", "layer_norm", "cross_entropy"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "embedding":
        return dict(op=op, N=_log_size(rng, 1, 16384), D=8 * _log_size(rng, 4, 336),
                    V=_log_size(rng, 100, 131072), dtype=dtype, grad=rng.random() < 0.7)
    if op == "dropout":
        return dict(op=op, N=_log_size(rng, 1, 16384), D=_log_size(rng, 32, 2688), dtype=dtype,
                    p=rng.choice([0.05, 0.1, 0.2, 0.5]))
    if op == "layer_norm":
        return dict(op=op, N=_log_size(rng, 1, 16384), D=_log_size(rng, 32, 2688), dtype=dtype,
                    wdtype=rng.choice([dtype, "fp32"]), grad=rng.random() < 0.7)
    while True:
        case = dict(op=op, N=_log_size(rng, 1, 8192), D=32 * _log_size(rng, 2, 84),
                    V=_log_size(rng, 500, 131072), dtype=dtype,
                    smoothing=rng.choice([0.0, 0.1]), z_loss=rng.choice([0.0, 1e-4]),
                    bias=rng.random() < 0.5, reduction=rng.choice(["mean", "sum", "none"]),
                    ignored=rng.choice([0.0, 0.1]), grad=rng.random() < 0.7)
        # fp32 products run at a small fraction of the 16-bit rate
        cost = case["N"] * case["D"] * case["V"] * (16 if dtype == "fp32" else 1)
        if cost <= _N * _D * _V:
            return case


# ---- inputs ------------------------------------------------------------------------------------

def _skewed_ids(n, V, g):
    """Token ids whose frequency falls with their rank, as in text."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1.0)).floor().long() - 1).clamp_(0, V - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]
    N, D = case["N"], case["D"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = dict(case=case)
    if case["op"] == "embedding":
        V = case["V"]
        s["weight"] = normal(V, D, std=0.02)
        s["ids"] = _skewed_ids(N, V, g)
        # one position in fifty is padding, marked by an id outside the table
        pad = torch.rand(N, generator=g, device="cuda") < 0.02
        s["ids"] = torch.where(pad, torch.full_like(s["ids"], -1), s["ids"])
        s["scale"] = math.sqrt(D)
        if case["grad"]:
            s["grad_out"] = normal(N, D)
    elif case["op"] == "dropout":
        s["x"] = normal(N, D)
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
        s["grad_out"] = normal(N, D)
    elif case["op"] == "layer_norm":
        wd = _DTYPES[case["wdtype"]]
        # rows of different size and offset, as a residual stream has them
        size = torch.rand(N, 1, generator=g, device="cuda") * 4 + 0.5
        s["x"] = (torch.randn(N, D, generator=g, device="cuda") * size + 0.3 * size).to(dt)
        s["weight"] = normal(D, std=0.1, mean=1.0, dtype=wd)
        s["bias"] = normal(D, std=0.1, dtype=wd)
        if case["grad"]:
            s["grad_out"] = normal(N, D)
    else:
        V = case["V"]
        s["hidden"] = normal(N, D)
        s["weight"] = normal(V, D, std=0.02)
        s["bias"] = normal(V, std=0.1, dtype=torch.float32) if case["bias"] else None
        t = _skewed_ids(N, V, g)
        pad = torch.rand(N, generator=g, device="cuda") < case["ignored"]
        s["targets"] = torch.where(pad, torch.full_like(t, -100), t)
        if case["grad"] and case["reduction"] == "none":
            s["grad_out"] = normal(N, dtype=torch.float32)
    # what a training program holds as parameters and activations to differentiate by
    if case.get("grad", True):
        for k in ("x", "hidden", "weight", "bias"):
            if s.get(k) is not None:
                s[k].requires_grad_(True)
    return s


# ---- the plain form: elementary operations in 32 bits, one rounding at the end ------------------

def _plain_embedding(s):
    w, ids, scale = s["weight"], s["ids"], s["scale"]
    ok = (ids >= 0) & (ids < w.shape[0])
    rows = w[torch.where(ok, ids, torch.zeros_like(ids))].float() * scale
    out = torch.where(ok[:, None], rows, torch.zeros_like(rows)).to(w.dtype)
    if "grad_out" not in s:
        return out
    acc = torch.zeros(w.shape, device=w.device)
    acc.index_add_(0, ids[ok], s["grad_out"][ok].float())
    return out, (acc * scale).to(w.dtype)


def _keep(rng, n, p):
    """keep[e] for elements e = 0 .. n - 1: ten rounds of the 4 x 32 counter-based generator
    of Salmon et al. (2011), key = rng[0], counter = (e / 8, rng[1]); element e takes the
    16-bit piece e % 8 of the four words, and is kept where it is at least 65536 p."""
    m32 = 0xFFFFFFFF
    blocks = torch.arange((n + 7) // 8, device=rng.device, dtype=torch.int64)
    c = [blocks & m32, (blocks >> 32) & m32,
         (rng[1] & m32).expand_as(blocks), ((rng[1] >> 32) & m32).expand_as(blocks)]
    k0, k1 = rng[0] & m32, (rng[0] >> 32) & m32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & m32) ^ c[1] ^ k0, b & m32, ((a >> 32) & m32) ^ c[3] ^ k1, a & m32]
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    pieces = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], dim=1)
    return pieces.reshape(-1)[:n] >= int(p * 65536 + 0.5)


def _plain_dropout(s):
    x, p = s["x"], s["case"]["p"]
    drop = int(p * 65536 + 0.5)
    keep = _keep(s["rng"], x.numel(), p).view(x.shape)
    scale = 65536.0 / (65536 - drop)
    zero = torch.zeros((), device=x.device)
    return tuple(torch.where(keep, v.float() * scale, zero).to(x.dtype)
                 for v in (x, s["grad_out"]))


_EPS = 1e-5


def _plain_layer_norm(s):
    x = s["x"].float()
    w, b = s["weight"].float(), s["bias"].float()
    c = x - x.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((c * c).mean(dim=1, keepdim=True) + _EPS)
    xhat = c * rstd
    y = (xhat * w + b).to(s["x"].dtype)
    if "grad_out" not in s:
        return y
    g = s["grad_out"].float()
    gw = g * w
    dx = (gw - gw.mean(dim=1, keepdim=True) - xhat * (gw * xhat).mean(dim=1, keepdim=True)) * rstd
    return (y, dx.to(s["x"].dtype), (g * xhat).sum(dim=0).to(s["weight"].dtype),
            g.sum(dim=0).to(s["bias"].dtype))


def _plain_cross_entropy(s):
    case = s["case"]
    V = case["V"]
    h, w, t = s["hidden"].float(), s["weight"].float(), s["targets"]
    eps, zl = case["smoothing"], case["z_loss"]
    ok = (t >= 0) & (t < V)
    count = ok.sum().clamp(min=1)
    tc = torch.where(ok, t, torch.zeros_like(t))[:, None]
    z = h @ w.t()
    if s["bias"] is not None:
        z += s["bias"]
    m = z.max(dim=1, keepdim=True).values
    lse = m[:, 0] + torch.log(torch.exp(z - m).sum(dim=1))
    val = lse - (1.0 - eps) * z.gather(1, tc)[:, 0] - eps * z.mean(dim=1) + zl * lse * lse
    rows = torch.where(ok, val, torch.zeros_like(val))
    loss = {"none": rows, "sum": rows.sum(), "mean": rows.sum() / count}[case["reduction"]]
    if not case["grad"]:
        return loss
    up = {"none": s.get("grad_out", rows), "sum": torch.ones_like(rows),
          "mean": torch.ones_like(rows) / count}[case["reduction"]]
    up = torch.where(ok, up, torch.zeros_like(up))[:, None]
    dz = torch.exp(z - lse[:, None]) * (1.0 + 2.0 * zl * lse)[:, None] - eps / V
    dz.scatter_add_(1, tc, torch.full_like(rows, eps - 1.0)[:, None])
    dz *= up
    grads = (loss, (dz @ w).to(s["hidden"].dtype), (dz.t() @ h).to(s["weight"].dtype))
    return grads if s["bias"] is None else grads + (dz.sum(dim=0),)


# ---- this package's entry points -----------------------------------------------------------------

def _own(s):
    import lm_head_selected_bf16_amd as flp
    case = s["case"]
    if case["op"] == "embedding":
        out = flp.embedding(s["weight"], s["ids"], scale=s["scale"])
        if not case["grad"]:
            return out
        return (out,) + torch.autograd.grad(out, [s["weight"]], s["grad_out"])
    if case["op"] == "dropout":
        out = flp.dropout(s["x"], case["p"], s["rng"])
        return (out,) + torch.autograd.grad(out, [s["x"]], s["grad_out"])
    if case["op"] == "layer_norm":
        y = flp.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS)
        if not case["grad"]:
            return y
        return (y,) + torch.autograd.grad(y, [s["x"], s["weight"], s["bias"]], s["grad_out"])
    loss = flp.linear_cross_entropy(s["hidden"], s["weight"], s["targets"], bias=s["bias"],
                                    label_smoothing=case["smoothing"], z_loss=case["z_loss"],
                                    reduction=case["reduction"])
    if not case["grad"]:
        return loss
    leaves = [s["hidden"], s["weight"]] + ([] if s["bias"] is None else [s["bias"]])
    return (loss,) + torch.autograd.grad(loss, leaves, s.get("grad_out"))


def run(state):
    if own:
        return _own(state)
    plain = {"embedding": _plain_embedding, "dropout": _plain_dropout,
             "layer_norm": _plain_layer_norm, "cross_entropy": _plain_cross_entropy}
    with torch.no_grad():
        return plain[state["case"]["op"]](state)


def work(case):
    N, D, e = case["N"], case["D"], _SIZE[case["dtype"]]
    if case["op"] == "embedding":
        V = case["V"]
        b = N * 8 + min(N, V) * D * e + N * D * e
        if case["grad"]:
            b += N * D * e + V * D * e
        return {"bytes": b, "flops": N * D * (2 if case["grad"] else 1)}
    if case["op"] == "dropout":
        # two passes; ten rounds of two products per eight elements and pass
        return {"bytes": 4 * N * D * e, "flops": 2 * N * D}
    if case["op"] == "layer_norm":
        we = _SIZE[case["wdtype"]]
        b, f = 2 * N * D * e + 2 * D * we, 8 * N * D
        if case["grad"]:
            b += 2 * N * D * e + 2 * D * we
            f += 14 * N * D
        return {"bytes": b, "flops": f}
    V = case["V"]
    b = N * D * e + V * D * e + N * 8 + (V * 4 if case["bias"] else 0)
    b += N * 4 if case["reduction"] == "none" else 4
    if case["grad"]:
        b += N * D * e + V * D * e + (V * 4 if case["bias"] else 0)
    return {"bytes": b, "flops": (6 if case["grad"] else 2) * N * D * V}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _words(seed, block, offset):
    """The generator's four 32-bit words of each block, in host integers (numpy uint64)."""
    import numpy as np
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x0, x1 = block & low, block >> half
    x2, x3 = np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        ka = np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF)
        kb = np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        pa, pb = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (pb >> half) ^ x1 ^ ka, pb & low, (pa >> half) ^ x3 ^ kb, pa & low
    return x0, x1, x2, x3


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.detach() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    if case["op"] == "embedding":
        V = case["V"]
        ids = s["ids"]
        # row V of the extended table is the zero row of ids outside the table
        slot = torch.where((ids < 0) | (ids >= V), V, ids)
        table = torch.cat([s["weight"].double() * s["scale"],
                           torch.zeros(1, case["D"], dtype=torch.float64, device="cuda")])
        out = table.index_select(0, slot)
        if not case["grad"]:
            return out
        del table
        d = torch.zeros(V + 1, case["D"], dtype=torch.float64, device="cuda")
        d.index_add_(0, slot, s["grad_out"].double())
        return out, d[:V] * s["scale"]
    if case["op"] == "dropout":
        import numpy as np
        n = case["N"] * case["D"]
        drop = math.floor(case["p"] * 65536 + 0.5)
        seed64, off64 = (int(v) & 0xFFFFFFFFFFFFFFFF for v in s["rng"].tolist())
        words = _words(seed64, np.arange(-(-n // 8), dtype=np.uint64), off64)
        bits = np.stack(words, axis=1).astype("<u4").view("<u2").reshape(-1)[:n]
        keep = torch.from_numpy((bits.astype(np.int32) >= drop)).cuda().view(case["N"], case["D"])
        q = 65536 / (65536 - drop)
        return tuple((v.double() * q).masked_fill(~keep, 0.0) for v in (s["x"], s["grad_out"]))
    if case["op"] == "layer_norm":
        x, w, b = (s[k].double().requires_grad_(True) for k in ("x", "weight", "bias"))
        var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + _EPS) * w + b
        if not case["grad"]:
            return y.detach()
        return (y.detach(),) + torch.autograd.grad(y, [x, w, b], s["grad_out"].double())
    N, D, V = case["N"], case["D"], case["V"]
    w = s["weight"].double()
    t = s["targets"]
    valid = (t >= 0) & (t < V)
    n_valid = max(int(valid.sum()), 1)
    losses = torch.zeros(N, dtype=torch.float64, device="cuda")
    gh = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    gw = torch.zeros(V, D, dtype=torch.float64, device="cuda") if case["grad"] else None
    gb = torch.zeros(V, dtype=torch.float64, device="cuda")
    rows = torch.nonzero(valid)[:, 0]
    for part in rows.split(1024):
        h = s["hidden"][part].double()
        z = h @ w.T
        if s["bias"] is not None:
            z = z + s["bias"].double()
        logp = torch.log_softmax(z, dim=1)
        lse = (z[:, 0] - logp[:, 0])
        goal = torch.full_like(z, case["smoothing"] / V)
        goal[torch.arange(len(part), device="cuda"), t[part]] += 1.0 - case["smoothing"]
        losses[part] = -(goal * logp).sum(dim=1) + case["z_loss"] * lse ** 2
        if not case["grad"]:
            continue
        d = logp.exp() * (1.0 + 2.0 * case["z_loss"] * lse[:, None]) - goal
        if case["reduction"] == "none":
            d = d * s["grad_out"][part].double()[:, None]
        elif case["reduction"] == "mean":
            d = d / n_valid
        gh[part] = d @ w
        gw += d.T @ h
        gb += d.sum(dim=0)
    total = {"none": losses, "sum": losses.sum(), "mean": losses.sum() / n_valid}
    loss = total[case["reduction"]]
    if not case["grad"]:
        return loss
    return (loss, gh, gw) + ((gb,) if case["bias"] else ())
