"""The operators around a model's body run together, as a training step of a small language model
uses them: scaled embedding, dropout, a body (one linear layer with a residual), the final layer
norm and the linear cross entropy; forward and gradients against the same step in 64 bits, and
the step captured in a graph."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu


def step_inputs(dtype, B=3, S=41, D=96, V=777, seed=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (B, S), generator=g)
    ids[:, S - 5:] = -1                       # padding at the end of every sequence
    targets = torch.roll(ids, -1, 1)
    targets[:, -6:] = -100
    p = dict(table=torch.randn(V, D, generator=g) * 0.05,
             mix=torch.randn(D, D, generator=g) / math.sqrt(D),
             w=1 + 0.1 * torch.randn(D, generator=g), b=0.1 * torch.randn(D, generator=g),
             head=torch.randn(V, D, generator=g) * 0.05)
    p = {k: v.to(dtype).cuda().requires_grad_(True) for k, v in p.items()}
    rng = torch.tensor([1234, 7], device="cuda")
    return ids.cuda(), targets.cuda(), p, rng


def step(m, ids, targets, p, rng, scale):
    x = m.embedding(p["table"], ids, scale=scale)
    x = m.dropout(x, 0.1, rng)
    x = x + x @ p["mix"]
    x = m.layer_norm(x, p["w"], p["b"])
    return m.linear_cross_entropy(x, p["head"], targets, label_smoothing=0.1, z_loss=1e-3)


def step64(ids, targets, p, keep, scale):
    D = p["mix"].shape[0]
    p = {k: v.detach().double().requires_grad_(True) for k, v in p.items()}
    V = p["table"].shape[0]
    ok = (ids >= 0) & (ids < V)
    x = torch.where(ok[..., None], p["table"][ids.clamp(0, V - 1)] * scale, 0.0)
    q = round(0.1 * 65536) / 65536
    x = torch.where(keep.view(x.shape), x / (1 - q), 0.0)
    x = x + (x.view(-1, D) @ p["mix"]).view(x.shape)
    mean = x.mean(-1, keepdim=True)
    x = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + 1e-5) * p["w"] + p["b"]
    z = x.view(-1, D) @ p["head"].t()
    lse = torch.logsumexp(z, 1)
    t = targets.view(-1)
    valid = (t >= 0) & (t < V)
    zt = z.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
    rows = 0.9 * (lse - zt) + 0.1 * (lse - z.mean(1)) + 1e-3 * lse ** 2
    loss = torch.where(valid, rows, 0.0).sum() / valid.sum()
    names = list(p)
    return loss, dict(zip(names, torch.autograd.grad(loss, [p[n] for n in names])))


# Relative 2-norm of the difference.  fp32: about a hundred fp32 roundings in a row, each below
# 2^-24 and far from aligned: 2^-17.  bf16: the five tensors between the operators, the
# parameters' products and the gradients are each rounded to 2^-8 half steps, about twelve
# roundings between the loss and the table's gradient: sqrt(12) 2^-9 rms, doubled.
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2.0 ** -17),
                                       (torch.bfloat16, 2 * math.sqrt(12) * 2.0 ** -9)])
def test_training_step(dtype, tol):
    m = flp()
    ids, targets, p, rng = step_inputs(dtype)
    scale = math.sqrt(96)
    loss = step(m, ids, targets, p, rng, scale)
    loss.backward()
    n = ids.numel() * 96
    keep = m.dropout(torch.ones(n, device="cuda"), 0.1, rng) != 0
    ref, grads = step64(ids, targets, p, keep, scale)
    loss, ref = float(loss.detach()), float(ref.detach())
    say(f"loss {loss} against {ref}")
    assert abs(loss - ref) <= tol * abs(ref)
    for k, v in p.items():
        rel = float((v.grad.double() - grads[k]).norm() / grads[k].norm())
        say(f"  {k}: {rel:.2e} (bound {tol:.2e})")
        assert rel <= tol


def test_padding_reaches_no_gradient():
    """The table row that only padded positions would touch, and any content of the rows of
    padded targets, leave the gradients alone."""
    m = flp()
    ids, targets, p, rng = step_inputs(torch.float32)
    loss = step(m, ids, targets, p, rng, 2.0)
    g = torch.autograd.grad(loss, list(p.values()))
    changed = ids.clone()
    changed[targets < 0] = 5                  # other tokens where nothing is counted
    loss2 = step(m, changed, targets, p, rng, 2.0)
    g2 = torch.autograd.grad(loss2, list(p.values()))
    assert torch.equal(loss, loss2)
    assert torch.equal(g[-1], g2[-1])         # the head


def test_step_in_a_graph():
    """The operators' forward and backward calls of one step, captured once and replayed with new
    ids, targets and dropout offsets between the program's own work: every replay equals the
    eager calls bit for bit."""
    m = flp()
    ids, targets, p, rng = step_inputs(torch.bfloat16)
    p = {k: v.detach() for k, v in p.items()}
    one = torch.ones((), device="cuda")
    V = p["table"].shape[0]

    def calls():
        x0 = m.embedding_forward(p["table"], ids, 4.0)
        x1 = m.dropout_forward(x0, 0.1, rng)
        x2, mean, rstd = m.layer_norm_forward(x1, p["w"], p["b"])
        loss, stats = m.cross_entropy_forward(x2, p["head"], targets, None, 0.1, 1e-3)
        d2, dhead, _ = m.cross_entropy_backward(one, stats, x2, p["head"], targets, None, 0.1,
                                                1e-3)
        d1, dw, db = m.layer_norm_backward(d2, x1, mean, rstd, p["w"])
        d0 = m.dropout_forward(d1, 0.1, rng)
        return loss, dhead, dw, db, m.embedding_backward(d0, ids, V, scale=4.0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for rep in range(4):
        nids, ntargets, _, _ = step_inputs(torch.bfloat16, seed=10 + rep)
        ids.copy_(nids)
        targets.copy_(ntargets)
        rng[1] = rep
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, calls()):
            assert torch.equal(a, b), rep


def autograd_step(p, ids, targets, rng):
    """Loss and gradients of one step, on leaves of its own."""
    m = flp()
    leaf = {k: v.detach().requires_grad_() for k, v in p.items() if k != "mix"}
    x = m.dropout(m.embedding(leaf["table"], ids, 4.0), 0.1, rng)
    loss = m.linear_cross_entropy(m.layer_norm(x, leaf["w"], leaf["b"]), leaf["head"], targets,
                                  None, 0.1, 1e-3)
    names = sorted(leaf)
    return (loss.detach(),) + torch.autograd.grad(loss, [leaf[k] for k in names])


def test_autograd_step_in_a_graph():
    """The same through autograd, whose backward runs on a thread of its own: captured once,
    replayed with new inputs between eager steps, the same bits."""
    ids, targets, p, rng = step_inputs(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        autograd_step(p, ids, targets, rng)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = autograd_step(p, ids, targets, rng)
    for rep in range(4):
        nids, ntargets, _, _ = step_inputs(torch.bfloat16, seed=30 + rep)
        ids.copy_(nids)
        targets.copy_(ntargets)
        rng[1] = rep
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, autograd_step(p, ids, targets, rng)):
            assert torch.equal(a, b), rep


def test_autograd_steps_on_two_streams():
    """Two steps, each on a stream of its own: forward and backward stay on it."""
    steps = [step_inputs(torch.bfloat16, seed=50 + k) for k in range(2)]
    want = [autograd_step(p, ids, t, rng) for ids, t, p, rng in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        got = []
        for (ids, t, p, rng), s in zip(steps, streams):
            with torch.cuda.stream(s):
                got.append(autograd_step(p, ids, t, rng))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_forward_mode_differentiation_is_refused():
    """An input with a tangent: an error, where a plain call would give an output without one;
    inside a dual level without tangents nothing changes."""
    from torch.autograd import forward_ad
    m = flp()
    ids, targets, p, rng = step_inputs(torch.float32)
    x = torch.randn(targets.numel(), p["head"].shape[1], device="cuda")
    t = targets.reshape(-1)
    calls = [(lambda w: m.embedding(w, ids), p["table"].detach()),
             (lambda x: m.dropout(x, 0.1, rng), x),
             (lambda x: m.layer_norm(x, p["w"].detach(), p["b"].detach()), x),
             (lambda x: m.linear_cross_entropy(x, p["head"].detach(), t), x)]
    want = [f(v) for f, v in calls]
    with forward_ad.dual_level():
        for (f, v), y in zip(calls, want):
            assert torch.equal(f(v), y)
            with pytest.raises(NotImplementedError):
                f(forward_ad.make_dual(v, torch.ones_like(v)))
            with pytest.raises(NotImplementedError):
                f(forward_ad.make_dual(v.clone().requires_grad_(), torch.ones_like(v)))


@pytest.mark.parametrize("up", [None, "constant", "differentiable"])
@pytest.mark.parametrize("op", ["layer_norm", "cross_entropy", "cross_entropy_at_once"])
def test_a_penalty_on_a_first_gradient_is_refused(op, up):
    """The first gradients of layer norm and of the loss depend on their inputs: a term made of
    them cannot be differentiated, and says so beside other terms that can."""
    from lm_head_selected_bf16_amd import torch_ops
    m = flp()
    g = torch.Generator().manual_seed(5)
    x = torch.randn(12, 64, generator=g).cuda().requires_grad_()
    w = torch.randn(90, 64, generator=g).cuda().requires_grad_()
    b = torch.randn(90, generator=g).cuda().requires_grad_()
    t = torch.arange(12, device="cuda")
    if op == "layer_norm":
        w, b = (v[0:1].expand(64).detach().clone().requires_grad_() for v in (w[0, :1], b))
        out = m.layer_norm(x, w, b)
    elif op == "cross_entropy":
        out = m.linear_cross_entropy(x, w, t, b)
    else:
        out = torch_ops.LossAndGradients.apply(x, w, t, b, 0.0, 0.0, "mean")
    seed = None if up is None and out.dim() == 0 else torch.ones_like(out)
    if up == "differentiable":
        seed = seed if seed is not None else torch.ones_like(out)
        seed.requires_grad_()
    first = torch.autograd.grad(out, [x, w, b], seed, create_graph=True)
    # d_bias of the norm is a sum of the upstream gradient alone
    depends = [True, True, op != "layer_norm" or up == "differentiable"]
    for d, dep in zip(first, depends):
        assert d.requires_grad == dep
        if dep:
            with pytest.raises(RuntimeError, match="differentiate twice"):
                (out.sum() + d.pow(2).sum()).backward(retain_graph=True)
    for v, d in zip((x, w, b), first):
        v.grad = None
    again = torch.autograd.grad(out, [x, w, b], None if seed is None else seed.detach())
    for a, d in zip(again, first):
        assert not a.requires_grad and torch.equal(a, d)


def test_a_penalty_on_the_gradient_of_a_linear_operator():
    """Dropout's and the embedding's gradients do not depend on their inputs: with a constant
    upstream gradient they are constants."""
    m = flp()
    ids, _, p, rng = step_inputs(torch.float32)
    x = torch.randn(3, 64, device="cuda", requires_grad=True)
    for out, leaf in ((m.dropout(x, 0.1, rng), x), (m.embedding(p["table"], ids, 2.0), p["table"])):
        (d,) = torch.autograd.grad(out, [leaf], torch.ones_like(out), create_graph=True)
        assert not d.requires_grad
        (out.sum() + d.pow(2).sum()).backward()
        assert torch.equal(leaf.grad, d)
        out = m.dropout(x, 0.1, rng)
    up = torch.ones(*ids.shape, 96, device="cuda", requires_grad=True)
    (d,) = torch.autograd.grad(m.embedding(p["table"], ids, 2.0), [p["table"]], up,
                               create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        d.sum().backward()


@pytest.mark.parametrize("how", ["grad", "backward"])
def test_a_status_inside_a_backward_is_the_librarys_error(how):
    """Data exchanged for a view off the 16-byte grid between forward and backward: the library
    refuses it inside autograd's engine, and the error keeps its type and status.  The next step
    is not touched by it."""
    m = flp()
    g = torch.Generator().manual_seed(6)
    w = torch.randn(90, 64, generator=g).cuda()
    t = torch.arange(12, device="cuda")
    x = torch.randn(12, 64, generator=g).cuda().requires_grad_()
    loss = m.linear_cross_entropy(x, w, t)
    (want,) = torch.autograd.grad(loss, [x], retain_graph=True)
    kept = x.data
    x.data = torch.cat([kept.flatten()[:1], kept.flatten()])[1:].view(12, 64)
    with pytest.raises(m.FlpError, match="flp_cross_entropy_backward failed: FLP_MISALIGNED") as e:
        loss.backward() if how == "backward" else torch.autograd.grad(loss, [x])
    assert e.value.status == 4
    x.data = kept
    assert torch.equal(torch.autograd.grad(m.linear_cross_entropy(x, w, t), [x])[0], want)
    with pytest.raises(m.FlpError, match="flp_layer_norm_forward failed: FLP_INVALID_ARGUMENT"):
        m.layer_norm(x, eps=-1.0)
