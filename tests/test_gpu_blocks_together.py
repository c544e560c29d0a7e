"""The operators of a model's blocks run together with those around them, as a training step uses
them: scaled embedding, norms in front of and behind each gated feed-forward block with its gate
and residual scale, the head's loss, and the AdamW step over all tensors; against the same step in
64 bits, captured in a graph with its own counters, on another stream, and decoding row by row."""
import math

import pytest
import torch
from torch.autograd import forward_ad

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24
LAYERS, SCALE = 2, 0.7


def model(dtype, D=96, F=130, V=777, seed=0):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, std, mean=0.0):
        return (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda().requires_grad_(True)
    p = dict(table=t(V, D, std=0.3), first=t(D, std=0.1, mean=1.0), head=t(V, D, std=1 / math.sqrt(D)))
    for k in range(LAYERS):
        p[f"wg{k}"], p[f"wu{k}"] = t(F, D, std=1 / math.sqrt(D)), t(F, D, std=1 / math.sqrt(D))
        p[f"wd{k}"] = t(D, F, std=1 / math.sqrt(F))
        p[f"post{k}"], p[f"next{k}"] = t(D, std=0.1, mean=1.0), t(D, std=0.1, mean=1.0)
        p[f"gate{k}"] = t(D, std=0.2, mean=0.6)
    return p


def batch(B=3, S=41, V=777, seed=0):
    g = torch.Generator().manual_seed(100 + seed)
    ids = torch.randint(0, V, (B, S), generator=g)
    ids[:, S - 5:] = -1                       # padding at the end of every sequence
    targets = torch.roll(ids, -1, 1)
    targets[:, -6:] = -100
    return ids.cuda(), targets.cuda()


def loss_of(m, p, ids, targets):
    x = m.embedding(p["table"], ids)
    n = m.rms_norm(x, p["first"])
    for k in range(LAYERS):
        h = m.gated_linear(n, p[f"wg{k}"], p[f"wu{k}"], activation="silu" if k else "gelu")
        # a 2-D product: a batched one has a transposed operand in its backward
        y = (h.reshape(-1, h.shape[-1]) @ p[f"wd{k}"].t()).view(x.shape)
        x, n = m.residual_rms_norm(x, y, p[f"next{k}"], post_weight=p[f"post{k}"],
                                   gate=p[f"gate{k}"], scale=SCALE)
    return m.linear_cross_entropy(n, p["head"], targets, z_loss=1e-3)


def loss64(p, ids, targets):
    V, D = p["table"].shape

    def rms(v, w):
        return v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w
    ok = (ids >= 0) & (ids < V)
    x = torch.where(ok[..., None], p["table"][ids.clamp(0, V - 1)], 0.0).view(-1, D)
    n = rms(x, p["first"])
    for k in range(LAYERS):
        z = n @ p[f"wg{k}"].T
        a = torch.nn.functional.silu(z) if k else torch.nn.functional.gelu(z)
        y = (a * (n @ p[f"wu{k}"].T)) @ p[f"wd{k}"].T
        x = x + SCALE * p[f"gate{k}"] * rms(y, p[f"post{k}"])
        n = rms(x, p[f"next{k}"])
    z = n @ p["head"].T
    lse = torch.logsumexp(z, 1)
    t = targets.view(-1)
    valid = (t >= 0) & (t < V)
    rows = lse - z.gather(1, t.clamp(0, V - 1)[:, None])[:, 0] + 1e-3 * lse ** 2
    return torch.where(valid, rows, 0.0).sum() / valid.sum()


# Relative 2-norm of a gradient's error: some 16 operators in a row (8 of each pass), each rounding
# its operands or results a few times (three half steps at most: dz, its result, the stream) and
# passing on what it got with a gain near one.  fp32's sums of up to 260 terms add 130 U each.
BOUND = {F32: 16 * 140 * U, BF16: 16 * 3 * 2.0 ** -9, F16: 16 * 3 * 2.0 ** -12}


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_step_against_64_bits(dtype):
    m = flp()
    p = model(dtype)
    ids, targets = batch()
    loss = loss_of(m, p, ids, targets)
    grads = torch.autograd.grad(loss, list(p.values()))
    q = {k: v.detach().double().requires_grad_(True) for k, v in p.items()}
    ref = loss64(q, ids, targets)
    want = torch.autograd.grad(ref, list(q.values()))
    assert abs(float(loss) - float(ref)) <= BOUND[dtype] * float(ref)
    for k, g, w in zip(p, grads, want):
        off = float((g.double() - w).norm() / w.norm())
        say(f"  {k}: {off:.2e} of {BOUND[dtype]:.2e}")
        assert off <= BOUND[dtype], (k, off)


def test_padding_rows_have_no_part():
    """What a padded position holds changes no gradient: an id outside the table reads as zeros and
    its target counts for nothing."""
    m = flp()
    p = model(BF16)
    ids, targets = batch()
    ref = torch.autograd.grad(loss_of(m, p, ids, targets), list(p.values()))
    other = torch.where(ids < 0, torch.full_like(ids, 10 ** 6), ids)
    got = torch.autograd.grad(loss_of(m, p, other, targets), list(p.values()))
    for k, a, b in zip(p, ref, got):
        assert torch.equal(a, b), k


def optimizer(m, p, bits, master):
    leaves = list(p.values())
    decay = [0.1 if t.dim() == 2 else 0.0 for t in leaves]
    return leaves, decay, m.adamw_state(leaves, bits=bits, master=master)


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps(bits):
    """Several whole steps: gradients of the changed parameters are those of a fresh model with the
    same values, and every parameter is finite and moved."""
    m = flp()
    p = model(BF16)
    leaves, decay, state = optimizer(m, p, bits, True)
    for t in (1, 2, 3):
        ids, targets = batch(seed=t)
        grads = torch.autograd.grad(loss_of(m, p, ids, targets), leaves)
        fresh = {k: v.detach().clone().requires_grad_(True) for k, v in p.items()}
        again = torch.autograd.grad(loss_of(m, fresh, ids, targets), list(fresh.values()))
        for k, a, b in zip(p, grads, again):
            assert torch.equal(a, b), (t, k)
        m.adamw_step(leaves, grads, state, t, 1e-2, weight_decay=decay)
        for k, v in p.items():
            assert bool(v.isfinite().all()), k
            assert not torch.equal(v, fresh[k]), k


def test_captured_training_steps():
    """Forward, backward and optimizer captured once; each replay takes its own batch, step number
    and rate, and gives the bits of eager steps."""
    m = flp()
    pa, pb = model(BF16), model(BF16)
    (la, da, sa), (lb, db, sb) = optimizer(m, pa, 8, True), optimizer(m, pb, 8, True)
    ids, targets = batch()
    t, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-2, device="cuda")

    def step(p, leaves, decay, state, i, j):
        loss = loss_of(m, p, i, j)
        m.adamw_step(leaves, torch.autograd.grad(loss, leaves), state, t, lr, weight_decay=decay)
        return loss.detach()
    warm = model(BF16, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the libraries' first calls
        lw, dw, sw = optimizer(m, warm, 8, True)
        step(warm, lw, dw, sw, ids, targets)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step(pa, la, da, sa, ids, targets)
    for k in range(1, 5):
        i, j = batch(seed=k)
        ids.copy_(i), targets.copy_(j), t.fill_(k), lr.fill_(1e-2 / k)
        graph.replay()
        torch.cuda.synchronize()
        kept = loss.clone()
        assert torch.equal(kept, step(pb, lb, db, sb, i, j)), k
        torch.cuda.synchronize()
        for name in pa:
            assert torch.equal(pa[name], pb[name]), (k, name)
        for f, h in zip(sa, sb):
            for x, y in zip(f, h):
                assert x is y is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_another_stream():
    m = flp()
    pa, pb = model(F32), model(F32)
    ids, targets = batch()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000)
        grads = torch.autograd.grad(loss_of(m, pa, ids, targets), list(pa.values()))
        la, da, sa = optimizer(m, pa, 32, False)
        m.adamw_step(la, grads, sa, 1, 1e-2, weight_decay=da)
    lb, db, sb = optimizer(m, pb, 32, False)
    m.adamw_step(lb, torch.autograd.grad(loss_of(m, pb, ids, targets), lb), sb, 1, 1e-2,
                 weight_decay=db)
    torch.cuda.current_stream().wait_stream(side)
    for k in pa:
        assert torch.equal(pa[k], pb[k]), k


def test_two_streams_at_once():
    """Two models' blocks interleaved on two streams, each with its own workspaces."""
    m = flp()
    ps = [model(BF16, seed=k) for k in range(2)]
    ids, targets = batch()
    ref = [torch.autograd.grad(loss_of(m, p, ids, targets), list(p.values())) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for turn in range(3):
        got = []
        for s, p in zip(streams, ps):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(torch.autograd.grad(loss_of(m, p, ids, targets), list(p.values())))
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y), turn


def test_decoding_a_row_at_a_time():
    """The serving form: blocks without gradients, one row at a time, have the bits of the batch."""
    m = flp()
    p = model(BF16, D=256, F=700)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(9, 256, generator=g).to(BF16).cuda()
    y = torch.randn(9, 256, generator=g).to(BF16).cuda()

    def block(x, y):
        r, n = m.residual_rms_norm(x, y, p["next0"], post_weight=p["post0"], gate=p["gate0"],
                                   scale=SCALE)
        return r, m.gated_linear(n, p["wg0"], p["wu0"])
    with torch.no_grad():
        whole = block(x, y)
        for i in range(9):
            one = block(x[i:i + 1].contiguous(), y[i:i + 1].contiguous())
            for a, b in zip(one, whole):
                assert torch.equal(a[0], b[i]), i


def test_backward_twice_and_forward_mode():
    """A retained graph gives the same gradients again; forward-mode differentiation is refused."""
    m = flp()
    p = model(F32)
    ids, targets = batch()
    x = torch.randn(20, 96, device="cuda", requires_grad=True)
    y = torch.randn(20, 96, device="cuda", requires_grad=True)
    r, n = m.residual_rms_norm(x, y, p["next0"], gate=p["gate0"])
    out = m.gated_linear(n, p["wg0"], p["wu0"])
    leaves = [x, y, p["next0"], p["gate0"], p["wg0"], p["wu0"]]
    one = torch.autograd.grad(out.sum() + r.sum(), leaves, retain_graph=True)
    two = torch.autograd.grad(out.sum() + r.sum(), leaves)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    with forward_ad.dual_level():
        for leaf in (x, x.detach()):
            dual = forward_ad.make_dual(leaf.detach() if leaf is not x else leaf, torch.ones_like(leaf))
            for call in (lambda: m.rms_norm(dual, p["next0"]),
                         lambda: m.residual_rms_norm(dual, y, p["next0"]),
                         lambda: m.gated_linear(dual, p["wg0"], p["wu0"])):
                with pytest.raises((NotImplementedError, RuntimeError)):
                    call()
