"""Layer norm against its definition in 64 bits: widths from one element to rows wider than a
workgroup holds, rows off the 16-byte grid, every type and parameter combination, the gradients
against the formula and against differences, determinism, streams and graphs."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative


def rounding(t, ref):
    """Half a step of the type at ref: relative for normal values, and the constant
    smallest_normal * eps / 2 below the smallest normal one (fp16 steps there are 2^-24, which
    an entry of 4e-5 cannot meet relatively)."""
    f = torch.finfo(t)
    return (f.eps / 2) * ref.abs().clamp(min=f.smallest_normal)


def make(N, D, dtype, wdtype, seed, offset=0.5, weight=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, D, generator=g) * (torch.rand(N, 1, generator=g) * 3 + 0.2)
         + offset).to(dtype)
    w = (torch.randn(D, generator=g) * 0.3 + 1).to(wdtype) if weight else None
    b = (torch.randn(D, generator=g) * 0.3).to(wdtype) if bias else None
    go = torch.randn(N, D, generator=g).to(dtype)
    return tuple(None if t is None else t.cuda() for t in (x, w, b, go))


def reference(x, w, b, go, eps):
    x, go = x.double(), go.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = (x - mean) * rstd
    y = xhat * w + (0 if b is None else b.double())
    g = go * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return dict(y=y, mean=mean[..., 0], rstd=rstd[..., 0], xhat=xhat, dx=dx, g=g,
                dw=(go * xhat).sum(0), db=go.sum(0))


def row_error(x, r):
    """Bound on the fp32 error of a row's xhat: a sum of D terms in chains of at most D / 256
    plus a tree of depth below 32 is off by at most (D / 256 + 32) U times the sum of the terms'
    sizes; the mean's error enters xhat times rstd, the variance's (relative) by half."""
    D = x.shape[-1]
    k = (D / 256 + 32) * U
    mean_abs = x.double().abs().mean(-1, keepdim=True)
    rstd = r["rstd"][:, None]
    e_mean = k * mean_abs * rstd          # of (mean) * rstd
    # the centred values are rounded once (U |c|) and carry the mean's error
    e_rstd = k + 4 * U + 2 * e_mean       # relative, of rstd
    return e_mean + r["xhat"].abs() * (e_rstd + 4 * U)


def check(name, got, ref, tol):
    err = (got.double() - ref).abs()
    worst = float((err / tol).max()) if err.numel() else 0.0
    say(f"  {name}: worst error {worst:.3f} of its bound")
    assert bool((err <= tol).all()), (name, worst)


def compare(x, w, b, go, eps=1e-5):
    m = flp()
    y, mean, rstd = m.layer_norm_forward(x, w, b, eps)
    dx, dw, db = m.layer_norm_backward(go, x, mean, rstd, w,
                                       w_dtype=None if b is None else b.dtype)
    r = reference(x, w, b, go, eps)
    N, D = x.shape
    ex = row_error(x, r)
    wa = 1.0 if w is None else w.double().abs()
    check("out", y, r["y"], rounding(x.dtype, r["y"]) + ex * wa + 4 * U * r["y"].abs()
          + 4 * U * (r["xhat"] * wa).abs())
    # d_x: the two means over D of g and g xhat, and xhat's own error
    k = (D / 256 + 32) * U
    g, xh, rs = r["g"].abs(), r["xhat"].abs(), r["rstd"][:, None]
    m1, m2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    e2 = (k + 8 * U) * m2 + (g * ex).mean(-1, keepdim=True)
    tol = rs * ((k + 4 * U) * m1 + 8 * U * g + xh * e2 + ex * m2 + 8 * U * xh * m2)
    rel = 4 * U + k + 2 * k * x.double().abs().mean(-1, keepdim=True) * rs  # of rstd
    check("d_x", dx, r["dx"], rounding(x.dtype, r["dx"]) * (1 + 2 ** -6) + 2 * tol
          + 2 * rel * rs * (g + m1 + xh * m2))
    # a sum of N terms in chains of at most N / 256 + 8 rows (or 256 slabs), then trees
    n = (N + 64) * U
    go64 = go.double().abs()
    wt = dw.dtype
    check("d_weight", dw, r["dw"], rounding(wt, r["dw"]) + n * (go64 * xh).sum(0)
          + (go64 * ex).sum(0) + 4 * U * (go64 * xh).sum(0))
    check("d_bias", db, r["db"], rounding(wt, r["db"]) + n * go64.sum(0))
    return y, mean, rstd, dx, dw, db


WIDTHS = [1, 2, 7, 8, 64, 129, 520, 1000, 1345, 2688, 4096, 4097, 8200, 12288, 12289, 16384, 16385, 40001]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32),
                                          (F32, F32)])
def test_widths(D, dtype, wdtype):
    for N in (1, 37):
        say(f"N={N} D={D} {dtype} {wdtype}")
        compare(*make(N, D, dtype, wdtype, 7 * D + N))


@pytest.mark.parametrize("N", [1, 7, 8, 9, 255, 256, 257, 2049, 5000, 20011])
def test_row_counts(N):
    for D, dtype in ((24, BF16), (777, F32), (2688, BF16)):
        say(f"N={N} D={D} {dtype}")
        compare(*make(N, D, dtype, dtype, N + D))


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_optional_parameters(weight, bias):
    compare(*make(33, 1000, BF16, BF16, 3, weight=weight, bias=bias))
    x, w, b, go = make(33, 1000, F16, F32, 4, weight=weight, bias=bias)
    m = flp()
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b) if t is not None]
    it = iter(leaves)
    args = [next(it) if t is not None else None for t in (x, w, b)]
    y = m.layer_norm(*args)
    grads = torch.autograd.grad(y, leaves, go)
    y2, mean, rstd = m.layer_norm_forward(x, w, b)
    ref = m.layer_norm_backward(go, x, mean, rstd, w, w_dtype=F32)
    keep = [True, weight, bias]
    assert torch.equal(y, y2)
    for got, want in zip(grads, [t for t, k in zip(ref, keep) if k]):
        assert torch.equal(got, want)


def test_only_what_is_asked_for():
    x, w, b, go = make(300, 1345, BF16, F32, 5)
    m = flp()
    y, mean, rstd = m.layer_norm_forward(x, w, b)
    full = m.layer_norm_backward(go, x, mean, rstd, w)
    for need in ((True, False, False), (False, True, False), (False, False, True),
                 (False, True, True), (True, True, False)):
        part = m.layer_norm_backward(go, x, mean, rstd, w, *need)
        for k in range(3):
            assert (part[k] is None) == (not need[k])
            assert part[k] is None or torch.equal(part[k], full[k])


def test_large_offsets_and_scales():
    """Rows whose mean is far larger than their spread, tiny rows (eps decides) and large ones:
    the variance comes from centred values."""
    x, w, b, go = make(64, 2688, F32, F32, 6)
    x[:16] = x[:16] + 1000.0
    x[16:32] = x[16:32] * 1e-6
    x[32:48] = x[32:48] * 1e8
    compare(x, w, b, go)


def test_degenerate_rows():
    """A constant row is its bias (eps > 0); an infinite or NaN row is NaN and touches no other
    row; eps = 0 leaves ordinary rows alone; D = 1 has no spread at all."""
    m = flp()
    x, w, b, go = make(40, 1000, F32, F32, 8)
    x[3] = 2.0
    clean = m.layer_norm(x, w, b)
    assert torch.equal(clean[3], b)
    bad = x.clone()
    bad[5, 17] = float("inf")
    bad[9, 0] = float("nan")
    y = m.layer_norm(bad, w, b)
    assert y[5].isnan().all() and y[9].isnan().all()
    keep = [i for i in range(40) if i not in (5, 9)]
    assert torch.equal(y[keep], clean[keep])
    rows = [i for i in range(40) if i != 3]
    compare(x[rows].contiguous(), w, b, go[rows].contiguous(), eps=0.0)
    one = torch.full((5, 1), 3.0, device="cuda")
    assert torch.equal(m.layer_norm(one, w[:1], b[:1]), b[:1].expand(5, 1))


@pytest.mark.parametrize("D", [1, 7, 520, 1000, 1345, 2000, 2688, 5000, 12000, 16385, 20000])
@pytest.mark.parametrize("dtype,values", [(BF16, (3.0, 4080.0, -0.0996)), (F16, (3.0, 2047.0, -6e4)),
                                          (F32, (3.0, 4080.3, -0.1, 1e30))])
def test_constant_rows_are_their_bias(D, dtype, values):
    """Whatever the value: the mean is the value itself and nothing is left of the row.  rstd is
    that of the variance 0, which the first mean's error e <= k |x| enters only through the
    rounding of e^2 - e^2 (at most 4 U e^2)."""
    m = flp()
    x = torch.tensor(values, device="cuda").to(dtype)[:, None].expand(-1, D).contiguous()
    _, w, b, _ = make(1, D, dtype, dtype, 14)
    y, mean, rstd = m.layer_norm_forward(x, w, b)
    assert torch.equal(y, b.expand_as(y))
    assert torch.equal(mean, x[:, 0].float())
    e = (D / 256 + 32) * U * x[:, 0].double().abs()
    rel = (rstd.double() * math.sqrt(1e-5) - 1).abs()
    ok = e < 1e15  # beyond, e^2 passes fp32
    assert bool((rel <= 4 * U + 2 * U * e ** 2 / 1e-5)[ok].all())


@pytest.mark.parametrize("D", [520, 1000, 2688, 6000, 20000])
def test_mean_of_rows_far_from_zero(D):
    """Rows whose spread is a small part of their offset.  The first mean is off by k |x|, with
    k the error of a sum as above; the values centred by it are rounded once, their mean is off by
    k + 4 U of their mean size, and the corrected mean is rounded to half a step."""
    m = flp()
    g = torch.Generator().manual_seed(15)
    x = torch.randn(16, D, generator=g)
    x = (x * torch.logspace(-3, 1, 16)[:, None] + torch.logspace(1, 5, 16)[:, None]).cuda()
    y, mean, rstd = m.layer_norm_forward(x)
    ref = x.double().mean(1)
    c = (x.double() - ref[:, None]).abs().mean(1)
    k = (D / 256 + 32) * U
    off = k * x.double().abs().mean(1)
    check("mean", mean, ref, 1.01 * U * ref.abs() + (k + 5 * U) * (c + off))


@pytest.mark.parametrize("D", [64, 777, 3000, 9000, 12289])
@pytest.mark.parametrize("k", [-62, 55])
def test_scale_of_the_rows(D, k):
    """Without eps the norm does not depend on the rows' scale, and a power of two changes no
    rounding: with x times 2^k and grad_out times 2^-30, out has the same bits, d_weight and
    d_bias those times 2^-30 and d_x those times 2^(-30 - k)."""
    m = flp()
    g = torch.Generator().manual_seed(16)
    x = (torch.randn(9, D, generator=g) + 0.25).cuda()
    _, w, b, go = make(9, D, F32, F32, 17)
    y, mean, rstd = m.layer_norm_forward(x, w, b, 0.0)
    dx, dw, db = m.layer_norm_backward(go, x, mean, rstd, w)
    x2, go2 = x * 2.0 ** k, go * 2.0 ** -30
    y2, mean2, rstd2 = m.layer_norm_forward(x2, w, b, 0.0)
    dx2, dw2, db2 = m.layer_norm_backward(go2, x2, mean2, rstd2, w)
    assert torch.equal(y2, y) and torch.equal(rstd2 * 2.0 ** k, rstd)
    assert torch.equal(dx2.double() * 2.0 ** (30 + k), dx.double())
    assert torch.equal(dw2 * 2.0 ** 30, dw) and torch.equal(db2 * 2.0 ** 30, db)


@pytest.mark.parametrize("D", [64, 777, 3000, 9000, 12289])
def test_rows_whose_variance_is_subnormal(D):
    """A spread of 2^-65 and eps = 0: the variance 2^-130 is held to steps of 2^-149, so each
    square and their mean are off by half a step: 2^-19 of the variance, 2^-20 of rstd (times 2:
    a row's variance is above half its expectation).  1 / rstd^2 passes fp32, rstd does not."""
    m = flp()
    g = torch.Generator().manual_seed(18)
    x = torch.randn(9, D, generator=g).cuda()
    _, w, b, go = make(9, D, F32, F32, 19)
    y, mean, rstd = m.layer_norm_forward(x, w, b, 0.0)
    dx, dw, db = m.layer_norm_backward(go, x, mean, rstd, w)
    x2 = x * 2.0 ** -65
    y2, mean2, rstd2 = m.layer_norm_forward(x2, w, b, 0.0)
    dx2, dw2, db2 = m.layer_norm_backward(go, x2, mean2, rstd2, w)
    rel = 2.0 ** -19 + 8 * U
    r = reference(x, w, b, go, 0.0)
    # out = fma(xhat, w, b): each of the two is rounded by itself, off by U |out| from the sum
    check("out", y2, y.double(), rel * (r["xhat"] * w.double()).abs() + 2.1 * U * y.double().abs())
    gw, xh = r["g"].abs(), r["xhat"].abs()
    size = r["rstd"][:, None] * (gw + gw.mean(1, keepdim=True)
                                 + 3 * xh * (gw * xh).mean(1, keepdim=True))
    # each d_x is off by a rounding of each term and the sums' (k), with its own order of rows
    check("d_x", dx2.double() * 2.0 ** -65, dx.double(), (rel + 2 * (D / 256 + 40) * U) * size)
    # nine terms added in the same order
    check("d_weight", dw2, dw.double(), (rel + 20 * U) * (go.double().abs() * xh).sum(0))
    assert torch.equal(db2, db)


def test_empty_batch():
    m = flp()
    x = torch.empty(0, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    b = torch.ones(64, device="cuda", requires_grad=True)
    y = m.layer_norm(x, w, b)
    dx, dw, db = torch.autograd.grad(y, [x, w, b], torch.empty_like(y))
    assert y.shape == (0, 64) and dx.shape == (0, 64)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("D", [1345, 2688, 9000])
def test_rows_do_not_depend_on_each_other(D):
    m = flp()
    x, w, b, go = make(530, D, BF16, BF16, 9)
    y, mean, rstd = m.layer_norm_forward(x, w, b)
    dx, dw, db = m.layer_norm_backward(go, x, mean, rstd, w)
    again = m.layer_norm_backward(go, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    for lo, hi in ((0, 1), (529, 530), (100, 357)):
        s = slice(lo, hi)
        y1, m1, r1 = m.layer_norm_forward(x[s].contiguous(), w, b)
        d1, _, _ = m.layer_norm_backward(go[s].contiguous(), x[s].contiguous(), m1, r1, w)
        assert torch.equal(y1, y[s]) and torch.equal(m1, mean[s]) and torch.equal(r1, rstd[s])
        assert torch.equal(d1, dx[s])


def test_views_off_the_16_byte_grid():
    """A contiguous view that starts one element into its storage, and outputs that leave what
    lies behind the last row alone."""
    m = flp()
    for dtype in (BF16, F32):
        for D in (63, 64, 1344):
            x, w, b, go = make(9, D, dtype, dtype, 10)
            want = m.layer_norm_forward(x, w, b)
            shift = torch.empty(9 * D + 1, dtype=dtype, device="cuda")
            xs = shift[1:].view(9, D).copy_(x)
            out = torch.full((9 * D + 9,), 7.0, dtype=dtype, device="cuda")
            st = m.flp_layer_norm_forward(9, D, {BF16: m.FLP_BF16, F32: m.FLP_F32}[dtype],
                                          xs.data_ptr(), {BF16: m.FLP_BF16, F32: m.FLP_F32}[dtype],
                                          w.data_ptr(), b.data_ptr(), 1e-5,
                                          out.data_ptr() + out.element_size(), 0, 0,
                                          torch.cuda.current_stream().cuda_stream)
            assert st == m.FLP_OK
            assert torch.equal(out[1:9 * D + 1].view(9, D), want[0])
            assert out[0] == 7.0 and bool((out[9 * D + 1:] == 7.0).all())


def test_gradient_against_differences():
    m = flp()
    x, w, b, go = make(3, 12, F32, F32, 11)

    def loss(x, w, b):
        return float((m.layer_norm(x, w, b).double() * go.double()).sum())

    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    m.layer_norm(*leaves).backward(go)
    h = 2.0 ** -7
    for k, t in enumerate((x, w, b)):
        flat = t.view(-1)
        for e in range(0, flat.numel(), 5):
            old = float(flat[e])
            flat[e] = old + h
            up = loss(x, w, b)
            flat[e] = old - h
            down = loss(x, w, b)
            flat[e] = old
            # second-order error h^2 f''' / 6 with f''' below 100 here, and fp32 rounding of the
            # 36 outputs (each off by at most 8 U 8) over 2 h
            assert abs((up - down) / (2 * h) - float(leaves[k].grad.view(-1)[e])) < \
                100 * h * h / 6 + 36 * 64 * U / (2 * h)


def test_leading_shapes_and_other_stream():
    m = flp()
    x, w, b, go = make(24, 520, BF16, F32, 12)
    want = m.layer_norm(x, w, b)
    assert torch.equal(m.layer_norm(x.view(2, 3, 4, 520), w, b), want.view(2, 3, 4, 520))
    assert torch.equal(m.layer_norm(x[0], w, b), want[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = m.layer_norm(x, w, b)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_refusals():
    m = flp()
    x, w, b, go = make(8, 64, BF16, BF16, 13)
    with pytest.raises(ValueError):
        m.layer_norm(x.t())
    with pytest.raises(TypeError):
        m.layer_norm(x, w.half())
    with pytest.raises(TypeError):
        m.layer_norm(x, w, b.float())
    with pytest.raises(ValueError):
        m.layer_norm(x, w[:32])
    with pytest.raises(ValueError):
        m.layer_norm(x, w.cpu())
    with pytest.raises(m.FlpError):
        m.layer_norm(x, w, b, eps=-1.0)
    y, mean, rstd = m.layer_norm_forward(x, w, b)
    with pytest.raises(ValueError):
        m.layer_norm_backward(go[:4], x, mean, rstd, w)
    with pytest.raises(ValueError):
        m.layer_norm_backward(go, x, mean[:4], rstd, w)
    with pytest.raises(TypeError):
        m.layer_norm_backward(go, x, mean, rstd, w, w_dtype=F32)


@pytest.mark.parametrize("which", ["weight", "x", "device", "dtype"])
def test_data_exchanged_before_the_backward_is_refused(which):
    x, w, b, go = make(5, 96, F32, F32, seed=31)
    x, w, b = (t.requires_grad_() for t in (x, w, b))
    out = flp().layer_norm(x, w, b)
    if which == "weight":
        w.data = w.data[:48].clone()
    elif which == "x":
        x.data = x.data[:2].clone()
    elif which == "device":
        w.data = w.data.cpu()
    else:
        w.data = w.data.to(BF16)
    with pytest.raises((ValueError, TypeError)):
        torch.autograd.grad(out, [x], go)


@pytest.mark.parametrize("need", range(1, 8))
@pytest.mark.parametrize("weight,bias", [(True, True), (True, False), (False, True), (False, False)])
def test_autograd_gives_each_leaf_its_gradient(weight, bias, need):
    """Every combination of parameters that are there and of leaves that ask, with an upstream
    gradient that is a broadcast view, against the functional calls."""
    m = flp()
    x, w, b, go = make(37, 193, BF16, F32, 41, weight=weight, bias=bias)
    ask = [need & 1, need & 2 and w is not None, need & 4 and b is not None]
    if not any(ask):
        return
    _, mean, rstd = m.layer_norm_forward(x, w, b)
    up = go[:1].expand(37, 193)
    want = m.layer_norm_backward(up.contiguous(), x, mean, rstd, w, w_dtype=None if w is not None
                                 else F32 if b is not None else BF16)
    leaves = [None if t is None else t.clone().requires_grad_(bool(a))
              for t, a in zip((x, w, b), ask)]
    out = m.layer_norm(*leaves)
    asked = [t for t, a in zip(leaves, ask) if a]
    first = torch.autograd.grad(out, asked, up, retain_graph=True)
    again = torch.autograd.grad(out, asked, up)
    for f, a, v in zip(first, again, [v for v, a in zip(want, ask) if a]):
        assert torch.equal(f, v) and torch.equal(a, v)
    with pytest.raises(RuntimeError):  # the graph is gone
        torch.autograd.grad(out, asked, up)
