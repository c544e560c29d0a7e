"""Linear cross entropy against its definition in 64 bits: every type, ragged rows and
vocabularies, label smoothing, z-loss and the three reductions, padded rows that hold infinities
and NaN, vocabulary entries masked by the bias, row chunks, fp16 gradients far below the type's
range, differences, determinism, streams and graphs."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def make(N, D, V, dtype, seed, bias=True, ignored=0.1, w_std=0.05):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, D, generator=g).to(dtype).cuda()
    w = (torch.randn(V, D, generator=g) * w_std).to(dtype).cuda()
    b = (torch.randn(V, generator=g) * 0.3).cuda() if bias else None
    t = torch.randint(0, V, (N,), generator=g)
    t[torch.rand(N, generator=g) < ignored] = -100
    if N > 3 and ignored:
        t[1], t[2] = V, -1
    up = torch.randn(N, generator=g).cuda()
    return h, w, b, t.cuda(), up


def reference(h, w, b, t, s, c, reduction, up):
    """Losses, lse and gradients in 64 bits, with the logits and dz for the error bounds."""
    V = w.shape[0]
    ok = (t >= 0) & (t < V)
    h = torch.where(ok[:, None], h.double(), 0.0)
    w = w.double()
    z = h @ w.t()
    if b is not None:
        z = z + b.double()
    lse = torch.logsumexp(z, 1)
    tc = torch.where(ok, t, 0)[:, None]
    loss = (1 - s) * (lse - z.gather(1, tc)[:, 0]) + c * lse ** 2
    if s:
        loss = loss + s * (lse - z.mean(1))
    loss = torch.where(ok, loss, 0.0)
    n = max(int(ok.sum()), 1)
    g = {"none": up.double(), "sum": torch.ones_like(lse) * float(up[0]),
         "mean": torch.ones_like(lse) * float(up[0]) / n}[reduction]
    g = torch.where(ok, g, 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    onehot = torch.zeros_like(z).scatter_(1, tc, 1.0)
    dz = g * ((1 + 2 * c * lse)[:, None] * p - (1 - s) * onehot - s / V)
    dz = torch.where(ok[:, None], dz, 0.0)
    total = {"none": loss, "sum": loss.sum(), "mean": loss.sum() / n}[reduction]
    return dict(loss=total, rows=loss, lse=lse, ok=ok, n=n, z=z, p=p, g=g, dz=dz, h=h, w=w,
                dh=dz @ w, dw=dz.t() @ h, db=dz.sum(0))


def rounding(t, ref):
    f = torch.finfo(t)
    return (f.eps / 2) * ref.abs().clamp(min=f.smallest_normal)


def check(name, got, ref, tol):
    err = (got.double() - ref).abs()
    worst = float((err / tol).max()) if err.numel() else 0.0
    say(f"  {name}: worst error {worst:.3f} of its bound")
    assert bool((err <= tol).all()), (name, worst)


def bounds(r, s, c, reduction, dtype):
    """Error bounds.  A logit is a chain of D fp32 products (D U times the sum of their sizes),
    plus the bias; exp and its argument are off by (|z| + 4) 4 U; sums of V exponentials by
    (V / 256 + 32) U at most.  dz then holds one rounding to the inputs' type, and each gradient
    a chain of fp32 products and one rounding."""
    D, V, N = r["h"].shape[1], r["w"].shape[0], r["h"].shape[0]
    ez = (r["h"].abs() @ r["w"].abs().t()) * D * U + 2 * U * r["z"].abs()
    top = ez.max(1).values
    zmax = r["z"].abs().max(1).values
    elog = (zmax + 4) * 4 * U + (V / 256 + 32) * U
    elss = 2 * top + 2 * elog
    erow = (2 + 2 * c * r["lse"].abs()) * elss + 8 * U * (r["rows"].abs() + zmax * (1 + V * U)
                                                          + c * r["lse"] ** 2)
    if s:
        erow = erow + s * (V / 256 + 64) * U * zmax
    erow = torch.where(r["ok"], erow, 0.0)
    rel = (2 * top + 2 * elog)[:, None]  # of p
    a = (1 + 2 * c * r["lse"].abs())[:, None]
    ga = r["g"].abs()
    edz = ga * a * r["p"] * (rel + 8 * U) + 2 * c * ga * r["p"] * elss[:, None] + 4 * U * ga * (
        r["p"] * a + (r["dz"].abs() / ga.clamp(min=1e-300)).clamp(max=2 + float(a.max())))
    # the exponential and the matrix products flush what is below the smallest normal number,
    # 2^-126 (logits spread over several hundred reach it): p, and dz itself
    edz = edz + torch.where(r["ok"][:, None], 2.0 ** -126 * (1 + ga * a), 0.0)
    half = torch.finfo(dtype).eps / 2 if dtype != F32 else 0.0
    return erow, edz + (r["dz"].abs() + edz) * half


def run(h, w, b, t, up, s=0.0, c=0.0, reduction="mean", **kw):
    m = flp()
    loss, stats = m.cross_entropy_forward(h, w, t, b, s, c, reduction)
    g = up if reduction == "none" else up[0].clone()
    dh, dw, db = m.cross_entropy_backward(g, stats, h, w, t, b, s, c, reduction,
                                          need_bias=True, **kw)
    return loss, stats[0], dh, dw, db


def compare(h, w, b, t, up, s=0.0, c=0.0, reduction="mean", **kw):
    loss, lse, dh, dw, db = run(h, w, b, t, up, s, c, reduction, **kw)
    r = reference(h, w, b, t, s, c, reduction, up)
    erow, edz = bounds(r, s, c, reduction, h.dtype)
    N, D = h.shape
    V = w.shape[0]
    if reduction == "none":
        check("loss", loss, r["loss"], erow + 2 * U * r["rows"].abs() + 1e-300)
    else:
        div = r["n"] if reduction == "mean" else 1
        tol = (erow.sum() + (N / 1024 + 16) * U * r["rows"].abs().sum()) / div
        check("loss", loss, r["loss"], tol + 2 * U * r["loss"].abs() + 1e-300)
    # fp16: entries of dz below 2^-24 / 2^10 of the largest row factor are lost (subnormal step)
    sub = 0.0
    if h.dtype == F16:
        sub = float((r["g"].abs() * (1 + 2 * c * r["lse"].abs())[:, None]).max()) * 2.0 ** -34
    edz = edz + torch.where(r["ok"][:, None], sub, 0.0)
    check("d_hidden", dh, r["dh"], edz @ r["w"].abs() + V * U * (r["dz"].abs() @ r["w"].abs())
          + rounding(h.dtype, r["dh"]) * 1.01 + 1e-300)
    check("d_weight", dw, r["dw"], edz.t() @ r["h"].abs()
          + N * U * (r["dz"].abs().t() @ r["h"].abs()) + rounding(h.dtype, r["dw"]) * 1.01 + 1e-300)
    # d_bias adds the unrounded fp32 entries
    check("d_bias", db, r["db"], edz.sum(0) + N * U * r["dz"].abs().sum(0) + 1e-300)
    assert not dh[~r["ok"]].any()
    return loss, lse, dh, dw, db


SHAPES = [(1, 32, 1), (1, 64, 255), (3, 32, 256), (33, 96, 257), (64, 256, 4096), (65, 160, 1000),
          (130, 96, 2049), (300, 64, 777), (600, 224, 5003),
          (5, 32, 70001), (9, 32, 140001), (2100, 32, 70001)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_shapes(k, dtype):
    N, D, V = SHAPES[k]
    args = make(N, D, V, dtype, 10 * k, ignored=0.1 if N > 1 else 0.0)
    for s, c, red in ((0.0, 0.0, "mean"), (0.1, 1e-3, "none")):
        say(f"N={N} D={D} V={V} {dtype} s={s} c={c} {red}")
        compare(*args, s=s, c=c, reduction=red)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("s,c,bias", [(0.0, 1e-2, False), (0.3, 0.0, True), (1.0, 1e-4, True)])
def test_terms(dtype, reduction, s, c, bias):
    compare(*make(130, 64, 1300, dtype, 5, bias=bias), s=s, c=c, reduction=reduction)


def test_int32_targets_and_leading_shape():
    m = flp()
    h, w, b, t, up = make(24, 64, 500, BF16, 6)
    want = m.linear_cross_entropy(h, w, t, b, 0.1, 1e-3, "none")
    got = m.linear_cross_entropy(h.view(2, 3, 4, 64), w, t.int().view(2, 3, 4), b, 0.1, 1e-3,
                                 "none")
    assert got.shape == (2, 3, 4) and torch.equal(got.view(-1), want)


def test_plain_loss_is_minus_logp():
    m = flp()
    h, w, b, t, up = make(300, 96, 3001, BF16, 7)
    loss = m.linear_cross_entropy(h, w, t, b, reduction="none")
    assert torch.equal(loss, -m.linear_logp(h, w, t, b) + 0.0)


def test_padded_rows_hold_anything():
    """Rows whose target is outside the vocabulary: infinities and NaN in their hidden rows reach
    neither a loss nor a gradient."""
    for dtype in (BF16, F16, F32):
        h, w, b, t, up = make(70, 64, 600, dtype, 8)
        clean = run(h, w, b, t, up, 0.1, 1e-3, "mean")
        pad = (t < 0) | (t >= 600)
        assert int(pad.sum()) > 3
        bad = h.clone()
        bad[pad] = float("nan")
        bad[pad.nonzero()[0]] = float("inf")
        got = run(bad, w, b, t, up, 0.1, 1e-3, "mean")
        for k, (x, y) in enumerate(zip(got, clean)):
            if k == 1:  # lse of a padded row is whatever its logits are
                x, y = x[~pad], y[~pad]
            assert torch.equal(x, y), k


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nothing_but_padding(dtype):
    h, w, b, t, up = make(40, 64, 300, dtype, 9)
    t.fill_(-100)
    for reduction in ("none", "sum", "mean"):
        loss, lse, dh, dw, db = run(h, w, b, t, up, 0.1, 1e-3, reduction)
        for x in (loss, dh, dw, db):
            assert not x.any()


@pytest.mark.parametrize("low", [-math.inf, torch.finfo(F32).min, -1e30])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masked_vocabulary(dtype, low):
    """Entries masked through the bias, whole 256-column tiles among them: probability 0 and no
    gradient, the loss that of the remaining vocabulary."""
    m = flp()
    h, w, b, t, up = make(50, 64, 1500, dtype, 10, ignored=0.0)
    keep = torch.zeros(1500, dtype=torch.bool, device="cuda")
    keep[256:300] = True
    keep[1024:1400] = True
    masked = torch.where(keep, b, torch.full_like(b, low))
    t = keep.nonzero()[:, 0][t % int(keep.sum())]
    loss, lse, dh, dw, db = run(h, w, masked, t, up, 0.0, 1e-3, "none")
    index = torch.cumsum(keep, 0) - 1
    r = reference(h, w[keep].contiguous(), b[keep].contiguous(), index[t], 0.0, 1e-3, "none", up)
    erow, edz = bounds(r, 0.0, 1e-3, "none", dtype)
    check("loss", loss, r["loss"], erow + 2 * U * r["rows"].abs())
    assert not dw[~keep].any() and not db[~keep].any()
    check("d_bias", db[keep], r["db"], edz.sum(0) + 50 * U * r["dz"].abs().sum(0))
    check("d_hidden", dh, r["dh"], edz @ r["w"].abs()
          + 1500 * U * (r["dz"].abs() @ r["w"].abs()) + rounding(dtype, r["dh"]) * 1.01)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("V", [700, 1500, 70001, 140001])
def test_nan_logits_reach_the_loss(V, dtype):
    """NaN rows of W that fill whole vocabulary tiles (and one that does not): the loss of every
    counted row is NaN, its log-probability too, and a padded row's loss stays 0.  Tiles of
    nothing but -infinity beside them add nothing."""
    m = flp()
    h, w, b, t, up = make(20, 64, V, dtype, 22)
    t = torch.where(t >= 0, t % 200, t)
    ok = (t >= 0) & (t < V)
    for lo, hi in ((256, 512), (300, 301), (256, V)):
        bad = w.clone()
        bad[lo:hi] = float("nan")
        for bias in (None, torch.where(torch.arange(V, device="cuda") < 210, b, -math.inf)):
            for s, c in ((0.0, 0.0), (0.1, 1e-3)):
                loss, stats = m.cross_entropy_forward(h, bad, t, bias, s, c, "none")
                assert bool(loss[ok].isnan().all()) and not loss[~ok].any()
                assert bool(stats[0][ok].isnan().all())
                assert bool(m.linear_cross_entropy(h, bad, t, bias, s, c).isnan())
            assert bool(m.linear_logp(h, bad, t, bias)[ok].isnan().all())
            if dtype != F16:
                assert bool(m.cross_entropy_gradients(h, bad, t, bias)[0].isnan())
    # the masked vocabulary alone
    bias = torch.where(torch.arange(V, device="cuda") < 210, b, -math.inf)
    part, _ = m.forward_partial(h, w, t, 0, V, bias)
    assert bool((part[1:, :, 0] == -math.inf).all()) and not part[1:, :, 1].any()
    loss = m.linear_cross_entropy(h, w, t, bias, reduction="none")
    few = m.linear_cross_entropy(h, w[:210].contiguous(), torch.where(ok, t, -1),
                                 b[:210].contiguous(), reduction="none")
    assert torch.equal(loss, few) and bool(loss.isfinite().all())


def test_lowest_everywhere_is_uniform():
    """Every entry masked with the lowest fp32 value: the row is uniform over the vocabulary."""
    h, w, b, t, up = make(20, 64, 700, F32, 11, ignored=0.0)
    b = torch.full_like(b, torch.finfo(F32).min)
    loss, lse, dh, dw, db = run(h, w, b, t, up, 0.0, 0.0, "none")
    assert bool((loss.double() - math.log(700)).abs().max() <= 64 * U * math.log(700))
    p = torch.full((20, 700), 1.0 / 700, device="cuda", dtype=torch.float64)
    dz = up.double()[:, None] * (p - torch.nn.functional.one_hot(t, 700))
    check("d_bias", db, dz.sum(0), 64 * U * dz.abs().sum(0))


def test_smoothing_over_the_lowest_value_stays_finite():
    """Half the vocabulary at the lowest fp32 value, label smoothing on: the mean of the logits
    is representable although their sum is not."""
    m = flp()
    h, w, b, t, up = make(20, 64, 4096, F32, 12, ignored=0.0)
    b[2048:] = torch.finfo(F32).min
    loss = m.linear_cross_entropy(h, w, t % 2048, b, label_smoothing=0.25, reduction="none")
    want = 0.25 * 0.5 * -float(torch.finfo(F32).min)
    assert bool((loss.double() / want - 1).abs().max() < 1e-5)


def test_large_and_confident_logits():
    """Logits of several hundred, and rows whose target has probability 1 up to rounding."""
    for dtype in (BF16, F32):
        h, w, b, t, up = make(40, 64, 900, dtype, 13, w_std=6.0, ignored=0.0)
        with torch.no_grad():
            t[:20] = (h[:20].float() @ w.float().t() + b).argmax(1)
        compare(h, w, b, t, up, c=1e-4, reduction="none")


def test_small_fp16_gradients_do_not_underflow():
    """A mean over 2000 rows, and an upstream gradient of 2^-12: dz is below what fp16 holds."""
    h, w, b, t, up = make(2000, 64, 3000, F16, 14)
    up[0] = 2.0 ** -12
    compare(h, w, b, t, up, s=0.1, reduction="mean")
    up = up * 2.0 ** 40  # and gradients beyond its largest value, over a sum in range
    r = reference(h, w, b, t, 0.0, 0.0, "mean", up)
    loss, lse, dh, dw, db = run(h, w, b, t, up, 0.0, 0.0, "mean")
    check("d_bias", db, r["db"], r["dz"].abs().sum(0) * 1e-3)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_row_chunks_keep_the_bits(dtype):
    """The smallest workspace (256-row chunks) and the largest give the same gradients."""
    m = flp()
    h, w, b, t, up = make(700, 64, 2000, dtype, 15)
    code = {BF16: m.FLP_BF16, F16: m.FLP_F16, F32: m.FLP_F32}[dtype]
    least = m.flp_cross_entropy_backward_workspace_bytes(700, 64, 2000, code, 256)
    one = m.flp_cross_entropy_backward_workspace_bytes(700, 64, 2000, code, 700)
    a = run(h, w, b, t, up, 0.1, 1e-3, "mean", workspace_bytes=least)
    z = run(h, w, b, t, up, 0.1, 1e-3, "mean", workspace_bytes=one)
    assert all(torch.equal(x, y) for x, y in zip(a, z))


def at_once(h, w, b, t, s, c, reduction, **kw):
    m = flp()
    loss, stats, dh, dw, db = m.cross_entropy_gradients(h, w, t, b, s, c, reduction,
                                                        need_bias=True, **kw)
    return loss, stats[0], dh, dw, db


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_gradients_at_once_have_the_bits_of_two_calls(k, dtype):
    N, D, V = SHAPES[k]
    h, w, b, t, up = make(N, D, V, dtype, 10 * k, ignored=0.1 if N > 1 else 0.0)
    for s, c, red, bias in ((0.0, 0.0, "mean", None), (0.1, 1e-3, "sum", b)):
        want = run(h, w, bias, t, torch.ones_like(up), s, c, red)
        got = at_once(h, w, bias, t, s, c, red)
        for name, x, y in zip(("loss", "lse", "d_hidden", "d_weight", "d_bias"), got, want):
            assert torch.equal(x, y), (N, D, V, red, name)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_at_once_in_chunks_and_parts(dtype):
    m = flp()
    h, w, b, t, up = make(1100, 96, 2500, dtype, 50)
    want = run(h, w, b, t, torch.ones_like(up), 0.1, 1e-3, "mean")
    code = {BF16: m.FLP_BF16, F32: m.FLP_F32}[dtype]
    size = m.flp_cross_entropy_gradients_workspace_bytes
    sizes = [size(1100, 96, 2500, code, r) for r in (256, 512, 1100)]
    assert sizes == sorted(sizes) and size(1100, 96, 2500, code, 0) <= sizes[-1]
    for wsb in sizes + [size(1100, 96, 2500, code, 0)]:
        got = at_once(h, w, b, t, 0.1, 1e-3, "mean", workspace_bytes=wsb)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), wsb
    for need in ((True, False), (False, True), (False, False)):
        loss, stats, dh, dw, db = m.cross_entropy_gradients(h, w, t, b, 0.1, 1e-3,
                                                            need_hidden=need[0],
                                                            need_weight=need[1], need_bias=False)
        assert torch.equal(loss, want[0]) and db is None
        assert (dh is None) != need[0] and (dw is None) != need[1]
        assert dh is None or torch.equal(dh, want[2])
        assert dw is None or torch.equal(dw, want[3])


def test_gradients_at_once_with_padding_and_masks():
    """Padded rows of NaN, a vocabulary masked with the lowest value, nothing but padding, and an
    empty batch."""
    m = flp()
    h, w, b, t, up = make(300, 64, 1500, BF16, 51)
    b[256:600] = torch.finfo(F32).min
    t = torch.where((t >= 256) & (t < 600), t - 256, t)
    want = run(h, w, b, t, torch.ones_like(up), 0.0, 1e-3, "mean")
    bad = h.clone()
    pad = (t < 0) | (t >= 1500)
    bad[pad] = float("nan")
    got = at_once(bad, w, b, t, 0.0, 1e-3, "mean")
    for k in (0, 2, 3, 4):
        assert torch.equal(got[k], want[k]), k
    for x in at_once(h, w, b, torch.full_like(t, -1), 0.0, 1e-3, "mean")[::2]:
        assert not x.any()
    loss, stats, dh, dw, db = m.cross_entropy_gradients(h[:0], w, t[:0], b)
    assert not loss.any() and dh.shape == (0, 64) and not dw.any() and not db.any()


# the sizes from which a step's loss and gradients come from one call
@pytest.mark.parametrize("dtype,N,D,V", [(BF16, 300, 1024, 70000), (F32, 200, 128, 100000)])
def test_autograd_of_large_steps(dtype, N, D, V):
    m = flp()
    h, w, b, t, up = make(N, D, V, dtype, 52, w_std=0.02)
    unit = run(h, w, b, t, torch.ones_like(up), 0.1, 1e-3, "mean")
    names = ("hidden", "weight", "bias")
    leaves = [x.clone().requires_grad_(True) for x in (h, w, b)]
    loss = m.linear_cross_entropy(leaves[0], leaves[1], t, leaves[2], 0.1, 1e-3)
    assert torch.equal(loss, unit[0])
    # first backward (made with the loss), a second one (recomputed), and one with a factor
    first = torch.autograd.grad(loss, leaves, retain_graph=True)
    again = torch.autograd.grad(loss, leaves, retain_graph=True)
    for n, x, y, z in zip(names, first, again, unit[2:]):
        assert torch.equal(x, z) and torch.equal(y, z), n
    loss = m.linear_cross_entropy(leaves[0], leaves[1], t, leaves[2], 0.1, 1e-3)
    half = torch.autograd.grad(loss * 0.5, leaves)
    for n, x, z in zip(names, half, unit[2:]):
        assert torch.equal(x.double(), 0.5 * z.double()), n
    loss = m.linear_cross_entropy(leaves[0], leaves[1], t, leaves[2], 0.1, 1e-3)
    third = torch.autograd.grad(loss * 3, leaves)
    for n, x, z in zip(names, third, unit[2:]):
        # rounded at 1, times 3 in fp32, rounded once more
        assert bool(((x.double() - 3 * z.double()).abs()
                     <= torch.finfo(x.dtype).eps / 2 * 3 * z.double().abs() + 1e-300).all()), n
    # only one leaf asks
    x = h.clone().requires_grad_(True)
    (dh,) = torch.autograd.grad(m.linear_cross_entropy(x, w, t, b, 0.1, 1e-3), [x])
    assert torch.equal(dh, unit[2])


def test_a_captured_backward_of_gradients_made_at_once():
    """A backward that is captured by itself: every replay multiplies the forward's gradients by
    the upstream gradient of the time, not what the replay before left, and an eager backward
    beside it does too."""
    from lm_head_selected_bf16_amd import torch_ops
    m = flp()
    h, w, b, t, up = make(70, 64, 900, BF16, 53)
    _, _, *unit = at_once(h, w, b, t, 0.1, 1e-3, "mean")
    leaves = [x.requires_grad_() for x in (h, w, b)]
    loss = torch_ops.LossAndGradients.apply(h, w, t, b, 0.1, 1e-3, "mean")
    g = torch.ones((), device="cuda")

    def backward():  # the node's, without autograd around it
        got = torch_ops.LossAndGradients.backward(loss.grad_fn, g)
        return got[0], got[1], got[3]

    def check_times(got, f):
        for x, u in zip(got, unit):
            assert torch.equal(x, (u.float() * f).to(x.dtype)), f

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = backward()
    for f in (3.0, 3.0, 0.7, 1.0):
        g.fill_(f)
        graph.replay()
        torch.cuda.synchronize()
        check_times(out, f)
        check_times(torch.autograd.grad(loss, leaves, g, retain_graph=True), f)


def test_an_eager_backward_of_a_captured_forward():
    """What one replay's backward gave is not touched by the next replay."""
    from lm_head_selected_bf16_amd import torch_ops
    h, w, b, t, up = make(70, 64, 900, BF16, 54)
    h.requires_grad_()
    torch_ops.LossAndGradients.apply(h, w, t, b, 0.1, 1e-3, "mean")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = torch_ops.LossAndGradients.apply(h, w, t, b, 0.1, 1e-3, "mean")
    g = torch.full((), 3.0, device="cuda")
    seen = []
    for rep in range(3):
        with torch.no_grad():
            h.data.copy_(make(70, 64, 900, BF16, 200 + rep)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = torch_ops.LossAndGradients.backward(loss.grad_fn, g)[0]
        unit = at_once(h.detach(), w, b, t, 0.1, 1e-3, "mean")[2]
        seen.append((got, (unit.float() * 3).to(BF16)))
        for x, y in seen:
            assert torch.equal(x, y), rep


@pytest.mark.parametrize("call", ["at once", "functional", "autograd"])
def test_little_memory_means_smaller_chunks(call):
    """With room for the outputs, the least workspace and a little beside (the allocator takes
    20 MB at least for a tensor of over 1 MB), where a whole chunk of 4096 x 20000 takes 330 (two
    calls) to 650 MB: the same bits.  With room for nothing, torch's error."""
    from lm_head_selected_bf16_amd import torch_ops
    m = flp()
    h, w, b, t, up = make(4096, 64, 20000, BF16, 55)
    one = torch.ones((), device="cuda")
    leaf = h.clone().requires_grad_()
    loss, stats = m.cross_entropy_forward(h, w, t, b)
    kept = m.linear_cross_entropy(leaf, w, t, b)
    assert not torch_ops._gradients_at_once(leaf, w, "mean")

    def step():
        if call == "at once":
            return m.cross_entropy_gradients(h, w, t, b)[2:]
        if call == "functional":
            return m.cross_entropy_backward(one, stats, h, w, t, b)
        return torch.autograd.grad(kept, [leaf], retain_graph=True)

    want = step()
    code = m.FLP_BF16
    size = {"at once": m.flp_cross_entropy_gradients_workspace_bytes}.get(
        call, m.flp_cross_entropy_backward_workspace_bytes)
    room = (size(4096, 64, 20000, code, 0) >> 20) + 48
    assert size(4096, 64, 20000, code, 4096) > 2 * room << 20
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    try:
        torch.cuda.set_per_process_memory_fraction(
            (torch.cuda.memory_reserved() + (room << 20)) / total)
        got = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        del got
        torch.cuda.empty_cache()
        torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() / total)
        with pytest.raises(torch.OutOfMemoryError):
            step()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert all(torch.equal(x, y) for x, y in zip(step(), want))


def test_scale_inplace():
    m = flp()
    code = {BF16: m.FLP_BF16, F16: m.FLP_F16, F32: m.FLP_F32}
    stream = torch.cuda.current_stream().cuda_stream
    for dtype in (BF16, F16, F32):
        for n in (1, 7, 8, 4099):
            base = torch.randn(n + 9, device="cuda").to(dtype)
            for f in (1.0, 0.5, 3.0):
                x = base.clone()
                factor = torch.tensor(f, device="cuda")
                # starts one element in: off the 16-byte grid
                assert m.flp_scale_inplace(n, code[dtype], x[1:].data_ptr(), factor.data_ptr(),
                                           stream) == m.FLP_OK
                want = base.clone()
                want[1:n + 1] = (base[1:n + 1].float() * f).to(dtype)
                assert torch.equal(x, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_do_not_depend_on_the_batch(dtype):
    m = flp()
    h, w, b, t, up = make(333, 96, 2500, dtype, 16)
    loss, lse, dh, dw, db = run(h, w, b, t, up, 0.1, 1e-3, "none")
    again = run(h, w, b, t, up, 0.1, 1e-3, "none")
    assert all(torch.equal(x, y) for x, y in zip((loss, lse, dh, dw, db), again))
    for lo, hi in ((0, 1), (100, 133), (200, 333)):
        s = slice(lo, hi)
        part = run(h[s].contiguous(), w, b, t[s].contiguous(), up[s].contiguous(), 0.1, 1e-3,
                   "none")
        for x, y in zip(part[:3], (loss, lse, dh)):
            assert torch.equal(x, y[s])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N", [5, 64, 65, 128, 129, 512, 513, 1025, 2050])
def test_slabs_of_the_vocabulary(dtype, N):
    """Row counts around every tile of d_hidden, over a vocabulary of several slabs and a ragged
    last one, and past the last row count that takes slabs."""
    compare(*make(N, 96, 9001, dtype, 30 + N), s=0.1, c=1e-3, reduction="mean")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [4100, 9001])
def test_padding_rows_change_no_bit(V, dtype):
    """More rows, all of them padding, move the batch through the tiles of every row count: each
    sum keeps its order, so nothing changes."""
    h, w, b, t, up = make(60, 96, V, dtype, 33)
    want = run(h, w, b, t, up, 0.1, 1e-3, "sum")
    for N in (64, 100, 128, 250, 300, 700, 2100, 4200):
        x = torch.cat([h, torch.randn(N - 60, 96, device="cuda").to(dtype)])
        y = torch.cat([t, torch.full((N - 60,), -1, device="cuda", dtype=t.dtype)])
        got = run(x, w, b, y, up, 0.1, 1e-3, "sum")
        assert torch.equal(got[1][:60], want[1]) and torch.equal(got[2][:60], want[2]), N
        assert not got[2][60:].any(), N
        assert torch.equal(got[3], want[3]) and torch.equal(got[4], want[4]), N


@pytest.mark.parametrize("N", [8192, 8193])
def test_last_row_count_of_slabs(N):
    compare(*make(N, 32, 4500, BF16, 29), s=0.1, reduction="sum")


def test_slabs_keep_rows_apart():
    m = flp()
    h, w, b, t, up = make(1024, 64, 9000, BF16, 31)
    dh = run(h, w, b, t, up, reduction="none")[2]
    for lo, hi in ((0, 1), (3, 60), (200, 330), (300, 1000)):
        s = slice(lo, hi)
        part = run(h[s].contiguous(), w, b, t[s].contiguous(), up[s].contiguous(),
                   reduction="none")[2]
        assert torch.equal(part, dh[s])


def test_gradient_against_differences():
    m = flp()
    h, w, b, t, up = make(6, 32, 40, F32, 17, ignored=0.0, w_std=0.3)
    t[5] = -1
    leaves = [x.clone().requires_grad_(True) for x in (h, w, b)]
    for reduction in ("mean", "sum"):
        loss = m.linear_cross_entropy(leaves[0], leaves[1], t, leaves[2], 0.1, 1e-2, reduction)
        grads = torch.autograd.grad(loss, leaves)
        step = 2.0 ** -6
        for k, x in enumerate((h, w, b)):
            flat = x.view(-1)
            for e in range(0, flat.numel(), 37):
                old = float(flat[e])
                vals = []
                for d in (step, -step):
                    flat[e] = old + d
                    vals.append(float(m.linear_cross_entropy(h, w, t, b, 0.1, 1e-2, reduction)))
                flat[e] = old
                diff = (vals[0] - vals[1]) / (2 * step)
                # a third derivative below 40 over six rows, and 64 U of a loss below 64
                assert abs(diff - float(grads[k].view(-1)[e])) < 40 * 6 * step ** 2 / 6 * 0.05 \
                    + 64 * 64 * U / (2 * step)


def test_autograd_asks_only_for_what_needs_a_gradient():
    m = flp()
    h, w, b, t, up = make(60, 64, 500, BF16, 18)
    _, _, dh, dw, db = run(h, w, b, t, torch.ones_like(up), 0.1, 0.0, "mean")
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        leaves = [x.clone().requires_grad_(bool(n)) for x, n in zip((h, w, b), need)]
        m.linear_cross_entropy(leaves[0], leaves[1], t, leaves[2], 0.1).backward()
        for x, n, want in zip(leaves, need, (dh, dw, db)):
            assert (x.grad is not None) == bool(n)
            assert x.grad is None or torch.equal(x.grad, want)
    # twice through the same graph
    x = h.clone().requires_grad_(True)
    loss = m.linear_cross_entropy(x, w, t, b, 0.1)
    one = torch.autograd.grad(loss, [x], retain_graph=True)[0]
    two = torch.autograd.grad(loss * 2, [x])[0]
    assert torch.equal(one, dh) and torch.equal(one.float() * 2, two.float())


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("need", range(1, 8))
def test_autograd_gives_each_leaf_its_gradient(need, bias):
    m = flp()
    h, w, b, t, up = make(33, 64, 700, F16, 61, bias=bias)
    ask = [need & 1, need & 2, need & 4 and bias]
    if not any(ask):
        return
    _, stats = m.cross_entropy_forward(h, w, t, b, 0.1, 1e-3, "none")
    g = up[:1].expand(33)
    want = m.cross_entropy_backward(g.contiguous(), stats, h, w, t, b, 0.1, 1e-3, "none")
    leaves = [None if x is None else x.clone().requires_grad_(bool(a))
              for x, a in zip((h, w, b), ask)]
    loss = m.linear_cross_entropy(leaves[0], leaves[1], t, leaves[2], 0.1, 1e-3, "none")
    got = torch.autograd.grad(loss, [x for x, a in zip(leaves, ask) if a], g)
    for x, v in zip(got, [v for v, a in zip(want, ask) if a]):
        assert torch.equal(x, v)


@pytest.mark.parametrize("which", ["hidden", "weight", "bias", "device", "dtype"])
def test_data_exchanged_before_the_backward_is_refused(which):
    h, w, b, t, up = make(9, 64, 300, F32, 62)
    h, w, b = (x.requires_grad_() for x in (h, w, b))
    loss = flp().linear_cross_entropy(h, w, t, b)
    if which == "hidden":
        h.data = h.data[:4].clone()
    elif which == "weight":
        w.data = w.data[:100].clone()
    elif which == "bias":
        b.data = b.data[:100].clone()
    elif which == "device":
        w.data = w.data.cpu()
    else:
        w.data = w.data.to(BF16)
    with pytest.raises((ValueError, TypeError)):
        torch.autograd.grad(loss, [h])


def test_empty_batch():
    m = flp()
    w = torch.randn(300, 64, device="cuda", dtype=BF16, requires_grad=True)
    h = torch.empty(0, 64, device="cuda", dtype=BF16, requires_grad=True)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    for reduction in ("none", "sum", "mean"):
        loss = m.linear_cross_entropy(h, w, t, reduction=reduction)
        assert loss.numel() == (0 if reduction == "none" else 1) and not loss.any()
        dw, dh = torch.autograd.grad(loss.sum(), [w, h])
        assert not dw.any() and dh.shape == (0, 64)


@pytest.mark.parametrize("at_once", [False, True])
def test_graph_replays_with_new_inputs(at_once):
    m = flp()
    h, w, b, t, up = make(260, 64, 1500, BF16, 19)
    g = torch.ones((), device="cuda")

    def step():
        if at_once:
            return m.cross_entropy_gradients(h, w, t, b, 0.1, 1e-3)
        loss, stats = m.cross_entropy_forward(h, w, t, b, 0.1, 1e-3)
        return (loss,) + m.cross_entropy_backward(g, stats, h, w, t, b, 0.1, 1e-3)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        nh, _, _, nt, _ = make(260, 64, 1500, BF16, 100 + rep)
        h.copy_(nh)
        t.copy_(nt)
        g.fill_(0.5 + rep)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, step())), rep


def test_second_derivatives_are_refused():
    m = flp()
    h, w, b, t, up = make(8, 64, 100, F32, 21)
    h.requires_grad_(True)
    # with a constant upstream gradient the first derivative is a constant to autograd
    (g,) = torch.autograd.grad(m.linear_cross_entropy(h, w, t, b), [h], create_graph=True)
    with pytest.raises(RuntimeError, match="does not require grad"):
        g.sum().backward()
    one = torch.ones((), device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad(m.linear_cross_entropy(h, w, t, b), [h], one, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_two_streams_at_once():
    """Two batches on two streams, each with its own workspaces, give what they give alone."""
    m = flp()
    batches = [make(300, 64, 3000, BF16, 40 + k) for k in range(2)]
    want = [run(*b, 0.1, 1e-3, "mean") for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(3):
        got = []
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                got.append(run(*b, 0.1, 1e-3, "mean"))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_refusals():
    m = flp()
    h, w, b, t, up = make(8, 64, 100, BF16, 20)
    for kw in (dict(label_smoothing=-0.1), dict(label_smoothing=1.5), dict(z_loss=-1.0),
               dict(z_loss=float("nan"))):
        with pytest.raises(m.FlpError):
            m.linear_cross_entropy(h, w, t, **kw)
    with pytest.raises(ValueError):
        m.linear_cross_entropy(h, w, t, reduction="max")
    with pytest.raises(ValueError):
        m.linear_cross_entropy(h, w, t.cpu())
    with pytest.raises(ValueError):
        m.linear_cross_entropy(h, w, t, b.double())
    with pytest.raises(TypeError):
        m.linear_cross_entropy(h, w.float(), t)
    with pytest.raises(m.FlpError):
        m.linear_cross_entropy(h[:, :40].contiguous(), w[:, :40].contiguous(), t)
    with pytest.raises(m.FlpError):
        m.cross_entropy_gradients(h, w, t, reduction="none")
    with pytest.raises(m.FlpError):
        m.cross_entropy_gradients(h.half(), w.half(), t)
    loss, stats = m.cross_entropy_forward(h, w, t, b)
    with pytest.raises(ValueError):
        m.cross_entropy_backward(up, stats, h, w, t, b)  # a scalar is wanted
    with pytest.raises(ValueError):
        m.cross_entropy_backward(torch.ones((), device="cuda"), stats[:1], h, w, t, b)
