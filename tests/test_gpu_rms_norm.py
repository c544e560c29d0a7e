"""The root mean square norms around a block against their definition in 64 bits: widths from one
element to the widest row, every type, gates per channel, per sequence and per element, with and
without a norm behind the block; gradients against the formula and against differences, batches
that do not depend on each other, views, streams and graphs."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative
EPS = 1e-6


def rounding(t, ref):
    """Half a step of the type at ref."""
    f = torch.finfo(t)
    return (f.eps / 2) * ref.abs().clamp(min=f.smallest_normal)


def make(N, D, dtype, wdtype, seed, gates=0, block=True, post=False, weight=True):
    g = torch.Generator().manual_seed(seed)
    size = torch.rand(N, 1, generator=g) * 3 + 0.2
    a = dict(x=(torch.randn(N, D, generator=g) * size).to(dtype),
             grad_n=torch.randn(N, D, generator=g).to(dtype), scale=0.7)
    if weight:
        a["weight"] = (torch.randn(D, generator=g) * 0.3 + 1).to(wdtype)
    if block:
        a["y"] = (torch.randn(N, D, generator=g) * (size * 0.5 + 0.1)).to(dtype)
        a["grad_r"] = torch.randn(N, D, generator=g).to(dtype)
        a["post_norm"] = post
        if post and weight:
            a["post_weight"] = (torch.randn(D, generator=g) * 0.3 + 1).to(wdtype)
        if gates:
            a["gate"] = (torch.randn(gates, D, generator=g) * 0.4 + 0.5).to(wdtype)
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()}


# A sum over D elements has chains of at most 8 elements, 8 chunks and a tree of 9 levels: 25
# roundings, so 33 U with those of its terms.  A norm's factor: half of that, and four of its own.
SUM = 33 * U
NORM = SUM / 2 + 4 * U


def reference(a, eps=EPS):
    """Values and bounds on what fp32 makes of them, by the roundings that the formula has."""
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    x = d["x"]
    N, D = x.shape
    one = torch.ones(D, dtype=torch.float64, device=x.device)
    w = d.get("weight", one)
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    out, tol = {}, {}
    r, er = x, torch.zeros_like(x)
    if "y" in d:
        y = d["y"]
        pw = d.get("post_weight", one)
        post = d["post_norm"]
        ry = 1 / torch.sqrt(mean(y * y) + eps) if post else torch.ones_like(mean(y))
        yh = y * ry
        eyh = yh.abs() * (NORM + U if post else 0.0)
        gate = d.get("gate", torch.ones(1, D, dtype=torch.float64, device=x.device))
        each = gate.repeat_interleave(N // gate.shape[0], 0)
        f = d["scale"] * each * pw
        r = x + yh * f
        er = eyh * f.abs() + 5 * U * (yh * f).abs() + U * r.abs()
        out["r"], tol["r"] = r, er
    ms = mean(r * r)
    rstd = 1 / torch.sqrt(ms + eps)
    err = NORM + mean(r.abs() * er) / (ms + eps)  # of rstd, relative
    rh = r * rstd
    erh = rstd * er + rh.abs() * (err + U)
    out["n"], tol["n"] = rh * w, w.abs() * (erh + 2 * U * rh.abs())
    gn = d["grad_n"]
    gw = gn * w
    m2 = mean(gw * rh)
    em2 = (SUM + 2 * U) * mean((gw * rh).abs()) + mean(gw.abs() * erh)
    dr = rstd * (gw - rh * m2)
    both = gw.abs() + (rh * m2).abs()
    edr = rstd * (erh * m2.abs() + rh.abs() * em2 + 4 * U * both) + (err + 2 * U) * rstd * both
    rows = (N + 64) * U  # chains of at most N / 256 + 8 rows (or slabs), then trees
    out["d_weight"] = (gn * rh).sum(0)
    tol["d_weight"] = rows * (gn * rh).abs().sum(0) + (gn.abs() * erh).sum(0)
    if "y" in d:
        dr = dr + d["grad_r"]
        edr = edr + U * dr.abs()
        g = dr * f
        eg = edr * f.abs() + 6 * U * g.abs()
        if post:
            m3 = mean(g * yh)
            em3 = (SUM + 2 * U) * mean((g * yh).abs()) + mean(yh.abs() * eg + g.abs() * eyh)
            out["d_y"] = ry * (g - yh * m3)
            s = g.abs() + (yh * m3).abs()
            tol["d_y"] = ry * (eg + yh.abs() * em3 + m3.abs() * eyh + (NORM + 5 * U) * s)
            t = d["scale"] * each * dr * yh
            out["d_post_weight"] = t.sum(0)
            tol["d_post_weight"] = ((rows + 8 * U) * t.abs().sum(0) + (
                (d["scale"] * each).abs() * (edr * yh.abs() + dr.abs() * eyh)).sum(0))
        else:
            out["d_y"], tol["d_y"] = g, eg
        t = d["scale"] * pw * dr * yh
        et = (rows + 8 * U) * t.abs() + (d["scale"] * pw).abs() * (edr * yh.abs() + dr.abs() * eyh)
        G = gate.shape[0]
        out["d_gate"], tol["d_gate"] = (v.view(G, -1, D).sum(1) for v in (t, et))
    out["d_x"], tol["d_x"] = dr, edr
    return out, tol


def run(a, eps=EPS):
    m = flp()
    got = {}
    if "y" not in a:
        got["n"], rstd = m.rms_norm_forward(a["x"], a.get("weight"), eps)
        got["d_x"], got["d_weight"] = m.rms_norm_backward(a["grad_n"], a["x"], rstd, a.get("weight"))
        return got
    kw = dict(weight=a.get("weight"), post_weight=a.get("post_weight"), gate=a.get("gate"),
              scale=a["scale"], post_norm=a["post_norm"])
    got["r"], got["n"], rstd, prstd = m.residual_rms_norm_forward(a["x"], a["y"], eps=eps, **kw)
    names = ("d_x", "d_y", "d_weight", "d_post_weight", "d_gate")
    grads = m.residual_rms_norm_backward(a["grad_r"], a["grad_n"], a["x"], a["y"], rstd, prstd, **kw)
    got.update({k: v for k, v in zip(names, grads) if v is not None})
    return got


def compare(a, eps=EPS):
    got = run(a, eps)
    ref, tol = reference(a, eps)
    for k, v in got.items():
        bound = rounding(v.dtype, ref[k]) * (1 + 2.0 ** -6) + tol[k] * (1 + 2.0 ** -6) + 1e-45
        err = (v.double() - ref[k]).abs()
        worst = float((err / bound).max())
        say(f"  {k}: worst error {worst:.3f} of its bound")
        assert worst <= 1.0, (k, worst)
    return got


TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]
WIDTHS = [1, 2, 7, 8, 9, 64, 511, 520, 777, 1025, 1345, 2048, 2056, 2688, 4100, 8192, 8200, 16383,
          16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_widths(D, dtype, wdtype):
    for N, gates, block, post in ((1, 1, True, True), (36, 0, False, False), (36, 0, True, False),
                                  (36, 1, True, True), (36, 4, True, True), (36, 36, True, True),
                                  (36, 36, True, False)):
        say(f"N={N} D={D} {dtype} {wdtype} gates={gates} block={block} post={post}")
        compare(make(N, D, dtype, wdtype, 7 * D + N + gates, gates, block, post))


@pytest.mark.parametrize("N,gates", [(1, 0), (7, 7), (8, 2), (255, 5), (256, 256), (257, 1),
                                     (2049, 3), (4097, 17), (20011, 1), (20010, 10005)])
def test_row_counts(N, gates):
    for D, dtype in ((24, BF16), (777, F32), (2688, BF16)):
        say(f"N={N} D={D} {dtype} gates={gates}")
        compare(make(N, D, dtype, dtype, N + D, gates, True, True))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gates", [0, 1, 3, 33])
def test_without_weights(gates, post):
    compare(make(33, 1000, BF16, BF16, 3, gates, True, post, weight=False))


def test_sizes_of_the_rows():
    """Rows of 1e-18 to 1e18, eps = 0."""
    a = make(37, 1001, F32, F32, 5, 1, True, True)
    k = torch.logspace(-18, 18, 37, device="cuda")[:, None]
    a["x"], a["y"] = a["x"] * k, a["y"] * k
    compare(a, eps=0.0)


def test_rows_of_zeros():
    a = make(9, 640, BF16, BF16, 6, 1, True, True)
    a["x"][3], a["y"][3], a["y"][5] = 0, 0, 0
    got = compare(a)
    assert not bool(got["r"][3].any()) and not bool(got["n"][3].any())


def test_infinite_and_nan_rows_stay_by_themselves():
    a = make(40, 520, BF16, BF16, 7, 1, True, True)
    clean = run(a)
    b = dict(a, x=a["x"].clone(), y=a["y"].clone())
    b["x"][7, 3], b["y"][19, 11] = math.inf, math.nan
    got = run(b)
    ok = [i for i in range(40) if i not in (7, 19)]
    for k in ("r", "n", "d_x", "d_y"):
        assert torch.equal(got[k][ok], clean[k][ok]), k
    assert bool(got["n"][19].isnan().all())
    # grad_r alone goes through the sum: it is d_x, whatever the row holds
    m = flp()
    rstd = torch.zeros(40, device="cuda")
    dx, dy, *_ = m.residual_rms_norm_backward(b["grad_r"], None, b["x"], b["y"], rstd, None,
                                              need_weight=False)
    assert torch.equal(dx, b["grad_r"]) and torch.equal(dy, b["grad_r"])


def test_without_a_residual_it_is_the_plain_norm():
    """scale = 0 leaves x: the same bits as the plain norm of x."""
    a = make(50, 1345, F16, F32, 8)
    a["scale"] = 0.0
    m = flp()
    got = run(a)
    n, rstd = m.rms_norm_forward(a["x"], a["weight"])
    assert torch.equal(got["r"], a["x"]) and torch.equal(got["n"], n)
    assert not bool(got["d_y"].any())


@pytest.mark.parametrize("gates", [1, 5, 300])
def test_rows_do_not_depend_on_each_other(gates):
    a = make(300, 1000, BF16, BF16, 9, gates, True, True)
    whole = run(a)
    each = a["gate"].repeat_interleave(300 // gates, 0)
    for i in (0, 123, 299):
        one = {k: v[i:i + 1].contiguous() if isinstance(v, torch.Tensor) and v.shape[0] == 300 else v
               for k, v in a.items()}
        one["gate"] = each[i:i + 1].contiguous()
        got = run(one)
        for k in ("r", "n", "d_x", "d_y"):
            assert torch.equal(got[k][0], whole[k][i]), (k, i)
    again = run(a)
    for k in whole:
        assert torch.equal(whole[k], again[k]), k


def test_views_off_the_16_byte_grid_and_what_surrounds_them():
    m = flp()
    N, D = 33, 1345
    for dtype in (BF16, F32):
        a = make(N, D, dtype, dtype, 10, 3, True, True)

        def moved(t):
            flat = torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")[3:]
            return flat.copy_(t.reshape(-1)).view(t.shape)
        b = {k: moved(v) if isinstance(v, torch.Tensor) else v for k, v in a.items()}
        x, y = run(a), run(b)
        for k in x:
            assert torch.equal(x[k], y[k]), k
        big = torch.full((N * D + 16,), 7.0, dtype=dtype, device="cuda")
        out = big[5:5 + N * D]
        from lm_head_selected_bf16_amd import _abi
        code = _abi.FLP_BF16 if dtype == BF16 else _abi.FLP_F32
        assert m.flp_rms_norm_forward(N, D, code, a["x"].data_ptr(), code, 0, EPS, out.data_ptr(),
                                      0, torch.cuda.current_stream().cuda_stream) == 0
        assert bool((big[:5] == 7).all()) and bool((big[5 + N * D:] == 7).all())
        assert torch.equal(out.view(N, D), m.rms_norm_forward(a["x"])[0])


def test_empty_batch():
    m = flp()
    x = torch.empty(0, 64, device="cuda", requires_grad=True)
    y = torch.empty(0, 64, device="cuda", requires_grad=True)
    w, pw, g = (torch.ones(64, device="cuda", requires_grad=True) for _ in range(3))
    r, n = m.residual_rms_norm(x, y, w, pw, g)
    assert r.shape == n.shape == (0, 64)
    grads = torch.autograd.grad([r, n], [x, y, w, pw, g], [torch.empty_like(r)] * 2)
    assert grads[0].shape == (0, 64) and all(not bool(v.any()) for v in grads[2:])


@pytest.mark.parametrize("gates", [0, 1, 3])
def test_no_rows_through_the_abi(gates):
    """Without rows nothing is read, null pointers and infinite parameters neither: the sums over
    rows are zeros."""
    m = flp()
    D = 37
    w = torch.full((D,), math.inf, device="cuda", dtype=F16)
    out = [torch.ones(n, D, device="cuda", dtype=F16) for n in (1, 1, max(gates, 1))]
    for gate, post in ((0, 0), (0, w.data_ptr()), (out[0].data_ptr(), 0)):
        for t in out[1:]:
            t.fill_(1)
        st = m._abi.flp_residual_rms_norm_backward(
            0, D, m.FLP_F16, 0, 0, 0, 0, m.FLP_F16, 0, 1, post, gates, 0 if gates != 1 else gate, 0.5,
            0, 0, 0, 0, 0, out[1].data_ptr(), out[2].data_ptr() if gates else 0, 0, 0,
            torch.cuda.current_stream().cuda_stream)
        assert st == m.FLP_OK
        assert not bool(out[1].any()) and not (gates and bool(out[2].any()))


@pytest.mark.parametrize("gates", [0, 1, 6, 24])
@pytest.mark.parametrize("post", [False, True])
def test_gradient_against_differences(gates, post):
    """fp32, a fixed random functional, central differences of the 64-bit formula's step: the
    difference quotient's own error is h^2 times a third derivative of the size of the gradient."""
    m = flp()
    a = make(24, 40, F32, F32, 11, gates, True, post)
    names = [k for k in ("x", "y", "weight", "post_weight", "gate") if k in a]
    leaves = {k: a[k].clone().requires_grad_(True) for k in names}
    r, n = m.residual_rms_norm(leaves["x"], leaves["y"], leaves["weight"],
                               post_weight=leaves.get("post_weight"), gate=leaves.get("gate"),
                               scale=a["scale"], post_norm=post)
    loss = (r * a["grad_r"]).sum() + (n * a["grad_n"]).sum()
    grads = dict(zip(names, torch.autograd.grad(loss, list(leaves.values()))))
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in a.items()}

    def value(**kw):
        o, _ = reference(dict(d, **kw))
        return float((o["r"] * d["grad_r"]).sum() + (o["n"] * d["grad_n"]).sum())
    h = 1e-5
    g = torch.Generator().manual_seed(12)
    for k in names:
        way = torch.randn(a[k].shape, generator=g).double().cuda()
        num = (value(**{k: d[k] + h * way}) - value(**{k: d[k] - h * way})) / (2 * h)
        ana = float((grads[k].double() * way).sum())
        scale = float((grads[k].double() * way).abs().sum())
        assert abs(num - ana) <= 1e-5 * scale + 1e-6, (k, num, ana)


@pytest.mark.parametrize("need", ["x", "y", "weight", "post_weight", "gate", "all"])
@pytest.mark.parametrize("used", ["r", "n", "both"])
def test_autograd_gives_each_leaf_its_gradient(need, used):
    m = flp()
    a = make(34, 520, BF16, F32, 13, 2, True, True)
    names = ["x", "y", "weight", "post_weight", "gate"]
    leaves = {k: a[k].clone().requires_grad_(need in (k, "all")) for k in names}
    r, n = m.residual_rms_norm(leaves["x"], leaves["y"], leaves["weight"], leaves["post_weight"],
                               leaves["gate"], scale=a["scale"])
    outs, ups = [], []
    if used in ("r", "both"):
        outs, ups = [r], [a["grad_r"]]
    if used in ("n", "both"):
        outs, ups = outs + [n], ups + [a["grad_n"]]
    wanted = [k for k in names if need in (k, "all")]
    got = torch.autograd.grad(outs, [leaves[k] for k in wanted], ups, allow_unused=True)
    _, _, rstd, prstd = m.residual_rms_norm_forward(a["x"], a["y"], a["weight"], a["post_weight"],
                                                    a["gate"], a["scale"])
    ref = m.residual_rms_norm_backward(a["grad_r"] if used != "n" else None,
                                       a["grad_n"] if used != "r" else None, a["x"], a["y"], rstd,
                                       prstd, a["weight"], a["post_weight"], a["gate"], a["scale"])
    for k, g in zip(wanted, got):
        assert torch.equal(g, ref[names.index(k)]), k
    if used == "r":
        assert not bool(ref[2].any())  # the next norm's weight has no part in r


def test_leading_shapes_and_gates_of_sequences():
    m = flp()
    a = make(24, 96, F32, F32, 14, 4, True, True)
    whole = m.residual_rms_norm(a["x"], a["y"], a["weight"], a["post_weight"], a["gate"])
    x, y = a["x"].view(4, 6, 96), a["y"].view(4, 6, 96)
    for gate in (a["gate"], a["gate"].view(4, 1, 96)):
        r, n = m.residual_rms_norm(x, y, a["weight"], a["post_weight"], gate)
        assert torch.equal(r.view(24, 96), whole[0]) and torch.equal(n.view(24, 96), whole[1])
    full = a["gate"].repeat_interleave(6, 0)
    r, n = m.residual_rms_norm(x, y, a["weight"], a["post_weight"], full.view(4, 6, 96))
    assert torch.equal(r.view(24, 96), whole[0])
    row = m.rms_norm(a["x"][0], a["weight"])
    assert torch.equal(row, m.rms_norm(a["x"], a["weight"])[0])


def test_refusals():
    m = flp()
    a = make(12, 64, F32, F32, 15, 1, True, True)
    x, y, w, g = a["x"], a["y"], a["weight"], a["gate"]
    for args, kw, err in [
            ((x.double(), y.double()), {}, TypeError), ((x, y.half()), {}, ValueError),
            ((x, y[:6]), {}, ValueError), ((x.t(), y.t()), {}, ValueError),
            ((x, y, w.half()), {}, TypeError), ((x, y, w[:32]), {}, ValueError),
            ((x, y, w.cpu()), {}, ValueError), ((x.cpu(), y.cpu()), {}, ValueError),
            ((x, y, w), dict(gate=g.expand(5, 64).contiguous()), ValueError),   # 12 rows
            ((x, y, w), dict(gate=g[:, :32].contiguous()), ValueError),
            ((x.view(3, 4, 64), y.view(3, 4, 64)), dict(gate=g.expand(4, 64).contiguous()),
             ValueError),                                                      # not the leading size
            ((x, y), dict(post_weight=w, post_norm=False), ValueError),
            ((x, y), dict(scale=math.nan), m.FlpError), ((x, y), dict(scale=math.inf), m.FlpError),
            ((x, y), dict(eps=-1.0), m.FlpError)]:
        with pytest.raises(err):
            m.residual_rms_norm(*args, **kw)
    half = torch.ones(64, device="cuda", dtype=F16)
    with pytest.raises(TypeError):
        m.residual_rms_norm(x.half(), y.half(), half, gate=g)  # fp16 and fp32 parameters
    with pytest.raises(m.FlpError, match="UNSUPPORTED_SHAPE"):
        m.rms_norm(torch.zeros(2, 16385, device="cuda"))
    r, n = m.residual_rms_norm(x.clone().requires_grad_(True), y)
    gx, = torch.autograd.grad(n, [r.grad_fn.next_functions[0][0].variable], torch.ones_like(n),
                              create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        gx.sum().backward()


@pytest.mark.parametrize("which", ["x", "y", "weight", "gate"])
def test_data_exchanged_before_the_backward_is_refused(which):
    m = flp()
    a = make(12, 64, F32, F32, 16, 3, True, True)
    leaves = {k: a[k].clone().requires_grad_(True) for k in ("x", "y", "weight", "gate")}
    r, n = m.residual_rms_norm(leaves["x"], leaves["y"], leaves["weight"], gate=leaves["gate"])
    leaves[which].data = torch.zeros(3, 2, device="cuda")
    with pytest.raises((ValueError, RuntimeError)):
        n.sum().backward()


def test_streams_and_graphs():
    m = flp()
    a = make(700, 1345, BF16, F32, 17, 7, True, True)
    names = ["x", "y", "weight", "post_weight", "gate"]
    leaves = [a[k].clone().requires_grad_(True) for k in names]

    def step():
        r, n = m.residual_rms_norm(*leaves, scale=0.7)
        return (r, n) + torch.autograd.grad([r, n], leaves, [a["grad_r"], a["grad_n"]])
    ref = [t.detach().clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for u, v in zip(ref, got):
        assert torch.equal(u, v)
    del got
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        with torch.no_grad():
            leaves[0].mul_(0.5), leaves[1].add_(0.25), leaves[4].mul_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.detach().clone() for t in held]
        for u, v in zip(kept, step()):
            assert torch.equal(u, v), k
        torch.cuda.synchronize()


def test_more_elements_than_32_bits_count():
    """2^31 elements and more in x alone: the first and the last rows."""
    m = flp()
    N, D = (1 << 31) // 1024 + 5, 1024
    x = torch.ones(N, D, dtype=BF16, device="cuda")
    y = torch.full((N, D), 2.0, dtype=BF16, device="cuda")
    x[-1], y[-1] = 3.0, 5.0
    r, n, rstd, _ = m.residual_rms_norm_forward(x, y, eps=0.0)
    assert bool((r[:3] == 3).all()) and bool((r[-1] == 8).all()) and bool((r[-2] == 3).all())
    assert bool((n[-3:] == 1).all())
    dx, dy, *_ = m.residual_rms_norm_backward(y, None, x, y, rstd, need_weight=False)
    assert bool((dx[-1] == 5).all()) and bool((dy[-2] == 2).all())
