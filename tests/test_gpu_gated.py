"""The gated projection against its formula in 64 bits: every type and activation, sizes around
the tiles and the padding, one row and thousands, both gradients of the weights from one tensor,
rows that do not depend on each other, streams and graphs."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative
ACTS = ["silu", "gelu", "gelu_tanh"]


def half_step(t):
    return torch.finfo(t).eps / 2


def rounding(t, ref):
    """Half a step of the type at ref."""
    return half_step(t) * ref.abs().clamp(min=torch.finfo(t).smallest_normal)


def make(N, D, F, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, D, generator=g).to(dtype)
    wg = (torch.randn(F, D, generator=g) * std / math.sqrt(D)).to(dtype)
    wu = (torch.randn(F, D, generator=g) * std / math.sqrt(D)).to(dtype)
    go = torch.randn(N, F, generator=g).to(dtype)
    return tuple(t.cuda() for t in (x, wg, wu, go))


def act(name, z):
    """act(z) / z, act'(z) and a bound on |act''|, in 64 bits."""
    if name == "gelu":
        f = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return f, f + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), 0.8
    if name == "silu":
        f = torch.sigmoid(z)
        return f, f * (1 + z * (1 - f)), 0.5
    a, b = 2 * math.sqrt(2 / math.pi), 0.044715
    f = torch.sigmoid(a * (z + b * z ** 3))
    return f, f + z * f * (1 - f) * a * (1 + 3 * b * z * z), 0.85


# |act''|: silu 2 s (1 - s) at 0 is 1/2, its largest.  gelu (2 - z^2) phi(z) at 0 is 0.798.
# gelu_tanh: at 0 it is a / 2 = 0.798, and it stays within 0.03 of gelu's.

# fp32's own error in the factors.  exp(v) by exp2 of a rounded product: (|v| + 2) U relative, so
# the logistic function (|v| + 6) U, and |v| f(v) z stays below 0.28 |z| where v < 0 (for v > 0
# the factor's error is that of exp(-v) <= 1 times |v| exp(-v) <= 0.37): 8 U of max(f, .28) z.
# gelu's erfc has 16 ulp at most, and its argument's rounding |z|^2 U relative on the far side,
# where z^2 f < 0.2.  gelu_tanh: v is rounded five times, |v| <= 1.6 |z| (1 + 0.05 z^2).
ACT_ERR = 40 * U


def reference(x, wg, wu, go, name):
    """Values, and bounds on the fp32 error and on the roundings of dz and du."""
    t = x.dtype
    X, G, P, go = (v.double() for v in (x, wg, wu, go))
    D, F, N = x.shape[1], wg.shape[0], x.shape[0]
    # products: sums of D terms in fp32, every partial sum rounded once
    z, u = X @ G.T, X @ P.T
    ez, eu = (D + 2) * U * (X.abs() @ G.abs().T), (D + 2) * U * (X.abs() @ P.abs().T)
    f, slope, bend = act(name, z)
    a = z * f
    ea = 1.2 * ez + ACT_ERR * (z.abs() + 1e-30)   # |act'| <= 1.13
    out = dict(out=a * u)
    tol = dict(out=ea * u.abs() + a.abs() * eu + ea * eu + 2 * U * (a * u).abs())
    r = half_step(t) if t != F32 else 0.0
    tiny = torch.finfo(t).smallest_normal * r
    # the backward sees act(z) and u act'(z) in 24 bits (16 of them mantissa), and rounds dz and du
    k = 2.0 ** -16 if t != F32 else 0.0
    eslope = bend * ez + ACT_ERR * (1 + z.abs())
    dz, du = go * u * slope, go * a
    edz = go.abs() * (eu * slope.abs() + u.abs() * eslope + eu * eslope) + (k + 3 * U) * dz.abs()
    edu = go.abs() * ea + (k + 2 * U) * du.abs()
    edz, edu = edz + r * (dz.abs() + edz) + tiny, edu + r * (du.abs() + edu) + tiny
    out["dx"] = dz @ G + du @ P
    out["out_terms"] = a * u if t == F32 else torch.zeros(1)
    out["dx_terms"] = (dz ** 2 @ G ** 2 + du ** 2 @ P ** 2).sqrt()
    out["dwg_terms"], out["dwu_terms"] = (dz.T ** 2 @ X ** 2).sqrt(), (du.T ** 2 @ X ** 2).sqrt()
    tol["dx"] = edz @ G.abs() + edu @ P.abs() + (2 * F + 8) * U * (dz.abs() @ G.abs() + du.abs() @ P.abs())
    out["dwg"], out["dwu"] = dz.T @ X, du.T @ X
    tol["dwg"] = edz.T @ X.abs() + (N + 2) * U * (dz.abs().T @ X.abs())
    tol["dwu"] = edu.T @ X.abs() + (N + 2) * U * (du.abs().T @ X.abs())
    return out, tol


def run(x, wg, wu, go, name):
    m = flp()
    out, saved = m.gated_linear_forward(x, wg, wu, name)
    plain, none = m.gated_linear_forward(x, wg, wu, name, return_saved=False)
    assert none is None and torch.equal(out.view(torch.uint8), plain.view(torch.uint8))
    dx, dwg, dwu = m.gated_linear_backward(go, saved, x, wg, wu, name)
    return dict(out=out, dx=dx, dwg=dwg, dwu=dwu)


def compare(x, wg, wu, go, name):
    got = run(x, wg, wu, go, name)
    ref, tol = reference(x, wg, wu, go, name)
    for k, v in got.items():
        bound = rounding(v.dtype, ref[k]) * (1 + 2.0 ** -6) + tol[k] * (1 + 2.0 ** -6)
        worst = float(((v.double() - ref[k]).abs() / bound).max())
        # The bounds add absolute values; what is typical must not hide behind them.  The roundings
        # of dz and du are independent, at most half a step of each term: their sum's size is that
        # of the terms' squares (with a factor 2 for few elements), then the result's rounding.
        h = half_step(v.dtype) if v.dtype != F32 else 1e-6
        size = float(ref[k].norm()) + 2 * float(ref[k + "_terms"].norm())
        off = float((v.double() - ref[k]).norm()) / max(size, 1e-300)
        say(f"  {k}: worst error {worst:.3f} of its bound, typical {off / h:.2f}")
        assert worst <= 1.0, (k, worst)
        assert off <= h, (k, off)
    return got


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N,D,F", [(1, 32, 1), (1, 64, 2), (2, 96, 31), (7, 32, 33), (16, 160, 64),
                                   (17, 64, 65), (33, 2688, 100), (65, 128, 127), (129, 96, 300),
                                   (200, 288, 771), (257, 224, 513), (300, 1344, 1025)])
def test_sizes(N, D, F, dtype, name):
    say(f"N={N} D={D} F={F} {dtype} {name}")
    compare(*make(N, D, F, dtype, N + D + F), name)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N,D,F", [(1, 2688, 7168), (5, 2688, 1000), (1000, 544, 3587),
                                   (2048, 256, 1024), (2049, 256, 1024), (4100, 96, 2500)])
def test_larger_sizes(N, D, F, dtype):
    say(f"N={N} D={D} F={F} {dtype}")
    compare(*make(N, D, F, dtype, N + F), "silu")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_arguments(name, dtype):
    """z of up to hundreds on both sides: the factor ends at 0 and 1 without a NaN."""
    x, wg, wu, go = make(40, 64, 130, dtype, 3, std=60.0)
    wu = (wu.double() / 60).to(dtype)
    got = run(x, wg, wu, go, name)
    ref, _ = reference(x, wg, wu, go, name)
    for k, v in got.items():
        assert bool(v.isfinite().all()), k
        assert float((v.double() - ref[k]).norm() / ref[k].norm()) <= 4 * half_step(dtype) + 1e-5


@pytest.mark.parametrize("big", [2.0 ** 65, 2.0 ** 70, 2.0 ** 120])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ACTS)
def test_arguments_whose_squares_pass_fp32(name, dtype, big):
    """act(z) is z or 0 there and its slope 1 or 0, exactly."""
    m = flp()
    x = torch.zeros(2, 32, dtype=dtype, device="cuda")
    x[0, 0], x[1, 0], x[:, 1] = big, -big, 1.0
    wg, wu = (torch.zeros(1, 32, dtype=dtype, device="cuda") for _ in range(2))
    wg[0, 0] = wu[0, 1] = 1.0
    out, saved = m.gated_linear_forward(x, wg, wu, name)
    assert out.view(-1).tolist() == [big, 0.0]
    go = torch.ones_like(out)
    dx = m.gated_linear_backward(go, saved, x, wg, wu, name, need_gate=False, need_up=False)[0]
    assert dx[:, 0].tolist() == [1.0, 0.0] and dx[:, 1].tolist() == [big, 0.0]


def test_infinite_and_nan_rows_stay_by_themselves():
    x, wg, wu, go = make(70, 96, 200, BF16, 4)
    clean = run(x, wg, wu, go, "silu")
    y = x.clone()
    y[3, 5], y[69, 0] = math.inf, math.nan
    got = run(y, wg, wu, go, "silu")
    ok = [i for i in range(70) if i not in (3, 69)]
    for k in ("out", "dx"):
        assert torch.equal(got[k][ok], clean[k][ok])
    assert bool(got["out"][69].isnan().all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rows_do_not_depend_on_each_other(dtype):
    x, wg, wu, go = make(3000, 224, 300, dtype, 5)
    m = flp()
    for many in (600, 3000):   # d_x in slabs, and in one walk
        whole = run(x[:many].contiguous(), wg, wu, go[:many].contiguous(), "silu")
        part = run(x[:many - 300].contiguous(), wg, wu, go[:many - 300].contiguous(), "silu")
        for k in ("out", "dx"):
            assert torch.equal(whole[k][:many - 300], part[k]), (many, k)
        again = run(x[:many].contiguous(), wg, wu, go[:many].contiguous(), "silu")
        for k in whole:
            assert torch.equal(whole[k], again[k]), k
    moved = torch.cat([x[1000:1020], x[:40]])
    out = m.gated_linear(moved, wg, wu)
    assert torch.equal(out[20:], m.gated_linear(x[:40].contiguous(), wg, wu))


@pytest.mark.parametrize("few,many", [(1, 512), (513, 1024), (1025, 2048), (2049, 2100)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_d_x_within_a_class_of_batches(dtype, few, many):
    """The batch sizes between which d_x has the same slabs, from their smallest to their largest."""
    x, wg, wu, go = make(many, 672, 1500, dtype, 6)
    whole = run(x, wg, wu, go, "silu")
    part = run(x[-few:].contiguous(), wg, wu, go[-few:].contiguous(), "silu")
    for k in ("out", "dx"):
        assert torch.equal(whole[k][-few:], part[k]), k


def test_halves_of_one_weight_and_odd_offsets():
    m = flp()
    x, wg, wu, go = make(50, 96, 129, BF16, 6)
    both = torch.cat([wg, wu])
    ref = run(x, wg, wu, go, "gelu")
    out, saved = m.gated_linear_forward(x, both[:129], both[129:], "gelu")
    assert torch.equal(out, ref["out"])
    flat = torch.empty(go.numel() + 3, dtype=BF16, device="cuda")[3:]
    moved = flat.copy_(go.reshape(-1)).view(go.shape)
    dx, dwg, dwu = m.gated_linear_backward(moved, saved, x, both[:129], both[129:], "gelu")
    for k, v in (("dx", dx), ("dwg", dwg), ("dwu", dwu)):
        assert torch.equal(v, ref[k]), k
    # an output off the grid, and what surrounds it
    from lm_head_selected_bf16_amd import _abi
    big = torch.full((50 * 129 + 16,), 7.0, dtype=BF16, device="cuda")
    at = big[5:5 + 50 * 129]
    assert m.flp_gated_linear_forward(50, 96, 129, _abi.FLP_BF16, x.data_ptr(), wg.data_ptr(),
                                      wu.data_ptr(), m.FLP_ACT_GELU, at.data_ptr(), 0,
                                      torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(at.view(50, 129), ref["out"])
    assert bool((big[:5] == 7).all()) and bool((big[5 + 50 * 129:] == 7).all())


@pytest.mark.parametrize("need", ["x", "w_gate", "w_up", "all"])
def test_autograd_gives_each_leaf_its_gradient(need):
    m = flp()
    x, wg, wu, go = make(66, 64, 130, F16, 7)
    leaves = [t.clone().requires_grad_(need in (k, "all"))
              for k, t in (("x", x), ("w_gate", wg), ("w_up", wu))]
    out = m.gated_linear(*leaves, activation="gelu_tanh")
    wanted = [t for t in leaves if t.requires_grad]
    got = torch.autograd.grad(out, wanted, go)
    ref = run(x, wg, wu, go, "gelu_tanh")
    names = [k for k, t in zip(("dx", "dwg", "dwu"), leaves) if t.requires_grad]
    assert torch.equal(out, ref["out"])
    for k, g in zip(names, got):
        assert torch.equal(g, ref[k]), k


def test_one_weight_for_both():
    """The same leaf as w_gate and w_up gets both gradients."""
    m = flp()
    x, wg, _, go = make(30, 64, 70, F32, 8)
    w = wg.clone().requires_grad_(True)
    g, = torch.autograd.grad(m.gated_linear(x, w, w), [w], go)
    ref = run(x, wg, wg, go, "silu")
    assert torch.equal(g, ref["dwg"] + ref["dwu"])


@pytest.mark.parametrize("name", ACTS)
def test_gradient_against_differences(name):
    """fp32 against central differences of the formula in 64 bits."""
    x, wg, wu, go = make(20, 32, 45, F32, 9)
    got = run(x, wg, wu, go, name)
    v = [t.double() for t in (x, wg, wu)]

    def value(a, b, c):
        z = a @ b.T
        return float((z * act(name, z)[0] * (a @ c.T) * go.double()).sum())
    h = 1e-5
    g = torch.Generator().manual_seed(10)
    for j, k in enumerate(("dx", "dwg", "dwu")):
        way = torch.randn(v[j].shape, generator=g).double().cuda()
        up, down = [list(v) for _ in range(2)]
        up[j], down[j] = v[j] + h * way, v[j] - h * way
        num = (value(*up) - value(*down)) / (2 * h)
        ana = float((got[k].double() * way).sum())
        assert abs(num - ana) <= 1e-5 * float((got[k].double() * way).abs().sum()) + 1e-6, k


def test_empty_batch_and_leading_shapes():
    m = flp()
    x, wg, wu, go = make(12, 64, 40, F32, 11)
    w1, w2 = wg.clone().requires_grad_(True), wu.clone().requires_grad_(True)
    e = torch.empty(0, 64, device="cuda", requires_grad=True)
    out = m.gated_linear(e, w1, w2)
    assert out.shape == (0, 40)
    ge, g1, g2 = torch.autograd.grad(out, [e, w1, w2], torch.empty_like(out))
    assert ge.shape == (0, 64) and not bool(g1.any()) and not bool(g2.any())
    ref = m.gated_linear(x, wg, wu)
    assert torch.equal(m.gated_linear(x.view(3, 4, 64), wg, wu).view(12, 40), ref)
    assert torch.equal(m.gated_linear(x[0], wg, wu), ref[0])


def test_refusals():
    m = flp()
    x, wg, wu, go = make(12, 64, 40, F32, 12)
    for args, kw, err in [((x.double(), wg, wu), {}, TypeError), ((x, wg.half(), wu), {}, TypeError),
                          ((x, wg, wu.half()), {}, TypeError),
                          ((x, wg[:, :32], wu[:, :32]), {}, ValueError),
                          ((x, wg, wu[:20]), {}, ValueError), ((x.cpu(), wg, wu), {}, ValueError),
                          ((x, wg.cpu(), wu), {}, ValueError), ((x.t(), wg, wu), {}, ValueError),
                          ((x, wg, wu), dict(activation="relu"), ValueError),
                          ((x, wg, wu, 3), {}, ValueError)]:
        with pytest.raises(err):
            m.gated_linear(*args, **kw)
    with pytest.raises(m.FlpError, match="UNSUPPORTED_SHAPE"):  # D not a multiple of 32
        m.gated_linear(torch.zeros(2, 48, device="cuda"), torch.zeros(8, 48, device="cuda"),
                       torch.zeros(8, 48, device="cuda"))
    with pytest.raises(m.FlpError, match="MISALIGNED"):
        m.gated_linear(torch.zeros(12 * 64 + 1, device="cuda")[1:].view(12, 64), wg, wu)
    out, saved = m.gated_linear_forward(x, wg, wu)
    with pytest.raises(ValueError):
        m.gated_linear_backward(go, saved[:100], x, wg, wu)
    with pytest.raises(ValueError):
        m.gated_linear_backward(go[:, :20], saved, x, wg, wu)
    y = x.clone().requires_grad_(True)
    gx, = torch.autograd.grad(m.gated_linear(y, wg, wu), [y], go, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        gx.sum().backward()
    for k in range(3):
        leaves = [t.clone().requires_grad_(True) for t in (x, wg, wu)]
        out = m.gated_linear(*leaves)
        leaves[k].data = torch.zeros(5, 3, device="cuda")
        with pytest.raises((ValueError, RuntimeError)):
            out.sum().backward()


def test_streams_and_graphs():
    m = flp()
    x, wg, wu, go = make(700, 96, 333, BF16, 13)
    leaves = [t.clone().requires_grad_(True) for t in (x, wg, wu)]

    def step():
        out = m.gated_linear(*leaves)
        return (out,) + torch.autograd.grad(out, leaves, go)
    ref = [t.detach().clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    del got
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        with torch.no_grad():
            leaves[0].mul_(0.5), leaves[1].mul_(-1.5), leaves[2].add_(0.01)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.detach().clone() for t in held]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b), k
        torch.cuda.synchronize()


def test_more_elements_than_32_bits_count():
    """An output of 2^31 elements and more: its first and last rows."""
    m = flp()
    N, F = (1 << 31) // 8192 + 3, 8192
    g = torch.Generator().manual_seed(14)
    x = torch.randn(N, 32, generator=g).to(BF16).cuda()
    wg, wu = (torch.randn(F, 32, generator=g).div(6).to(BF16).cuda() for _ in range(2))
    out = m.gated_linear(x, wg, wu)
    for rows in (slice(0, 5), slice(N - 5, N)):
        part = x[rows].contiguous()
        assert torch.equal(out[rows], m.gated_linear(torch.cat([part] * 30), wg, wu)[:5])
