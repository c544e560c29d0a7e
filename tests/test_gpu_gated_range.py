"""fp16 gradients of the gated projection with upstream gradients far from 1: dz and du, which the
matrix instructions take in fp16, keep their bits where they lie below its normal range, and stay
finite where they pass its largest value."""
import math

import pytest
import torch

from gpu_common import flp, say
from test_gpu_gated import act

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = 2.0 ** -11  # half a step of fp16, relative


def make(N, D, F, seed, size, up, dtype=F16):
    """z and u around 1 from x of `size` and weights of 1 / size; upstream gradients around `up`."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, D, generator=g) * size
    wg, wu = (torch.randn(F, D, generator=g) / (size * math.sqrt(D)) for _ in range(2))
    go = torch.randn(N, F, generator=g) * up
    return tuple(t.to(dtype).cuda() for t in (x, wg, wu, go))


def gradients(x, wg, wu, go, name="silu", **need):
    m = flp()
    _, saved = m.gated_linear_forward(x, wg, wu, name)
    return m.gated_linear_backward(go, saved, x, wg, wu, name, **need)


def reference(x, wg, wu, go, name="silu"):
    """The gradients in 64 bits, and the roots of their terms' squares summed."""
    x, wg, wu, go = (t.double() for t in (x, wg, wu, go))
    z, u = x @ wg.T, x @ wu.T
    f, slope, _ = act(name, z)
    dz, du = go * u * slope, go * z * f
    out = dz @ wg + du @ wu, dz.T @ x, du.T @ x
    size = ((dz ** 2 @ wg ** 2 + du ** 2 @ wu ** 2).sqrt(), (dz.T ** 2 @ x ** 2).sqrt(),
            (du.T ** 2 @ x ** 2).sqrt())
    return out, size


def check(got, ref, size):
    """The roundings of dz and du are independent and at most half a step of their terms, then the
    result's own half step; below 2^-14, where the result itself has fewer bits, its step."""
    for k, (v, r, s) in enumerate(zip(got, ref, size)):
        if v is None:
            continue
        err = (v.double() - r).abs() - 2.0 ** -25
        off = float(err.clamp(min=0).norm()) / (float(r.norm()) + 2 * float(s.norm()))
        say(f"  gradient {k}: {off / HALF:.2f} half steps")
        assert off <= HALF, (k, off)


@pytest.mark.parametrize("up", [1.0, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 3e-7])
@pytest.mark.parametrize("N,D,F", [(1024, 64, 200), (40, 96, 1500), (1000, 544, 515), (3000, 64, 64),
                                   (7, 32, 33)])
def test_small_upstream_gradients(N, D, F, up):
    # d_x from large weights, the weights' gradients from large inputs: inside fp16's normal range
    say(f"N={N} D={D} F={F} up={up}")
    for size, need in ((1 / 512, (True, False, False)), (64.0, (False, True, True))):
        a = make(N, D, F, N + F, size, up)
        got = gradients(*a, need_input=need[0], need_gate=need[1], need_up=need[2])
        ref, terms = reference(*a)
        check(got, ref, terms)


@pytest.mark.parametrize("N,D,F", [(30, 64, 64), (700, 64, 64)])
def test_products_above_the_largest_value(N, D, F):
    """z and u around 100, upstream gradients around 400: dz passes 65504, d_x does not."""
    x, wg, wu, go = make(N, D, F, 3, 512.0, 400.0)
    wg, wu = ((w.double() * 100).to(F16) for w in (wg, wu))
    ref, terms = reference(x, wg, wu, go)
    assert float(ref[0].abs().max()) < 65504 and float(terms[0].max()) < 65504
    dx = gradients(x, wg, wu, go, need_gate=False, need_up=False)[0]
    assert bool(dx.isfinite().all())
    check([dx], ref, terms)


def test_infinite_and_nan_rows_stay_by_themselves():
    """They say nothing of the others' size either."""
    a = make(600, 96, 333, 5, 1 / 512, 1e-6)
    clean = gradients(*a, need_gate=False, need_up=False)[0]
    go = a[3].clone()
    go[7, 3], go[8, 4], go[599, 332] = math.inf, math.nan, -math.inf
    dx = gradients(*a[:3], go, need_gate=False, need_up=False)[0]
    rest = [i for i in range(600) if i not in (7, 8, 599)]
    assert torch.equal(dx[rest], clean[rest])
    assert not bool(dx[[7, 8, 599]].isfinite().any())


def test_zero_gradients_and_few_numbers():
    for N, D, F in ((1, 32, 1), (17, 64, 65)):
        a = make(N, D, F, 6, 1.0, 0.0)
        assert all(not bool(g.any()) for g in gradients(*a))
    # a single product, below the least fp16 value of 2^-24 but for its factor
    x = torch.zeros(1, 32, dtype=F16, device="cuda")
    w = torch.zeros(1, 32, dtype=F16, device="cuda")
    x[0, 0], w[0, 0] = 1.0, 2.0 ** 10
    wu = w * 2.0 ** -24
    go = torch.full((1, 1), 2.0 ** -20, dtype=F16, device="cuda")
    # z = 2^10, u = 2^-14: dz = 2^-34, du = 2^-10; d_x = dz 2^10 + du 2^-14 = 2^-24 + 2^-24
    dx, dwg, dwu = gradients(x, w, wu, go)
    assert float(dx[0, 0]) == 2.0 ** -23 and float(dwu[0, 0]) == 2.0 ** -10
    assert float(dwg[0, 0]) == 0.0   # 2^-34


def test_same_rows_among_batches_and_replayed():
    m = flp()
    x, wg, wu, go = make(512, 64, 300, 7, 1 / 512, 1e-5)
    go[0, 0] = 2e-4  # the largest, in every batch
    whole = gradients(x, wg, wu, go)
    part = gradients(x[:100].contiguous(), wg, wu, go[:100].contiguous())
    assert torch.equal(whole[0][:100], part[0])
    leaves = [t.clone().requires_grad_(True) for t in (x, wg, wu)]

    def step():
        return torch.autograd.grad(m.gated_linear(*leaves), leaves, go)
    for a, b in zip(step(), whole):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for factor in (1.0, 2.0 ** -4, 2.0 ** 9, 2.0 ** -3):
        go.mul_(factor)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b), factor
        torch.cuda.synchronize()
