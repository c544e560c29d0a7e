"""The AdamW step against its formula in 64 bits: every mix of types, states in 32 bits and in 8,
sizes around the 256 elements of a scale and the 2048 of a tile, many tensors in one call, views
off the 16-byte grid, gradients that are not finite, counters on the device, graphs and streams."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative
BETAS, EPS, LR, DECAY = (0.9, 0.95), 1e-8, 1e-2, 0.1
SIZES = [1, 7, 255, 256, 257, 2047, 2048, 2049, 5003, 70001]


def rounding(t, ref):
    """Half a step of the type at ref."""
    f = torch.finfo(t)
    return (f.eps / 2) * ref.abs().clamp(min=f.smallest_normal)


def held(codes, scale):
    """What 8-bit states stand for, in 64 bits."""
    n = codes.numel()
    return (codes.reshape(-1).double() * scale.double().repeat_interleave(256)[:n]).view(codes.shape)


def snapshot(state, k):
    m, v = state.exp_avg[k], state.exp_avg_sq[k]
    if state.exp_avg_scale is None:
        return m.double(), v.double()
    return held(m, state.exp_avg_scale[k]), held(v, state.exp_avg_sq_scale[k]) ** 2


def formula(p, g, m, v, t, lr, decay, betas=BETAS, eps=EPS):
    """The step in 64 bits, and bounds on what fp32 makes of m, v and the parameter."""
    b1, b2 = betas
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    c2 = math.sqrt(1 - b2 ** t)
    denom = v1.sqrt() / c2 + eps
    rate = lr / (1 - b1 ** t)
    p1 = p * (1 - lr * decay) - rate * (m1 / denom)
    # m: the constants, g times its factor, the product, a decoded m0 and the sum are rounded once
    em = 4 * U * (b1 * m.abs() + (1 - b1) * g.abs())
    # v (all terms positive): g twice, its square, the product with a constant, the constants, a
    # decoded root twice and its square, the sum
    ev = 8 * U * v1 + 2.0 ** -149
    # the root has half of that and its own rounding; its scale, eps and the sum one each, the
    # quotient, the rate and their product one each
    ratio = (m1 / denom).abs()
    ep = rate * (em / denom + 11 * U * ratio) + 3 * U * p.abs() + 2 * U * p1.abs()
    return p1, m1, v1, em, ev, ep


def check(name, got, ref, tol):
    got = got.double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    worst = float(torch.where(same, 0.0, (got - ref).abs() / tol).max()) if got.numel() else 0.0
    assert worst <= 1.0, (name, worst)
    return worst


def check_codes(name, codes, scale, ref, err, divisor):
    """Codes of ref, which fp32 holds up to err: half a step of e4m3 at the ratio, and where a
    positive divisor was raised to the smallest code, at most that."""
    n = ref.numel()
    blocks = torch.nn.functional.pad(ref.reshape(-1), (0, -n % 256)).view(-1, 256)
    top = blocks.abs().amax(1).clamp(min=2.0 ** -100)
    top_err = torch.nn.functional.pad(err.reshape(-1), (0, -n % 256)).view(-1, 256).amax(1)
    check(name + " scale", scale, top / 448, top / 448 * 3 * U + top_err / 448)
    unit = scale.double().repeat_interleave(256)[:n]
    got, r, e = codes.reshape(-1).double(), ref.reshape(-1) / unit, err.reshape(-1) / unit
    tol = (r.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 2.0 ** -4) + r.abs() * 4 * U + e
    if divisor:
        tol = torch.where((r > 0) & (r < 2.0 ** -9), torch.full_like(tol, 2.0 ** -9), tol)
        assert bool((got[ref.reshape(-1) > 0] > 0).all()), "a positive root became 0"
        assert bool((got[ref.reshape(-1) == 0] == 0).all())
    check(name + " codes", codes.reshape(-1), r, tol)


def make(sizes, pdt, gdt, seed):
    g = torch.Generator().manual_seed(seed)
    params = [(torch.randn(n, generator=g) * 0.5).to(pdt).cuda() for n in sizes]

    def grads():
        # sizes that differ by e^3 within a block
        return [(torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))
                 * 0.05).to(gdt).cuda() for n in sizes]
    return params, grads


def step_and_compare(params, grads, state, t, decay, gs=None, lr=LR, device=False):
    before = []
    for k, p in enumerate(params):
        w = state.master[k] if state.master and state.master[k] is not None else p
        before.append((w.double().clone(),) + tuple(x.clone() for x in snapshot(state, k)))
    at, rate = t, lr
    if device:
        at, rate = torch.tensor([t], device="cuda"), torch.tensor(lr, device="cuda")
        lr = float(rate)  # as float32 holds it
    scale = None if gs is None else torch.tensor([gs], device="cuda")
    flp().adamw_step(params, grads, state, at, rate, betas=BETAS, eps=EPS, weight_decay=decay,
                     grad_scale=scale)
    factor = 1.0 if gs is None else float(scale)
    for k, (p, g) in enumerate(zip(params, grads)):
        w0, m0, v0 = before[k]
        p1, m1, v1, em, ev, ep = formula(w0, g.double() * factor, m0, v0, t, lr, decay[k])
        if state.master and state.master[k] is not None:
            check("master", state.master[k], p1, ep)
            assert torch.equal(p, state.master[k].to(p.dtype))
        else:
            check("param", p, p1, ep + rounding(p.dtype, p1) * (1 + 2 ** -7))
        if state.exp_avg_scale is None:
            check("m", state.exp_avg[k], m1, em)
            check("v", state.exp_avg_sq[k], v1, ev)
        else:
            check_codes("m", state.exp_avg[k], state.exp_avg_scale[k], m1, em, False)
            root = v1.sqrt()
            check_codes("v", state.exp_avg_sq[k], state.exp_avg_sq_scale[k], root,
                        6 * U * root + 1e-30, True)


MIXES = [(F32, F32, False), (BF16, BF16, False), (BF16, BF16, True), (BF16, F32, False),
         (BF16, F32, True), (F16, F16, False), (F16, F16, True), (F16, F32, False),
         (F16, F32, True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt,master", MIXES)
def test_steps(pdt, gdt, master, bits):
    params, grads = make(SIZES, pdt, gdt, 1)
    state = flp().adamw_state(params, bits=bits, master=master)
    decay = [DECAY if k % 2 else 0.0 for k in range(len(SIZES))]
    for t in (1, 2, 3):
        step_and_compare(params, grads(), state, t, decay)


@pytest.mark.parametrize("bits", [32, 8])
def test_factors_and_counters_on_the_device(bits):
    params, grads = make([300, 4099], BF16, BF16, 2)
    state = flp().adamw_state(params, bits=bits, master=True)
    for t in (1, 7, 123457):
        step_and_compare(params, grads(), state, t, [0.0, DECAY], gs=0.37, device=True)


def test_late_and_early_steps_of_a_beta_near_one():
    """1 - b2^t in 64 bits: fp32 would lose it to a part in 20 at b2 = 1 - 1e-6 and t = 1."""
    m = flp()
    for t in (1, 2, 10 ** 6, 10 ** 12):
        p, g = torch.zeros(8, device="cuda"), torch.full((8,), 0.5, device="cuda")
        betas = (0.9, 1 - 1e-6)
        for at in (t, torch.tensor([t], device="cuda")):
            state = m.adamw_state([p])
            p.zero_()
            m.adamw_step([p], [g], state, at, 1.0, betas=betas, eps=0.0, weight_decay=0.0)
            z = torch.zeros(8, dtype=torch.float64, device="cuda")
            p1, _, _, _, _, ep = formula(z, g.double(), z, z, t, 1.0, 0.0, betas, 0.0)
            # fp32 holds 1 - b2 and 1 - b1 (computed in 64 bits) to half a step: in the bound
            check("param", p, p1, ep)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_of_every_type_at_once(bits):
    """130 tensors (several launches) of nine mixes in one call: the bits of a call each."""
    m = flp()
    sizes = [1 + (k * 397) % 3001 for k in range(130)]
    ps, gs = [], []
    for k, n in enumerate(sizes):
        pdt, gdt, _ = MIXES[k % 9]
        p, g = make([n], pdt, gdt, 100 + k)
        ps += p
        gs += g()
    copies = [k % 9 for k in range(130)]

    def fresh():
        s = m.adamw_state(ps, bits=bits, master=True)
        return s._replace(master=[w if MIXES[c][2] else None for w, c in zip(s.master, copies)])
    a, b = fresh(), fresh()
    pa, pb = [p.clone() for p in ps], [p.clone() for p in ps]
    decay = [0.01 * (k % 3) for k in range(130)]
    m.adamw_step(pa, gs, a, 1, LR, weight_decay=decay)
    for k in range(130):
        one = m.AdamWState(*[None if f is None else [f[k]] for f in b])
        m.adamw_step([pb[k]], [gs[k]], one, 1, LR, weight_decay=decay[k])
    for x, y in zip(pa, pb):
        assert torch.equal(x, y)
    for f, h in zip(a, b):
        for x, y in zip(f or [], h or []):
            assert x is y is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_views_off_the_grid_and_what_surrounds_them(pdt, gdt, bits):
    m = flp()
    n, off = 3001, 3
    params, grads = make([n + 2 * off], pdt, gdt, 5)
    whole_p, whole_g = params[0], grads()[0]
    base = m.adamw_state([whole_p], bits=bits)
    cut = lambda t: t.view(-1)[off:off + n]  # noqa: E731
    for t in (base.exp_avg[0], base.exp_avg_sq[0]):
        t.view(torch.uint8).fill_(0x11)
    kept = [t.clone() for t in (whole_p, base.exp_avg[0], base.exp_avg_sq[0])]
    scales = [torch.full((14,), 3.0, device="cuda") for _ in range(2)] if bits == 8 else None
    aligned = m.AdamWState([cut(base.exp_avg[0]).clone()], [cut(base.exp_avg_sq[0]).clone()],
                           scales and [scales[0][1:13].clone()],
                           scales and [scales[1][1:13].clone()])
    views = m.AdamWState([cut(base.exp_avg[0])], [cut(base.exp_avg_sq[0])],
                         scales and [scales[0][1:13]], scales and [scales[1][1:13]])
    p2 = cut(whole_p).clone()
    m.adamw_step([cut(whole_p)], [cut(whole_g)], views, 3, LR)
    m.adamw_step([p2], [cut(whole_g).clone()], aligned, 3, LR)
    assert torch.equal(cut(whole_p), p2)
    for whole, one, was in ((base.exp_avg[0], aligned.exp_avg[0], kept[1]),
                            (base.exp_avg_sq[0], aligned.exp_avg_sq[0], kept[2])):
        assert torch.equal(cut(whole).view(torch.uint8), one.view(torch.uint8))
        assert torch.equal(whole[:off].view(torch.uint8), was[:off].view(torch.uint8))
        assert torch.equal(whole[off + n:].view(torch.uint8), was[off + n:].view(torch.uint8))
    assert torch.equal(whole_p[:off], kept[0][:off])
    assert torch.equal(whole_p[off + n:], kept[0][off + n:])
    if scales:
        for s in scales:
            assert float(s[0]) == 3.0 and float(s[13]) == 3.0


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_gradient_that_is_not_finite(bad, bits):
    """It reaches its element (in 8 bits: the states of its block), and no other's bits."""
    m = flp()
    params, grads = make([1024], F32, F32, 6)
    g = grads()[0]
    p, q = params[0].clone(), params[0].clone()
    a, b = m.adamw_state([p], bits=bits), m.adamw_state([q], bits=bits)
    wrong = g.clone()
    wrong[300] = bad
    m.adamw_step([p], [wrong], a, 1, LR)
    m.adamw_step([q], [g], b, 1, LR)
    others = torch.ones(1024, dtype=torch.bool, device="cuda")
    others[300] = False
    assert torch.equal(p[others], q[others]) and not bool(p[300].isfinite())
    if bits == 8:
        others[256:512] = False
        assert bool(snapshot(a, 0)[0][300].isnan()) and bool(snapshot(a, 0)[1][300].isnan())
    else:
        assert not bool(a.exp_avg[0][300].isfinite())
    for x, y in ((a.exp_avg[0], b.exp_avg[0]), (a.exp_avg_sq[0], b.exp_avg_sq[0])):
        assert torch.equal(x[others].view(torch.uint8), y[others].view(torch.uint8))


def test_small_roots_of_a_block_are_never_divided_away():
    """A block with one gradient of 1 and others of 2^-24: their roots are below the range of the
    codes, and a root of 0 would send them off by lr m / eps once their gradient is 0."""
    m = flp()
    p = torch.zeros(256, device="cuda")
    g = torch.full((256,), 2.0 ** -24, device="cuda")
    g[0] = 1.0
    g[2] = 2.0 ** -10
    g[3] = 0.0
    state = m.adamw_state([p], bits=8)
    m.adamw_step([p], [g], state, 1, LR, weight_decay=0.0)
    codes = state.exp_avg_sq[0].float()
    assert bool((codes[[1, 2] + list(range(4, 256))] >= 2.0 ** -9).all()) and float(codes[3]) == 0
    for t in range(2, 40):
        m.adamw_step([p], [torch.zeros_like(g)], state, t, LR, weight_decay=0.0)
    assert bool((p.abs() <= 12 * LR).all()), float(p.abs().max())
    assert float(p[3]) == 0.0


def test_zeros_stay_zeros():
    m = flp()
    for bits in (32, 8):
        p = torch.zeros(700, device="cuda", dtype=BF16)
        state = m.adamw_state([p], bits=bits, master=True)
        for t in (1, 2):
            m.adamw_step([p], [torch.zeros_like(p)], state, t, LR)
        assert not bool(p.any())
        assert not bool(state.exp_avg[0].float().any()) and not bool(state.exp_avg_sq[0].float().any())


def test_missing_gradients_empty_tensors_and_versions():
    m = flp()
    params, grads = make([10, 0, 20], F32, F32, 8)
    g = grads()
    state = m.adamw_state(params)
    kept = params[0].clone()
    v = [p._version for p in params]
    m.adamw_step(params, [None, g[1], g[2]], state, 1, LR)
    assert torch.equal(params[0], kept) and not bool(state.exp_avg[0].any())
    assert params[0]._version == v[0] and params[2]._version == v[2] + 1
    assert state.exp_avg[2]._version == 1
    assert m.adamw_step([], [], m.AdamWState([], []), 1, LR) is None
    # a parameter that a pending backward has saved
    w = torch.ones(4, device="cuda", requires_grad=True)
    y = (w * w).sum()
    m.adamw_step([w], [torch.ones(4, device="cuda")], m.adamw_state([w]), 1, LR)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_shared_gradient_and_refused_shares():
    m = flp()
    params, grads = make([64, 64], F32, F32, 9)
    g = grads()[0]
    state = m.adamw_state(params)
    m.adamw_step(params, [g, g], state, 1, LR)
    with pytest.raises(m.FlpError, match="INVALID_ARGUMENT"):
        m.adamw_step([params[0], params[0]], [g, g], state, 2, LR)
    with pytest.raises(m.FlpError, match="INVALID_ARGUMENT"):
        m.adamw_step([params[0]], [params[0]], m.adamw_state([params[0]]), 2, LR)
    twice = state._replace(exp_avg_sq=state.exp_avg)
    with pytest.raises(m.FlpError, match="INVALID_ARGUMENT"):
        m.adamw_step(params, [g, g], twice, 2, LR)


def test_python_refusals():
    m = flp()
    p, g = torch.zeros(4, 6, device="cuda"), torch.zeros(4, 6, device="cuda")
    s = m.adamw_state([p])
    for args, err in [
            (([p], [g.t().contiguous()], s, 1, LR), ValueError),        # another shape
            (([p.t()], [g.t()], s, 1, LR), ValueError),                 # not contiguous
            (([p], [g.half()], s, 1, LR), TypeError),
            (([p.double()], [g.double()], s, 1, LR), TypeError),
            (([p], [g.cpu()], s, 1, LR), ValueError),
            (([p], [g], m.adamw_state([p], bits=8)._replace(exp_avg_scale=None), 1, LR), ValueError),
            (([p], [g], m.adamw_state([p], bits=8)._replace(exp_avg=s.exp_avg), 1, LR), TypeError),
            (([p], [g], s._replace(exp_avg=[torch.zeros(5, device="cuda")]), 1, LR), ValueError),
            (([p], [g], s._replace(master=[p.half()]), 1, LR), ValueError),
            (([p], [], s, 1, LR), ValueError),
            (([p], [g], s, torch.ones(2, dtype=torch.int64, device="cuda"), LR), ValueError),
            (([p], [g], s, torch.ones(1, device="cuda"), LR), ValueError),
            (([p], [g], s, 1, torch.ones(1, dtype=torch.float64, device="cuda")), ValueError)]:
        with pytest.raises(err):
            m.adamw_step(*args)
    for kw in (dict(step=0), dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(lr=math.nan),
               dict(weight_decay=math.inf)):
        kw = dict(dict(step=1, lr=LR), **kw)
        with pytest.raises(m.FlpError):
            m.adamw_step([p], [g], s, **kw)
    assert not bool(p.any())


def test_captured_and_replayed_with_its_own_counters():
    m = flp()
    params, grads = make([1000, 2049], BF16, BF16, 11)
    gs = grads()
    eager = [p.clone() for p in params]
    a, b = m.adamw_state(params, bits=8, master=True), m.adamw_state(eager, bits=8, master=True)
    t = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.zeros(1, device="cuda")
    kept = [p.clone() for p in params]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        m.adamw_step(params, gs, a, t, lr)
    for p, k in zip(params, kept):
        assert torch.equal(p, k)  # capturing runs nothing
    for step in (1, 2, 3, 4):
        t.fill_(step)
        lr.fill_(LR / step)
        for g in gs:
            g.mul_(1.5 - 0.25 * step)
        graph.replay()
        torch.cuda.synchronize()
        m.adamw_step(eager, gs, b, torch.tensor([step], device="cuda"),
                     torch.tensor([LR / step], device="cuda"))
        torch.cuda.synchronize()
        for x, y in zip(params + a.master, eager + b.master):
            assert torch.equal(x, y), step
        for f, h in zip(a[:4], b[:4]):
            for x, y in zip(f, h):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_on_another_stream():
    m = flp()
    params, grads = make([70001], F32, F32, 12)
    g = grads()
    q = [p.clone() for p in params]
    a, b = m.adamw_state(params), m.adamw_state(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        h = [x * 2 for x in g]
        m.adamw_step(params, h, a, 1, LR)
    torch.cuda.current_stream().wait_stream(side)
    m.adamw_step(q, [x * 2 for x in g], b, 1, LR)
    assert torch.equal(params[0], q[0])


def test_more_elements_than_32_bits_count():
    """2^31 + 777 elements: the first, the last and those around 2^31."""
    m = flp()
    n = 2 ** 31 + 777
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.full((n,), 0.25, dtype=BF16, device="cuda")
    state = m.adamw_state([p], bits=8)
    m.adamw_step([p], [g], state, 1, 0.5, weight_decay=0.0)
    for part in (slice(0, 300), slice(2 ** 31 - 300, 2 ** 31 + 300), slice(n - 300, n)):
        # m / root = 1 up to fp32's roundings: -0.5 in bfloat16
        assert bool((p[part] == -0.5).all())
        assert bool((state.exp_avg[0][part].float() == 448).all())
    assert bool((state.exp_avg_scale[0] > 0).all())
