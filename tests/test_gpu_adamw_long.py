"""AdamW states in 8 bits over thousands of steps against those in 32 bits: a second moment follows
gradients that shrink and grow beside others of its block, one step moving it by a hundredth of a
code's half step; an m without gradients ends at 0; each code is one of the two around its value."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BLOCKS = 16
PARTS = {"same": (0, 1.0), "tenth": (64, 0.1), "threefold": (128, 3.0), "none": (192, 0.0)}


def pattern():
    """What the gradients of a block's quarters are multiplied by after the first steps."""
    f = torch.empty(256)
    for first, factor in PARTS.values():
        f[first:first + 64] = factor
    return f.repeat(BLOCKS).cuda()


def part(t, name):
    first = PARTS[name][0]
    return t.view(BLOCKS, 256)[:, first:first + 64]


def held(codes, scale):
    return codes.view(-1).double() * scale.double().repeat_interleave(256)[:codes.numel()]


# A held root's error, relative: a rounding moves it by at most s = 1/8 (a code's step), and by s with
# probability |d| / s where the step moves the root's ratio to its block's largest by d; so the
# variance grows by at most s |d| a step, and the error shrinks by 1 - b2 a step.  d is
# (1 - b2) / 2 |g^2 / v - 1|, 0.97 (1 - b2) / 2 on average for normal gradients, and as much again for the
# movement of the largest: a variance of at most s 0.97 / 2 = 0.061, a deviation of 0.25.  (It is
# 0.15: s is 0.09 on average, and the thresholds are spread more evenly than random ones.)
SPREAD = 0.25


@pytest.mark.parametrize("betas,before,after", [
    ((0.9, 0.999), 2000, 7000), ((0.9, 0.99), 400, 1600), ((0.9, 0.97), 200, 800),
    ((0.95, 0.95), 200, 600)])
def test_second_moments_follow_their_gradients(betas, before, after):
    m = flp()
    n = 256 * BLOCKS
    g = torch.Generator(device="cuda").manual_seed(1)
    few, wide = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    a, b = m.adamw_state([few], bits=8), m.adamw_state([wide], bits=32)
    f = pattern()
    for t in range(1, before + after + 1):
        grad = torch.randn(n, generator=g, device="cuda") + 0.3
        if t > before:
            grad *= f
        for p, s in ((few, a), (wide, b)):
            m.adamw_step([p], [grad], s, t, 1e-3, betas=betas, weight_decay=0.0)
    ratio = held(a.exp_avg_sq[0], a.exp_avg_sq_scale[0]) / b.exp_avg_sq[0].double().sqrt()
    for name in ("same", "tenth", "threefold"):
        q = part(ratio, name).reshape(-1).quantile(
            torch.tensor([0.05, 0.5, 0.95], dtype=torch.float64, device="cuda")).tolist()
        say(f"  {betas} {name}: {q}")
        # the median of 1024 and the skew of the spread, sd^2 / 2: 0.01 + 0.03
        assert abs(q[1] - 1) <= 0.1, (name, q)
        assert q[0] >= 1 - 2 * SPREAD and q[2] <= 1 + 2 * SPREAD, (name, q)
        # the parameter's way: its mean over a part (a path's own deviation is SPREAD of it at most,
        # that of 1024 elements' mean a thirty-second of that; 1 / root adds SPREAD^2)
        x, y = part(few, name).double().mean(), part(wide, name).double().mean()
        assert abs(float(x / y) - 1) <= SPREAD ** 2 + 3 * SPREAD / 32, (name, float(x), float(y))


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.95, 0.99), (0.9, 0.95), (0.5, 0.9)])
def test_elements_without_gradients_come_to_rest(betas, spread):
    """Beside elements that have some, with constant size too (the block's scale stands still)."""
    m = flp()
    n = 256 * BLOCKS
    p = torch.zeros(n, device="cuda")
    state = m.adamw_state([p], bits=8)
    g = torch.Generator(device="cuda").manual_seed(7)
    has = (pattern() != 0).float()

    def draw():
        return 1 + spread * torch.randn(n, generator=g, device="cuda")
    for t in range(1, 100):
        m.adamw_step([p], [draw()], state, t, 1e-3, betas=betas, weight_decay=0.0)
    # from 448 to below the least code's half in log(448 * 1024) / (1 - b1) steps; from code 1 to 0 in
    # a visit of the thresholds to 1 - b1 of their range, some 3 / (1 - b1) steps at most
    last = 100 + int((math.log(448 * 1024) + 30) / (1 - betas[0]))
    for t in range(100, last):
        m.adamw_step([p], [draw() * has], state, t, 1e-3, betas=betas, weight_decay=0.0)
    assert not bool(part(state.exp_avg[0].float(), "none").any())
    assert bool((part(state.exp_avg_sq[0].float(), "none") > 0).all())
    was = p.clone()
    for t in range(last, last + 50):
        m.adamw_step([p], [draw() * has], state, t, 1e-3, betas=betas, weight_decay=0.0)
    assert torch.equal(part(p, "none"), part(was, "none"))
    assert bool((part(p, "same") != part(was, "same")).all())


def grid_step(r):
    """The distance of e4m3's values around |r|."""
    return torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)


@pytest.mark.parametrize("pdt,gdt,master", [(F32, F32, False), (BF16, BF16, True), (F16, F32, False)])
def test_codes_are_the_nearest_below_or_above_and_right_on_average(pdt, gdt, master):
    m = flp()
    sizes = [1, 255, 257, 2049, 70001]
    g = torch.Generator().manual_seed(2)
    params = [(torch.randn(n, generator=g) * 0.5).to(pdt).cuda() for n in sizes]
    state = m.adamw_state(params, bits=8, master=master)
    b1, b2 = 0.9, 0.999
    for t in (1, 2, 3, 2 ** 32 + 4):
        grads = [(torch.randn(n, generator=g) * torch.exp(2 * torch.randn(n, generator=g))
                  * 0.05).to(gdt).cuda() for n in sizes]
        old = [[held(c[k], s[k]) for c, s in ((state.exp_avg, state.exp_avg_scale),
                                              (state.exp_avg_sq, state.exp_avg_sq_scale))]
               for k in range(len(sizes))]
        m.adamw_step(params, grads, state, t, 1e-3)
        for k, (m0, r0) in enumerate(old):
            x = grads[k].double()
            root = (b2 * r0 * r0 + (1 - b2) * x * x).sqrt()
            for what, codes, scale, ref, mag in (
                    ("m", state.exp_avg[k], state.exp_avg_scale[k], b1 * m0 + (1 - b1) * x,
                     b1 * m0.abs() + (1 - b1) * x.abs()),
                    ("root", state.exp_avg_sq[k], state.exp_avg_sq_scale[k], root, root)):
                unit = scale.double().repeat_interleave(256)[:ref.numel()]
                r, got = ref / unit, codes.view(-1).double()
                # fp32: eight roundings of the terms, the scale's and the ratio's three
                err = 12 * 2.0 ** -24 * mag / unit
                off = (got - r).abs()
                s = grid_step(r) * (1 + 2.0 ** -20)
                low = (r > 0) & (got == 2.0 ** -9) if what == "root" else torch.zeros_like(r).bool()
                assert bool(((off <= s + err) | (low & (off <= 2.0 ** -9 + err))).all()), (t, what)
                # errors of at most s^2 / 4 in variance each, of all that is not raised to the least
                d, s = (got - r)[~low], s[~low]
                if what == "m":
                    d = d * r[~low].sign()
                assert abs(float((d / s).sum())) <= 6 * math.sqrt(0.25 * max(d.numel(), 1)), (t, what)


def test_the_same_bits_from_the_hosts_and_the_devices_number():
    m = flp()
    g = torch.Generator().manual_seed(3)
    start = torch.randn(5003, generator=g).to(BF16).cuda()
    runs = []
    for device in (False, True, False):
        p = start.clone()
        state = m.adamw_state([p], bits=8, master=True)
        h = torch.Generator().manual_seed(4)
        at = torch.zeros(1, dtype=torch.int64, device="cuda")
        for t in list(range(1, 60)) + [2 ** 31, 2 ** 32 + 1, 10 ** 12]:
            grad = torch.randn(5003, generator=h).to(BF16).cuda()
            m.adamw_step([p], [grad], state, at.fill_(t) if device else t, 1e-3)
        runs.append([p, state.master[0]] + [f[0].view(torch.uint8) for f in state[:4]])
    for other in runs[1:]:
        for x, y in zip(runs[0], other):
            assert torch.equal(x, y)


@pytest.mark.parametrize("betas", [(0.9, 0.95), (0.9, 0.999)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_an_infinite_gradient_takes_its_blocks_states(bad, betas):
    """All states of the block become NaN with an infinite gradient, whatever its other roots are; with a
    NaN its element's own."""
    m = flp()
    g = torch.Generator().manual_seed(5)
    p = torch.randn(1024, generator=g).cuda()
    grad = torch.randn(1024, generator=g).cuda()
    grad[400:420] = 0.0
    state = m.adamw_state([p], bits=8)
    grad[300] = bad
    before = p.clone()
    m.adamw_step([p], [grad], state, 1, 1e-3, betas=betas)
    rest = torch.ones(1024, dtype=torch.bool, device="cuda")
    rest[300] = False
    assert bool(p[rest].isfinite().all()) and not bool(p[300].isfinite())
    assert bool((p != before)[rest & (grad != 0)].all())
    gone = ~rest if math.isnan(bad) else (torch.arange(1024, device="cuda") // 256) == 1
    for codes, scale in ((state.exp_avg, state.exp_avg_scale),
                         (state.exp_avg_sq, state.exp_avg_sq_scale)):
        assert torch.equal(held(codes[0], scale[0]).isnan(), gone)
