"""Dropout against the definition: the generator in host integers, every type, lengths around
a block of eight, probabilities 0 and 1, infinite values in dropped places, the backward's
mask, graphs that draw a new mask per replay."""
import numpy as np
import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
M32 = 0xFFFFFFFF


def block_words(block, seed, offset):
    """Ten rounds of the 4 x 32 generator for one block, in Python integers."""
    c = [block & M32, block >> 32, offset & M32, offset >> 32]
    k = [seed & M32, seed >> 32]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def keep_mask(n, p, seed, offset):
    thr = int(p * 65536 + 0.5)
    bits = []
    for b in range(-(-n // 8)):
        for w in block_words(b, seed, offset):
            bits += [w & 0xFFFF, w >> 16]
    return np.array(bits[:n]) >= thr, 65536 / (65536 - thr) if thr < 65536 else 0.0


def rng_tensor(seed, offset):
    return torch.from_numpy(np.array([seed, offset], dtype=np.uint64).view(np.int64)).cuda()


def test_generator_known_answers():
    """The published known answers of the generator (all-zero and all-one inputs)."""
    assert block_words(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = (1 << 64) - 1
    assert block_words(ones, ones, ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 1000, 2047, 2048, 2049, 5003])
def test_against_definition(dtype, n):
    m = flp()
    for p, seed, offset in ((0.1, 5, 0), (0.5, (1 << 64) - 3, 1 << 40), (0.9999, 7, 2 ** 63)):
        x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dtype).cuda()
        keep, scale = keep_mask(n, p, seed, offset)
        y = m.dropout(x, p, rng_tensor(seed, offset))
        ref = np.where(keep, x.double().cpu().numpy() * scale, 0.0)
        got = y.double().cpu().numpy()
        assert ((got == 0) | keep).all()
        # the scale is rounded once to fp32, the product once to fp32 and once to the type
        tol = np.abs(ref) * (torch.finfo(dtype).eps / 2 + 2 ** -23)
        assert (np.abs(got - ref) <= tol + float(torch.finfo(dtype).smallest_normal)
                * torch.finfo(dtype).eps).all()


def test_probabilities_zero_and_one():
    m = flp()
    for dtype in TYPES:
        x = torch.randn(4099, device="cuda").to(dtype)
        assert torch.equal(m.dropout(x, 0.0, rng_tensor(1, 2)), x)
        assert not m.dropout(x, 1.0, rng_tensor(1, 2)).any()
        assert torch.equal(m.dropout(x, 2.0 ** -18, rng_tensor(1, 2)), x)  # rounds to p = 0


def test_share_kept_and_expectation():
    """Over n = 2^22 elements the share kept is within six standard deviations of 1 - p, and
    masks of two offsets agree as often as independent ones."""
    m = flp()
    n, p = 1 << 22, 0.3
    q = round(p * 65536) / 65536
    one = torch.ones(n, device="cuda")
    a = m.dropout(one, p, rng_tensor(11, 0)) != 0
    b = m.dropout(one, p, rng_tensor(11, 1)) != 0
    for share, want in ((a.double().mean(), 1 - q), ((a & b).double().mean(), (1 - q) ** 2)):
        say(f"  {float(share):.6f} against {want:.6f}")
        assert abs(float(share) - want) < 6 * (want * (1 - want) / n) ** 0.5


def test_dropped_places_hide_infinities_and_nan():
    m = flp()
    n, p = 4000, 0.5
    keep, scale = keep_mask(n, p, 3, 4)
    drop = torch.from_numpy(~keep).cuda()
    for dtype in TYPES:
        x = torch.ones(n, device="cuda", dtype=dtype)
        x[drop] = float("nan")
        x[drop & (torch.arange(n, device="cuda") % 2 == 0)] = float("inf")
        y = m.dropout(x, p, rng_tensor(3, 4))
        assert torch.equal(y, torch.where(drop, 0.0, scale).to(dtype))


def test_backward_draws_the_forward_mask():
    m = flp()
    x = torch.randn(3, 5, 1003, device="cuda", requires_grad=True)
    rng = rng_tensor(21, 9)
    y = m.dropout(x, 0.2, rng)
    g = torch.randn_like(y)
    (dx,) = torch.autograd.grad(y, [x], g)
    assert torch.equal(dx, m.dropout(g, 0.2, rng))
    assert torch.equal(dx != 0, y != 0)
    # a pair that was changed in between is refused, not used
    y = m.dropout(x, 0.2, rng)
    rng += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_views_off_the_16_byte_grid_and_tails():
    m = flp()
    for dtype in TYPES:
        base = torch.randn(1000, device="cuda").to(dtype)
        want = m.dropout(base[1:].clone(), 0.4, rng_tensor(1, 1))
        code = {torch.bfloat16: m.FLP_BF16, torch.float16: m.FLP_F16, torch.float32: m.FLP_F32}
        out = torch.full((1010,), 7.0, device="cuda", dtype=dtype)
        rng = rng_tensor(1, 1)
        st = m.flp_dropout(999, code[dtype], base[1:].data_ptr(), 0.4, rng.data_ptr(),
                           out[3:].data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == m.FLP_OK
        assert torch.equal(out[3:1002], want)
        assert bool((out[:3] == 7).all()) and bool((out[1002:] == 7).all())


def test_graph_draws_a_new_mask_per_replay():
    m = flp()
    x = torch.randn(777, 65, device="cuda")
    rng = rng_tensor(5, 0)
    m.dropout_forward(x, 0.3, rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.dropout_forward(x, 0.3, rng)
    for step in range(4):
        rng[1] = step
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, m.dropout_forward(x, 0.3, rng_tensor(5, step)))


def test_second_derivatives_are_refused():
    m = flp()
    x = torch.randn(64, device="cuda", requires_grad=True)
    y = m.dropout(x, 0.5, rng_tensor(1, 1))
    (g,) = torch.autograd.grad(y, [x], torch.ones_like(y, requires_grad=True), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_empty_and_refusals():
    m = flp()
    rng = rng_tensor(0, 0)
    x = torch.randn(4, 6, device="cuda")
    assert m.dropout(x[:0], 0.5, rng).shape == (0, 6)
    for bad in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError):
            m.dropout(x, bad, rng)
    with pytest.raises(ValueError):
        m.dropout(x.t(), 0.5, rng)
    with pytest.raises(ValueError):
        m.dropout(x, 0.5, rng.int())
    with pytest.raises(ValueError):
        m.dropout(x, 0.5, rng.cpu())
    with pytest.raises(TypeError):
        m.dropout(x.double(), 0.5, rng)
