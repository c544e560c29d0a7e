"""The scaled embedding against its definition in 64 bits, and against the plain lookup at
scale 1 (the same bits)."""
import math

import pytest
import torch

import flp_inputs
import oracle
from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

CASES = [  # dtype, N, D, V, ids, ids outside the table, id type, d_weight type
    (BF16, 3000, 64, 5000, "zipf", (-1, 5000), torch.int64, None),
    (BF16, 700, 2688, 900, "uniform", (), torch.int32, F32),
    (F16, 700, 96, 300, "zipf", (300,), torch.int64, None),
    (F32, 900, 36, 2000, "zipf", (-2,), torch.int32, None),
    (BF16, 1500, 64, 4000, "same", (), torch.int64, None),
    (F32, 1, 4, 1, "uniform", (), torch.int64, None),
]


@pytest.mark.parametrize("scale", [math.sqrt(2688), -0.3, 2.0 ** -40, 0.0])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_parity(k, scale):
    dtype, N, D, V, draw, bad, idt, dwt = CASES[k]
    inp = flp_inputs.make_embedding_inputs(N, D, V, dtype, 60 + k, ids=draw, invalid=bad)
    m = flp()
    ids = inp["ids"].to(idt).cuda()
    w, g = inp["weight"].cuda(), inp["grad"].cuda()
    out = m.embedding_forward(w, ids, scale)
    dw = m.embedding_backward(g, ids, V, dw_dtype=dwt, scale=scale)
    s32 = float(torch.tensor(scale, dtype=F32))  # the factor enters in fp32
    ref = torch.from_numpy(oracle.embedding_forward(inp["weight"], inp["ids"])) * s32
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = (out.double().cpu() - ref).abs()
    # the product is exact to 24 bits in fp32, then rounded to the type
    assert bool((err <= ref.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -24) + tiny).all())
    exact = torch.from_numpy(oracle.embedding_backward(inp["grad"], inp["ids"], V)) * s32
    size = torch.from_numpy(oracle.embedding_backward(inp["grad"].abs(), inp["ids"], V)) * abs(s32)
    wt = dw.dtype
    # at most N fp32 additions, the product and the final rounding
    tol = size * N * 2.0 ** -24 + exact.abs() * (torch.finfo(wt).eps / 2 + 2.0 ** -24)
    tiny = torch.finfo(wt).smallest_normal * torch.finfo(wt).eps
    err = (dw.double().cpu() - exact).abs()
    say(f"  case {k} scale {scale}: d_weight max error {float(err.max()):.3e}")
    assert bool((err <= tol + tiny).all())


def test_scale_one_is_the_plain_lookup():
    inp = flp_inputs.make_embedding_inputs(2000, 128, 700, BF16, 70, ids="zipf", invalid=(-1,))
    m = flp()
    w, ids, g = inp["weight"].cuda(), inp["ids"].cuda(), inp["grad"].cuda()
    w[3, 5] = float("nan")
    w[4, 6] = float("inf")
    plain, scaled = torch.empty(2000, 128, dtype=BF16, device="cuda"), None
    st = m.flp_embedding_forward(2000, 128, 700, m.FLP_BF16, w.data_ptr(), ids.data_ptr(),
                                 m.FLP_I64, plain.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream)
    assert st == m.FLP_OK
    scaled = m.embedding(w, ids, scale=1.0)
    assert torch.equal(plain.view(torch.int16), scaled.view(torch.int16))
    # a power of two scales every gradient exactly
    a, b = m.embedding_backward(g, ids, 700), m.embedding_backward(g, ids, 700, scale=0.5)
    assert torch.equal(a.float() * 0.5, b.float())


def test_autograd_and_ids_outside_the_table():
    m = flp()
    w = torch.randn(50, 64, device="cuda", requires_grad=True)
    ids = torch.tensor([[3, -1, 50], [3, 49, 1 << 40]], device="cuda")
    out = m.embedding(w, ids, scale=8.0)
    assert out.shape == (2, 3, 64)
    assert not out[0, 1:].any() and not out[1, 2].any()
    g = torch.randn_like(out)
    (dw,) = torch.autograd.grad(out, [w], g)
    ref = torch.zeros(50, 64, device="cuda", dtype=torch.float64)
    ref[3] = 8 * (g[0, 0].double() + g[1, 0].double())
    ref[49] = 8 * g[1, 1].double()
    assert bool(((dw.double() - ref).abs() <= ref.abs() * 2 ** -23 + 16 * 2.0 ** -24).all())
    empty = m.embedding(w, ids[:0], scale=8.0)
    (dw,) = torch.autograd.grad(empty, [w], torch.empty_like(empty))
    assert empty.shape == (0, 3, 64) and not dw.any()


@pytest.mark.parametrize("ids", ["uniform", "few", "same", "dropped"])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_sorting_by_counting_keeps_the_order_of_the_radix_passes(ids, idt):
    """Up to 4096 tokens are sorted in another way.  Dropped ids behind them change nothing else,
    so the longer list has to give the same bits (of sums whose order shows in the last bit), and
    shorter ones are checked with whole numbers."""
    V, D = 3001, 40
    g = torch.Generator().manual_seed(9)
    top = {"uniform": V, "few": 7, "same": 1, "dropped": V}[ids]
    t = torch.randint(0, top, (4096,), generator=g)
    if ids == "dropped":
        t[torch.rand(4096, generator=g) < 0.4] = V
        t[::11] = -5
    grad = torch.randn(4096, D, generator=g)
    t, grad = t.to(idt).cuda(), grad.cuda()
    m = flp()
    short = m.embedding_backward(grad, t, V)
    longer = m.embedding_backward(torch.cat([grad, torch.ones(1000, D, device="cuda")]),
                                  torch.cat([t, torch.full((1000,), -1, dtype=idt, device="cuda")]), V)
    assert torch.equal(short, longer)
    whole = (grad * 8).round()
    for N in (1, 2, 63, 64, 65, 255, 257, 1000, 2047, 2049, 4095):
        want = torch.zeros(V, D, dtype=torch.float64, device="cuda")
        ok = (t[:N] >= 0) & (t[:N] < V)
        want.index_add_(0, t[:N][ok].long(), whole[:N][ok].double())
        assert torch.equal(m.embedding_backward(whole[:N].contiguous(), t[:N].contiguous(), V).double(),
                           want), N


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("off", [1, 3, 8])
def test_upstream_gradient_off_the_16_byte_grid(dtype, off):
    """A dense view that begins `off` elements into its storage, given as it is and made by the
    backward of a concatenation."""
    m = flp()
    w = torch.randn(50, 64, device="cuda").to(dtype).requires_grad_()
    ids = torch.tensor([4, 9, -1, 4, 49, 0], device="cuda")
    whole = torch.randn(off + 6 * 64, device="cuda").to(dtype)
    up = whole[off:].view(6, 64)
    want = m.embedding_backward(up.clone(), ids, 50, scale=3.0)
    (got,) = torch.autograd.grad(m.embedding(w, ids, 3.0), [w], up)
    assert torch.equal(got, want)
    cat = torch.cat([torch.zeros(off, device="cuda", dtype=dtype),
                     m.embedding(w, ids, 3.0).flatten()])
    (got,) = torch.autograd.grad(cat, [w], whole)
    assert torch.equal(got, want)


@pytest.mark.parametrize("args", [(), (1.0,), (3.0,)])
def test_the_function_of_the_lookup(args):
    """Embedding is an autograd.Function with forward and backward of its own, and gives the bits
    of embedding(); its backward needs no second library."""
    m = flp()
    assert issubclass(m.Embedding, torch.autograd.Function)
    ids = torch.tensor([[4, 9, -1], [4, 49, 50]], device="cuda")
    w = torch.randn(50, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    whole = torch.randn(3 + 6 * 64, device="cuda").bfloat16()
    for up in (torch.randn(2, 3, 64, device="cuda").bfloat16(), whole[3:].view(2, 3, 64),
               whole[:64].expand(2, 3, 64)):
        out, want = m.Embedding.apply(w, ids, *args), m.embedding(w, ids, *args)
        assert torch.equal(out, want) and type(out.grad_fn).__name__ == "EmbeddingBackward"
        assert torch.equal(torch.autograd.grad(out, [w], up)[0],
                           torch.autograd.grad(want, [w], up)[0])


@pytest.mark.parametrize("scale", [1.0, 0.5])
def test_more_rows_than_one_launch_has_waves(scale):
    N = 2 ** 26 + 37
    w = torch.randn(50, 8, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, 50, (N,), device="cuda", dtype=torch.int32)
    out = flp().embedding_forward(w, ids, scale)
    for lo in (0, 2 ** 25 - 20, 2 ** 26 - 20, N - 40):  # a half is exact
        assert torch.equal(out[lo:lo + 40], w[ids[lo:lo + 40].long()] * scale)


def test_refusals():
    m = flp()
    w = torch.randn(50, 64, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (float("nan"), float("inf")):
        with pytest.raises(ValueError):
            m.embedding(w, ids, scale=bad)
    with pytest.raises(ValueError):
        m.embedding(w, ids.cpu(), scale=2.0)
    with pytest.raises(m.FlpError):
        m.embedding(torch.randn(5, 6, device="cuda"), ids, scale=2.0)
