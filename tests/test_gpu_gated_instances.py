"""The gated projection's kernels that training batches run, each reached and named by a trace:
against 64 bits with ragged sizes, and d_x of the same rows from the smaller and the larger tile of
each class of batches, bit for bit."""
import re

import pytest
import torch

from gpu_common import flp, say
from test_gpu_gated import compare, half_step, make, reference, rounding

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAME = {BF16: "BF16", F16: "F16", F32: "F32"}


def traced(call):
    """What `call` returns, and the names of the library's kernels that it ran."""
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        out = call()
        torch.cuda.synchronize()
    names = [e.name.replace("flp::", "").replace("(anonymous namespace)::", "").replace("void ", "")
             for e in p.events()]
    return out, {m.group(0) for m in (re.match(r"k_\w+(<[^()]*>)?", n) for n in names) if m}


def forward(dtype, bm, bn, odd, act=0):
    waves = "4, 2, 2" if bm == 256 else "2, 2, 2" if bm == 128 else "2, 2, 4"
    return f"k_gated_fwd<{NAME[dtype]}, {bm}, {bn}, {waves}, {str(odd).lower()}, {act}>"


def product(dtype, turned, large, slabs):
    tile = "256, 224, 4, 2" if large else "128, 128, 2, 2"
    return f"k_gated_gemm<{NAME[dtype]}, {str(turned).lower()}, {tile}, {str(slabs).lower()}>"




@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("N,D,F,bm,odd", [
    (2571, 64, 2021, 256, False), (2600, 96, 2000, 256, True), (4097, 256, 1300, 256, False),
    (1000, 544, 1601, 128, True), (777, 128, 1601, 128, False), (150, 160, 400, 64, True),
    (150, 192, 401, 64, False), (31, 192, 401, 32, False), (20, 2688, 130, 32, False),
    (9, 672, 65, 32, True)])
def test_forward_tiles(N, D, F, bm, odd, dtype):
    say(f"N={N} D={D} F={F} {dtype}")
    args = make(N, D, F, dtype, N + F)
    _, ran = traced(lambda: compare(*args, "silu"))
    assert forward(dtype, bm, max(bm, 64), odd) in ran, ran


@pytest.mark.parametrize("N,D,F,bm", [(2571, 64, 2021, 256), (777, 128, 1601, 128),
                                      (150, 192, 401, 64), (31, 96, 401, 32)])
def test_forward_tiles_fp32(N, D, F, bm):
    say(f"N={N} D={D} F={F}")
    args = make(N, D, F, F32, N + F)
    _, ran = traced(lambda: compare(*args, "gelu"))
    assert forward(F32, bm, max(bm, 64), False, 1) in ran, ran


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("N,D,F,dx,dw", [
    # (large tile, slabs) of d_x and of the weights' product; K of several stages and a part of one
    (501, 2688, 2021, (True, True), (True, False)),
    (1001, 1344, 3587, (False, True), (True, False)),
    (777, 2688, 1700, (True, True), (True, False)),
    (3333, 2688, 130, (True, False), (False, True)),
    (8200, 1376, 200, (True, False), (False, True)),
    (300, 160, 1500, (False, True), (False, False)),
    (2100, 160, 100, (False, False), (False, True)),
    (4111, 992, 1001, (True, True), (False, False)),
    (2500, 1376, 130, (False, False), (False, True))])
def test_backward_tiles(N, D, F, dx, dw, dtype):
    say(f"N={N} D={D} F={F} {dtype}")
    args = make(N, D, F, dtype, N + F)
    _, ran = traced(lambda: compare(*args, "silu"))
    assert product(dtype, False, *dx) in ran, ran
    assert product(dtype, True, *dw) in ran, ran


@pytest.mark.parametrize("N,D,F,dx,dw", [
    (129, 1344, 2000, "128, 128, 2, 2, false, 2", "128, 128, 2, 2, false, 0"),
    (200, 288, 1500, "64, 64, 2, 2, false, 2", "64, 64, 2, 2, false, 0"),
    (33, 64, 700, "64, 32, 4, 1, false, 2", "64, 32, 4, 1, false, 0"),
    (2300, 1344, 200, "128, 128, 2, 2, false, 0", "64, 64, 2, 2, false, 0")])
def test_backward_tiles_fp32(N, D, F, dx, dw):
    say(f"N={N} D={D} F={F}")
    args = make(N, D, F, F32, N + F)
    _, ran = traced(lambda: compare(*args, "silu"))
    for tile, two in ((dx, "false>"), (dw, "true>")):
        assert any(k.startswith(f"k_gemm<F32, {tile}") and k.endswith(two) for k in ran), (tile, ran)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("few,many,D,F", [
    (130, 512, 2688, 2048),       # up to 512 rows: eight slabs
    (1, 512, 2688, 2048),
    (513, 1024, 1600, 640),       # up to 1024: five
    (1025, 2048, 2688, 300),      # up to 2048: two
    (2049, 8192, 2688, 200),      # up to 8192, and above: one walk
    (8193, 16384, 672, 200)])
def test_d_x_from_both_tiles_of_a_class(few, many, D, F, dtype):
    """The smallest batch of a class by the smaller tile, the largest by the larger one."""
    m = flp()
    x, wg, wu, go = make(many, D, F, dtype, 6)
    seen = []
    for part in (slice(many - few, None), slice(None)):
        a, g = x[part].contiguous(), go[part].contiguous()
        _, saved = m.gated_linear_forward(a, wg, wu)
        dx, ran = traced(lambda: m.gated_linear_backward(g, saved, a, wg, wu, need_gate=False,
                                                         need_up=False)[0])
        seen.append((dx, {"256, 224" in k for k in ran if k.startswith("k_gated_gemm")}))
    assert torch.equal(seen[0][0], seen[1][0][-few:])
    assert seen[0][1] == {False} and seen[1][1] == {True}, [s[1] for s in seen]
    # some rows against 64 bits
    rows = torch.tensor([0, few // 2, few - 1], device="cuda")
    at = many - few + rows
    ref, tol = reference(x[at], wg, wu, go[at], "silu")
    err = (seen[0][0][rows].double() - ref["dx"]).abs()
    assert bool((err <= (rounding(dtype, ref["dx"]) + tol["dx"]) * (1 + 2.0 ** -6)).all())
    # typical: the roundings of dz and du and the result's (compare() has the same)
    size = float(ref["dx"].norm()) + 2 * float(ref["dx_terms"].norm())
    assert float(err.norm()) <= half_step(dtype) * size
