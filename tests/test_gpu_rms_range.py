"""Rows of the root mean square norms at the ends of fp32: values of 2^127 and more, whose power of
two has no normal inverse, and values below its normal range."""
import math

import pytest
import torch

from gpu_common import flp, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative
# a sum has 25 roundings on its longest chain (8 elements, 8 chunks, a tree of 9 levels) and those of
# its terms; a norm's factor half of that and four of its own
NORM = 33 * U / 2 + 4 * U


@pytest.mark.parametrize("D", [8, 777, 2688, 4104, 16384])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top", [2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 127, 1.99 * 2.0 ** 127,
                                 2.0 ** -60, 2.0 ** -120])
def test_rows_at_the_ends_of_the_range(top, dtype, D):
    """n and rstd, which may lie below fp32's normal range itself (then to its step, 2^-149)."""
    m = flp()
    say(f"top={top} D={D} {dtype}")
    g = torch.Generator().manual_seed(D)
    x = (torch.rand(5, D, generator=g, dtype=torch.float64) * 2 - 1)
    x[:, D // 2] = 1.0
    x[3, :] = 0.0
    x[3, 1] = -1.0          # alone in its row
    x = (x * top).to(dtype).cuda()
    w = (torch.rand(D, generator=g) + 0.5).cuda()
    n, rstd = m.rms_norm_forward(x, w, eps=0.0)
    d = x.double()
    ref = 1 / torch.sqrt(d.square().mean(-1))
    assert bool(((rstd.double() - ref).abs() <= ref * NORM + 2.0 ** -149).all()), (rstd, ref)
    # n has the relative error of the stored rstd, and two roundings of its own
    out = d * ref[:, None] * w.double()
    rel = NORM + 2.0 ** -149 / ref + 2 * U + torch.finfo(dtype).eps / 2
    assert bool(((n.double() - out).abs() <= out.abs() * (rel[:, None] * (1 + 2.0 ** -7))
                 + 2.0 ** -133).all())
    # the same rows as a residual stream's sum (half of each), behind a norm of the block's output
    r, n2, rstd2, _ = m.residual_rms_norm_forward((x / 2), (x / 2), w, eps=0.0)
    if top > 1:
        assert torch.equal(rstd2, rstd) and torch.equal(n2, n)


def test_one_such_row_among_others():
    m = flp()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 4100, generator=g).cuda()
    clean, stat = m.rms_norm_forward(x)
    y = x.clone()
    y[17, 5] = 3e38
    n, rstd = m.rms_norm_forward(y)
    rest = [i for i in range(40) if i != 17]
    assert torch.equal(n[rest], clean[rest]) and torch.equal(rstd[rest], stat[rest])
    assert abs(float(n[17, 5]) - math.sqrt(4100)) <= 1e-4 * math.sqrt(4100)
    assert bool(n[17].isfinite().all())
