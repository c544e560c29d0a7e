"""Gates of the operators between a model's ends and of its optimizer's step on a machine without
a GPU: fake addresses, every call returns before the device is touched; and the argument checks of
their Python entry points that need no device."""
import os

import pytest
import torch

abi = pytest.importorskip("lm_head_selected_bf16_amd._abi")

if not os.path.exists(abi.LIB_PATH):
    pytest.skip("libflp.so not built (run __graft_entry__.build())", allow_module_level=True)

import lm_head_selected_bf16_amd as flp  # noqa: E402

abi.load()
BF16, F16, F32, I64, I32 = abi.FLP_BF16, abi.FLP_F16, abi.FLP_F32, abi.FLP_I64, abi.FLP_I32
A = [0x10000000 * (k + 1) for k in range(16)]  # fake, 16-byte aligned, non-overlapping
INF, NAN = float("inf"), float("nan")


def name(st):
    return abi.STATUS_NAMES[st]


# ---- AdamW -------------------------------------------------------------------------------------

def tensor(k=0, n=1000, **kw):
    base = dict(param=A[0], grad=A[1], exp_avg=A[2], exp_avg_sq=A[3], exp_avg_scale=A[4],
                exp_avg_sq_scale=A[5], master=A[6], n=n, weight_decay=0.1, p_dtype=BF16,
                g_dtype=F32)
    base.update(kw)
    t = abi.flp_adamw_tensor()
    for f, v in base.items():
        if f in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale",
                 "master") and v:
            v += k * 0x100000
        setattr(t, f, v)
    return t


def adamw(tensors, **kw):
    a = dict(n=len(tensors), bits=8, step=1, step_dev=0, lr=1e-3, lr_dev=0, b1=0.9, b2=0.999,
             eps=1e-8, gs=0)
    a.update(kw)
    arr = (abi.flp_adamw_tensor * max(len(tensors), 1))(*tensors)
    return name(abi.flp_adamw_step(a["n"], arr, a["bits"], a["step"], a["step_dev"], a["lr"],
                                   a["lr_dev"], a["b1"], a["b2"], a["eps"], a["gs"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), "FLP_INVALID_ARGUMENT"),
    (dict(bits=16), "FLP_UNSUPPORTED_DTYPE"),
    (dict(step=0), "FLP_INVALID_ARGUMENT"),
    (dict(lr=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(lr=INF), "FLP_INVALID_ARGUMENT"),
    (dict(b1=1.0), "FLP_INVALID_ARGUMENT"),
    (dict(b2=-0.1), "FLP_INVALID_ARGUMENT"),
    (dict(b2=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(eps=-1e-8), "FLP_INVALID_ARGUMENT"),
    (dict(eps=INF), "FLP_INVALID_ARGUMENT"),
    (dict(step_dev=A[8] + 4), "FLP_MISALIGNED"),
    (dict(lr_dev=A[8] + 2), "FLP_MISALIGNED"),
    (dict(gs=A[8] + 1), "FLP_MISALIGNED"),
    (dict(gs=A[0]), "FLP_INVALID_ARGUMENT"),             # a counter inside a parameter
    (dict(step_dev=A[6] + 8), "FLP_INVALID_ARGUMENT"),
])
def test_adamw_gates(kw, expect):
    assert adamw([tensor()], **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), "FLP_INVALID_ARGUMENT"),
    (dict(n=1 << 62), "FLP_UNSUPPORTED_SHAPE"),
    (dict(weight_decay=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(p_dtype=I64), "FLP_UNSUPPORTED_DTYPE"),
    (dict(g_dtype=F16), "FLP_UNSUPPORTED_DTYPE"),        # neither the parameter's type nor fp32
    (dict(p_dtype=F32, g_dtype=BF16), "FLP_UNSUPPORTED_DTYPE"),
    (dict(param=0), "FLP_INVALID_ARGUMENT"),
    (dict(grad=0), "FLP_INVALID_ARGUMENT"),
    (dict(exp_avg=0), "FLP_INVALID_ARGUMENT"),
    (dict(exp_avg_sq_scale=0), "FLP_INVALID_ARGUMENT"),
    (dict(param=A[0] + 1), "FLP_MISALIGNED"),
    (dict(grad=A[1] + 2), "FLP_MISALIGNED"),
    (dict(master=A[6] + 2), "FLP_MISALIGNED"),
    (dict(exp_avg_scale=A[4] + 2), "FLP_MISALIGNED"),
    (dict(exp_avg=A[3] - 999), "FLP_INVALID_ARGUMENT"),  # the last code is exp_avg_sq's first
    (dict(param=A[1]), "FLP_INVALID_ARGUMENT"),          # the gradient
    (dict(exp_avg_scale=A[5] + 12), "FLP_INVALID_ARGUMENT"),  # four scales each
    (dict(param=A[0] + 0x100000 + 1998), "FLP_INVALID_ARGUMENT"),  # the first tensor's last element
])
def test_adamw_tensor_gates(kw, expect):
    """The second of two tensors is the wrong one."""
    assert adamw([tensor(k=1), tensor(**kw)]) == expect


def test_adamw_python_checks():
    p = torch.zeros(4)
    with pytest.raises(ValueError):
        flp.adamw_step([p], [p], flp.adamw_state([p]), 1, 1e-3)
    with pytest.raises(ValueError):
        flp.adamw_state([p], bits=16)
    s = flp.adamw_state([torch.zeros(3, 100), torch.zeros(1, dtype=torch.bfloat16)], bits=8,
                        master=True)
    assert [t.shape for t in s.exp_avg] == [(3, 100), (1,)]
    assert [t.numel() for t in s.exp_avg_scale] == [2, 1]
    assert s.master[0] is None and s.master[1].dtype == torch.float32
    assert s.exp_avg_sq[0].dtype == torch.float8_e4m3fn


def test_adamw_state_of_an_iterator():
    """As of a module's parameters()."""
    p = [torch.ones(3, dtype=torch.bfloat16), torch.ones(2, 2)]
    for bits in (8, 32):
        s = flp.adamw_state(iter(p), bits=bits, master=True)
        assert [t.shape for t in s.exp_avg] == [t.shape for t in s.exp_avg_sq] == [(3,), (2, 2)]
        assert len(s.master) == 2


# ---- root mean square norms --------------------------------------------------------------------

N, D = 40, 64


def rms_fwd(**kw):
    a = dict(N=N, D=D, x=BF16, xp=A[0], y=A[1], w=F32, wp=A[2], post=1, pw=A[3], gates=4, gate=A[4],
             scale=0.5, eps=1e-6, r=A[5], n=A[6], rstd=A[7], prstd=A[8])
    a.update(kw)
    return name(abi.flp_residual_rms_norm_forward(
        a["N"], a["D"], a["x"], a["xp"], a["y"], a["w"], a["wp"], a["post"], a["pw"], a["gates"],
        a["gate"], a["scale"], a["eps"], a["r"], a["n"], a["rstd"], a["prstd"], 0))


SHARED = [
    (dict(N=-1), "FLP_INVALID_ARGUMENT"),
    (dict(D=0), "FLP_INVALID_ARGUMENT"),
    (dict(D=16385), "FLP_UNSUPPORTED_SHAPE"),
    (dict(N=1 << 31, gates=1), "FLP_UNSUPPORTED_SHAPE"),
    (dict(x=I64), "FLP_UNSUPPORTED_DTYPE"),
    (dict(w=F16), "FLP_UNSUPPORTED_DTYPE"),
    (dict(scale=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(scale=1e39), "FLP_INVALID_ARGUMENT"),
    (dict(gates=3), "FLP_INVALID_ARGUMENT"),             # 40 rows
    (dict(gates=-1), "FLP_INVALID_ARGUMENT"),
    (dict(N=1 << 24, gates=1 << 23), "FLP_UNSUPPORTED_SHAPE"),
    (dict(gates=0), "FLP_INVALID_ARGUMENT"),             # a gate without rows
    (dict(gate=0), "FLP_INVALID_ARGUMENT"),              # rows without a gate
    (dict(post=0), "FLP_INVALID_ARGUMENT"),              # post_weight without post_norm
    (dict(xp=0), "FLP_INVALID_ARGUMENT"),
    (dict(y=0), "FLP_INVALID_ARGUMENT"),
    (dict(xp=A[0] + 1), "FLP_MISALIGNED"),
    (dict(gate=A[4] + 2), "FLP_MISALIGNED"),
]


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(eps=-1e-6), "FLP_INVALID_ARGUMENT"),
    (dict(eps=INF), "FLP_INVALID_ARGUMENT"),
    (dict(n=0), "FLP_INVALID_ARGUMENT"),
    (dict(r=0), "FLP_INVALID_ARGUMENT"),
    (dict(y=0, post=0, pw=0, gates=0, gate=0), "FLP_INVALID_ARGUMENT"),  # r without y
    (dict(n=A[6] + 1), "FLP_MISALIGNED"),
    (dict(rstd=A[7] + 2), "FLP_MISALIGNED"),
    (dict(r=A[0]), "FLP_INVALID_ARGUMENT"),              # in place
    (dict(n=A[1] + 64), "FLP_INVALID_ARGUMENT"),
    (dict(n=A[4] + 512), "FLP_INVALID_ARGUMENT"),        # inside the third gate row
    (dict(prstd=A[7] + 156), "FLP_INVALID_ARGUMENT"),    # the last statistic
    (dict(N=0, xp=0, y=0, r=0, n=0), "FLP_OK"),
])
def test_residual_rms_norm_forward_gates(kw, expect):
    assert rms_fwd(**kw) == expect


def rms_bwd(**kw):
    a = dict(N=N, D=D, x=BF16, gr=A[0], gn=A[1], xp=A[2], y=A[3], w=F32, wp=A[4], post=1, pw=A[5],
             gates=4, gate=A[6], scale=0.5, rstd=A[7], prstd=A[8], dx=A[9], dy=A[10], dw=A[11],
             dpw=A[12], dg=A[13], ws=A[14],
             wsb=abi.flp_residual_rms_norm_backward_workspace_bytes(N, D, 4))
    a.update(kw)
    return name(abi.flp_residual_rms_norm_backward(
        a["N"], a["D"], a["x"], a["gr"], a["gn"], a["xp"], a["y"], a["w"], a["wp"], a["post"],
        a["pw"], a["gates"], a["gate"], a["scale"], a["rstd"], a["prstd"], a["dx"], a["dy"],
        a["dw"], a["dpw"], a["dg"], a["ws"], a["wsb"], 0))


NONE = dict(dx=0, dy=0, dw=0, dpw=0, dg=0, ws=0, wsb=0)


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(gr=0, gn=0), "FLP_INVALID_ARGUMENT"),
    (dict(rstd=0), "FLP_INVALID_ARGUMENT"),
    (dict(prstd=0), "FLP_INVALID_ARGUMENT"),
    (dict(ws=0), "FLP_INVALID_ARGUMENT"),
    (dict(gates=0, gate=0), "FLP_INVALID_ARGUMENT"),     # d_gate without a gate
    (dict(post=0, pw=0), "FLP_INVALID_ARGUMENT"),        # d_post_weight without post_norm
    (dict(ws=A[14] + 4), "FLP_MISALIGNED"),
    (dict(dg=A[13] + 2), "FLP_MISALIGNED"),
    (dict(wsb=4095), "FLP_WORKSPACE_TOO_SMALL"),
    (dict(dx=A[0]), "FLP_INVALID_ARGUMENT"),             # d_x over grad_r
    (dict(dy=A[9] + 128), "FLP_INVALID_ARGUMENT"),
    (dict(dpw=A[11] + 64), "FLP_INVALID_ARGUMENT"),
    (dict(ws=A[13] + 256), "FLP_INVALID_ARGUMENT"),      # workspace inside d_gate
    (NONE, "FLP_OK"),
    (dict(NONE, N=0, gr=0, gn=0, xp=0, y=0, rstd=0, prstd=0), "FLP_OK"),
])
def test_residual_rms_norm_backward_gates(kw, expect):
    assert rms_bwd(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(xp=0), "FLP_INVALID_ARGUMENT"), (dict(out=0), "FLP_INVALID_ARGUMENT"),
    (dict(out=A[0]), "FLP_INVALID_ARGUMENT"), (dict(D=0), "FLP_INVALID_ARGUMENT"),
    (dict(wp=A[1] + 2), "FLP_MISALIGNED"), (dict(eps=NAN), "FLP_INVALID_ARGUMENT"),
])
def test_rms_norm_gates(kw, expect):
    a = dict(D=D, xp=A[0], wp=A[1], eps=1e-6, out=A[2])
    a.update(kw)
    assert name(abi.flp_rms_norm_forward(N, a["D"], BF16, a["xp"], F32, a["wp"], a["eps"], a["out"],
                                         A[3], 0)) == expect
    if "out" not in kw and "eps" not in kw:
        assert name(abi.flp_rms_norm_backward(N, a["D"], BF16, A[4], a["xp"], F32, a["wp"], A[3],
                                              A[5], A[6], A[7], 1 << 20, 0)) == expect


def test_rms_norm_workspace_bytes():
    size = abi.flp_residual_rms_norm_backward_workspace_bytes
    # two fp32 rows of D per slab: at most 256 slabs, more where gates cut the rows finer
    assert size(16384, 2688, 0) == size(16384, 2688, 1) == size(16384, 2688, 16384) \
        == 256 * 2 * 2688 * 4
    assert size(4097, 64, 17) == 17 * 15 * 2 * 64 * 4      # 241 rows a gate, slabs of 17
    assert size(20, 64, 10) == 10 * 2 * 64 * 4
    assert size(0, 64, 0) == 0


# ---- gated projection --------------------------------------------------------------------------

F = 100


def gated_fwd(**kw):
    a = dict(N=N, D=D, F=F, x=BF16, xp=A[0], wg=A[1], wu=A[2], act=0, out=A[3], saved=A[4])
    a.update(kw)
    return name(abi.flp_gated_linear_forward(a["N"], a["D"], a["F"], a["x"], a["xp"], a["wg"],
                                             a["wu"], a["act"], a["out"], a["saved"], 0))


GATED = [
    (dict(N=-1), "FLP_INVALID_ARGUMENT"),
    (dict(F=0), "FLP_INVALID_ARGUMENT"),
    (dict(D=48), "FLP_UNSUPPORTED_SHAPE"),               # no multiple of 32
    (dict(D=1 << 23), "FLP_UNSUPPORTED_SHAPE"),          # 256 rows pass 2^31 bytes
    (dict(F=64 * 32767 + 1), "FLP_UNSUPPORTED_SHAPE"),
    (dict(N=64 * 65535 + 1), "FLP_UNSUPPORTED_SHAPE"),
    (dict(N=64 * 65535, F=64 * 256 + 1), "FLP_UNSUPPORTED_SHAPE"),
    (dict(x=I32), "FLP_UNSUPPORTED_DTYPE"),
    (dict(act=3), "FLP_INVALID_ARGUMENT"),
    (dict(act=-1), "FLP_INVALID_ARGUMENT"),
    (dict(wg=0), "FLP_INVALID_ARGUMENT"),
    (dict(wu=0), "FLP_INVALID_ARGUMENT"),
    (dict(xp=A[0] + 8), "FLP_MISALIGNED"),
    (dict(wu=A[2] + 2), "FLP_MISALIGNED"),
    (dict(saved=A[4] + 8), "FLP_MISALIGNED"),
]


@pytest.mark.parametrize("kw,expect", GATED + [
    (dict(xp=0), "FLP_INVALID_ARGUMENT"),
    (dict(out=0), "FLP_INVALID_ARGUMENT"),
    (dict(out=A[3] + 1), "FLP_MISALIGNED"),
    (dict(out=A[0]), "FLP_INVALID_ARGUMENT"),
    (dict(out=A[2] + F * D * 2 - 2), "FLP_INVALID_ARGUMENT"),      # the last weight
    (dict(out=A[4] + 48 * 128 * 6 - 2), "FLP_INVALID_ARGUMENT"),   # saved: 48 rows of 128
    (dict(N=0, xp=0, wg=0, wu=0, out=0, saved=0), "FLP_OK"),
])
def test_gated_linear_forward_gates(kw, expect):
    assert gated_fwd(**kw) == expect


def gated_bwd(**kw):
    a = dict(N=N, D=D, F=F, x=BF16, g=A[0], saved=A[1], xp=A[2], wg=A[3], wu=A[4], act=1, dx=A[5],
             dwg=A[6], dwu=A[7], ws=A[8],
             wsb=abi.flp_gated_linear_backward_workspace_bytes(N, D, F, BF16, 1, 1))
    a.update(kw)
    return name(abi.flp_gated_linear_backward(a["N"], a["D"], a["F"], a["x"], a["g"], a["saved"],
                                              a["xp"], a["wg"], a["wu"], a["act"], a["dx"],
                                              a["dwg"], a["dwu"], a["ws"], a["wsb"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(kw, saved=A[1] + 8) if "saved" in kw else kw, e) for kw, e in GATED] + [
    (dict(g=0), "FLP_INVALID_ARGUMENT"),
    (dict(saved=0), "FLP_INVALID_ARGUMENT"),
    (dict(ws=0), "FLP_INVALID_ARGUMENT"),
    (dict(xp=0), "FLP_INVALID_ARGUMENT"),                # the weight gradients need x
    (dict(g=A[0] + 1), "FLP_MISALIGNED"),
    (dict(dx=A[5] + 2), "FLP_MISALIGNED"),
    (dict(dwu=A[7] + 8), "FLP_MISALIGNED"),
    (dict(ws=A[8] + 8), "FLP_MISALIGNED"),
    (dict(wsb=abi.flp_gated_linear_backward_workspace_bytes(N, D, F, BF16, 1, 1) - 1),
     "FLP_WORKSPACE_TOO_SMALL"),
    (dict(dx=A[0]), "FLP_INVALID_ARGUMENT"),
    (dict(dwu=A[6] + 64), "FLP_INVALID_ARGUMENT"),
    (dict(ws=A[7] + 64), "FLP_INVALID_ARGUMENT"),
    (dict(dx=0, dwg=0, dwu=0, ws=0, g=0), "FLP_OK"),     # nothing requested
    (dict(N=0, g=0, saved=0, xp=0, dwg=0, dwu=0, ws=0, wsb=0), "FLP_OK"),
])
def test_gated_linear_backward_gates(kw, expect):
    assert gated_bwd(**kw) == expect


def test_gated_linear_sizes():
    assert abi.flp_gated_linear_saved_bytes(40, 100, BF16) == 48 * 128 * 6
    assert abi.flp_gated_linear_saved_bytes(40, 100, F32) == 48 * 128 * 8
    assert abi.flp_gated_linear_saved_bytes(0, 100, BF16) == 0
    size = abi.flp_gated_linear_backward_workspace_bytes
    # 16 bits: [dz | du], and fp32 sums over slabs of its 256 columns or tokens (none of 64 tokens)
    assert size(64, 64, 128, BF16, 1, 1) == size(64, 64, 128, BF16, 0, 1) == 256 * 64 * 2
    assert size(64, 64, 256, BF16, 1, 0) == 512 * 64 * 2 + 2 * 64 * 64 * 4
    assert size(1024, 64, 128, BF16, 0, 1) == 256 * 1024 * 2 + 4 * 256 * 64 * 4
    # fp32: beside it [Wg; Wu]^T; its transpose over 64 tokens and x^T
    assert size(64, 64, 128, F32, 1, 0) == 2 * 128 * 64 * 4 + 2 * 128 * 64 * 4
    assert size(40, 64, 128, F32, 0, 1) == 2 * 128 * 64 * 4 + 64 * 64 * 4
    assert size(0, 64, 128, BF16, 1, 1) == 0


def test_residual_rms_norm_needs_the_block():
    for x in (torch.ones(2, 4), torch.ones(2, 4, requires_grad=True)):
        with pytest.raises(TypeError):
            flp.residual_rms_norm(x, None)
    with pytest.raises(TypeError):
        flp.residual_rms_norm_forward(torch.ones(2, 4), None)


@pytest.mark.parametrize("eps,expect", [
    (1e-40, "FLP_INVALID_ARGUMENT"), (1e-300, "FLP_INVALID_ARGUMENT"),
    (2.0 ** -126 * (1 - 2.0 ** -20), "FLP_INVALID_ARGUMENT")])
def test_adamw_eps_below_the_normal_range(eps, expect):
    """Its reciprocal is no fp32 number: an element without gradients would become NaN."""
    assert adamw([tensor()], eps=eps) == expect


def test_adamw_eps_at_the_edges():
    """0 and the least normal value pass this gate (another argument is refused)."""
    for eps in (0.0, 2.0 ** -126):
        assert adamw([tensor(n=1 << 62)], eps=eps) == "FLP_UNSUPPORTED_SHAPE"
