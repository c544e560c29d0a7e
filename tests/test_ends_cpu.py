"""Gates of the scaled embedding, dropout and layer norm on a machine without a GPU: fake
addresses, every call returns before the device is touched; and the argument checks of their
Python entry points that need no device."""
import pytest
import torch

abi = pytest.importorskip("lm_head_selected_bf16_amd._abi")
import os  # noqa: E402

if not os.path.exists(abi.LIB_PATH):
    pytest.skip("libflp.so not built (run __graft_entry__.build())", allow_module_level=True)

import lm_head_selected_bf16_amd as flp  # noqa: E402

abi.load()
BF16, F16, F32, I64, I32 = abi.FLP_BF16, abi.FLP_F16, abi.FLP_F32, abi.FLP_I64, abi.FLP_I32
A = [0x10000000 * (k + 1) for k in range(12)]  # fake, 16-byte aligned, non-overlapping
N, D, V = 40, 64, 1000
INF, NAN = float("inf"), float("nan")


def name(st):
    return abi.STATUS_NAMES[st]


def norm_fwd(**kw):
    a = dict(N=N, D=D, x=BF16, xp=A[0], w=BF16, wp=A[1], bp=A[2], eps=1e-5, out=A[3], mean=A[4],
             rstd=A[5])
    a.update(kw)
    return name(abi.flp_layer_norm_forward(a["N"], a["D"], a["x"], a["xp"], a["w"], a["wp"],
                                           a["bp"], a["eps"], a["out"], a["mean"], a["rstd"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "FLP_INVALID_ARGUMENT"),
    (dict(D=0), "FLP_INVALID_ARGUMENT"),
    (dict(D=1 << 28), "FLP_UNSUPPORTED_SHAPE"),
    (dict(N=1 << 50, D=1 << 20), "FLP_UNSUPPORTED_SHAPE"),
    (dict(x=I64), "FLP_UNSUPPORTED_DTYPE"),
    (dict(w=F16), "FLP_UNSUPPORTED_DTYPE"),              # neither the rows' type nor fp32
    (dict(x=F32, w=BF16), "FLP_UNSUPPORTED_DTYPE"),
    (dict(eps=-1e-6), "FLP_INVALID_ARGUMENT"),
    (dict(eps=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(eps=INF), "FLP_INVALID_ARGUMENT"),
    (dict(xp=0), "FLP_INVALID_ARGUMENT"),
    (dict(out=0), "FLP_INVALID_ARGUMENT"),
    (dict(xp=A[0] + 1), "FLP_MISALIGNED"),
    (dict(w=F32, wp=A[1] + 2), "FLP_MISALIGNED"),
    (dict(mean=A[4] + 2), "FLP_MISALIGNED"),
    (dict(out=A[0]), "FLP_INVALID_ARGUMENT"),            # in place
    (dict(rstd=A[4] + 16), "FLP_INVALID_ARGUMENT"),      # the two statistics overlap
    (dict(out=A[1] - 64), "FLP_INVALID_ARGUMENT"),       # out runs into the weight
    (dict(N=0, xp=0, out=0), "FLP_OK"),
])
def test_layer_norm_forward_gates(kw, expect):
    assert norm_fwd(**kw) == expect


def norm_bwd(**kw):
    a = dict(N=N, D=D, x=BF16, g=A[0], xp=A[1], w=F32, wp=A[2], mean=A[3], rstd=A[4], dx=A[5],
             dw=A[6], db=A[7], ws=A[8], wsb=abi.flp_layer_norm_backward_workspace_bytes(N, D))
    a.update(kw)
    return name(abi.flp_layer_norm_backward(a["N"], a["D"], a["x"], a["g"], a["xp"], a["w"],
                                            a["wp"], a["mean"], a["rstd"], a["dx"], a["dw"],
                                            a["db"], a["ws"], a["wsb"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "FLP_INVALID_ARGUMENT"),
    (dict(w=F16), "FLP_UNSUPPORTED_DTYPE"),
    (dict(g=0), "FLP_INVALID_ARGUMENT"),
    (dict(xp=0), "FLP_INVALID_ARGUMENT"),
    (dict(mean=0), "FLP_INVALID_ARGUMENT"),
    (dict(rstd=0), "FLP_INVALID_ARGUMENT"),
    (dict(ws=0), "FLP_INVALID_ARGUMENT"),
    (dict(ws=A[8] + 4), "FLP_MISALIGNED"),
    (dict(dw=A[6] + 2), "FLP_MISALIGNED"),
    (dict(wsb=64), "FLP_WORKSPACE_TOO_SMALL"),
    (dict(dx=A[0]), "FLP_INVALID_ARGUMENT"),             # d_x over grad_out
    (dict(ws=A[5] + 64), "FLP_INVALID_ARGUMENT"),        # workspace inside d_x
    (dict(db=A[6] + 128), "FLP_INVALID_ARGUMENT"),       # d_bias inside d_weight
    (dict(dx=0, dw=0, db=0, ws=0, wsb=0, g=0), "FLP_OK"),  # nothing requested
    (dict(N=0, g=0, xp=0, mean=0, rstd=0, dw=0, db=0, ws=0, wsb=0), "FLP_OK"),
    (dict(N=0, g=0, xp=0, mean=0, rstd=0, dw=A[6] + 2, ws=0, wsb=0), "FLP_MISALIGNED"),
])
def test_layer_norm_backward_gates(kw, expect):
    assert norm_bwd(**kw) == expect


def test_layer_norm_workspace_bytes():
    # two fp32 rows of D per slab, at most 256 slabs
    assert abi.flp_layer_norm_backward_workspace_bytes(16384, 2688) == 256 * 2 * 2688 * 4
    assert abi.flp_layer_norm_backward_workspace_bytes(1, 5) == 256
    assert abi.flp_layer_norm_backward_workspace_bytes(0, 64) == 0


def drop(**kw):
    a = dict(n=1000, x=BF16, xp=A[0], p=0.1, rng=A[1], out=A[2])
    a.update(kw)
    return name(abi.flp_dropout(a["n"], a["x"], a["xp"], a["p"], a["rng"], a["out"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), "FLP_INVALID_ARGUMENT"),
    (dict(n=1 << 62), "FLP_UNSUPPORTED_SHAPE"),
    (dict(x=I32), "FLP_UNSUPPORTED_DTYPE"),
    (dict(p=-0.01), "FLP_INVALID_ARGUMENT"),
    (dict(p=1.01), "FLP_INVALID_ARGUMENT"),
    (dict(p=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(xp=0), "FLP_INVALID_ARGUMENT"),
    (dict(rng=0), "FLP_INVALID_ARGUMENT"),
    (dict(out=0), "FLP_INVALID_ARGUMENT"),
    (dict(rng=A[1] + 4), "FLP_MISALIGNED"),
    (dict(xp=A[0] + 1), "FLP_MISALIGNED"),
    (dict(out=A[0]), "FLP_INVALID_ARGUMENT"),            # in place
    (dict(out=A[1] - 1992), "FLP_INVALID_ARGUMENT"),     # out runs into rng
    (dict(n=0, xp=0, rng=0, out=0), "FLP_OK"),
])
def test_dropout_gates(kw, expect):
    assert drop(**kw) == expect


@pytest.mark.parametrize("scale", [INF, -INF, NAN])
def test_scaled_embedding_refuses_a_scale_that_is_not_finite(scale):
    assert name(abi.flp_embedding_scaled_forward(N, D, V, BF16, A[0], A[1], I64, scale, A[2],
                                                 0)) == "FLP_INVALID_ARGUMENT"
    wsb = abi.flp_embedding_backward_workspace_bytes(N, D, V)
    assert name(abi.flp_embedding_scaled_backward(N, D, V, BF16, A[0], A[1], I64, scale, A[2],
                                                  BF16, A[3], wsb, 0)) == "FLP_INVALID_ARGUMENT"


def test_scaled_embedding_keeps_the_gates_of_the_lookup():
    assert name(abi.flp_embedding_scaled_forward(N, 4, V, BF16, A[0], A[1], I64, 2.0, A[2],
                                                 0)) == "FLP_UNSUPPORTED_SHAPE"
    assert name(abi.flp_embedding_scaled_forward(N, D, V, BF16, A[0], A[1], I64, 2.0, A[0] + 64,
                                                 0)) == "FLP_INVALID_ARGUMENT"
    assert name(abi.flp_embedding_scaled_backward(N, D, V, BF16, A[0], A[1], I64, 2.0, A[2], BF16,
                                                  A[3], 64, 0)) == "FLP_WORKSPACE_TOO_SMALL"


def test_python_checks():
    x = torch.zeros(4, 8)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU tensor"):
        flp.layer_norm(x)
    with pytest.raises(TypeError):
        flp.layer_norm(x.double())
    with pytest.raises(ValueError, match="GPU tensor"):
        flp.dropout(x, 0.1, rng)
    with pytest.raises(TypeError):
        flp.dropout(x.long(), 0.1, rng)
    with pytest.raises(ValueError, match="GPU"):
        flp.embedding(x, torch.zeros(3, dtype=torch.int64), scale=2.0)
