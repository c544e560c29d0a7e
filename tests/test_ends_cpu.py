"""Gates of the scaled embedding, dropout, layer norm and linear cross entropy on a machine without a GPU: fake
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
    (dict(D=1 << 27), "FLP_UNSUPPORTED_SHAPE"),
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
    # more positions than one launch takes
    assert name(abi.flp_embedding_scaled_backward(2 ** 30, 8, V, BF16, A[0], A[1], I64, 2.0, A[2],
                                                  BF16, A[3], 2 ** 60, 0)) == "FLP_UNSUPPORTED_SHAPE"


def ce_fwd(**kw):
    a = dict(N=N, D=D, V=V, x=BF16, h=A[0], w=A[1], b=A[2], t=A[3], td=I64, s=0.1, c=1e-4,
             red=abi.FLP_REDUCE_MEAN, loss=A[4], lse=A[5], ws=A[6],
             wsb=abi.flp_cross_entropy_forward_workspace_bytes(N, D, V))
    a.update(kw)
    return name(abi.flp_cross_entropy_forward(a["N"], a["D"], a["V"], a["x"], a["h"], a["w"],
                                              a["b"], a["t"], a["td"], a["s"], a["c"], a["red"],
                                              a["loss"], a["lse"], a["ws"], a["wsb"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "FLP_INVALID_ARGUMENT"),
    (dict(D=48), "FLP_UNSUPPORTED_SHAPE"),
    (dict(x=I64), "FLP_UNSUPPORTED_DTYPE"),
    (dict(td=F32), "FLP_UNSUPPORTED_DTYPE"),
    (dict(s=-0.1), "FLP_INVALID_ARGUMENT"),
    (dict(s=1.1), "FLP_INVALID_ARGUMENT"),
    (dict(s=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(c=-1.0), "FLP_INVALID_ARGUMENT"),
    (dict(c=INF), "FLP_INVALID_ARGUMENT"),
    (dict(red=3), "FLP_INVALID_ARGUMENT"),
    (dict(h=0), "FLP_INVALID_ARGUMENT"),
    (dict(t=0), "FLP_INVALID_ARGUMENT"),
    (dict(loss=0), "FLP_INVALID_ARGUMENT"),
    (dict(ws=0), "FLP_INVALID_ARGUMENT"),
    (dict(h=A[0] + 8), "FLP_MISALIGNED"),
    (dict(loss=A[4] + 2), "FLP_MISALIGNED"),
    (dict(t=A[3] + 4), "FLP_MISALIGNED"),
    (dict(loss=A[5] + 8 * N - 4), "FLP_INVALID_ARGUMENT"),  # the loss inside the statistics
    (dict(ws=A[1] + 256), "FLP_INVALID_ARGUMENT"),          # workspace inside the weight
    (dict(wsb=256), "FLP_WORKSPACE_TOO_SMALL"),
    (dict(N=0, loss=0), "FLP_INVALID_ARGUMENT"),            # a reduced loss is written
    (dict(N=0, loss=A[4] + 1), "FLP_MISALIGNED"),
    (dict(N=0, red=abi.FLP_REDUCE_NONE, h=0, t=0, loss=0, lse=0, ws=0), "FLP_OK"),
])
def test_cross_entropy_forward_gates(kw, expect):
    assert ce_fwd(**kw) == expect


def ce_bwd(**kw):
    a = dict(N=N, D=D, V=V, x=BF16, g=A[0], lse=A[1], h=A[2], w=A[3], b=A[4], t=A[5], td=I32,
             s=0.0, c=0.0, red=abi.FLP_REDUCE_MEAN, dh=A[6], dw=A[7], db=A[8], ws=A[9],
             wsb=abi.flp_cross_entropy_backward_workspace_bytes(N, D, V, BF16, 0))
    a.update(kw)
    return name(abi.flp_cross_entropy_backward(a["N"], a["D"], a["V"], a["x"], a["g"], a["lse"],
                                               a["h"], a["w"], a["b"], a["t"], a["td"], a["s"],
                                               a["c"], a["red"], a["dh"], a["dw"], a["db"],
                                               a["ws"], a["wsb"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(D=100), "FLP_UNSUPPORTED_SHAPE"),
    (dict(s=2.0), "FLP_INVALID_ARGUMENT"),
    (dict(c=NAN), "FLP_INVALID_ARGUMENT"),
    (dict(red=-1), "FLP_INVALID_ARGUMENT"),
    (dict(g=0), "FLP_INVALID_ARGUMENT"),
    (dict(lse=0), "FLP_INVALID_ARGUMENT"),
    (dict(ws=0), "FLP_INVALID_ARGUMENT"),
    (dict(dh=A[6] + 2), "FLP_MISALIGNED"),
    (dict(dh=A[2]), "FLP_INVALID_ARGUMENT"),
    (dict(db=A[7] + 64), "FLP_INVALID_ARGUMENT"),
    (dict(ws=A[0] - 256), "FLP_INVALID_ARGUMENT"),          # workspace runs into grad_out
    (dict(wsb=64), "FLP_WORKSPACE_TOO_SMALL"),
    (dict(wsb=abi.flp_cross_entropy_backward_workspace_bytes(N, D, V, BF16, 0) - 1),
     "FLP_WORKSPACE_TOO_SMALL"),
    (dict(dh=0, dw=0, db=0, ws=0), "FLP_OK"),
    (dict(N=0, g=0, lse=0, h=0, t=0, dw=0, db=0, ws=0), "FLP_OK"),
    (dict(N=0, g=0, lse=0, h=0, t=0, dw=A[7] + 8, ws=0), "FLP_MISALIGNED"),
])
def test_cross_entropy_backward_gates(kw, expect):
    assert ce_bwd(**kw) == expect


def ce_all(**kw):
    a = dict(N=N, D=D, V=V, x=BF16, h=A[0], w=A[1], b=A[2], t=A[3], td=I64, s=0.1, c=1e-4,
             red=abi.FLP_REDUCE_SUM, loss=A[4], st=A[5], dh=A[6], dw=A[7], db=A[8], ws=A[9],
             wsb=abi.flp_cross_entropy_gradients_workspace_bytes(N, D, V, BF16, 0))
    a.update(kw)
    return name(abi.flp_cross_entropy_gradients(a["N"], a["D"], a["V"], a["x"], a["h"], a["w"],
                                                a["b"], a["t"], a["td"], a["s"], a["c"], a["red"],
                                                a["loss"], a["st"], a["dh"], a["dw"], a["db"],
                                                a["ws"], a["wsb"], 0))


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "FLP_INVALID_ARGUMENT"),
    (dict(D=40), "FLP_UNSUPPORTED_SHAPE"),
    (dict(x=F16), "FLP_UNSUPPORTED_DTYPE"),
    (dict(s=-1.0), "FLP_INVALID_ARGUMENT"),
    (dict(red=abi.FLP_REDUCE_NONE), "FLP_INVALID_ARGUMENT"),
    (dict(loss=0), "FLP_INVALID_ARGUMENT"),
    (dict(h=0), "FLP_INVALID_ARGUMENT"),
    (dict(ws=0), "FLP_INVALID_ARGUMENT"),
    (dict(dw=A[7] + 8), "FLP_MISALIGNED"),
    (dict(dh=A[1] + 64), "FLP_INVALID_ARGUMENT"),
    (dict(st=A[4] - 8 * N + 4), "FLP_INVALID_ARGUMENT"),    # the statistics run into the loss
    (dict(ws=A[6] + 16), "FLP_INVALID_ARGUMENT"),
    (dict(wsb=4096), "FLP_WORKSPACE_TOO_SMALL"),
    (dict(wsb=abi.flp_cross_entropy_gradients_workspace_bytes(N, D, V, BF16, 0) - 1),
     "FLP_WORKSPACE_TOO_SMALL"),
    (dict(N=0, loss=0), "FLP_INVALID_ARGUMENT"),
])
def test_cross_entropy_gradients_gates(kw, expect):
    assert ce_all(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), "FLP_INVALID_ARGUMENT"),
    (dict(x=I64), "FLP_UNSUPPORTED_DTYPE"),
    (dict(p=0), "FLP_INVALID_ARGUMENT"),
    (dict(f=0), "FLP_INVALID_ARGUMENT"),
    (dict(p=A[0] + 1), "FLP_MISALIGNED"),
    (dict(f=A[0] + 16), "FLP_INVALID_ARGUMENT"),            # the factor inside x
    (dict(n=0, p=0, f=0), "FLP_OK"),
])
def test_scale_inplace_gates(kw, expect):
    a = dict(n=100, x=BF16, p=A[0], f=A[1])
    a.update(kw)
    assert name(abi.flp_scale_inplace(a["n"], a["x"], a["p"], a["f"], 0)) == expect


def test_gradients_workspace_holds_the_chunk():
    """A whole chunk keeps 4 bytes per logit beside dz and dz^T; the least workspace is a chunk
    of 256 rows or one of all of them, whichever is smaller."""
    size = abi.flp_cross_entropy_gradients_workspace_bytes
    one = size(16384, 2688, 131072, BF16, 16384)
    assert one >= 16384 * 131072 * 8
    assert one <= 24 << 30  # what the Python entry point takes without chunks
    for shape in ((16384, 2688, 131072), (600, 64, 1000), (257, 96, 300)):
        n = shape[0]
        assert size(*shape, BF16, 0) == min(size(*shape, BF16, 256), size(*shape, BF16, n))
    assert size(0, 64, 100, BF16, 0) == 0 and size(10, 64, 100, F16, 0) == 0


def test_cross_entropy_workspace_bytes():
    n_vt = -(-V // 256)
    assert (abi.flp_cross_entropy_forward_workspace_bytes(N, D, V)
            >= abi.flp_forward_workspace_bytes(N, D, V) + n_vt * N * 4 + N * 4)
    assert (abi.flp_cross_entropy_backward_workspace_bytes(N, D, V, BF16, 0)
            >= abi.flp_backward_workspace_bytes(N, D, V, BF16, BF16, 0) + 3 * N * 4 + 4)
    assert abi.flp_cross_entropy_backward_workspace_bytes(0, D, V, BF16, 0) == 0


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
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="reduction"):
        flp.linear_cross_entropy(x, x, t, reduction="average")
    with pytest.raises(ValueError, match="GPU"):
        flp.linear_cross_entropy(x, x, t)


def test_a_status_inside_an_autograd_node_is_the_librarys_error():
    """A tensor that never reached a GPU: the library refuses the call (there is no GPU here, or
    the scale is not finite), and the node's exception is the one of every other entry point."""
    import torch

    from lm_head_selected_bf16_amd import torch_ops
    w = torch.zeros(4, 8, requires_grad=True)
    ids = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(abi.FlpError, match="flp_embedding_scaled_forward failed: "
                                           "FLP_INVALID_ARGUMENT") as e:
        torch_ops._nodes().embedding(w, ids, INF, 0)
    assert e.value.status != 0


@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_differentiation_is_refused(grad):
    """An input with a tangent, whether or not anything requires a gradient: an error, not an
    output without a tangent."""
    from torch.autograd import forward_ad
    x, w, b = torch.ones(4, 32), torch.ones(7, 32), torch.ones(7)
    p, q = torch.ones(32), torch.ones(32)
    ids = torch.zeros(4, dtype=torch.int64)
    rng = torch.zeros(2, dtype=torch.int64)
    calls = [(lambda w: flp.embedding(w, ids), [w]),
             (lambda x: flp.dropout(x, 0.1, rng), [x]),
             (lambda *a: flp.layer_norm(*a), [x, p, q]),
             (lambda x, w, b: flp.linear_cross_entropy(x, w, ids, b), [x, w, b])]
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        for call, args in calls:
            for k, t in enumerate(args):
                dual = forward_ad.make_dual(t, torch.ones_like(t))
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    call(*args[:k], dual, *args[k + 1:])


def test_missing_nodes_are_an_error(monkeypatch):
    import sys

    import lm_head_selected_bf16_amd as m
    from lm_head_selected_bf16_amd import torch_ops
    torch_ops._nodes()
    monkeypatch.setattr(torch_ops, "_NODES", None)
    monkeypatch.delattr(m, "_flp_torch")
    monkeypatch.setitem(sys.modules, "lm_head_selected_bf16_amd._flp_torch", None)
    with pytest.raises(ImportError, match="_flp_torch.so is missing"):
        torch_ops._nodes()
