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
