"""PyTorch-facing wrapper of the C ABI: device buffers, streams and autograd.

Argument marshalling only: shapes are checked and flattened, outputs and
workspaces are allocated with torch on the inputs' device, pointers and the
current HIP stream are passed to libflp.so.  Nothing here computes any part of
the operator.

Semantics ("Fused Linear LogP" docs page, sections "Entry Point" and "Tensor
Contract"): hidden [B, S, D] or [N, D], weight [V, D], targets [B, S] or [N]
(int64 or int32), optional float32 bias [V]; hidden and weight bfloat16, float16 or
float32; output float32 with the leading
shape of targets.  The optional per-row temperature [B, S] / [N] divides the
logits of its row (PR #555 summary).  Gradients flow to hidden, weight and bias;
targets and temperature are not differentiable.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import List, NamedTuple, Optional, Sequence, Tuple, Union

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _abi
from ._abi import FLP_BF16, FLP_F16, FLP_F32, FLP_I32, FLP_I64, FLP_OK, FlpError

# Default cap on the backward workspace: a larger workspace only means larger row
# chunks (same bits); 16 GiB keeps a whole 16384-row chunk of dz and dz^T.
DEFAULT_BWD_WORKSPACE = 16 << 30
# The same for the cross entropy's loss-and-gradients call, which keeps a chunk's fp32 logits as
# well: a whole chunk of 16384 rows over 131072 columns in bfloat16.
DEFAULT_GRADIENTS_WORKSPACE = 24 << 30

_X_DTYPES = {torch.bfloat16: FLP_BF16, torch.float16: FLP_F16, torch.float32: FLP_F32}
_T_DTYPES = {torch.int64: FLP_I64, torch.int32: FLP_I32}


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(device: torch.device) -> int:
    # the raw handle, without the Stream object around it (2 us of a small call)
    return torch._C._cuda_getCurrentRawStream(device.index)


_ON_IT = contextlib.nullcontext()


def _on(device: torch.device):
    """The device as the current one while a call is made (the library works on the current
    HIP device)."""
    if device.index == torch.cuda.current_device():
        return _ON_IT
    return torch.cuda.device(device)


_NODES = None


def _nodes():
    """The autograd nodes of csrc/flp_torch.cpp, bound to the loaded library."""
    global _NODES
    if _NODES is None:
        lib = _abi.load()
        try:
            from . import _flp_torch
        except ModuleNotFoundError as e:
            raise ImportError("_flp_torch.so is missing: build it with `python -m "
                              "lm_head_selected_bf16_amd.build`") from e
        _flp_torch.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                         for name in _abi.SIGNATURES})
        _NODES = _flp_torch
    return _NODES


def _wants_grad(*tensors) -> bool:
    """Whether a gradient is asked for.  Forward-mode differentiation is refused, as the autograd
    nodes refuse it: a plain call would drop the inputs' tangents in silence."""
    if forward_ad._current_level >= 0:  # inside a dual level (unpack_dual: 1 us per tensor)
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("forward-mode differentiation of this operator is not "
                                          "implemented")
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _check(fn: str, status: int) -> None:
    if status != FLP_OK:
        raise FlpError(fn, status)


def _prepare(hidden, weight, targets, bias, temperature):
    if hidden.dtype not in _X_DTYPES or weight.dtype != hidden.dtype:
        raise TypeError("hidden and weight must have the same dtype: bfloat16, float16 or float32")
    if targets.dtype not in _T_DTYPES:
        raise TypeError("targets must be int64 or int32")
    if not (hidden.is_cuda and weight.is_cuda and targets.is_cuda):
        raise ValueError("hidden, weight and targets must be on the GPU")
    for name, t in (("hidden", hidden), ("weight", weight), ("targets", targets),
                    ("bias", bias), ("temperature", temperature)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if weight.dim() != 2 or hidden.shape[-1] != weight.shape[1]:
        raise ValueError("weight must be [V, D] with D = hidden.shape[-1]")
    lead = tuple(targets.shape)
    if tuple(hidden.shape[:-1]) != lead:
        raise ValueError("hidden leading shape must equal the targets shape")
    D = int(hidden.shape[-1])
    V = int(weight.shape[0])
    h2 = hidden.reshape(-1, D)
    t1 = targets.reshape(-1)
    N = int(t1.shape[0])
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (V,)):
        raise ValueError("bias must be float32 [V]")
    temp1 = None
    if temperature is not None:
        if temperature.dtype != torch.float32 or tuple(temperature.shape) != lead:
            raise ValueError("temperature must be float32 with the targets shape")
        temp1 = temperature.reshape(-1)
    return h2, t1, temp1, lead, N, D, V


def forward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
            bias: Optional[torch.Tensor] = None, temperature: Optional[torch.Tensor] = None,
            return_lse: bool = True, workspace: Optional[torch.Tensor] = None
            ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """logp (and lse) float32 with the targets' leading shape, through flp_forward."""
    h2, t1, temp1, lead, N, D, V = _prepare(hidden, weight, targets, bias, temperature)
    dev = hidden.device
    logp = torch.empty(lead, dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev) if return_lse else None
    need = _abi.flp_forward_workspace_bytes(N, D, V)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    st = _abi.flp_forward(N, D, V, _X_DTYPES[hidden.dtype], _ptr(h2), _ptr(weight), _ptr(bias),
                          _ptr(t1), _T_DTYPES[targets.dtype], _ptr(temp1), _ptr(logp), _ptr(lse),
                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                          _stream(dev))
    _check("flp_forward", st)
    return logp, lse


def forward_partial(hidden: torch.Tensor, weight_shard: torch.Tensor, targets: torch.Tensor,
                    vocab_start: int, vocab_size: int, bias_shard: Optional[torch.Tensor] = None,
                    temperature: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-tile (max, sum-of-exp) partials [ceil(V_local / 256), N, 2] and the zt [N] of one
    vocabulary shard (rows vocab_start .. vocab_start + V_local - 1 of the weight), through
    flp_forward_partial.  Targets are global ids; vocab_size is the full vocabulary."""
    h2, t1, temp1, lead, N, D, V_local = _prepare(hidden, weight_shard, targets, bias_shard,
                                                  temperature)
    dev = hidden.device
    partial = torch.empty(((V_local + 255) // 256, N, 2), dtype=torch.float32, device=dev)
    zt = torch.empty(N, dtype=torch.float32, device=dev)
    st = _abi.flp_forward_partial(N, D, V_local, int(vocab_start), int(vocab_size),
                                  _X_DTYPES[hidden.dtype], _ptr(h2), _ptr(weight_shard),
                                  _ptr(bias_shard), _ptr(t1), _T_DTYPES[targets.dtype],
                                  _ptr(temp1), _ptr(partial), _ptr(zt), _stream(dev))
    _check("flp_forward_partial", st)
    return partial, zt


def merge(partials: torch.Tensor, zt: torch.Tensor, targets: torch.Tensor, vocab_size: int,
          return_lse: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """logp (and lse) from the shards' partials concatenated in ascending vocabulary order
    ([ceil(vocab_size / 256), N, 2]) and the sum of their zt, through flp_merge."""
    if targets.dtype not in _T_DTYPES:
        raise TypeError("targets must be int64 or int32")
    lead = tuple(targets.shape)
    t1 = targets.reshape(-1)
    N = int(t1.shape[0])
    n_vt = (int(vocab_size) + 255) // 256
    if (partials.dtype != torch.float32 or tuple(partials.shape) != (n_vt, N, 2)
            or not partials.is_contiguous()):
        raise ValueError(f"partials must be contiguous float32 [{n_vt}, {N}, 2]")
    if zt.dtype != torch.float32 or tuple(zt.shape) != (N,) or not zt.is_contiguous():
        raise ValueError("zt must be contiguous float32 [N]")
    if not t1.is_contiguous():
        raise ValueError("targets must be contiguous")
    dev = partials.device
    logp = torch.empty(lead, dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev) if return_lse else None
    st = _abi.flp_merge(N, int(vocab_size), _ptr(partials), _ptr(zt), _ptr(t1),
                        _T_DTYPES[targets.dtype], _ptr(logp), _ptr(lse), _stream(dev))
    _check("flp_merge", st)
    return logp, lse


def backward_workspace_bytes(N: int, D: int, V: int, x_dtype: torch.dtype,
                             dw_dtype: Optional[torch.dtype] = None, chunk_rows: int = 0) -> int:
    dw = _X_DTYPES[x_dtype if dw_dtype is None else dw_dtype]
    return _abi.flp_backward_workspace_bytes(N, D, V, _X_DTYPES[x_dtype], dw, chunk_rows)


def default_backward_workspace_bytes(N: int, D: int, V: int, x_dtype: torch.dtype,
                                     dw_dtype: Optional[torch.dtype] = None,
                                     cap: int = DEFAULT_BWD_WORKSPACE) -> int:
    """The whole batch as one chunk if that fits under ``cap``, else the minimum
    plus as many 256-row quanta as fit (same bits either way)."""
    full = backward_workspace_bytes(N, D, V, x_dtype, dw_dtype, chunk_rows=max(N, 1))
    if full <= cap:
        return full
    lo = backward_workspace_bytes(N, D, V, x_dtype, dw_dtype, chunk_rows=0)
    return max(lo, cap)


def backward(grad_out: torch.Tensor, lse: torch.Tensor, hidden: torch.Tensor, weight: torch.Tensor,
             targets: torch.Tensor, bias: Optional[torch.Tensor] = None,
             temperature: Optional[torch.Tensor] = None, need_hidden: bool = True,
             need_weight: bool = True, need_bias: Optional[bool] = None,
             dw_dtype: Optional[torch.dtype] = None, workspace_bytes: Optional[int] = None,
             workspace: Optional[torch.Tensor] = None):
    """(d_hidden, d_weight, d_bias) through flp_backward; unrequested ones are None."""
    h2, t1, temp1, lead, N, D, V = _prepare(hidden, weight, targets, bias, temperature)
    dev = hidden.device
    if need_bias is None:
        need_bias = bias is not None
    if grad_out.dtype != torch.float32 or tuple(grad_out.shape) != lead or not grad_out.is_contiguous():
        raise ValueError("grad_out must be contiguous float32 with the targets shape")
    if lse.dtype != torch.float32 or tuple(lse.shape) != lead or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 with the targets shape")
    dwt = hidden.dtype if dw_dtype is None else dw_dtype
    d_hidden = torch.empty_like(hidden) if need_hidden else None
    d_weight = torch.empty(weight.shape, dtype=dwt, device=dev) if need_weight else None
    d_bias = torch.empty(V, dtype=torch.float32, device=dev) if need_bias else None
    if workspace is None:
        if workspace_bytes is None:
            workspace_bytes = default_backward_workspace_bytes(N, D, V, hidden.dtype, dwt)
        workspace = torch.empty(max(int(workspace_bytes), 16), dtype=torch.uint8, device=dev)
    st = _abi.flp_backward(N, D, V, _X_DTYPES[hidden.dtype], _ptr(grad_out), _ptr(lse), _ptr(h2),
                           _ptr(weight), _ptr(bias), _ptr(t1), _T_DTYPES[targets.dtype],
                           _ptr(temp1), _ptr(d_hidden), _ptr(d_weight), _X_DTYPES[dwt],
                           _ptr(d_bias), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(dev))
    _check("flp_backward", st)
    return d_hidden, d_weight, d_bias


class LinearLogp(torch.autograd.Function):
    """Autograd node: the forward saves lse; the backward recomputes the logits."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, bias, temperature):
        logp, lse = forward(hidden, weight, targets, bias, temperature, return_lse=True)
        ctx.save_for_backward(hidden, weight, targets, bias, temperature, lse)
        ctx.mark_non_differentiable(lse)
        return logp, lse

    @staticmethod
    def backward(ctx, g_logp, g_lse):
        hidden, weight, targets, bias, temperature, lse = ctx.saved_tensors
        need_h, need_w, _, need_b, _ = ctx.needs_input_grad
        if not (need_h or need_w or need_b):
            return None, None, None, None, None
        g = g_logp.contiguous().to(torch.float32)
        dh, dw, db = backward(g, lse, hidden, weight, targets, bias, temperature,
                              need_hidden=need_h, need_weight=need_w,
                              need_bias=bool(need_b and bias is not None))
        return dh, dw, None, db, None


def linear_logp_with_lse(hidden, weight, targets, bias=None, temperature=None):
    """(logp, lse): selected-token log-probabilities and the per-row log-sum-exp."""
    return LinearLogp.apply(hidden, weight, targets, bias, temperature)


def linear_logp(hidden, weight, targets, bias=None, temperature=None):
    """logp[..] = log_softmax((hidden @ weight^T + bias) / T)[target], 0 for out-of-range targets."""
    return linear_logp_with_lse(hidden, weight, targets, bias, temperature)[0]


# ---- the operator on materialised logits ------------------------------------------------------

def _prepare_logits(logits, targets):
    if logits.dtype not in _X_DTYPES:
        raise TypeError("logits must be bfloat16, float16 or float32")
    if targets.dtype not in _T_DTYPES:
        raise TypeError("targets must be int64 or int32")
    if not (logits.is_cuda and targets.is_cuda):
        raise ValueError("logits and targets must be on the GPU")
    if not (logits.is_contiguous() and targets.is_contiguous()):
        raise ValueError("logits and targets must be contiguous")
    lead = tuple(targets.shape)
    if tuple(logits.shape[:-1]) != lead:
        raise ValueError("logits leading shape must equal the targets shape")
    V = int(logits.shape[-1])
    t1 = targets.reshape(-1)
    return logits.reshape(-1, V), t1, lead, int(t1.shape[0]), V


def logits_forward(logits: torch.Tensor, targets: torch.Tensor, return_lse: bool = True
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """logp (and lse) of given logits [.., V] through flp_logits_forward."""
    z2, t1, lead, N, V = _prepare_logits(logits, targets)
    dev = logits.device
    logp = torch.empty(lead, dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev) if return_lse else None
    st = _abi.flp_logits_forward(N, V, _X_DTYPES[logits.dtype], _ptr(z2), _ptr(t1),
                                 _T_DTYPES[targets.dtype], _ptr(logp), _ptr(lse), _stream(dev))
    _check("flp_logits_forward", st)
    return logp, lse


def logits_backward(grad_out: torch.Tensor, lse: torch.Tensor, logits: torch.Tensor,
                    targets: torch.Tensor) -> torch.Tensor:
    """d logits (logits dtype) through flp_logits_backward."""
    z2, t1, lead, N, V = _prepare_logits(logits, targets)
    for name, x in (("grad_out", grad_out), ("lse", lse)):
        if x.dtype != torch.float32 or tuple(x.shape) != lead or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with the targets shape")
    d = torch.empty_like(logits)
    st = _abi.flp_logits_backward(N, V, _X_DTYPES[logits.dtype], _ptr(grad_out), _ptr(lse),
                                  _ptr(z2), _ptr(t1), _T_DTYPES[targets.dtype], _ptr(d),
                                  _stream(logits.device))
    _check("flp_logits_backward", st)
    return d


class LogitsLogp(torch.autograd.Function):
    """Autograd node of the operator on materialised logits; the forward saves lse."""

    @staticmethod
    def forward(ctx, logits, targets):
        logp, lse = logits_forward(logits, targets, return_lse=True)
        ctx.save_for_backward(logits, targets, lse)
        return logp

    @staticmethod
    def backward(ctx, g_logp):
        logits, targets, lse = ctx.saved_tensors
        if not ctx.needs_input_grad[0]:
            return None, None
        return logits_backward(g_logp.contiguous().to(torch.float32), lse, logits, targets), None


def logits_logp(logits, targets):
    """logp[..] = log_softmax(logits)[target], 0 for out-of-range targets (differentiable)."""
    return LogitsLogp.apply(logits, targets)


# ---- indexed (row-subset) variants ------------------------------------------------------------
#
# rows: 1-D int64 / int32 ids into the flattened batch (PR #547 "What", indexed
# semantics): outputs keep the full row shape, a duplicated id selects its row
# once, ids outside [0, N) are ignored, rows left out get logp = lse = 0 and zero
# gradients; d_weight and d_bias sum over the selected rows.

def _prepare_rows(rows: torch.Tensor, dev: torch.device):
    if rows.dtype not in _T_DTYPES:
        raise TypeError("rows must be int64 or int32")
    if rows.dim() != 1 or not rows.is_contiguous() or rows.device != dev:
        raise ValueError("rows must be a contiguous 1-D tensor on the inputs' device")
    return rows, int(rows.shape[0]), _T_DTYPES[rows.dtype]


def forward_indexed(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                    rows: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    temperature: Optional[torch.Tensor] = None, return_lse: bool = True
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """logp (and lse) of the selected rows, zeros elsewhere, through flp_forward_indexed."""
    h2, t1, temp1, lead, N, D, V = _prepare(hidden, weight, targets, bias, temperature)
    dev = hidden.device
    rows, n_rows, r_dt = _prepare_rows(rows, dev)
    logp = torch.empty(lead, dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev) if return_lse else None
    need = _abi.flp_forward_indexed_workspace_bytes(N, D, V, _X_DTYPES[hidden.dtype], n_rows)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    st = _abi.flp_forward_indexed(N, D, V, _X_DTYPES[hidden.dtype], _ptr(h2), _ptr(weight),
                                  _ptr(bias), _ptr(t1), _T_DTYPES[targets.dtype], _ptr(temp1),
                                  _ptr(rows), r_dt, n_rows, _ptr(logp), _ptr(lse), _ptr(ws),
                                  ws.numel(), _stream(dev))
    _check("flp_forward_indexed", st)
    return logp, lse


def backward_indexed(grad_out: torch.Tensor, lse: torch.Tensor, hidden: torch.Tensor,
                     weight: torch.Tensor, targets: torch.Tensor, rows: torch.Tensor,
                     bias: Optional[torch.Tensor] = None,
                     temperature: Optional[torch.Tensor] = None, need_hidden: bool = True,
                     need_weight: bool = True, need_bias: Optional[bool] = None,
                     dw_dtype: Optional[torch.dtype] = None,
                     workspace_bytes: Optional[int] = None):
    """(d_hidden, d_weight, d_bias) of the selected rows through flp_backward_indexed."""
    h2, t1, temp1, lead, N, D, V = _prepare(hidden, weight, targets, bias, temperature)
    dev = hidden.device
    rows, n_rows, r_dt = _prepare_rows(rows, dev)
    if need_bias is None:
        need_bias = bias is not None
    for name, x in (("grad_out", grad_out), ("lse", lse)):
        if x.dtype != torch.float32 or tuple(x.shape) != lead or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with the targets shape")
    dwt = hidden.dtype if dw_dtype is None else dw_dtype
    xd, wd = _X_DTYPES[hidden.dtype], _X_DTYPES[dwt]
    d_hidden = torch.empty_like(hidden) if need_hidden else None
    d_weight = torch.empty(weight.shape, dtype=dwt, device=dev) if need_weight else None
    d_bias = torch.empty(V, dtype=torch.float32, device=dev) if need_bias else None
    if workspace_bytes is None:
        cap = max(min(n_rows, N), 1)
        workspace_bytes = _abi.flp_backward_indexed_workspace_bytes(N, D, V, xd, wd, n_rows, cap)
        if workspace_bytes > DEFAULT_BWD_WORKSPACE:
            workspace_bytes = max(DEFAULT_BWD_WORKSPACE,
                                  _abi.flp_backward_indexed_workspace_bytes(N, D, V, xd, wd,
                                                                            n_rows, 0))
    ws = torch.empty(max(int(workspace_bytes), 16), dtype=torch.uint8, device=dev)
    st = _abi.flp_backward_indexed(N, D, V, xd, _ptr(grad_out), _ptr(lse), _ptr(h2),
                                   _ptr(weight), _ptr(bias), _ptr(t1), _T_DTYPES[targets.dtype],
                                   _ptr(temp1), _ptr(rows), r_dt, n_rows, _ptr(d_hidden),
                                   _ptr(d_weight), wd, _ptr(d_bias), _ptr(ws), ws.numel(),
                                   _stream(dev))
    _check("flp_backward_indexed", st)
    return d_hidden, d_weight, d_bias


class LinearLogpIndexed(torch.autograd.Function):
    """Autograd node of the indexed linear operator; the forward saves lse."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, rows, bias, temperature):
        logp, lse = forward_indexed(hidden, weight, targets, rows, bias, temperature)
        ctx.save_for_backward(hidden, weight, targets, rows, bias, temperature, lse)
        ctx.mark_non_differentiable(lse)
        return logp, lse

    @staticmethod
    def backward(ctx, g_logp, g_lse):
        hidden, weight, targets, rows, bias, temperature, lse = ctx.saved_tensors
        need_h, need_w, _, _, need_b, _ = ctx.needs_input_grad
        if not (need_h or need_w or need_b):
            return None, None, None, None, None, None
        dh, dw, db = backward_indexed(g_logp.contiguous().to(torch.float32), lse, hidden, weight,
                                      targets, rows, bias, temperature, need_hidden=need_h,
                                      need_weight=need_w,
                                      need_bias=bool(need_b and bias is not None))
        return dh, dw, None, None, db, None


def linear_logp_indexed(hidden, weight, targets, rows, bias=None, temperature=None):
    """linear_logp restricted to the rows listed in ``rows`` (full shape, zeros elsewhere)."""
    return LinearLogpIndexed.apply(hidden, weight, targets, rows, bias, temperature)[0]


def logits_forward_indexed(logits: torch.Tensor, targets: torch.Tensor, rows: torch.Tensor,
                           return_lse: bool = True
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """logp (and lse) of the selected rows of given logits through flp_logits_forward_indexed."""
    z2, t1, lead, N, V = _prepare_logits(logits, targets)
    dev = logits.device
    rows, n_rows, r_dt = _prepare_rows(rows, dev)
    logp = torch.empty(lead, dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev) if return_lse else None
    ws = torch.empty(max(_abi.flp_logits_indexed_workspace_bytes(N), 16), dtype=torch.uint8,
                     device=dev)
    st = _abi.flp_logits_forward_indexed(N, V, _X_DTYPES[logits.dtype], _ptr(z2), _ptr(t1),
                                         _T_DTYPES[targets.dtype], _ptr(rows), r_dt, n_rows,
                                         _ptr(logp), _ptr(lse), _ptr(ws), ws.numel(), _stream(dev))
    _check("flp_logits_forward_indexed", st)
    return logp, lse


def logits_backward_indexed(grad_out: torch.Tensor, lse: torch.Tensor, logits: torch.Tensor,
                            targets: torch.Tensor, rows: torch.Tensor) -> torch.Tensor:
    """d logits of the selected rows (zero rows elsewhere) through flp_logits_backward_indexed."""
    z2, t1, lead, N, V = _prepare_logits(logits, targets)
    dev = logits.device
    rows, n_rows, r_dt = _prepare_rows(rows, dev)
    for name, x in (("grad_out", grad_out), ("lse", lse)):
        if x.dtype != torch.float32 or tuple(x.shape) != lead or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with the targets shape")
    d = torch.empty_like(logits)
    ws = torch.empty(max(_abi.flp_logits_indexed_workspace_bytes(N), 16), dtype=torch.uint8,
                     device=dev)
    st = _abi.flp_logits_backward_indexed(N, V, _X_DTYPES[logits.dtype], _ptr(grad_out),
                                          _ptr(lse), _ptr(z2), _ptr(t1), _T_DTYPES[targets.dtype],
                                          _ptr(rows), r_dt, n_rows, _ptr(d), _ptr(ws), ws.numel(),
                                          _stream(dev))
    _check("flp_logits_backward_indexed", st)
    return d


class LogitsLogpIndexed(torch.autograd.Function):
    """Autograd node of the indexed operator on materialised logits."""

    @staticmethod
    def forward(ctx, logits, targets, rows):
        logp, lse = logits_forward_indexed(logits, targets, rows, return_lse=True)
        ctx.save_for_backward(logits, targets, rows, lse)
        return logp

    @staticmethod
    def backward(ctx, g_logp):
        logits, targets, rows, lse = ctx.saved_tensors
        if not ctx.needs_input_grad[0]:
            return None, None, None
        d = logits_backward_indexed(g_logp.contiguous().to(torch.float32), lse, logits, targets,
                                    rows)
        return d, None, None


def logits_logp_indexed(logits, targets, rows):
    """logits_logp restricted to the rows listed in ``rows`` (full shape, zeros elsewhere)."""
    return LogitsLogpIndexed.apply(logits, targets, rows)


# ---- untied embedding lookup -------------------------------------------------------------------
#
# out = weight[ids] (a zero row for ids outside [0, V)); d_weight sums the gradient rows of each
# id in ascending token order in fp32 (PR #555 summary bullets: sorted-segment deterministic
# grad_weight).

def _prepare_embedding(weight, ids):
    if weight.dtype not in _X_DTYPES:
        raise TypeError("weight must be bfloat16, float16 or float32")
    if ids.dtype not in _T_DTYPES:
        raise TypeError("ids must be int64 or int32")
    if not (weight.is_cuda and ids.is_cuda):
        raise ValueError("weight and ids must be on the GPU")
    if weight.dim() != 2 or not weight.is_contiguous() or not ids.is_contiguous():
        raise ValueError("weight must be a contiguous [V, D] tensor and ids contiguous")
    V, D = int(weight.shape[0]), int(weight.shape[1])
    return V, D, ids.reshape(-1), int(ids.numel())


def _embedding_scale(scale) -> float:
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    return scale


def embedding_forward(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """scale * weight[ids] with the ids' shape + [D], through flp_embedding_scaled_forward."""
    V, D, i1, N = _prepare_embedding(weight, ids)
    scale = _embedding_scale(scale)
    dev = weight.device
    if ids.device != dev:
        raise ValueError("weight and ids must be on one device")
    with _on(dev):
        out = torch.empty(tuple(ids.shape) + (D,), dtype=weight.dtype, device=dev)
        st = _abi.flp_embedding_scaled_forward(N, D, V, _X_DTYPES[weight.dtype], _ptr(weight),
                                               _ptr(i1), _T_DTYPES[ids.dtype], scale, _ptr(out),
                                               _stream(dev))
    _check("flp_embedding_scaled_forward", st)
    return out


def embedding_backward(grad: torch.Tensor, ids: torch.Tensor, num_embeddings: int,
                       dw_dtype: Optional[torch.dtype] = None, scale: float = 1.0) -> torch.Tensor:
    """d_weight [V, D] of sum(grad * scale * weight[ids]) through flp_embedding_scaled_backward."""
    if grad.dtype not in _X_DTYPES or not grad.is_contiguous() or not grad.is_cuda:
        raise ValueError("grad must be a contiguous bfloat16 / float16 / float32 GPU tensor")
    if ids.dtype not in _T_DTYPES or not ids.is_contiguous():
        raise ValueError("ids must be contiguous int64 or int32")
    D = int(grad.shape[-1])
    if tuple(grad.shape[:-1]) != tuple(ids.shape):
        raise ValueError("grad must have the ids' shape + [D]")
    scale = _embedding_scale(scale)
    N, V = int(ids.numel()), int(num_embeddings)
    dwt = grad.dtype if dw_dtype is None else dw_dtype
    dev = grad.device
    if ids.device != dev:
        raise ValueError("grad and ids must be on one device")
    with _on(dev):
        d_weight = torch.empty((V, D), dtype=dwt, device=dev)
        size = max(_abi.flp_embedding_backward_workspace_bytes(N, D, V), 16)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        st = _abi.flp_embedding_scaled_backward(N, D, V, _X_DTYPES[grad.dtype], grad.data_ptr(),
                                                ids.data_ptr(), _T_DTYPES[ids.dtype], scale,
                                                d_weight.data_ptr(), _X_DTYPES[dwt],
                                                ws.data_ptr(), size, _stream(dev))
    _check("flp_embedding_scaled_backward", st)
    return d_weight


class Embedding(torch.autograd.Function):
    """Autograd node of the lookup in Python, over libflp.so alone; the ids are not
    differentiable.  embedding() takes the node of csrc/flp_torch.cpp, with the same bits."""

    @staticmethod
    def forward(ctx, weight, ids, scale=1.0):
        ctx.save_for_backward(ids)
        ctx.num_embeddings, ctx.scale = int(weight.shape[0]), scale
        return embedding_forward(weight, ids, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        (ids,) = ctx.saved_tensors
        if not ctx.needs_input_grad[0]:
            return None, None, None
        grad = grad.contiguous()
        if grad.data_ptr() % 16:  # a dense view at any offset of its storage
            grad = grad.clone()
        return embedding_backward(grad, ids, ctx.num_embeddings, scale=ctx.scale), None, None


def embedding(weight, ids, scale=1.0):
    """scale * weight[ids] (zero rows for ids outside [0, V)), differentiable in weight."""
    if not _wants_grad(weight):
        return embedding_forward(weight, ids, scale)
    _prepare_embedding(weight, ids)
    dev = weight.device
    if ids.device != dev:
        raise ValueError("weight and ids must be on one device")
    with _on(dev):
        return _nodes().embedding(weight, ids, _embedding_scale(scale), _stream(dev))


# ---- linear cross entropy -----------------------------------------------------------------------
#
# The training loss of the head: -logp with label smoothing, a squared log-partition term and a
# reduction, without an [N, V] tensor of logits.  Targets outside [0, V) are padding: loss 0, not
# counted, zero gradients.

_REDUCTIONS = {"none": _abi.FLP_REDUCE_NONE, "sum": _abi.FLP_REDUCE_SUM,
               "mean": _abi.FLP_REDUCE_MEAN}


def _chunked_workspace(size: int, least: int, device) -> torch.Tensor:
    """A workspace of `size` bytes, or of as many, halved as often as needed and at least `least`,
    as the device has room for: a smaller one runs more row chunks, with the same bits."""
    while True:
        try:
            return torch.empty(max(size, 16), dtype=torch.uint8, device=device)
        except torch.OutOfMemoryError:
            if size <= least:
                raise
            size = max(size // 2, least)


def _prepare_loss(hidden, weight, targets, bias, reduction):
    if reduction not in _REDUCTIONS:
        raise ValueError("reduction must be 'none', 'sum' or 'mean'")
    prep = _prepare(hidden, weight, targets, bias, None)
    if any(t is not None and t.device != hidden.device for t in (weight, targets, bias)):
        raise ValueError("hidden, weight, targets and bias must be on one device")
    return prep, _REDUCTIONS[reduction]


def cross_entropy_forward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                          bias: Optional[torch.Tensor] = None, label_smoothing: float = 0.0,
                          z_loss: float = 0.0, reduction: str = "mean", return_stats: bool = True
                          ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(loss, stats) through flp_cross_entropy_forward: loss float32 with the targets' shape
    (reduction "none") or a scalar; stats float32 [2, *targets' shape], stats[0] = lse."""
    (h2, t1, _, lead, N, D, V), red = _prepare_loss(hidden, weight, targets, bias, reduction)
    dev = hidden.device
    with _on(dev):
        loss = torch.empty(lead if reduction == "none" else (), dtype=torch.float32, device=dev)
        stats = None
        if return_stats:
            stats = torch.empty((2,) + lead, dtype=torch.float32, device=dev)
        ws = torch.empty(max(_abi.flp_cross_entropy_forward_workspace_bytes(N, D, V), 16),
                         dtype=torch.uint8, device=dev)
        st = _abi.flp_cross_entropy_forward(N, D, V, _X_DTYPES[hidden.dtype], _ptr(h2),
                                            _ptr(weight), _ptr(bias), _ptr(t1),
                                            _T_DTYPES[targets.dtype], float(label_smoothing),
                                            float(z_loss), red, _ptr(loss), _ptr(stats), _ptr(ws),
                                            ws.numel(), _stream(dev))
    _check("flp_cross_entropy_forward", st)
    return loss, stats


def cross_entropy_backward(grad_out: torch.Tensor, stats: torch.Tensor, hidden: torch.Tensor,
                           weight: torch.Tensor, targets: torch.Tensor,
                           bias: Optional[torch.Tensor] = None, label_smoothing: float = 0.0,
                           z_loss: float = 0.0, reduction: str = "mean", need_hidden: bool = True,
                           need_weight: bool = True, need_bias: Optional[bool] = None,
                           workspace_bytes: Optional[int] = None):
    """(d_hidden, d_weight, d_bias) through flp_cross_entropy_backward; unrequested ones are
    None.  grad_out: float32, of the loss's shape.  The workspace is as large as the backward of
    linear_logp takes by default, or as the device has room for; a smaller one runs more row
    chunks with the same bits."""
    (h2, t1, _, lead, N, D, V), red = _prepare_loss(hidden, weight, targets, bias, reduction)
    dev = hidden.device
    want = lead if reduction == "none" else ()
    for name, x, shape in (("grad_out", grad_out, want), ("stats", stats, (2,) + lead)):
        if (x.dtype != torch.float32 or tuple(x.shape) != shape or not x.is_contiguous()
                or x.device != dev):
            raise ValueError(f"{name} must be contiguous float32 of shape {tuple(shape)} on the "
                             "device of hidden")
    if need_bias is None:
        need_bias = bias is not None
    xd = _X_DTYPES[hidden.dtype]
    size = _abi.flp_cross_entropy_backward_workspace_bytes
    most = least = workspace_bytes
    if workspace_bytes is None:
        most, least = size(N, D, V, xd, max(N, 1)), size(N, D, V, xd, 0)
        most = min(most, max(least, DEFAULT_BWD_WORKSPACE))
    with _on(dev):
        d_hidden = torch.empty_like(hidden) if need_hidden else None
        d_weight = torch.empty_like(weight) if need_weight else None
        d_bias = torch.empty(V, dtype=torch.float32, device=dev) if need_bias else None
        ws = _chunked_workspace(int(most), int(least), dev)
        st = _abi.flp_cross_entropy_backward(N, D, V, xd, _ptr(grad_out), _ptr(stats), _ptr(h2),
                                             _ptr(weight), _ptr(bias), _ptr(t1),
                                             _T_DTYPES[targets.dtype], float(label_smoothing),
                                             float(z_loss), red, _ptr(d_hidden), _ptr(d_weight),
                                             _ptr(d_bias), _ptr(ws), ws.numel(), _stream(dev))
    _check("flp_cross_entropy_backward", st)
    return d_hidden, d_weight, d_bias


def cross_entropy_gradients(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                            bias: Optional[torch.Tensor] = None, label_smoothing: float = 0.0,
                            z_loss: float = 0.0, reduction: str = "mean",
                            need_hidden: bool = True, need_weight: bool = True,
                            need_bias: Optional[bool] = None,
                            workspace_bytes: Optional[int] = None):
    """(loss, stats, d_hidden, d_weight, d_bias) for an upstream gradient of 1 through
    flp_cross_entropy_gradients (bfloat16 or float32, reduction "sum" or "mean"): the bits of
    cross_entropy_forward and cross_entropy_backward with one matrix product less."""
    (h2, t1, _, lead, N, D, V), red = _prepare_loss(hidden, weight, targets, bias, reduction)
    dev = hidden.device
    if need_bias is None:
        need_bias = bias is not None
    xd = _X_DTYPES[hidden.dtype]
    size = _abi.flp_cross_entropy_gradients_workspace_bytes
    most = least = workspace_bytes
    if workspace_bytes is None:
        most, least = size(N, D, V, xd, max(N, 1)), size(N, D, V, xd, 0)
        most = min(most, max(least, DEFAULT_GRADIENTS_WORKSPACE))
    with _on(dev):
        loss = torch.empty((), dtype=torch.float32, device=dev)
        stats = torch.empty((2,) + lead, dtype=torch.float32, device=dev)
        d_hidden = torch.empty_like(hidden) if need_hidden else None
        d_weight = torch.empty_like(weight) if need_weight else None
        d_bias = torch.empty(V, dtype=torch.float32, device=dev) if need_bias else None
        ws = _chunked_workspace(int(most), int(least), dev)
        st = _abi.flp_cross_entropy_gradients(N, D, V, xd, _ptr(h2), _ptr(weight), _ptr(bias),
                                              _ptr(t1), _T_DTYPES[targets.dtype],
                                              float(label_smoothing), float(z_loss), red,
                                              _ptr(loss), _ptr(stats), _ptr(d_hidden),
                                              _ptr(d_weight), _ptr(d_bias), _ptr(ws), ws.numel(),
                                              _stream(dev))
    _check("flp_cross_entropy_gradients", st)
    return loss, stats, d_hidden, d_weight, d_bias


def _gradients_at_once(hidden, weight, reduction) -> bool:
    """Whether a training step's loss and gradients come from one call (the same bits).  It saves
    a product of N D V multiply-adds and moves 8 bytes per logit more, and a few launches more:
    measured on MI355X, it wins from D = 1024 on in bfloat16 (4096 x 512 x 50257: 1090 us in two
    calls, 1207 in one; 4096 x 2048 x 50257: 3092 and 2816), in float32 where its tiles of 256
    rows by 256 columns give most compute units a workgroup (the two calls take smaller ones:
    1000 x 1024 x 8192 548 us in two calls, 556 in one, 1000 x 512 x 16384 560 and 464), and where
    that product takes 20 us."""
    D = hidden.shape[-1]
    N, V = hidden.numel() // max(D, 1), weight.shape[0]
    if reduction == "none":
        return False
    if hidden.dtype == torch.bfloat16:
        return D >= 1024 and N * D * V >= 2 * 10 ** 10
    tiles = -(-N // 256) * -(-V // 256)
    return (hidden.dtype == torch.float32 and D >= 128 and N > 128 and tiles >= 192
            and N * D * V >= 2 * 10 ** 9)


class LossAndGradients(torch.autograd.Function):
    """Autograd node of the linear cross entropy where its forward makes the gradients for an
    upstream gradient of 1 along with the loss: the first backward multiplies them by the
    upstream gradient in place (a second rounding unless that is a power of two) and hands them
    over.  Any further backward through the same node recomputes.  Once a graph capture has seen
    the forward or a backward, the gradients stay as they are, since a replay fills or reads them
    again, and every backward hands over copies."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, bias, label_smoothing, z_loss, reduction):
        ctx.terms = (label_smoothing, z_loss, reduction)
        need_h, need_w, _, need_b = ctx.needs_input_grad[:4]
        loss, stats, *ctx.grads = cross_entropy_gradients(
            hidden, weight, targets, bias, *ctx.terms, need_hidden=need_h, need_weight=need_w,
            need_bias=need_b)
        ctx.replayed = torch.cuda.is_current_stream_capturing()
        ctx.save_for_backward(hidden, weight, targets, bias, stats)
        return loss

    @staticmethod
    def backward(ctx, g):
        ctx.replayed = ctx.replayed or torch.cuda.is_current_stream_capturing()
        if ctx.grads is not None and ctx.replayed:
            grads = [None if x is None else _scaled(x.clone(), g) for x in ctx.grads]
        elif ctx.grads is not None:
            grads, ctx.grads = [_scaled(x, g) for x in ctx.grads], None
        else:
            hidden, weight, targets, bias, stats = ctx.saved_tensors
            need_h, need_w, _, need_b = ctx.needs_input_grad[:4]
            grads = cross_entropy_backward(g.contiguous(), stats, hidden, weight, targets, bias,
                                           *ctx.terms, need_hidden=need_h, need_weight=need_w,
                                           need_bias=need_b)
        if torch.is_grad_enabled():  # a graph of the backward is asked for: it has none
            grads = [None if x is None else _nodes().first_order(x) for x in grads]
        dh, dw, db = grads
        return dh, dw, None, db, None, None, None


def _scaled(x, factor):
    """x *= factor in place (a scalar float32 tensor), through flp_scale_inplace."""
    if x is not None:
        with _on(x.device):
            st = _abi.flp_scale_inplace(x.numel(), _X_DTYPES[x.dtype], x.data_ptr(),
                                        factor.data_ptr(), _stream(x.device))
        _check("flp_scale_inplace", st)
    return x


def linear_cross_entropy(hidden, weight, targets, bias=None, label_smoothing=0.0, z_loss=0.0,
                         reduction="mean"):
    """Cross entropy of hidden @ weight^T + bias against targets, differentiable in hidden, weight
    and bias:

        (1 - s) (lse - z[target]) + s (lse - mean(z)) + z_loss lse^2,   s = label_smoothing

    per row ("none"), summed ("sum") or averaged over the rows whose target lies in [0, V)
    ("mean", 0 when there are none); the other rows are padding with loss 0 and no gradient.

    Where that is faster (reduced bfloat16 losses from D = 1024 on and large float32 ones, see
    _gradients_at_once) the call makes the gradients along with the loss when one is asked for:
    - it takes the three products of a whole step at once, so a loss without a backward belongs
      under torch.no_grad();
    - its workspace, freed on return, holds a row chunk's fp32 logits beside dz and dz^T: 8 bytes
      per logit in bfloat16, 12 in float32, up to torch_ops.DEFAULT_GRADIENTS_WORKSPACE (24 GiB)
      or what the device has room for;
    - the gradients stay on the node until its first backward, which multiplies them by the
      upstream gradient: one more rounding to their type unless that is a power of two.
    cross_entropy_forward and cross_entropy_backward make none of these choices."""
    if not _wants_grad(hidden, weight, bias):
        return cross_entropy_forward(hidden, weight, targets, bias, label_smoothing, z_loss,
                                     reduction, return_stats=False)[0]
    if _gradients_at_once(hidden, weight, reduction):
        return LossAndGradients.apply(hidden, weight, targets, bias, label_smoothing, z_loss,
                                      reduction)
    _, red = _prepare_loss(hidden, weight, targets, bias, reduction)
    dev = hidden.device
    with _on(dev):
        return _nodes().cross_entropy(hidden, weight, targets, bias, label_smoothing, z_loss, red,
                                      DEFAULT_BWD_WORKSPACE, _stream(dev))


# ---- dropout ------------------------------------------------------------------------------------
#
# The mask is a function of the element's position, p and rng (int64 [2] on the device: seed and
# offset), so it is drawn again in the backward instead of being stored.

def _prepare_dropout(x, p, rng) -> float:
    if x.dtype not in _X_DTYPES:
        raise TypeError("x must be bfloat16, float16 or float32")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous GPU tensor")
    if rng.dtype != torch.int64 or tuple(rng.shape) != (2,):
        raise ValueError("rng must be int64 [2]: seed and offset")
    if rng.device != x.device or not rng.is_contiguous():
        raise ValueError("rng must be contiguous and on the device of x")
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be between 0 and 1")
    return p


def dropout_forward(x: torch.Tensor, p: float, rng: torch.Tensor) -> torch.Tensor:
    """x with each element dropped with probability p and the others scaled, through flp_dropout."""
    p = _prepare_dropout(x, p, rng)
    dev = x.device
    with _on(dev):
        out = torch.empty_like(x)
        st = _abi.flp_dropout(x.numel(), _X_DTYPES[x.dtype], x.data_ptr(), p, rng.data_ptr(),
                              out.data_ptr(), _stream(dev))
    _check("flp_dropout", st)
    return out


def dropout(x, p, rng):
    """x with each element dropped with probability p and the others times 1 / (1 - p),
    differentiable in x.  rng: int64 [2] on the device of x, (seed, offset); give every call of a
    step its own offset.  The backward reads rng again, so write a new pair into a new tensor
    rather than changing this one before the backward has run."""
    if not _wants_grad(x):
        return dropout_forward(x, p, rng)
    p = _prepare_dropout(x, p, rng)
    dev = x.device
    with _on(dev):
        return _nodes().dropout(x, p, rng, _stream(dev))


# ---- layer norm ---------------------------------------------------------------------------------

def _prepare_norm(x, weight, bias):
    if x.dtype not in _X_DTYPES:
        raise TypeError("x must be bfloat16, float16 or float32")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least one element")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous GPU tensor")
    D = int(x.shape[-1])
    wd = x.dtype
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        if t.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"{name} must have the dtype of x or float32")
        if tuple(t.shape) != (D,) or not t.is_contiguous() or t.device != x.device:
            raise ValueError(f"{name} must be contiguous [D] on the device of x")
        wd = t.dtype
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    return x.numel() // D, D, wd


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       return_stats: bool = True):
    """(out, mean, rstd) of the layer norm over the last dimension through
    flp_layer_norm_forward; mean and rstd are float32 of the leading shape, or None."""
    N, D, wd = _prepare_norm(x, weight, bias)
    dev = x.device
    with _on(dev):
        out = torch.empty_like(x)
        mean = rstd = None
        if return_stats:
            mean, rstd = torch.empty((2,) + x.shape[:-1], dtype=torch.float32, device=dev)
        st = _abi.flp_layer_norm_forward(N, D, _X_DTYPES[x.dtype], x.data_ptr(), _X_DTYPES[wd],
                                         _ptr(weight), _ptr(bias), float(eps), out.data_ptr(),
                                         _ptr(mean), _ptr(rstd), _stream(dev))
    _check("flp_layer_norm_forward", st)
    return out, mean, rstd


def layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                        need_input: bool = True, need_weight: bool = True, need_bias: bool = True,
                        w_dtype: Optional[torch.dtype] = None):
    """(d_x, d_weight, d_bias) through flp_layer_norm_backward; unrequested ones are None.
    d_weight and d_bias have w_dtype (the weight's, by default)."""
    _, D, wd = _prepare_norm(x, weight, None)
    if w_dtype is not None:
        if w_dtype not in (x.dtype, torch.float32) or (weight is not None and w_dtype != wd):
            raise TypeError("w_dtype must be the weight's dtype, or that of x or float32")
        wd = w_dtype
    if grad_out.dtype != x.dtype or grad_out.shape != x.shape or not grad_out.is_contiguous():
        raise ValueError("grad_out must be contiguous with the dtype and shape of x")
    lead = tuple(x.shape[:-1])
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or tuple(t.shape) != lead or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with the leading shape of x")
    if any(t.device != x.device for t in (grad_out, mean, rstd)):
        raise ValueError("grad_out, mean and rstd must be on the device of x")
    dev = x.device
    N = x.numel() // D
    with _on(dev):
        d_x = torch.empty_like(x) if need_input else None
        d_weight = torch.empty(D, dtype=wd, device=dev) if need_weight else None
        d_bias = torch.empty(D, dtype=wd, device=dev) if need_bias else None
        ws, size = None, 0
        if need_weight or need_bias:
            size = max(_abi.flp_layer_norm_backward_workspace_bytes(N, D), 16)
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
        st = _abi.flp_layer_norm_backward(N, D, _X_DTYPES[x.dtype], grad_out.data_ptr(),
                                          x.data_ptr(), _X_DTYPES[wd], _ptr(weight),
                                          mean.data_ptr(), rstd.data_ptr(), _ptr(d_x),
                                          _ptr(d_weight), _ptr(d_bias), _ptr(ws), size,
                                          _stream(dev))
    _check("flp_layer_norm_backward", st)
    return d_x, d_weight, d_bias


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension, differentiable in
    x, weight and bias; weight and bias [D] in the dtype of x or float32."""
    if not _wants_grad(x, weight, bias):
        return layer_norm_forward(x, weight, bias, eps, return_stats=False)[0]
    _prepare_norm(x, weight, bias)
    dev = x.device
    with _on(dev):
        return _nodes().layer_norm(x, weight, bias, eps, _stream(dev))


# ---- gated projection of a feed-forward block ----------------------------------------------------

_ACTIVATIONS = {"silu": _abi.FLP_ACT_SILU, "gelu": _abi.FLP_ACT_GELU,
                "gelu_tanh": _abi.FLP_ACT_GELU_TANH}


def _prepare_gated(x, w_gate, w_up, activation):
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be 'silu', 'gelu' or 'gelu_tanh'")
    if x.dtype not in _X_DTYPES or w_gate.dtype != x.dtype or w_up.dtype != x.dtype:
        raise TypeError("x, w_gate and w_up must have the same dtype: bfloat16, float16 or float32")
    if not (x.is_cuda and w_gate.device == x.device and w_up.device == x.device):
        raise ValueError("x, w_gate and w_up must be on one GPU")
    for name, t in (("x", x), ("w_gate", w_gate), ("w_up", w_up)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if (w_gate.dim() != 2 or w_up.shape != w_gate.shape or x.dim() < 1
            or x.shape[-1] != w_gate.shape[1] or x.shape[-1] < 1):
        raise ValueError("w_gate and w_up must be [F, D] with D = x.shape[-1]")
    F, D = int(w_gate.shape[0]), int(w_gate.shape[1])
    return x.numel() // D, D, F, _ACTIVATIONS[activation]


def gated_linear_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                         activation: str = "silu", return_saved: bool = True
                         ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(out, saved) through flp_gated_linear_forward; saved (bytes, for the backward) or None."""
    N, D, F, act = _prepare_gated(x, w_gate, w_up, activation)
    dev, xd = x.device, _X_DTYPES[x.dtype]
    with _on(dev):
        out = torch.empty(x.shape[:-1] + (F,), dtype=x.dtype, device=dev)
        saved = None
        if return_saved:
            saved = torch.empty(max(_abi.flp_gated_linear_saved_bytes(N, F, xd), 16),
                                dtype=torch.uint8, device=dev)
        st = _abi.flp_gated_linear_forward(N, D, F, xd, x.data_ptr(), w_gate.data_ptr(),
                                           w_up.data_ptr(), act, out.data_ptr(), _ptr(saved),
                                           _stream(dev))
    _check("flp_gated_linear_forward", st)
    return out, saved


def gated_linear_backward(grad_out: torch.Tensor, saved: torch.Tensor, x: torch.Tensor,
                          w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu",
                          need_input: bool = True, need_gate: bool = True, need_up: bool = True):
    """(d_x, d_w_gate, d_w_up) through flp_gated_linear_backward; unrequested ones are None.  The
    activation is the one that saved was made with (which holds its values already)."""
    N, D, F, act = _prepare_gated(x, w_gate, w_up, activation)
    dev, xd = x.device, _X_DTYPES[x.dtype]
    if (grad_out.dtype != x.dtype or grad_out.shape != x.shape[:-1] + (F,)
            or not grad_out.is_contiguous() or grad_out.device != dev):
        raise ValueError("grad_out must be contiguous with the dtype, shape and device of the output")
    if (saved.dtype != torch.uint8 or not saved.is_contiguous() or saved.device != dev
            or saved.numel() < _abi.flp_gated_linear_saved_bytes(N, F, xd)):
        raise ValueError("saved must be what gated_linear_forward returned")
    with _on(dev):
        dx = torch.empty_like(x) if need_input else None
        dwg = torch.empty_like(w_gate) if need_gate else None
        dwu = torch.empty_like(w_up) if need_up else None
        size = _abi.flp_gated_linear_backward_workspace_bytes(N, D, F, xd, int(need_input),
                                                              int(need_gate or need_up))
        ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
        st = _abi.flp_gated_linear_backward(N, D, F, xd, grad_out.data_ptr(), saved.data_ptr(),
                                            x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), act,
                                            _ptr(dx), _ptr(dwg), _ptr(dwu), ws.data_ptr(),
                                            ws.numel(), _stream(dev))
    _check("flp_gated_linear_backward", st)
    return dx, dwg, dwu


def gated_linear(x, w_gate, w_up, activation="silu"):
    """act(x @ w_gate^T) * (x @ w_up^T), the first half of a gated feed-forward block,
    differentiable in x, w_gate and w_up.  x [.., D] with D a multiple of 32, w_gate and w_up
    [F, D] (they may be the halves of one [2 F, D] tensor); activation "silu", "gelu" (the exact
    one) or "gelu_tanh".  For the backward two numbers per element of the output are kept, 6 bytes (float32:
    8)."""
    if not _wants_grad(x, w_gate, w_up):
        return gated_linear_forward(x, w_gate, w_up, activation, return_saved=False)[0]
    act = _prepare_gated(x, w_gate, w_up, activation)[3]
    dev = x.device
    with _on(dev):
        return _nodes().gated_linear(x, w_gate, w_up, act, _stream(dev))


# ---- root mean square norms around a block ------------------------------------------------------

def _prepare_rms(x, y, weight, post_weight, gate, post_norm):
    """(rows, width, parameters' dtype, gate rows)."""
    if x.dtype not in _X_DTYPES:
        raise TypeError("x must be bfloat16, float16 or float32")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least one element")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous GPU tensor")
    D = int(x.shape[-1])
    if y is not None and (y.dtype != x.dtype or y.shape != x.shape or not y.is_contiguous()
                          or y.device != x.device):
        raise ValueError("y must be contiguous with the dtype, shape and device of x")
    wd = None
    for name, t in (("weight", weight), ("post_weight", post_weight), ("gate", gate)):
        if t is None:
            continue
        if t.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"{name} must have the dtype of x or float32")
        if wd is not None and t.dtype != wd:
            raise TypeError("weight, post_weight and gate must have the same dtype")
        if not t.is_contiguous() or t.device != x.device:
            raise ValueError(f"{name} must be contiguous and on the device of x")
        if name != "gate" and tuple(t.shape) != (D,):
            raise ValueError(f"{name} must be [D]")
        wd = t.dtype
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight goes with post_norm")
    N = x.numel() // D
    return N, D, x.dtype if wd is None else wd, _gate_rows(x, gate, N, D)


def _gate_rows(x, gate, N, D) -> int:
    """How many gate rows there are, each for as many consecutive rows of x."""
    if gate is None:
        return 0
    lead = list(gate.shape[:-1])
    if gate.dim() < 1 or gate.shape[-1] != D:
        raise ValueError("gate must be [.., D]")
    while lead and lead[-1] == 1:
        lead.pop()
    G = math.prod(lead)
    # leading dimensions of x, or so many groups of the rows of a 2-D one
    ok = tuple(lead) == tuple(x.shape[:len(lead)]) and len(lead) < x.dim()
    if not ok and not (x.dim() == 2 and len(lead) == 1 and G > 0 and N % G == 0):
        raise ValueError("gate must be [D], begin with the leading sizes of x ([B, D] or [B, 1, D] "
                         "for x [B, S, D]), or be [G, D] for x [N, D] with N a multiple of G")
    return G


def rms_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     return_stats: bool = True):
    """(out, rstd) of the root mean square norm over the last dimension through
    flp_rms_norm_forward; rstd is float32 of the leading shape, or None."""
    N, D, wd, _ = _prepare_rms(x, None, weight, None, None, False)
    dev = x.device
    with _on(dev):
        out = torch.empty_like(x)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev) if return_stats else None
        st = _abi.flp_rms_norm_forward(N, D, _X_DTYPES[x.dtype], x.data_ptr(), _X_DTYPES[wd],
                                       _ptr(weight), float(eps), out.data_ptr(), _ptr(rstd),
                                       _stream(dev))
    _check("flp_rms_norm_forward", st)
    return out, rstd


def rms_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, rstd: torch.Tensor,
                      weight: Optional[torch.Tensor] = None, need_input: bool = True,
                      need_weight: bool = True):
    """(d_x, d_weight) through flp_rms_norm_backward; unrequested ones are None, d_weight has the
    dtype of weight (of x without one)."""
    dx, _, dw, _, _ = residual_rms_norm_backward(None, grad_out, x, None, rstd, None, weight,
                                                 need_input=need_input, need_weight=need_weight)
    return dx, dw


def rms_norm(x, weight=None, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * weight over the last dimension, differentiable in x and weight;
    weight [D] in the dtype of x or float32."""
    if not _wants_grad(x, weight):
        return rms_norm_forward(x, weight, eps, return_stats=False)[0]
    _prepare_rms(x, None, weight, None, None, False)
    dev = x.device
    with _on(dev):
        return _nodes().rms_norm(x, None, weight, None, None, False, 1.0, eps, _stream(dev))[0]


def residual_rms_norm_forward(x: torch.Tensor, y: torch.Tensor,
                              weight: Optional[torch.Tensor] = None,
                              post_weight: Optional[torch.Tensor] = None,
                              gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                              eps: float = 1e-6, post_norm: Optional[bool] = None,
                              return_stats: bool = True):
    """(r, n, rstd, post_rstd) of residual_rms_norm through flp_residual_rms_norm_forward; the
    statistics are float32 of the leading shape, or None (post_rstd without post_norm)."""
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a tensor (rms_norm has none)")
    post = post_weight is not None if post_norm is None else bool(post_norm)
    N, D, wd, G = _prepare_rms(x, y, weight, post_weight, gate, post)
    dev = x.device
    with _on(dev):
        r, n = torch.empty_like(x), torch.empty_like(x)
        rstd = post_rstd = None
        if return_stats:
            rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
            post_rstd = torch.empty_like(rstd) if post else None
        st = _abi.flp_residual_rms_norm_forward(
            N, D, _X_DTYPES[x.dtype], x.data_ptr(), y.data_ptr(), _X_DTYPES[wd], _ptr(weight),
            int(post), _ptr(post_weight), G, _ptr(gate), float(scale), float(eps), r.data_ptr(),
            n.data_ptr(), _ptr(rstd), _ptr(post_rstd), _stream(dev))
    _check("flp_residual_rms_norm_forward", st)
    return r, n, rstd, post_rstd


def residual_rms_norm_backward(grad_r: Optional[torch.Tensor], grad_n: Optional[torch.Tensor],
                               x: torch.Tensor, y: Optional[torch.Tensor], rstd: torch.Tensor,
                               post_rstd: Optional[torch.Tensor] = None,
                               weight: Optional[torch.Tensor] = None,
                               post_weight: Optional[torch.Tensor] = None,
                               gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                               post_norm: Optional[bool] = None, need_input: bool = True,
                               need_block: bool = True, need_weight: bool = True,
                               need_post_weight: Optional[bool] = None,
                               need_gate: Optional[bool] = None):
    """(d_x, d_y, d_weight, d_post_weight, d_gate) through flp_residual_rms_norm_backward;
    unrequested ones are None.  grad_r or grad_n may be None (zero)."""
    post = post_weight is not None if post_norm is None else bool(post_norm)
    N, D, wd, G = _prepare_rms(x, y, weight, post_weight, gate, post)
    need_post_weight = post if need_post_weight is None else need_post_weight and post
    need_gate = gate is not None if need_gate is None else need_gate and gate is not None
    for name, t in (("grad_r", grad_r), ("grad_n", grad_n)):
        if t is not None and (t.dtype != x.dtype or t.shape != x.shape or not t.is_contiguous()
                              or t.device != x.device):
            raise ValueError(f"{name} must be contiguous with the dtype, shape and device of x")
    for name, t in (("rstd", rstd), ("post_rstd", post_rstd)):
        if t is None and (name == "rstd" or post):
            raise ValueError(f"{name} is needed")
        if t is not None and (t.dtype != torch.float32 or t.shape != x.shape[:-1]
                              or not t.is_contiguous() or t.device != x.device):
            raise ValueError(f"{name} must be contiguous float32 with the leading shape of x")
    dev = x.device
    with _on(dev):
        dx = torch.empty_like(x) if need_input else None
        dy = torch.empty_like(x) if need_block and y is not None else None
        dw = torch.empty(D, dtype=wd, device=dev) if need_weight else None
        dpw = torch.empty(D, dtype=wd, device=dev) if need_post_weight else None
        dg = torch.empty_like(gate) if need_gate else None
        ws, size = None, 0
        if need_weight or need_post_weight or need_gate:
            size = max(_abi.flp_residual_rms_norm_backward_workspace_bytes(N, D, G), 16)
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
        st = _abi.flp_residual_rms_norm_backward(
            N, D, _X_DTYPES[x.dtype], _ptr(grad_r), _ptr(grad_n), x.data_ptr(), _ptr(y),
            _X_DTYPES[wd], _ptr(weight), int(post), _ptr(post_weight), G, _ptr(gate), float(scale),
            rstd.data_ptr(), _ptr(post_rstd), _ptr(dx), _ptr(dy), _ptr(dw), _ptr(dpw), _ptr(dg),
            _ptr(ws), size, _stream(dev))
    _check("flp_residual_rms_norm_backward", st)
    return dx, dy, dw, dpw, dg


def residual_rms_norm(x, y, weight=None, post_weight=None, gate=None, scale=1.0, eps=1e-6,
                      post_norm=None):
    """(r, n): the residual stream x with the block's output y taken in, and its norm for the next
    block or the head, in one pass:

        p = rms_norm(y, post_weight) where post_norm (by default where post_weight is given), or y
        r = x + scale * gate * p,    n = rms_norm(r, weight)

    differentiable in x, y, weight, post_weight and gate.  weight and post_weight [D], gate [D],
    or with a row for each leading index of x ([B, D] or [B, 1, D] for x [B, S, D]; x's own shape
    for a gate per element), or [G, D] for x [N, D], each row for N / G rows in turn; all of them
    in the dtype of x or all in float32."""
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a tensor (rms_norm has none)")
    if not _wants_grad(x, y, weight, post_weight, gate):
        return residual_rms_norm_forward(x, y, weight, post_weight, gate, scale, eps, post_norm,
                                         return_stats=False)[:2]
    post = post_weight is not None if post_norm is None else bool(post_norm)
    _prepare_rms(x, y, weight, post_weight, gate, post)
    dev = x.device
    with _on(dev):
        return tuple(_nodes().rms_norm(x, y, weight, post_weight, gate, post, float(scale), eps,
                                       _stream(dev)))


# ---- AdamW --------------------------------------------------------------------------------------

class AdamWState(NamedTuple):
    """What adamw_step keeps of each parameter between steps, in lists as long as theirs.

    States in 32 bits are float32 tensors of the parameters' shapes: exp_avg holds the running
    mean m of the gradients, exp_avg_sq that of their squares, v.  States in 8 bits are
    float8_e4m3fn, exp_avg_sq holding the root of v, with float32 scales for 256 consecutive
    elements each: element i of tensor k stands for
    exp_avg[k].view(-1)[i] * exp_avg_scale[k][i // 256].  Steps with beta1 > 0.9 or beta2 > 0.95
    round them up or down by a threshold of the step's number and the element's index, so that they
    are right on average over the steps.  master: float32 copies of the
    parameters (None for a parameter without one), or None."""
    exp_avg: List[torch.Tensor]
    exp_avg_sq: List[torch.Tensor]
    exp_avg_scale: Optional[List[torch.Tensor]] = None
    exp_avg_sq_scale: Optional[List[torch.Tensor]] = None
    master: Optional[List[Optional[torch.Tensor]]] = None


def adamw_state(params: Sequence[torch.Tensor], bits: int = 32, master: bool = False
                ) -> AdamWState:
    """The state before the first step: zeros, in 32 or 8 bits per element; with master, a float32
    copy of every 16-bit parameter."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    params = list(params)
    copies = None
    if master:
        copies = [None if p.dtype == torch.float32 else p.detach().float().contiguous()
                  for p in params]

    def zeros(p, n, dtype):
        return torch.zeros(n, dtype=dtype, device=p.device)

    if bits == 32:
        m, v = ([zeros(p, p.shape, torch.float32) for p in params] for _ in range(2))
        return AdamWState(m, v, None, None, copies)
    m, v = ([zeros(p, p.shape, torch.uint8).view(torch.float8_e4m3fn) for p in params]
            for _ in range(2))
    ms, vs = ([zeros(p, -(-p.numel() // 256), torch.float32) for p in params] for _ in range(2))
    return AdamWState(m, v, ms, vs, copies)


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[Optional[torch.Tensor]],
               state: AdamWState, step: Union[int, torch.Tensor],
               lr: Union[float, torch.Tensor], betas: Tuple[float, float] = (0.9, 0.999),
               eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.01,
               grad_scale: Optional[torch.Tensor] = None) -> None:
    """One AdamW step over all params at once, in place, through flp_adamw_step:

        m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,   g = grad * grad_scale
        p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)

    params: bfloat16, float16 or float32, in any mix; grads: each of its parameter's dtype or
    float32, None leaves its parameter alone.  step: the number t of this step, from 1.
    weight_decay: one number, or one for each parameter.  step (int64), lr and grad_scale (float32)
    may be one-element tensors on the device, which a captured call reads at every replay."""
    if not isinstance(params, (list, tuple)):
        params = list(params)
    if not params:
        return
    if not isinstance(weight_decay, (list, tuple)):
        weight_decay = float(weight_decay)
    at_step, at_lr = (x if isinstance(x, torch.Tensor) else None for x in (step, lr))
    dev = params[0].device
    if not params[0].is_cuda:
        raise ValueError("parameters must be contiguous GPU tensors on one device")
    with _on(dev):
        _nodes().adamw_step(params, grads, state.exp_avg, state.exp_avg_sq, state.exp_avg_scale,
                            state.exp_avg_sq_scale, state.master, weight_decay,
                            1 if at_step is not None else int(step), at_step,
                            0.0 if at_lr is not None else float(lr), at_lr, float(betas[0]),
                            float(betas[1]), float(eps), grad_scale, _stream(dev))
