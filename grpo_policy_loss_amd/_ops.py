"""ctypes binding of the operators around the loss (include/grpo.h): the norm in
front of the LM head.

Argument marshalling only, as in _lib.  Every call checks that its tensors share
one GPU and runs on that GPU's current torch stream, whichever device is current.
"""
from __future__ import annotations

import contextlib

import torch

from ._lib import _arg, _check, _dev, _dt, _matrix, _ptr, lib

# grpo_norm_kind
NORM_LAYER, NORM_RMS = 0, 1


def _on(*ts):
    """The tensors' one GPU made current, and its current stream: (context, stream)."""
    _dev(*ts)
    dev = ts[0].device
    for t in ts:
        if t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}: one call runs on one GPU")
    ctx = contextlib.nullcontext() if dev.index == torch.cuda.current_device() else \
        torch.cuda.device(dev)
    return ctx, torch.cuda.current_stream(dev).cuda_stream


def _workspace(need, device, workspace):
    """The caller's workspace (uint8, at least `need` bytes) or a new one."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _arg(workspace, "workspace", dtype=torch.uint8)
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; this call needs at least {need}")
    return workspace


# ---------------------------------------------------------------- norm
def grpo_norm_fwd(X, weight, bias=None, eps: float = 1e-5, kind: int = NORM_RMS, out=None):
    """(Y, mean, rstd) of the rows of X [rows, cols] (float32 or bfloat16; weight and
    bias [cols] of the same type).  mean and rstd [rows] are float32; mean is None for
    NORM_RMS."""
    rows, cols = _matrix(X, "X")
    dt = _dt(X)
    _arg(weight, "weight", dtype=X.dtype, numel=cols)
    if bias is not None:
        _arg(bias, "bias", dtype=X.dtype, numel=cols)
    Y = torch.empty_like(X) if out is None else _arg(out, "out", dtype=X.dtype, shape=(rows, cols))
    ctx, stream = _on(*(t for t in (X, weight, bias, Y) if t is not None))
    rstd = torch.empty(rows, dtype=torch.float32, device=X.device)
    mean = torch.empty_like(rstd) if kind == NORM_LAYER else None
    with ctx:
        _check("grpo_norm_fwd", lib().grpo_norm_fwd(
            _ptr(X), _ptr(weight), _ptr(bias), rows, cols, dt, kind, eps, _ptr(Y), _ptr(mean),
            _ptr(rstd), stream))
    return Y, mean, rstd


def grpo_norm_bwd(dY, X, weight, mean, rstd, kind: int = NORM_RMS, bias: bool = False, dX=None,
                  dweight=None, dbias=None, workspace=None):
    """(dX, dweight, dbias): dX in X's type; dweight and dbias [cols] float32,
    accumulated into when given (zeros are allocated otherwise).  dbias is formed
    if `bias` is true or dbias is given, and None otherwise.  mean and rstd are
    grpo_norm_fwd's (mean None for NORM_RMS)."""
    rows, cols = _matrix(X, "X")
    dt = _dt(X)
    _arg(dY, "dY", dtype=X.dtype, shape=(rows, cols))
    _arg(weight, "weight", dtype=X.dtype, numel=cols)
    _arg(rstd, "rstd", dtype=torch.float32, numel=rows)
    if kind == NORM_LAYER:
        _arg(mean, "mean", dtype=torch.float32, numel=rows)
    else:
        mean = None
    dev = X.device
    dX = torch.empty_like(X) if dX is None else _arg(dX, "dX", dtype=X.dtype, shape=(rows, cols))
    dweight = torch.zeros(cols, dtype=torch.float32, device=dev) if dweight is None else \
        _arg(dweight, "dweight", dtype=torch.float32, numel=cols)
    if dbias is not None:
        _arg(dbias, "dbias", dtype=torch.float32, numel=cols)
    elif bias:
        dbias = torch.zeros(cols, dtype=torch.float32, device=dev)
    need = int(lib().grpo_norm_workspace_bytes(rows, cols, dt))
    if need == 0:
        _check("grpo_norm_workspace_bytes", -1)
    if workspace is not None:
        workspace = _workspace(need, dev, workspace)
    ctx, stream = _on(*(t for t in (dY, X, weight, mean, rstd, dX, dweight, dbias, workspace)
                        if t is not None))
    with ctx:
        ws = _workspace(need, dev, workspace)
        _check("grpo_norm_bwd", lib().grpo_norm_bwd(
            _ptr(dY), _ptr(X), _ptr(weight), _ptr(mean), _ptr(rstd), rows, cols, dt, kind,
            _ptr(dX), _ptr(dweight), _ptr(dbias), _ptr(ws), ws.numel(), stream))
    return dX, dweight, dbias
