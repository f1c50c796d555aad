"""ctypes binding of the operators around the loss (include/grpo.h): the norm in
front of the LM head, the optimizer's step, the gradients' norm and the sampling of
tokens.

Argument marshalling only, as in _lib.  Every call checks that its tensors share
one GPU and runs on that GPU's current torch stream, whichever device is current.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from ._lib import (AdamWOpts, AdamWTensor, GradTensor, SampleOpts, _arg, _check, _dev, _dt, _matrix,
                   _ptr, lib)

# grpo_norm_kind
NORM_LAYER, NORM_RMS = 0, 1


_HERE = contextlib.nullcontext()


def _on(*ts, strided=()):
    """The tensors' one GPU made current, and its current stream: (context, stream).
    All of them are contiguous, except those of `strided`."""
    at = ts[0].get_device()
    for t in ts:
        if at < 0 or t.get_device() != at or not t.is_contiguous():
            _refuse(ts + strided, ts)
    for t in strided:
        if t.get_device() != at:
            _refuse(ts + strided, ts)
    ctx = _HERE if at == torch._C._cuda_getDevice() else torch.cuda.device(at)
    return ctx, torch._C._cuda_getCurrentRawStream(at)


def _refuse(ts, contiguous):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be on the GPU")
    _dev(*contiguous)
    raise ValueError("tensors on %s: one call runs on one GPU"
                     % " and ".join(sorted({str(t.device) for t in ts})))


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


@functools.lru_cache(maxsize=256)
def _norm_bytes(rows, cols, dt):
    need = int(lib().grpo_norm_workspace_bytes(rows, cols, dt))
    if need == 0:
        _check("grpo_norm_workspace_bytes", -1)
    return need


def grpo_norm_bwd(dY, X, weight, mean, rstd, kind: int = NORM_RMS, bias: bool = False, dX=None,
                  dweight=None, dbias=None, workspace=None):
    """(dX, dweight, dbias): dX in X's type; dweight and dbias [cols] float32,
    accumulated into when given.  dbias is formed
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
    # into the caller's accumulators, or new tensors that the call fills
    accumulate = dweight is not None or dbias is not None
    new = torch.zeros if accumulate else torch.empty
    if dweight is not None:
        _arg(dweight, "dweight", dtype=torch.float32, numel=cols)
    else:
        dweight = new(cols, dtype=torch.float32, device=dev)
    if dbias is not None:
        _arg(dbias, "dbias", dtype=torch.float32, numel=cols)
    elif bias:
        dbias = new(cols, dtype=torch.float32, device=dev)
    need = _norm_bytes(rows, cols, dt)
    if workspace is not None:
        workspace = _workspace(need, dev, workspace)
    ctx, stream = _on(*(t for t in (dY, X, weight, mean, rstd, dX, dweight, dbias, workspace)
                        if t is not None))
    with ctx:
        ws = _workspace(need, dev, workspace)
        _check("grpo_norm_bwd", lib().grpo_norm_bwd(
            _ptr(dY), _ptr(X), _ptr(weight), _ptr(mean), _ptr(rstd), rows, cols, dt, kind,
            int(accumulate), _ptr(dX), _ptr(dweight), _ptr(dbias), _ptr(ws), ws.numel(), stream))
    return dX, dweight, dbias


# ---------------------------------------------------------------- AdamW
QUANT_BLOCK = 256   # elements per scale of an 8-bit moment


class Moment8:
    """A moment in 8 bits: codes (int8 for the first moment, uint8 for the second, in
    the parameter's shape) and one float32 scale per 256 elements."""

    def __init__(self, codes, scales):
        if codes.dtype not in (torch.int8, torch.uint8):
            raise TypeError(f"codes must be int8 or uint8, got {codes.dtype}")
        _arg(scales, "scales", dtype=torch.float32, numel=-(-codes.numel() // QUANT_BLOCK))
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return self.codes.shape


def dequantize_moment(q: Moment8, out=None):
    """grpo_moment_values: the float32 values of q."""
    out = torch.empty(q.codes.shape, dtype=torch.float32, device=q.codes.device) if out is None \
        else _arg(out, "out", dtype=torch.float32, numel=q.codes.numel())
    ctx, stream = _on(q.codes, q.scales, out)
    with ctx:
        _check("grpo_moment_values", lib().grpo_moment_values(
            _ptr(q.codes), _ptr(q.scales), q.codes.numel(), int(q.codes.dtype == torch.uint8),
            _ptr(out), stream))
    return out


def adamw_moments(params, bits: int = 32):
    """The moments before the first step: (exp_avg, exp_avg_sq), lists of float32 zeros
    (bits 32) or of Moment8 zeros (bits 8) for each parameter."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")

    def zeros(p, dtype):
        if bits == 32:
            return torch.zeros(p.shape, dtype=torch.float32, device=p.device)
        return Moment8(torch.zeros(p.shape, dtype=dtype, device=p.device),
                       torch.zeros(-(-p.numel() // QUANT_BLOCK), dtype=torch.float32, device=p.device))
    return [zeros(p, torch.int8) for p in params], [zeros(p, torch.uint8) for p in params]


class AdamWPlan:
    """What grpo_adamw needs of its tensors, made once by adamw_plan.  It keeps the
    tensors' memory alive and holds their addresses: a parameter or gradient that is
    replaced (p.data = ..., zero_grad(set_to_none=True), the default) or whose storage is
    freed in place (resize_(0)) needs a new plan.  The step goes by the old addresses
    without noticing, since it looks at no tensor; holds() tells."""

    def __init__(self, tensors, params, image, table, lists):
        self.tensors, self.image, self.table = tensors, image, table
        self.lists = lists      # params, grads and, with masters, those: first in each of tensors
        self.places = [[t.data_ptr() for t in row] for row in tensors]
        self.versioned = [p for p in params if not p.is_inference()]
        self.device = table.device
        self.stream = torch._C._cuda_getCurrentRawStream(table.get_device())

    def holds(self, params, grads, master=None) -> bool:
        """Whether these are still the tensors that the plan steps, at the addresses that it
        holds, and its moments have not moved: adamw_plan's params, grads and master (None
        where it had none; a gradient of None is not held).  Host work of some 0.8 us a
        tensor, so it is the caller's to ask where tensors may have been replaced."""
        lists = [list(x) for x in (params, grads) + (() if master is None else (master,))]
        if len(lists) != self.lists or any(len(x) != len(self.places) for x in lists):
            return False
        for now, row, at in zip(zip(*lists), self.tensors, self.places):
            if any(t is None or t.data_ptr() != a or t.numel() != row[0].numel() for t, a in zip(now, at)):
                return False
            if any(t.data_ptr() != a for t, a in zip(row, at)):
                return False
        return True


def adamw_plan(params, grads, exp_avg, exp_avg_sq, master=None) -> AdamWPlan:
    """The plan of an AdamW step over lists of tensors of one GPU: params (all float32 or
    all bfloat16), grads (all float32 or all bfloat16, in the parameters' sizes), the
    moments (float32 tensors, or Moment8) and optionally float32 masters of bfloat16
    parameters.  Tensors that share memory are refused."""
    params, grads, exp_avg, exp_avg_sq = (list(x) for x in (params, grads, exp_avg, exp_avg_sq))
    master = None if master is None else list(master)
    if not params:
        raise ValueError("params is empty")
    for name, x in (("grads", grads), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq),
                    ("master", master)):
        if x is not None and len(x) != len(params):
            raise ValueError(f"{name} has {len(x)} tensors, params has {len(params)}")
    eight = isinstance(exp_avg[0], Moment8)
    _arg(params[0], "params[0]")
    _arg(grads[0], "grads[0]")
    pt, gt = _dt(params[0]), _dt(grads[0])
    rows, keep = (AdamWTensor * len(params))(), []
    for i, (p, g, m, v) in enumerate(zip(params, grads, exp_avg, exp_avg_sq)):
        _arg(p, f"params[{i}]", dtype=params[0].dtype)
        n = p.numel()
        parts = {"param": p, "grad": _arg(g, f"grads[{i}]", dtype=grads[0].dtype, numel=n)}
        if master is not None:
            parts["master"] = _arg(master[i], f"master[{i}]", dtype=torch.float32, numel=n)
        for name, x, dtype in (("exp_avg", m, torch.int8), ("exp_avg_sq", v, torch.uint8)):
            if isinstance(x, Moment8) != eight:
                raise TypeError("the moments must be all float32 tensors or all Moment8")
            if eight:
                parts[name] = _arg(x.codes, f"{name}[{i}].codes", dtype=dtype, numel=n)
                parts[name + "_scales"] = x.scales
            else:
                parts[name] = _arg(x, f"{name}[{i}]", dtype=torch.float32, numel=n)
        keep.append(tuple(t.detach() for t in parts.values()))
        rows[i].n = n
        for name, t in parts.items():
            setattr(rows[i], name, t.data_ptr())
    ctx, _ = _on(*(t for row in keep for t in row))
    size = int(lib().grpo_adamw_plan_bytes(len(params)))
    image = (ctypes.c_uint8 * size)()
    _check("grpo_adamw_plan", lib().grpo_adamw_plan(rows, len(params), pt, gt, 8 if eight else 32,
                                                    image, size))
    with ctx:
        # a copy from pageable memory: it has arrived when the call returns
        table = torch.frombuffer(image, dtype=torch.uint8).to(params[0].device)
        return AdamWPlan(keep, params, image, table, 2 if master is None else 3)


def _scalar(x, name, dtype):
    """A device scalar's tensor, or None for a host number."""
    return _arg(x, name, dtype=dtype, numel=1) if isinstance(x, torch.Tensor) else None


def grpo_adamw(plan: AdamWPlan, step, lr=1e-6, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 0.01, grad_scale=None):
    """One AdamW step of the plan's tensors, in place, in one launch.  step counts from 1;
    a tensor for step (int64, one element) or lr (float32, one element) is read when the
    kernel runs, so a captured step follows it.  grad_scale: a float32 tensor of one
    element that multiplies every gradient (a clipping factor), or None.  Gradients are
    left as they are.  A captured graph needs the plan to live as long as it does."""
    step_dev, lr_dev = _scalar(step, "step", torch.int64), _scalar(lr, "lr", torch.float32)
    if grad_scale is not None:
        _arg(grad_scale, "grad_scale", dtype=torch.float32, numel=1)
    ctx, stream = _on(*(t for t in (plan.table, step_dev, lr_dev, grad_scale) if t is not None))
    opts = AdamWOpts(0.0 if lr_dev is not None else lr, betas[0], betas[1], eps, weight_decay,
                     0 if step_dev is not None else step, _ptr(step_dev), _ptr(lr_dev),
                     _ptr(grad_scale))
    with ctx:
        if stream != plan.stream:   # the allocator must not hand the table on too early
            plan.table.record_stream(torch.cuda.current_stream(plan.device))
        _check("grpo_adamw", lib().grpo_adamw(plan.image, _ptr(plan.table), ctypes.byref(opts),
                                              stream))
    # autograd has to see that the parameters changed
    torch.autograd.graph.increment_version(plan.versioned)


# ---------------------------------------------------------------- gradient norm
# grpo_grad_norm_kind
GRAD_NORM_L2, GRAD_NORM_MAX = 0, 1


class GradPlan:
    """What grpo_grad_norm and grpo_grad_clip need of the gradients, made once by grad_plan.
    Like an AdamWPlan it keeps the tensors' memory alive and holds their addresses: gradients
    that are replaced need a new plan, and holds() tells."""

    def __init__(self, tensors, grads, image, table):
        self.tensors, self.image, self.table = tensors, image, table
        self.places = [t.data_ptr() for t in tensors]
        self.versioned = [g for g in grads if not g.is_inference()]
        self.device = table.device
        self.stream = torch._C._cuda_getCurrentRawStream(table.get_device())

    def holds(self, grads) -> bool:
        """Whether these are still the gradients of the plan, at the addresses that it holds
        (a gradient of None is not held)."""
        grads = list(grads)
        return len(grads) == len(self.tensors) and all(
            g is not None and g.data_ptr() == a and t.data_ptr() == a and g.numel() == t.numel()
            and g.dtype == t.dtype for g, t, a in zip(grads, self.tensors, self.places))


def grad_plan(grads) -> GradPlan:
    """The plan of the norm of a list of gradients of one GPU, float32 and bfloat16 in any
    mixture.  Tensors that share memory are refused."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads is empty")
    rows = (GradTensor * len(grads))()
    for i, g in enumerate(grads):
        _arg(g, f"grads[{i}]")
        rows[i] = GradTensor(g.data_ptr(), g.numel(), _dt(g), 0)
    ctx, _ = _on(*grads)
    size = int(lib().grpo_grad_plan_bytes(len(grads)))
    image = (ctypes.c_uint8 * size)()
    _check("grpo_grad_plan", lib().grpo_grad_plan(rows, len(grads), image, size))
    with ctx:
        # a copy from pageable memory: it has arrived when the call returns
        table = torch.frombuffer(image, dtype=torch.uint8).to(grads[0].device)
        return GradPlan([g.detach() for g in grads], grads, image, table)


@functools.lru_cache(maxsize=1)
def _grad_bytes():
    return int(lib().grpo_grad_norm_workspace_bytes())


def grpo_grad_norm(plan: GradPlan, max_norm: float = 0.0, kind: int = GRAD_NORM_L2, workspace=None):
    """(norm, scale), float32 tensors of one element: the norm of all gradients of the plan
    as one vector (of kind GRAD_NORM_L2, or GRAD_NORM_MAX, the largest magnitude), and
    min(1, max_norm / (norm + 1e-6)), which grpo_adamw takes as its grad_scale and
    grpo_grad_clip applies in place (max_norm 0: 1).  A captured graph needs the plan to live
    as long as it does."""
    need = _grad_bytes()
    ts = (plan.table,) if workspace is None else (plan.table, _workspace(need, plan.device, workspace))
    ctx, stream = _on(*ts)
    with ctx:
        _keep(plan, stream)
        norm = torch.empty(1, dtype=torch.float32, device=plan.device)
        scale = torch.empty(1, dtype=torch.float32, device=plan.device)
        ws = _workspace(need, plan.device, workspace)
        _check("grpo_grad_norm", lib().grpo_grad_norm(
            plan.image, plan.table.data_ptr(), kind, max_norm, norm.data_ptr(), scale.data_ptr(),
            ws.data_ptr(), ws.numel(), stream))
    return norm, scale


def grpo_grad_clip(plan: GradPlan, scale):
    """Every gradient of the plan times scale (a float32 tensor of one element), in place,
    rounded to its type.  For an optimizer that takes no scale of its own."""
    _arg(scale, "scale", dtype=torch.float32, numel=1)
    ctx, stream = _on(plan.table, scale)
    with ctx:
        _keep(plan, stream)
        _check("grpo_grad_clip", lib().grpo_grad_clip(plan.image, plan.table.data_ptr(),
                                                      scale.data_ptr(), stream))
    # autograd has to see that the gradients changed
    torch.autograd.graph.increment_version(plan.versioned)


def _keep(plan, stream):
    if stream != plan.stream:   # the allocator must not hand the table on too early
        plan.table.record_stream(torch.cuda.current_stream(plan.device))


# ---------------------------------------------------------------- sampling
@functools.lru_cache(maxsize=256)
def _sample_bytes(B, V):
    need = int(lib().grpo_sample_workspace_bytes(B, V))
    if need == 0:
        _check("grpo_sample_workspace_bytes", -3)
    return need


def grpo_sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None,
                workspace=None):
    """(token, lp): one token (int32 [B]) for each row of logits [B, V] (float32 or
    bfloat16; rows may lie any distance apart), from u [B] float32 in [0, 1), and its
    log-probability (float32 [B]) under softmax(logits / temperature) of the whole row.
    temperature, top_k, top_p and min_p are numbers, or tensors [B] with one for each row
    (float32; int32 for top_k).  0 is off for each, and so is top_p 1: temperature 0 samples
    at temperature 1 and top_p 0 keeps the whole row; top_k 1 takes the largest logit.
    out: (token, lp) to write into.  See grpo_sample in include/grpo.h for the order of the
    filters and rows without a distribution."""
    B, V = _matrix(logits, "logits")
    dt = _dt(logits)
    if V > 1 and logits.stride(1) != 1 or B > 1 and logits.stride(0) < V:
        raise ValueError("the logits of a row must be adjacent and rows must not overlap")
    stride = max(V, logits.stride(0))
    _arg(u, "u", dtype=torch.float32, numel=B)
    # numbers, and device arrays in their places
    numbers, arrays, rows = [], [], []
    for name, x in (("temperature", temperature), ("top_p", top_p), ("min_p", min_p), ("top_k", top_k)):
        if isinstance(x, torch.Tensor):
            rows.append(_arg(x, name, dtype=torch.int32 if name == "top_k" else torch.float32, numel=B))
            numbers.append(0)
            arrays.append(x.data_ptr())
        else:
            # ctypes drops what does not fit 32 bits
            numbers.append(min(max(x, -1), 2**31 - 1) if name == "top_k" else x)
            arrays.append(None)
    opts = SampleOpts(*numbers, 0, *arrays)
    token, lp = (None, None) if out is None else out
    dev = logits.device
    token = torch.empty(B, dtype=torch.int32, device=dev) if token is None else \
        _arg(token, "token", dtype=torch.int32, numel=B)
    lp = torch.empty(B, dtype=torch.float32, device=dev) if lp is None else \
        _arg(lp, "lp", dtype=torch.float32, numel=B)
    need = _sample_bytes(B, V)
    if workspace is not None:
        rows.append(_workspace(need, dev, workspace))
    ctx, stream = _on(u, token, lp, *rows, strided=(logits,))
    with ctx:
        ws = _workspace(need, dev, workspace)
        _check("grpo_sample", lib().grpo_sample(
            _ptr(logits), dt, B, V, stride, _ptr(u), ctypes.byref(opts), _ptr(token), _ptr(lp),
            _ptr(ws), ws.numel(), stream))
    return token, lp
