"""A dense layer with bias, activation and residual in its epilogue, and its gradients.

    y = act(x W + bias) + residual

for the layers below the head and, with fp32 out, the head's own logits for a sampler.  x, W and
bias are bf16; W is [K, N] (weight_layout 'hv') or [N, K] ('vh', nn.Linear), as the head's.
Argument marshalling only; the library's kernels do the work.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B
from .losses import _addr, _current_device, _on, _raw_stream, _workspace, _written

_ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_OUT = {torch.bfloat16: 1, torch.float32: 0}
_LAYOUTS = {"hv": 0, "vh": 1, 0: 0, 1: 1}
_HEADER = 256  # bytes of workspace of the forward, whatever the shape


def linear_params(M, N, K, activation=None, weight_layout="hv", out_dtype=torch.bfloat16,
                  validate=False):
    """FlceLinearParams of a flce_linear call."""
    if out_dtype not in _OUT:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be one of relu/gelu/gelu_tanh/silu or None, got "
                         f"{activation!r}")
    return B.FlceLinearParams(M, N, K, B.layout_code(weight_layout), _ACTIVATIONS[activation],
                              _OUT[out_dtype], bool(validate))


def linear_workspace_size(params: "B.FlceLinearParams", backward: bool = False) -> int:
    """Bytes of workspace a flce_linear (flce_linear_backward) call with these parameters needs."""
    lib = B._lib or B.load_library()
    size = lib.flce_linear_workspace_size(ctypes.byref(params), int(backward))
    if size == 0:
        B._check(lib.flce_linear_check_params(ctypes.byref(params)))
    return size


def _shapes(x, weight, weight_layout):
    """(M, N, K, device) of x [..., K] and the weight, checked."""
    for t, name in ((x, "x"), (weight, "weight")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if x.dim() < 1 or weight.dim() != 2:
        raise ValueError(f"x must be [..., K] and weight 2-D, got {tuple(x.shape)} and "
                         f"{tuple(weight.shape)}")
    dev = B._on_current_device(x)
    if weight.device != dev:
        raise ValueError(f"weight is on {weight.device}, the other tensors on {dev}")
    N, K = weight.shape if B.layout_code(weight_layout) == B.WEIGHT_VH else weight.shape[::-1]
    if x.shape[-1] != K:
        raise ValueError(f"x has rows of {x.shape[-1]}, the weight takes {K}")
    M = 1
    for n in x.shape[:-1]:
        M *= n
    return M, N, K, dev


def _apart(outs, inputs):
    """Refuses outputs (name, tensor or None) that share memory with one another or with an input, which
    would be read after it is overwritten."""
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name)
             for name, t in (*outs, *inputs) if t is not None and t.numel()]
    for i, (a, b, name) in enumerate(spans[:sum(t is not None and t.numel() > 0 for _, t in outs)]):
        for c, d, other in spans[i + 1:]:
            if a < d and c < b:
                raise ValueError(f"{name} shares memory with {other}")


def _aligned(t):
    """t, or a copy of it from a 16-byte boundary on: a row slice of odd width, as the gradient behind a
    torch.cat over tokens is, begins anywhere."""
    return t if t is None or t.data_ptr() & 15 == 0 else t.clone()


def flce_linear(x, weight, bias=None, activation=None, residual=None, weight_layout="hv",
                out_dtype=torch.bfloat16, need_preact=False, validate=False, workspace=None,
                stream=None, out=None):
    """y [..., N] = act(x W + bias) + residual, in bf16 or (out_dtype) fp32.

    x [..., K] and weight bf16, K a multiple of 8, and N too for a [K, N] weight; bias bf16 [N];
    activation: None, 'relu', 'gelu', 'gelu_tanh' or 'silu'; residual of y's shape and type (out
    may be the residual itself).  Sums are fp32, rounded once.  With need_preact returns (y, z): z =
    x W + bias in bf16, as the backward takes it.  x and weight begin at a 16-byte boundary; a
    residual or out that does not is copied.
    """
    if stream is not None:
        return _on(stream, flce_linear, x, weight, bias, activation, residual, weight_layout,
                   out_dtype, need_preact, validate, workspace, out=out)
    lib = B._lib or B.load_library()
    # one pass over what is right, as a small layer's time is these checks; _refuse says what is
    # wrong
    try:
        bf16, dev = torch.bfloat16, x.get_device()
        layout, act, out_code = _LAYOUTS[weight_layout], _ACTIVATIONS[activation], _OUT[out_dtype]
        N, K = weight.shape if layout else weight.shape[::-1]
        shape = (*x.shape[:-1], N)
        if not (dev >= 0 and x.dtype is bf16 and weight.dtype is bf16 and x.shape[-1] == K
                and weight.get_device() == dev == _current_device() and x.is_contiguous() and weight.is_contiguous()):
            raise ValueError
        for t, dtype, size in ((bias, bf16, (N,)), (residual, out_dtype, shape), (out, out_dtype, shape)):
            if t is not None and not (t.dtype is dtype and t.shape == size
                                      and t.get_device() == dev and t.is_contiguous()):
                raise ValueError
    except (AttributeError, IndexError, KeyError, TypeError, ValueError):
        _refuse(x, weight, bias, activation, residual, weight_layout, out_dtype, out)
        raise
    p = B.FlceLinearParams(x.numel() // K if K else 0, N, K, layout, act, out_code, bool(validate))
    given = out
    if given is None:
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
    else:
        own = residual is not None and out.data_ptr() == residual.data_ptr()
        _apart([("out", out)], [("x", x), ("weight", weight), ("bias", bias),
                                ("residual", None if own else residual)])
        if out.data_ptr() & 15:
            out = torch.empty(shape, dtype=out_dtype, device=x.device)
    residual = _aligned(residual)
    z = torch.empty(shape, dtype=bf16, device=x.device) if need_preact else None
    ws = torch.empty(_HEADER, dtype=torch.uint8, device=x.device) if workspace is None \
        else _workspace(linear_workspace_size(p), dev, workspace)
    code = lib.flce_linear(ctypes.byref(p), x.data_ptr(), weight.data_ptr(), _addr(bias),
                           _addr(residual), out.data_ptr(), _addr(z), ws.data_ptr(), ws.numel(),
                           _raw_stream(dev))
    if code:
        B._check(code)
    if given is not None:
        if out is not given:
            given.detach().copy_(out)
            out = given
        _written(out)
    return (out, z) if need_preact else out


def _refuse(x, weight, bias, activation, residual, weight_layout, out_dtype, out):
    """Says what is wrong with flce_linear's arguments."""
    M, N, K, dev = _shapes(x, weight, weight_layout)
    linear_params(M, N, K, activation, weight_layout, out_dtype)
    shape = (*x.shape[:-1], N)
    if bias is not None:
        B._need(bias, "bias", torch.bfloat16, (N,), dev)
    for t, name in ((residual, "residual"), (out, "out")):
        if t is not None:
            B._need(t, name, out_dtype, shape, dev)


def flce_linear_backward(dout, x, weight, preact=None, activation=None, weight_layout="hv",
                         need_dx=True, need_dweight=True, need_dbias=True, validate=False,
                         workspace=None, stream=None, out=None):
    """(dx, dweight, dbias) of flce_linear, bf16, shaped like x, weight and [N]; None where not
    wanted.  dout: of y's shape and type (bf16 or fp32); it is the residual's gradient as it is.
    preact: z of the forward, where there is an activation; it and dout are copied where they do
    not begin at a 16-byte boundary.  dz = dout act'(z), of the bf16 z, is rounded to bf16 for the
    products; dbias sums it unrounded.  out: (dx, dweight, dbias) to write into."""
    if stream is not None:
        return _on(stream, flce_linear_backward, dout, x, weight, preact, activation,
                   weight_layout, need_dx, need_dweight, need_dbias, validate, workspace, out=out)
    lib = B._lib or B.load_library()
    try:  # as in flce_linear
        bf16, dev = torch.bfloat16, x.get_device()
        layout, act, code = _LAYOUTS[weight_layout], _ACTIVATIONS[activation], _OUT[dout.dtype]
        N, K = weight.shape if layout else weight.shape[::-1]
        shape = (*x.shape[:-1], N)
        if not (dev >= 0 and x.dtype is bf16 and weight.dtype is bf16 and x.shape[-1] == K
                and weight.get_device() == dev == _current_device() and x.is_contiguous()
                and weight.is_contiguous()):
            raise ValueError
        for t in (dout, preact) if act else (dout,):
            if not (t.shape == shape and t.get_device() == dev and t.is_contiguous()):
                raise ValueError
        if act and preact.dtype is not bf16:
            raise ValueError
    except (AttributeError, IndexError, KeyError, TypeError, ValueError):
        _refuse_backward(dout, x, weight, preact, activation, weight_layout)
        raise
    p = B.FlceLinearParams(x.numel() // K if K else 0, N, K, layout, act, code, bool(validate))
    size = linear_workspace_size(p, True)
    wanted = (("dx", need_dx, x.shape), ("dweight", need_dweight, weight.shape),
              ("dbias", need_dbias, (N,)))
    given = out is not None
    if not given:
        out = [torch.empty(s, dtype=bf16, device=dev) if need else None for _, need, s in wanted]
    else:
        if len(out) != 3:
            raise ValueError("out must hold dx, dweight and dbias")
        out = [t if need else None for t, (_, need, _) in zip(out, wanted)]
        for t, (name, need, s) in zip(out, wanted):
            if need:
                B._need(t, name, bf16, s, x.device)
        _apart([(name, t) for (name, _, _), t in zip(wanted, out)],
               [("dout", dout), ("x", x), ("weight", weight), ("preact", preact if act else None)])
    dx, dw, db = out
    dout, preact = _aligned(dout), _aligned(preact) if act else None
    ws = _workspace(size, dev, workspace)
    code = lib.flce_linear_backward(
        ctypes.byref(p), dout.data_ptr(), x.data_ptr(), weight.data_ptr(),
        preact.data_ptr() if act else None, _addr(dx), _addr(dw), _addr(db),
        ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if code:
        B._check(code)
    if given:
        _written([t for t in (dx, dw, db) if t is not None])
    return dx, dw, db


def _refuse_backward(dout, x, weight, preact, activation, weight_layout):
    """Says what is wrong with flce_linear_backward's arguments."""
    M, N, K, dev = _shapes(x, weight, weight_layout)
    shape = (*x.shape[:-1], N)
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a CUDA tensor")
    p = linear_params(M, N, K, activation, weight_layout, dout.dtype)
    B._need(dout, "dout", dout.dtype, shape, dev)
    if p.activation:
        if preact is None:
            raise ValueError("an activation's gradient needs preact")
        B._need(preact, "preact", torch.bfloat16, shape, dev)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation, weight_layout, out_dtype):
        needs = any(ctx.needs_input_grad[:3])
        keep = needs and _ACTIVATIONS.get(activation, 0) != 0
        y = flce_linear(x, weight, bias, activation, residual, weight_layout, out_dtype, keep)
        y, z = y if keep else (y, None)
        ctx.save_for_backward(x, weight, z)
        ctx.cfg = activation, weight_layout
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dw = db = None
        if any(need[:3]):
            dx, dw, db = flce_linear_backward(g.contiguous(), x, weight, z, *ctx.cfg, *need[:3])
        return dx, dw, db, g if need[3] else None, None, None, None


def linear(x, weight, bias=None, activation=None, residual=None, weight_layout="hv",
           out_dtype=torch.bfloat16):
    """act(x W + bias) + residual, differentiable by x, weight, bias and residual; see
    flce_linear."""
    if not torch.is_grad_enabled():  # (a Function is told that its inputs want gradients all the same)
        return flce_linear(x, weight, bias, activation, residual, weight_layout, out_dtype)
    return _Linear.apply(x, weight, bias, residual, activation, weight_layout, out_dtype)
