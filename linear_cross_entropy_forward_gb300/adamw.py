"""AdamW over many tensors at once, with states in 32 or 8 bits, and the norm of their gradients.

The step after the head's backward: dweight, the lookup's gradient and those of the layers go in
as they are (bf16, fp16 or fp32), the norm and the step are a launch each however many tensors
there are (up to 680; the next 680 are another), and neither copies anything from the host or waits,
so both can be captured in a graph.  Argument marshalling only; the library's kernels do the
work.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _binding as B
from .losses import _DTYPES, _current_device, _on, _raw_stream, _written

BLOCK = 128  # elements that share a scale of the 8-bit states
_TENSOR = np.dtype([("param", np.uint64), ("grad", np.uint64), ("n", np.int64),
                    ("offset", np.int64), ("weight_decay", np.float32), ("dtype", np.int32),
                    ("grad_dtype", np.int32)], align=True)
_STATE = {32: ("step", "master", "exp_avg", "exp_avg_sq"),
          8: ("step", "master", "exp_avg", "exp_avg_scale", "exp_rms", "exp_rms_scale")}


def _refuse_grad(g, name, shape, dtypes, index):
    if not isinstance(g, torch.Tensor) or not g.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor, got {type(g).__name__}")
    if g.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {g.dtype}")
    if shape is not None and g.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(g.shape)}")
    if not g.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {g.device}, not on cuda:{index}")


def _adamw_params(n_tensors, numel=0, lr=0.0, betas=(0.9, 0.999), eps=1e-8, grad_scale=1.0,
                  max_norm=None, state_bits=32, seed=0, skip_nonfinite=False):
    return B.FlceAdamwParams(n_tensors, numel, lr, betas[0], betas[1], eps, grad_scale,
                             max_norm or 0.0, state_bits, seed & 0xFFFFFFFF, bool(skip_nonfinite))


def flce_grad_norm(grads, scale=1.0, workspace=None, stream=None):
    """2-norm [1] fp32 of scale * all the given tensors together (bf16, fp16 or fp32, contiguous).

    Squares are summed in fp32 by eight (one that leaves fp32's range is infinite, or 0), these in
    a pair of floats per thread and in 64 bits from the blocks on, in a fixed order.
    workspace: uint8, zero at first and left so, as flce_adamw_workspace_size says."""
    if stream is not None:
        return _on(stream, flce_grad_norm, grads, scale, workspace)
    lib = B._lib or B.load_library()
    grads = list(grads)
    index = _current_device()
    table = np.zeros(len(grads), _TENSOR)
    for i, g in enumerate(grads):
        if not (isinstance(g, torch.Tensor) and g.dtype in _DTYPES and g.get_device() == index
                and g.is_contiguous()):
            _refuse_grad(g, f"tensor {i}", None, tuple(_DTYPES), index)
    table["grad"] = [g.data_ptr() for g in grads]
    table["n"] = [g.numel() for g in grads]
    table["dtype"] = table["grad_dtype"] = [_DTYPES[g.dtype] for g in grads]
    p = _adamw_params(len(grads), grad_scale=scale)
    ref = ctypes.byref(p)
    size = lib.flce_adamw_workspace_size(ref)
    if size == 0:
        B._check(lib.flce_adamw_check_params(ref))
    if workspace is None:
        workspace = torch.zeros(size, dtype=torch.uint8, device=index)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 \
            or not workspace.is_contiguous() or workspace.get_device() != index:
        raise TypeError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    elif workspace.numel() < size:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; this call needs {size}")
    norm = torch.empty(1, dtype=torch.float32, device=index)
    code = lib.flce_grad_norm(ref, table.ctypes.data, norm.data_ptr(), workspace.data_ptr(),
                              workspace.numel(), _raw_stream(index))
    if code:
        B._check(code)
    return norm


def _refuse_max_norm(max_norm):
    if max_norm is not None and not max_norm > 0:
        raise ValueError(f"max_norm must be positive or None, got {max_norm}")


class AdamW:
    """AdamW on a list of CUDA tensors (bf16, fp16 or fp32, contiguous, of one device).

    With t the step, c = grad_scale * min(1, max_norm / (norm + 1e-6)) and g = c * grad:
    m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
    p = p (1 - lr weight_decay) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).

    lr: a number, or a CUDA fp32 tensor of one element that is read by the step (a schedule
        under a captured graph).
    weight_decay: a number, or one per tensor.
    state_bits: 32 (m and v in fp32) or 8: m and sqrt(v) as float8_e4m3fn with an fp32 scale per
        128 elements, rounded up or down at random (by `seed`, the step and the element, so a
        run repeats bit for bit), which keeps their means where changes are below a code's step.
    master: keep fp32 weights beside the parameters, which then get them rounded; without, a
        16-bit parameter is updated and rounded in its own type (where a change below half its
        step is lost).
    max_norm: clip the gradients' norm; each step then returns it.  skip_nonfinite: a step whose
        norm is infinite or NaN changes nothing (fp16 gradients under a loss scale, which
        grad_scale divides out).

    lr, max_norm and grad_scale are attributes that each step reads, so that a schedule or a loss scale
    may change them; a captured step keeps those of its capture, but for an lr that is a tensor.

    The states of all tensors lie in flat tensors, each tensor's from a multiple of 128 on
    (`offsets`): state_dict() has them, as they are, not copies.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, master=False, max_norm=None, grad_scale=1.0,
                 skip_nonfinite=False, seed=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs at least one tensor")
        if state_bits not in _STATE:
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits!r}")
        _refuse_max_norm(max_norm)
        index = _current_device()
        for i, p in enumerate(self.params):
            if not (isinstance(p, torch.Tensor) and p.dtype in _DTYPES
                    and p.get_device() == index and p.is_contiguous()):
                _refuse_grad(p, f"parameter {i}", None, tuple(_DTYPES), index)
        n = len(self.params)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(decay) != n:
            raise ValueError(f"{len(decay)} weight decays for {n} tensors")
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size(), i)
                       for i, p in enumerate(self.params) if p.numel())
        for (_, end, i), (start, _, j) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"parameters {min(i, j)} and {max(i, j)} share memory")
        self._index, self._shapes = index, [p.shape for p in self.params]
        self._wanted = [(p.dtype,) if p.dtype is torch.float32 else (p.dtype, torch.float32)
                        for p in self.params]
        self._table = np.zeros(n, _TENSOR)
        self._table_at = self._table.ctypes.data
        self._columns = [self._table[name] for name in ("param", "grad", "grad_dtype")]
        self._table["n"] = [p.numel() for p in self.params]
        self._table["dtype"] = [_DTYPES[p.dtype] for p in self.params]
        self._table["weight_decay"] = decay
        padded = -(-self._table["n"] // BLOCK) * BLOCK
        self._table["offset"] = np.cumsum(padded) - padded
        self.offsets = self._table["offset"].tolist()
        numel = int(padded.sum())
        self.lr, self.state_bits = lr, state_bits
        self.max_norm, self.grad_scale, self._skip = max_norm, grad_scale, bool(skip_nonfinite)
        self._params = _adamw_params(n, numel, 0.0 if isinstance(lr, torch.Tensor) else lr, betas,
                                     eps, grad_scale, max_norm, state_bits, seed, skip_nonfinite)
        self._ref = ctypes.byref(self._params)
        lib = B._lib or B.load_library()
        size = lib.flce_adamw_workspace_size(self._ref)
        if size == 0:
            B._check(lib.flce_adamw_check_params(self._ref))
        self._workspace = torch.zeros(size, dtype=torch.uint8, device=index)
        self.step_count = torch.zeros(1, dtype=torch.int64, device=index)
        self.master = torch.zeros(numel, device=index) if master else None
        if state_bits == 32:
            self._state = {"exp_avg": torch.zeros(numel, device=index),
                           "exp_avg_sq": torch.zeros(numel, device=index)}
        else:
            self._state = {}
            for name in ("exp_avg", "exp_rms"):
                codes = torch.zeros(numel, dtype=torch.uint8, device=index)
                self._state[name] = codes.view(torch.float8_e4m3fn)
                self._state[name + "_scale"] = torch.zeros(numel // BLOCK, device=index)
        self._kept = [t for t in self.state_dict().values() if t is not None]
        if master:
            self.load_master()

    def load_master(self):
        """Takes the fp32 weights from the parameters (after they were changed from outside)."""
        for p, at in zip(self.params, self.offsets):
            self.master[at:at + p.numel()].copy_(p.detach().reshape(-1))

    def state_dict(self):
        """The states themselves, flat: step, master (or None) and the moments."""
        return {"step": self.step_count, "master": self.master, **self._state}

    def load_state_dict(self, state):
        """Copies what state_dict() of an optimizer over the same tensors, in the same order, gave.
        (Of the flat tensors only the sizes together can be compared.)"""
        mine = self.state_dict()
        if set(state) != set(mine):
            raise ValueError(f"state must hold {sorted(mine)}, got {sorted(state)}")
        for name, t in mine.items():
            other = state[name]
            if (t is None) != (other is None):
                raise ValueError(f"state {name} is {'missing' if other is None else 'not kept'}")
            if t is not None and (other.shape != t.shape or other.dtype != t.dtype):
                raise ValueError(f"state {name} must be {t.dtype} {tuple(t.shape)}, got "
                                 f"{other.dtype} {tuple(other.shape)}")
        for name, t in mine.items():
            if t is not None:
                t.copy_(state[name])

    def step(self, grads=None, stream=None):
        """One step with the given gradients (None: the parameters' .grad), in the parameters'
        types or fp32; every tensor has one.  Returns the gradients' norm [1] (before
        clipping), or None where nothing asks for it."""
        if stream is not None:
            return _on(stream, self.step, grads)
        lib = B._lib or B.load_library()
        index = self._index
        if index != _current_device():
            B._on_current_device(self.params[0])
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} tensors")
        for i, (p, g, shape, dtypes) in enumerate(zip(self.params, grads, self._shapes,
                                                      self._wanted)):
            if not (isinstance(g, torch.Tensor) and g.dtype in dtypes and g.shape == shape
                    and g.get_device() == index and g.is_contiguous()):
                _refuse_grad(g, f"gradient {i}", shape, dtypes, index)
            # (a parameter's data may have been exchanged since)
            if not (p.dtype is dtypes[0] and p.shape == shape and p.get_device() == index
                    and p.is_contiguous()):
                _refuse_grad(p, f"parameter {i}", shape, dtypes[:1], index)
        param, grad, grad_dtype = self._columns
        param[:] = [p.data_ptr() for p in self.params]
        grad[:] = [g.data_ptr() for g in grads]
        grad_dtype[:] = [_DTYPES[g.dtype] for g in grads]
        table = self._table_at
        lr_ptr = None
        if isinstance(self.lr, torch.Tensor):
            B._need(self.lr.reshape(1), "lr", torch.float32, (1,), self.step_count.device)
            lr_ptr = self.lr.data_ptr()
        else:
            self._params.lr = self.lr
        _refuse_max_norm(self.max_norm)
        self._params.max_norm, self._params.grad_scale = self.max_norm or 0.0, self.grad_scale
        stream = _raw_stream(index)
        ws = self._workspace
        norm = None
        if self._skip or self.max_norm is not None:
            norm = torch.empty(1, dtype=torch.float32, device=index)
            code = lib.flce_grad_norm(self._ref, table, norm.data_ptr(),
                                      ws.data_ptr(), ws.numel(), stream)
            if code:
                B._check(code)
        s = self._state
        if self.state_bits == 32:
            states = s["exp_avg"].data_ptr(), s["exp_avg_sq"].data_ptr(), None, None
        else:
            states = (s["exp_avg"].data_ptr(), s["exp_rms"].data_ptr(),
                      s["exp_avg_scale"].data_ptr(), s["exp_rms_scale"].data_ptr())
        code = lib.flce_adamw_step(
            self._ref, table, None if self.master is None else self.master.data_ptr(),
            *states, lr_ptr, None if norm is None else norm.data_ptr(),
            self.step_count.data_ptr(), ws.data_ptr(), ws.numel(), stream)
        if code:
            B._check(code)
        _written(self.params + self._kept)
        return norm
