"""Embedding lookup with scaling, and its gradient by sorted tokens.

The table is [V, H], the layout of an LM head with weight_layout 'vh', so that one matrix
can be both (a tied model): the head's dweight then takes the lookup's gradient in place
with accumulate=True.  Argument marshalling only; the library's kernels do the work.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B
from .losses import _DTYPES, _current_device, _on, _raw_stream, _workspace


def embedding_params(N, H, V, scale=1.0, dtype=torch.bfloat16, grad_dtype=None, ids_int64=True,
                     accumulate=False, padding_idx=None, v_offset=0, v_total=0, validate=False):
    """FlceEmbeddingParams; padding_idx None: none (the C struct's -1; no row counts from the end)."""
    if padding_idx is not None and padding_idx < 0:
        raise ValueError(f"padding_idx must be a row of the table or None, got {padding_idx}")
    try:
        dt, gdt = _DTYPES[dtype], _DTYPES[grad_dtype or dtype]
    except KeyError as e:
        raise TypeError(f"embedding types are float32, bfloat16 and float16, got {e}") from None
    return B.FlceEmbeddingParams(N, H, V, v_offset, v_total,
                                 -1 if padding_idx is None else padding_idx, scale, dt, gdt,
                                 bool(ids_int64), bool(accumulate), bool(validate))


def embedding_workspace_size(params: "B.FlceEmbeddingParams") -> int:
    """Bytes of workspace a flce_embedding_backward call with these parameters needs."""
    lib = B._lib or B.load_library()
    size = lib.flce_embedding_workspace_size(ctypes.byref(params))
    if size == 0:
        B._check(lib.flce_embedding_check_params(ctypes.byref(params)))
    return size


def _need_ids(ids):
    """Checks the ids; their device's index."""
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise TypeError("ids must be a CUDA tensor")
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"ids must be int64 or int32, got {ids.dtype}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    index = ids.get_device()
    if index != _current_device():
        B._on_current_device(ids)
    return index


_IDS = {torch.int64: 1, torch.int32: 0}


def _refuse_lookup(ids, weight):
    _need_ids(ids)
    if not isinstance(weight, torch.Tensor) or not weight.is_cuda or weight.dtype not in _DTYPES:
        raise TypeError("weight must be a bf16, fp16 or fp32 CUDA tensor")
    if weight.dim() != 2 or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [V, H], got shape {tuple(weight.shape)}")
    if weight.get_device() != ids.get_device():
        raise ValueError(f"weight is on {weight.device}, ids on {ids.device}")


def flce_embedding(ids, weight, scale=1.0, v_offset=0, v_total=0, validate=False, stream=None,
                   out=None):
    """scale * weight[ids], of shape [*ids.shape, H].

    weight [V, H] bf16, fp16 or fp32; ids int64 or int32 of any shape.  With v_total > 0
    weight holds rows [v_offset, v_offset + V) of a table of v_total rows and other shards'
    rows are zero, so that the shards' sum is the lookup.  An id outside the table gives a
    row of NaN; with validate the call waits and raises.
    """
    if stream is not None:
        return _on(stream, flce_embedding, ids, weight, scale, v_offset, v_total, validate,
                   out=out)
    lib = B._lib or B.load_library()
    # one pass over what is right, as a small lookup's time is these checks; _refuse_lookup
    # says what is wrong
    try:
        ids64, dt, dev = _IDS[ids.dtype], _DTYPES[weight.dtype], ids.get_device()
        V, H = weight.shape
        if not (dev >= 0 and dev == weight.get_device() and dev == _current_device()
                and ids.is_contiguous() and weight.is_contiguous()):
            raise ValueError
    except (AttributeError, KeyError, ValueError):
        _refuse_lookup(ids, weight)
        raise
    shape = (*ids.shape, H)
    p = B.FlceEmbeddingParams(ids.numel(), H, V, v_offset, v_total, -1, scale, dt, dt, ids64, 0,
                              bool(validate))
    if out is None:
        out = torch.empty(shape, dtype=weight.dtype, device=dev)
    else:
        B._need(out, "out", weight.dtype, shape, ids.device)
    ws = torch.empty(256, dtype=torch.uint8, device=dev) if validate else None
    code = lib.flce_embedding(ctypes.byref(p), ids.data_ptr(), weight.data_ptr(), out.data_ptr(),
                              None if ws is None else ws.data_ptr(), 256 if validate else 0,
                              _raw_stream(dev))
    if code:
        B._check(code)
    return out


def flce_embedding_backward(dout, ids, V, scale=1.0, padding_idx=None, dweight=None,
                            accumulate=False, grad_dtype=None, v_offset=0, v_total=0,
                            validate=False, workspace=None, stream=None):
    """The gradient [V, H] of flce_embedding by weight: row v is scale times the sum of
    dout's rows whose id is v, summed in fp32 in a fixed order (the tokens', in groups of up
    to 32 that are then added) and rounded once.

    dweight: where it goes (dout's type, or fp32), a new tensor if None; accumulate=True adds
    to it and touches no other row.  Ids equal to padding_idx (a row of the whole table) have
    no gradient, nor have those of other shards.
    """
    if stream is not None:
        return _on(stream, flce_embedding_backward, dout, ids, V, scale, padding_idx, dweight,
                   accumulate, grad_dtype, v_offset, v_total, validate, workspace)
    lib = B._lib or B.load_library()
    dev = _need_ids(ids)
    if not isinstance(dout, torch.Tensor) or not dout.is_cuda or dout.dtype not in _DTYPES:
        raise TypeError("dout must be a bf16, fp16 or fp32 CUDA tensor")
    if dout.dim() < 1:
        raise ValueError("dout must be [*ids.shape, H]")
    H = dout.shape[-1]
    B._need(dout, "dout", dout.dtype, (*ids.shape, H), ids.device)
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate needs dweight")
        gdt = grad_dtype or dout.dtype
    else:
        gdt = dweight.dtype if isinstance(dweight, torch.Tensor) else None
        if grad_dtype is not None and grad_dtype != gdt:
            raise TypeError(f"dweight must be {grad_dtype}, got {gdt}")
        B._need(dweight, "dweight", gdt, (V, H), ids.device)
    if gdt not in (dout.dtype, torch.float32):
        raise TypeError(f"dweight must be {dout.dtype} or float32, got {gdt}")
    p = embedding_params(ids.numel(), H, V, scale, dout.dtype, gdt, ids.dtype is torch.int64,
                         accumulate, padding_idx, v_offset, v_total, validate)
    size = embedding_workspace_size(p)
    if dweight is None:
        dweight = torch.empty(V, H, dtype=gdt, device=dev)
    ws = _workspace(size, dev, workspace)
    code = lib.flce_embedding_backward(
        ctypes.byref(p), dout.data_ptr(), ids.data_ptr(), dweight.data_ptr(), ws.data_ptr(),
        ws.numel(), _raw_stream(dev))
    if code:
        B._check(code)
    return dweight


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, padding_idx, v_offset, v_total):
        out = flce_embedding(ids, weight, scale, v_offset, v_total)
        V, H = weight.shape
        if padding_idx is not None:  # the lookup has no use for it: refused here, not in the backward
            p = embedding_params(ids.numel(), H, V, scale, weight.dtype, None, True, False,
                                 padding_idx, v_offset, v_total)
            B._check(B.load_library().flce_embedding_check_params(ctypes.byref(p)))
        ctx.save_for_backward(ids)
        ctx.cfg = (V, scale, padding_idx, v_offset, v_total)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        (ids,) = ctx.saved_tensors
        V, scale, padding_idx, v_offset, v_total = ctx.cfg
        dw = flce_embedding_backward(g.contiguous(), ids, V, scale, padding_idx,
                                     v_offset=v_offset, v_total=v_total)
        return None, dw, None, None, None, None


def embedding(ids, weight, scale=1.0, padding_idx=None, v_offset=0, v_total=0):
    """scale * weight[ids], differentiable by weight (a dense gradient of weight's type; ids
    equal to padding_idx get none)."""
    return _Embedding.apply(ids, weight, scale, padding_idx, v_offset, v_total)
