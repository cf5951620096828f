"""The distribution that a sampler sees: penalties for repeated tokens, biases, a mask of allowed
tokens and the temperature on rows of logits, and what training needs of it.

A rollout samples from it; the policy loss needs the log-probabilities (and entropies) of the
sampled tokens under the same distribution, and a constrained or penalised step needs its
gradient.  Per row, in fp32:

    l = l / repetition_penalty where l > 0, else l * repetition_penalty,   for seen tokens
    l = l - frequency_penalty * n - presence_penalty * [n > 0] + the sum of its biases
    l = -inf where not allowed;   z = l / temperature

with n a token's occurrences among the row's generated tokens; prompt and generated tokens are
seen.  Argument marshalling only; one launch of the library per call.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B
from .losses import _DTYPES, _addr, _current_device, _on, _raw_stream, _written
from .workloads import IGNORE_INDEX

_WHOLE = {torch.int64: 1, torch.int32: 0}


def _per_row(value, name, R, index, none):
    """(number, address) of a number or a [R] fp32 tensor."""
    if not isinstance(value, torch.Tensor):
        return float(value), None
    if value.dtype is not torch.float32 or value.shape != (R,) or value.get_device() != index \
            or not value.is_contiguous():
        raise TypeError(f"{name} must be a number or a contiguous fp32 [{R}] tensor on "
                        f"cuda:{index}, got {value.dtype} {tuple(value.shape)} on {value.device}")
    return none, value.data_ptr()


def _lists(t, name, R, index, dtypes):
    """Row stride of a [R, n] tensor whose rows are dense (expanded rows have stride 0)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a CUDA tensor of "
                        f"{' or '.join(str(d) for d in dtypes)}")
    if t.dim() != 2 or t.shape[0] != R:
        raise ValueError(f"{name} must be [{R}, n], got shape {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the logits on cuda:{index}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    return t.stride(0)


def _lens(t, name, R, index):
    if not isinstance(t, torch.Tensor) or t.dtype not in _WHOLE or t.shape != (R,) \
            or t.get_device() != index or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int64 or int32 [{R}] tensor on cuda:{index}")
    return _WHOLE[t.dtype]


class _Call:
    """The C parameters of one set of options, and the tensors they point at."""

    def __init__(self, logits, tokens, prompt_lens, lengths, repetition_penalty,
                 frequency_penalty, presence_penalty, bias_ids, bias_values, allowed, temperature,
                 ignore_index, out_dtype, validate):
        if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
            raise TypeError("logits must be a CUDA tensor")
        if logits.dtype not in _DTYPES:
            raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
        if logits.dim() != 2 or logits.shape[1] < 1:
            raise ValueError(f"logits must be [R, V], got shape {tuple(logits.shape)}")
        self.index = index = logits.get_device()
        if index != _current_device():
            B._on_current_device(logits)
        R, V = logits.shape
        if logits.stride(1) != 1 and V > 1:
            raise ValueError("logits' last dimension must be dense")
        out_dtype = out_dtype or logits.dtype
        if out_dtype not in (logits.dtype, torch.float32):
            raise TypeError(f"out must be {logits.dtype} or float32, got {out_dtype}")
        # where an array says what is changed, the number stands for no change
        rep, rep_at = _per_row(repetition_penalty, "repetition_penalty", R, index, 1.0)
        freq, freq_at = _per_row(frequency_penalty, "frequency_penalty", R, index, 0.0)
        pres, pres_at = _per_row(presence_penalty, "presence_penalty", R, index, 0.0)
        temp, temp_at = _per_row(temperature, "temperature", R, index, 1.0)
        p = B.FlceLogitsParams(R, V, 0, logits.stride(0), V, 0, 0, 0, 0, 0, ignore_index, rep, freq,
                               pres, temp, _DTYPES[logits.dtype], _DTYPES[out_dtype], 0, 0, 0, 0,
                               bool(validate), 0)
        rows = B.FlceLogitsRows(None, None, None, rep_at, freq_at, pres_at, temp_at)
        if tokens is not None:
            p.ld_tokens = _lists(tokens, "tokens", R, index, tuple(_WHOLE))
            p.tokens_int64, p.T = _WHOLE[tokens.dtype], tokens.shape[1]
            rows.tokens = tokens.data_ptr()
            if prompt_lens is not None:
                p.lens_int64 = _lens(prompt_lens, "prompt_lens", R, index)
                rows.prompt_lens = prompt_lens.data_ptr()
            if lengths is not None:
                if prompt_lens is not None and lengths.dtype is not prompt_lens.dtype:
                    raise TypeError("prompt_lens and lengths must have the same type")
                p.lens_int64 = _lens(lengths, "lengths", R, index)
                rows.lengths = lengths.data_ptr()
        elif prompt_lens is not None or lengths is not None:
            raise ValueError("prompt_lens and lengths need tokens")
        if (bias_ids is None) != (bias_values is None):
            raise ValueError("bias_ids and bias_values come together")
        if bias_ids is not None:
            p.ld_bias_ids = _lists(bias_ids, "bias_ids", R, index, tuple(_WHOLE))
            p.ld_bias_values = _lists(bias_values, "bias_values", R, index, (torch.float32,))
            if bias_values.shape != bias_ids.shape:
                raise ValueError(f"bias_values must have shape {tuple(bias_ids.shape)}, got "
                                 f"{tuple(bias_values.shape)}")
            p.n_bias, p.bias_int64 = bias_ids.shape[1], _WHOLE[bias_ids.dtype]
            rows.bias_ids, rows.bias_values = bias_ids.data_ptr(), bias_values.data_ptr()
        if allowed is not None:
            p.ld_allowed = _lists(allowed, "allowed", R, index,
                                  (torch.bool, torch.uint8, torch.int32))
            p.mask_kind = 2 if allowed.dtype is torch.int32 else 1
            need = (V + 31) // 32 if p.mask_kind == 2 else V
            if allowed.shape[1] != need:
                raise ValueError(f"allowed must be [{R}, {need}] for {allowed.dtype}, got "
                                 f"{tuple(allowed.shape)}")
            rows.allowed = allowed.data_ptr()
        self.p, self.rows, self.R, self.V, self.out_dtype = p, rows, R, V, out_dtype
        # whose addresses are in rows
        self.keep = (tokens, prompt_lens, lengths, repetition_penalty, frequency_penalty,
                     presence_penalty, bias_ids, bias_values, allowed, temperature)

    def workspace(self):
        return torch.empty(256, dtype=torch.uint8, device=self.index) if self.p.validate else None


def _labels(labels, R, index):
    if not isinstance(labels, torch.Tensor) or labels.dtype is not torch.int64 \
            or labels.shape != (R,) or labels.get_device() != index or not labels.is_contiguous():
        raise TypeError(f"labels must be a contiguous int64 [{R}] tensor on cuda:{index}")


def flce_process_logits(logits, tokens=None, prompt_lens=None, lengths=None,
                        repetition_penalty=1.0, frequency_penalty=0.0, presence_penalty=0.0,
                        bias_ids=None, bias_values=None, allowed=None, temperature=1.0,
                        out=None, out_dtype=None, need_lse=False, stream=None):
    """z [R, V] of logits [R, V] (bf16, fp16 or fp32; rows may have a stride).

    tokens [R, T] int64 or int32: the row's prompt and then its generated tokens; the first
        lengths[r] count (None: all), the first prompt_lens[r] of them are the prompt's (None:
        none).  Ids outside [0, V) (padding) are left out.
    repetition_penalty, frequency_penalty, presence_penalty, temperature: a number, or fp32 [R].
        A temperature of 0 (a greedy row) leaves the row unscaled.
    bias_ids (int64 or int32), bias_values (fp32), [R, n], n <= 2048: added to their columns; ids
        outside [0, V) are left out, an id that comes twice has both.
    allowed: bool or uint8 [R, V], or int32 [R, (V + 31) // 32] with column v at bit v % 32 of
        word v // 32.  A row that allows nothing is all -inf.
    Any [R, n] argument may be one row expanded.  out: where z goes (logits' type or fp32; logits
    itself for in place), a new tensor if None.
    Returns z, or with need_lse (z, lse [R] fp32), so that log_softmax(z) = z - lse.
    """
    if stream is not None:
        return _on(stream, flce_process_logits, logits, tokens, prompt_lens, lengths,
                   repetition_penalty, frequency_penalty, presence_penalty, bias_ids, bias_values,
                   allowed, temperature, out, out_dtype, need_lse)
    lib = B._lib or B.load_library()
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise TypeError("out must be a CUDA tensor")
        if out_dtype is not None and out_dtype != out.dtype:
            raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
        out_dtype = out.dtype
    c = _Call(logits, tokens, prompt_lens, lengths, repetition_penalty, frequency_penalty,
              presence_penalty, bias_ids, bias_values, allowed, temperature, IGNORE_INDEX,
              out_dtype, False)
    given = out is not None
    if not given:
        out = torch.empty(c.R, c.V, dtype=c.out_dtype, device=c.index)
    else:
        if out.shape != (c.R, c.V) or out.get_device() != c.index:
            raise ValueError(f"out must be [{c.R}, {c.V}] on cuda:{c.index}, got "
                             f"{tuple(out.shape)} on {out.device}")
        c.p.ld_out = _lists(out, "out", c.R, c.index, (out.dtype,))
        _refuse_overlap(out, logits)
    lse = torch.empty(c.R, dtype=torch.float32, device=c.index) if need_lse else None
    code = lib.flce_logits(ctypes.byref(c.p), ctypes.byref(c.rows), logits.data_ptr(), None,
                           out.data_ptr(), _addr(lse), None, None, None, 0, _raw_stream(c.index))
    if code:
        B._check(code)
    if given:
        _written(out)
    return (out, lse) if need_lse else out


def _refuse_overlap(out, logits):
    """In place is out = logits, element for element; any other overlap would read what is written."""
    a, b = out.data_ptr(), logits.data_ptr()
    if a == b and out.dtype == logits.dtype and out.stride(0) == logits.stride(0):
        return

    def end(t):
        return t.data_ptr() + ((t.shape[0] - 1) * t.stride(0) + t.shape[1]) * t.element_size()

    if out.numel() and a < end(logits) and b < end(out):
        raise ValueError("out overlaps logits without being logits")


def flce_logits_logprob(logits, labels, tokens=None, prompt_lens=None, lengths=None,
                        repetition_penalty=1.0, frequency_penalty=0.0, presence_penalty=0.0,
                        bias_ids=None, bias_values=None, allowed=None, temperature=1.0,
                        ignore_index=IGNORE_INDEX, validate=False, stream=None, split_lse=False):
    """(logp, entropy, lse), fp32 [R]: of labels [R] int64 under softmax(z), z not stored.

    With split_lse, lse is [2, R]: behind each row's, what its rounding to fp32 left off, for a
    gradient that keeps its digits where logits are large.  The options are flce_process_logits'.
    A row whose label is ignore_index has logp and entropy 0; a label outside [0, V) gives NaN
    (with validate the call waits and raises); one that is not allowed -inf."""
    if stream is not None:
        return _on(stream, flce_logits_logprob, logits, labels, tokens, prompt_lens, lengths,
                   repetition_penalty, frequency_penalty, presence_penalty, bias_ids, bias_values,
                   allowed, temperature, ignore_index, validate, split_lse=split_lse)
    lib = B._lib or B.load_library()
    c = _Call(logits, tokens, prompt_lens, lengths, repetition_penalty, frequency_penalty,
              presence_penalty, bias_ids, bias_values, allowed, temperature, ignore_index, None,
              validate)
    _labels(labels, c.R, c.index)
    return _logprob(lib, c, logits, labels, split_lse)


def _logprob(lib, c, logits, labels, split_lse):
    c.p.split_lse = bool(split_lse)
    # (each a tensor of its own: views of one could not be changed in place behind autograd, and would
    # share the version that its check goes by)
    logp, ent, lse = (torch.empty(shape, dtype=torch.float32, device=c.index)
                      for shape in (c.R, c.R, (2, c.R) if split_lse else c.R))
    ws = c.workspace()
    code = lib.flce_logits(ctypes.byref(c.p), ctypes.byref(c.rows), logits.data_ptr(),
                           labels.data_ptr(), None, lse.data_ptr(), logp.data_ptr(),
                           ent.data_ptr(), _addr(ws), 256 if c.p.validate else 0,
                           _raw_stream(c.index))
    if code:
        B._check(code)
    return logp, ent, lse


def _row_grad(g, name, R, index, shape=None):
    shape = shape or (R,)
    if g is not None and (g.dtype is not torch.float32 or g.shape != shape
                          or g.get_device() != index or not g.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous fp32 {list(shape)} tensor on cuda:{index}")


def flce_logits_logprob_backward(logits, labels, lse, entropy, g_logp, g_entropy, tokens=None,
                                 prompt_lens=None, lengths=None, repetition_penalty=1.0,
                                 frequency_penalty=0.0, presence_penalty=0.0, bias_ids=None,
                                 bias_values=None, allowed=None, temperature=1.0,
                                 ignore_index=IGNORE_INDEX, grad_dtype=None, stream=None):
    """dlogits [R, V] (logits' type, or fp32 with grad_dtype) for upstream gradients g_logp and
    g_entropy, fp32 [R] or None (zero); lse ([R] or [2, R]) and entropy as flce_logits_logprob gave
    them.  With lse [R] a probability is off by its rounding, 2^-24 |lse| of itself.  Rows
    that are ignored, or of which the mask leaves nothing, get zeros."""
    if stream is not None:
        return _on(stream, flce_logits_logprob_backward, logits, labels, lse, entropy, g_logp,
                   g_entropy, tokens, prompt_lens, lengths, repetition_penalty,
                   frequency_penalty, presence_penalty, bias_ids, bias_values, allowed,
                   temperature, ignore_index, grad_dtype)
    lib = B._lib or B.load_library()
    c = _Call(logits, tokens, prompt_lens, lengths, repetition_penalty, frequency_penalty,
              presence_penalty, bias_ids, bias_values, allowed, temperature, ignore_index,
              grad_dtype, False)
    _labels(labels, c.R, c.index)
    split = isinstance(lse, torch.Tensor) and lse.dim() == 2
    _row_grad(lse, "lse", c.R, c.index, (2, c.R) if split else None)
    for name, t in (("entropy", entropy), ("g_logp", g_logp), ("g_entropy", g_entropy)):
        _row_grad(t, name, c.R, c.index)
    c.p.split_lse = split
    if lse is None or (g_entropy is not None and entropy is None):
        raise ValueError("the gradient needs lse, and that of the entropy needs entropy")
    return _logprob_backward(lib, c, logits, labels, lse, entropy, g_logp, g_entropy)


def _logprob_backward(lib, c, logits, labels, lse, entropy, g_logp, g_entropy):
    d = torch.empty(c.R, c.V, dtype=c.out_dtype, device=c.index)
    code = lib.flce_logits_backward(ctypes.byref(c.p), ctypes.byref(c.rows), logits.data_ptr(),
                                    labels.data_ptr(), lse.data_ptr(), _addr(entropy),
                                    _addr(g_logp), _addr(g_entropy), d.data_ptr(), None, 0,
                                    _raw_stream(c.index))
    if code:
        B._check(code)
    return d


class _LogitsLogprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, options):
        lib = B._lib or B.load_library()
        c = _Call(logits, *options)
        _labels(labels, c.R, c.index)
        logp, ent, lse = _logprob(lib, c, logits, labels, True)
        # the options' tensors are saved for the check that nothing has changed them since
        ctx.save_for_backward(logits, labels, lse, ent,
                              *(t for t in options if isinstance(t, torch.Tensor)))
        c.p.validate = 0
        ctx.call = c
        ctx.set_materialize_grads(False)
        return logp, ent

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logp, g_ent):
        logits, labels, lse, ent = ctx.saved_tensors[:4]
        if g_logp is None and g_ent is None:
            return None, None, None
        g_logp, g_ent = (None if g is None else g.contiguous() for g in (g_logp, g_ent))
        c = ctx.call
        if c.index != _current_device():
            B._on_current_device(logits)
        if logits.stride(1) != 1:
            logits = logits.contiguous()
        c.p.ld_logits = logits.stride(0)  # a saved tensor may come back as a copy
        for name, g in (("g_logp", g_logp), ("g_entropy", g_ent)):
            _row_grad(g, name, c.R, c.index)
        return _logprob_backward(B._lib, c, logits, labels, lse, ent, g_logp, g_ent), None, None


def logits_logprob(logits, labels, tokens=None, prompt_lens=None, lengths=None,
                   repetition_penalty=1.0, frequency_penalty=0.0, presence_penalty=0.0,
                   bias_ids=None, bias_values=None, allowed=None, temperature=1.0,
                   ignore_index=IGNORE_INDEX, validate=False):
    """(logp, entropy) of labels under the processed distribution, differentiable by logits (the
    options have no gradient); see flce_logits_logprob."""
    return _LogitsLogprob.apply(logits, labels, (
        tokens, prompt_lens, lengths, repetition_penalty, frequency_penalty, presence_penalty,
        bias_ids, bias_values, allowed, temperature, ignore_index, None, validate))
