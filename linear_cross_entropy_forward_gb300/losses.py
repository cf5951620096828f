"""Losses over sequences of tokens: the clipped policy loss and the preference loss.

Both read the log-probabilities that linear_cross_entropy's head gives (logp = -loss with
reduction 'none') and return the gradients its backward takes.  A batch is padded,
[B, S], or packed, [T] with cu_seqlens [B + 1]; a 1-D batch without cu_seqlens is one
sequence.  `mask` says which tokens count: bool or uint8 (non-zero counts), or the int64
labels themselves (those other than ignore_index count).  What does not count may hold
anything.  Arguments of a padded batch may have row strides (slices, expanded rows);
the last dimension must be dense.  Gradients are dense.

Argument marshalling only, as in the rest of the binding: the computation, one launch
per call, is the library's.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B
from .workloads import IGNORE_INDEX, RED_NONE, reduction_code

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_KL = {"k1": 1, "k2": 2, "k3": 3}
_RATIO = {"token": 0, "sequence": 1}
_AGGREGATE = {"token_mean": 0, "seq_mean_token_mean": 1, "seq_mean_token_sum": 2, "sum": 3}
_PREFERENCE = {"sigmoid": 0, "robust": 1, "hinge": 2, "ipo": 3}
_PAIRS = {"halves": 0, "interleaved": 1}


def _code(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {'/'.join(table)}, got {value!r}") from None


_MASKS = {torch.bool: 1, torch.uint8: 1, torch.int64: 2}

# the plain integers behind torch.cuda.current_device() and current_stream(), which cost
# a few microseconds where a small call takes twenty
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _on(stream, call, *args, **kw):
    """call(...) with `stream` current: new tensors then belong to the stream that the kernels
    run on (memory of another stream's pool could still be in use there)."""
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _refuse(t, name, dtype, shape, index):
    """Says what is wrong with one array of a batch."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")


def _rows(t, name, dtype, shape, index):
    """Checks one array of a batch; its row stride in elements."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == index):
        _refuse(t, name, dtype, shape, index)
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    return s[0]


def _batch(logp, mask, cu_seqlens, ignore_index):
    """(FlceSeqs, device index, number of sequences) of a batch laid out like logp."""
    if not isinstance(logp, torch.Tensor) or not logp.is_cuda:
        raise TypeError("logp must be a CUDA tensor")
    dt = _DTYPES.get(logp.dtype)
    if dt is None:
        raise TypeError(f"logp must be float32, bfloat16 or float16, got {logp.dtype}")
    index = logp.get_device()
    if index != _current_device():
        B._on_current_device(logp)
    shape = logp.shape
    cu_kind = cu_ptr = mask_kind = mask_ptr = ld_mask = 0
    if cu_seqlens is not None:
        if len(shape) != 1:
            raise ValueError("with cu_seqlens, logp must be 1-D")
        if not isinstance(cu_seqlens, torch.Tensor) or not cu_seqlens.is_cuda \
                or cu_seqlens.dtype not in (torch.int32, torch.int64):
            raise TypeError("cu_seqlens must be an int32 or int64 CUDA tensor")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous [B + 1] tensor")
        if cu_seqlens.get_device() != index:
            raise ValueError(f"cu_seqlens is on {cu_seqlens.device}, logp on {logp.device}")
        n_seq, S = cu_seqlens.numel() - 1, shape[0]
        cu_kind = 1 if cu_seqlens.dtype is torch.int32 else 2
        cu_ptr = cu_seqlens.data_ptr()
    elif len(shape) == 1:
        n_seq, S = 1, shape[0]
    elif len(shape) == 2:
        n_seq, S = shape
    else:
        raise ValueError(f"logp must be [B, S] or [T], got shape {tuple(shape)}")
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype not in _MASKS:
            raise TypeError("mask must be a bool, uint8 or int64 (labels) tensor")
        ld_mask = _rows(mask, "mask", mask.dtype, shape, index)
        mask_kind = _MASKS[mask.dtype]
        mask_ptr = mask.data_ptr() or 8  # an array of no elements has no address
    return B.FlceSeqs(n_seq, S, cu_ptr, mask_ptr, ld_mask, ignore_index, cu_kind, mask_kind,
                      dt), index, n_seq


def _scalar_grad(g, n, index):
    if g is not None:
        _rows(g, "g_loss", torch.float32, torch.Size((n,)), index)


def policy_params(logp, old_logp=None, advantages=None, ref_logp=None, entropy=None, mask=None,
                  cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0,
                  kl="k3", entropy_coef=0.0, ratio="token", aggregate="token_mean", scale=1.0,
                  ignore_index=IGNORE_INDEX, validate=False, adv_per_token=None):
    """(FlcePolicyParams, device index) of a flce_policy_loss call, its tensors checked."""
    seqs, index, n_seq = _batch(logp, mask, cu_seqlens, ignore_index)
    shape, dt = logp.shape, logp.dtype
    ld_logp = _rows(logp, "logp", dt, shape, index)
    ld_old = ld_ref = ld_ent = 0
    if old_logp is not None:
        ld_old = _rows(old_logp, "old_logp", dt, shape, index)
    if ref_logp is not None:
        ld_ref = _rows(ref_logp, "ref_logp", dt, shape, index)
    elif kl_coef:
        raise ValueError("kl_coef needs ref_logp")
    if entropy is not None:
        ld_ent = _rows(entropy, "entropy", dt, shape, index)
    elif entropy_coef:
        raise ValueError("entropy_coef needs entropy")
    if not isinstance(advantages, torch.Tensor):
        raise TypeError("advantages must be a CUDA tensor")
    per_seq = torch.Size((n_seq,))
    if adv_per_token is None:
        # one per sequence, unless the shape is the tokens' and that reading is the only one
        per_token = advantages.shape != per_seq and ratio != "sequence"
    else:
        per_token = bool(adv_per_token)
    ld_adv = _rows(advantages, "advantages", torch.float32, shape if per_token else per_seq, index)
    if not per_token and not advantages.is_contiguous():
        raise ValueError("advantages must be contiguous")
    return B.FlcePolicyParams(
        seqs, ld_logp, ld_old, ld_ref, ld_ent, ld_adv, clip_low, clip_high, dual_clip, kl_coef,
        entropy_coef, scale, _code(_KL, kl, "kl"), _code(_RATIO, ratio, "ratio"),
        _code(_AGGREGATE, aggregate, "aggregate"), per_token, bool(validate)), index


def _workspace(size, index, workspace):
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=index)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 \
            or not workspace.is_contiguous() or workspace.get_device() != index:
        raise TypeError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    if workspace.numel() < size:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; this call needs {size}")
    return workspace


def _size(lib, name, ref):
    size = getattr(lib, f"flce_{name}_workspace_size")(ref)
    if size == 0:
        B._check(getattr(lib, f"flce_{name}_check_params")(ref))
    return size


def policy_workspace_size(params: "B.FlcePolicyParams") -> int:
    """Bytes of workspace a flce_policy_loss call with these parameters needs."""
    return int(_size(B.load_library(), "policy", ctypes.byref(params)))


def _addr(t):
    return None if t is None else t.data_ptr()


def flce_policy_loss(logp, old_logp, advantages, ref_logp=None, entropy=None, mask=None,
                     cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0,
                     kl="k3", entropy_coef=0.0, ratio="token", aggregate="token_mean", scale=1.0,
                     ignore_index=IGNORE_INDEX, g_loss=None, need_loss=True, need_grad=True,
                     need_entropy_grad=True, validate=False, workspace=None, stream=None,
                     adv_per_token=None):
    """Clipped policy loss and its gradients, in one launch.

    Per counted token, with d = logp - old_logp, r = exp(d) and A its advantage:
    -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) -- for A < 0 and dual_clip c > 1 at
    most -c A -- plus kl_coef K(logp, ref_logp) minus entropy_coef * entropy.  old_logp None:
    d = 0 (the policy itself).  kl: 'k1' logp - ref, 'k2' its half square, 'k3'
    exp(-k1) - 1 + k1.  Log-ratios are clamped to +-20, with zero gradient beyond.
    ratio 'sequence' takes the mean of d over each sequence's counted tokens.
    advantages: fp32 [B], one per sequence, or one per token (logp's shape); adv_per_token says
    which where a packed batch has as many tokens as sequences (None: one per sequence there).
    aggregate: 'token_mean', 'seq_mean_token_mean', 'seq_mean_token_sum', or 'sum' (times
    scale); sequences without a counted token do not count.

    Returns (loss [1], stats [4], counts [4], dlogp, dentropy).  stats: the aggregated
    policy term, mean KL to the reference, mean entropy, mean k3 to the old policy.
    counts (int64): counted tokens, sequences with one, clipped tokens (sequences),
    dual-clipped ones.  The gradients are times g_loss ([1] fp32, None: 1).  Parts that
    are not wanted (need_loss, need_grad, need_entropy_grad) or not there (dentropy without
    entropy) are None.
    """
    if stream is not None:
        return _on(stream, flce_policy_loss, logp, old_logp, advantages, ref_logp, entropy, mask,
                   cu_seqlens, clip_low, clip_high, dual_clip, kl_coef, kl, entropy_coef, ratio,
                   aggregate, scale, ignore_index, g_loss, need_loss, need_grad,
                   need_entropy_grad, validate, workspace, adv_per_token=adv_per_token)
    lib = B._lib or B.load_library()
    p, dev = policy_params(logp, old_logp, advantages, ref_logp, entropy, mask, cu_seqlens,
                           clip_low, clip_high, dual_clip, kl_coef, kl, entropy_coef, ratio,
                           aggregate, scale, ignore_index, validate, adv_per_token)
    if not need_loss and not need_grad:
        raise ValueError("neither the loss nor the gradients are wanted")
    _scalar_grad(g_loss, 1, dev)
    ref = ctypes.byref(p)
    size = _size(lib, "policy", ref)
    loss = stats = counts = dlogp = dent = None
    if need_loss:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        stats = torch.empty(4, dtype=torch.float32, device=dev)
        counts = torch.empty(4, dtype=torch.int64, device=dev)
    if need_grad:
        dlogp = torch.empty(logp.shape, dtype=logp.dtype, device=dev)
        if entropy is not None and need_entropy_grad:
            dent = torch.empty(logp.shape, dtype=logp.dtype, device=dev)
    ws = _workspace(size, dev, workspace)
    if not need_loss and logp.numel() == 0:
        return loss, stats, counts, dlogp, dent
    code = lib.flce_policy_loss(
        ref, logp.data_ptr(), _addr(old_logp), _addr(ref_logp), _addr(entropy),
        advantages.data_ptr(), _addr(g_loss), _addr(loss), _addr(stats), _addr(counts),
        _addr(dlogp), _addr(dent), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if code:
        B._check(code)
    return loss, stats, counts, dlogp, dent


def _upstream(g):
    """An upstream gradient as the library takes it: dense fp32 of one dimension."""
    g = g.reshape(-1)
    return g if g.dtype is torch.float32 and g.is_contiguous() else g.float().contiguous()


class _PolicyLoss(torch.autograd.Function):
    """fp32: the launch that forms the loss forms the gradients of it, and the backward
    multiplies them by the upstream gradient (as the kernel would, with the same rounding;
    290 us a step with autograd against 340).  A 16-bit gradient would be rounded twice that
    way: there the backward is a launch of its own."""

    @staticmethod
    def forward(ctx, logp, entropy, old_logp, advantages, ref_logp, mask, cu_seqlens, kw):
        need_lp, need_ent = ctx.needs_input_grad[:2]
        ctx.formed = logp.dtype is torch.float32
        loss, stats, counts, dlogp, dent = flce_policy_loss(
            logp, old_logp, advantages, ref_logp, entropy, mask, cu_seqlens,
            need_grad=ctx.formed and (need_lp or need_ent), need_entropy_grad=need_ent, **kw)
        if ctx.formed:
            ctx.save_for_backward(dlogp, dent)
        else:
            ctx.save_for_backward(logp, entropy, old_logp, advantages, ref_logp, mask, cu_seqlens)
            ctx.kw = kw
        ctx.mark_non_differentiable(stats, counts)
        return loss[0], stats, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, _g_stats, _g_counts):
        need_lp, need_ent = ctx.needs_input_grad[:2]
        if ctx.formed:
            dlogp, dent = ctx.saved_tensors
            dlogp = dlogp * g_loss if need_lp else None
            dent = dent * g_loss if need_ent else None
        else:
            logp, entropy, old_logp, advantages, ref_logp, mask, cu = ctx.saved_tensors
            _, _, _, dlogp, dent = flce_policy_loss(
                logp, old_logp, advantages, ref_logp, entropy, mask, cu, g_loss=_upstream(g_loss),
                need_loss=False, need_entropy_grad=need_ent, **ctx.kw)
        return dlogp, dent, None, None, None, None, None, None


def policy_loss(logp, old_logp, advantages, ref_logp=None, entropy=None, mask=None,
                cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl="k3",
                entropy_coef=0.0, ratio="token", aggregate="token_mean", scale=1.0,
                ignore_index=IGNORE_INDEX, adv_per_token=None):
    """loss, stats, counts = policy_loss(logp, old_logp, advantages, ...)

    flce_policy_loss as a differentiable function of logp and entropy (the other tensors are
    constants): loss is a scalar, stats and counts carry no gradient.  With the head:

        nll, entropy = linear_cross_entropy(hidden, weight, labels, reduction="none")
        loss, stats, counts = policy_loss(-nll, old_logp, advantages, entropy=entropy,
                                          mask=labels, cu_seqlens=cu, entropy_coef=0.01)

    linear_policy_loss does the two in one call without recomputing the logits.
    """
    kw = dict(clip_low=clip_low, clip_high=clip_high, dual_clip=dual_clip, kl_coef=kl_coef, kl=kl,
              entropy_coef=entropy_coef, ratio=ratio, aggregate=aggregate, scale=scale,
              ignore_index=ignore_index, adv_per_token=adv_per_token)
    return _PolicyLoss.apply(logp, entropy, old_logp, advantages, ref_logp, mask, cu_seqlens, kw)


def flce_policy_forward_backward(hidden, weight, labels, old_logp, advantages, ref_logp=None,
                                 cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0,
                                 kl_coef=0.0, kl="k3", entropy_coef=0.0, ratio="token",
                                 aggregate="token_mean", scale=1.0, ignore_index=IGNORE_INDEX,
                                 softcap=0.0, weight_layout="hv", chunk_n=0, dhidden_fp32=False,
                                 g_loss=None, validate=False, workspace=None, stream=None,
                                 adv_per_token=None):
    """The policy loss on top of the LM head, with dhidden and dweight, in one call.

    hidden [N, H], weight and labels as in flce_forward_backward; old_logp, ref_logp fp32 [N];
    advantages fp32 [B] or [N] (adv_per_token as in flce_policy_loss); cu_seqlens [B + 1] cuts
    the N tokens into sequences (None: one).  Tokens whose label is ignore_index do not count.  ratio 'sequence' needs all
    tokens in one chunk (chunk_n >= N).
    Returns (loss [1], stats [4], counts [4], logp [N], entropy [N], dhidden, dweight);
    the gradients are times g_loss ([1] fp32, None: 1).  As in flce_forward_backward, the
    gradients of the logits are rounded to bf16 before the products with weight and hidden.
    """
    if stream is not None:
        return _on(stream, flce_policy_forward_backward, hidden, weight, labels, old_logp,
                   advantages, ref_logp, cu_seqlens, clip_low, clip_high, dual_clip, kl_coef, kl,
                   entropy_coef, ratio, aggregate, scale, ignore_index, softcap, weight_layout,
                   chunk_n, dhidden_fp32, g_loss, validate, workspace, adv_per_token=adv_per_token)
    lib = B._lib or B.load_library()
    N, H, V, wshape = B._dims(hidden, weight, weight_layout)
    B._need(hidden, "hidden", torch.bfloat16, (N, H))
    dev = B._on_current_device(hidden)
    B._need(weight, "weight", torch.bfloat16, wshape, dev)
    B._need(labels, "labels", torch.int64, (N,), dev)
    p = B.make_params(N, H, V, "none", ignore_index, 0.0, softcap, validate,
                      weight_layout=weight_layout, chunk_n=chunk_n, dhidden_fp32=dhidden_fp32)
    logp = torch.empty(N, dtype=torch.float32, device=dev)
    entropy = torch.empty(N, dtype=torch.float32, device=dev)
    q, index = policy_params(logp, old_logp, advantages, ref_logp, entropy, None, cu_seqlens,
                             clip_low, clip_high, dual_clip, kl_coef, kl, entropy_coef, ratio,
                             aggregate, scale, ignore_index, validate, adv_per_token)
    _scalar_grad(g_loss, 1, index)
    size = lib.flce_policy_head_workspace_size(ctypes.byref(p), ctypes.byref(q))
    if size == 0:
        B._check(lib.flce_check_params(ctypes.byref(p)))
        _size(lib, "policy", ctypes.byref(q))
        raise B.FlceError(1, "the head cannot take these parameters (a sequence ratio needs all "
                             "tokens in one chunk)")
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    stats = torch.empty(4, dtype=torch.float32, device=dev)
    counts = torch.empty(4, dtype=torch.int64, device=dev)
    dh = torch.empty(N, H, dtype=torch.float32 if dhidden_fp32 else torch.bfloat16, device=dev)
    dw = torch.empty(wshape, dtype=torch.bfloat16, device=dev)
    ws = _workspace(size, index, workspace)
    B._check(lib.flce_policy_forward_backward(
        ctypes.byref(p), ctypes.byref(q), _addr(hidden), _addr(weight), _addr(labels),
        _addr(old_logp), _addr(ref_logp), _addr(advantages), _addr(g_loss), _addr(loss),
        _addr(stats), _addr(counts), _addr(logp), _addr(entropy), _addr(dh), _addr(dw),
        ws.data_ptr(), ws.numel(), _raw_stream(index)))
    return loss, stats, counts, logp, entropy, dh, dw


class _LinearPolicyLoss(torch.autograd.Function):
    """The gradients are formed in the forward, for an upstream gradient of 1, and scaled in
    the backward (a copy: the saved ones serve another backward pass).  Scaled by anything but
    a power of two, a bf16 gradient is rounded a second time, as with grad_in_forward."""

    @staticmethod
    def forward(ctx, hidden, weight, labels, old_logp, advantages, ref_logp, cu_seqlens, kw):
        loss, stats, counts, logp, entropy, dh, dw = flce_policy_forward_backward(
            hidden, weight, labels, old_logp, advantages, ref_logp, cu_seqlens, **kw)
        ctx.save_for_backward(dh, dw)
        ctx.mark_non_differentiable(stats, counts, logp, entropy)
        return loss[0], stats, counts, logp, entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, *_):
        dh, dw = ctx.saved_tensors
        g = _upstream(g_loss)
        dh = B.flce_scale_bf16(dh.clone(), g) if ctx.needs_input_grad[0] else None
        dw = B.flce_scale_bf16(dw.clone(), g) if ctx.needs_input_grad[1] else None
        return dh, dw, None, None, None, None, None, None


def linear_policy_loss(hidden, weight, labels, old_logp, advantages, ref_logp=None,
                       cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0,
                       kl="k3", entropy_coef=0.0, ratio="token", aggregate="token_mean",
                       scale=1.0, ignore_index=IGNORE_INDEX, softcap=0.0, weight_layout="hv",
                       chunk_n=0, adv_per_token=None):
    """loss, stats, counts, logp, entropy = linear_policy_loss(hidden, weight, labels, ...)

    policy_loss(-nll, ...) of linear_cross_entropy's per-token nll and entropy, with the
    gradients by hidden and weight formed in the forward: the logits are computed once.
    Differentiable by hidden and weight through loss alone.  An upstream gradient that is no
    power of two costs the bf16 gradients a second rounding (flce_policy_forward_backward's
    g_loss does not).
    """
    kw = dict(clip_low=clip_low, clip_high=clip_high, dual_clip=dual_clip, kl_coef=kl_coef, kl=kl,
              entropy_coef=entropy_coef, ratio=ratio, aggregate=aggregate, scale=scale,
              ignore_index=ignore_index, softcap=softcap, weight_layout=weight_layout,
              chunk_n=chunk_n, adv_per_token=adv_per_token)
    return _LinearPolicyLoss.apply(hidden, weight, labels, old_logp, advantages, ref_logp,
                                   cu_seqlens, kw)


def preference_params(logp, ref_logp=None, ref_scores=None, mask=None, cu_seqlens=None, beta=0.1,
                      loss_type="sigmoid", label_smoothing=0.0, margin=0.0,
                      length_normalised=False, nll_coef=0.0, pairs="halves", reduction="mean",
                      ignore_index=IGNORE_INDEX, validate=False):
    """(FlcePreferenceParams, device index) of a flce_preference_loss call, its tensors checked."""
    seqs, index, n_seq = _batch(logp, mask, cu_seqlens, ignore_index)
    if n_seq % 2:
        raise ValueError(f"pairs need an even number of sequences, got {n_seq}")
    ld_logp = _rows(logp, "logp", logp.dtype, logp.shape, index)
    ld_ref = 0
    if ref_logp is not None:
        ld_ref = _rows(ref_logp, "ref_logp", logp.dtype, logp.shape, index)
    if ref_scores is not None:
        _rows(ref_scores, "ref_scores", torch.float32, torch.Size((n_seq,)), index)
    return B.FlcePreferenceParams(
        seqs, ld_logp, ld_ref, beta, margin, label_smoothing, nll_coef,
        _code(_PREFERENCE, loss_type, "loss_type"), bool(length_normalised),
        _code(_PAIRS, pairs, "pairs"), reduction_code(reduction), bool(validate)), index


def preference_workspace_size(params: "B.FlcePreferenceParams") -> int:
    """Bytes of workspace a flce_preference_loss call with these parameters needs."""
    return int(_size(B.load_library(), "preference", ctypes.byref(params)))


def flce_preference_loss(logp, ref_logp=None, ref_scores=None, mask=None, cu_seqlens=None,
                         beta=0.1, loss_type="sigmoid", label_smoothing=0.0, margin=0.0,
                         length_normalised=False, nll_coef=0.0, pairs="halves", reduction="mean",
                         ignore_index=IGNORE_INDEX, g_loss=None, need_loss=True, need_grad=True,
                         validate=False, workspace=None, stream=None):
    """Preference loss over pairs of sequences and its gradient, in one launch.

    s_i = sum over sequence i's counted tokens of logp - ref_logp (divided by their number
    with length_normalised), minus ref_scores[i] (fp32 [B], reference scores kept from
    before); h = beta (s_chosen - s_rejected) - margin.  loss_type 'sigmoid' (with
    label_smoothing), 'robust', 'hinge' or 'ipo'; nll_coef adds the chosen side's mean
    negative log-likelihood.  pairs 'halves': the first half of the sequences are the
    chosen ones, the second half the rejected; 'interleaved': they alternate.  Pairs with a
    side without a counted token do not count.

    Returns (loss, rewards [B], dlogp): loss [1], or [B / 2] with reduction 'none'; rewards =
    beta s_i; dlogp times g_loss (fp32, loss's shape, None: 1).
    """
    if stream is not None:
        return _on(stream, flce_preference_loss, logp, ref_logp, ref_scores, mask, cu_seqlens,
                   beta, loss_type, label_smoothing, margin, length_normalised, nll_coef, pairs,
                   reduction, ignore_index, g_loss, need_loss, need_grad, validate, workspace)
    lib = B._lib or B.load_library()
    p, dev = preference_params(logp, ref_logp, ref_scores, mask, cu_seqlens, beta, loss_type,
                               label_smoothing, margin, length_normalised, nll_coef, pairs,
                               reduction, ignore_index, validate)
    if not need_loss and not need_grad:
        raise ValueError("neither the loss nor the gradient is wanted")
    n_seq = p.seqs.B
    n_out = n_seq // 2 if p.reduction == RED_NONE else 1
    _scalar_grad(g_loss, n_out, dev)
    ref = ctypes.byref(p)
    size = _size(lib, "preference", ref)
    loss = rewards = dlogp = None
    if need_loss:
        loss = torch.empty(n_out, dtype=torch.float32, device=dev)
        rewards = torch.empty(n_seq, dtype=torch.float32, device=dev)
    if need_grad:
        dlogp = torch.empty(logp.shape, dtype=logp.dtype, device=dev)
    ws = _workspace(size, dev, workspace)
    if n_out == 0 or (not need_loss and logp.numel() == 0):
        # no pair: nothing to compute
        return loss, rewards, None if dlogp is None else dlogp.zero_()
    code = lib.flce_preference_loss(
        ref, logp.data_ptr(), _addr(ref_logp), _addr(ref_scores), _addr(g_loss), _addr(loss),
        _addr(rewards), _addr(dlogp), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if code:
        B._check(code)
    return loss, rewards, dlogp


class _PreferenceLoss(torch.autograd.Function):
    """As _PolicyLoss; a loss per pair has an upstream gradient per pair, which the kernel
    spreads over the tokens."""

    @staticmethod
    def forward(ctx, logp, ref_logp, ref_scores, mask, cu_seqlens, kw):
        per_pair = reduction_code(kw["reduction"]) == RED_NONE
        ctx.formed = logp.dtype is torch.float32 and not per_pair
        loss, rewards, dlogp = flce_preference_loss(
            logp, ref_logp, ref_scores, mask, cu_seqlens,
            need_grad=ctx.formed and ctx.needs_input_grad[0], **kw)
        if ctx.formed:
            ctx.save_for_backward(dlogp)
        else:
            ctx.save_for_backward(logp, ref_logp, ref_scores, mask, cu_seqlens)
            ctx.kw = kw
        ctx.mark_non_differentiable(rewards)
        return loss if per_pair else loss[0], rewards

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, _g_rewards):
        if ctx.formed:
            return ctx.saved_tensors[0] * g_loss, None, None, None, None, None
        logp, ref_logp, ref_scores, mask, cu = ctx.saved_tensors
        _, _, dlogp = flce_preference_loss(logp, ref_logp, ref_scores, mask, cu,
                                           g_loss=_upstream(g_loss), need_loss=False, **ctx.kw)
        return dlogp, None, None, None, None, None


def preference_loss(logp, ref_logp=None, ref_scores=None, mask=None, cu_seqlens=None, beta=0.1,
                    loss_type="sigmoid", label_smoothing=0.0, margin=0.0,
                    length_normalised=False, nll_coef=0.0, pairs="halves", reduction="mean",
                    ignore_index=IGNORE_INDEX):
    """loss, rewards = preference_loss(logp, ref_logp, ...): flce_preference_loss as a
    differentiable function of logp (the other tensors are constants)."""
    kw = dict(beta=beta, loss_type=loss_type, label_smoothing=label_smoothing, margin=margin,
              length_normalised=length_normalised, nll_coef=nll_coef, pairs=pairs,
              reduction=reduction, ignore_index=ignore_index)
    return _PreferenceLoss.apply(logp, ref_logp, ref_scores, mask, cu_seqlens, kw)
