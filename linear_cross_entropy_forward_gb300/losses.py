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

import contextlib
import ctypes

import torch

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


def _allocate_on(stream):
    """New tensors belong to the stream that the call runs on: memory of another stream's
    pool could still be in use there."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _rows(t, name, dtype, shape, device):
    """Checks one array of a batch; its row stride in elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    return t.stride(0) if len(shape) == 2 else 0


def _batch(logp, mask, cu_seqlens, ignore_index):
    """(FlceSeqs, device, number of sequences) of a batch laid out like logp."""
    if not isinstance(logp, torch.Tensor) or not logp.is_cuda:
        raise TypeError("logp must be a CUDA tensor")
    if logp.dtype not in _DTYPES:
        raise TypeError(f"logp must be float32, bfloat16 or float16, got {logp.dtype}")
    dev = B._on_current_device(logp)
    q = B.FlceSeqs()
    q.dtype = _DTYPES[logp.dtype]
    q.ignore_index = ignore_index
    shape = logp.shape
    if cu_seqlens is not None:
        if len(shape) != 1:
            raise ValueError("with cu_seqlens, logp must be 1-D")
        if not isinstance(cu_seqlens, torch.Tensor) or not cu_seqlens.is_cuda \
                or cu_seqlens.dtype not in (torch.int32, torch.int64):
            raise TypeError("cu_seqlens must be an int32 or int64 CUDA tensor")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous [B + 1] tensor")
        if cu_seqlens.device != dev:
            raise ValueError(f"cu_seqlens is on {cu_seqlens.device}, logp on {dev}")
        q.B, q.S = cu_seqlens.numel() - 1, shape[0]
        q.cu_kind = 1 if cu_seqlens.dtype == torch.int32 else 2
        q.cu_seqlens = cu_seqlens.data_ptr()
    elif len(shape) == 1:
        q.B, q.S = 1, shape[0]
    elif len(shape) == 2:
        q.B, q.S = shape
    else:
        raise ValueError(f"logp must be [B, S] or [T], got shape {tuple(shape)}")
    if mask is not None:
        if not isinstance(mask, torch.Tensor) \
                or mask.dtype not in (torch.bool, torch.uint8, torch.int64):
            raise TypeError("mask must be a bool, uint8 or int64 (labels) tensor")
        q.ld_mask = _rows(mask, "mask", mask.dtype, shape, dev)
        # an array of no elements has no address; the kind still needs one
        q.mask_kind = 2 if mask.dtype == torch.int64 else 1
        q.mask = mask.data_ptr() or 8
    return q, dev, q.B


def _check_cu(q):
    if q.cu_kind and not q.cu_seqlens:
        raise ValueError("cu_seqlens is empty")


def _scalar_grad(g, n, device):
    if g is None:
        return None
    B._need(g, "g_loss", torch.float32, (n,), device)
    return g


def policy_params(logp, old_logp=None, advantages=None, ref_logp=None, entropy=None, mask=None,
                  cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0,
                  kl="k3", entropy_coef=0.0, ratio="token", aggregate="token_mean", scale=1.0,
                  ignore_index=IGNORE_INDEX, validate=False):
    """(FlcePolicyParams, device) of a flce_policy_loss call, its tensors checked."""
    p = B.FlcePolicyParams()
    q, dev, n_seq = _batch(logp, mask, cu_seqlens, ignore_index)
    p.seqs = q
    shape, dt = logp.shape, logp.dtype
    p.ld_logp = _rows(logp, "logp", dt, shape, dev)
    if old_logp is not None:
        p.ld_old = _rows(old_logp, "old_logp", dt, shape, dev)
    if ref_logp is not None:
        p.ld_ref = _rows(ref_logp, "ref_logp", dt, shape, dev)
    elif kl_coef:
        raise ValueError("kl_coef needs ref_logp")
    if entropy is not None:
        p.ld_entropy = _rows(entropy, "entropy", dt, shape, dev)
    elif entropy_coef:
        raise ValueError("entropy_coef needs entropy")
    if not isinstance(advantages, torch.Tensor):
        raise TypeError("advantages must be a CUDA tensor")
    # one per sequence, unless the shape is the tokens' and that reading is the only one
    per_token = advantages.shape == shape and (ratio != "sequence") and not (
        advantages.dim() == 1 and n_seq == advantages.shape[0])
    p.adv_per_token = per_token
    p.ld_adv = _rows(advantages, "advantages", torch.float32, shape if per_token else
                     torch.Size((n_seq,)), dev)
    p.clip_low, p.clip_high, p.dual_clip = clip_low, clip_high, dual_clip
    p.kl_coef, p.entropy_coef, p.scale = kl_coef, entropy_coef, scale
    p.kl = _code(_KL, kl, "kl")
    p.ratio = _code(_RATIO, ratio, "ratio")
    p.aggregate = _code(_AGGREGATE, aggregate, "aggregate")
    p.validate = bool(validate)
    return p, dev


def _workspace(size, device, workspace):
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 \
            or not workspace.is_contiguous() or workspace.device != device:
        raise TypeError(f"workspace must be a contiguous uint8 tensor on {device}")
    if workspace.numel() < size:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; this call needs {size}")
    return workspace


def _size(lib, name, p):
    B._check(getattr(lib, f"flce_{name}_check_params")(ctypes.byref(p)))
    return getattr(lib, f"flce_{name}_workspace_size")(ctypes.byref(p))


def policy_workspace_size(params: "B.FlcePolicyParams") -> int:
    """Bytes of workspace a flce_policy_loss call with these parameters needs."""
    return int(_size(B.load_library(), "policy", params))


def _addr(t):
    return None if t is None else t.data_ptr()


def flce_policy_loss(logp, old_logp, advantages, ref_logp=None, entropy=None, mask=None,
                     cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0,
                     kl="k3", entropy_coef=0.0, ratio="token", aggregate="token_mean", scale=1.0,
                     ignore_index=IGNORE_INDEX, g_loss=None, need_loss=True, need_grad=True,
                     validate=False, workspace=None, stream=None):
    """Clipped policy loss and its gradients, in one launch.

    Per counted token, with d = logp - old_logp, r = exp(d) and A its advantage:
    -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) -- for A < 0 and dual_clip c > 1 at
    most -c A -- plus kl_coef K(logp, ref_logp) minus entropy_coef * entropy.  old_logp None:
    d = 0 (the policy itself).  kl: 'k1' logp - ref, 'k2' its half square, 'k3'
    exp(-k1) - 1 + k1.  Log-ratios are clamped to +-20, with zero gradient beyond.
    ratio 'sequence' takes the mean of d over each sequence's counted tokens.
    advantages: fp32 [B], one per sequence, or one per token (logp's shape).
    aggregate: 'token_mean', 'seq_mean_token_mean', 'seq_mean_token_sum', or 'sum' (times
    scale); sequences without a counted token do not count.

    Returns (loss [1], stats [4], counts [4], dlogp, dentropy).  stats: the aggregated
    policy term, mean KL to the reference, mean entropy, mean k3 to the old policy.
    counts (int64): counted tokens, sequences with one, clipped tokens (sequences),
    dual-clipped ones.  The gradients are times g_loss ([1] fp32, None: 1).  Parts that
    are not wanted (need_loss, need_grad; dentropy without entropy) are None.
    """
    lib = B.load_library()
    p, dev = policy_params(logp, old_logp, advantages, ref_logp, entropy, mask, cu_seqlens,
                           clip_low, clip_high, dual_clip, kl_coef, kl, entropy_coef, ratio,
                           aggregate, scale, ignore_index, validate)
    if not need_loss and not need_grad:
        raise ValueError("neither the loss nor the gradients are wanted")
    _scalar_grad(g_loss, 1, dev)
    size = _size(lib, "policy", p)
    loss = stats = counts = dlogp = dent = None
    with _allocate_on(stream):
        if need_loss:
            loss = torch.empty(1, dtype=torch.float32, device=dev)
            stats = torch.empty(4, dtype=torch.float32, device=dev)
            counts = torch.empty(4, dtype=torch.int64, device=dev)
        if need_grad:
            dlogp = torch.empty(logp.shape, dtype=logp.dtype, device=dev)
            if entropy is not None:
                dent = torch.empty(logp.shape, dtype=logp.dtype, device=dev)
        ws = _workspace(size, dev, workspace)
        if need_grad and not need_loss and logp.numel() == 0:
            return loss, stats, counts, dlogp, dent
        B._check(lib.flce_policy_loss(
            ctypes.byref(p), _addr(logp), _addr(old_logp), _addr(ref_logp), _addr(entropy),
            _addr(advantages), _addr(g_loss), _addr(loss), _addr(stats), _addr(counts),
            _addr(dlogp), _addr(dent), ws.data_ptr(), ws.numel(), B._stream(stream)))
    return loss, stats, counts, dlogp, dent


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, entropy, old_logp, advantages, ref_logp, mask, cu_seqlens, kw):
        loss, stats, counts, _, _ = flce_policy_loss(logp, old_logp, advantages, ref_logp,
                                                     entropy, mask, cu_seqlens, need_grad=False,
                                                     **kw)
        ctx.save_for_backward(logp, entropy, old_logp, advantages, ref_logp, mask, cu_seqlens)
        ctx.kw = kw
        ctx.mark_non_differentiable(stats, counts)
        return loss[0], stats, counts

    @staticmethod
    def backward(ctx, g_loss, _g_stats, _g_counts):
        logp, entropy, old_logp, advantages, ref_logp, mask, cu = ctx.saved_tensors
        g = g_loss.detach().reshape(1).to(torch.float32).contiguous()
        _, _, _, dlogp, dent = flce_policy_loss(logp, old_logp, advantages, ref_logp, entropy,
                                                mask, cu, g_loss=g, need_loss=False, **ctx.kw)
        return dlogp, dent, None, None, None, None, None, None


def policy_loss(logp, old_logp, advantages, ref_logp=None, entropy=None, mask=None,
                cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl="k3",
                entropy_coef=0.0, ratio="token", aggregate="token_mean", scale=1.0,
                ignore_index=IGNORE_INDEX):
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
              ignore_index=ignore_index)
    return _PolicyLoss.apply(logp, entropy, old_logp, advantages, ref_logp, mask, cu_seqlens, kw)


def flce_policy_forward_backward(hidden, weight, labels, old_logp, advantages, ref_logp=None,
                                 cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0,
                                 kl_coef=0.0, kl="k3", entropy_coef=0.0, ratio="token",
                                 aggregate="token_mean", scale=1.0, ignore_index=IGNORE_INDEX,
                                 softcap=0.0, weight_layout="hv", chunk_n=0, dhidden_fp32=False,
                                 g_loss=None, validate=False, workspace=None, stream=None):
    """The policy loss on top of the LM head, with dhidden and dweight, in one call.

    hidden [N, H], weight and labels as in flce_forward_backward; old_logp, ref_logp fp32 [N];
    advantages fp32 [B] or [N]; cu_seqlens [B + 1] cuts the N tokens into sequences (None:
    one).  Tokens whose label is ignore_index do not count.  ratio 'sequence' needs all
    tokens in one chunk (chunk_n >= N).
    Returns (loss [1], stats [4], counts [4], logp [N], entropy [N], dhidden, dweight);
    the gradients are times g_loss ([1] fp32, None: 1).
    """
    lib = B.load_library()
    N, H, V, wshape = B._dims(hidden, weight, weight_layout)
    B._need(hidden, "hidden", torch.bfloat16, (N, H))
    dev = B._on_current_device(hidden)
    B._need(weight, "weight", torch.bfloat16, wshape, dev)
    B._need(labels, "labels", torch.int64, (N,), dev)
    p = B.make_params(N, H, V, "none", ignore_index, 0.0, softcap, validate,
                      weight_layout=weight_layout, chunk_n=chunk_n, dhidden_fp32=dhidden_fp32)
    with _allocate_on(stream):
        logp = torch.empty(N, dtype=torch.float32, device=dev)
        entropy = torch.empty(N, dtype=torch.float32, device=dev)
        q, _ = policy_params(logp, old_logp, advantages, ref_logp, entropy, None, cu_seqlens,
                             clip_low, clip_high, dual_clip, kl_coef, kl, entropy_coef, ratio,
                             aggregate, scale, ignore_index, validate)
        _scalar_grad(g_loss, 1, dev)
        B._check(lib.flce_check_params(ctypes.byref(p)))
        _size(lib, "policy", q)
        size = lib.flce_policy_head_workspace_size(ctypes.byref(p), ctypes.byref(q))
        if size == 0:
            raise B.FlceError(1, "the head cannot take these parameters (a sequence ratio needs "
                                 "all tokens in one chunk)")
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        stats = torch.empty(4, dtype=torch.float32, device=dev)
        counts = torch.empty(4, dtype=torch.int64, device=dev)
        dh = torch.empty(N, H, dtype=torch.float32 if dhidden_fp32 else torch.bfloat16, device=dev)
        dw = torch.empty(wshape, dtype=torch.bfloat16, device=dev)
        ws = _workspace(size, dev, workspace)
        B._check(lib.flce_policy_forward_backward(
            ctypes.byref(p), ctypes.byref(q), _addr(hidden), _addr(weight), _addr(labels),
            _addr(old_logp), _addr(ref_logp), _addr(advantages), _addr(g_loss), _addr(loss),
            _addr(stats), _addr(counts), _addr(logp), _addr(entropy), _addr(dh), _addr(dw),
            ws.data_ptr(), ws.numel(), B._stream(stream)))
    return loss, stats, counts, logp, entropy, dh, dw


class _LinearPolicyLoss(torch.autograd.Function):
    """The gradients are formed in the forward, for an upstream gradient of 1, and scaled in
    the backward (a copy: the saved ones serve another backward pass)."""

    @staticmethod
    def forward(ctx, hidden, weight, labels, old_logp, advantages, ref_logp, cu_seqlens, kw):
        loss, stats, counts, logp, entropy, dh, dw = flce_policy_forward_backward(
            hidden, weight, labels, old_logp, advantages, ref_logp, cu_seqlens, **kw)
        ctx.save_for_backward(dh, dw)
        ctx.mark_non_differentiable(stats, counts, logp, entropy)
        return loss[0], stats, counts, logp, entropy

    @staticmethod
    def backward(ctx, g_loss, *_):
        dh, dw = ctx.saved_tensors
        g = g_loss.detach().reshape(1).to(torch.float32).contiguous()
        dh = B.flce_scale_bf16(dh.clone(), g) if ctx.needs_input_grad[0] else None
        dw = B.flce_scale_bf16(dw.clone(), g) if ctx.needs_input_grad[1] else None
        return dh, dw, None, None, None, None, None, None


def linear_policy_loss(hidden, weight, labels, old_logp, advantages, ref_logp=None,
                       cu_seqlens=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0,
                       kl="k3", entropy_coef=0.0, ratio="token", aggregate="token_mean",
                       scale=1.0, ignore_index=IGNORE_INDEX, softcap=0.0, weight_layout="hv",
                       chunk_n=0):
    """loss, stats, counts, logp, entropy = linear_policy_loss(hidden, weight, labels, ...)

    policy_loss(-nll, ...) of linear_cross_entropy's per-token nll and entropy, with the
    gradients by hidden and weight formed in the forward: the logits are computed once.
    Differentiable by hidden and weight through loss alone.
    """
    kw = dict(clip_low=clip_low, clip_high=clip_high, dual_clip=dual_clip, kl_coef=kl_coef, kl=kl,
              entropy_coef=entropy_coef, ratio=ratio, aggregate=aggregate, scale=scale,
              ignore_index=ignore_index, softcap=softcap, weight_layout=weight_layout,
              chunk_n=chunk_n)
    return _LinearPolicyLoss.apply(hidden, weight, labels, old_logp, advantages, ref_logp,
                                   cu_seqlens, kw)


def preference_params(logp, ref_logp=None, ref_scores=None, mask=None, cu_seqlens=None, beta=0.1,
                      loss_type="sigmoid", label_smoothing=0.0, margin=0.0,
                      length_normalised=False, nll_coef=0.0, pairs="halves", reduction="mean",
                      ignore_index=IGNORE_INDEX, validate=False):
    """(FlcePreferenceParams, device) of a flce_preference_loss call, its tensors checked."""
    p = B.FlcePreferenceParams()
    q, dev, n_seq = _batch(logp, mask, cu_seqlens, ignore_index)
    p.seqs = q
    if n_seq % 2:
        raise ValueError(f"pairs need an even number of sequences, got {n_seq}")
    p.ld_logp = _rows(logp, "logp", logp.dtype, logp.shape, dev)
    if ref_logp is not None:
        p.ld_ref = _rows(ref_logp, "ref_logp", logp.dtype, logp.shape, dev)
    if ref_scores is not None:
        B._need(ref_scores, "ref_scores", torch.float32, (n_seq,), dev)
    p.beta, p.margin, p.label_smoothing, p.nll_coef = beta, margin, label_smoothing, nll_coef
    p.kind = _code(_PREFERENCE, loss_type, "loss_type")
    p.length_normalised = bool(length_normalised)
    p.interleaved = _code(_PAIRS, pairs, "pairs")
    p.reduction = reduction_code(reduction)
    p.validate = bool(validate)
    return p, dev


def preference_workspace_size(params: "B.FlcePreferenceParams") -> int:
    """Bytes of workspace a flce_preference_loss call with these parameters needs."""
    return int(_size(B.load_library(), "preference", params))


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
    lib = B.load_library()
    p, dev = preference_params(logp, ref_logp, ref_scores, mask, cu_seqlens, beta, loss_type,
                               label_smoothing, margin, length_normalised, nll_coef, pairs,
                               reduction, ignore_index, validate)
    if not need_loss and not need_grad:
        raise ValueError("neither the loss nor the gradient is wanted")
    n_out = p.seqs.B // 2 if p.reduction == RED_NONE else 1
    _scalar_grad(g_loss, n_out, dev)
    size = _size(lib, "preference", p)
    loss = rewards = dlogp = None
    with _allocate_on(stream):
        if need_loss:
            loss = torch.empty(n_out, dtype=torch.float32, device=dev)
            rewards = torch.empty(p.seqs.B, dtype=torch.float32, device=dev)
        if need_grad:
            dlogp = torch.empty(logp.shape, dtype=logp.dtype, device=dev)
        ws = _workspace(size, dev, workspace)
        if p.seqs.B == 0 and n_out == 0 or (not need_loss and logp.numel() == 0):
            # no pair: nothing to compute
            return loss, rewards, None if dlogp is None else dlogp.zero_()
        B._check(lib.flce_preference_loss(
            ctypes.byref(p), _addr(logp), _addr(ref_logp), _addr(ref_scores), _addr(g_loss),
            _addr(loss), _addr(rewards), _addr(dlogp), ws.data_ptr(), ws.numel(),
            B._stream(stream)))
    return loss, rewards, dlogp


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, ref_logp, ref_scores, mask, cu_seqlens, kw):
        loss, rewards, _ = flce_preference_loss(logp, ref_logp, ref_scores, mask, cu_seqlens,
                                                need_grad=False, **kw)
        ctx.save_for_backward(logp, ref_logp, ref_scores, mask, cu_seqlens)
        ctx.kw = kw
        ctx.mark_non_differentiable(rewards)
        return loss if reduction_code(kw["reduction"]) == RED_NONE else loss[0], rewards

    @staticmethod
    def backward(ctx, g_loss, _g_rewards):
        logp, ref_logp, ref_scores, mask, cu = ctx.saved_tensors
        g = g_loss.detach().reshape(-1).to(torch.float32).contiguous()
        _, _, dlogp = flce_preference_loss(logp, ref_logp, ref_scores, mask, cu, g_loss=g,
                                           need_loss=False, **ctx.kw)
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
