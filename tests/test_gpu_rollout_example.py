"""The dense layer, the processed logits, the policy loss and the optimizer as a run of them together
uses them: the example runs, its rollout and its scoring agree, and its gradients are those of the
same model in 64 bits."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_runs():
    import rollout_and_update as ex
    for loss, norm, apart in ex.main(rounds=2, quiet=True):
        assert math.isfinite(loss) and norm > 0
        # the two products of a bf16 state and table sum in another order where the tiles differ: a
        # bf16 rounding of a state (2^-8 of values below 4) times a table's row of 128 values of 0.3
        assert apart < 0.5


def test_gradients():
    import linear_cross_entropy_forward_gb300 as flce
    import rollout_and_update as ex

    g = torch.Generator().manual_seed(3)
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = (torch.randn(ex.V, ex.H, generator=g) * 0.3).bfloat16().cuda().requires_grad_(True)
    weight = (torch.randn(ex.H, ex.H, generator=g) / ex.H ** 0.5).bfloat16().cuda().requires_grad_(True)
    bias = (torch.randn(ex.H, generator=g) * 0.1).bfloat16().cuda().requires_grad_(True)
    allowed = ex.allowed_tokens("cuda")
    tokens, old = ex.rollout(torch.randint(0, ex.V, (ex.B, ex.PROMPT), generator=g).cuda(),
                             table, weight, bias, allowed, gen)
    assert bool((tokens[:, ex.PROMPT:] % 7 != 6).all()) and bool((tokens >= 0).all())
    adv = torch.randn(ex.B, generator=g).cuda()
    logp, ent = ex.score(tokens, table, weight, bias, allowed)
    loss, _, _ = flce.policy_loss(logp, old, adv, entropy=ent, entropy_coef=0.01)
    grads = torch.autograd.grad(loss.sum(), [table, weight, bias])

    # the same in 64 bits by autograd over the definitions
    T, W, b = (t.detach().double().requires_grad_(True) for t in (table, weight, bias))
    pairs = torch.stack([tokens[:, ex.PROMPT - 2:-2], tokens[:, ex.PROMPT - 1:-1]], 2).view(-1, 2)
    x = T[pairs[:, 1]] + T[pairs[:, 0]]
    logits = (x + torch.nn.functional.silu(x @ W.t() + b)) @ T.t()
    rows, n = [], logits.shape[0]
    ok = torch.arange(ex.V, device="cuda") % 7 != 6
    P = ex.PENALTIES
    for i in range(n):
        r, s = divmod(i, ex.NEW)
        seen = torch.bincount(tokens[r, :ex.PROMPT + s], minlength=ex.V) > 0
        made = torch.bincount(tokens[r, ex.PROMPT:ex.PROMPT + s], minlength=ex.V).double()
        z = logits[i]
        z = torch.where(seen, torch.where(z > 0, z / P["repetition_penalty"], z * P["repetition_penalty"]), z)
        z = z - P["frequency_penalty"] * made - P["presence_penalty"] * (made > 0)
        rows.append(torch.log_softmax(z.masked_fill(~ok, -math.inf) / P["temperature"], 0))
    logq = torch.stack(rows)
    lp = logq.gather(1, tokens[:, ex.PROMPT:].reshape(-1, 1)).view(ex.B, ex.NEW)
    H = -torch.where(ok, logq.exp() * logq.masked_fill(~ok, 0.0), torch.zeros_like(logq)).sum(1)
    ratio = (lp - old.double()).exp()
    a = adv.double()[:, None]
    per = -torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a) - 0.01 * H.view(ex.B, ex.NEW)
    want = torch.autograd.grad(per.mean(), [T, W, b])
    # states, dz and the gradients are bf16: a few roundings of 2^-8 along the way, some of the
    # clipped borders crossed by them
    for d, w in zip(grads, want):
        assert float((d.double() - w).norm() / w.norm()) < 0.1
    assert float((logp.double() - lp).abs().max()) < 0.5
