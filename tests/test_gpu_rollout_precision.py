"""The rollout example's scores and gradients against 64 bits that round where the model does: states and
layers' outputs to bf16, and nothing else.

Tolerances.  Behind the same bf16 states a log-probability is off by fp32's roundings, 16 * 2^-24 of the
logits' size (below 64), twice: 1.3e-4.  A state whose 64-bit and fp32 sums fall on either side of a
rounding's border is a step of 2^-7 of itself apart; that is rare (one element in thousands), so the median has none of
it, and a few of them, each times a row of the table, stay below 0.05.  A gradient passes at most six
roundings to bf16 on its way (of the head's product, dz, dx, the sum of a state's two parts, the lookup's
and the head's sum), 2^-8 of the value each at most: 0.024 by 2-norm.
"""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def bf16(x):
    """x rounded, with the gradient of x."""
    return x + (x.detach().float().bfloat16().double() - x.detach())


@pytest.mark.parametrize("seed", [3])
def test_scores_and_gradients(seed):
    import linear_cross_entropy_forward_gb300 as flce
    import rollout_and_update as ex

    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table = (torch.randn(ex.V, ex.H, generator=g) * 0.3).bfloat16().cuda().requires_grad_(True)
    weight = (torch.randn(ex.H, ex.H, generator=g) / ex.H ** 0.5).bfloat16().cuda().requires_grad_(True)
    bias = (torch.randn(ex.H, generator=g) * 0.1).bfloat16().cuda().requires_grad_(True)
    allowed = ex.allowed_tokens("cuda")
    tokens, _ = ex.rollout(torch.randint(0, ex.V, (ex.B, ex.PROMPT), generator=g).cuda(),
                           table, weight, bias, allowed, gen)
    logp, ent = ex.score(tokens, table, weight, bias, allowed)
    adv = torch.randn(ex.B, generator=g).cuda()
    loss, _, _ = flce.policy_loss(logp, logp.detach(), adv, entropy=ent, entropy_coef=0.01)
    grads = torch.autograd.grad(loss.sum(), [table, weight, bias])

    T, W, b = (t.detach().double().requires_grad_(True) for t in (table, weight, bias))
    x = bf16(T[tokens[:, ex.PROMPT - 1:-1]] + T[tokens[:, ex.PROMPT - 2:-2]]).reshape(-1, ex.H)
    h = bf16(x + torch.nn.functional.silu(x @ W.t() + b))
    z, P, n = h @ T.t(), ex.PENALTIES, ex.B * ex.NEW
    made, seen = torch.zeros(2, n, ex.V, dtype=torch.float64, device="cuda").unbind(0)
    for i in range(n):
        r, s = divmod(i, ex.NEW)
        made[i] = torch.bincount(tokens[r, ex.PROMPT:ex.PROMPT + s], minlength=ex.V)
        seen[i] = torch.bincount(tokens[r, :ex.PROMPT + s], minlength=ex.V)
    z = torch.where(seen > 0, torch.where(z > 0, z / P["repetition_penalty"], z * P["repetition_penalty"]), z)
    z = z - P["frequency_penalty"] * made - P["presence_penalty"] * (made > 0)
    ok = torch.arange(ex.V, device="cuda") % 7 != 6
    logq = torch.log_softmax(z.masked_fill(~ok, -math.inf) / P["temperature"], 1)
    lp = logq.gather(1, tokens[:, ex.PROMPT:].reshape(-1, 1)).view(ex.B, ex.NEW)
    H = -torch.where(ok, logq.exp() * logq.masked_fill(~ok, 0.0), torch.zeros_like(logq)).sum(1)
    assert float(z.detach()[:, ok].abs().max()) < 64
    off = (logp.detach().double() - lp.detach()).abs()
    assert float(off.median()) < 1.3e-4 and float(off.max()) < 0.05
    ratio = (lp - lp.detach()).exp()
    per = -ratio * adv.double()[:, None] - 0.01 * H.view(ex.B, ex.NEW)  # at a ratio of 1 nothing is clipped
    want = torch.autograd.grad(per.mean(), [T, W, b])
    for name, d, w in zip(("table", "weight", "bias"), grads, want):
        assert float((d.double() - w).norm() / w.norm()) < 6 * 2.0 ** -8, name
