"""A row of logits with a NaN or +inf left has NaN for its log-probability whatever its label: one that is
not allowed too, whose -inf would hide it."""
import math

import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [100, 5001, 70000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_labels(V, dtype):
    x = torch.randn(4, V, device="cuda").to(dtype)
    x[1, V - 2], x[2, V - 3] = float("nan"), float("inf")
    a = torch.ones(4, V, dtype=torch.bool, device="cuda")
    a[:, 7] = False
    a[3, :] = False
    y = torch.full((4,), 7, device="cuda")
    logp, ent, lse = flce.flce_logits_logprob(x, y, allowed=a)
    assert float(logp[0]) == -math.inf and float(logp[3]) == -math.inf  # nothing is wrong there
    assert bool(logp[1:3].isnan().all()) and bool(ent[1:3].isnan().all()) and bool(lse[1:3].isnan().all())
    # an ignored row stays 0, an unmasked label of the same rows is NaN
    assert float(flce.flce_logits_logprob(x, torch.full_like(y, -100), allowed=a)[0].abs().max()) == 0
    assert bool(flce.flce_logits_logprob(x, torch.full_like(y, 8), allowed=a)[0][1:3].isnan().all())
