"""What the log-probabilities' call returns are tensors of the caller's own, to be changed in place."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu


def test_log_probabilities_changed_in_place():
    x, y = torch.randn(5, 300, device="cuda"), torch.arange(5, device="cuda")
    want = []
    for place in (False, True):
        leaf = x.clone().requires_grad_(True)
        logp, ent = flce.logits_logprob(leaf, y)
        if place:
            logp.sub_(1.0).mul_(2.0)  # the difference to a reference's, say
        else:
            logp = (logp - 1.0) * 2.0
        (logp.sum() + ent.sum()).backward()
        want.append(leaf.grad)
    assert torch.equal(*want)
    # the entropy is what its gradient takes: changed in place, it is missed
    leaf = x.clone().requires_grad_(True)
    logp, ent = flce.logits_logprob(leaf, y)
    ent.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (logp.sum() + ent.sum()).backward()


def test_outputs_share_no_memory():
    x, y = torch.randn(5, 300, device="cuda"), torch.arange(5, device="cuda")
    outs = flce.flce_logits_logprob(x, y)
    assert len({t.untyped_storage().data_ptr() for t in outs}) == 3
    before = outs[1]._version
    outs[0].zero_()
    assert outs[1]._version == before
