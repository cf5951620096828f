"""What an optimizer is told after it was made: the clipping norm and the loss scale of the next step, as
its learning rate."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu


def make(**kw):
    g = torch.Generator(device="cuda").manual_seed(1)
    ps = [torch.randn(n, generator=g, device="cuda").half() for n in (3000, 50)]
    gs = [torch.randn(n, generator=g, device="cuda").half() for n in (3000, 50)]
    return flce.AdamW(ps, betas=(0.0, 0.5), weight_decay=0.0, master=True, **kw), gs


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a.params + list(a.state_dict().values()),
                                                 b.params + list(b.state_dict().values())))


@pytest.mark.parametrize("bits", [32, 8])
def test_each_step_reads_them(bits):
    """Against optimizers that were made with the values, and hold the same states."""
    opt, gs = make(state_bits=bits)
    assert opt.step(gs) is None
    for max_norm, scale in ((0.5, 1.0), (0.25, 0.125), (None, 4.0), (8.0, 0.5), (None, 1.0)):
        other, _ = make(state_bits=bits, max_norm=max_norm, grad_scale=scale)
        for p, q in zip(other.params, opt.params):
            p.copy_(q)
        other.load_state_dict(opt.state_dict())
        opt.max_norm, opt.grad_scale = max_norm, scale
        got, want = opt.step(gs), other.step(gs)
        assert (got is None) == (max_norm is None) and (got is None or torch.equal(got, want))
        assert same(opt, other), (max_norm, scale)


def test_a_loss_scale_that_falls():
    opt, gs = make(skip_nonfinite=True, grad_scale=2.0 ** -10, lr=0.1)
    broken = [g.clone() for g in gs]
    broken[0][7] = float("inf")
    before = [p.clone() for p in opt.params]
    assert not bool(torch.isfinite(opt.step(broken)))
    assert all(torch.equal(p, q) for p, q in zip(opt.params, before)) and int(opt.step_count) == 0
    opt.grad_scale = 2.0 ** -9  # the next backward runs under half the loss scale
    exact = float(torch.cat(gs).double().norm()) / 512
    assert abs(float(opt.step(gs)) - exact) <= 1e-6 * exact and int(opt.step_count) == 1


def test_refusals():
    opt, gs = make()
    for bad in (0.0, -1.0, float("nan")):
        opt.max_norm = bad
        with pytest.raises(ValueError, match="max_norm"):
            opt.step(gs)
    opt.max_norm, opt.grad_scale = None, float("inf")
    with pytest.raises(flce.FlceError, match="BAD_ARG"):
        opt.step(gs)
    assert int(opt.step_count) == 0
