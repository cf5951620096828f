"""The gradient of the processed logits' log-probabilities keeps its digits whatever their size.

z is exact in every case (values of few bits, temperatures that are powers of two), so all that is lost is
lost behind it.  Tolerances: ln p = (z - m) - ln d is off by the rounding of z - lse (none within a
factor of two), of d (2^-22 of it, in all its sums) and of ln d; a probability by that and by the
exponential's 2^-22; together less than (8 + |ln p|) 2^-23 of itself.  The entropy behind its
gradient is off by as much as its terms, (8 + H) 2^-23.  A label's own g (1 - p) has the rounding of 1
and p, 2^-23 |g|, beside.
"""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu


def rows(size, V, temperature, seed=0):
    """Three rows: a likely label (about 0.9998), two likely columns, an even row; a label at an end."""
    g = torch.Generator().manual_seed(seed)
    z = size - 12 - torch.randint(0, 64, (3, V), generator=g).double() / 16
    at = V // 3
    z[0, at] = size
    z[1, at], z[1, V - 1] = size, size - 0.5
    z[2] = size - torch.randint(0, 16, (V,), generator=g).double() / 64
    x = (z * temperature).float()
    assert bool((x.double() == z * temperature).all())
    return x.cuda(), z.cuda(), torch.tensor([at, V - 1, 0]).cuda()


@pytest.mark.parametrize("V", [300, 1021, 40007])
@pytest.mark.parametrize("size,temperature", [(20.0, 1.0), (100.0, 1.0), (-100.0, 1.0), (3000.0, 1.0),
                                              (3200.0, 1 / 32), (30000.0, 0.25)])
def test_gradient(size, temperature, V):
    x, z, y = rows(size, V, temperature)
    gl, ge = torch.tensor([1.0, -0.7, 0.3], device="cuda"), torch.tensor([0.5, 1.0, -1.0], device="cuda")
    logq = torch.log_softmax(z, 1)
    p, H = logq.exp(), -(logq.exp() * logq).sum(1, keepdim=True)
    one = torch.zeros_like(z).scatter_(1, y[:, None], 1.0)
    a, b = gl.double()[:, None], ge.double()[:, None]
    want = (a * (one - p) - b * p * (logq + H)) / temperature
    off = (8 + logq.abs()) * 2.0 ** -23
    tol = p * off * (a.abs() + b.abs() * (logq + H).abs()) + b.abs() * p * (off + (8 + H) * 2.0 ** -23) \
        + one * a.abs() * 2.0 ** -23
    tol = tol / temperature + 2.0 ** -23 * want.abs() + 1e-37

    def check(d, what):
        err = (d.double() - want).abs()
        assert bool((err <= tol).all()), (what, float((err / tol).max()))

    leaf = x.clone().requires_grad_(True)
    logp, ent = flce.logits_logprob(leaf, y, temperature=temperature)
    check(torch.autograd.grad([logp, ent], [leaf], [gl, ge])[0], "autograd")
    assert bool(((logp.detach().double() - logq.gather(1, y[:, None])[:, 0]).abs()
                 <= off.gather(1, y[:, None])[:, 0]).all())
    logp, ent, lse = flce.flce_logits_logprob(x, y, temperature=temperature, split_lse=True)
    assert lse.shape == (2, 3)
    exact = torch.logsumexp(z, 1)
    assert bool((lse[1].abs() <= 2.0 ** -24 * lse[0].abs() * (1 + 2.0 ** -20)).all())
    assert bool(((lse.double().sum(0) - exact).abs() <= 2.0 ** -20 + 2.0 ** -45 * abs(size)).all())
    check(flce.flce_logits_logprob_backward(x, y, lse, ent, gl, ge, temperature=temperature), "split")
    # rows that begin anywhere, whose ends go element by element
    wide = torch.zeros(3, V + 3, device="cuda")
    for skew in (1, 2):
        v = wide[:, skew:skew + V]
        v.copy_(x)
        leaf = v.detach().requires_grad_(True)
        logp, ent = flce.logits_logprob(leaf, y, temperature=temperature)
        check(torch.autograd.grad([logp, ent], [leaf], [gl, ge])[0], skew)


def test_rows_without_an_lse():
    x = torch.randn(4, 50, device="cuda")
    x[1] = -float("inf")
    x[2, 3] = float("nan")
    x[3, 4] = float("inf")
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    _, ent, lse = flce.flce_logits_logprob(x, y, split_lse=True)
    plain = flce.flce_logits_logprob(x, y)[2]
    assert torch.equal(lse[0].nan_to_num(7, 8, 9), plain.nan_to_num(7, 8, 9))
    assert bool((lse[1, 1:] == 0).all())
    d = flce.flce_logits_logprob_backward(x, y, lse, ent, torch.ones(4, device="cuda"), torch.ones(4, device="cuda"))
    assert float(d[1].abs().max()) == 0 and bool(d[2:].isnan().all()) and bool(torch.isfinite(d[0]).all())
    empty = flce.flce_logits_logprob(x[:0], y[:0], split_lse=True)
    assert [t.shape for t in empty] == [(0,), (0,), (2, 0)]


def test_refusals():
    x, y = torch.zeros(4, 50, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    g = torch.ones(4, device="cuda")
    for lse in (torch.zeros(3, 4, device="cuda"), torch.zeros(2, 5, device="cuda"), torch.zeros(5, device="cuda"),
                torch.zeros(2, 4, device="cuda", dtype=torch.float64), torch.zeros(4, 2, device="cuda").t()):
        with pytest.raises(TypeError, match="lse"):
            flce.flce_logits_logprob_backward(x, y, lse, None, g, None)
