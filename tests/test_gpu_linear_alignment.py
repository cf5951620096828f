"""Rows of a dense layer's odd widths that begin anywhere: the gradient behind a torch.cat over tokens, a
slice of a residual, a slice to write to.  The same values from an aligned address give the same
results bit for bit."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu


def make(M, K, N, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(N)
    x, w = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((M, K), (N, K)))
    return x, w, torch.randn(M, N, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("N", [1001, 1003, 5, 1])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_gradient_behind_a_cat(N, act, dtype):
    x, w, dy = make(40, 64, N, dtype)
    skew = []

    def run(before):
        leaves = [t.clone().requires_grad_(True) for t in (x, w)]
        y = flce.linear(*leaves, activation=act, weight_layout="vh", out_dtype=dtype)
        y.register_hook(lambda g: skew.append(g.data_ptr() % 16))
        rows = torch.cat([torch.zeros(before, N, device="cuda", dtype=dtype), y])
        return torch.autograd.grad(rows, leaves, torch.cat([torch.zeros_like(rows[:before]), dy]))

    want = run(0)
    for before in (1, 2, 3):
        assert all(torch.equal(a, b) for a, b in zip(run(before), want))
    assert any(skew), "no gradient here begins off a 16-byte boundary"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slices_of_a_residual_and_an_output(dtype):
    M, K, N = 40, 64, 1001
    x, w, r = make(M, K, N, dtype)
    args = dict(activation="gelu", weight_layout="vh", out_dtype=dtype)
    want = flce.flce_linear(x, w, residual=r, **args)
    big = torch.zeros(M + 4, N, device="cuda", dtype=dtype)
    for at in (1, 2, 3):
        big.zero_()
        big[at:at + M] = r
        res = big[at:at + M]
        assert res.data_ptr() % 16
        assert torch.equal(flce.flce_linear(x, w, residual=res, **args), want)
        # written over the residual itself, and beside it
        version = res._version
        assert flce.flce_linear(x, w, residual=res, out=res, **args) is res
        assert res._version > version
        assert torch.equal(res, want)
        assert float(big[:at].abs().max()) == 0 and float(big[at + M:].abs().max()) == 0
        out = torch.zeros(M + 4, N, device="cuda", dtype=dtype)
        y, z = flce.flce_linear(x, w, residual=r, out=out[at:at + M], need_preact=True, **args)
        assert torch.equal(out[at:at + M], want) and y.data_ptr() == out[at:at + M].data_ptr()
        leaf = r.clone().requires_grad_(True)
        y = flce.linear(x, w, None, "gelu", torch.cat([leaf[:at], leaf])[at:], "vh", dtype)
        y.float().sum().backward()
        assert bool((leaf.grad == 1).all())
    with pytest.raises(ValueError, match="out shares memory with residual"):
        flce.flce_linear(x, w, residual=big[1:M + 1], out=big[2:M + 2], **args)


def test_slices_of_what_the_gradients_read():
    M, K, N = 40, 64, 1001
    x, w, dy = make(M, K, N)
    z = torch.randn(M, N, device="cuda").bfloat16()
    want = flce.flce_linear_backward(dy, x, w, z, "silu", "vh")
    a, b = (torch.cat([t[:3], t])[3:] for t in (dy, z))
    assert a.data_ptr() % 16 and b.data_ptr() % 16
    got = flce.flce_linear_backward(a, x, w, b, "silu", "vh")
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    # x and weight are read in whole pieces
    with pytest.raises(flce.FlceError, match="ALIGN"):
        flce.flce_linear_backward(dy, torch.cat([x.flatten()[:1], x.flatten()])[1:].view(M, K), w, weight_layout="vh")
