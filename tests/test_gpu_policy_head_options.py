"""The policy loss at the head with each of its options against the calls it joins: the same
kernels on the same values, so results are equal bit for bit."""
import pytest
import torch

from test_gpu_policy_loss import KW, _head_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


def two_calls(F, hidden, weight, labels, old, adv, ref, cu, layout, softcap, fp32, g, chunk_n, kw):
    nll, ent, _, _ = F.flce_forward(hidden, weight, labels, "none", softcap=softcap,
                                    weight_layout=layout)
    loss, stats, counts, dl, de = F.flce_policy_loss(0 - nll, old, adv, ref_logp=ref, entropy=ent,
                                                     mask=labels, cu_seqlens=cu, g_loss=g, **kw)
    dh, dw = F.flce_forward_backward(hidden, weight, labels, -dl, de, "none", softcap=softcap,
                                     weight_layout=layout, chunk_n=chunk_n, dhidden_fp32=fp32)[4:]
    return loss, stats, counts, 0 - nll, ent, dh, dw


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("g", [None, -2.5])
@pytest.mark.parametrize("chunk_n", [0, 512])
@pytest.mark.parametrize("per_token", [False, True])
def test_options(F, layout, softcap, fp32, g, chunk_n, per_token):
    N = 1300
    hidden, weight, labels, old, ref, adv, cu = _head_inputs(N=N, layout=layout)
    if per_token:
        adv = torch.randn(N, generator=torch.Generator().manual_seed(9)).cuda()
    up = None if g is None else torch.full((1,), g, device="cuda")
    kw = dict(KW, aggregate="seq_mean_token_mean")
    got = F.flce_policy_forward_backward(
        hidden, weight, labels, old, adv, ref_logp=ref, cu_seqlens=cu, weight_layout=layout,
        softcap=softcap, dhidden_fp32=fp32, g_loss=up, chunk_n=chunk_n, validate=True, **kw)
    want = two_calls(F, hidden, weight, labels, old, adv, ref, cu, layout, softcap, fp32, up,
                     chunk_n, kw)
    names = ("loss", "stats", "counts", "logp", "entropy", "dhidden", "dweight")
    for name, x, y in zip(names, got, want):
        assert x.dtype == y.dtype and torch.equal(x, y), name


def test_softcapped_head_against_the_definition(F):
    """Gradients within the head's bound of 1e-2 (dlogits and outputs are rounded to bf16)."""
    hidden, weight, labels, old, ref, adv, cu = _head_inputs()
    weight = weight * 4  # logits that the cap bends
    a, b = hidden.clone().requires_grad_(True), weight.clone().requires_grad_(True)
    kw = dict(clip_low=0.9, clip_high=50.0, kl_coef=0.02, entropy_coef=0.01, aggregate="token_mean")
    loss, _, _, _, _ = F.linear_policy_loss(a, b, labels, old, adv, ref_logp=ref, cu_seqlens=cu,
                                            softcap=5.0, **kw)
    got = torch.autograd.grad(loss * 3.0, (a, b))
    h, w = hidden.double().requires_grad_(True), weight.double().requires_grad_(True)
    z = 5.0 * torch.tanh(h @ w / 5.0)
    logq = torch.log_softmax(z, 1)
    m = labels != -100
    lp = logq.gather(1, labels.clamp(min=0)[:, None])[:, 0][m]
    ent = -(logq.exp() * logq).sum(1)[m]
    seq = torch.bucketize(torch.arange(len(m), device="cuda"), cu[1:].long(), right=True)
    d = (lp - old.double()[m]).clamp(-20, 20)
    A = adv.double()[seq][m]
    obj = torch.minimum(d.exp() * A, d.exp().clamp(0.1, 51.0) * A)
    e = (ref.double()[m] - lp).clamp(-20, 20)
    terms = -obj + 0.02 * (torch.expm1(e) - e) - 0.01 * ent
    want = terms.mean()
    grads = torch.autograd.grad(want * 3.0, (h, w))
    # log-probabilities within 1e-5 move a term by 1e-5 of its ratio's size at most
    assert abs(float(loss.detach()) - float(want.detach())) <= 2e-5 * float(terms.detach().abs().mean())
    for x, y in zip(got, grads):
        assert float((x.double() - y).norm() / y.norm()) <= 1e-2
