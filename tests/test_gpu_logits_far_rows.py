"""Rows of logits on both sides of an array's 2^31st element: what is read, written and differentiated there
is what the same rows alone give."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu
R, V = 9000, 256000  # row 8388 holds element 2^31
AT = [0, 1, 8387, 8388, 8389, 8390, 8999]


@pytest.fixture(scope="module")
def batch():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros(R, V, device="cuda", dtype=torch.bfloat16)
    x[AT] = (3 * torch.randn(len(AT), V, generator=g, device="cuda")).bfloat16()
    o = dict(tokens=torch.randint(0, V, (R, 40), generator=g, device="cuda"),
             lengths=torch.randint(0, 41, (R,), generator=g, device="cuda"),
             repetition_penalty=0.7 + torch.rand(R, generator=g, device="cuda"),
             presence_penalty=torch.rand(R, generator=g, device="cuda"),
             temperature=0.3 + torch.rand(R, generator=g, device="cuda"))
    yield x, o, {k: t[AT].contiguous() for k, t in o.items()}
    del x
    torch.cuda.empty_cache()


def test_processed(batch):
    x, o, few = batch
    rows = x[AT].clone()
    want, lse = flce.flce_process_logits(rows, need_lse=True, **few)
    assert not bool((want == rows).all(1).any())
    z, l = flce.flce_process_logits(x, need_lse=True, **o)
    assert torch.equal(z[AT], want)
    # blocks of a row join their sums in another order: tens of fp32 roundings of a logsumexp near 20
    assert bool(((l[AT] - lse).abs() <= 32 * 2.0 ** -24 * lse.abs()).all())
    assert torch.equal(x[AT], rows)  # nothing was written to
    # a row of zeros in between is changed by its penalties alone, and so is the last one before 2^31
    for r in (100, 8386, 8391):
        one = {k: t[r:r + 1].contiguous() for k, t in o.items()}
        assert torch.equal(z[r:r + 1], flce.flce_process_logits(torch.zeros_like(rows[:1]), **one))
    same = x.clone()
    del z
    assert flce.flce_process_logits(same, out=same, **o) is same
    assert torch.equal(same[AT], want)


def test_log_probabilities_and_gradient(batch):
    x, o, few = batch
    labels = torch.arange(R, device="cuda") * 28  # to the row's end
    ones = torch.ones(R, device="cuda")
    logp, ent, lse = flce.flce_logits_logprob(x, labels, split_lse=True, **o)
    y = labels[AT].contiguous()
    want = flce.flce_logits_logprob(x[AT].contiguous(), y, split_lse=True, **few)
    for a, b in zip((logp, ent, lse[0]), (want[0], want[1], want[2][0])):
        assert bool(((a[AT] - b).abs() <= 32 * 2.0 ** -24 * b.abs() + 1e-6).all())
    d = flce.flce_logits_logprob_backward(x, labels, lse, ent, ones, ones, **o)
    # with the same statistics the same bits
    part = flce.flce_logits_logprob_backward(x[AT].contiguous(), y, lse[:, AT].contiguous(), ent[AT].contiguous(),
                                             ones[AT].contiguous(), ones[AT].contiguous(), **few)
    assert torch.equal(d[AT], part) and bool((part.gather(1, y[:, None]) > 0).all())
