"""padding_idx: what is refused, and when."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


@pytest.mark.parametrize("padding,err", [(-1, ValueError), (-10, ValueError), (10, "flce"),
                                         (1 << 40, "flce")])
def test_refused_in_the_forward_as_in_the_backward(F, padding, err):
    ids, w = torch.zeros(5, dtype=torch.int64).cuda(), torch.ones(10, 8).cuda().requires_grad_(True)
    kind = F.FlceError if err == "flce" else err
    with pytest.raises(kind):
        F.embedding(ids, w, padding_idx=padding)
    with pytest.raises(kind):
        F.flce_embedding_backward(torch.ones(5, 8).cuda(), ids, 10, padding_idx=padding)


def test_a_row_of_another_shard_is_taken(F):
    ids = torch.tensor([3, 12, 12, 17]).cuda()
    w = torch.ones(10, 8).cuda().requires_grad_(True)
    for padding, rows in ((None, [2, 7]), (12, [7]), (3, [2, 7]), (19, [2, 7])):
        out = F.embedding(ids, w, padding_idx=padding, v_offset=10, v_total=20)
        (g,) = torch.autograd.grad(out.sum(), w)
        assert g.abs().sum(1).nonzero().flatten().tolist() == rows
