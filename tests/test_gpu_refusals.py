"""What the Python calls of the sequence losses and the embedding refuse, with CUDA tensors:
each refusal comes before anything is launched."""
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


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_losses(F):
    x, a = z(4, 10), z(4)
    cu = torch.tensor([0, 5, 10], dtype=torch.int32).cuda()
    p, q = F.flce_policy_loss, F.flce_preference_loss
    for err, call in [
            (TypeError, lambda: p(x.double(), x, a)), (TypeError, lambda: p(x, x.half(), a)),
            (TypeError, lambda: p(x, x, a.double())), (TypeError, lambda: p(x, x, None)),
            (TypeError, lambda: p(x, x.cpu(), a)), (TypeError, lambda: p(x, x, a, mask=z(4, 10))),
            (TypeError, lambda: p(z(10), None, z(2), cu_seqlens=cu.float())),
            (TypeError, lambda: p(x, x, a, g_loss=z(1).half())),
            (TypeError, lambda: p(x, x, a, workspace=z(10))),
            (ValueError, lambda: p(x, z(4, 9), a)), (ValueError, lambda: p(x, x, z(3))),
            (ValueError, lambda: p(x, x, a, mask=z(4, 9, dtype=torch.bool))),
            (ValueError, lambda: p(x, x, a, kl_coef=0.1)),
            (ValueError, lambda: p(x, x, a, entropy_coef=0.1)),
            (ValueError, lambda: p(x, x, a, kl="kl")),
            (ValueError, lambda: p(x, x, a, aggregate="mean")),
            (ValueError, lambda: p(x, x, x, ratio="sequence")),
            (ValueError, lambda: p(z(10, 4).t(), x, a)), (ValueError, lambda: p(x, z(10, 4).t(), a)),
            (ValueError, lambda: p(z(2, 2, 2), None, a)),
            (ValueError, lambda: p(x, x, a, cu_seqlens=cu)),
            (ValueError, lambda: p(z(10), None, z(2), cu_seqlens=cu.view(1, 3))),
            (ValueError, lambda: p(x, x, z(8)[::2])),
            (ValueError, lambda: p(x, x, a, g_loss=z(2))),
            (ValueError, lambda: p(x, x, a, need_loss=False, need_grad=False)),
            (ValueError, lambda: p(x, x, a, workspace=z(10, dtype=torch.uint8))),
            (F.FlceError, lambda: p(x, x, a, clip_low=1.0)),
            (F.FlceError, lambda: p(x, x, a, dual_clip=0.5)),
            (TypeError, lambda: q(x, ref_scores=a.half())), (ValueError, lambda: q(z(3, 10))),
            (ValueError, lambda: q(x, z(4, 9))), (ValueError, lambda: q(x, ref_scores=z(3))),
            (ValueError, lambda: q(x, pairs="pairs")), (ValueError, lambda: q(x, loss_type="x")),
            (ValueError, lambda: q(x, reduction="x")), (ValueError, lambda: q(x, g_loss=z(2))),
            (F.FlceError, lambda: q(x, beta=0.0)),
            (F.FlceError, lambda: q(x, loss_type="hinge", label_smoothing=0.1))]:
        with pytest.raises(err):
            call()


def test_embedding(F):
    ids, w = torch.zeros(5, dtype=torch.int64, device="cuda"), z(7, 8)
    f, b = F.flce_embedding, F.flce_embedding_backward
    for err, call in [
            (TypeError, lambda: f(ids.float(), w)), (TypeError, lambda: f(ids, w.double())),
            (TypeError, lambda: f(ids.cpu(), w)), (TypeError, lambda: f(ids, w.cpu())),
            (TypeError, lambda: f(ids, None)), (ValueError, lambda: f(ids, z(7))),
            (ValueError, lambda: f(ids, z(8, 7).t())),
            (ValueError, lambda: f(torch.zeros(10, dtype=torch.int64, device="cuda")[::2], w)),
            (ValueError, lambda: f(ids, w, out=z(5, 7))), (F.FlceError, lambda: f(ids, w, v_offset=3)),
            (F.FlceError, lambda: f(ids, w, float("nan"))),
            (TypeError, lambda: b(z(5, 8).double(), ids, 7)), (ValueError, lambda: b(z(4, 8), ids, 7)),
            (ValueError, lambda: b(z(8, 5).t(), ids, 7)),
            (ValueError, lambda: b(z(5, 8), ids, 7, accumulate=True)),
            (ValueError, lambda: b(z(5, 8), ids, 7, dweight=z(6, 8))),
            (TypeError, lambda: b(z(5, 8), ids, 7, dweight=z(7, 8).half())),
            (TypeError, lambda: b(z(5, 8).half(), ids, 7, grad_dtype=torch.bfloat16)),
            (F.FlceError, lambda: b(z(5, 8), ids, 7, padding_idx=7)),
            (ValueError, lambda: b(z(5, 8), ids, 7, workspace=z(8, dtype=torch.uint8)))]:
        with pytest.raises(err):
            call()
