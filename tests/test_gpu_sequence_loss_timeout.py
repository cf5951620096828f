"""The wait between the blocks of the losses over sequences, with a sequence that never comes: it
ends after its limit of 2 s, is reported, and leaves no result that could be taken for one."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

FLCE_ERR_TIMEOUT = 6


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


def f32(*shape):
    return torch.full(shape, 7.0, device="cuda")


def mask_of(shape):
    return torch.rand(shape, generator=torch.Generator().manual_seed(1)).lt(0.7).cuda()


def test_policy(F):
    """Padded: 600 pieces, a grid."""
    lib = F.load_library()
    lp, adv, mask = f32(300, 500), f32(300), mask_of((300, 500))
    p, _ = F.policy_params(lp, None, adv, mask=mask)
    ws = torch.empty(F.policy_workspace_size(p), dtype=torch.uint8, device="cuda")
    loss, stats, dlp = f32(1), f32(4), f32(300, 500)
    counts = torch.zeros(4, dtype=torch.int64, device="cuda")
    code = lib.flce_selftest_policy_timeout(
        ctypes.byref(p), lp.data_ptr(), adv.data_ptr(), loss.data_ptr(), stats.data_ptr(),
        counts.data_ptr(), dlp.data_ptr(), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert F.flce_status(ws) == FLCE_ERR_TIMEOUT
    assert bool(loss.isnan().all()) and bool(stats.isnan().all())
    assert bool(dlp[mask].isnan().all()) and bool((dlp[~mask] == 0).all())
    # the context is usable, and so is the workspace
    again = F.flce_policy_loss(lp, None, adv, mask=mask, workspace=ws)
    assert F.flce_status(ws) == 0
    assert float(again[0]) == -7.0 and not bool(again[3].isnan().any())


@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_preference(F, reduction):
    """Packed: 400 tokens each of 300 sequences, a grid."""
    lib = F.load_library()
    lp, mask = f32(120000), mask_of((120000,))
    cu = torch.arange(0, 120001, 400, dtype=torch.int32).cuda()
    p, _ = F.preference_params(lp, mask=mask, cu_seqlens=cu, reduction=reduction)
    ws = torch.empty(F.preference_workspace_size(p), dtype=torch.uint8, device="cuda")
    loss, rewards, dlp = f32(150 if reduction == "none" else 1), f32(300), f32(120000)
    code = lib.flce_selftest_preference_timeout(
        ctypes.byref(p), lp.data_ptr(), loss.data_ptr(), rewards.data_ptr(), dlp.data_ptr(),
        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert F.flce_status(ws) == FLCE_ERR_TIMEOUT
    assert bool(loss.isnan().all())
    assert bool(dlp[mask].isnan().all()) and bool((dlp[~mask] == 0).all())
    F.flce_preference_loss(lp, mask=mask, cu_seqlens=cu, reduction=reduction, workspace=ws)
    assert F.flce_status(ws) == 0
