"""A dense layer where no gradient will be asked for keeps nothing for one."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu


def peak(call):
    """Bytes that the call holds at most beyond what was there, and its result."""
    call()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    y = call()
    return torch.cuda.max_memory_allocated() - before, y


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_preactivation_is_kept(mode):
    M, K, N = 2048, 64, 1024
    x, w = torch.randn(M, K, device="cuda").bfloat16(), torch.randn(N, K, device="cuda").bfloat16()
    w.requires_grad_(True)
    size = 2 * M * N

    def call():
        return flce.linear(x, w, activation="silu", weight_layout="vh")

    held, with_gradient = peak(call)
    assert held >= 2 * size  # y and z
    with mode():
        held, y = peak(call)
    assert size <= held < size + (1 << 20)
    assert torch.equal(y, with_gradient) and not y.requires_grad
