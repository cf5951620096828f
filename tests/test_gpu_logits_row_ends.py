"""Processed logits do not depend on where a row begins: its ends that are no whole 16 bytes, worked off
element by element, give the same bits as the vectors between them."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [24, 1000])
@pytest.mark.parametrize("T", [200, 20000])
def test_any_beginning(V, T, dtype):
    R, n = 3, 40
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (3 * torch.randn(R, V, generator=g, device="cuda")).to(dtype)
    ends = torch.cat([torch.arange(0, 10), torch.arange(V - 10, V)]).cuda()
    ids = ends[torch.randint(0, 20, (R, n), generator=g, device="cuda")]  # most of them several times
    o = dict(bias_ids=ids, bias_values=3 * torch.randn(R, n, generator=g, device="cuda"),
             tokens=torch.randint(0, V, (R, T), generator=g, device="cuda"),
             prompt_lens=torch.full((R,), T // 2, device="cuda"), repetition_penalty=1.3,
             frequency_penalty=0.01, presence_penalty=0.3, temperature=0.7, out_dtype=torch.float32)
    want = flce.flce_process_logits(x, **o)
    for skew in range(1, 8):
        buf = torch.zeros(R, V + 9, device="cuda", dtype=dtype)
        buf[:, skew:skew + V] = x
        assert torch.equal(flce.flce_process_logits(buf[:, skew:skew + V], **o), want), skew
