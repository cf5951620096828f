"""Positions and row strides past 32 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 4096


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    yield pkg
    torch.cuda.empty_cache()


def test_packed(F):
    """Two long sequences and a short one at the end of the axis, whose values alone are not zero:
    the ratios of the others are 1, their KL terms 0."""
    T, n = FAR + 5000, 777
    lp = torch.zeros(T, dtype=torch.bfloat16, device="cuda")
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    cu = torch.tensor([0, T // 2 + 13, T - n, T], device="cuda")
    tail = torch.linspace(-2.0, -0.25, n).to(torch.bfloat16)
    lp[T - n:] = tail.cuda()
    mask[T - n:T - n + 10] = False
    loss, _, counts, dlp, _ = F.flce_policy_loss(
        lp, None, torch.tensor([0.0, 0.0, 2.0], device="cuda"), mask=mask, cu_seqlens=cu,
        aggregate="seq_mean_token_mean", validate=True)
    # a ratio of 1 everywhere: -(0 + 0 + 2) / 3, and -2 / (3 (n - 10)) per token of the last
    assert abs(float(loss) + 2 / 3) <= 2.0 ** -22
    assert counts.tolist() == [T - 10, 3, 0, 0]
    want = torch.tensor(-2 / (3 * (n - 10)), dtype=torch.float64).to(torch.bfloat16).cuda()
    assert bool((dlp[T - n + 10:] == want).all()) and bool((dlp[T - n:T - n + 10] == 0).all())
    assert bool((dlp[:T - n] == 0).all())
    del dlp
    # the last two as a pair: h = 0.1 (0 - sum of the tail)
    pair = torch.tensor([0, T - n, T], device="cuda")
    loss, rewards, dlp = F.flce_preference_loss(lp, mask=mask, cu_seqlens=pair, validate=True)
    s = float(tail[10:].double().sum())
    h = -0.1 * s
    exact = torch.nn.functional.softplus(torch.tensor(-h, dtype=torch.float64))
    assert abs(float(loss) - float(exact)) <= 2.0 ** -19 * 0.1 * abs(s) + 1e-30
    assert float(rewards[0]) == 0 and abs(float(rewards[1]) - 0.1 * s) <= 2.0 ** -19 * 0.1 * abs(s)
    assert bool((dlp[:T - n] == dlp[0]).all()) and bool((dlp[T - n + 10:] == -dlp[0]).all())


def test_row_strides(F):
    """Three rows, each 2^30 elements or more behind the one before it."""
    S, ld = 3001, (1 << 30) + 3000
    lens = [(name, torch.empty(2 * ld + S, dtype=torch.bfloat16, device="cuda")) for name in "ab"]
    g = torch.Generator().manual_seed(2)
    small = [(-torch.rand(3, S, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    lp, old = (x.as_strided((3, S), (ld, 1)) for _, x in lens)
    lp.copy_(small[0])
    old.copy_(small[1])
    adv = torch.tensor([1.0, -1.0, 0.5], device="cuda")
    far = F.flce_policy_loss(lp, old, adv, ref_logp=old, kl_coef=0.1, validate=True)
    near = F.flce_policy_loss(small[0], small[1], adv, ref_logp=small[1], kl_coef=0.1, validate=True)
    for x, y in zip(far[:4], near[:4]):
        assert torch.equal(x, y)
    far = F.flce_preference_loss(lp[:2], old[:2], validate=True)
    near = F.flce_preference_loss(small[0][:2], small[1][:2], validate=True)
    for x, y in zip(far, near):
        assert torch.equal(x, y)
