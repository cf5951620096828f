"""Edges of the losses over sequences.  Tolerances are those that test_gpu_policy_loss.py derives,
where nothing else is said."""
import math
import threading

import pytest
import torch

from test_gpu_policy_loss import KW, check, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


def round_tokens():
    """Tokens of which every warp of the GPU takes one piece."""
    return torch.cuda.get_device_properties(0).multi_processor_count * 32 * 256


def test_threads_whose_launches_keep_different_amounts(F):
    """Two and four pieces per warp, whose gradients wait in shared memory of different sizes."""
    per = round_tokens()
    wrong = []

    def work(rounds):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                lp = torch.zeros(int((rounds - 0.5) * per), device="cuda")
                adv = torch.ones(1, device="cuda")
                p, _ = F.policy_params(lp, None, adv)
                ws = torch.empty(F.policy_workspace_size(p), dtype=torch.uint8, device="cuda")
                for k in range(1500):
                    out = F.flce_policy_loss(lp, None, adv, workspace=ws)
                    if k % 16 == 15:
                        s.synchronize()
                if float(out[0]) != -1.0:
                    wrong.append(float(out[0]))
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(r,)) for r in (2, 4, 3, 4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


BAD_OFFSETS = [[0, 5000, 100, 5100], [0, 50, 6000], [-5, 50, 5100], [5100, 0], [0, 2000, 1000, 5100]]


def stale(*shape, dtype=torch.float32):
    """Leaves 7s in memory that the next tensor of this size is likely to get."""
    for _ in range(4):
        torch.full(shape, 7.0, dtype=dtype, device="cuda")


@pytest.mark.parametrize("cu", BAD_OFFSETS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_offsets_out_of_order_leave_no_result(F, cu, dtype):
    """Neither a finite one nor what the memory held before."""
    T = 5100
    x, ent = torch.zeros(T, dtype=dtype).cuda(), torch.ones(T, dtype=dtype).cuda()
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    adv = torch.ones(len(cu) - 1).cuda()
    stale(T, dtype=dtype)
    loss, stats, _, dl, de = F.flce_policy_loss(x, x, adv, entropy=ent, entropy_coef=0.1, cu_seqlens=c)
    for t in (loss, stats, dl, de):
        assert bool(t.isnan().all())
    g = torch.ones(1).cuda()
    dl = F.flce_policy_loss(x, x, adv, cu_seqlens=c, g_loss=g, need_loss=False)[3]
    assert bool(dl.isnan().all())
    if len(adv) % 2 == 0:
        stale(T, dtype=dtype)
        for reduction in ("mean", "none"):
            loss, rewards, dl = F.flce_preference_loss(x, cu_seqlens=c, reduction=reduction)
            for t in (loss, rewards, dl):
                assert bool(t.isnan().all())


@pytest.mark.parametrize("chunk_n", [0, 512])
def test_offsets_out_of_order_leave_no_result_of_the_head(F, chunk_n):
    N, H, V = 1300, 64, 512
    g = torch.Generator().manual_seed(3)
    hidden = torch.randn(N, H, generator=g).to(torch.bfloat16).cuda()
    weight = torch.randn(H, V, generator=g).to(torch.bfloat16).cuda()
    labels = torch.randint(0, V, (N,), generator=g).cuda()
    c = torch.tensor([0, 1300, 10, 1300], dtype=torch.int64).cuda()
    loss, stats, _, _, _, dh, dw = F.flce_policy_forward_backward(
        hidden, weight, labels, torch.zeros(N).cuda(), torch.ones(3).cuda(), cu_seqlens=c,
        chunk_n=chunk_n)
    for t in (loss, stats, dh, dw):
        assert bool(t.isnan().all())


@pytest.mark.parametrize("n", [1, 2, 4, 7, 300, 1025])
def test_sequence_ratios_at_the_borders(F, n):
    """Means of log-ratios that lie within rounding of a border: logp is the border's fp32 value,
    old_logp the few bits that the border has beyond it, a little more or less."""
    spans, lps, olds, advs = [], [], [], []
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=3.0, ratio="sequence")
    for border, a in ((math.log1p(0.28), 1.0), (math.log1p(-0.2), -1.0), (math.log(3.0), -1.0)):
        h = torch.tensor(border, dtype=torch.float32)
        low = border - float(h)
        for off in (0.5, 0.9, 1.1, 1.5, -0.5, 2.5):
            spans.append((len(lps), len(lps) + n))
            lps += [float(h)] * n
            olds += [-low * off] * n
            advs.append(a)
    lp, old, adv = (torch.tensor(v, dtype=torch.float32) for v in (lps, olds, advs))
    mask = torch.ones(len(lps), dtype=torch.bool)
    cu = torch.arange(0, len(lps) + 1, n, dtype=torch.int32)
    got = F.flce_policy_loss(lp.cuda(), old.cuda(), adv.cuda(), cu_seqlens=cu.cuda(), **kw)
    want = reference(lp.double(), old.double(), None, None, adv.repeat_interleave(n).double(), mask,
                     spans, kw)
    assert 0 < want[2][2] and 0 < want[2][3]
    check(want, *got[:4], None, torch.float32)


@pytest.mark.parametrize("kw,a,d", [(dict(clip_high=1e9), 1.0, 25.0),
                                    (dict(clip_low=1 - 1e-10), -1.0, -25.0),
                                    (dict(dual_clip=1e9), -1.0, 25.0),
                                    (dict(clip_high=1e9, dual_clip=2e9), -1.0, 25.0),
                                    (dict(clip_high=4e8), 1.0, 25.0),
                                    (dict(clip_low=1 - 1e-8), -1.0, -25.0),
                                    (dict(dual_clip=4e8), -1.0, 25.0),
                                    (dict(clip_high=math.inf), 1.0, math.inf)])
@pytest.mark.parametrize("ratio", ["token", "sequence"])
def test_borders_beyond_the_clamp(F, kw, a, d, ratio):
    """The definition itself: r is the exponential of the clamped log-ratio, and the objective is
    clipped where clip(r) makes it smaller.  A ratio of e^20 in fp32 is off by a few steps of
    expf, as the tolerance of 2^-19 covers."""
    lp = torch.tensor([0.0, d], dtype=torch.float32)
    lo, hi, c = kw.get("clip_low", 0.2), kw.get("clip_high", 0.2), kw.get("dual_clip", 0.0)
    want, clipped, dual = 0.0, 0, 0
    for x in lp.tolist():
        r = math.exp(max(-20.0, min(20.0, x)))
        rc = max(1 - lo, min(1 + hi, r))
        obj = min(r * a, rc * a)
        clipped += rc * a < r * a
        if c and a < 0 and c * a > obj:
            obj, dual = c * a, dual + 1
        want -= obj
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    adv = torch.full((2,), a).cuda()
    loss, _, counts, dl, _ = F.flce_policy_loss(lp.cuda(), torch.zeros(2).cuda(), adv, cu_seqlens=cu,
                                                aggregate="sum", ratio=ratio, **kw)
    assert abs(float(loss) - want) <= 2.0 ** -19 * abs(want)
    assert counts.tolist() == [2, 2, clipped, dual]
    assert dl.tolist() == [-a, 0.0]


def test_advantages_of_as_many_sequences_as_tokens(F):
    """A packed batch of three sequences, two of them empty, with three tokens: an advantage per
    token has the shape of one per sequence, and the call says which it is."""
    lp, old, ref, ent, adv, mask = make([0, 3, 0], 3, adv_token=True, mask_rate=1.0)
    cu = torch.tensor([0, 0, 3, 3], dtype=torch.int32).cuda()
    for per_token, a in ((True, adv), (False, adv[[1, 1, 1]]), (None, adv[[1, 1, 1]])):
        got = F.flce_policy_loss(lp.cuda(), old.cuda(), adv.cuda(), cu_seqlens=cu,
                                 adv_per_token=per_token)
        want = reference(lp.double(), old.double(), None, None, a.double(), mask, [(0, 3)], {})
        check(want, *got[:4], None, torch.float32)
        x = lp.cuda().requires_grad_(True)
        loss = F.policy_loss(x, old.cuda(), adv.cuda(), cu_seqlens=cu, adv_per_token=per_token)[0]
        assert torch.equal(loss.detach(), got[0][0])
    with pytest.raises(ValueError, match="advantages"):
        F.flce_policy_loss(lp.cuda(), old.cuda(), adv.cuda()[:2], cu_seqlens=cu, adv_per_token=True)
    with pytest.raises(ValueError, match="advantages"):
        F.flce_policy_loss(lp.cuda().view(1, 3), None, adv.cuda().view(1, 3), adv_per_token=False)
    with pytest.raises(F.FlceError):
        F.flce_policy_loss(lp.cuda(), old.cuda(), adv.cuda(), cu_seqlens=cu, ratio="sequence",
                           adv_per_token=True)


def test_advantages_of_as_many_sequences_as_tokens_at_the_head(F):
    g = torch.Generator().manual_seed(4)
    hidden = torch.randn(3, 64, generator=g).to(torch.bfloat16).cuda()
    weight = torch.randn(64, 512, generator=g).to(torch.bfloat16).cuda()
    labels = torch.randint(0, 512, (3,), generator=g).cuda()
    adv, old = torch.tensor([1.0, -2.0, 3.0]).cuda(), torch.zeros(3).cuda()
    cu = torch.tensor([0, 0, 3, 3], dtype=torch.int32).cuda()
    for per_token in (True, False, None):
        got = F.flce_policy_forward_backward(hidden, weight, labels, old, adv, cu_seqlens=cu,
                                             adv_per_token=per_token)
        want = F.flce_policy_loss(got[3], old, adv, mask=labels, cu_seqlens=cu,
                                  adv_per_token=per_token)
        auto = F.linear_policy_loss(hidden, weight, labels, old, adv, cu_seqlens=cu,
                                    adv_per_token=per_token)
        assert torch.equal(got[0], want[0]) and torch.equal(auto[0], want[0][0])


def test_no_sequences_at_all(F):
    """Tokens that no sequence owns: nothing counts."""
    x = torch.zeros(300).cuda()
    cu = torch.zeros(1, dtype=torch.int32).cuda()
    loss, stats, counts, dl, de = F.flce_policy_loss(x, x, torch.empty(0).cuda(), entropy=x,
                                                     entropy_coef=0.1, cu_seqlens=cu, validate=True)
    assert float(loss) == 0 and stats.tolist() == [0] * 4 and counts.tolist() == [0] * 4
    assert bool((dl == 0).all()) and bool((de == 0).all())
    loss, rewards, dl = F.flce_preference_loss(x, cu_seqlens=cu, validate=True)
    assert float(loss) == 0 and rewards.numel() == 0 and bool((dl == 0).all())
    w = torch.zeros(64, 128, dtype=torch.bfloat16).cuda()
    h = torch.ones(10, 64, dtype=torch.bfloat16).cuda()
    got = F.flce_policy_forward_backward(h, w, torch.zeros(10, dtype=torch.int64).cuda(), x[:10],
                                         torch.empty(0).cuda(), cu_seqlens=cu, validate=True)
    assert float(got[0]) == 0 and got[2].tolist() == [0] * 4
    assert bool((got[5] == 0).all()) and bool((got[6] == 0).all())


@pytest.mark.parametrize("ratio", ["token", "sequence"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rounds", [3.4, 4.5])
def test_several_pieces_per_warp(F, ratio, dtype, rounds):
    """Three and four pieces per warp whose gradients are kept; beyond four, kept and recomputed
    ones in one launch."""
    per = round_tokens()
    lens = [int(1.2 * per) + 7, 5, int((rounds - 1.3) * per) + 13, int(0.1 * per)]
    run(F, lens, seed=int(10 * rounds), dtype=dtype,
        kw=dict(KW, ratio=ratio, aggregate="seq_mean_token_mean"))
