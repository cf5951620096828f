"""The preference loss against a plain loop over pairs in 64 bits.

Tolerances.  A sequence's score is a sum over tokens of fp32 differences (half a step each)
added in fp32 or wider: within 2^-19 of the summed magnitudes M.  h is then off by beta 2^-19 M at most; the losses' derivatives by h are bounded by the
factors below (curvature 1/4 for the logistic ones, scaled for robust; ipo's is 2 / beta^2).
A gradient stored in 16 bits adds half a step of its type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


def softplus(x):
    return max(x, 0.0) + math.log1p(math.exp(-abs(x)))


def sig(x):
    return 1 / (1 + math.exp(-x)) if x >= 0 else math.exp(x) / (1 + math.exp(x))


def reference(lp, ref, scores, mask, spans, kw):
    P = len(spans) // 2
    beta, eps, margin = kw.get("beta", 0.1), kw.get("label_smoothing", 0.0), kw.get("margin", 0.0)
    nll, norm = kw.get("nll_coef", 0.0), kw.get("length_normalised", False)
    kind, red = kw.get("loss_type", "sigmoid"), kw.get("reduction", "mean")
    s, n, like, mag = [], [], [], []
    for i, (a, b) in enumerate(spans):
        idx = torch.arange(a, b)[mask[a:b]]
        d = lp[idx] - (ref[idx] if ref is not None else 0.0)
        k = len(idx)
        n.append(k)
        x, m = float(d.sum()), float(d.abs().sum()) + float(lp[idx].abs().sum())
        if norm and k:
            x, m = x / k, m / k
        if scores is not None:
            x -= float(scores[i])
            m += abs(float(scores[i]))
        s.append(x if k else 0.0)
        mag.append(m)
        like.append(float(lp[idx].sum()))
    per_pair, coef, tol_l, tol_c, ok = [], [0.0] * len(spans), [], [0.0] * len(spans), []
    for i in range(P):
        c, r = (i, P + i) if kw.get("pairs", "halves") == "halves" else (2 * i, 2 * i + 1)
        ok.append(n[c] > 0 and n[r] > 0)
        if not ok[-1]:
            per_pair.append(0.0)
            tol_l.append(0.0)
            continue
        h = beta * (s[c] - s[r]) - margin
        dh_err = beta * 2.0 ** -19 * (mag[c] + mag[r])
        if kind == "sigmoid":
            l, g, first, curv = ((1 - eps) * softplus(-h) + eps * softplus(h),
                                 -(1 - eps) * sig(-h) + eps * sig(h), 1.0, 0.25)
        elif kind == "robust":
            q = 1 - 2 * eps
            l, g, first, curv = (((1 - eps) * softplus(-h) - eps * softplus(h)) / q,
                                 (-(1 - eps) * sig(-h) - eps * sig(h)) / q, 1 / q, 0.25 / q)
        elif kind == "hinge":
            l, g, first, curv = max(0.0, 1 - h), -1.0 if h < 1 else 0.0, 1.0, 0.0
        else:
            u = (h - 0.5) / beta
            l, g, first, curv = u * u, 2 * u / beta, abs(2 * u / beta) + 1, 2 / beta ** 2
        per_pair.append(l - nll * like[c] / n[c])
        tol_l.append(dh_err * first + 2.0 ** -19 * (abs(l) + nll * mag[c]))
        pc, pr = (1 / n[c], 1 / n[r]) if norm else (1.0, 1.0)
        coef[c], coef[r] = beta * g * pc - nll / n[c], -beta * g * pr
        tol_c[c] = beta * pc * (curv * dh_err + 2.0 ** -20 * abs(g)) + 2.0 ** -20 * nll / n[c]
        tol_c[r] = beta * pr * (curv * dh_err + 2.0 ** -20 * abs(g))
    div = max(1, sum(ok)) if red == "mean" else 1
    return s, [beta * x for x in s], per_pair, tol_l, [x / div for x in coef], \
        [x / div for x in tol_c], div, mag


def run(F, lens, seed=0, dtype="fp32", kw=None, ref="token", mask_rate=0.8, check_only=None,
        mask=None):
    kw = dict(kw or {})
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    lp = (-torch.randn(T, generator=g).abs()).to(dt)
    rf = (lp.float() + 0.2 * torch.randn(T, generator=g)).to(dt)
    if mask is None:
        mask = torch.rand(T, generator=g) < mask_rate
    scores = torch.randn(len(lens), generator=g) * 3 - 2 if ref == "scores" else None
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    rf_arg = rf if ref == "token" else None
    loss, rewards, dl = F.flce_preference_loss(
        lp.cuda(), ref_logp=None if rf_arg is None else rf_arg.cuda(),
        ref_scores=None if scores is None else scores.cuda(), mask=mask.cuda(),
        cu_seqlens=cu.cuda(), validate=True, **kw)
    spans = [(int(cu[i]), int(cu[i + 1])) for i in range(len(lens))]
    verify(loss, rewards, dl, reference(lp.double(), None if rf_arg is None else rf.double(), scores,
                                        mask, spans, kw), mask, spans, dt, kw)


def verify(loss, rewards, dl, want, mask, spans, dt, kw):
    s, w_rew, per_pair, tol_l, coef, tol_c, div, mag = want
    beta = kw.get("beta", 0.1)
    if kw.get("reduction", "mean") == "none":
        for x, y, t in zip(loss.tolist(), per_pair, tol_l):
            assert abs(x - y) <= t + 1e-30
    else:
        assert abs(float(loss) - sum(per_pair) / div) <= sum(tol_l) / div + 1e-30
    for x, y, m in zip(rewards.tolist(), w_rew, mag):
        assert abs(x - y) <= beta * 2.0 ** -19 * m + 1e-30
    got = dl.double().cpu().reshape(-1)
    covered = torch.zeros(len(got), dtype=torch.bool)
    for (a, b), c, t in zip(spans, coef, tol_c):
        covered[a:b] = True
        x = got[a:b][mask[a:b]]
        if dt != torch.float32:
            t = t + torch.finfo(dt).eps / 2 * abs(c) * 1.001 + (2.0 ** -25 if dt == torch.float16 else 0)
        assert bool(((x - c).abs() <= t + 1e-30).all()), (c, t, x[:4])
        assert bool((got[a:b][~mask[a:b]] == 0).all())
    assert bool((got[~covered] == 0).all())


LENS = [[1, 1], [0, 5], [1024, 1], [333] * 4, [700, 0, 1, 2000, 37, 9], [5000, 70001], [3] * 600, []]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("pairs", ["halves", "interleaved"])
def test_lengths(F, lens, pairs):
    run(F, lens, seed=len(lens), kw=dict(pairs=pairs, nll_coef=0.1))


@pytest.mark.parametrize("kind,eps", [("sigmoid", 0.0), ("sigmoid", 0.1), ("robust", 0.2),
                                      ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("ref", ["token", "scores", "none"])
def test_kinds(F, kind, eps, norm, ref):
    run(F, [200, 1100, 40, 7, 555, 90], seed=3, ref=ref,
        kw=dict(loss_type=kind, label_smoothing=eps, length_normalised=norm,
                beta=2.0 if norm else 0.1, margin=0.4, nll_coef=0.2, reduction="sum"))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
def test_types_and_reductions(F, dtype, reduction):
    run(F, [200, 1100, 40, 7], seed=4, dtype=dtype, kw=dict(reduction=reduction, beta=0.05))


def test_large_margins_do_not_overflow(F):
    for beta in (50.0, 1e4):
        run(F, [500, 500, 500, 500], seed=5, ref="none", kw=dict(beta=beta, reduction="none"))


def test_pairs_with_an_empty_side_do_not_count(F):
    mask = torch.ones(40, dtype=torch.bool)
    mask[10:20] = False
    run(F, [10, 10, 10, 10], seed=6, mask=mask, kw=dict(pairs="interleaved", nll_coef=0.3))
    run(F, [10, 10, 10, 10], seed=6, mask=torch.zeros(40, dtype=torch.bool), kw=dict())


@pytest.mark.parametrize("v", [math.nan, math.inf, torch.finfo(torch.float32).min])
def test_masked_places_may_hold_anything(F, v):
    g = torch.Generator().manual_seed(1)
    lp, ref = -torch.rand(4, 300, generator=g), -torch.rand(4, 300, generator=g)
    mask = torch.rand(4, 300, generator=g) < 0.5
    a = F.flce_preference_loss(lp.cuda(), ref.cuda(), mask=mask.cuda(), nll_coef=0.1)
    lp2, ref2 = (torch.where(mask, x, torch.full_like(x, v)) for x in (lp, ref))
    b = F.flce_preference_loss(lp2.cuda(), ref2.cuda(), mask=mask.cuda(), nll_coef=0.1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_row_strides_and_labels(F):
    g = torch.Generator().manual_seed(2)
    B_, S = 6, 257
    lp, ref = -torch.rand(B_, S + 3, generator=g), -torch.rand(B_, S + 9, generator=g)
    labels = torch.randint(0, 5, (B_, S + 1), generator=g)
    labels[:, ::3] = -100
    mask = (labels[:, 1:] != -100).reshape(-1)
    kw = dict(beta=0.3)
    got = F.flce_preference_loss(lp.cuda()[:, 2:S + 2], ref.cuda()[:, :S], mask=labels.cuda()[:, 1:], **kw)
    spans = [(i * S, (i + 1) * S) for i in range(B_)]
    want = reference(lp[:, 2:S + 2].reshape(-1).double(), ref[:, :S].reshape(-1).double(), None, mask,
                     spans, kw)
    verify(*got, want, mask, spans, torch.float32, kw)


def test_offsets_out_of_order_are_reported(F):
    x = torch.zeros(100).cuda()
    for cu in ([0, 60, 40], [0, 50, 200], [-1, 50, 100]):
        c = torch.tensor(cu, dtype=torch.int64).cuda()
        with pytest.raises(F.FlceError) as e:
            F.flce_preference_loss(x, cu_seqlens=c, validate=True)
        assert e.value.code == 2
        assert math.isnan(float(F.flce_preference_loss(x, cu_seqlens=c)[0]))


def test_tokens_outside_the_sequences(F):
    g = torch.Generator().manual_seed(9)
    lp = -torch.rand(3000, generator=g)
    cu = torch.tensor([100, 1500, 2600], dtype=torch.int32)
    got = F.flce_preference_loss(lp.cuda(), cu_seqlens=cu.cuda(), validate=True)
    m = torch.ones(3000, dtype=torch.bool)
    spans = [(100, 1500), (1500, 2600)]
    verify(*got, reference(lp.double(), None, None, m, spans, {}), m, spans, torch.float32, {})


@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_autograd(F, reduction):
    g = torch.Generator().manual_seed(7)
    lp, ref = (-torch.rand(6, 400, generator=g).cuda() for _ in range(2))
    n = 3 if reduction == "none" else 1
    up = torch.randn(n, generator=g).cuda()
    base = F.flce_preference_loss(lp, ref, reduction=reduction, g_loss=up)
    a = lp.clone().requires_grad_(True)
    loss, rewards = F.preference_loss(a, ref, reduction=reduction)
    assert torch.equal(rewards, base[1]) and torch.equal(loss.detach().reshape(-1), base[0])
    for _ in range(2):
        (ga,) = torch.autograd.grad((loss * (up if n > 1 else up[0])).sum(), a, retain_graph=True)
        assert torch.equal(ga, base[2])


def test_gradient_against_differences(F):
    """Step 2^-5 of one token moves h by beta 2^-5; the sigmoid loss's third derivative is below
    1/8: a central difference is off by less than beta^3 2^-10 / 8, its rounding by 2^-24 * 2^5."""
    g = torch.Generator().manual_seed(8)
    lp, ref = -torch.rand(4, 6, generator=g), -torch.rand(4, 6, generator=g)
    f = lambda x: float(F.flce_preference_loss(x.cuda(), ref.cuda(), beta=0.5, nll_coef=0.1)[0])  # noqa: E731
    dl = F.flce_preference_loss(lp.cuda(), ref.cuda(), beta=0.5, nll_coef=0.1)[2].cpu()
    for i in range(4):
        for j in (0, 3):
            e = torch.zeros(4, 6)
            e[i, j] = 2.0 ** -5
            hi, lo = lp + e, lp - e
            d = (f(hi) - f(lo)) / float(hi[i, j].double() - lo[i, j].double())
            assert abs(d - float(dl[i, j])) < 2.0 ** -13 + 2.0 ** -17


def test_other_stream_graph_and_repeats(F):
    g = torch.Generator().manual_seed(10)
    lp, ref = (-torch.rand(8, 3000, generator=g).cuda() for _ in range(2))
    want = F.flce_preference_loss(lp, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = F.flce_preference_loss(lp, ref, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cap = F.flce_preference_loss(lp, ref)
    for x in cap:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, cap))


def test_few_long_pairs(F):
    """Pairs whose sums a block adds up."""
    for pairs in ("halves", "interleaved"):
        run(F, [200000, 90000, 150001, 300000], seed=12, kw=dict(pairs=pairs, beta=0.01, nll_coef=0.1))
        run(F, [400000, 0], seed=13, ref="scores", kw=dict(pairs=pairs, beta=0.01))
