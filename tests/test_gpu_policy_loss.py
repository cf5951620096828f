"""The policy loss against a plain loop over sequences in 64 bits.

Tolerances.  A token's term is a product of a ratio (exp of an exact difference rounded to
fp32: |d| <= 20 makes that 20 half steps of 2^-24 at most, and two steps of expf), an
advantage and a weight, plus a KL term with a few roundings of its own: 2^-19 of the sum of
the terms' magnitudes covers them (32 half steps).  Sums over tokens add at most 2^-19 of
the summed magnitudes as well (a tree over 256 fp32 values, then pairs of floats).  A gradient stored
in 16 bits adds half a step of its type, and fp16 half of its smallest subnormal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

LIMIT = 20.0
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


def reference(lp, old, ref, ent, adv, mask, spans, kw):
    """loss, stats, counts, dlogp, dentropy and the magnitudes of the loss's terms, in 64 bits.
    lp, old, ref, ent: flat fp64 CPU tensors; adv: per token; spans: [(begin, end)]."""
    g_lp, g_ent = torch.zeros_like(lp), torch.zeros_like(lp)
    mag = torch.zeros_like(lp)
    lo, hi, c = kw.get("clip_low", 0.2), kw.get("clip_high", 0.2), kw.get("dual_clip", 0.0)
    klc, entc = kw.get("kl_coef", 0.0), kw.get("entropy_coef", 0.0)
    agg = kw.get("aggregate", "token_mean")
    live = [(a, b) for a, b in spans if bool(mask[a:b].any())]
    tokens = sum(int(mask[a:b].sum()) for a, b in spans)
    loss = pg_sum = kl_sum = h_sum = okl_sum = 0.0
    total = 0.0
    clipped = dual = 0
    for a, b in live:
        idx = torch.arange(a, b)[mask[a:b]]
        n = len(idx)
        w = {"token_mean": 1.0 / tokens, "seq_mean_token_mean": 1.0 / (len(live) * n),
             "seq_mean_token_sum": 1.0 / len(live), "sum": kw.get("scale", 1.0)}[agg]
        d = lp[idx] - old[idx] if old is not None else torch.zeros(n, dtype=torch.float64)
        d_tok = d
        seq = kw.get("ratio", "token") == "sequence"
        if seq:
            d = d.mean().expand(n)
        A = adv[idx]
        dc = d.clamp(-LIMIT, LIMIT)
        r = dc.exp()
        inside = (d.abs() <= LIMIT).double()
        obj, dobj = r * A, r * A * inside
        up, down = (A > 0) & (d > math.log1p(hi)), (A < 0) & (d < math.log1p(-lo))
        obj = torch.where(up, (1 + hi) * A, torch.where(down, (1 - lo) * A, obj))
        du = (A < 0) & (d > math.log(c)) if c else torch.zeros(n, dtype=torch.bool)
        obj = torch.where(du, c * A, obj)
        dobj = torch.where(up | down | du, torch.zeros_like(dobj), dobj)
        if seq:
            clipped += int((up | down).any())
            dual += int(du.any())
        else:
            clipped += int((up | down).sum())
            dual += int(du.sum())
        kl, dkl = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
        if ref is not None:
            e = ref[idx] - lp[idx]
            kind = kw.get("kl", "k3")
            if kind == "k1":
                kl, dkl = -e, torch.ones_like(e)
            elif kind == "k2":
                kl, dkl = e * e / 2, -e
            else:
                ec = e.clamp(-LIMIT, LIMIT)
                kl = torch.expm1(ec) - ec
                dkl = torch.where(e.abs() <= LIMIT, -torch.expm1(ec), torch.zeros_like(e))
        h = ent[idx] if ent is not None else torch.zeros(n, dtype=torch.float64)
        pg_sum += float((-w * obj).sum())
        loss += float((w * (-obj + klc * kl - entc * h)).sum())
        total += float((w * (obj.abs() + (klc * kl).abs() + (entc * h).abs())).sum())
        kl_sum += float(kl.sum())
        h_sum += float(h.sum())
        oc = d_tok.clamp(-LIMIT, LIMIT)
        okl_sum += float((torch.expm1(oc) - oc).sum())
        g_lp[idx] = w * (-dobj + klc * dkl)
        mag[idx] = w * (dobj.abs() + (klc * dkl).abs())
        g_ent[idx] = -w * entc
    t = max(tokens, 1)
    stats = [pg_sum, kl_sum / t, h_sum / t, okl_sum / t]
    return loss, stats, [tokens, len(live), clipped, dual], g_lp, g_ent, mag, total


def close(got, want, mag, dtype, what):
    tol = 2.0 ** -19 * mag + 1e-30
    if dtype != torch.float32:
        tol = tol + (torch.finfo(dtype).eps / 2) * want.abs() * 1.001
        if dtype == torch.float16:
            tol = tol + 2.0 ** -25
    err = (got.double().cpu() - want).abs()
    bad = err > tol
    assert not bool(bad.any()), (what, float((err / tol).max()), int(bad.sum()))


def make(lens, seed, dtype=torch.float32, adv_token=False, mask_rate=0.7, spread=0.15):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    lp = (-1.2 * torch.randn(T, generator=g).abs() ** 1.5).to(dtype)
    old = (lp.float() + spread * torch.randn(T, generator=g)).to(dtype)
    ref = (lp.float() + 0.25 * torch.randn(T, generator=g)).to(dtype)
    ent = (0.5 + torch.randn(T, generator=g).abs()).to(dtype)
    mask = torch.rand(T, generator=g) < mask_rate
    adv = torch.randn(T if adv_token else len(lens), generator=g)
    return lp, old, ref, ent, adv, mask


def run(F, lens, seed=0, dtype="fp32", adv_token=False, kw=None, use=("old", "ref", "ent"),
        mask_rate=0.7, spread=0.15, cu_dtype=torch.int32):
    kw = dict(kw or {})
    dt = DTYPES[dtype]
    lp, old, ref, ent, adv, mask = make(lens, seed, dt, adv_token, mask_rate, spread)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=cu_dtype)
    c = lambda x: x.cuda()  # noqa: E731
    loss, stats, counts, dl, de = F.flce_policy_loss(
        c(lp), c(old) if "old" in use else None, c(adv), ref_logp=c(ref) if "ref" in use else None,
        entropy=c(ent) if "ent" in use else None, mask=c(mask), cu_seqlens=c(cu), validate=True,
        **kw)
    spans = [(int(cu[i]), int(cu[i + 1])) for i in range(len(lens))]
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
    adv_t = (adv if adv_token else adv[seq]).double()
    want = reference(lp.double(), old.double() if "old" in use else None,
                     ref.double() if "ref" in use else None,
                     ent.double() if "ent" in use else None, adv_t, mask, spans, kw)
    check(want, loss, stats, counts, dl, de, dt)


def check(want, loss, stats, counts, dl, de, dt):
    w_loss, w_stats, w_counts, g_lp, g_ent, mag, total = want
    assert counts.tolist() == w_counts
    assert abs(float(loss) - w_loss) <= 2.0 ** -19 * total + 1e-30
    for k, (x, y) in enumerate(zip(stats.tolist(), w_stats)):
        # k1's mean cancels: its terms are of size |ref - lp| < 2
        assert abs(x - y) <= 2.0 ** -19 * max(total if k == 0 else 4.0, abs(y)) + 1e-30, (k, x, y)
    if dl is not None:
        close(dl, g_lp.view(dl.shape), mag.view(dl.shape), dt, "dlogp")
    if de is not None:
        close(de, g_ent.view(de.shape), g_ent.abs().view(de.shape), dt, "dentropy")


KW = dict(kl_coef=0.02, entropy_coef=0.01, clip_low=0.2, clip_high=0.28)


@pytest.mark.parametrize("lens", [[1], [5], [0, 3, 0], [1023], [1024], [1025], [1, 1, 1, 1, 1],
                                  [700, 0, 1, 2000, 37], [2048, 1024, 1024], [70001],
                                  [3] * 700, [0, 0, 0]])
@pytest.mark.parametrize("aggregate", ["token_mean", "seq_mean_token_mean"])
def test_lengths(F, lens, aggregate):
    run(F, lens, seed=len(lens), kw=dict(KW, aggregate=aggregate))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("adv_token", [False, True])
def test_types_and_kl(F, dtype, kl, adv_token):
    run(F, [400, 13, 1100, 260], seed=3, dtype=dtype, adv_token=adv_token,
        kw=dict(KW, kl=kl, dual_clip=1.1, aggregate="seq_mean_token_sum"),
        cu_dtype=torch.int64)


@pytest.mark.parametrize("use", [(), ("old",), ("ref",), ("ent",), ("old", "ent")])
def test_absent_arguments(F, use):
    run(F, [100, 57], seed=5, use=use,
        kw=dict(kl_coef=0.1 if "ref" in use else 0.0, entropy_coef=0.1 if "ent" in use else 0.0,
                aggregate="sum", scale=1 / 64))


@pytest.mark.parametrize("aggregate", ["token_mean", "seq_mean_token_mean", "seq_mean_token_sum",
                                       "sum"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sequence_ratio(F, aggregate, dtype):
    # the mean of few tokens moves enough to be clipped both ways
    run(F, [1, 2, 3, 0, 5, 9, 1500, 4, 4, 2, 1, 1], seed=11, dtype=dtype, spread=0.5,
        kw=dict(KW, ratio="sequence", aggregate=aggregate, dual_clip=1.2, scale=0.01))


def test_extreme_ratios_stay_finite_where_the_formula_is(F):
    run(F, [300, 300], seed=7, spread=15.0, kw=dict(KW, dual_clip=3.0))


def test_many_tokens_of_one_sequence(F):
    run(F, [1 << 20], seed=8, kw=dict(KW))


def test_clipping_borders_fall_as_the_exact_difference_does(F):
    """lp - old within a few steps of the borders, where neither fp32 difference nor exp would do."""
    lps, olds, advs = [], [], []
    for border, a in ((math.log1p(0.28), 1.0), (math.log1p(-0.2), -1.0), (math.log(3.0), -1.0)):
        for old in (0.0, -0.7, -3.3, -11.0):
            o = torch.tensor(old, dtype=torch.float32)
            x = (o.double() + border).float()
            for k in range(-3, 4):
                y = x
                for _ in range(abs(k)):
                    y = torch.nextafter(y, torch.tensor(math.inf if k > 0 else -math.inf))
                lps.append(float(y))
                olds.append(float(o))
                advs.append(a)
    lp, old, adv = (torch.tensor(v, dtype=torch.float32) for v in (lps, olds, advs))
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=3.0)
    n = len(lps)
    mask = torch.ones(n, dtype=torch.bool)
    got = F.flce_policy_loss(lp.cuda(), old.cuda(), adv.cuda(), **kw)
    want = reference(lp.double(), old.double(), None, None, adv.double(), mask, [(0, n)], kw)
    assert want[2][2] > 0 and want[2][3] > 0
    check(want, *got[:4], None, torch.float32)


@pytest.mark.parametrize("what", ["nan", "inf", "-inf", "lowest"])
def test_masked_places_may_hold_anything(F, what):
    v = {"nan": math.nan, "inf": math.inf, "-inf": -math.inf,
         "lowest": torch.finfo(torch.float32).min}[what]
    lp, old, ref, ent, adv, mask = make([200, 300, 100], 21, adv_token=True)
    mask[200:500] = False  # a sequence whose mask leaves nothing
    cu = torch.tensor([0, 200, 500, 600], dtype=torch.int32).cuda()
    bad = [torch.where(mask, x, torch.full_like(x, v)) for x in (lp, old, ref, ent, adv)]
    kw = dict(KW, aggregate="seq_mean_token_mean", dual_clip=2.0)
    outs = []
    for a in ((lp, old, ref, ent, adv), bad):
        a = [x.cuda() for x in a]
        outs.append(F.flce_policy_loss(a[0], a[1], a[4], ref_logp=a[2], entropy=a[3],
                                       mask=mask.cuda(), cu_seqlens=cu, **kw))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    assert bool((outs[1][3][~mask.cuda()] == 0).all()) and bool((outs[1][4][~mask.cuda()] == 0).all())


def test_everything_masked(F):
    x = torch.full((3, 50), math.nan).cuda()
    loss, stats, counts, dl, de = F.flce_policy_loss(
        x, x, torch.ones(3).cuda(), ref_logp=x, entropy=x, mask=torch.zeros(3, 50).bool().cuda(),
        kl_coef=0.1, entropy_coef=0.1)
    assert float(loss) == 0 and stats.tolist() == [0] * 4 and counts.tolist() == [0] * 4
    assert bool((dl == 0).all()) and bool((de == 0).all())


def test_a_counted_nan_is_seen(F):
    lp = torch.zeros(10).cuda()
    lp[4] = math.nan
    loss, _, _, dl, _ = F.flce_policy_loss(lp, torch.zeros(10).cuda(), torch.ones(1).cuda())
    assert math.isnan(float(loss)) and math.isnan(float(dl[4])) and not math.isnan(float(dl[3]))


@pytest.mark.parametrize("mask_kind", ["bool", "uint8", "labels"])
def test_row_strides_and_masks(F, mask_kind):
    B_, S = 5, 333
    lp, old, ref, ent, adv, mask = make([S] * B_, 31, adv_token=True)
    v = lambda x: x.view(B_, S)  # noqa: E731

    def wide(x, extra):
        y = torch.full((B_, S + extra), math.nan if x.is_floating_point() else 1, dtype=x.dtype)
        y[:, :S] = v(x)
        return y.cuda()[:, :S]

    m = wide(mask, 3)
    if mask_kind == "uint8":
        m = wide(mask.to(torch.uint8) * 7, 5)
    if mask_kind == "labels":
        m = wide(torch.where(mask, 12, -7), 2)
    kw = dict(KW, aggregate="seq_mean_token_mean")
    got = F.flce_policy_loss(wide(lp, 1), wide(old, 7), wide(adv, 2), ref_logp=wide(ref, 64),
                             entropy=wide(ent, 3), mask=m, ignore_index=-7, **kw)
    want = reference(lp.double(), old.double(), ref.double(), ent.double(), adv.double(), mask,
                     [(i * S, (i + 1) * S) for i in range(B_)], kw)
    check(want, *got, torch.float32)


def test_expanded_rows(F):
    S = 100
    lp, old, _, _, adv, mask = make([S] * 3, 33)
    old1 = old.view(3, S)[:1]
    got = F.flce_policy_loss(lp.view(3, S).cuda(), old1.cuda().expand(3, S), adv.cuda(),
                             mask=mask.view(3, S).cuda())
    want = reference(lp.double(), old1.expand(3, S).reshape(-1).double(), None, None,
                     adv.repeat_interleave(S).double(), mask,
                     [(i * S, (i + 1) * S) for i in range(3)], {})
    check(want, *got[:4], None, torch.float32)


def test_tokens_outside_the_sequences(F):
    lp, old, ref, ent, adv, mask = make([3000], 41)
    cu = torch.tensor([17, 1400, 1400, 2500], dtype=torch.int64)
    adv = torch.randn(3)
    a = torch.zeros(3000)
    for i in range(3):
        a[int(cu[i]):int(cu[i + 1])] = adv[i]
    got = F.flce_policy_loss(lp.cuda(), old.cuda(), adv.cuda(), ref_logp=ref.cuda(),
                             entropy=ent.cuda(), cu_seqlens=cu.cuda(), validate=True, **KW)
    m = torch.zeros(3000, dtype=torch.bool)
    m[17:2500] = True
    want = reference(lp.double(), old.double(), ref.double(), ent.double(), a.double(), m,
                     [(int(cu[i]), int(cu[i + 1])) for i in range(3)], KW)
    check(want, *got, torch.float32)


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [0, 50, 120], [-5, 50, 100], [100, 0]])
def test_offsets_out_of_order_are_reported(F, cu):
    x = torch.zeros(100).cuda()
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    adv = torch.ones(len(cu) - 1).cuda()
    with pytest.raises(F.FlceError) as e:
        F.flce_policy_loss(x, x, adv, cu_seqlens=c, validate=True)
    assert e.value.code == 2
    assert math.isnan(float(F.flce_policy_loss(x, x, adv, cu_seqlens=c)[0]))


def test_gradient_against_differences(F):
    """Differences of the loss itself: step 2^-6 in lp; the loss is smooth there (no token near a
    border), its third derivatives at most ~2 w, so a central difference is off by less than
    2^-12 w, and the fp32 loss's own rounding by 2^-24 |loss| / 2^-6."""
    lens = [5, 4]
    lp, old, ref, ent, adv, mask = make(lens, 51, mask_rate=1.0, spread=0.05)
    cu = torch.tensor([0, 5, 9], dtype=torch.int32).cuda()
    c = [x.cuda() for x in (old, adv, ref, ent)]
    kw = dict(clip_low=0.9, clip_high=9.0, kl_coef=0.5, aggregate="sum", scale=1.0)

    def loss(x):
        return float(F.flce_policy_loss(x.cuda(), c[0], c[1], ref_logp=c[2], cu_seqlens=cu, **kw)[0])

    dl = F.flce_policy_loss(lp.cuda(), c[0], c[1], ref_logp=c[2], cu_seqlens=cu, **kw)[3].cpu()
    h = 2.0 ** -6
    for i in range(9):
        e = torch.zeros(9)
        e[i] = h
        a, b = lp + e, lp - e
        d = (loss(a) - loss(b)) / float(a[i].double() - b[i].double())
        assert abs(d - float(dl[i])) < 2.0 ** -12 * 2 * (1 + float(adv.abs().max())) + 2.0 ** -14


@pytest.mark.parametrize("ratio", ["token", "sequence"])
def test_autograd(F, ratio):
    lens = [1500, 300, 9]
    lp, old, ref, ent, adv, mask = (x.cuda() for x in make(lens, 61))
    cu = torch.tensor([0, 1500, 1800, 1809], dtype=torch.int32).cuda()
    kw = dict(KW, ratio=ratio, aggregate="seq_mean_token_mean")
    base = F.flce_policy_loss(lp, old, adv, ref_logp=ref, entropy=ent, mask=mask, cu_seqlens=cu,
                              g_loss=torch.full((1,), -2.5, device="cuda"), **kw)
    a, b = lp.clone().requires_grad_(True), ent.clone().requires_grad_(True)
    loss, stats, counts = F.policy_loss(a, old, adv, ref_logp=ref, entropy=b, mask=mask,
                                        cu_seqlens=cu, **kw)
    assert loss.shape == () and float(loss.detach()) == float(base[0])
    assert torch.equal(stats, base[1]) and torch.equal(counts, base[2])
    for _ in range(2):  # a second backward pass of the same graph gives the same
        ga, gb = torch.autograd.grad(loss * -2.5, (a, b), retain_graph=True)
        assert torch.equal(ga, base[3]) and torch.equal(gb, base[4])
    # a float64 upstream gradient, and entropy as a constant
    loss2, _, _ = F.policy_loss(a, old, adv, ref_logp=ref, entropy=ent, mask=mask, cu_seqlens=cu, **kw)
    (ga2,) = torch.autograd.grad(loss2.double() * -2.5, (a,))
    assert torch.equal(ga2, base[3])


def test_repeats_bit_for_bit_and_workspace_contents_do_not_matter(F):
    lens = [20000, 1, 30000, 777]
    lp, old, ref, ent, adv, mask = (x.cuda() for x in make(lens, 71))
    cu = torch.tensor([0, 20000, 20001, 50001, 50778], dtype=torch.int32).cuda()
    kw = dict(KW, aggregate="seq_mean_token_mean", ref_logp=ref, entropy=ent, mask=mask, cu_seqlens=cu)
    p, _ = F.policy_params(lp, old, adv, **kw)
    ws = torch.empty(F.policy_workspace_size(p), dtype=torch.uint8, device="cuda")
    first = F.flce_policy_loss(lp, old, adv, workspace=ws, **kw)
    for fill in (0, 255, 77):
        ws.fill_(fill)
        again = F.flce_policy_loss(lp, old, adv, workspace=ws, **kw)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_other_stream_and_graph(F):
    lens = [3000, 500]
    lp, old, ref, ent, adv, mask = (x.cuda() for x in make(lens, 81))
    cu = torch.tensor([0, 3000, 3500], dtype=torch.int32).cuda()
    kw = dict(KW, ref_logp=ref, entropy=ent, mask=mask, cu_seqlens=cu)
    want = F.flce_policy_loss(lp, old, adv, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = F.flce_policy_loss(lp, old, adv, stream=s, **kw)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cap = F.flce_policy_loss(lp, old, adv, **kw)
    for x in cap:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, cap))


# ------------------------------------------------------------------ on top of the head
def _head_inputs(N=700, H=256, V=1536, layout="hv", seed=5):
    g = torch.Generator().manual_seed(seed)
    hidden = torch.randn(N, H, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(H, V, generator=g) / H ** 0.5).to(torch.bfloat16)
    weight = (w if layout == "hv" else w.t().contiguous()).cuda()
    labels = torch.randint(0, V, (N,), generator=g)
    labels[torch.rand(N, generator=g) < 0.2] = -100
    cu = torch.tensor([0, N // 3, N // 3, N - 5, N], dtype=torch.int32).cuda()
    z = hidden.double() @ (weight.double() if layout == "hv" else weight.double().t())
    logq = torch.log_softmax(z, 1)
    lp = logq.gather(1, labels.cuda().clamp(min=0)[:, None])[:, 0].float().cpu()
    old = (lp + 0.15 * torch.randn(N, generator=g)).cuda()
    ref = (lp + 0.25 * torch.randn(N, generator=g)).cuda()
    return hidden, weight, labels.cuda(), old, ref, torch.randn(4, generator=g).cuda(), cu


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("chunk_n", [0, 512])
def test_head_gives_what_the_two_calls_give(F, layout, chunk_n):
    """The same kernels on the same values: the loss, its parts and the log-probabilities are
    equal, and with one chunk the gradients of the gradient-in-forward call are too."""
    N = 1300
    hidden, weight, labels, old, ref, adv, cu = _head_inputs(N=N, layout=layout)
    kw = dict(KW, aggregate="seq_mean_token_mean")
    got = F.flce_policy_forward_backward(hidden, weight, labels, old, adv, ref_logp=ref,
                                         cu_seqlens=cu, weight_layout=layout, chunk_n=chunk_n,
                                         validate=True, **kw)
    ce, ent, _, _ = F.flce_forward(hidden, weight, labels, "none", weight_layout=layout)
    assert torch.equal(got[3], 0 - ce) and torch.equal(got[4], ent)
    loss, stats, counts, dl, de = F.flce_policy_loss(0 - ce, old, adv, ref_logp=ref, entropy=ent,
                                                     mask=labels, cu_seqlens=cu, **kw)
    assert torch.equal(got[0], loss) and torch.equal(got[1], stats) and torch.equal(got[2], counts)
    dh, dw = F.flce_forward_backward(hidden, weight, labels, -dl, de, "none",
                                     weight_layout=layout, chunk_n=chunk_n)[4:]
    assert torch.equal(got[5], dh) and torch.equal(got[6], dw)


def test_head_against_the_definition(F):
    hidden, weight, labels, old, ref, adv, cu = _head_inputs()
    kw = dict(KW, aggregate="token_mean")
    a = hidden.clone().requires_grad_(True)
    b = weight.clone().requires_grad_(True)
    loss, _, _, _, _ = F.linear_policy_loss(a, b, labels, old, adv, ref_logp=ref, cu_seqlens=cu, **kw)
    g1 = torch.autograd.grad(loss * 3.0, (a, b), retain_graph=True)
    g2 = torch.autograd.grad(loss * 3.0, (a, b))
    assert all(torch.equal(x, y) for x, y in zip(g1, g2))
    h = hidden.double().requires_grad_(True)
    w = weight.double().requires_grad_(True)
    logq = torch.log_softmax(h @ w, 1)
    m = labels != -100
    lp = logq.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    ent = -(logq.exp() * logq).sum(1)
    seq = torch.bucketize(torch.arange(len(m), device="cuda"), cu[1:].long(), right=True)
    want = reference(lp.detach().cpu(), old.double().cpu(), ref.double().cpu(), ent.detach().cpu(),
                     adv.double()[seq].cpu(), m.cpu(),
                     [(int(cu[i]), int(cu[i + 1])) for i in range(4)], kw)
    # the head's log-probabilities are within 1e-5 of the exact ones here
    assert abs(float(loss.detach()) - want[0]) <= 1e-5 * want[6]
    gh, gw = torch.autograd.grad([lp, ent], [h, w], [want[3].cuda() * 3, want[4].cuda() * 3])
    for got, exact in zip(g1, (gh, gw)):
        rel = float((got.double() - exact).norm() / exact.norm())
        assert rel <= 1e-2  # the head's bound: dlogits and outputs are rounded to bf16


def test_head_sequence_ratio_needs_one_chunk(F):
    hidden, weight, labels, old, ref, adv, cu = _head_inputs(N=1300)
    with pytest.raises(F.FlceError):
        F.flce_policy_forward_backward(hidden, weight, labels, old, adv, cu_seqlens=cu,
                                       ratio="sequence", chunk_n=512)
    got = F.flce_policy_forward_backward(hidden, weight, labels, old, adv, cu_seqlens=cu,
                                         ratio="sequence")
    want = F.flce_policy_loss(got[3], old, adv, mask=labels, cu_seqlens=cu, ratio="sequence")
    assert torch.equal(got[0], want[0])


def test_head_no_rows(F):
    w = torch.zeros(64, 128, dtype=torch.bfloat16).cuda()
    e = torch.empty(0).cuda()
    got = F.flce_policy_forward_backward(torch.empty(0, 64, dtype=torch.bfloat16).cuda(), w,
                                         torch.empty(0, dtype=torch.int64).cuda(), e,
                                         torch.ones(1).cuda(), validate=True)
    assert float(got[0]) == 0 and got[2].tolist() == [0] * 4 and bool((got[6] == 0).all())


def test_head_bad_label_is_reported(F):
    hidden, weight, labels, old, ref, adv, cu = _head_inputs()
    labels[3] = 1 << 20
    with pytest.raises(F.FlceError) as e:
        F.flce_policy_forward_backward(hidden, weight, labels, old, adv, cu_seqlens=cu, validate=True)
    assert e.value.code == 5


@pytest.mark.parametrize("lens", [[5000] * 9, [90000, 3, 40000]])
def test_clusters_and_grids_in_a_graph(F, lens):
    """More pieces than one block takes: a cluster's launch, and a cooperative grid's."""
    lp, old, ref, ent, adv, mask = (x.cuda() for x in make(lens, 91))
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32).cuda()
    kw = dict(KW, aggregate="seq_mean_token_mean", ref_logp=ref, entropy=ent, mask=mask, cu_seqlens=cu)
    want = F.flce_policy_loss(lp, old, adv, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cap = F.flce_policy_loss(lp, old, adv, **kw)
    for _ in range(3):
        for x in cap:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, cap))


def test_many_short_sequences(F):
    run(F, [3, 0, 1, 7] * 20000, seed=95, kw=dict(KW, aggregate="seq_mean_token_mean"))


@pytest.mark.parametrize("ratio", ["token", "sequence"])
def test_more_tokens_than_warps_keep(F, ratio):
    """Beyond a piece per warp of the GPU: kept gradients and recomputed ones in one launch."""
    run(F, [700000, 5, 900000, 30000], seed=97, dtype="bf16",
        kw=dict(KW, ratio=ratio, aggregate="seq_mean_token_mean"))


@pytest.mark.parametrize("ratio", ["token", "sequence"])
def test_few_long_sequences(F, ratio):
    """Sequences whose sums a block adds up."""
    run(F, [200000, 0, 150001], seed=99, kw=dict(KW, ratio=ratio, aggregate="seq_mean_token_mean"))


@pytest.mark.parametrize("ratio", ["token", "sequence"])
def test_counted_infinities_follow_the_formula(F, ratio):
    """A token of probability zero under the policy, or under the old one: the clamped ratio where
    it is not clipped, the border where it is, and no gradient either way."""
    n = 40
    lp = -torch.rand(n, generator=torch.Generator().manual_seed(4))
    old = lp + 0.01
    lp[3], lp[13], old[23], old[33] = -math.inf, -math.inf, -math.inf, -math.inf
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0])
    cu = torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32)
    mask = torch.ones(n, dtype=torch.bool)
    for kw in (dict(ratio=ratio), dict(ratio=ratio, dual_clip=3.0)):
        got = F.flce_policy_loss(lp.cuda(), old.cuda(), adv.cuda(), cu_seqlens=cu.cuda(), **kw)
        want = reference(lp.double(), old.double(), None, None, adv.repeat_interleave(10).double(),
                         mask, [(i * 10, (i + 1) * 10) for i in range(4)], kw)
        check(want, *got[:4], None, torch.float32)
