"""Cases of the training-loss and embedding operators, their plain forms and their 64-bit values.

`run` computes a case with elementary torch operations where `own` is false, and through
the package's public calls where it is true.  The operators:

policy       clipped policy loss with a KL term and an entropy bonus over the log-probabilities
             of the sampled tokens, and its gradients;
preference   a preference loss over pairs of sequences, and its gradient;
embed        embedding lookup with scaling;
embed_grad   its gradient by sorted tokens, dense or added to a tied head's gradient;
head         the policy loss on top of the fused LM head: loss, dhidden and dweight in one call.
"""
import math

import numpy as np
import torch

own = False

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
LIMIT = 20.0  # log-ratios are clamped to +-20 before the exponential


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one rollout group of a small run: a few hundred tokens, latency is everything
        dict(name="policy_small_group", op="policy", layout="padded", B=4, S=64, dtype="fp32",
             adv="seq", agg="token_mean", ratio="token", kl="k3", ref=True, ent=True, dual=0.0,
             api="call"),
        # the RL batch of the 16384-token head workload, packed and ragged, one advantage per
        # sequence, through autograd as a training loop would
        dict(name="policy_packed_rl_batch", op="policy", layout="packed", B=61, S=16384,
             dtype="fp32", adv="seq", agg="seq_mean_token_mean", ratio="token", kl="k3", ref=True,
             ent=True, dual=3.0, api="autograd"),
        # a whole rollout batch scored at once: a million tokens, an advantage per token
        dict(name="policy_rollout_batch", op="policy", layout="padded", B=256, S=4096,
             dtype="fp32", adv="token", agg="token_mean", ratio="token", kl="k2", ref=True,
             ent=True, dual=0.0, api="call"),
        # sequence-level ratios over long bf16 sequences, no reference policy
        dict(name="policy_sequence_ratio", op="policy", layout="packed", B=97, S=300007,
             dtype="bf16", adv="seq", agg="seq_mean_token_mean", ratio="sequence", kl="k3",
             ref=False, ent=False, dual=0.0, api="call"),
        # a micro-batch of two preference pairs
        dict(name="preference_two_pairs", op="preference", layout="padded", B=4, S=333,
             dtype="fp32", loss="sigmoid", ref="token", norm=False, smooth=0.0, nll=0.0,
             pairs="halves"),
        # a large batch of ragged pairs, label smoothing and the chosen side's likelihood
        dict(name="preference_packed_pairs", op="preference", layout="packed", B=512, S=1 << 20,
             dtype="fp32", loss="sigmoid", ref="token", norm=False, smooth=0.1, nll=0.05,
             pairs="interleaved"),
        # the lookup of a few tokens in a decoding or scoring loop
        dict(name="embed_few_tokens", op="embed", N=8, H=4096, V=32000, dtype="bf16", scaled=False),
        # the lookup of a training batch, tied table with scaling
        dict(name="embed_batch", op="embed", N=16384, H=3584, V=152064, dtype="bf16", scaled=True),
        # a tied table: the lookup's gradient added to the head's gradient, a tenth padding
        dict(name="embed_grad_tied", op="embed_grad", N=16384, H=2304, V=32768, dtype="bf16",
             accumulate=True, pad=0.1),
        # the dense gradient of a large table, untouched rows zero
        dict(name="embed_grad_dense", op="embed_grad", N=4096, H=2304, V=256000, dtype="bf16",
             accumulate=False, pad=0.0),
        # the head and the loss of a small model in one call
        dict(name="head_small", op="head", N=256, H=512, V=4096, B=4, layout="hv", agg="token_mean",
             kl="k3"),
        # the head and the loss of a 32000-entry vocabulary
        dict(name="head_batch", op="head", N=4096, H=4096, V=32000, B=16, layout="hv",
             agg="seq_mean_token_mean", kl="k3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["policy", "preference", "embed", "embed_grad", "head"])
    if op == "policy":
        layout = rng.choice(["padded", "packed"])
        ratio = rng.choice(["token", "token", "sequence"])
        B = _log(rng, 1, 256)
        return dict(op=op, layout=layout, B=B,
                    S=_log(rng, 1, 4096) if layout == "padded" else _log(rng, B, 1 << 20),
                    dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    adv="seq" if ratio == "sequence" else rng.choice(["seq", "token"]),
                    agg=rng.choice(["token_mean", "seq_mean_token_mean", "seq_mean_token_sum",
                                    "sum"]),
                    ratio=ratio, kl=rng.choice(["k1", "k2", "k3"]), ref=rng.random() < 0.7,
                    ent=rng.random() < 0.6, dual=rng.choice([0.0, 3.0]),
                    api=rng.choice(["call", "autograd"]))
    if op == "preference":
        layout = rng.choice(["padded", "packed"])
        P = _log(rng, 1, 256)
        loss = rng.choice(["sigmoid", "hinge", "ipo", "robust"])
        return dict(op=op, layout=layout, B=2 * P,
                    S=_log(rng, 1, 2048) if layout == "padded" else _log(rng, 2 * P, 1 << 20),
                    dtype=rng.choice(["fp32", "bf16", "fp16"]),
                    loss=loss,
                    ref=rng.choice(["token", "scores", "none"]), norm=rng.random() < 0.3,
                    smooth=rng.choice([0.0, 0.1]) if loss in ("sigmoid", "robust") else 0.0,
                    nll=rng.choice([0.0, 0.05]), pairs=rng.choice(["halves", "interleaved"]))
    if op == "embed":
        return dict(op=op, N=_log(rng, 1, 16384), H=_log(rng, 32, 3584), V=_log(rng, 100, 152064),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), scaled=rng.random() < 0.5)
    if op == "embed_grad":
        return dict(op=op, N=_log(rng, 1, 16384), H=_log(rng, 32, 2304), V=_log(rng, 100, 256000),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    accumulate=rng.random() < 0.5, pad=rng.choice([0.0, 0.1, 0.5]))
    layout = rng.choice(["hv", "vh"])
    V = _log(rng, 200, 32000)
    return dict(op=op, N=_log(rng, 16, 4096), H=8 * _log(rng, 8, 512),
                V=V if layout == "vh" else 8 * (V // 8), B=_log(rng, 1, 16), layout=layout,
                agg=rng.choice(["token_mean", "seq_mean_token_mean", "sum"]),
                kl=rng.choice(["k1", "k2", "k3"]))


# ---------------------------------------------------------------------------- inputs
def _gen(seed, k=0):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + 7919 * k) % (1 << 62))
    return g


def _lens(total, count, rs):
    """Lengths of `count` ragged sequences that sum to `total`; one is empty where many are."""
    w = np.exp(rs.uniform(0.0, 2.5, count))
    if count >= 8:
        w[rs.randint(count)] = 0.0
    ln = np.floor(w / w.sum() * total).astype(np.int64)
    ln[int(np.argmax(ln))] += total - int(ln.sum())
    return ln


def _mask(B, starts, lens, total, rs, pad_tail):
    """The response part of each sequence: a prompt before it, padding after it where padded."""
    m = np.zeros(total, dtype=np.bool_)
    for s, n in zip(starts.tolist(), lens.tolist()):
        a = int(n * rs.uniform(0.0, 0.4))
        b = n - int(n * rs.uniform(0.0, 0.5)) if pad_tail else n
        m[s + a:s + b] = True
    if B >= 8:  # a sequence whose mask leaves nothing
        i = rs.randint(B)
        m[starts[i]:starts[i] + lens[i]] = False
    return m


def _sequences(case, seed):
    """(shape, sequence number of each token, cu_seqlens or None, mask, the sequences' ends) of a
    padded or packed batch."""
    rs = np.random.RandomState(int(seed) % (1 << 31))
    B, S = case["B"], case["S"]
    if case["layout"] == "padded":
        lens, shape = np.full(B, S, dtype=np.int64), (B, S)
    else:
        lens, shape = _lens(S, B, rs), (S,)
    cu = np.concatenate([[0], np.cumsum(lens)])
    m = _mask(B, cu[:-1], lens, int(cu[-1]), rs, case["layout"] == "padded")
    cu = torch.from_numpy(cu).cuda()
    return (shape, torch.from_numpy(np.repeat(np.arange(B), lens)).cuda(),
            None if case["layout"] == "padded" else cu.to(torch.int32),
            torch.from_numpy(m).cuda().view(shape), cu)


def _logps(shape, mask, dtype, seed):
    """Sampled tokens' log-probabilities under the policy, the rollout's policy and the reference:
    zero on the tokens that do not count, as the fused head leaves ignored rows."""
    g = _gen(seed)
    r = lambda: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    lp = -1.2 * r().abs() ** 1.5
    out = [lp, lp + 0.15 * r(), lp + 0.25 * r(), 0.5 + r().abs()]
    return [torch.where(mask, x, torch.zeros_like(x)).to(dtype) for x in out]


def _ids(N, V, seed, pad=0.0):
    """Token ids with frequencies that fall as 1/rank, spread over the table; a share `pad` of one id."""
    g = _gen(seed, 3)
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    k = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    step = 7919 if V % 7919 else 7907
    ids = (k * step + 13) % V
    if pad:
        ids = torch.where(torch.rand(N, generator=g, device="cuda") < pad, torch.zeros_like(ids), ids)
    return ids


def _policy_kw(case):
    return dict(clip_low=0.2, clip_high=0.28, dual_clip=case["dual"],
                kl_coef=0.02 if case["ref"] else 0.0, kl=case["kl"],
                entropy_coef=0.01 if case["ent"] else 0.0, ratio=case["ratio"],
                aggregate=case["agg"], scale=1.0 / 1024 if case["agg"] == "sum" else 1.0)


def _prepare_policy(case, seed):
    shape, seq, cu, mask, ends = _sequences(case, seed)
    lp, old, ref, ent = _logps(shape, mask, DT[case["dtype"]], seed)
    adv = torch.randn(case["B"] if case["adv"] == "seq" else shape, generator=_gen(seed, 1),
                      device="cuda")
    return dict(case=case, kw=_policy_kw(case), lp=lp, old=old, ref=ref if case["ref"] else None,
                ent=ent if case["ent"] else None, adv=adv, mask=mask, cu=cu, seq=seq,
                ends=ends)


def _prepare_preference(case, seed):
    shape, seq, cu, mask, ends = _sequences(case, seed)
    lp, _, ref, _ = _logps(shape, mask, DT[case["dtype"]], seed)
    scores = None
    if case["ref"] == "scores":
        scores = torch.zeros(case["B"], device="cuda", dtype=torch.float64)
        scores = scores.index_add_(0, seq, ref.reshape(-1).double()).float()
        if case["norm"]:
            n = torch.zeros_like(scores).index_add_(0, seq, mask.reshape(-1).float())
            scores = scores / n.clamp(min=1)
    kw = dict(beta=2.0 if case["norm"] else 0.1, loss_type=case["loss"],
              label_smoothing=case["smooth"], margin=0.3 if case["norm"] else 0.0,
              length_normalised=case["norm"], nll_coef=case["nll"], pairs=case["pairs"])
    return dict(case=case, kw=kw, lp=lp, ref=ref if case["ref"] == "token" else None,
                scores=scores, mask=mask, cu=cu, seq=seq, ends=ends)


def _prepare_embed(case, seed):
    g, dt = _gen(seed), DT[case["dtype"]]
    N, H, V = case["N"], case["H"], case["V"]
    w = torch.empty(V, H, dtype=dt, device="cuda").normal_(0.0, 0.02, generator=g)
    return dict(case=case, ids=_ids(N, V, seed), w=w,
                scale=math.sqrt(H) if case["scaled"] else 1.0)


def _prepare_embed_grad(case, seed):
    g, dt = _gen(seed), DT[case["dtype"]]
    N, H, V = case["N"], case["H"], case["V"]
    dout = torch.empty(N, H, dtype=dt, device="cuda").normal_(0.0, 0.1, generator=g)
    dw = None
    if case["accumulate"]:
        dw = torch.empty(V, H, dtype=dt, device="cuda").normal_(0.0, 0.1, generator=g)
    return dict(case=case, ids=_ids(N, V, seed, case["pad"]), dout=dout, dw=dw,
                scale=math.sqrt(H) if case["accumulate"] else 1.0)


def _prepare_head(case, seed):
    N, H, V = case["N"], case["H"], case["V"]
    rs = np.random.RandomState(int(seed) % (1 << 31))
    g = _gen(seed)
    hidden = torch.randn(N, H, generator=g, device="cuda").to(torch.bfloat16)
    shape = (H, V) if case["layout"] == "hv" else (V, H)
    weight = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(
        0.0, 1.0 / math.sqrt(H), generator=g)
    lens = _lens(N, case["B"], rs)
    cu = np.concatenate([[0], np.cumsum(lens)])
    mask = torch.from_numpy(_mask(case["B"], cu[:-1], lens, N, rs, False)).cuda()
    ends = torch.from_numpy(cu).cuda()
    labels = torch.randint(0, V, (N,), generator=g, device="cuda")
    labels = torch.where(mask, labels, torch.full_like(labels, -100))
    # the rollout's and the reference's log-probabilities lie near the present policy's
    lp = torch.empty(N, device="cuda")
    for a in range(0, N, 1024):
        h = hidden[a:a + 1024].float()
        z = h @ (weight if case["layout"] == "hv" else weight.t()).float()
        y = labels[a:a + 1024].clamp(min=0)
        lp[a:a + 1024] = z.gather(1, y[:, None])[:, 0] - torch.logsumexp(z, 1)
    old = lp + 0.15 * torch.randn(N, generator=g, device="cuda")
    ref = lp + 0.25 * torch.randn(N, generator=g, device="cuda")
    adv = torch.randn(case["B"], generator=g, device="cuda")
    kw = _policy_kw(dict(case, dual=0.0, ref=True, ent=True, ratio="token"))
    return dict(case=case, kw=kw, hidden=hidden, weight=weight, labels=labels, old=old, ref=ref,
                adv=adv, cu=ends.to(torch.int32), ends=ends,
                seq=torch.from_numpy(np.repeat(np.arange(case["B"]), lens)).cuda(), mask=mask)


def prepare(case, seed):
    return {"policy": _prepare_policy, "preference": _prepare_preference, "embed": _prepare_embed,
            "embed_grad": _prepare_embed_grad, "head": _prepare_head}[case["op"]](case, seed)


# ---------------------------------------------------------------------------- plain forms
def _seq_sum(x, cu):
    """Sums of 64-bit x over the tokens [cu[i], cu[i + 1])."""
    c = torch.cat([x.new_zeros(1), torch.cumsum(x, 0)])
    return c[cu[1:]] - c[cu[:-1]]


def _plain_policy(lp, old, ref, ent, adv, mask, seq, cu, B, kw):
    """loss, means, counts, dlp, dent of flat fp32 tokens.  The log-ratios, the KL terms and the sums
    are held in 64 bits: the first lie next to the clipping borders, the others cancel."""
    zero = torch.zeros((), device=lp.device, dtype=torch.float64)
    m = mask
    d = torch.where(m, lp.double() - old.double(), zero)
    n_i = _seq_sum(m.double(), cu)
    valid, seqs = n_i.sum(), (n_i > 0).sum()
    if kw["aggregate"] == "token_mean":
        w = 1.0 / valid.clamp(min=1).expand(B)
    elif kw["aggregate"] == "seq_mean_token_mean":
        w = 1.0 / (seqs.clamp(min=1) * n_i.clamp(min=1))
    elif kw["aggregate"] == "seq_mean_token_sum":
        w = 1.0 / seqs.clamp(min=1).double().expand(B)
    else:
        w = torch.full((B,), kw["scale"], device=lp.device, dtype=torch.float64)
    wt = w[seq]
    old_kl = torch.exp(d.clamp(-LIMIT, LIMIT)) - 1.0 - d.clamp(-LIMIT, LIMIT)
    a = adv if kw["adv_token"] else adv[seq]
    if kw["ratio"] == "sequence":
        d = (_seq_sum(d, cu) / n_i.clamp(min=1))[seq]
    above = (a > 0) & (d > math.log1p(kw["clip_high"]))
    below = (a < 0) & (d < math.log1p(-kw["clip_low"]))
    dual = torch.zeros_like(above)
    if kw["dual_clip"]:
        dual = (a < 0) & (d > math.log(kw["dual_clip"]))
    out = above | below | dual | (d.abs() > LIMIT)
    r = torch.exp(d.clamp(-LIMIT, LIMIT)).float()
    r = torch.where(above, 1.0 + kw["clip_high"], r)
    r = torch.where(below, 1.0 - kw["clip_low"], r)
    r = torch.where(dual, kw["dual_clip"], r)
    pg = torch.where(m, -r * a, 0.0)
    dlp = torch.where(out, 0.0, -r * a)
    kl = zero
    if ref is not None:
        e = torch.where(m, ref.double() - lp.double(), zero)
        if kw["kl"] == "k1":
            kl, dkl = -e, torch.ones_like(e)
        elif kw["kl"] == "k2":
            kl, dkl = 0.5 * e * e, -e
        else:
            c = e.clamp(-LIMIT, LIMIT)
            kl = torch.exp(c) - 1.0 - c
            dkl = torch.where(e.abs() > LIMIT, 0.0, 1.0 - torch.exp(c))
        dlp = dlp + kw["kl_coef"] * dkl.float()
        kl = torch.where(m, kl, zero)
    dlp = torch.where(m, wt.float() * dlp, 0.0)
    pg_sum = (wt * pg.double()).sum()
    loss = pg_sum + kw["kl_coef"] * (wt * kl).sum()
    mean = 1.0 / valid.clamp(min=1)
    h_mean, dent = zero, None
    if ent is not None:
        h = torch.where(m, ent.double(), zero)
        loss = loss - kw["entropy_coef"] * (wt * h).sum()
        h_mean = h.sum() * mean
        dent = torch.where(m, -kw["entropy_coef"] * wt.float(), 0.0)
    stats = torch.stack([pg_sum, (torch.zeros_like(d) + kl).sum() * mean, h_mean,
                         torch.where(m, old_kl, zero).sum() * mean]).float()
    if kw["ratio"] == "sequence":
        n_clip = _seq_sum(((above | below) & m).double(), cu).gt(0).sum()
        n_dual = _seq_sum((dual & m).double(), cu).gt(0).sum()
    else:
        n_clip, n_dual = ((above | below) & m).sum(), (dual & m).sum()
    counts = torch.stack([valid.long(), seqs, n_clip, n_dual])
    return loss.float().reshape(1), stats, counts, dlp, dent


def _run_policy_plain(s):
    case, shape, dt = s["case"], s["lp"].shape, s["lp"].dtype
    flat = lambda x: None if x is None else x.reshape(-1).float()  # noqa: E731
    kw = dict(s["kw"], adv_token=case["adv"] == "token")
    loss, stats, counts, dlp, dent = _plain_policy(
        flat(s["lp"]), flat(s["old"]), flat(s["ref"]), flat(s["ent"]), s["adv"].reshape(-1),
        s["mask"].reshape(-1), s["seq"], s["ends"], case["B"], kw)
    out = dict(loss=loss, stats=stats, counts=counts, dlogp=dlp.to(dt).view(shape))
    if dent is not None:
        out["dentropy"] = dent.to(dt).view(shape)
    return out


def _log_sigmoid(x):
    return torch.clamp(x, max=0.0) - torch.log1p(torch.exp(-x.abs()))


def _run_preference_plain(s):
    case, kw, B = s["case"], s["kw"], s["case"]["B"]
    lp, m, seq = s["lp"].reshape(-1).float(), s["mask"].reshape(-1), s["seq"]
    diff = lp if s["ref"] is None else lp - s["ref"].reshape(-1).float()
    n = _seq_sum(m.double(), s["ends"])
    # sums of thousands of terms of both signs: in 64 bits
    score = _seq_sum(torch.where(m, diff.double(), 0.0), s["ends"])
    like = _seq_sum(torch.where(m, lp.double(), 0.0), s["ends"])
    if kw["length_normalised"]:
        score = score / n.clamp(min=1)
    if s["scores"] is not None:
        score = score - s["scores"].double()
    score = torch.where(n > 0, score, 0.0)
    if kw["pairs"] == "halves":
        c, r = torch.arange(B // 2, device=lp.device), torch.arange(B // 2, B, device=lp.device)
    else:
        c, r = torch.arange(0, B, 2, device=lp.device), torch.arange(1, B, 2, device=lp.device)
    beta, eps = kw["beta"], kw["label_smoothing"]
    ok = (n[c] > 0) & (n[r] > 0)
    h = beta * (score[c] - score[r]) - kw["margin"]
    if kw["loss_type"] == "sigmoid":
        ls = -(1 - eps) * _log_sigmoid(h) - eps * _log_sigmoid(-h)
        dh = -(1 - eps) * torch.sigmoid(-h) + eps * torch.sigmoid(h)
    elif kw["loss_type"] == "robust":
        ls = (-(1 - eps) * _log_sigmoid(h) + eps * _log_sigmoid(-h)) / (1 - 2 * eps)
        dh = (-(1 - eps) * torch.sigmoid(-h) - eps * torch.sigmoid(h)) / (1 - 2 * eps)
    elif kw["loss_type"] == "hinge":
        ls, dh = torch.clamp(1 - h, min=0.0), -(h < 1).double()
    else:
        u = score[c] - score[r] - kw["margin"] / beta - 0.5 / beta
        ls, dh = u * u, 2 * u / beta
    nc = n.clamp(min=1)
    ls = ls - kw["nll_coef"] * like[c] / nc[c]
    pairs = ok.sum().clamp(min=1)
    loss = torch.where(ok, ls, 0.0).sum() / pairs
    per = 1.0 / nc if kw["length_normalised"] else torch.ones_like(n)
    gc = torch.where(ok, (beta * dh * per[c] - kw["nll_coef"] / nc[c]) / pairs, 0.0)
    gr = torch.where(ok, -beta * dh * per[r] / pairs, 0.0)
    coef = torch.zeros(B, device=lp.device, dtype=torch.float64)
    coef[c], coef[r] = gc, gr
    dlp = torch.where(m, coef.float()[seq], 0.0)
    return dict(loss=loss.float().reshape(1), rewards=(beta * score).float(),
                dlogp=dlp.to(s["lp"].dtype).view(s["lp"].shape))


def _run_embed_plain(s):
    return (s["w"][s["ids"]].float() * s["scale"]).to(s["w"].dtype)


def _run_embed_grad_plain(s):
    case = s["case"]
    acc = torch.zeros(case["V"], case["H"], device="cuda")
    acc.index_add_(0, s["ids"], s["dout"].float())
    acc.mul_(s["scale"])
    if s["dw"] is not None:
        acc.add_(s["dw"].float())
    return acc.to(s["dout"].dtype)


def _run_head_plain(s):
    case, kw = s["case"], dict(s["kw"], adv_token=False)
    h = s["hidden"].float()
    w = (s["weight"] if case["layout"] == "hv" else s["weight"].t()).float()
    z = h @ w
    y, m = s["labels"].clamp(min=0), s["mask"]
    z = z - z.amax(1, keepdim=True)
    lse = torch.log(torch.exp(z).sum(1, keepdim=True))
    z = z - lse
    p = torch.exp(z)
    neg_ent = (p * z).sum(1, keepdim=True)
    lp = torch.where(m, z.gather(1, y[:, None])[:, 0], 0.0)
    ent = torch.where(m, -neg_ent[:, 0], 0.0)
    loss, stats, counts, dlp, dent = _plain_policy(lp, s["old"], s["ref"], ent, s["adv"], m,
                                                   s["seq"], s["ends"], case["B"], kw)
    # d lp / dz = onehot - p,  d H / dz = -p (log p + H)
    dz = p * (-dlp[:, None] - dent[:, None] * (z - neg_ent))
    dz.scatter_add_(1, y[:, None], dlp[:, None])
    dhidden, dweight = dz @ w.t(), h.t() @ dz
    if case["layout"] == "vh":
        dweight = dweight.t()
    return dict(loss=loss, stats=stats, counts=counts, logp=lp, entropy=ent,
                dhidden=dhidden.to(torch.bfloat16), dweight=dweight.to(torch.bfloat16))


# ---------------------------------------------------------------------------- the package's calls
def _run_policy_own(s):
    import linear_cross_entropy_forward_gb300 as F
    kw = dict(s["kw"], ref_logp=s["ref"], mask=s["mask"], cu_seqlens=s["cu"])
    if s["case"]["api"] == "autograd":
        lp = s["lp"].detach().requires_grad_(True)
        ent = None if s["ent"] is None else s["ent"].detach().requires_grad_(True)
        loss, stats, counts = F.policy_loss(lp, s["old"], s["adv"], entropy=ent, **kw)
        loss.backward()
        out = dict(loss=loss.detach().reshape(1), stats=stats, counts=counts, dlogp=lp.grad)
        if ent is not None:
            out["dentropy"] = ent.grad
        return out
    loss, stats, counts, dlp, dent = F.flce_policy_loss(s["lp"], s["old"], s["adv"],
                                                        entropy=s["ent"], **kw)
    out = dict(loss=loss, stats=stats, counts=counts, dlogp=dlp)
    if dent is not None:
        out["dentropy"] = dent
    return out


def _run_preference_own(s):
    import linear_cross_entropy_forward_gb300 as F
    loss, rewards, dlp = F.flce_preference_loss(s["lp"], ref_logp=s["ref"], ref_scores=s["scores"],
                                                mask=s["mask"], cu_seqlens=s["cu"], **s["kw"])
    return dict(loss=loss, rewards=rewards, dlogp=dlp)


def _run_embed_own(s):
    import linear_cross_entropy_forward_gb300 as F
    return F.flce_embedding(s["ids"], s["w"], scale=s["scale"])


def _run_embed_grad_own(s):
    import linear_cross_entropy_forward_gb300 as F
    if s["dw"] is None:
        return F.flce_embedding_backward(s["dout"], s["ids"], s["case"]["V"], scale=s["scale"])
    # the head's gradient is new in each step: here, a copy of it
    dw = s["dw"].clone()
    return F.flce_embedding_backward(s["dout"], s["ids"], s["case"]["V"], scale=s["scale"],
                                     dweight=dw, accumulate=True)


def _run_head_own(s):
    import linear_cross_entropy_forward_gb300 as F
    loss, stats, counts, lp, ent, dh, dw = F.flce_policy_forward_backward(
        s["hidden"], s["weight"], s["labels"], s["old"], s["adv"], ref_logp=s["ref"],
        cu_seqlens=s["cu"], weight_layout=s["case"]["layout"], **s["kw"])
    return dict(loss=loss, stats=stats, counts=counts, logp=lp, entropy=ent, dhidden=dh,
                dweight=dw)


def run(state):
    if own:
        return {"policy": _run_policy_own, "preference": _run_preference_own,
                "embed": _run_embed_own, "embed_grad": _run_embed_grad_own,
                "head": _run_head_own}[state["case"]["op"]](state)
    return {"policy": _run_policy_plain, "preference": _run_preference_plain,
            "embed": _run_embed_plain, "embed_grad": _run_embed_grad_plain,
            "head": _run_head_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- work
def _distinct(case):
    """Expected number of distinct ids of a draw of _ids()."""
    N, V = case["N"], case["V"]
    k = np.arange(V, dtype=np.float64)
    p = (np.log(k + 2) - np.log(k + 1)) / math.log(V + 1.0) * (1.0 - case.get("pad", 0.0))
    return float((1.0 - np.exp(N * np.log1p(-np.minimum(p, 1 - 1e-12)))).sum())


def work(case):
    op = case["op"]
    if op in ("policy", "preference"):
        T = case["B"] * case["S"] if case["layout"] == "padded" else case["S"]
        b = SIZE[case["dtype"]]
        if op == "policy":
            n_in = 2 + int(case["ref"]) + int(case["ent"])
            per = b * (n_in + 1 + int(case["ent"])) + 1 + (4 if case["adv"] == "token" else 0)
            return {"bytes": T * per + 16 * case["B"], "flops": 30 * T}
        return {"bytes": T * (b * (2 + int(case["ref"] == "token")) + 1) + 16 * case["B"],
                "flops": 6 * T}
    if op == "head":
        N, H, V = case["N"], case["H"], case["V"]
        return {"bytes": 4 * N * H + 4 * H * V + 28 * N, "flops": 6 * N * H * V}
    N, H, V, b = case["N"], case["H"], case["V"], SIZE[case["dtype"]]
    if op == "embed":
        return {"bytes": 8 * N + b * H * (N + _distinct(case)), "flops": N * H}
    if case["accumulate"]:
        # the whole gradient comes out: the copy of the head's part is read and written
        return {"bytes": 8 * N + b * H * (N + 2 * V), "flops": N * H}
    return {"bytes": 8 * N + b * H * (N + V), "flops": N * H}


# ---------------------------------------------------------------------------- 64-bit values
def _exact_policy(lp, old, ref, ent, adv_tok, m, seq, B, kw):
    """The definition with automatic differentiation in 64 bits; lp and ent are leaves."""
    pick = lambda x: x[m]  # noqa: E731
    sq = pick(seq)
    n = torch.bincount(sq, minlength=B).double()
    live = n > 0
    valid, seqs = max(1, int(n.sum())), max(1, int(live.sum()))
    d0 = pick(lp) - pick(old)
    d = d0
    if kw["ratio"] == "sequence":
        d = (torch.zeros(B, dtype=torch.float64, device=lp.device).index_add(0, sq, d0)
             / n.clamp(min=1))[sq]
    a = pick(adv_tok)
    r = d.clamp(-LIMIT, LIMIT).exp()
    rc = r.clamp(1 - kw["clip_low"], 1 + kw["clip_high"])
    obj = torch.minimum(r * a, rc * a)
    clipped = rc * a < r * a
    dual = torch.zeros_like(clipped)
    if kw["dual_clip"]:
        floor = kw["dual_clip"] * a
        dual = (a < 0) & (floor > obj)
        obj = torch.where(a < 0, torch.maximum(obj, floor), obj)
    w = {"token_mean": torch.full_like(n, 1.0 / valid),
         "seq_mean_token_mean": 1.0 / (n.clamp(min=1) * seqs),
         "seq_mean_token_sum": torch.full_like(n, 1.0 / seqs),
         "sum": torch.full_like(n, kw["scale"])}[kw["aggregate"]][sq]
    pg = -(w * obj).sum()
    kl = torch.zeros_like(d0)
    if ref is not None:
        e = pick(ref) - pick(lp)
        c = e.clamp(-LIMIT, LIMIT)
        kl = {"k1": -e, "k2": e.square() / 2, "k3": torch.expm1(c) - c}[kw["kl"]]
    loss = pg + kw["kl_coef"] * (w * kl).sum()
    h = torch.zeros_like(d0) if ent is None else pick(ent)
    loss = loss - kw["entropy_coef"] * (w * h).sum()
    c0 = d0.clamp(-LIMIT, LIMIT)
    stats = torch.stack([pg, kl.sum() / valid, h.sum() / valid,
                         (torch.expm1(c0) - c0).sum() / valid])
    grads = [x for x in (lp, ent) if x is not None]
    got = torch.autograd.grad(loss, grads, allow_unused=True) if int(n.sum()) else \
        [torch.zeros_like(x) for x in grads]
    return loss.detach().reshape(1), stats.detach(), got


def exact(case, seed):
    s = prepare(case, seed)
    d64 = lambda x: None if x is None else x.detach().reshape(-1).double()  # noqa: E731
    op = case["op"]
    if op == "policy":
        lp = d64(s["lp"]).requires_grad_(True)
        ent = None if s["ent"] is None else d64(s["ent"]).requires_grad_(True)
        adv = d64(s["adv"])
        loss, stats, got = _exact_policy(lp, d64(s["old"]), d64(s["ref"]), ent,
                                         adv if case["adv"] == "token" else adv[s["seq"]],
                                         s["mask"].reshape(-1), s["seq"], case["B"], s["kw"])
        out = dict(loss=loss, stats=stats, counts=None, dlogp=got[0].view(s["lp"].shape))
        if ent is not None:
            out["dentropy"] = got[1].view(s["lp"].shape)
        return out
    if op == "preference":
        B, kw, m = case["B"], s["kw"], s["mask"].reshape(-1)
        lp = d64(s["lp"]).requires_grad_(True)
        sq = s["seq"][m]
        total = lambda x: torch.zeros(B, dtype=torch.float64, device="cuda").index_add(  # noqa: E731
            0, sq, x[m])
        n = torch.bincount(sq, minlength=B).double()
        like = total(lp)
        score = like if s["ref"] is None else like - total(d64(s["ref"]))
        if kw["length_normalised"]:
            score = score / n.clamp(min=1)
        if s["scores"] is not None:
            score = score - s["scores"].double()
        score = score * (n > 0)
        two = (lambda x: x.view(2, -1)) if kw["pairs"] == "halves" else (  # noqa: E731
            lambda x: x.view(-1, 2).t())
        (sc, sr), (nc, nr), (lc, _) = two(score), two(n), two(like)
        eps, lg = kw["label_smoothing"], torch.nn.functional.logsigmoid
        h = kw["beta"] * (sc - sr) - kw["margin"]
        per = {"sigmoid": lambda: -(1 - eps) * lg(h) - eps * lg(-h),
               "robust": lambda: ((eps - 1) * lg(h) + eps * lg(-h)) / (1 - 2 * eps),
               "hinge": lambda: torch.relu(1 - h),
               "ipo": lambda: (h / kw["beta"] - 1 / (2 * kw["beta"])).square()}[kw["loss_type"]]()
        per = per - kw["nll_coef"] * lc / nc.clamp(min=1)
        ok = (nc > 0) & (nr > 0)
        loss = (per * ok).sum() / max(1, int(ok.sum()))
        (g,) = torch.autograd.grad(loss, lp)
        return dict(loss=loss.detach().reshape(1), rewards=(kw["beta"] * score).detach(),
                    dlogp=g.view(s["lp"].shape))
    if op == "embed":
        return torch.index_select(s["w"].double(), 0, s["ids"]) * s["scale"]
    if op == "embed_grad":
        order = torch.argsort(s["ids"], stable=True)
        base = torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda") \
            if s["dw"] is None else s["dw"].double()
        for a in range(0, case["N"], 4096):
            part = order[a:a + 4096]
            base.index_add_(0, s["ids"][part], s["dout"][part].double() * s["scale"])
        return base
    if 6.0 * case["N"] * case["H"] * case["V"] > 5e12:
        return None  # over 20 seconds of 64-bit products
    h = s["hidden"].double().requires_grad_(True)
    w = s["weight"].double().requires_grad_(True)
    logits = h @ (w if case["layout"] == "hv" else w.t())
    logq = torch.log_softmax(logits, 1)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    lp = torch.where(s["mask"], logq.gather(1, s["labels"].clamp(min=0)[:, None])[:, 0], zero)
    ent = torch.where(s["mask"], -(logq.exp() * logq).sum(1), zero)
    lp_leaf, ent_leaf = (x.detach().requires_grad_(True) for x in (lp, ent))
    loss, stats, (glp, gent) = _exact_policy(lp_leaf, s["old"].double(), s["ref"].double(), ent_leaf,
                                             s["adv"].double()[s["seq"]], s["mask"], s["seq"],
                                             case["B"], s["kw"])
    gh, gw = torch.autograd.grad([lp, ent], [h, w], [glp, gent])
    return dict(loss=loss, stats=stats, counts=None, logp=lp.detach(), entropy=ent.detach(),
                dhidden=gh, dweight=gw)
