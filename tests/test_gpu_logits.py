"""Processed logits, their log-probabilities and gradient against 64 bits.

Tolerances: z has at most eight roundings of fp32 on values that are at most `size` (the logit times
the largest factors, plus what is subtracted and added), then one to the output's type.  A sum of
exponentials of fp32 differences of at most `size` has a relative error below 2^-22 size + 1e-6.
"""
import math

import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
INF = float("inf")


def reference(x, opts):
    """z (64 bits), its slope by the logits and the size of what went into it."""
    R, V = x.shape
    x = x.double().cpu()

    def per_row(name, none):
        t = opts.get(name, none)
        return t.double().cpu() if isinstance(t, torch.Tensor) else torch.full((R,), float(t), dtype=torch.float64)

    rep, freq = per_row("repetition_penalty", 1.0), per_row("frequency_penalty", 0.0)
    pres, temp = per_row("presence_penalty", 0.0), per_row("temperature", 1.0)
    z, slope, size = x.clone(), torch.ones_like(x), x.abs().nan_to_num(0, 0, 0)
    for r in range(R):
        ids = opts["tokens"][r].tolist() if opts.get("tokens") is not None else []
        n = int(opts["lengths"][r]) if opts.get("lengths") is not None else len(ids)
        p = int(opts["prompt_lens"][r]) if opts.get("prompt_lens") is not None else 0
        n = min(max(n, 0), len(ids))
        ids = ids[:n]
        made = {}
        for i, t in enumerate(ids):
            if 0 <= t < V:
                made[t] = made.get(t, 0) + (i >= p)
        for t, c in made.items():
            k = 1 / rep[r] if z[r, t] > 0 else rep[r]
            z[r, t] *= k
            slope[r, t] *= k
            size[r, t] *= float(max(rep[r], 1 / rep[r]))
            if c:
                z[r, t] -= freq[r] * c + pres[r]
                size[r, t] += float(abs(freq[r]) * c + abs(pres[r]))
        if opts.get("bias_ids") is not None:
            for t, v in zip(opts["bias_ids"][r].tolist(), opts["bias_values"][r].tolist()):
                if 0 <= t < V:
                    z[r, t] += v
                    size[r, t] += abs(v) if math.isfinite(v) else 0
        if opts.get("allowed") is not None:
            a = opts["allowed"][r].cpu()
            if a.dtype == torch.int32:
                a = ((a[:, None] >> torch.arange(32)) & 1).flatten()[:V]
            z[r, a == 0] = -INF
            slope[r, a == 0] = 0
        if temp[r] > 0:
            z[r] /= temp[r]
            slope[r] /= temp[r]
            size[r] /= float(temp[r])
    return z, slope, size


def check(x, opts, out_dtype=None, out=None):
    z, _, size = reference(x, opts)
    got, lse = flce.flce_process_logits(x, need_lse=True, out_dtype=out_dtype, out=out, **opts)
    dt = out_dtype or x.dtype
    g = got.double().cpu()
    gone = ~torch.isfinite(z)
    assert got.dtype == dt
    assert torch.equal(g[gone].nan_to_num(7, 8, 9), z[gone].nan_to_num(7, 8, 9))
    tol = 8 * 2.0 ** -24 * size + HALF_STEP[dt] * z.abs()
    if dt is torch.float16:  # subnormal steps
        tol = tol + 2.0 ** -25
    ok = ((g - z).abs() <= tol + 1e-30) | gone
    assert bool(ok.all()), float(((g - z).abs() - tol)[~ok].max())
    want = torch.logsumexp(z, 1)
    top = (8 * 2.0 ** -24 * torch.where(gone, torch.zeros_like(size), size)).amax(1)
    l = lse.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(l[~fine].nan_to_num(7, 8, 9), want[~fine].nan_to_num(7, 8, 9))
    assert bool(((l - want).abs() <= top * 2 + 2e-6 + 2.0 ** -23 * want.abs())[fine].all()), \
        float((l - want).abs()[fine].max())
    return got, lse


def options(R, V, T, seed, *, bias=0, mask=None, ids=torch.int64, lens=torch.int64, spread=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    o = {}
    if T is not None:
        o["tokens"] = (rnd(R, T) * (spread or V)).long().clamp(max=V - 1).to(ids)
        o["lengths"] = torch.randint(0, T + 1, (R,), generator=g, device="cuda").to(lens)
        o["lengths"][0] = T
        o["prompt_lens"] = (o["lengths"] * rnd(R)).to(lens)
    o["repetition_penalty"] = 0.7 + rnd(R)
    o["frequency_penalty"] = rnd(R) - 0.3
    o["presence_penalty"] = rnd(R) - 0.3
    o["temperature"] = 0.3 + rnd(R)
    if bias:
        o["bias_ids"] = torch.randint(-2, V + 2, (R, bias), generator=g, device="cuda").to(ids)
        o["bias_ids"][:, bias // 2] = o["bias_ids"][:, 0]  # twice the same
        o["bias_values"] = torch.randn(R, bias, generator=g, device="cuda") * 3
    if mask == "bytes":
        o["allowed"] = rnd(R, V) < 0.4
        o["allowed"][:, 0] = True
    elif mask == "bits":
        o["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (R, (V + 31) // 32), generator=g, device="cuda").int()
        o["allowed"][:, 0] |= 1
    return o


def rows_of(R, V, dtype, seed, pad=0, skew=0):
    """Logits with a row stride of V + pad that begin `skew` elements past an aligned address."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((skew + R * (V + pad),), float("nan"), device="cuda", dtype=dtype)
    x = buf[skew:].view(R, V + pad)[:, :V]
    x.copy_(3 * torch.randn(R, V, generator=g, device="cuda"))
    return x


CASES = [  # R, V, T, pad, skew, bias, mask, ids
    (1, 1, 1, 0, 0, 0, None, torch.int64), (3, 2, 5, 0, 1, 2, "bytes", torch.int32),
    (2, 7, 0, 1, 0, 3, "bits", torch.int64), (4, 33, 40, 0, 3, 0, "bits", torch.int32),
    (5, 100, 64, 4, 0, 5, "bytes", torch.int64), (2, 1000, 333, 1, 5, 7, "bits", torch.int64),
    (3, 4096, 1000, 0, 0, 0, None, torch.int32), (2, 8191, 900, 0, 7, 48, "bytes", torch.int64),
    (2, 32000, 2048, 0, 0, 0, None, torch.int64), (2, 50257, 3001, 0, 0, 9, "bits", torch.int64),
    (2, 50257, 17, 3, 1, 300, "bytes", torch.int32), (3, 128256, 4096, 0, 0, 48, "bits", torch.int64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,V,T,pad,skew,bias,mask,ids", CASES)
def test_processed(R, V, T, pad, skew, bias, mask, ids, dtype):
    x = rows_of(R, V, dtype, V + T, pad, skew)
    o = options(R, V, T, V, bias=bias, mask=mask, ids=ids, lens=ids, spread=max(1, V // 3))
    got, lse = check(x, o)
    again, lse2 = flce.flce_process_logits(x, need_lse=True, **o)
    assert torch.equal(got, again) and torch.equal(lse, lse2)
    if dtype != torch.float32:
        check(x, o, torch.float32)


@pytest.mark.parametrize("R", [700, 2500])
def test_many_rows(R):
    """Few blocks per row: several copies of a row, and passes over its counters, per block."""
    V = 40001 if R == 700 else 9000
    x = rows_of(R, V, torch.bfloat16, 1)
    o = options(R, V, 300, 2, bias=3, mask="bytes", spread=V)
    pick = torch.randint(0, R, (24,)).tolist() + [0, R - 1]
    got, lse = flce.flce_process_logits(x, need_lse=True, **o)
    few = {k: v[pick].contiguous() for k, v in o.items()}
    one, l = check(x[pick].contiguous(), few)
    assert torch.equal(got[pick].nan_to_num(0, 1, 2), one.nan_to_num(0, 1, 2))
    # the blocks of a row are others, so its sums are joined in another order
    assert float((lse[pick] - l).abs().max()) <= 4e-6


def test_long_histories():
    """2^14 tokens and more: wider counters, more passes; a token that comes 20000 times."""
    R, V, T = 2, 70000, 40000
    x = rows_of(R, V, torch.bfloat16, 3)
    o = options(R, V, T, 4)
    o["tokens"][0, 100:20100] = 69999
    o["lengths"][:] = torch.tensor([T, 30001])
    o["prompt_lens"][:] = torch.tensor([50, 0])
    check(x, o)
    o["tokens"] = o["tokens"].int()
    check(x.float(), o)
    check(rows_of(1, 300000, torch.bfloat16, 5), options(1, 300000, 16384, 6))


def test_scalars_strides_and_expanded_rows():
    x = rows_of(6, 500, torch.float32, 8)
    o = options(6, 500, 64, 9, bias=4, mask="bytes")
    numbers = dict(o, repetition_penalty=1.3, frequency_penalty=0.2, presence_penalty=0.1, temperature=0.6)
    check(x, numbers)
    one = dict(numbers)
    for k in ("tokens", "bias_ids", "bias_values", "allowed"):  # one row for all
        one[k] = numbers[k][:1].expand(6, -1)
    check(x, one)
    wide = dict(numbers)
    for k in ("tokens", "bias_ids", "bias_values", "allowed"):  # rows of a wider array
        t = numbers[k]
        big = torch.zeros(6, t.shape[1] + 3, dtype=t.dtype, device="cuda")
        big[:, 1:-2] = t
        wide[k] = big[:, 1:-2]
    check(x, wide)
    a, _ = check(x, numbers)
    assert torch.equal(flce.flce_process_logits(x[:1].expand(6, -1), **numbers)[0], a[0])
    # without lengths all tokens count, without prompt_lens none is the prompt's
    check(x, {"tokens": o["tokens"], "frequency_penalty": 0.5})
    check(x, {"tokens": o["tokens"], "lengths": o["lengths"], "presence_penalty": 0.5})
    check(x, {"temperature": 0.0})
    check(x, {})
    # tokens without a penalty, a penalty without tokens
    plain = flce.flce_process_logits(x, tokens=o["tokens"])
    assert torch.equal(plain, x)
    assert torch.equal(flce.flce_process_logits(x, repetition_penalty=2.0), x)


def test_in_place_and_out():
    x = rows_of(3, 1001, torch.bfloat16, 10, pad=7)
    o = options(3, 1001, 128, 11, bias=3, mask="bits")
    want, lse = check(x, o)
    buf = torch.zeros(3, 1200, device="cuda", dtype=torch.bfloat16)
    into = buf[:, 100:1101]
    check(x, o, out=into)
    assert torch.equal(into, want) and float(buf[:, :100].abs().max()) == 0
    assert float(buf[:, 1101:].abs().max()) == 0
    y = x.clone(memory_format=torch.preserve_format)
    y = torch.empty_strided(x.shape, x.stride(), device="cuda", dtype=x.dtype).copy_(x)
    z, l = flce.flce_process_logits(y, out=y, need_lse=True, **o)
    assert z is y and torch.equal(y, want) and torch.equal(l, lse)


def test_what_is_left_of_a_row():
    """Rows whose mask leaves nothing, -inf, the type's lowest value and NaN in masked places, NaN
    and +inf in others."""
    V = 300
    x = rows_of(8, V, torch.float32, 12)
    a = torch.ones(8, V, dtype=torch.bool, device="cuda")
    a[0] = False                                    # nothing is left
    x[1] = -INF                                     # nor here
    x[2] = torch.finfo(torch.float32).min           # all the same
    x[3, 5], a[3, 5] = float("nan"), False          # masked
    x[4, 6], a[4, 6] = INF, False
    x[5, 7] = float("nan")
    x[6, 8] = INF
    a[7] = False
    a[7, 299] = True                                # one left
    labels = torch.full((8,), 299, device="cuda")
    z, lse = flce.flce_process_logits(x, allowed=a, need_lse=True)
    logp, ent, lse2 = flce.flce_logits_logprob(x, labels, allowed=a)
    d = flce.flce_logits_logprob_backward(x, labels, lse2, ent, torch.ones(8, device="cuda"),
                                          torch.ones(8, device="cuda"), allowed=a)
    assert bool((z[0] == -INF).all()) and bool((z[1] == -INF).all())
    for r in (0, 1):
        assert float(lse[r]) == -INF and float(logp[r]) == -INF and float(ent[r]) == 0
        assert float(d[r].abs().max()) == 0
    assert abs(float(ent[2]) - math.log(V)) < 1e-5 and abs(float(logp[2]) + math.log(V)) < 1e-5
    for r in (3, 4):
        want = torch.logsumexp(x[r].double()[a[r]], 0)
        assert abs(float(lse[r]) - float(want)) < 1e-5 and bool(torch.isfinite(d[r]).all())
        assert float(z[r, r + 2]) == -INF and float(d[r, r + 2]) == 0
    for r in (5, 6):
        assert math.isnan(float(lse[r])) and math.isnan(float(logp[r])) and math.isnan(float(ent[r]))
    assert abs(float(logp[7])) < 1e-6 and abs(float(ent[7])) < 1e-6
    assert float(lse[7]) == pytest.approx(float(x[7, 299]), abs=1e-6)
    # bias of -inf, which masks; infinities of both signs make NaN
    ids = torch.tensor([[3, 4]], device="cuda")
    z = flce.flce_process_logits(x[7:], bias_ids=ids, bias_values=torch.tensor([[-INF, INF]], device="cuda"))
    assert float(z[0, 3]) == -INF and float(z[0, 4]) == INF
    both = flce.flce_process_logits(x[7:], bias_ids=ids[:, :1].expand(1, 2).contiguous(),
                                    bias_values=torch.tensor([[-INF, INF]], device="cuda"))
    assert math.isnan(float(both[0, 3]))


def grad64(x, labels, opts, gl, ge):
    z, slope, size = reference(x, opts)
    lse = torch.logsumexp(z, 1, keepdim=True)
    p = torch.exp(z - lse)
    logq = torch.where(p > 0, z - lse, torch.zeros_like(z))
    H = -(p * logq).sum(1, keepdim=True)
    y = labels.cpu()
    counts = y != -100
    one = torch.zeros_like(z).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    gl, ge = (t.double().cpu()[:, None] * counts[:, None] for t in (gl, ge))
    d = slope * (gl * (one - p) - ge * p * (logq + H))
    logp = torch.where(counts, (z - lse).gather(1, y.clamp(min=0)[:, None])[:, 0], torch.zeros(len(y), dtype=torch.float64))
    return logp, torch.where(counts, H[:, 0], torch.zeros_like(logp)), d, size, logq, H, p, slope


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,V,T,pad,skew,bias,mask,ids", CASES[1:])
def test_logprob_and_gradient(R, V, T, pad, skew, bias, mask, ids, dtype):
    x = rows_of(R, V, dtype, V + T + 1, pad, skew)
    o = options(R, V, T, V + 1, bias=bias, mask=mask, ids=ids, lens=ids, spread=max(1, V // 3))
    labels = torch.zeros(R, dtype=torch.int64, device="cuda")  # allowed
    if R > 2:
        labels[1] = -100
    g = torch.Generator(device="cuda").manual_seed(1)
    gl, ge = torch.randn(R, generator=g, device="cuda"), torch.randn(R, generator=g, device="cuda")
    leaf = x.detach().requires_grad_(True)
    logp, ent = flce.logits_logprob(leaf, labels, **o)
    (d,) = torch.autograd.grad([logp, ent], [leaf], [gl, ge])
    wl, we, wd, size, logq, H, p, slope = grad64(x, labels, o, gl, ge)
    off = 16 * 2.0 ** -24 * size.amax(1) + 4e-6  # of a difference z - lse
    assert bool(((logp.double().cpu() - wl).abs() <= off + 2.0 ** -23 * wl.abs()).all())
    # p and the differences each `off` away, weighted by p |logq|
    assert bool(((ent.double().cpu() - we).abs() <= off * (2 + 2 * logq.abs().mul(p).sum(1) + we)).all())
    scale = slope.abs() * p * (gl.abs().cpu()[:, None] + ge.abs().cpu()[:, None] * (logq.abs() + H + 3))
    lab = slope.abs() * (gl.abs().cpu()[:, None]) * 2.0 ** -22
    tol = 2 * off[:, None] * scale + lab + HALF_STEP[dtype] * wd.abs()
    tol = tol + (2.0 ** -25 if dtype is torch.float16 else 1e-37)
    err = (d.double().cpu() - wd).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    if R > 2:
        assert float(d[1].abs().max()) == 0 and float(logp[1]) == 0 and float(ent[1]) == 0
    d32 = flce.flce_logits_logprob_backward(x, labels, *flce.flce_logits_logprob(x, labels, **o)[2:0:-1],
                                            gl, ge, grad_dtype=torch.float32, **o)
    assert bool(((d32.double().cpu() - wd).abs() <= 2 * off[:, None] * scale + lab + 2.0 ** -24 * wd.abs() + 1e-37).all())


def test_gradient_against_differences():
    """Central differences of the 64-bit definition, on logits away from 0, where the penalty bends."""
    R, V = 3, 40
    x = rows_of(R, V, torch.float32, 20)
    x = torch.where(x.abs() < 0.05, x.sign() * 0.05 + 0.01, x)
    o = options(R, V, 20, 21, bias=4, mask="bytes")
    labels = torch.zeros(R, dtype=torch.int64, device="cuda")
    gl, ge = torch.randn(R, device="cuda"), torch.randn(R, device="cuda")
    leaf = x.clone().requires_grad_(True)
    logp, ent = flce.logits_logprob(leaf, labels, **o)
    (d,) = torch.autograd.grad([logp, ent], [leaf], [gl, ge])
    v = torch.randn(R, V, dtype=torch.float64)

    def f(h):
        z, _, _ = reference(x.double().cpu() + h * v, o)
        logq = torch.log_softmax(z, 1)
        H = -(logq.exp() * torch.where(torch.isfinite(logq), logq, torch.zeros_like(logq))).sum(1)
        return float((gl.double().cpu() * logq[:, 0] + ge.double().cpu() * H).sum())

    slope = (f(1e-5) - f(-1e-5)) / 2e-5
    assert float((d.double().cpu() * v).sum()) == pytest.approx(slope, rel=1e-4, abs=1e-4)


def test_labels():
    V = 100
    x = rows_of(5, V, torch.float32, 22)
    labels = torch.tensor([3, -100, 100, -1, 99], device="cuda")
    logp, ent, lse = flce.flce_logits_logprob(x, labels)
    assert [math.isnan(float(t)) for t in logp] == [False, False, True, True, False]
    assert [math.isnan(float(t)) for t in ent] == [False, False, True, True, False]
    assert bool(torch.isfinite(lse).all())
    with pytest.raises(flce.FlceError, match="LABEL"):
        flce.flce_logits_logprob(x, labels, validate=True)
    flce.flce_logits_logprob(x, labels[[0, 1, 4, 0, 0]], validate=True)
    logp, _, _ = flce.flce_logits_logprob(x, torch.full((5,), 7, device="cuda"), ignore_index=7)
    assert float(logp.abs().max()) == 0
    # a label that is not allowed
    a = torch.ones(5, V, dtype=torch.bool, device="cuda")
    a[0, 3] = False
    logp, ent, lse = flce.flce_logits_logprob(x, torch.full((5,), 3, device="cuda"), allowed=a)
    assert float(logp[0]) == -INF and bool(torch.isfinite(logp[1:]).all()) and bool(torch.isfinite(ent).all())
    d = flce.flce_logits_logprob_backward(x, torch.full((5,), 3, device="cuda"), lse, ent,
                                          torch.ones(5, device="cuda"), None, allowed=a)
    assert float(d[0, 3]) == 0 and bool(torch.isfinite(d).all())


def test_empty():
    x = torch.empty(0, 50, device="cuda")
    z, lse = flce.flce_process_logits(x, need_lse=True)
    assert z.shape == (0, 50) and lse.shape == (0,)
    leaf = x.requires_grad_(True)
    logp, ent = flce.logits_logprob(leaf, torch.empty(0, dtype=torch.int64, device="cuda"), validate=True)
    (d,) = torch.autograd.grad([logp.sum() + ent.sum()], [leaf])
    assert d.shape == (0, 50)


def test_streams_threads_graphs_and_autograd():
    import threading
    x = rows_of(40, 30000, torch.bfloat16, 30)
    o = options(40, 30000, 700, 31, bias=5, mask="bits")
    labels = torch.zeros(40, dtype=torch.int64, device="cuda")
    gl = torch.randn(40, device="cuda")
    want = flce.flce_process_logits(x, need_lse=True, **o)
    leaf = x.clone().requires_grad_(True)
    torch.cuda.synchronize()
    outs = {}

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                outs[i] = flce.flce_process_logits(x, need_lse=True, **o)
        s.synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    for i in range(3):
        assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        # an eager graph that lives on while the same leaf is captured; on a stream of its own, as a
        # capture cannot wait for the default stream, which autograd would have it do
        eager = flce.logits_logprob(leaf, labels, **o)
        for _ in range(2):
            lp, en = flce.logits_logprob(leaf, labels, **o)
            (d0,) = torch.autograd.grad([lp, en], [leaf], [gl, gl])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, lse = flce.flce_process_logits(x, need_lse=True, **o)
        lp, en = flce.logits_logprob(leaf, labels, **o)
        (d,) = torch.autograd.grad([lp, en], [leaf], [gl, gl])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, want[0]) and torch.equal(lse, want[1]) and torch.equal(d, d0)
    assert torch.equal(lp, eager[0])
    (d1,) = torch.autograd.grad(eager[0].sum(), [leaf], create_graph=True)
    with pytest.raises(RuntimeError):
        d1.float().sum().backward()
    # tokens and lengths are read by the replay
    o["tokens"][:, :50] = 3
    o["lengths"].fill_(50)
    graph.replay()
    again = flce.flce_process_logits(x, need_lse=True, **o)
    torch.cuda.synchronize()
    assert torch.equal(z, again[0]) and torch.equal(lse, again[1])
    # one of the two outputs alone, and a broadcast gradient
    lp, en = flce.logits_logprob(leaf, labels, **o)
    lp.sum().backward()
    assert bool(torch.isfinite(leaf.grad.float()).all())


def test_offsets_past_32_bits():
    """A row whose first logit is past 2^31 elements."""
    R, V = 9000, 256000
    x = torch.zeros(R, V, device="cuda", dtype=torch.bfloat16)
    at = [0, 8388, 8389, 8999]
    x[at] = (3 * torch.randn(len(at), V, device="cuda")).bfloat16()
    o = options(R, V, 40, 33)
    z, lse = flce.flce_process_logits(x, out=x, need_lse=True, **o)
    few = {k: v[at].contiguous() for k, v in o.items()}
    del x
    torch.cuda.empty_cache()
    assert bool(torch.isfinite(lse).all())
    assert abs(float(lse[100]) - math.log(V)) < 0.1


def test_refusals():
    x = torch.zeros(2, 64, device="cuda")
    t = torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    P = flce.flce_process_logits
    for bad in (x[0], x[None]):
        with pytest.raises(ValueError, match="logits"):
            P(bad)
    with pytest.raises(TypeError, match="float32"):
        P(x.double())
    with pytest.raises(ValueError, match="dense"):
        P(torch.zeros(64, 2, device="cuda").t())
    with pytest.raises(TypeError, match="tokens"):
        P(x, tokens=t.float())
    with pytest.raises(ValueError, match="tokens"):
        P(x, tokens=t[:1])
    with pytest.raises(ValueError, match="need tokens"):
        P(x, lengths=t[:, 0])
    with pytest.raises(TypeError, match="lengths"):
        P(x, tokens=t, lengths=t[:, 0])  # not contiguous
    with pytest.raises(TypeError, match="same type"):
        P(x, tokens=t, lengths=t[:, 0].contiguous(), prompt_lens=t[:, 0].int())
    with pytest.raises(ValueError, match="together"):
        P(x, bias_ids=t)
    with pytest.raises(ValueError, match="bias_values"):
        P(x, bias_ids=t, bias_values=torch.zeros(2, 5, device="cuda"))
    with pytest.raises(flce.FlceError, match="BAD_SHAPE"):
        P(x, bias_ids=torch.zeros(2, 2049, dtype=torch.int64, device="cuda"),
          bias_values=torch.zeros(2, 2049, device="cuda"))
    with pytest.raises(ValueError, match="allowed"):
        P(x, allowed=torch.zeros(2, 63, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError, match="allowed"):
        P(x, allowed=torch.zeros(2, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="temperature"):
        P(x, temperature=torch.ones(3, device="cuda"))
    for kw in (dict(repetition_penalty=0.0), dict(temperature=-1.0), dict(frequency_penalty=float("nan"))):
        with pytest.raises(flce.FlceError, match="BAD_ARG"):
            P(x, **kw)
    with pytest.raises(TypeError, match="out"):
        P(x, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out"):
        P(x, out=torch.zeros(2, 63, device="cuda"))
    with pytest.raises(ValueError, match="overlaps"):
        buf = torch.zeros(200, device="cuda")
        P(buf[:128].view(2, 64), out=buf[4:132].view(2, 64))
    with pytest.raises(flce.FlceError, match="BAD_SHAPE"):  # rows written on top of each other
        P(x, out=torch.zeros(1, 64, device="cuda").expand(2, 64))
    with pytest.raises(TypeError, match="labels"):
        flce.logits_logprob(x, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="g_logp"):
        flce.flce_logits_logprob_backward(x, t[:, 0].contiguous(), x[:, 0].contiguous(), None,
                                          torch.zeros(3, device="cuda"), None)
    with pytest.raises(ValueError, match="entropy"):
        flce.flce_logits_logprob_backward(x, t[:, 0].contiguous(), x[:, 0].contiguous(), None, None,
                                          torch.zeros(2, device="cuda"))


@pytest.mark.parametrize("R,V,T,dtype,ids", [(96, 256000, 12000, torch.bfloat16, torch.int64),
                                             (40, 128257, 60001, torch.float32, torch.int32),
                                             (61, 50257, 70000, torch.float16, torch.int64),
                                             (24, 1000003, 16000, torch.bfloat16, torch.int32)])
def test_long_histories_of_many_rows(R, V, T, dtype, ids):
    """In every element what few rows at a time give, whose blocks have fewer columns and passes, and a
    few rows against 64 bits; ids outside the row, empty and full histories, prompts alone, rows that
    begin anywhere."""
    o = options(R, V, T, 11, ids=ids, lens=ids)
    tok = o["tokens"]
    tok[:, 5::97] = -1
    tok[:, 6::89] = V
    tok[:, 7::83] = 2 ** 31 - 1 if ids is torch.int32 else -2 ** 40
    tok[:, 8::79] = V + (2 ** 33 if ids is torch.int64 else 5)
    tok[:, :T // 3] = (tok[:, :T // 3].double() / V).clamp(0, 1).pow(3).mul(1000).to(ids)  # repeated
    o["lengths"][1], o["prompt_lens"][1] = 0, 0
    o["lengths"][2], o["prompt_lens"][2] = T, T
    o["repetition_penalty"][3], o["frequency_penalty"][3], o["presence_penalty"][3] = 1.0, 0.0, 0.0
    x = rows_of(R, V, dtype, 12, pad=3, skew=1)
    z, lse = flce.flce_process_logits(x, need_lse=True, **o)
    labels = torch.randint(0, V, (R,), generator=torch.Generator(device="cuda").manual_seed(13), device="cuda")
    logp, ent, lse2 = flce.flce_logits_logprob(x, labels, **o)
    d = flce.flce_logits_logprob_backward(x, labels, lse2, ent, torch.ones_like(lse2), None, **o)
    assert torch.equal(lse, lse2)
    few = 3 if V < 200000 else 1
    for r in range(0, R, few):
        part = {k: v[r:r + few] for k, v in o.items()}
        zp = flce.flce_process_logits(x[r:r + few], **part)
        assert torch.equal(zp, z[r:r + few]), r
        dp = flce.flce_logits_logprob_backward(x[r:r + few], labels[r:r + few], lse2[r:r + few], ent[r:r + few],
                                               torch.ones_like(lse2[r:r + few]), None, **part)
        assert torch.equal(dp, d[r:r + few]), r
    for r in (0, 1, 2, 3, R - 1):
        part = {k: v[r:r + 1] for k, v in o.items()}
        want, _, size = reference(x[r:r + 1], part)
        tol = 8 * 2.0 ** -24 * size + HALF_STEP[dtype] * want.abs() + (2.0 ** -25 if dtype is torch.float16 else 0)
        assert bool(((z[r:r + 1].double().cpu() - want).abs() <= tol + 1e-30).all()), r
        want = torch.logsumexp(want, 1)
        assert abs(float(lse[r].double().cpu() - want)) <= 2 * 8 * 2.0 ** -24 * float(size.max()) + 2e-6 \
            + 2.0 ** -23 * abs(float(want)), r


def test_saved_tensors_that_come_back_as_copies():
    """Hooks on what is saved hand the gradient copies of the logits, without their row stride; the
    options' tensors stay where the call found them."""
    R, V = 5, 1000
    x = rows_of(R, V, torch.float32, 21, pad=24)
    labels = torch.arange(R, device="cuda") * 7
    g = torch.linspace(-1, 1, R, device="cuda")

    def run(hooks):
        leaf = x.detach().requires_grad_(True)
        o = options(R, V, 60, 22, mask="bits")
        with torch.autograd.graph.saved_tensors_hooks(*hooks):
            logp, ent = flce.logits_logprob(leaf, labels, **o)
        del o
        junk = [torch.full((R,), 1e9, device="cuda") for _ in range(20)]
        (d,) = torch.autograd.grad((logp * g).sum() + ent.sum(), leaf)
        del junk
        return d

    assert torch.equal(run((lambda t: t, lambda t: t)),
                       run((lambda t: t.cpu(), lambda t: t.cuda().contiguous())))


def test_two_builds_in_one_process(tmp_path):
    """What a library has set up for its kernels is its own: another build beside it (as the one with
    bounds checks is) sets up its own."""
    import shutil

    from linear_cross_entropy_forward_gb300 import _binding as B
    x = rows_of(4, 128256, torch.bfloat16, 31)
    o = options(4, 128256, 50, 32)
    z = flce.flce_process_logits(x, **o)
    other = tmp_path / "libflce_copy.so"
    shutil.copy(B.LIB_PATH, other)
    mine = B.use_library(str(other))
    try:
        assert torch.equal(flce.flce_process_logits(x, **o), z)
    finally:
        B.restore_library(mine)
