"""The optimizer's step and the gradients' norm against 64 bits.

Tolerances: m and v are two products and a sum in fp32 (4 half steps of 2^-24 of their terms), a
weight moves by lr u with |u| computed to 2^-19 (a root, a reciprocal and the bias corrections, a few
units in the last place each); the factor 1 - lr decay, the weight's product with it and the sum are
a rounding each, 3 * 2^-24 of the weight together, and it is rounded once to its own type.  An 8-bit code is one of the two
neighbours of the exact quotient: a whole step of 1/8 of its binade off at most.
"""
import math

import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
B1, B2, EPS, LR = 0.9, 0.98, 1e-8, 1e-2


def params(sizes, dtype, seed=0, skew=0, scale=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n in sizes:
        buf = torch.empty(n + skew, device="cuda", dtype=dtype)
        out.append(buf[skew:].copy_(scale * torch.randn(n, generator=g, device="cuda")))
    return out


def grads(sizes, dtype, seed, skew=0):
    out = params(sizes, dtype, seed, skew, 1.0)
    for i, t in enumerate(out):
        t.mul_(10.0 ** (i % 5 - 3))
    return out


def update(w, g, m, v, t, c, decay, lr=LR, eps=EPS):
    """One step in 64 bits."""
    g = g.double() * c
    m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
    u = (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)).sqrt() + eps)
    return w * (1 - lr * decay) - lr * u, m, v, u


SIZES = [1, 7, 8, 127, 128, 129, 1000, 2047, 2048, 2049, 40000, 300001]


@pytest.mark.parametrize("dtype,gdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                          (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
                                          (torch.float16, torch.float32)])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("skew", [0, 1])
def test_32_bit_states(dtype, gdtype, master, skew):
    ps = params(SIZES, dtype, 1, skew)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    opt = flce.AdamW(ps, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay, master=master, max_norm=2.0)
    if master:  # what the masters know and the parameters do not
        g = torch.Generator(device="cuda").manual_seed(77)
        for p, at in zip(ps, opt.offsets):
            opt.master[at:at + p.numel()] += 1e-4 * torch.randn(p.numel(), generator=g, device="cuda")
    ws = [(opt.master[at:at + p.numel()] if master else p).double().clone() for p, at in zip(ps, opt.offsets)]
    ms, vs = [torch.zeros_like(w) for w in ws], [torch.zeros_like(w) for w in ws]
    for t in (1, 2, 3):
        gs = grads(SIZES, gdtype, 10 + t, skew)
        exact = math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))
        norm = opt.step(gs)
        assert abs(float(norm) - exact) <= 1e-6 * exact
        c = min(1.0, 2.0 / (exact + 1e-6))
        state = opt.state_dict()
        for i, (p, g, at) in enumerate(zip(ps, gs, opt.offsets)):
            start = ws[i] if master or t == 1 else before[i]
            w, m, v, u = update(start, g, ms[i], vs[i], t, c, decay[i])
            span = slice(at, at + p.numel())
            gm, gv = state["exp_avg"][span].double(), state["exp_avg_sq"][span].double()
            big = ms[i].abs() + (c * g.double()).abs()
            assert bool(((gm - m).abs() <= 2.0 ** -22 * big).all())
            assert bool(((gv - v).abs() <= 2.0 ** -21 * v + 1e-37).all())
            tol = LR * u.abs() * 2.0 ** -19 + LR * 2.0 ** -21 * (big / (1 - B1 ** t)) \
                / ((v / (1 - B2 ** t)).sqrt() + EPS) + 3 * 2.0 ** -24 * start.abs()
            if master:
                gw = state["master"][span].double()
                assert bool(((gw - w).abs() <= tol).all()), (t, i, float((gw - w).abs().max()))
                assert torch.equal(p, state["master"][span].to(dtype))
                ws[i] = gw.clone()
            else:
                floor = 2.0 ** -25 if dtype is torch.float16 else 0.0
                assert bool(((p.double() - w).abs() <= tol * 1.01 + HALF[dtype] * w.abs() + floor).all())
            ms[i], vs[i] = gm.clone(), gv.clone()
        before = [p.double().clone() for p in ps]
        assert int(state["step"]) == t
        for name in ("exp_avg", "exp_avg_sq") + (("master",) if master else ()):
            for n, at in zip(SIZES, opt.offsets):  # what is behind a tensor's last element
                pad = state[name][at + n:at + -(-n // 128) * 128]
                assert pad.numel() == 0 or float(pad.abs().max()) == 0


def decode(codes, scale):
    return (codes.float().view(-1, 128).double() * scale.double()[:, None]).view(-1)


@pytest.mark.parametrize("dtype,gdtype,master,skew", [
    (torch.float32, torch.float32, False, 0), (torch.bfloat16, torch.bfloat16, True, 0),
    (torch.bfloat16, torch.float32, False, 1), (torch.float16, torch.float16, True, 1)])
def test_8_bit_states(dtype, gdtype, master, skew):
    ps = params(SIZES, dtype, 2, skew)
    opt = flce.AdamW(ps, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.1, state_bits=8, master=master, seed=5)
    for t in (1, 2, 3):
        old = {k: v.clone() for k, v in opt.state_dict().items() if v is not None}
        start = [(old["master"][at:at + p.numel()] if master else p).double().clone()
                 for p, at in zip(ps, opt.offsets)]
        gs = grads(SIZES, gdtype, 20 + t, skew)
        assert opt.step(gs) is None
        new = opt.state_dict()
        m0 = decode(old["exp_avg"], old["exp_avg_scale"])
        v0 = decode(old["exp_rms"], old["exp_rms_scale"]) ** 2
        for i, (p, g, at) in enumerate(zip(ps, gs, opt.offsets)):
            span = slice(at, at + p.numel())
            w, m, v, u = update(start[i], g, m0[span], v0[span], t, 1.0, 0.1)
            big = (m0[span].abs() + g.double().abs()) / (1 - B1 ** t)
            tol = LR * u.abs() * 2.0 ** -19 + LR * 2.0 ** -21 * big / ((v / (1 - B2 ** t)).sqrt() + EPS) \
                + 3 * 2.0 ** -24 * start[i].abs()
            if master:
                assert bool(((new["master"][span].double() - w).abs() <= tol).all())
                assert torch.equal(p, new["master"][span].to(dtype))
            else:
                assert bool(((p.double() - w).abs() <= tol * 1.01 + HALF[dtype] * w.abs()).all())
            for name, x in (("exp_avg", m), ("exp_rms", v.sqrt())):
                n, blocks = p.numel(), -(-p.numel() // 128)
                full = torch.zeros(blocks * 128, dtype=torch.float64, device="cuda")
                full[:n] = x
                top = full.view(-1, 128).abs().amax(1)
                scale = new[name + "_scale"][at // 128:at // 128 + blocks].double()
                assert bool(((scale - top / 448).abs() <= 2.0 ** -20 * top / 448).all())
                codes = new[name][at:at + blocks * 128].float().double()
                q = full / (top / 448).repeat_interleave(128).clamp(min=1e-300)
                step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
                assert bool(((codes - q).abs() <= step * (1 + 1e-5) + 1e-5 * q.abs()).all())
                assert bool((codes[n:] == 0).all())
                assert bool(((codes * q) >= 0).all())
                if name == "exp_rms":
                    assert bool((codes[:n][full[:n] > 0] >= 2.0 ** -9).all())


def test_8_bit_rounding_keeps_the_mean():
    """Elements that sit between two codes: over many of them the mean is that of what was rounded,
    to five standard deviations (a code is up to half a step off on average, 1/8 of the value at
    most, over 2^17 elements)."""
    n = 1 << 17
    p = [torch.zeros(n, device="cuda")]
    opt = flce.AdamW(p, lr=0.0, betas=(0.0, 0.0), weight_decay=0.0, state_bits=8, seed=9)
    g = torch.full((n,), 0.07, device="cuda")
    g[::128] = 1.0  # each block's largest
    opt.step([g])
    s = opt.state_dict()
    small = torch.ones(n, dtype=torch.bool, device="cuda")
    small[::128] = False
    for name in ("exp_avg", "exp_rms"):
        x = decode(s[name], s[name + "_scale"])
        assert float((x[~small] - 1).abs().max()) < 1e-6
        assert len(torch.unique(s[name].float()[small])) == 2
        assert abs(float(x[small].mean()) - 0.07) <= 5 * 0.07 / 16 / math.sqrt(n) + 1e-7
    # another seed and another step round other elements up; the same ones repeat
    first = s["exp_avg"].float().clone()
    for seed, steps, same in ((9, 1, True), (10, 1, False), (9, 2, False)):
        other = flce.AdamW(p, lr=0.0, betas=(0.0, 0.0), weight_decay=0.0, state_bits=8, seed=seed)
        for _ in range(steps):
            other.step([g])
        differ = float((other.state_dict()["exp_avg"].float() != first).float().mean())
        assert (differ == 0) if same else (differ > 0.1)
    # a slow decay is followed on the average: 2 % a step for 30 steps, of a code whose neighbours are
    # 7 % away (each element 3 % off per step at random, 2^17 elements)
    opt = flce.AdamW(p, lr=0.0, betas=(0.98, 0.98), weight_decay=0.0, state_bits=8, seed=11)
    opt.state_dict()["exp_avg"].copy_(s["exp_avg"])
    opt.state_dict()["exp_avg_scale"].copy_(s["exp_avg_scale"])
    start = float(decode(s["exp_avg"], s["exp_avg_scale"])[small].mean())
    keep = torch.zeros(n, device="cuda")
    keep[::128] = 1.0  # the blocks' largest stay where they are
    for _ in range(30):
        opt.step([keep])
    now = opt.state_dict()
    mean = float(decode(now["exp_avg"], now["exp_avg_scale"])[small].mean())
    assert abs(mean / (start * 0.98 ** 30) - 1) <= 5 * 0.125 * math.sqrt(30) / math.sqrt(n) + 1e-4


def test_many_tensors_and_empty_ones():
    """More tensors than a launch's arguments hold, with empty ones among them."""
    sizes = [(i * 37) % 300 for i in range(1500)]
    ps = params(sizes, torch.bfloat16, 3)
    gs = grads(sizes, torch.bfloat16, 4)
    opt = flce.AdamW(ps, lr=LR, betas=(B1, B2), weight_decay=0.0, max_norm=1e9)
    one = flce.AdamW([torch.cat(ps)], lr=LR, betas=(B1, B2), weight_decay=0.0)
    norm = opt.step(gs)
    one.step([torch.cat(gs)])
    exact = math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))
    assert abs(float(norm) - exact) <= 1e-6 * exact
    assert torch.equal(torch.cat(ps), one.params[0])
    assert int(opt.step_count) == 1
    assert float(flce.flce_grad_norm([])) == 0 and float(flce.flce_grad_norm([ps[0]])) == 0
    nothing = flce.AdamW([torch.empty(0, device="cuda")], max_norm=1.0)
    assert float(nothing.step([torch.empty(0, device="cuda")])) == 0


def test_norm():
    sizes = [1, 127, 2049, 100000, 5000001]
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for skew in (0, 1):
            gs = params(sizes, dtype, 6, skew, 1.0)
            exact = math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))
            a, b = flce.flce_grad_norm(gs), flce.flce_grad_norm(gs)
            assert torch.equal(a, b) and abs(float(a) - exact) <= 1e-6 * exact
            assert abs(float(flce.flce_grad_norm(gs, scale=0.25)) - exact / 4) <= 1e-6 * exact
    mixed = [params([1000], d, 7)[0] for d in (torch.float32, torch.bfloat16, torch.float16)]
    exact = math.sqrt(sum(float((g.double() ** 2).sum()) for g in mixed))
    assert abs(float(flce.flce_grad_norm(mixed)) - exact) <= 1e-6 * exact
    gs[2][5] = float("inf")
    assert float(flce.flce_grad_norm(gs)) == float("inf")
    gs[2][6] = float("nan")
    assert math.isnan(float(flce.flce_grad_norm(gs)))


def test_skip_nonfinite_and_scale():
    ps = params([1000, 50], torch.float16, 8)
    opt = flce.AdamW(ps, lr=LR, betas=(B1, B2), weight_decay=0.1, master=True, skip_nonfinite=True,
                     grad_scale=1 / 1024.0)
    gs = [torch.randn(n, device="cuda").half() * 100 for n in (1000, 50)]
    opt.step(gs)
    before = [p.clone() for p in ps] + [t.clone() for t in opt.state_dict().values()]
    for bad in (float("inf"), float("nan")):
        broken = [g.clone() for g in gs]
        broken[1][3] = bad
        norm = opt.step(broken)
        assert not math.isfinite(float(norm))
        now = ps + list(opt.state_dict().values())
        assert all(torch.equal(a, b) for a, b in zip(before, now))
    opt.step(gs)
    assert int(opt.step_count) == 2
    # the scale is divided out
    plain = flce.AdamW([p.float() for p in params([1000, 50], torch.float16, 8)], lr=LR, betas=(B1, B2), weight_decay=0.1)
    for _ in range(2):
        plain.step([g.float() / 1024 for g in gs])
    for p, at, q in zip(ps, opt.offsets, plain.params):
        assert float((opt.master[at:at + p.numel()] - q).abs().max()) <= 1e-6
    # without skip_nonfinite a NaN gradient is seen in what it belongs to, with 8 bits in its block
    for bits in (32, 8):
        p = [torch.ones(1000, device="cuda")]
        o = flce.AdamW(p, state_bits=bits)
        g = torch.ones(1000, device="cuda")
        g[300] = float("nan")
        o.step([g])
        assert bool(torch.isnan(p[0][300])) and bool(torch.isfinite(p[0][:256]).all())
        assert int(torch.isnan(p[0]).sum()) == 1
        assert bool(torch.isnan(o.state_dict()["exp_avg"].float()[300]))


def test_zero_gradients_and_zero_eps():
    for bits in (32, 8):
        p = [torch.ones(500, device="cuda")]
        opt = flce.AdamW(p, lr=0.5, weight_decay=0.1, state_bits=bits)
        opt.step([torch.zeros(500, device="cuda")])
        assert float((p[0] - 0.95).abs().max()) < 1e-6
        assert all(float(t.float().abs().max()) == 0 for k, t in opt.state_dict().items()
                   if t is not None and k != "step")
    # the first step of any gradient moves by lr
    p = [torch.zeros(6, device="cuda")]
    opt = flce.AdamW(p, lr=0.5, eps=0.0, weight_decay=0.0)
    opt.step([torch.tensor([1e-15, 1.0, -1e15, 1e-4, -3.0, 7.0], device="cuda")])
    assert float((p[0].abs() - 0.5).abs().max()) < 1e-5


def test_learning_rate_tensor_graph_and_streams():
    lr = torch.tensor([0.01], device="cuda")
    gs = [torch.randn(n, device="cuda").bfloat16() for n in (5000, 33)]
    for bits in (32, 8):
        a = flce.AdamW(params([5000, 33], torch.bfloat16, 9), lr=lr, state_bits=bits, master=True, max_norm=1.0)
        b = flce.AdamW(params([5000, 33], torch.bfloat16, 9), lr=0.01, state_bits=bits, master=True, max_norm=1.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a.step(gs)  # warm
        torch.cuda.current_stream().wait_stream(side)
        graphs = []
        for _ in range(2):  # two graphs of the same handle, one after the other
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                norm = a.step(gs)
            graphs.append(g)
        b.step(gs)
        for k, rate in enumerate((0.01, 0.02, 0.04)):
            lr.fill_(rate)
            graphs[k % 2].replay()
            b.lr = rate
            want = b.step(gs, stream=side if k == 2 else None)
            torch.cuda.synchronize()
        assert torch.equal(norm, want) or k % 2 == 0
        assert int(a.step_count) == 4
        for x, y in zip(a.params + list(a.state_dict().values()), b.params + list(b.state_dict().values())):
            assert torch.equal(x, y)
        lr.fill_(0.01)


def test_state_dict_and_masters():
    def build():
        return flce.AdamW(params([300, 77], torch.bfloat16, 12), state_bits=8, master=True, seed=3)

    gs = [[torch.randn(n, device="cuda").bfloat16() for n in (300, 77)] for _ in range(4)]
    a = build()
    for g in gs[:2]:
        a.step(g)
    b = build()
    b.load_state_dict({k: v.clone() for k, v in a.state_dict().items()})
    for p, q in zip(b.params, a.params):
        p.copy_(q)
    for g in gs[2:]:
        a.step(g)
        b.step(g)
    for x, y in zip(a.params + list(a.state_dict().values()), b.params + list(b.state_dict().values())):
        assert torch.equal(x, y)
    a.params[0].fill_(0.5)
    a.load_master()
    assert float((a.master[:300] - 0.5).abs().max()) == 0
    with pytest.raises(ValueError, match="state must hold"):
        a.load_state_dict({})
    with pytest.raises(ValueError, match="missing"):
        a.load_state_dict(dict(b.state_dict(), master=None))
    with pytest.raises(ValueError, match="exp_avg"):
        a.load_state_dict(dict(b.state_dict(), exp_avg=b.state_dict()["exp_avg"][:128]))


def test_parameters_own_gradients():
    p = torch.nn.Parameter(torch.ones(10, device="cuda"))
    opt = flce.AdamW([p], lr=0.1, weight_decay=0.0)
    (p * p).sum().backward()
    opt.step()
    assert float((p.detach() - 0.9).abs().max()) < 1e-6


def test_offsets_past_32_bits():
    """A tensor of more than 2^32 elements: the random bits and the addresses of its far end."""
    n = (1 << 32) + 1000
    p = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    ends = torch.cat([torch.arange(0, 3000), torch.arange(n - 3000, n)]).cuda()
    g[ends] = torch.randn(6000, device="cuda").bfloat16()
    for bits in (8, 32):
        p.zero_()
        opt = flce.AdamW([p], lr=LR, betas=(B1, B2), weight_decay=0.0, state_bits=bits, max_norm=1e9)
        norm = opt.step([g])
        exact = float(g[ends].double().norm())
        assert abs(float(norm) - exact) <= 1e-6 * exact
        w, _, _, u = update(torch.zeros(6000, device="cuda", dtype=torch.float64), g[ends],
                            0.0, 0.0, 1, 1.0, 0.0)
        assert bool(((p[ends].double() - w).abs() <= (2.0 ** -8 + 2.0 ** -17) * w.abs()).all())
        assert float(p[1 << 31].abs()) == 0 and int(opt.step_count) == 1
        if bits == 8:
            s = opt.state_dict()
            near, far = s["exp_rms"][:2816].float(), s["exp_rms"][n - n % 128 - 2816:n - n % 128].float()
            assert float((near > 0).float().mean()) > 0.99 and float((far > 0).float().mean()) > 0.99
        del opt
        torch.cuda.empty_cache()


def test_refusals():
    p, q = torch.ones(10, device="cuda"), torch.ones(10, device="cuda").bfloat16()
    A = flce.AdamW
    with pytest.raises(TypeError, match="CUDA tensor"):
        A([p.cpu()])
    with pytest.raises(TypeError, match="parameter 1"):
        A([p, p.double()])
    with pytest.raises(ValueError, match="contiguous"):
        A([torch.ones(4, 4, device="cuda").t()])
    with pytest.raises(ValueError, match="share memory"):
        A([p, q, p])
    with pytest.raises(ValueError, match="share memory"):
        A([p[:6], p[5:]])
    A([p[:5], p[5:]])
    with pytest.raises(ValueError, match="weight decays"):
        A([p, q], weight_decay=[0.1])
    for kw in (dict(betas=(1.0, 0.9)), dict(lr=-1.0), dict(eps=-1.0), dict(betas=(0.9, float("nan")))):
        with pytest.raises(flce.FlceError, match="BAD_ARG"):
            A([p], **kw)
    opt = A([p, q], lr=0.1)
    with pytest.raises(ValueError, match="2 tensors"):
        opt.step([p])
    with pytest.raises(TypeError, match="gradient 1"):
        opt.step([p, None])
    with pytest.raises(TypeError, match="gradient 0"):
        opt.step([p.bfloat16(), q])
    with pytest.raises(TypeError, match="gradient 1"):
        opt.step([p, q.half()])
    with pytest.raises(ValueError, match="gradient 1"):
        opt.step([p, q[:5]])
    with pytest.raises(TypeError, match="gradient 0"):
        opt.step()  # no .grad
    opt.step([p.clone(), torch.ones(10, device="cuda")])  # an fp32 gradient of a bf16 parameter
    with pytest.raises(flce.FlceError, match="BAD_ARG"):
        A([p], weight_decay=-0.1).step([p.clone()])
    with pytest.raises(TypeError, match="tensor 0"):
        flce.flce_grad_norm([p.double()])
    with pytest.raises(TypeError, match="lr"):
        A([p], lr=torch.ones(1, device="cuda", dtype=torch.float64)).step([p.clone()])
    with pytest.raises(ValueError, match="workspace"):
        flce.flce_grad_norm([p], workspace=torch.zeros(10, dtype=torch.uint8, device="cuda"))


def test_exchanged_parameters():
    """A parameter's data may be exchanged for another tensor of its kind; for one of another size or
    type the step, whose table holds the old ones, is refused."""
    p = torch.nn.Parameter(torch.zeros(300, device="cuda"))
    opt = flce.AdamW([p], lr=0.1, weight_decay=0.0)
    g = torch.ones(300, device="cuda")
    opt.step([g])
    p.data = torch.full((300,), 5.0, device="cuda")
    opt.step([g])
    assert bool(((p.detach() - 4.9).abs() < 1e-4).all())
    for other, error in ((torch.zeros(20, device="cuda"), ValueError),
                         (torch.zeros(300, device="cuda").half(), TypeError),
                         (torch.zeros(300), TypeError),
                         (torch.zeros(600, device="cuda")[::2], ValueError)):
        kept, p.data = p.data, other
        with pytest.raises(error, match="parameter 0"):
            opt.step([g])
        p.data = kept
    opt.step([g])
