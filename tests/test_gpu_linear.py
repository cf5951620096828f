"""The dense layer and its gradients against 64 bits.

Tolerances, element by element.  A sum of K products of bf16 values is exact up to the additions, at
most 2^-23 of the absolute terms' sum each (the tensor cores cut off where fp32 rounds):
(K + 8) 2^-23 (|x| |W| + |b|).  Activations have slopes below 1.13 and their own error is below 1e-6
(|z| + 1).  A rounding to bf16 is 2^-8 of the value, to fp32 2^-24.
"""
import math

import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu
E8, E23 = 2.0 ** -8, 2.0 ** -23


def act64(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if kind == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(2 * u)
    return z.clone()


def slope64(z, kind):
    z = z.detach().requires_grad_(True)
    if kind in (None, "none"):
        return torch.ones_like(z)
    (d,) = torch.autograd.grad(act64(z, kind).sum(), z)
    return d


def make(M, K, N, layout, seed=0, bias=True, residual=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(*((N, K) if layout == "vh" else (K, N)), generator=g, device="cuda")
    w = (w / math.sqrt(K)).bfloat16()
    b = torch.randn(N, generator=g, device="cuda").bfloat16() if bias else None
    r = torch.randn(M, N, generator=g, device="cuda").to(residual) if residual else None
    return x, w, b, r


def exact(x, w, b, layout):
    """z and the bound of its error."""
    W = (w.t() if layout == "vh" else w).double()
    z, size = x.double() @ W, x.double().abs() @ W.abs()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    return z, (x.shape[-1] + 8) * E23 * size


def close(got, want, tol, what=""):
    d = (got.double() - want).abs()
    assert got.shape == want.shape and bool(torch.isfinite(got.float()).all()), what
    assert bool((d <= tol + 1e-30).all()), (what, float((d - tol).max()), float(d.max()))


# one token to many, odd sizes, tiles and clusters of every kind, depths of one block and less
SHAPES = [(1, 8, 1), (1, 64, 128), (1, 4096, 4096), (2, 72, 129), (16, 1000, 300), (17, 520, 33),
          (48, 4096, 640), (65, 136, 1000), (200, 2304, 512), (256, 64, 257), (257, 8, 8),
          (300, 1000, 1001), (600, 4096, 256), (1500, 776, 384), (2999, 256, 1001), (4100, 200, 2056)]


@pytest.mark.parametrize("layout", ["vh", "hv"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(M, K, N, layout):
    N = (N + 7) // 8 * 8 if layout == "hv" else N
    x, w, b, r = make(M, K, N, layout, residual=torch.float32)
    z, tol = exact(x, w, b, layout)
    y = flce.flce_linear(x, w, b, None, r, layout, torch.float32, validate=True)
    want = z + r.double()
    close(y, want, tol + E23 * want.abs())
    # without bias and residual, in bf16
    z, tol = exact(x, w, None, layout)
    y = flce.flce_linear(x, w, weight_layout=layout)
    close(y, z, tol + E8 * z.abs())


@pytest.mark.parametrize("M,K,N", [(3, 264, 100), (130, 512, 136), (1100, 640, 520)])
@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_epilogue_and_gradients(M, K, N, act, out):
    x, w, b, r = make(M, K, N, "vh", 3, residual=out)
    z, tol = exact(x, w, b, "vh")
    y, pre = flce.flce_linear(x, w, b, act, r, "vh", out, need_preact=True)
    want = act64(z, act) + r.double()
    rounding = (E8 if out is torch.bfloat16 else E23) * want.abs()
    close(y, want, 1.13 * tol + 1e-6 * (z.abs() + 1) + rounding, act)
    close(pre, z, tol + E8 * z.abs(), "preact")
    dy = torch.randn(M, N, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(out)
    dx, dw, db = flce.flce_linear_backward(dy, x, w, pre, act, "vh", validate=True)
    dz = dy.double() * slope64(pre.double(), act)
    off = 1e-6 * (pre.double().abs() + 1) * dy.double().abs() + E8 * dz.abs()  # of the rounded dz
    W = w.double()
    close(dx, dz @ W, off @ W.abs() + (N + 8) * E23 * (dz.abs() @ W.abs()) + E8 * (dz @ W).abs(), "dx")
    dW = dz.t() @ x.double()
    size = dz.abs().t() @ x.double().abs()
    close(dw, dW, off.t() @ x.double().abs() + (M + 8) * E23 * size + E8 * dW.abs(), "dw")
    s = dz.sum(0)
    close(db, s, (1e-6 * (pre.double().abs() + 1) * dy.double().abs()).sum(0)
          + (M + 8) * 2.0 ** -24 * dz.abs().sum(0) + E8 * s.abs(), "db")


@pytest.mark.parametrize("layout", ["vh", "hv"])
@pytest.mark.parametrize("M,K,N", [(1, 64, 8), (7, 64, 200), (300, 1000, 1000), (2999, 256, 1000),
                                   (5000, 768, 2304)])
def test_gradients_of_both_layouts(M, K, N, layout):
    x, w, b, _ = make(M, K, N, layout, 7)
    dy = torch.randn(M, N, device="cuda").bfloat16()
    dx, dw, db = flce.flce_linear_backward(dy, x, w, weight_layout=layout)
    W, g = (w.t() if layout == "vh" else w).double(), dy.double()
    dX, dW = g @ W.t(), x.double().t() @ g
    close(dx, dX, (N + 8) * E23 * (g.abs() @ W.abs().t()) + E8 * dX.abs(), "dx")
    size = x.double().abs().t() @ g.abs()
    if layout == "vh":
        dW, size = dW.t(), size.t()
    close(dw, dW, (M + 8) * E23 * size + E8 * dW.abs(), "dw")
    s = g.sum(0)
    close(db, s, (M + 8) * 2.0 ** -24 * g.abs().sum(0) + E8 * s.abs(), "db")
    # each gradient alone is the same
    for i, need in enumerate(("need_dx", "need_dweight", "need_dbias")):
        flags = {"need_dx": False, "need_dweight": False, "need_dbias": False, need: True}
        one = flce.flce_linear_backward(dy, x, w, weight_layout=layout, **flags)
        assert torch.equal(one[i], (dx, dw, db)[i])
        assert [t is None for t in one] == [j != i for j in range(3)]


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradient_against_differences(act):
    """A directional derivative of the 64-bit loss by central differences: the kernel's gradients,
    each rounded to 2^-8, along a random direction."""
    M, K, N = 40, 64, 56
    x, w, b, _ = make(M, K, N, "vh", 11)
    g = torch.randn(M, N, device="cuda").bfloat16()
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    y = flce.linear(*leaves[:2], leaves[2], act, weight_layout="vh")
    grads = torch.autograd.grad(y, leaves, g)
    dirs = [torch.randn_like(t.double()) for t in (x, w, b)]

    def loss(h):
        X, W, B = (t.double() + h * d for t, d in zip((x, w, b), dirs))
        return float((act64(X @ W.t() + B, act) * g.double()).sum())

    h = 1e-4
    slope = (loss(h) - loss(-h)) / (2 * h)
    got = sum(float((a.double() * d).sum()) for a, d in zip(grads, dirs))
    # roundings of z, dz and the result, 2^-8 each, of terms whose sizes add up at most like this
    size = sum(float((a.double() * d).norm()) for a, d in zip(grads, dirs))
    assert abs(got - slope) <= 6 * 3 * E8 * size + 1e-4 * abs(slope)


def test_far_values_of_activations():
    """Preactivations from -40 to 40, and the far tails: K = 8 picks one of them per row."""
    v = torch.cat([torch.linspace(-40, 40, 2001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e4, -3e4])])
    M = v.numel()
    x = torch.zeros(M, 8, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = v.to("cuda").bfloat16()
    w = torch.zeros(16, 8, device="cuda", dtype=torch.bfloat16)
    w[:, 0] = 1
    z = x[:, :1].double().expand(M, 16)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        y, pre = flce.flce_linear(x, w, activation=act, weight_layout="vh", out_dtype=torch.float32,
                                  need_preact=True)
        close(y, act64(z, act), 1e-6 * act64(z, act).abs() + 1e-9 + 4e-6 * act64(z, act).abs(), act)
        assert torch.equal(pre.double(), z)
        dx, _, db = flce.flce_linear_backward(torch.ones_like(y).bfloat16(), x, w, pre, act, "vh")
        want = 16 * slope64(z, act)[:, 0]
        close(dx[:, 0], want, 2 * E8 * want.abs() + 1e-5, act)


def test_nan_and_infinity_stay_in_their_row():
    x, w, b, _ = make(5, 64, 40, "vh", 2)
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    for act in (None, "relu", "gelu", "gelu_tanh", "silu"):
        y = flce.flce_linear(x, w, b, act, weight_layout="vh")
        assert bool(torch.isnan(y[2]).all()), act
        assert bool(torch.isfinite(y[[0, 1, 4]]).all())


def test_shapes_views_and_in_place():
    x, w, b, r = make(12, 64, 24, "vh", 4, residual=torch.bfloat16)
    y = flce.flce_linear(x.view(3, 2, 2, 64), w, b, "silu", r.view(3, 2, 2, 24), "vh")
    assert y.shape == (3, 2, 2, 24)
    flat = flce.flce_linear(x, w, b, "silu", r, "vh")
    assert torch.equal(y.view(12, 24), flat)
    assert torch.equal(flce.flce_linear(x[0], w, b, "silu", r[0], "vh"), flat[0])
    # the residual is where the output goes
    into = r.clone()
    assert flce.flce_linear(x, w, b, "silu", into, "vh", out=into) is into
    assert torch.equal(into, flat)
    empty = flce.flce_linear(x[:0], w, b, "silu", weight_layout="vh", validate=True)
    assert empty.shape == (0, 24)
    dx, dw, db = flce.flce_linear_backward(empty, x[:0], w, empty, "silu", "vh", validate=True)
    assert dx.shape == (0, 64) and float(dw.abs().max()) == 0 and float(db.abs().max()) == 0
    # a bias that is not 16-byte aligned
    odd = torch.empty(25, device="cuda", dtype=torch.bfloat16)[1:].copy_(b)
    assert torch.equal(flce.flce_linear(x, w, odd, "silu", r, "vh"), flat)


@pytest.mark.parametrize("M,K,N", [(4, 4096, 512), (2500, 512, 2304)])
def test_repeats_streams_threads_and_graphs(M, K, N):
    import threading
    x, w, b, r = make(M, K, N, "vh", 6, residual=torch.bfloat16)
    dy = torch.randn(M, N, device="cuda").bfloat16()
    y, z = flce.flce_linear(x, w, b, "gelu", r, "vh", need_preact=True)
    grads = flce.flce_linear_backward(dy, x, w, z, "gelu", "vh")
    torch.cuda.synchronize()
    outs = {}

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                yy, zz = flce.flce_linear(x, w, b, "gelu", r, "vh", need_preact=True)
                outs[i] = [yy, *flce.flce_linear_backward(dy, x, w, zz, "gelu", "vh")]
        s.synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    for i in range(3):
        assert all(torch.equal(a, c) for a, c in zip(outs[i], [y, *grads]))
    side = torch.cuda.Stream()
    assert torch.equal(flce.flce_linear(x, w, b, "gelu", r, "vh", stream=side), y)
    side.synchronize()
    # two graphs that share one workspace, one after the other
    p = flce.linear_params(M, N, K, "gelu", "vh")
    ws = torch.empty(max(flce.linear_workspace_size(p), flce.linear_workspace_size(p, True)),
                     dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            yy, zz = flce.flce_linear(x, w, b, "gelu", r, "vh", need_preact=True, workspace=ws)
            gg = flce.flce_linear_backward(dy, x, w, zz, "gelu", "vh", workspace=ws)
        graphs.append((g, [yy, *gg]))
    x.mul_(-1)
    want = [flce.flce_linear(x, w, b, "gelu", r, "vh")]
    want += flce.flce_linear_backward(dy, x, w, flce.flce_linear(x, w, b, "gelu", r, "vh",
                                                               need_preact=True)[1], "gelu", "vh")
    for g, out in graphs:
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want))


def test_autograd():
    x, w, b, r = make(33, 64, 48, "hv", 8, residual=torch.float32)
    dy = torch.randn(33, 48, device="cuda")
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b, r)]
    y = flce.linear(leaves[0], leaves[1], leaves[2], "silu", leaves[3], out_dtype=torch.float32)
    y.backward(dy)
    _, z = flce.flce_linear(x, w, b, "silu", r, out_dtype=torch.float32, need_preact=True)
    dx, dw, db = flce.flce_linear_backward(dy, x, w, z, "silu")
    for leaf, d in zip(leaves, (dx, dw, db, dy)):
        assert torch.equal(leaf.grad, d)
    # only some of them, a broadcast upstream gradient, and no second derivative
    a = x.clone().requires_grad_(True)
    flce.linear(a, w, b).sum().backward()
    assert torch.equal(a.grad, flce.flce_linear_backward(torch.ones_like(y).bfloat16(), x, w)[0])
    a = w.clone().requires_grad_(True)
    (g,) = torch.autograd.grad(flce.linear(x, a, activation="gelu").float().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()
    # a graph of the backward while an eager graph of the same leaves lives; the leaves' first use is on
    # a stream of its own, as a capture cannot wait for the default stream, which autograd would have it do
    a, v = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = flce.linear(a, v, activation="gelu")
        up = torch.ones_like(eager)
        for _ in range(2):
            want = torch.autograd.grad(flce.linear(a, v, activation="gelu"), [a, v], up)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(flce.linear(a, v, activation="gelu"), [a, v], up)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(torch.equal(p, q) for p, q in zip(torch.autograd.grad(eager, [a, v], up), want))


def test_offsets_past_32_bits():
    """Rows whose first element is past 2^31 elements: 300000 x 8192 in bf16."""
    M, K, N = 300000, 16, 8192
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    at = [0, 1, 262143, 262144, 299999]
    x[at] = torch.randn(len(at), K, device="cuda").bfloat16()
    w = torch.randn(N, K, device="cuda").bfloat16()
    y = flce.flce_linear(x, w, weight_layout="vh")
    z, tol = exact(x[at], w, None, "vh")
    close(y[at], z, tol + E8 * z.abs())
    assert float(y[100:200].abs().max()) == 0
    dx, dw, db = flce.flce_linear_backward(y, x, w, weight_layout="vh")
    g = y[at].double()
    close(dx[at], g @ w.double(), (N + 8) * E23 * (g.abs() @ w.double().abs()) + E8 * (g @ w.double()).abs())
    s = g.sum(0)
    close(db, s, 16 * 2.0 ** -24 * g.abs().sum(0) + E8 * s.abs())
    dW = g.t() @ x[at].double()
    close(dw, dW, 64 * E23 * (g.abs().t() @ x[at].double().abs()) + E8 * dW.abs())


def test_refusals():
    x, w, b, r = make(4, 16, 8, "vh", residual=torch.bfloat16)
    L = lambda *a, **k: flce.flce_linear(*a, weight_layout="vh", **k)  # noqa: E731
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        L(x.float(), w)
    with pytest.raises(TypeError, match="weight must be torch.bfloat16"):
        L(x, w.half())
    with pytest.raises(ValueError, match="rows of 16"):
        flce.flce_linear(x, w)
    with pytest.raises(ValueError, match="contiguous"):
        L(x.t().contiguous().t(), w)
    with pytest.raises(TypeError, match="bias"):
        L(x, w, b.float())
    with pytest.raises(ValueError, match="bias"):
        L(x, w, b[:4])
    with pytest.raises(TypeError, match="residual"):
        L(x, w, b, None, r.float())
    with pytest.raises(ValueError, match="residual"):
        L(x, w, b, None, r[:2])
    with pytest.raises(ValueError, match="activation"):
        L(x, w, activation="tanh")
    with pytest.raises(TypeError, match="out_dtype"):
        L(x, w, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="out must"):
        L(x, w, out=torch.empty(4, 8, device="cuda"))
    with pytest.raises(flce.FlceError, match="ALIGN"):
        L(x[:, :12].contiguous(), w[:, :12].contiguous())
    with pytest.raises(flce.FlceError, match="ALIGN"):  # x 2 bytes off
        L(torch.empty(65, device="cuda", dtype=torch.bfloat16)[1:].view(4, 16), w)
    with pytest.raises(ValueError, match="workspace"):
        L(x, w, workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))
    dy = torch.ones(4, 8, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="preact"):
        flce.flce_linear_backward(dy, x, w, None, "gelu", "vh")
    with pytest.raises(TypeError, match="out_dtype"):
        flce.flce_linear_backward(dy.half(), x, w, weight_layout="vh")
    with pytest.raises(ValueError, match="dout"):
        flce.flce_linear_backward(dy[:2], x, w, weight_layout="vh")


@pytest.mark.parametrize("M,K,N,layout", [(2600, 1032, 2301, "vh"), (2600, 1032, 2304, "hv"),
                                          (1100, 264, 4099, "vh"), (2049, 2048, 2047, "vh")])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_many_tokens_by_odd_widths(M, K, N, layout, out):
    """Tiles of every kind with rows that 16 bytes do not divide; everything in the output at once, in
    place of the residual too; and the gradients, dz unaligned."""
    x, w, b, r = make(M, K, N, layout, 9, residual=out)
    z, tol = exact(x, w, b, layout)
    want = act64(z, "silu") + r.double()
    y, pre = flce.flce_linear(x, w, b, "silu", r, layout, out, need_preact=True, validate=True)
    rounding = (E8 if out is torch.bfloat16 else E23) * want.abs()
    close(y, want, 1.13 * tol + 1e-6 * (z.abs() + 1) + rounding)
    close(pre, z, tol + E8 * z.abs())
    same = r.clone()
    flce.flce_linear(x, w, b, "silu", same, layout, out, out=same)
    assert torch.equal(same, y)
    dx, dw, db = flce.flce_linear_backward(r, x, w, pre, "silu", layout, validate=True)
    dz = r.double() * slope64(pre.double(), "silu")
    off = 1e-6 * (pre.double().abs() + 1) * r.double().abs() + E8 * dz.abs()
    W = (w if layout == "vh" else w.t()).double()
    close(dx, dz @ W, off @ W.abs() + (N + 8) * E23 * (dz.abs() @ W.abs()) + E8 * (dz @ W).abs(), "dx")
    dW = dz.t() @ x.double()
    close(dw if layout == "vh" else dw.t(), dW, off.t() @ x.double().abs()
          + (M + 8) * E23 * (dz.abs().t() @ x.double().abs()) + E8 * dW.abs(), "dw")
    s = dz.sum(0)
    close(db, s, (1e-6 * (pre.double().abs() + 1) * r.double().abs()).sum(0)
          + (M + 8) * 2.0 ** -24 * dz.abs().sum(0) + E8 * s.abs(), "db")


def test_outputs_that_share_memory_are_refused():
    """Tiles are read while others are written, so an output over an input would be read back."""
    x, w, b, r = make(16, 16, 16, "vh", residual=torch.bfloat16)
    big = torch.empty(16 * 16 + 8, device="cuda", dtype=torch.bfloat16)
    L = lambda **k: flce.flce_linear(x, w, b, weight_layout="vh", **k)  # noqa: E731
    with pytest.raises(ValueError, match="out shares memory with x"):
        L(out=x)
    with pytest.raises(ValueError, match="out shares memory with weight"):
        L(out=w)
    with pytest.raises(ValueError, match="out shares memory with residual"):
        L(residual=big[8:].view(16, 16), out=big[:256].view(16, 16))
    L(residual=r, out=r)
    dy = torch.ones_like(r)
    D = lambda *o: flce.flce_linear_backward(dy, x, w, weight_layout="vh", out=o)  # noqa: E731
    new = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    same = new(16, 16)
    with pytest.raises(ValueError, match="dx shares memory with dout"):
        D(dy, new(16, 16), new(16))
    with pytest.raises(ValueError, match="dx shares memory with dweight"):
        D(same, same, new(16))
    with pytest.raises(ValueError, match="dweight shares memory with x"):
        D(new(16, 16), x, new(16))
    D(new(16, 16), new(16, 16), new(16))
