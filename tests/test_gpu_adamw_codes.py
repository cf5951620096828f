"""The 8-bit states code for code against a restatement of their definition, the random bits among it,
and the captured step's norm replay for replay."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu
M32 = (1 << 32) - 1


def mix(x):
    x = x ^ (x >> np.uint64(16))
    x = x * np.uint64(0x7FEB352D) & np.uint64(M32)
    x = x ^ (x >> np.uint64(15))
    x = x * np.uint64(0x846CA68B) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def random_bits(n, seed, t):
    """Of the two states of elements 0 to n - 1 of the flat states, 20 each."""
    key = mix(np.uint64((seed + 0x9E3779B9 * t) & M32))
    i = np.arange(n, dtype=np.uint64)
    h = mix((i & np.uint64(M32)) ^ mix((key + (i >> np.uint64(32))) & np.uint64(M32)))
    return h >> np.uint64(12), (h * np.uint64(0x9E3779B1) & np.uint64(M32)) >> np.uint64(12)


def encode(x, r, root):
    """fp32 values of e4m3 codes, and scales, of x in blocks of 128; every operation in fp32."""
    f = np.float32
    x = x.reshape(-1, 128)
    top = np.abs(x).max(1, keepdims=True)
    none = top < f(2.0 ** -110)
    unit = np.where(none, f(0), f(448) * (f(1) / np.where(none, f(1), top)))
    a = np.abs(x) * unit
    low = np.where(a < f(2.0 ** -6), f(2.0 ** -6), f(0))
    bits = (a + low).view(np.uint32).astype(np.uint64) + r.reshape(-1, 128)
    q = (bits & np.uint64(0xFFF00000)).astype(np.uint32).view(f) - low
    q = np.minimum(q, f(448))
    if root:
        q = np.where((a > 0) & (q == 0), f(2.0 ** -9), q)
    else:
        q = np.copysign(q, x)
    return q.ravel(), np.where(none, f(0), top * f(1.0 / 448))[:, 0]


@pytest.mark.parametrize("dtype,master", [(torch.float32, False), (torch.bfloat16, True), (torch.float16, False)])
@pytest.mark.parametrize("seed", [0, 0x9ABCDEF0])
def test_codes(dtype, master, seed):
    f = np.float32
    sizes = [1, 100, 128, 2049, 70001]
    g = torch.Generator(device="cuda").manual_seed(5)
    ps = [torch.randn(n, generator=g, device="cuda").to(dtype) for n in sizes]
    b1, b2, scale = 0.9, 0.995, 0.37
    opt = flce.AdamW(ps, betas=(b1, b2), state_bits=8, master=master, seed=seed, grad_scale=scale)
    n = opt.state_dict()["exp_avg"].numel()
    for t in range(1, 5):
        old = {k: v.float().cpu().numpy() for k, v in opt.state_dict().items() if v is not None}
        gs = [(torch.randn(k, generator=g, device="cuda") * 10.0 ** (i - 3) * (2.0 if t % 2 else 0.1)).to(dtype)
              for i, k in enumerate(sizes)]
        gs[3][::7] = 0
        opt.step(gs)
        new = {k: v.float().cpu().numpy() for k, v in opt.state_dict().items() if v is not None}
        flat = np.zeros(n, f)
        for x, at in zip(gs, opt.offsets):
            flat[at:at + x.numel()] = x.float().cpu().numpy()
        x = flat * f(scale)
        m = old["exp_avg"] * np.repeat(old["exp_avg_scale"], 128)
        s = old["exp_rms"] * np.repeat(old["exp_rms_scale"], 128)
        m = m * f(b1) + x * f(1 - b1)
        v = (s * s) * f(b2) + (x * x) * f(1 - b2)
        r1, r2 = random_bits(n, seed, t)
        for name, value, r, root in (("exp_avg", m, r1, False), ("exp_rms", np.sqrt(v), r2, True)):
            assert value.dtype == f
            q, scales = encode(value, r, root)
            assert np.array_equal(new[name + "_scale"], scales), (name, t)
            assert np.array_equal(new[name], q), (name, t, int((new[name] != q).sum()))


@pytest.mark.parametrize("bits", [32, 8])
def test_the_captured_norm(bits):
    """Two graphs of one optimizer, each with a norm of its own, against eager steps."""
    sizes = [5000, 33]
    ps = [[torch.ones(n, device="cuda").bfloat16() for n in sizes] for _ in range(2)]
    gs = [torch.zeros(n, device="cuda").bfloat16() for n in sizes]
    a, b = (flce.AdamW(p, lr=0.01, state_bits=bits, master=True, max_norm=1.0) for p in ps)
    a.step(gs)
    b.step(gs)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = a.step(gs)
        graphs.append((graph, norm))
    seen = set()
    for k in range(4):
        for i, t in enumerate(gs):
            t.copy_(torch.randn(t.numel(), generator=torch.Generator(device="cuda").manual_seed(10 * k + i),
                                device="cuda") * (k + 1))
        graph, norm = graphs[k % 2]
        graph.replay()
        want = b.step(gs)
        torch.cuda.synchronize()
        exact = float(torch.cat(gs).double().norm())
        assert torch.equal(norm, want) and abs(float(norm) - exact) <= 1e-6 * exact
        seen.add(float(norm))
        for x, y in zip(a.params + list(a.state_dict().values()), b.params + list(b.state_dict().values())):
            assert torch.equal(x, y)
    assert len(seen) == 4
