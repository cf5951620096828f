"""The dense layer, the processed logits and the optimizer through libflce_debug.so, the FLCE_DEBUG build:
the layer's TMA boxes and output stores are checked against their arrays there, and a failed check
would raise from these calls with validate; the results are those of the regular build, bit for bit."""
import random

import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce
from linear_cross_entropy_forward_gb300 import _binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug():
    """Runs a call in the regular build and in the other, and compares."""
    from linear_cross_entropy_forward_gb300.build import build
    path = build(debug=True)

    def both(call):
        want = call()
        mine = B.use_library(path)
        try:
            got = call()
        finally:
            B.restore_library(mine)
        for a, b in zip(got, want):
            assert a is b is None or torch.equal(a.nan_to_num(7, 8, 9), b.nan_to_num(7, 8, 9))

    return both


def layers():
    r = random.Random(3)
    for M, K, N in ((1, 8, 1), (1, 4096, 4096), (200, 512, 1001), (24, 64, 40000), (3000, 1024, 1001),
                    (8192, 512, 4096), (2500, 2048, 2304)):
        yield M, K, N, "vh", torch.bfloat16 if M % 2 else torch.float32
    for _ in range(24):
        layout = r.choice(["vh", "hv"])
        N = r.randrange(1, 5000)
        yield (r.choice([1, 5, 33, 130, 700, 2600]), 8 * r.randrange(1, 300),
               (N + 7) // 8 * 8 if layout == "hv" else N, layout, r.choice([torch.bfloat16, torch.float32]))


@pytest.mark.parametrize("M,K,N,layout,dtype", list(layers()))
def test_layers(debug, M, K, N, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(*((N, K) if layout == "vh" else (K, N)), generator=g, device="cuda").bfloat16()
    r = torch.randn(M, N, generator=g, device="cuda").to(dtype)

    def call():
        y, z = flce.flce_linear(x, w, None, "silu", r, layout, dtype, need_preact=True, validate=True)
        return (y, z, *flce.flce_linear_backward(r, x, w, z, "silu", layout, validate=True))

    debug(call)


@pytest.mark.parametrize("R,V,mask", [(3, 33, "bits"), (5, 1001, "bytes"), (2, 50257, "bits"), (300, 9001, None)])
def test_logits(debug, R, V, mask):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(R, V, generator=g, device="cuda").bfloat16()
    y = torch.randint(0, V, (R,), generator=g, device="cuda")
    o = dict(tokens=torch.randint(-1, V + 1, (R, 100), generator=g, device="cuda"), frequency_penalty=0.1,
             bias_ids=torch.randint(-1, V + 1, (R, 9), generator=g, device="cuda"),
             bias_values=torch.randn(R, 9, generator=g, device="cuda"))
    if mask == "bytes":
        o["allowed"] = torch.rand(R, V, generator=g, device="cuda") < 0.5
    elif mask:
        o["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (R, (V + 31) // 32), generator=g, device="cuda").int()
    ones = torch.ones(R, device="cuda")

    def call():
        z, _ = flce.flce_process_logits(x, need_lse=True, **o)
        logp, ent, lse = flce.flce_logits_logprob(x, y, validate=True, split_lse=True, **o)
        return z, logp, ent, lse, flce.flce_logits_logprob_backward(x, y, lse, ent, ones, ones, **o)

    debug(call)


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer(debug, bits):
    sizes = [1, 127, 129, 2049, 300001] + [5] * 700

    def call():
        g = torch.Generator(device="cuda").manual_seed(1)
        ps = [torch.randn(n, generator=g, device="cuda").bfloat16() for n in sizes]
        opt = flce.AdamW(ps, state_bits=bits, master=True, max_norm=1.0)
        norms = [opt.step([p * 0.5 for p in ps]) for _ in range(2)]
        return [*norms, *ps, *(t.float() for t in opt.state_dict().values())]

    debug(call)
