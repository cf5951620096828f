"""The elements of the flat states behind a tensor's last stay 0, whatever the step makes of the others."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu
SIZES = [1, 7, 8, 9, 127, 128, 129, 250, 2041, 2049]


def behind(opt):
    """(name, what lies behind each tensor's last element) of the states with an entry per element."""
    for name, t in opt.state_dict().items():
        if t is None or name == "step" or name.endswith("_scale"):
            continue
        for p, at in zip(opt.params, opt.offsets):
            n = p.numel()
            yield name, t[at + n:at + -(-n // 128) * 128].float()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["no eps", "nan norm", "infinite rate", "nan gradient"])
def test_zeros_stay(bits, dtype, kind):
    ps = [torch.ones(n, device="cuda", dtype=dtype) for n in SIZES]
    gs = [torch.full((n,), 0.5, device="cuda", dtype=dtype) for n in SIZES]
    kw = {}
    if kind == "no eps":
        kw["eps"] = 0.0
    elif kind == "infinite rate":
        kw["lr"] = torch.tensor([float("inf")], device="cuda")
    else:
        gs[3][-1] = float("nan")
        if kind == "nan norm":
            kw["max_norm"] = 1.0
    opt = flce.AdamW(ps, master=True, state_bits=bits, **kw)
    for _ in range(2):
        opt.step(gs)
    for name, pad in behind(opt):
        assert bool((pad == 0).all()), (kind, name)
    if kind == "no eps":  # m / sqrt(v) is 1: the elements themselves move by the rate
        for p, at in zip(ps, opt.offsets):
            w = opt.master[at:at + p.numel()]
            assert float((w - 1).abs().max()) < 3e-3 and bool(torch.isfinite(p.float()).all())
    if kind == "nan gradient":
        assert bool(ps[3].isnan()[-1]) and sum(int(p.isnan().sum()) for p in ps) == 1
