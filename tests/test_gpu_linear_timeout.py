"""A dense layer's wait for copies that never come: it ends after its limit of 2 s, is reported, and
leaves nothing that could be taken for a result, although nobody need have asked for its status."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

FLCE_ERR_TIMEOUT = 6


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


def bf16(*shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()


# a cluster to a tile, one block, pairs in one round and in several, narrow ones, odd widths, sums
# that are drained; one 64-deep block
CASES = [(1, 4096, 4096, "vh", None), (200, 512, 1001, "vh", "silu"), (24, 64, 40000, "hv", None),
         (3000, 1024, 1001, "vh", "gelu"), (8192, 512, 4096, "hv", None), (2500, 2048, 2304, "vh", None)]


@pytest.mark.parametrize("M,K,N,layout,act", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward(F, M, K, N, layout, act, dtype):
    lib, stream = F.load_library(), torch.cuda.current_stream().cuda_stream
    x, w = bf16(M, K), bf16(*((N, K) if layout == "vh" else (K, N)))
    r = bf16(M, N).to(dtype)
    p = F.linear_params(M, N, K, act, layout, dtype)
    ws = torch.empty(F.linear_workspace_size(p), dtype=torch.uint8, device="cuda")
    guard = 64
    y = torch.zeros(M * N + guard, dtype=dtype, device="cuda")
    z = torch.zeros(M * N + guard, dtype=torch.bfloat16, device="cuda")
    code = lib.flce_selftest_linear_timeout(ctypes.byref(p), x.data_ptr(), w.data_ptr(), r.data_ptr(),
                                            y.data_ptr(), z.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    assert code == 0
    assert F.flce_status(ws) == FLCE_ERR_TIMEOUT
    for t in (y, z):
        assert bool(t[:M * N].isnan().all()) and float(t[M * N:].abs().max()) == 0
    # the context is usable, and so is the workspace
    args = (x, w, None, act, r, layout, dtype)
    again = F.flce_linear(*args, need_preact=True, workspace=ws)
    assert F.flce_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(again, F.flce_linear(*args, need_preact=True)))
    assert bool(torch.isfinite(again[0].float()).all())


@pytest.mark.parametrize("M,K,N,layout,act", [(7, 64, 200, "vh", "silu"), (2999, 1032, 1001, "vh", None),
                                              (8192, 2048, 4096, "hv", "gelu")])
def test_gradients(F, M, K, N, layout, act):
    lib, stream = F.load_library(), torch.cuda.current_stream().cuda_stream
    x, w, dy = bf16(M, K), bf16(*((N, K) if layout == "vh" else (K, N))), bf16(M, N)
    z = bf16(M, N)
    p = F.linear_params(M, N, K, act, layout)
    ws = torch.empty(F.linear_workspace_size(p, True), dtype=torch.uint8, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    code = lib.flce_selftest_linear_backward_timeout(
        ctypes.byref(p), dy.data_ptr(), x.data_ptr(), w.data_ptr(), z.data_ptr(), dx.data_ptr(), dw.data_ptr(),
        ws.data_ptr(), ws.numel(), stream)
    assert code == 0
    assert F.flce_status(ws) == FLCE_ERR_TIMEOUT
    assert bool(dx.isnan().all()) and bool(dw.isnan().all())
    again = F.flce_linear_backward(dy, x, w, z, act, layout, workspace=ws)
    assert F.flce_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(again, F.flce_linear_backward(dy, x, w, z, act, layout)))


def test_validate(F):
    """The same by the call's own code."""
    lib, stream = F.load_library(), torch.cuda.current_stream().cuda_stream
    x, w, y = bf16(4, 64), bf16(128, 64), bf16(4, 128)
    p = F.linear_params(4, 128, 64, None, "vh", validate=True)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    assert lib.flce_selftest_linear_timeout(ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, y.data_ptr(), None,
                                            ws.data_ptr(), 256, stream) == FLCE_ERR_TIMEOUT
    assert bool(y.isnan().all())
