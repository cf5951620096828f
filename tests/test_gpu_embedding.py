"""The embedding lookup and its gradient.

The lookup is compared bit for bit with the rounded fp32 product.  The gradient's sums are
in fp32 in a fixed order: of c rows they are within c 2^-24 of the summed magnitudes (times
the scale, two more half steps for the product and the addition to the old value), and the
stored value adds half a step of its type (fp16: and half its smallest subnormal)."""
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


def bits(x):
    return x.contiguous().view(torch.int32 if x.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [1, 7, 8, 64, 100, 1030, 2304, 4096])
@pytest.mark.parametrize("scale", [1.0, 48.0, -0.3])
def test_lookup(F, dtype, H, scale):
    g = torch.Generator().manual_seed(H)
    w = torch.randn(301, H, generator=g).to(DTYPES[dtype]).cuda()
    for shape in [(), (1,), (8,), (3, 111), (0,)]:
        for idt in (torch.int64, torch.int32):
            ids = torch.randint(0, 301, shape, generator=g).to(idt).cuda()
            got = F.flce_embedding(ids, w, scale, validate=True)
            s = torch.tensor(scale, dtype=torch.float32).cuda()
            want = (w[ids.long()].float() * s).to(w.dtype)
            assert got.shape == want.shape and torch.equal(bits(got), bits(want))


def test_lookup_unaligned_table(F):
    base = torch.randn(50 * 64 + 1).to(torch.bfloat16).cuda()
    w = base[1:].view(50, 64)
    ids = torch.randint(0, 50, (77,)).cuda()
    assert torch.equal(F.flce_embedding(ids, w), w[ids])


def test_lookup_shards_and_bad_ids(F):
    w = torch.randn(100, 40).cuda()
    ids = torch.randint(0, 100, (333,)).cuda()
    parts = [F.flce_embedding(ids, w[a:b].contiguous(), 2.0, v_offset=a, v_total=100, validate=True)
             for a, b in ((0, 33), (33, 34), (34, 100))]
    assert torch.equal(sum(parts), w[ids] * 2)
    ids[5], ids[9] = 100, -1
    got = F.flce_embedding(ids, w)
    assert bool(got[5].isnan().all()) and bool(got[9].isnan().all())
    ok = torch.ones(333, dtype=torch.bool).cuda()
    ok[5] = ok[9] = False
    assert torch.equal(got[ok], w[ids[ok]])
    with pytest.raises(F.FlceError) as e:
        F.flce_embedding(ids, w, validate=True)
    assert e.value.code == 5


def test_lookup_offsets_past_32_bits(F):
    """A table of 2^31 + elements and an output of as many."""
    V, H = (1 << 20) + 5, 2056
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = (torch.arange(V, device="cuda") % 251).to(torch.bfloat16)
    w[:, -1] = (torch.arange(V, device="cuda") % 127).to(torch.bfloat16)
    ids = torch.arange(V - 1, -1, -1, device="cuda")
    out = F.flce_embedding(ids, w)
    assert torch.equal(out[:, 0], w[:, 0].flip(0)) and torch.equal(out[:, -1], w[:, -1].flip(0))
    dw = F.flce_embedding_backward(out, ids, V)
    assert torch.equal(dw, w)


def grad_case(F, N, H, V, dtype="bf16", gdtype=None, scale=1.0, accumulate=False, padding=None,
              ids=None, ids32=False, v_offset=0, v_total=0, seed=0):
    dt = DTYPES[dtype]
    gdt = DTYPES[gdtype or dtype]
    g = torch.Generator().manual_seed(seed)
    if ids is None:
        ids = torch.randint(0, v_total or V, (N,), generator=g)
    dout = torch.randn(N, H, generator=g).to(dt)
    old = torch.randn(V, H, generator=g).to(gdt) if accumulate else None
    dw = old.cuda() if accumulate else None
    got = F.flce_embedding_backward(dout.cuda(), (ids.int() if ids32 else ids).cuda(), V, scale,
                                    padding, dweight=dw, accumulate=accumulate, grad_dtype=gdt,
                                    v_offset=v_offset, v_total=v_total, validate=True)
    assert got.dtype == gdt and (not accumulate or got is dw)
    s = float(torch.tensor(scale, dtype=torch.float32))
    row = ids - v_offset
    keep = (row >= 0) & (row < V)
    if padding is not None:
        keep &= ids != padding
    want = old.double() if accumulate else torch.zeros(V, H, dtype=torch.float64)
    mag, cnt = want.abs().clone(), torch.zeros(V, dtype=torch.float64)
    want.index_add_(0, row[keep], dout[keep].double() * s)
    mag.index_add_(0, row[keep], dout[keep].double().abs() * abs(s))
    cnt.index_add_(0, row[keep], torch.ones(int(keep.sum()), dtype=torch.float64))
    tol = (cnt[:, None] + 2) * 2.0 ** -24 * mag
    if gdt != torch.float32:
        tol = tol + torch.finfo(gdt).eps / 2 * want.abs() * 1.001 + (2.0 ** -25 if gdt == torch.float16
                                                                      else 0.0)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    untouched = cnt == 0
    if accumulate:
        assert torch.equal(bits(got.cpu()[untouched]), bits(old[untouched]))
    else:
        assert bool((got.cpu()[untouched] == 0).all())
    return got


@pytest.mark.parametrize("N", [0, 1, 2, 31, 32, 33, 64, 1000, 1024, 1025, 5000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_token_counts(F, N, accumulate):
    grad_case(F, N, 72, 500, accumulate=accumulate, seed=N)


@pytest.mark.parametrize("dtype,gdtype", [("bf16", None), ("fp16", None), ("fp32", None),
                                          ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("H", [1, 2, 7, 12, 256, 1000, 2304])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_types_and_widths(F, dtype, gdtype, H, accumulate):
    grad_case(F, 777, H, 333, dtype, gdtype, scale=48.0, accumulate=accumulate, seed=H)


@pytest.mark.parametrize("V", [1, 2, 511, 512, 513, 70000, (1 << 18) + 1, (1 << 20) + 3])
def test_gradient_table_sizes(F, V):
    """One to three passes of the sort."""
    grad_case(F, 3000, 16, V, seed=V)


@pytest.mark.parametrize("N", [4096, 70000, 200001])
def test_gradient_frequent_ids(F, N):
    """Half of the tokens share one id, a quarter another: runs over many units."""
    g = torch.Generator().manual_seed(N)
    ids = torch.randint(0, 3000, (N,), generator=g)
    r = torch.rand(N, generator=g)
    ids[r < 0.5] = 1234
    ids[r > 0.75] = 2999
    grad_case(F, N, 40, 3000, ids=ids, seed=N)
    grad_case(F, N, 40, 3000, "fp32", ids=ids, accumulate=True, seed=N)


def test_gradient_one_id_and_runs_that_end_at_units(F):
    grad_case(F, 4096, 64, 9, ids=torch.full((4096,), 4))
    # runs of 32, 64, 31, 33 ... sorted already and in reverse
    runs = torch.repeat_interleave(torch.arange(40), torch.tensor([32, 64, 31, 33, 1, 95, 32, 97] * 5))
    grad_case(F, len(runs), 64, 40, ids=runs)
    grad_case(F, len(runs), 64, 40, ids=runs.flip(0))


def test_gradient_is_summed_in_the_tokens_order(F):
    """Values whose fp32 sum depends on the order: the sum of each unit's rows in order."""
    N = 32
    dout = torch.zeros(N, 8)
    dout[0], dout[1], dout[2] = 2.0 ** 25, 1.0, -2.0 ** 25
    ids = torch.zeros(N, dtype=torch.int64)
    got = F.flce_embedding_backward(dout.cuda(), ids.cuda(), 3)
    assert bool((got[0] == 0).all())  # (2^25 + 1) - 2^25 in fp32
    dout[1], dout[2] = -2.0 ** 25, 1.0
    assert bool((F.flce_embedding_backward(dout.cuda(), ids.cuda(), 3)[0] == 1).all())


def test_gradient_padding_and_shards(F):
    grad_case(F, 2000, 48, 100, padding=7, accumulate=True)
    grad_case(F, 2000, 48, 100, padding=0)
    grad_case(F, 2000, 48, 30, v_offset=50, v_total=100, ids32=True)
    grad_case(F, 2000, 48, 30, v_offset=50, v_total=100, padding=60, accumulate=True)


def test_gradient_bad_ids(F):
    ids = torch.randint(0, 50, (3000,))
    ids[17], ids[2900] = -3, 50
    dout = torch.randn(3000, 16)
    got = F.flce_embedding_backward(dout.cuda(), ids.cuda(), 50)
    ok = (ids >= 0) & (ids < 50)
    want = torch.zeros(50, 16, dtype=torch.float64).index_add_(0, ids[ok], dout[ok].double())
    assert float((got.double().cpu() - want).abs().max()) < 1e-4
    with pytest.raises(F.FlceError) as e:
        F.flce_embedding_backward(dout.cuda(), ids.cuda(), 50, validate=True)
    assert e.value.code == 5


def test_gradient_against_differences(F):
    """The lookup is linear: a step of 1 in one weight changes sum(out * dout) by its gradient."""
    w = torch.randn(6, 5).cuda()
    ids = torch.tensor([3, 1, 3, 3, 0]).cuda()
    dout = torch.randn(5, 5).cuda()
    dw = F.flce_embedding_backward(dout, ids, 6, 2.0)
    f = lambda x: float((F.flce_embedding(ids, x, 2.0).double() * dout.double()).sum())  # noqa: E731
    for v in range(6):
        e = torch.zeros(6, 5).cuda()
        e[v, 2] = 1.0
        assert abs(f(w + e) - f(w) - float(dw[v, 2])) < 1e-4


def test_repeats_and_workspace_contents(F):
    ids = torch.randint(0, 1000, (20000,)).cuda()
    dout = torch.randn(20000, 96).to(torch.bfloat16).cuda()
    p = F.embedding_params(20000, 96, 1000)
    ws = torch.empty(F.embedding_workspace_size(p), dtype=torch.uint8, device="cuda")
    first = F.flce_embedding_backward(dout, ids, 1000, workspace=ws)
    for fill in (0, 255):
        ws.fill_(fill)
        assert torch.equal(first, F.flce_embedding_backward(dout, ids, 1000, workspace=ws))


def test_autograd_stream_and_graph(F):
    ids = torch.randint(0, 500, (3, 700)).cuda()
    w = torch.randn(500, 128).to(torch.bfloat16).cuda().requires_grad_(True)
    out = F.embedding(ids, w, 2.0, padding_idx=3)
    dout = torch.randn(3, 700, 128).to(torch.bfloat16).cuda()
    want = F.flce_embedding_backward(dout, ids, 500, 2.0, 3)
    (g1,) = torch.autograd.grad(out, w, dout, retain_graph=True)
    assert torch.equal(g1, want)
    # an expanded upstream gradient
    (g2,) = torch.autograd.grad(out.sum(), w)
    assert torch.equal(g2, F.flce_embedding_backward(torch.ones_like(dout), ids, 500, 2.0, 3))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = F.flce_embedding_backward(dout, ids, 500, 2.0, 3, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o = F.flce_embedding(ids, w.detach(), 2.0)
        c = F.flce_embedding_backward(dout, ids, 500, 2.0, 3)
    o.zero_()
    c.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out.detach()) and torch.equal(c, want)


def test_tied_table(F):
    """A table that is the head's weight too: the lookup's gradient joins the head's in place."""
    N, H, V = 600, 64, 800
    table = (torch.randn(V, H) / 8).to(torch.bfloat16).cuda()
    ids, labels = torch.randint(0, V, (N,)).cuda(), torch.randint(0, V, (N,)).cuda()
    x = F.flce_embedding(ids, table, 8.0)
    one = torch.ones(1).cuda()
    out = F.flce_forward_backward(x, table, labels, one, None, "mean", weight_layout="vh")
    dh, dw = out[4], out[5]
    head = dw.clone()
    both = F.flce_embedding_backward(dh, ids, V, 8.0, dweight=dw, accumulate=True)
    lookup = F.flce_embedding_backward(dh, ids, V, 8.0, grad_dtype=torch.float32)
    want = (head.float() + lookup).to(torch.bfloat16)
    diff = (both.float() - want.float()).abs()
    # the two roundings can differ by one step of the value
    assert bool((diff <= torch.finfo(torch.bfloat16).eps * want.float().abs()).all())
