"""The example's steps: they learn, and a policy step's gradient of the tied table is the
definition's."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "tied_policy_step.py")


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    spec = importlib.util.spec_from_file_location("tied_policy_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_losses_fall(ex):
    policy, preference = ex.main(steps=12, quiet=True)
    assert all(math.isfinite(x) for x in policy + preference)
    assert policy[-1] < policy[0] and preference[-1] < preference[0]
    # before the first update the policy is the reference: -ln sig(0)
    assert abs(preference[0] - math.log(2)) < 1e-4


def test_tied_gradient_is_the_definitions(ex):
    """Both uses of the table in one fp64 graph.  The head's gradients are within its bound
    (1e-2 relative: dlogits rounded to bf16), and so is their sum."""
    g = torch.Generator().manual_seed(3)
    table = (torch.randn(ex.V, ex.H, generator=g) / 8).to(torch.bfloat16).cuda()
    ids = torch.randint(0, ex.V, (ex.B, ex.S), generator=g).cuda()
    labels = ex.next_labels(ids, 16).view(-1)
    adv = torch.randn(ex.B, generator=g).cuda()
    old = ex.log_probs(table, ids, 16) + 0.1 * torch.randn(ex.B * ex.S, generator=g).cuda()
    before = table.clone()
    new = table.clone()
    loss, _, _ = ex.policy_step(new, ids, 16, adv, old, old, lr=1.0)
    # the step itself: bf16(table - grad); here from the calls' own gradient
    hidden = ex.hidden_states(before, ids)
    out = ex.flce.flce_policy_forward_backward(
        hidden, before, labels, old, adv, ref_logp=old, cu_seqlens=ex.sequence_ends("cuda"),
        clip_low=0.2, clip_high=0.28, kl_coef=0.01, entropy_coef=0.001,
        aggregate="seq_mean_token_mean", weight_layout="vh")
    grad = ex.add_lookup_gradient(out[6], out[5], ids)
    assert torch.equal(new, before.sub(grad, alpha=1.0)) and torch.equal(out[0], loss)

    w = before.double().requires_grad_(True)
    x = w[ids] * math.sqrt(ex.H)
    h = x + torch.nn.functional.pad(x[:, :-1], (0, 0, 1, 0))
    # the head reads the hidden states that the lookup and the addition rounded to bf16
    h = h + (hidden.double().view_as(h) - h).detach()
    logq = torch.log_softmax(h.reshape(-1, ex.H) @ w.t(), 1)
    m = labels != -100
    lp = logq.gather(1, labels.clamp(min=0)[:, None])[:, 0][m]
    ent = -(logq.exp() * logq).sum(1)[m]
    o = old.double()[m]
    a = adv.double().repeat_interleave(ex.S)[m]
    r = (lp - o).exp()
    obj = torch.minimum(r * a, r.clamp(0.8, 1.28) * a)
    e = o - lp
    per = -obj + 0.01 * (torch.expm1(e) - e) - 0.001 * ent
    n = m.view(ex.B, ex.S).sum(1)
    want = (per / n.repeat_interleave(ex.S)[m]).sum() / ex.B
    want.backward()
    want = want.detach()
    assert abs(float(loss) - float(want)) < 1e-4 * max(1.0, abs(float(want)))
    rel = float((grad.double() - w.grad).norm() / w.grad.norm())
    assert rel < 1e-2, rel


def _functions(ex):
    """Each differentiable call as (leaf, scalar of the leaf)."""
    F = ex.flce
    g = torch.Generator().manual_seed(5)
    lp = -torch.rand(4, 700, generator=g).cuda()
    adv = torch.randn(4, generator=g).cuda()
    table = torch.randn(50, 64, generator=g).cuda()
    ids = torch.randint(0, 50, (300,), generator=g).cuda()
    up = torch.randn(300, 64, generator=g).cuda()
    return {"policy": (lp, lambda x: F.policy_loss(x, lp - 0.1, adv)[0]),
            "policy_bf16": (lp.bfloat16(), lambda x: F.policy_loss(x, lp.bfloat16(), adv)[0]),
            "preference": (lp, lambda x: F.preference_loss(x, lp * 0.5)[0]),
            "embedding": (table, lambda x: (F.embedding(ids, x, 2.0) * up).sum())}


@pytest.mark.parametrize("name", ["policy", "policy_bf16", "preference", "embedding"])
def test_backward_passes_replay_from_a_graph(ex, name):
    """The gradient of a leaf captured on a stream of its own (torch.autograd.grad: a backward()
    into .grad would also need the leaf's accumulation on that stream)."""
    leaf, f = _functions(ex)[name]
    x = leaf.clone().requires_grad_(True)
    (want,) = torch.autograd.grad(f(x), x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.autograd.grad(f(x), x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        (got,) = torch.autograd.grad(f(x), x)
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", ["policy", "preference", "embedding"])
def test_second_derivatives_are_refused(ex, name):
    leaf, f = _functions(ex)[name]
    x = leaf.clone().requires_grad_(True)
    (g,) = torch.autograd.grad(f(x) ** 2, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_gradient_of_a_broadcast_input(ex):
    F = ex.flce
    base = -torch.rand(1, 700).cuda().requires_grad_(True)
    adv = torch.randn(4).cuda()
    old = base.detach().expand(4, 700) - 0.05
    loss, _, _ = F.policy_loss(base.expand(4, 700), old, adv)
    (got,) = torch.autograd.grad(loss, base)
    full = F.flce_policy_loss(base.detach().expand(4, 700), old, adv)[3]
    assert torch.allclose(got, full.sum(0, keepdim=True), rtol=1e-6, atol=1e-9)


def test_calls_on_several_streams_and_threads(ex):
    """Cooperative grids, clusters and the head's GEMMs side by side: the same results."""
    import threading
    F = ex.flce
    g = torch.Generator().manual_seed(9)
    lp = -torch.rand(64, 2000, generator=g).cuda()
    adv = torch.randn(64, generator=g).cuda()
    ids = torch.randint(0, 3000, (70000,), generator=g).cuda()
    dout = torch.randn(70000, 32, generator=g).cuda()
    hidden = torch.randn(512, 256, generator=g).to(torch.bfloat16).cuda()
    weight = torch.randn(256, 2048, generator=g).to(torch.bfloat16).cuda()
    labels = torch.randint(0, 2048, (512,), generator=g).cuda()
    one = torch.ones(1, device="cuda")

    def calls():
        return [F.flce_policy_loss(lp, lp - 0.1, adv)[3], F.flce_preference_loss(lp)[2],
                F.flce_embedding_backward(dout, ids, 3000),
                F.flce_forward_backward(hidden, weight, labels, one, None)[5],
                F.flce_policy_loss(lp[:4, :100], None, adv[:4])[3]]

    want = calls()
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(25):
                got = calls()
                s.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, want)):
                    wrong.append(1)
                del got

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
