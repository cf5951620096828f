"""What the calls write into tensors of the caller's is seen by autograd: a backward that saved such a
tensor raises, as it does after torch's own in-place operations, instead of using the new values."""
import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce

pytestmark = pytest.mark.gpu
CHANGED = "modified by an inplace operation"


def bf16(*shape, grad=False):
    return torch.randn(*shape, device="cuda").bfloat16().requires_grad_(grad)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_between_a_forward_and_its_backward(bits):
    x, w = bf16(4, 16), bf16(24, 16, grad=True)
    opt = flce.AdamW([w], state_bits=bits, master=True)
    y = flce.linear(x.requires_grad_(True), w, weight_layout="vh")
    opt.step([torch.ones_like(w)])
    with pytest.raises(RuntimeError, match=CHANGED):
        y.float().sum().backward()
    # behind the step everything is as ever
    flce.linear(x, w, weight_layout="vh").float().sum().backward()
    assert bool(torch.isfinite(w.grad).all())


def test_states_and_views_of_one_tensor():
    flat = torch.zeros(300, device="cuda")
    opt = flce.AdamW([flat[:100], flat[128:]], master=True)
    seen = [flat, *opt.state_dict().values()]
    before = [t._version for t in seen]
    opt.step([torch.ones(100, device="cuda"), torch.ones(172, device="cuda")])
    assert all(t._version > v for t, v in zip(seen, before))
    with torch.inference_mode():
        p = torch.zeros(10, device="cuda")  # has no version
        flce.AdamW([p], lr=0.5, weight_decay=0.0).step([torch.ones(10, device="cuda")])
        assert float((p + 0.5).abs().max()) < 1e-5


def test_processed_in_place():
    x = torch.randn(3, 100, device="cuda")
    labels = torch.arange(3, device="cuda")
    leaf = torch.zeros_like(x).requires_grad_(True)
    logits = leaf + x
    logp, _ = flce.logits_logprob(logits, labels)
    with torch.no_grad():
        flce.flce_process_logits(logits, out=logits, temperature=0.5)
    with pytest.raises(RuntimeError, match=CHANGED):
        logp.sum().backward()
    # a mask in memory that another call writes
    allowed = torch.zeros(3, 100, device="cuda")
    logp, _ = flce.logits_logprob(leaf + x, labels, bias_ids=labels[None].expand(3, -1),
                                  bias_values=allowed[:, :3])
    flce.flce_process_logits(x, out=allowed)
    with pytest.raises(RuntimeError, match=CHANGED):
        logp.sum().backward()


def test_outputs_of_the_dense_layer():
    x, w, r = bf16(6, 16), bf16(24, 16), bf16(6, 24)
    a = bf16(6, 24, grad=True)
    y = a * r  # saves r
    flce.flce_linear(x, w, residual=r, weight_layout="vh", out=r)
    with pytest.raises(RuntimeError, match=CHANGED):
        y.float().sum().backward()
    outs = [bf16(6, 16), bf16(24, 16), bf16(24)]
    before = [t._version for t in outs]
    flce.flce_linear_backward(r, x, w, weight_layout="vh", out=outs)
    assert all(t._version > v for t, v in zip(outs, before))
    before = [t._version for t in outs]
    flce.flce_linear_backward(r, x, w, weight_layout="vh", need_dx=False, out=outs)
    assert [t._version > v for t, v in zip(outs, before)] == [False, True, True]


def test_captured_and_replayed():
    w, g = torch.zeros(100, device="cuda"), torch.ones(100, device="cuda")
    opt = flce.AdamW([w], lr=0.1, weight_decay=0.0)
    opt.step([g])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step([g])
    graph.replay()
    torch.cuda.synchronize()
    assert int(opt.step_count) == 2 and float((w + 0.2).abs().max()) < 1e-5
