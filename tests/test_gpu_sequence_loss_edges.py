"""Edges of the losses over sequences."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_cross_entropy_forward_gb300.build import build
    build()
    import linear_cross_entropy_forward_gb300 as pkg
    return pkg


def round_tokens():
    """Tokens of which every warp of the GPU takes one piece."""
    return torch.cuda.get_device_properties(0).multi_processor_count * 32 * 256


def test_threads_whose_launches_keep_different_amounts(F):
    """Two and four pieces per warp, whose gradients wait in shared memory of different sizes."""
    per = round_tokens()
    wrong = []

    def work(rounds):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                lp = torch.zeros(int((rounds - 0.5) * per), device="cuda")
                adv = torch.ones(1, device="cuda")
                p, _ = F.policy_params(lp, None, adv)
                ws = torch.empty(F.policy_workspace_size(p), dtype=torch.uint8, device="cuda")
                for k in range(1500):
                    out = F.flce_policy_loss(lp, None, adv, workspace=ws)
                    if k % 16 == 15:
                        s.synchronize()
                if float(out[0]) != -1.0:
                    wrong.append(float(out[0]))
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(r,)) for r in (2, 4, 3, 4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
