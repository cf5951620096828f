"""Host-side checks of the sequence losses and the embedding that need no GPU: the C
parameters' layout, what the entry points refuse before they look at a device, and what the
Python calls refuse."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce
from linear_cross_entropy_forward_gb300 import _binding as B
from linear_cross_entropy_forward_gb300 import losses as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD_ARG, BAD_SHAPE, ALIGN, WS = 1, 2, 3, 4
PTR = 0x10000  # never read: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    from linear_cross_entropy_forward_gb300.build import build
    build()
    return flce.load_library()


def test_structs_match_the_c_compiler(tmp_path):
    src = tmp_path / "t.c"
    names = [("flce_seqs", B.FlceSeqs), ("flce_policy_params", B.FlcePolicyParams),
             ("flce_preference_params", B.FlcePreferenceParams),
             ("flce_embedding_params", B.FlceEmbeddingParams)]
    body = ""
    for name, st in names:
        body += f'printf("%zu\\n", sizeof({name}));'
        for f, _ in st._fields_:
            body += f'printf("%zu\\n", offsetof({name}, {f}));'
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "flce.h"\nint main(void){%s return 0;}'
                   % body)
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for _, st in names:
        want.append(ctypes.sizeof(st))
        want += [getattr(st, f).offset for f, _ in st._fields_]
    assert got == want


def seqs(**kw):
    q = B.FlceSeqs(B=4, S=10, cu_kind=0, mask_kind=0, dtype=0, ld_mask=10, ignore_index=-100)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def policy(seq=None, **kw):
    p = B.FlcePolicyParams(seqs=seq or seqs(), ld_logp=10, ld_old=10, ld_ref=10, ld_entropy=10,
                           ld_adv=10, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0,
                           entropy_coef=0.0, scale=1.0, kl=3, ratio=0, aggregate=0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def preference(seq=None, **kw):
    p = B.FlcePreferenceParams(seqs=seq or seqs(), ld_logp=10, ld_ref=10, beta=0.1, reduction=1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def embedding(**kw):
    p = B.FlceEmbeddingParams(N=16, H=64, V=100, padding_idx=-1, scale=1.0, dtype=1, grad_dtype=1,
                              ids_int64=1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD_SEQS = [(dict(B=-1), BAD_SHAPE), (dict(S=-1), BAD_SHAPE), (dict(B=1 << 40), BAD_SHAPE),
            (dict(B=1 << 20, S=1 << 30), BAD_SHAPE), (dict(dtype=3), BAD_ARG),
            (dict(cu_kind=3, cu_seqlens=PTR), BAD_ARG), (dict(cu_kind=1), BAD_ARG),
            (dict(cu_seqlens=PTR), BAD_ARG), (dict(mask_kind=1), BAD_ARG),
            (dict(mask=PTR), BAD_ARG), (dict(cu_kind=1, cu_seqlens=PTR + 2), ALIGN),
            (dict(cu_kind=2, cu_seqlens=PTR + 4), ALIGN), (dict(mask_kind=2, mask=PTR + 4), ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_SEQS)
def test_layouts_refused(lib, kw, code):
    for name, p in (("policy", policy(seqs(**kw))), ("preference", preference(seqs(**kw)))):
        assert getattr(lib, f"flce_{name}_check_params")(ctypes.byref(p)) == code
        assert getattr(lib, f"flce_{name}_workspace_size")(ctypes.byref(p)) == 0


@pytest.mark.parametrize("kw", [dict(clip_low=1.0), dict(clip_low=-0.1), dict(clip_high=-1.0),
                                dict(clip_high=float("nan")), dict(dual_clip=1.0),
                                dict(dual_clip=-2.0), dict(kl_coef=float("nan")),
                                dict(entropy_coef=float("inf")), dict(scale=float("nan")),
                                dict(kl=0), dict(kl=4), dict(ratio=2), dict(aggregate=4),
                                dict(adv_per_token=2), dict(ratio=1, adv_per_token=1)])
def test_policy_parameters_refused(lib, kw):
    assert lib.flce_policy_check_params(ctypes.byref(policy(**kw))) == BAD_ARG


def test_negative_strides_refused(lib):
    for f in ("ld_logp", "ld_old", "ld_ref", "ld_entropy", "ld_adv"):
        assert lib.flce_policy_check_params(ctypes.byref(policy(**{f: -1}))) == BAD_ARG
    for f in ("ld_logp", "ld_ref"):
        assert lib.flce_preference_check_params(ctypes.byref(preference(**{f: -1}))) == BAD_ARG
    assert lib.flce_policy_check_params(ctypes.byref(policy(seqs(ld_mask=-1)))) == BAD_ARG


def test_policy_pointers_refused(lib):
    p = policy()
    need = lib.flce_policy_workspace_size(ctypes.byref(p))
    assert need > 0

    def call(p=p, logp=PTR, old=PTR, ref=None, ent=None, adv=PTR, g=None, loss=PTR, stats=PTR,
             counts=PTR, dlogp=PTR, dent=None, ws=PTR, size=need):
        return lib.flce_policy_loss(ctypes.byref(p), logp, old, ref, ent, adv, g, loss, stats, counts,
                                    dlogp, dent, ws, size, None)

    assert call(logp=None) == BAD_ARG and call(adv=None) == BAD_ARG and call(ws=None) == BAD_ARG
    assert call(loss=None) == BAD_ARG and call(stats=None) == BAD_ARG
    assert call(loss=None, stats=None, counts=None, dlogp=None) == BAD_ARG
    assert call(dent=PTR) == BAD_ARG
    assert call(p=policy(kl_coef=0.1)) == BAD_ARG and call(p=policy(entropy_coef=0.1)) == BAD_ARG
    assert call(logp=PTR + 2) == ALIGN and call(adv=PTR + 2) == ALIGN and call(ws=PTR + 8) == ALIGN
    assert call(counts=PTR + 4) == ALIGN and call(g=PTR + 1) == ALIGN
    assert call(size=need - 1) == WS
    assert lib.flce_policy_loss(None, *[PTR] * 12, need, None) == BAD_ARG


@pytest.mark.parametrize("kw", [dict(beta=0.0), dict(beta=float("inf")), dict(margin=float("nan")),
                                dict(kind=4), dict(reduction=3), dict(label_smoothing=0.5),
                                dict(label_smoothing=-0.1), dict(kind=2, label_smoothing=0.1),
                                dict(kind=3, label_smoothing=0.1), dict(interleaved=2),
                                dict(length_normalised=2), dict(nll_coef=float("nan"))])
def test_preference_parameters_refused(lib, kw):
    assert lib.flce_preference_check_params(ctypes.byref(preference(**kw))) == BAD_ARG


def test_preference_pointers_refused(lib):
    assert lib.flce_preference_check_params(ctypes.byref(preference(seqs(B=3)))) == BAD_SHAPE
    p = preference()
    need = lib.flce_preference_workspace_size(ctypes.byref(p))

    def call(logp=PTR, ref=None, scores=None, g=None, loss=PTR, rewards=PTR, dlogp=PTR, ws=PTR, size=need):
        return lib.flce_preference_loss(ctypes.byref(p), logp, ref, scores, g, loss, rewards, dlogp,
                                        ws, size, None)

    assert call(logp=None) == BAD_ARG and call(ws=None) == BAD_ARG and call(rewards=None) == BAD_ARG
    assert call(loss=None, dlogp=None) == BAD_ARG
    assert call(ref=PTR + 2) == ALIGN and call(scores=PTR + 2) == ALIGN
    assert call(size=need - 1) == WS


@pytest.mark.parametrize("kw,code", [(dict(N=-1), BAD_SHAPE), (dict(H=0), BAD_SHAPE),
                                     (dict(V=0), BAD_SHAPE), (dict(V=1 << 31), BAD_SHAPE),
                                     (dict(H=1 << 29), BAD_SHAPE), (dict(dtype=5), BAD_ARG),
                                     (dict(dtype=0, grad_dtype=1), BAD_ARG),
                                     (dict(dtype=1, grad_dtype=2), BAD_ARG),
                                     (dict(scale=float("inf")), BAD_ARG),
                                     (dict(v_offset=5), BAD_ARG),
                                     (dict(v_offset=50, v_total=120), BAD_SHAPE),
                                     (dict(padding_idx=100), BAD_ARG), (dict(padding_idx=-2), BAD_ARG),
                                     (dict(ids_int64=2), BAD_ARG), (dict(accumulate=2), BAD_ARG)])
def test_embedding_parameters_refused(lib, kw, code):
    assert lib.flce_embedding_check_params(ctypes.byref(embedding(**kw))) == code


def test_embedding_pointers_refused(lib):
    p = embedding()
    need = lib.flce_embedding_workspace_size(ctypes.byref(p))
    bwd = lambda dout=PTR, ids=PTR, dw=PTR, ws=PTR, size=need: lib.flce_embedding_backward(  # noqa: E731
        ctypes.byref(p), dout, ids, dw, ws, size, None)
    assert bwd(dout=None) == BAD_ARG and bwd(ids=None) == BAD_ARG and bwd(dw=None) == BAD_ARG
    assert bwd(ws=None) == BAD_ARG and bwd(ids=PTR + 4) == ALIGN and bwd(dw=PTR + 1) == ALIGN
    assert bwd(size=need - 1) == WS
    fwd = lambda ids=PTR, w=PTR, out=PTR, ws=None, size=0: lib.flce_embedding(  # noqa: E731
        ctypes.byref(p), ids, w, out, ws, size, None)
    assert fwd(ids=None) == BAD_ARG and fwd(w=None) == BAD_ARG and fwd(out=PTR + 1) == ALIGN
    p.validate = 1
    assert fwd() == BAD_ARG and fwd(ws=PTR, size=100) == WS


def test_head_parameters_refused(lib):
    def size(N=10, q=None, **kw):
        p = flce.make_params(N, 64, 512, "none", **kw)
        return lib.flce_policy_head_workspace_size(
            ctypes.byref(p), ctypes.byref(q or policy(seqs(B=1, S=N))))

    assert size() > 0
    assert size(zloss_coef=0.1) == 0 and size(label_smoothing=0.1) == 0
    assert size(v_offset=0, v_total=1024) == 0
    assert size(q=policy(seqs(B=1, S=9))) == 0 and size(q=policy(seqs(B=2, S=5))) == 0
    assert size(q=policy(seqs(B=1, S=10, dtype=1))) == 0
    many = seqs(B=1, S=2000)
    assert size(N=2000, q=policy(many, ratio=1), chunk_n=512) == 0
    assert size(N=2000, q=policy(many, ratio=1)) > 0
    p = flce.make_params(10, 64, 512, "mean")
    assert lib.flce_policy_head_workspace_size(ctypes.byref(p), ctypes.byref(policy(seqs(B=1)))) == 0


def test_python_calls_need_cuda_tensors():
    x, a = torch.zeros(4, 8), torch.zeros(4)
    ids, w = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    for call in (lambda: flce.flce_policy_loss(x, x, a), lambda: flce.policy_loss(x, x, a),
                 lambda: flce.flce_preference_loss(x), lambda: flce.preference_loss(x),
                 lambda: flce.flce_embedding(ids, w), lambda: flce.embedding(ids, w),
                 lambda: flce.flce_embedding_backward(w[:3], ids, 5)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_names_refused():
    for table, value in ((L._KL, "k4"), (L._RATIO, "tokens"), (L._AGGREGATE, "mean"),
                         (L._PREFERENCE, "dpo"), (L._PAIRS, ["halves"])):
        with pytest.raises(ValueError, match="must be one of"):
            L._code(table, value, "x")


def test_random_cuts_of_the_token_axis():
    """The losses cut a packed axis into numbered pieces, piece i + j being sequence i's part of
    tile j.  Whatever the lengths, every token of a sequence is in one piece, and the pieces of a
    sequence are the numbers between its first and its last."""
    import random
    rng = random.Random(3)
    T = 256
    for _ in range(200):
        n, total = rng.choice([1, 2, 5, 31, 33, 300]), rng.choice([0, 1, 255, 256, 257, 5000])
        cu = sorted(rng.randint(0, total) for _ in range(n + 1))
        first = [c // T + i for i, c in enumerate(cu)]
        assert all(b > a for a, b in zip(first, first[1:]))
        seen = [0] * total
        for u in range(total // T + n + 1):
            i = max((k for k in range(n) if first[k] <= u), default=-1)
            if i < 0:
                continue
            lo, hi = max(cu[i], (u - i) * T), min(cu[i + 1], (u - i + 1) * T)
            for p in range(lo, hi):
                seen[p] += 1
            if hi > lo:
                assert first[i] <= u <= (cu[i + 1] - 1) // T + i
        assert seen == [int(cu[0] <= p < cu[n]) for p in range(total)]
