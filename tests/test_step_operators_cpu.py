"""Host-side checks of the dense layer, the processed logits and the optimizer that need no GPU:
the C parameters' layout, what the entry points refuse before they look at a device, and what the
Python calls refuse."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_cross_entropy_forward_gb300 as flce
from linear_cross_entropy_forward_gb300 import _binding as B
from linear_cross_entropy_forward_gb300 import adamw as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD_ARG, BAD_SHAPE, ALIGN, WS = 1, 2, 3, 4
PTR = 0x10000  # never read: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    from linear_cross_entropy_forward_gb300.build import build
    build()
    return flce.load_library()


def test_structs_match_the_c_compiler(tmp_path):
    names = [("flce_linear_params", B.FlceLinearParams), ("flce_logits_params", B.FlceLogitsParams),
             ("flce_logits_rows", B.FlceLogitsRows), ("flce_adamw_tensor", B.FlceAdamwTensor),
             ("flce_adamw_params", B.FlceAdamwParams)]
    body = ""
    for name, st in names:
        body += f'printf("%zu\\n", sizeof({name}));'
        for f, _ in st._fields_:
            body += f'printf("%zu\\n", offsetof({name}, {f}));'
    src = tmp_path / "t.c"
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
    # the table that a step fills is an array of the C struct
    assert A._TENSOR.itemsize == ctypes.sizeof(B.FlceAdamwTensor)
    assert [A._TENSOR.fields[f][1] for f, _ in B.FlceAdamwTensor._fields_] == \
        [getattr(B.FlceAdamwTensor, f).offset for f, _ in B.FlceAdamwTensor._fields_]


# ---------------------------------------------------------------------------- dense layer
def layer(**kw):
    p = B.FlceLinearParams(M=16, N=64, K=32, weight_layout=1, activation=2, out_dtype=1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(M=0), 0), (dict(N=1), 0), (dict(N=7), 0), (dict(out_dtype=0), 0),
    (dict(N=7, weight_layout=0), ALIGN), (dict(K=12), ALIGN), (dict(K=0), BAD_SHAPE),
    (dict(M=-1), BAD_SHAPE), (dict(N=0), BAD_SHAPE), (dict(M=1 << 31), BAD_SHAPE),
    (dict(activation=5), BAD_ARG), (dict(activation=-1), BAD_ARG), (dict(weight_layout=2), BAD_ARG),
    (dict(out_dtype=2), BAD_ARG)])
def test_linear_params(lib, kw, code):
    p = layer(**kw)
    assert lib.flce_linear_check_params(ctypes.byref(p)) == code
    for backward in (0, 1):
        assert (lib.flce_linear_workspace_size(ctypes.byref(p), backward) == 0) == (code != 0)


def test_linear_pointers(lib):
    p = layer()

    def forward(x=PTR, w=PTR, b=PTR, r=PTR, y=PTR, z=PTR, ws=PTR, n=256):
        return lib.flce_linear(ctypes.byref(p), x, w, b, r, y, z, ws, n, None)

    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None)):
        assert forward(**kw) == BAD_ARG, kw
    for kw in (dict(x=PTR + 8), dict(w=PTR + 2), dict(b=PTR + 1), dict(r=PTR + 4), dict(y=PTR + 8),
               dict(z=PTR + 2), dict(ws=PTR + 16)):
        assert forward(**kw) == ALIGN, kw
    assert forward(n=255) == WS

    def backward(dout=PTR, x=PTR, w=PTR, z=PTR, dx=PTR, dw=PTR, db=PTR, ws=PTR, n=1 << 20):
        return lib.flce_linear_backward(ctypes.byref(p), dout, x, w, z, dx, dw, db, ws, n, None)

    for kw in (dict(dout=None), dict(x=None), dict(w=None), dict(z=None), dict(ws=None)):
        assert backward(**kw) == BAD_ARG, kw
    for kw in (dict(dout=PTR + 8), dict(dx=PTR + 2), dict(dw=PTR + 4), dict(db=PTR + 1)):
        assert backward(**kw) == ALIGN, kw
    assert backward(n=256) == WS


def test_linear_workspace_holds_dz_and_the_strips(lib):
    p = layer(M=1000, N=1001)
    assert lib.flce_linear_workspace_size(ctypes.byref(p), 0) == 256
    assert lib.flce_linear_workspace_size(ctypes.byref(p), 1) >= 256 + 1000 * 1008 * 2


# ---------------------------------------------------------------------------- logits
def rows(**kw):
    r = B.FlceLogitsRows()
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def logits(**kw):
    p = B.FlceLogitsParams(R=4, V=100, T=0, ld_logits=100, ld_out=100, ignore_index=-100,
                           repetition_penalty=1.0, temperature=1.0, dtype=1, out_dtype=1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(R=0), 0), (dict(temperature=0.0), 0), (dict(out_dtype=0), 0),
    (dict(dtype=0, out_dtype=0), 0), (dict(n_bias=2048), 0), (dict(R=1, ld_out=0), 0),
    (dict(frequency_penalty=-2.0, presence_penalty=-2.0), 0),
    (dict(dtype=3), BAD_ARG), (dict(dtype=0, out_dtype=1), BAD_ARG), (dict(out_dtype=2), BAD_ARG),
    (dict(mask_kind=3), BAD_ARG), (dict(repetition_penalty=0.0), BAD_ARG),
    (dict(repetition_penalty=-1.0), BAD_ARG), (dict(repetition_penalty=NAN), BAD_ARG),
    (dict(repetition_penalty=INF), BAD_ARG), (dict(frequency_penalty=NAN), BAD_ARG),
    (dict(presence_penalty=INF), BAD_ARG), (dict(temperature=-0.5), BAD_ARG),
    (dict(temperature=NAN), BAD_ARG), (dict(R=-1), BAD_SHAPE), (dict(V=0), BAD_SHAPE),
    (dict(V=(1 << 30) + 1), BAD_SHAPE), (dict(T=1 << 30), BAD_SHAPE), (dict(n_bias=2049), BAD_SHAPE),
    (dict(ld_tokens=-1), BAD_SHAPE), (dict(ld_out=99), BAD_SHAPE), (dict(R=1 << 40), BAD_SHAPE)])
def test_logits_params(lib, kw, code):
    assert lib.flce_logits_check_params(ctypes.byref(logits(**kw))) == code


def test_logits_pointers(lib):
    def call(p=None, r=None, x=PTR, y=None, out=PTR, lse=PTR, logp=None, ent=None, ws=None, n=0):
        return lib.flce_logits(ctypes.byref(p or logits()), ctypes.byref(r or rows()), x, y, out, lse,
                               logp, ent, ws, n, None)

    assert call(x=None) == BAD_ARG
    assert call(out=None, lse=None) == BAD_ARG
    assert call(logp=PTR) == BAD_ARG  # of which label?
    assert call(p=logits(T=8)) == BAD_ARG
    assert call(p=logits(n_bias=2), r=rows(bias_ids=PTR)) == BAD_ARG
    assert call(p=logits(mask_kind=1)) == BAD_ARG
    assert call(p=logits(validate=1)) == BAD_ARG
    assert call(p=logits(validate=1), ws=PTR, n=255) == WS
    for kw in (dict(x=PTR + 1), dict(out=PTR + 1), dict(lse=PTR + 2), dict(y=PTR + 4, logp=PTR),
               dict(r=rows(temperature=PTR + 2)), dict(r=rows(lengths=PTR + 2)),
               dict(p=logits(mask_kind=2), r=rows(allowed=PTR + 2)),
               dict(p=logits(T=8, tokens_int64=1), r=rows(tokens=PTR + 4))):
        assert call(**kw) == ALIGN, kw

    def backward(y=PTR, lse=PTR, ent=PTR, gl=PTR, ge=PTR, d=PTR):
        return lib.flce_logits_backward(ctypes.byref(logits()), ctypes.byref(rows()), PTR, y, lse, ent,
                                        gl, ge, d, None, 0, None)

    for kw in (dict(y=None), dict(lse=None), dict(ent=None), dict(d=None)):
        assert backward(**kw) == BAD_ARG, kw
    assert backward(gl=PTR + 2) == ALIGN


# ---------------------------------------------------------------------------- optimizer
def optimizer(**kw):
    p = B.FlceAdamwParams(n_tensors=1, numel=256, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8,
                          grad_scale=1.0, max_norm=0.0, state_bits=32)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def tensor(**kw):
    t = B.FlceAdamwTensor(param=PTR, grad=PTR, n=200, offset=0, weight_decay=0.1, dtype=1, grad_dtype=1)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(beta1=0.0, beta2=0.0, eps=0.0, lr=0.0), 0), (dict(state_bits=8), 0),
    (dict(n_tensors=0, numel=0), 0), (dict(state_bits=16), BAD_ARG), (dict(beta1=1.0), BAD_ARG),
    (dict(beta2=-0.1), BAD_ARG), (dict(beta2=NAN), BAD_ARG), (dict(lr=-1.0), BAD_ARG),
    (dict(lr=INF), BAD_ARG), (dict(eps=-1e-8), BAD_ARG), (dict(max_norm=-1.0), BAD_ARG),
    (dict(grad_scale=INF), BAD_ARG), (dict(n_tensors=-1), BAD_SHAPE), (dict(numel=100), BAD_SHAPE),
    (dict(numel=-128), BAD_SHAPE)])
def test_adamw_params(lib, kw, code):
    p = optimizer(**kw)
    assert lib.flce_adamw_check_params(ctypes.byref(p)) == code
    assert (lib.flce_adamw_workspace_size(ctypes.byref(p)) == 0) == (code != 0)


def test_adamw_pointers(lib):
    def call(p=None, t=None, master=None, m=PTR, v=PTR, sm=None, ss=None, lr=None, norm=None, step=PTR,
             ws=PTR, n=256):
        p, t = p or optimizer(), t or tensor()
        return lib.flce_adamw_step(ctypes.byref(p), ctypes.addressof(t), master, m, v, sm, ss, lr, norm,
                                   step, ws, n, None)

    for kw in (dict(m=None), dict(v=None), dict(step=None), dict(ws=None), dict(t=tensor(param=None)),
               dict(t=tensor(grad=None)), dict(t=tensor(dtype=3, grad_dtype=3)),
               dict(t=tensor(grad_dtype=2)), dict(t=tensor(weight_decay=-1.0)),
               dict(t=tensor(weight_decay=NAN)), dict(p=optimizer(state_bits=8), sm=PTR),
               dict(p=optimizer(max_norm=1.0)), dict(p=optimizer(skip_nonfinite=1))):
        assert call(**kw) == BAD_ARG, kw
    for kw in (dict(t=tensor(offset=128)), dict(t=tensor(offset=-128)), dict(t=tensor(offset=64)),
               dict(t=tensor(n=257)), dict(t=tensor(n=-1))):
        assert call(**kw) == BAD_SHAPE, kw
    for kw in (dict(m=PTR + 16), dict(master=PTR + 4), dict(step=PTR + 4), dict(ws=PTR + 8),
               dict(lr=PTR + 2), dict(t=tensor(grad=PTR + 1)),
               dict(t=tensor(grad_dtype=0, grad=PTR + 2))):
        assert call(**kw) == ALIGN, kw
    assert call(n=255) == WS
    assert lib.flce_adamw_step(ctypes.byref(optimizer()), None, None, PTR, PTR, None, None, None, None,
                               PTR, PTR, 256, None) == BAD_ARG

    def norm(p=None, t=None, out=PTR, ws=PTR, n=1 << 20):
        p, t = p or optimizer(), t or tensor(param=None)
        return lib.flce_grad_norm(ctypes.byref(p), ctypes.addressof(t), out, ws, n, None)

    assert norm(out=None) == BAD_ARG and norm(ws=None) == BAD_ARG
    assert norm(t=tensor(grad=None)) == BAD_ARG
    assert norm(out=PTR + 2) == ALIGN and norm(n=256) == WS


# ---------------------------------------------------------------------------- Python calls
def test_python_calls_refuse_cpu_tensors(lib):
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    for call in (lambda: flce.flce_linear(x, w), lambda: flce.linear(x, w),
                 lambda: flce.flce_linear_backward(torch.zeros(4, 16), x, w),
                 lambda: flce.flce_process_logits(torch.zeros(2, 8)),
                 lambda: flce.logits_logprob(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_python_values(lib):
    with pytest.raises(ValueError, match="activation"):
        flce.linear_params(1, 8, 8, activation="swish")
    with pytest.raises(TypeError, match="out_dtype"):
        flce.linear_params(1, 8, 8, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="weight_layout"):
        flce.linear_params(1, 8, 8, weight_layout="kn")
    with pytest.raises(flce.FlceError, match="ALIGN"):
        flce.linear_workspace_size(flce.linear_params(1, 8, 12))
    with pytest.raises(ValueError, match="at least one"):
        flce.AdamW([])
    with pytest.raises(ValueError, match="state_bits"):
        flce.AdamW([torch.zeros(4)], state_bits=16)
    with pytest.raises(ValueError, match="max_norm"):
        flce.AdamW([torch.zeros(4)], max_norm=0.0)
