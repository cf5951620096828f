"""Cases of the dense layer, the processed logits and the optimizer step, their plain forms and
their 64-bit values.

`run` computes a case with elementary torch operations where `own` is false, and through
the package's public calls where it is true.  The operators:

linear        y = act(x W + b) + r, the product with its epilogue;
linear_train  the same and its gradients, through autograd;
logits        penalties for repeated tokens, biases, a mask of allowed tokens and the
              temperature on rows of logits, with each row's logsumexp;
logprob       log-probability and entropy of given tokens under that distribution, and the
              gradient by the logits, through autograd;
adamw         gradient norm, clipping and an AdamW step over many tensors, states in 32 or
              8 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
BLOCK = 128  # elements that share a scale of the 8-bit states; tensors start at multiples of it


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a square layer of a 4096-wide model: the weight's bytes and the latency
        dict(name="linear_token", op="linear", M=1, K=4096, N=4096, layout="vh", act="none",
             bias=True, res=True, out="bf16"),
        # the logits of a decode batch over the 128256-token head, fp32 for the sampler
        dict(name="linear_decode_logits", op="linear", M=24, K=4096, N=128256, layout="vh",
             act="none", bias=False, res=False, out="fp32"),
        # the wide layer of a training step of 8192 tokens
        dict(name="linear_train_wide", op="linear_train", M=8192, K=4096, N=16384, layout="vh",
             act="gelu", bias=True, res=False, out="bf16"),
        # a ragged batch through a layer with an odd number of outputs, added to its residual
        dict(name="linear_train_ragged", op="linear_train", M=2999, K=2304, N=1001, layout="vh",
             act="silu", bias=True, res=True, out="bf16"),
        # one sequence being sampled, a few hundred tokens in
        dict(name="logits_one_row", op="logits", R=1, V=32000, T=300, dtype="fp32", rep=True,
             freq=False, pres=False, bias=0, allowed="none", temp=True),
        # a decode batch of a constrained generation: every option at once
        dict(name="logits_decode_batch", op="logits", R=64, V=128256, T=2048, dtype="fp32",
             rep=True, freq=True, pres=True, bias=48, allowed="bits", temp=True),
        # a rollout batch over the largest table, long histories
        dict(name="logits_rollout_batch", op="logits", R=384, V=256000, T=8192, dtype="bf16",
             rep=True, freq=True, pres=True, bias=0, allowed="none", temp=True),
        # the sampled tokens of a short constrained answer
        dict(name="logprob_small", op="logprob", R=16, V=4096, T=100, dtype="fp32", rep=False,
             freq=False, pres=False, bias=0, allowed="bits", temp=True),
        # a chunk of rollout tokens scored under the distribution they were sampled from
        dict(name="logprob_rollout_chunk", op="logprob", R=700, V=152064, T=1500, dtype="bf16",
             rep=True, freq=False, pres=True, bias=0, allowed="bytes", temp=True),
        # the small head: a few tensors, latency is everything
        dict(name="adamw_small", op="adamw", total=2_100_000, count=5, split=1, dtype="bf16",
             grad="bf16", master=True, bits=32, clip=True),
        # a tied 128256 x 4096 table with a few layers, fp32 masters beside bf16 weights
        dict(name="adamw_tied_table", op="adamw", total=600_000_000, count=24, split=2,
             dtype="bf16", grad="bf16", master=True, bits=32, clip=True),
        # many tensors of all sizes with the moments in 8 bits
        dict(name="adamw_many_8bit", op="adamw", total=300_000_000, count=290, split=3,
             dtype="bf16", grad="bf16", master=True, bits=8, clip=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "linear_train", "logits", "logprob", "adamw", "adamw"])
    if op in ("linear", "linear_train"):
        layout = rng.choice(["vh", "vh", "hv"])
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        bias = rng.random() < 0.7
        K = 8 * _log(rng, 16, 1000)
        if op == "linear":
            M = rng.choice([_log(rng, 1, 16), _log(rng, 2, 700), _log(rng, 200, 9000)])
        else:
            M = _log(rng, 60, 9000)
        N = _log(rng, 100, 60000 if M < 300 else 12000)
        if layout == "hv":
            N = (N + 7) // 8 * 8
        out = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, M=M, K=K, N=N, layout=layout, act=act, bias=bias,
                    res=rng.random() < 0.5, out=out)
    if op in ("logits", "logprob"):
        V = rng.choice([_log(rng, 500, 250000), 128256, 152064, 32000, 50257])
        most = 90_000_000 if op == "logits" else 60_000_000
        R = min(_log(rng, 1, 512), max(1, most // V))
        return dict(op=op, R=R, V=V, T=_log(rng, 1, 16000 if op == "logits" else 3000),
                    dtype=rng.choice(["fp32", "bf16", "bf16", "fp16"]), rep=rng.random() < 0.7,
                    freq=rng.random() < 0.5, pres=rng.random() < 0.5,
                    bias=rng.choice([0, 0, _log(rng, 1, 300)]),
                    allowed=rng.choice(["none", "bits", "bytes"]), temp=rng.random() < 0.7)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    total = _log(rng, 20_000, 200_000_000)
    return dict(op=op, total=total, count=min(_log(rng, 1, 250), max(1, total // 300)),
                split=rng.randrange(1, 1 << 30), dtype=dtype,
                grad=rng.choice([dtype, "fp32"]), master=dtype != "fp32" and rng.random() < 0.7,
                bits=rng.choice([32, 8]), clip=rng.random() < 0.7)


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_linear(c, seed):
    g = _gen(seed)
    M, K, N = c["M"], c["K"], c["N"]
    s = dict(c)
    s["x"] = _randn(g, M, K).bfloat16()
    shape = (N, K) if c["layout"] == "vh" else (K, N)
    s["w"] = (_randn(g, *shape) / math.sqrt(K)).bfloat16()
    s["b"] = (0.5 * _randn(g, N)).bfloat16() if c["bias"] else None
    s["r"] = _randn(g, M, N).to(DT[c["out"]]) if c["res"] else None
    if c["op"] == "linear_train":
        s["gy"] = _randn(g, M, N).to(DT[c["out"]])
        for k in ("x", "w", "b", "r"):
            if s[k] is not None:
                s[k].requires_grad_(True)
    return s


def _prepare_logits(c, seed):
    g = _gen(seed)
    R, V, T = c["R"], c["V"], c["T"]
    s = dict(c, allowed_kind=c["allowed"])
    s["logits"] = (3.0 * _randn(g, R, V)).to(DT[c["dtype"]])
    # repeated tokens: ids crowd at the low end, as ids of frequent tokens do
    u = torch.rand(R, T, generator=g, device="cuda")
    s["tokens"] = (u.pow(4) * V).long().clamp_(max=V - 1)
    s["lengths"] = torch.randint(0, T + 1, (R,), generator=g, device="cuda")
    s["prompt_lens"] = (s["lengths"] * torch.rand(R, generator=g, device="cuda")).long()
    rand = torch.rand(4, R, generator=g, device="cuda")
    s["repetition_penalty"] = 0.8 + 0.7 * rand[0] if c["rep"] else None
    s["frequency_penalty"] = 0.4 * rand[1] if c["freq"] else None
    s["presence_penalty"] = rand[2] - 0.3 if c["pres"] else None
    s["temperature"] = 0.4 + 0.9 * rand[3] if c["temp"] else None
    s["bias_ids"] = s["bias_values"] = None
    if c["bias"]:
        s["bias_ids"] = torch.randint(-1, V, (R, c["bias"]), generator=g, device="cuda")
        s["bias_values"] = 4.0 * _randn(g, R, c["bias"])
    s["allowed"] = None
    if c["allowed"] != "none":
        ok = torch.rand(R, V, generator=g, device="cuda") < 0.3
        ok[:, : V // 50 + 1] = True
        if c["allowed"] == "bits":  # bit v % 32 of word v // 32
            W = (V + 31) // 32
            ok = torch.nn.functional.pad(ok, (0, W * 32 - V)).view(R, W, 32).long()
            word = (ok << torch.arange(32, device="cuda")).sum(-1)
            s["allowed"] = torch.where(word >= 1 << 31, word - (1 << 32), word).int()
        else:
            s["allowed"] = ok
    if c["op"] == "logprob":
        s["labels"] = (torch.rand(R, generator=g, device="cuda") * (V // 50 + 1)).long()
        s["labels"][torch.rand(R, generator=g, device="cuda") < 0.1] = -100
        s["g_logp"], s["g_ent"] = _randn(g, R), 0.1 * _randn(g, R)
        s["logits"].requires_grad_(True)
    return s


def _shapes(c):
    """Numbers of elements of the case's tensors: a few large, many small, odd ones among them."""
    r = np.random.RandomState(c["split"])
    share = r.dirichlet(np.full(c["count"], 0.5))
    return [max(1, int(x)) for x in share * c["total"]]


HYPER = dict(lr=1e-3, betas=(0.9, 0.98), eps=1e-8)
MAX_NORM, STEPS_DONE, SEED = 1.0, 7, 1234


def _adamw_inputs(c, seed):
    g = _gen(seed)
    sizes = _shapes(c)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    s = dict(c, n=at, views=list(zip(sizes, starts)))
    live = torch.zeros(at, dtype=torch.bool, device="cuda")
    for n, a in zip(sizes, starts):
        live[a:a + n] = True
    # every second tensor (norms, biases) has no weight decay
    s["decays"] = [0.1 if i % 2 == 0 else 0.0 for i in range(len(sizes))]
    s["decay"] = torch.zeros(at // BLOCK, device="cuda")
    for n, a, d in zip(sizes, starts, s["decays"]):
        s["decay"][a // BLOCK:(a + n + BLOCK - 1) // BLOCK] = d
    w = (0.02 * _randn(g, at)).mul_(live)
    s["p"] = w.to(DT[c["dtype"]])
    s["master"] = w if c["master"] else None
    scale = torch.exp(0.5 * _randn(g, at // BLOCK)).repeat_interleave(BLOCK)
    s["g"] = (1e-3 * _randn(g, at)).mul_(scale).mul_(live).to(DT[c["grad"]])
    m = (2e-4 * _randn(g, at)).mul_(scale).mul_(live)
    v = (1e-3 * _randn(g, at)).mul_(scale).mul_(live).square_().mul_(0.5).add_(m * m)
    del scale, w
    if c["bits"] == 8:  # states as an earlier step left them, rounded to nearest
        for k, x in (("m", m), ("s", v.sqrt())):
            top = x.abs().view(-1, BLOCK).amax(1)
            s[k + "_scale"] = top / 448.0
            unit = torch.where(top > 0, 448.0 / top, torch.zeros_like(top))
            s[k] = (x.view(-1, BLOCK) * unit[:, None]).view(-1).to(torch.float8_e4m3fn)
    else:
        s["m"], s["v"] = m, v
    del m, v, live
    s["step"] = torch.full((1,), STEPS_DONE, dtype=torch.int64, device="cuda")
    return s


def _adamw_handle(s):
    """The optimizer that a program keeps, in the state of `s`."""
    import linear_cross_entropy_forward_gb300 as flce
    opt = flce.AdamW([s["p"][a:a + n] for n, a in s["views"]], weight_decay=s["decays"],
                     state_bits=s["bits"], master=s["master"] is not None,
                     max_norm=MAX_NORM if s["clip"] else None, seed=SEED, **HYPER)
    state = {"step": s["step"], "master": s["master"], "exp_avg": s["m"]}
    if s["bits"] == 8:
        state.update(exp_avg_scale=s["m_scale"], exp_rms=s["s"], exp_rms_scale=s["s_scale"])
    else:
        state.update(exp_avg_sq=s["v"])
    opt.load_state_dict(state)
    kept = {k: s[k] for k in ("bits", "clip", "op", "p")}
    return dict(kept, opt=opt, grads=[s["g"][a:a + n] for n, a in s["views"]])


def prepare(case, seed):
    c = dict(case)
    if c["op"] in ("linear", "linear_train"):
        return _prepare_linear(c, seed)
    if c["op"] in ("logits", "logprob"):
        return _prepare_logits(c, seed)
    s = _adamw_inputs(c, seed)
    return _adamw_handle(s) if own else s


# ---------------------------------------------------------------------------- plain forms
def _act(z, kind):
    """act(z) and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if kind == "silu":
        q = 1 / (1 + torch.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    if kind == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k, a = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k * (z + a * z * z * z))
    return (0.5 * z * (1 + t),
            0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * a * z * z))


def _plain_linear(s):
    x, w = s["x"].detach().float(), s["w"].detach().float()
    w = w.t() if s["layout"] == "vh" else w
    z = x @ w
    if s["b"] is not None:
        z = z + s["b"].detach().float()
    y, slope = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].detach().float()
    y = y.to(DT[s["out"]])
    if s["op"] == "linear":
        return y
    dz = s["gy"].float() * slope
    dx = dz @ w.t()
    dw = x.t() @ dz if s["layout"] == "hv" else dz.t() @ x
    out = {"y": y, "dx": dx.bfloat16(), "dw": dw.bfloat16()}
    if s["b"] is not None:
        out["db"] = dz.sum(0).to(s["b"].dtype)
    if s["r"] is not None:
        out["dr"] = s["gy"]
    return out


def _plain_process(s):
    """Processed logits in fp32 and the slope of each by its input."""
    x = s["logits"].detach().float()
    R, V = x.shape
    ids, at = s["tokens"], torch.arange(s["T"], device=x.device)
    there = at < s["lengths"][:, None]
    made = there & (at >= s["prompt_lens"][:, None])
    seen = torch.zeros(R, V, device=x.device).scatter_add_(1, ids, there.float()) > 0
    slope = torch.ones_like(x)
    if s["repetition_penalty"] is not None:
        rp = s["repetition_penalty"][:, None]
        slope = torch.where(seen, torch.where(x > 0, 1 / rp, rp), slope)
        x = x * slope
    if s["frequency_penalty"] is not None or s["presence_penalty"] is not None:
        n = torch.zeros(R, V, device=x.device).scatter_add_(1, ids, made.float())
        if s["frequency_penalty"] is not None:
            x = x - s["frequency_penalty"][:, None] * n
        if s["presence_penalty"] is not None:
            x = x - s["presence_penalty"][:, None] * (n > 0).float()
    if s["bias_ids"] is not None:
        used = s["bias_ids"] >= 0
        x = x.scatter_add(1, s["bias_ids"].clamp(min=0), s["bias_values"] * used)
    if s["allowed"] is not None:
        ok = s["allowed"]
        if s["allowed_kind"] == "bits":
            v = torch.arange(V, device=x.device)
            ok = (ok[:, v // 32] >> (v % 32)) & 1 > 0
        x = torch.where(ok, x, torch.full_like(x, -math.inf))
        slope = torch.where(ok, slope, torch.zeros_like(slope))
    if s["temperature"] is not None:
        x = x / s["temperature"][:, None]
        slope = slope / s["temperature"][:, None]
    return x, slope


def _plain_logits(s):
    x, slope = _plain_process(s)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    if s["op"] == "logits":
        return {"out": x.to(s["logits"].dtype), "lse": lse[:, 0]}
    p = e / total
    counts = s["labels"] != -100
    y = s["labels"].clamp(min=0)[:, None]
    logq = torch.where(p > 0, x - lse, torch.zeros_like(x))
    logp = torch.where(counts, x.gather(1, y)[:, 0] - lse[:, 0], torch.zeros_like(lse[:, 0]))
    ent = torch.where(counts, -(p * logq).sum(1), torch.zeros_like(lse[:, 0]))
    g = torch.where(counts, s["g_logp"], torch.zeros_like(logp))[:, None]
    h = torch.where(counts, s["g_ent"], torch.zeros_like(logp))[:, None]
    d = -p * (g + h * (logq + ent[:, None]))
    d = slope * d.scatter_add(1, y, g)
    return {"logp": logp, "entropy": ent, "dlogits": d.to(s["logits"].dtype)}


M32 = 0xFFFFFFFF


def _mix(x):
    """A 32-bit mixing of whole numbers (held in 64 bits): xor-shifts and odd multipliers."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _random_bits(n, t):
    """20 random bits for each of the two states of n elements, in step t (a tensor [1])."""
    key = _mix((SEED + 0x9E3779B9 * t) & M32)
    i = torch.arange(n, device="cuda")
    h = _mix((i & M32) ^ _mix((key + (i >> 32)) & M32))
    return h >> 12, ((h * 0x9E3779B1) & M32) >> 12


def _plain_round8(x, r, positive):
    """(e4m3 codes, scales): blocks in units of their largest / 448, each magnitude to one of its
    two neighbours, the upper one where the random bits carry; positive: 0 is for 0 alone."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    none = top < 2.0 ** -110
    unit = torch.where(none, torch.zeros_like(top), 448.0 / top)
    a = (x.abs() * unit).clamp(max=448.0)
    low = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)
    a2 = (((a + low).view(torch.int32) + r.view(-1, BLOCK).int()) & -0x100000).view(torch.float32)
    a2 = a2 - low
    if positive:
        a2 = torch.where((a > 0) & (a2 == 0), torch.full_like(a2, 2.0 ** -9), a2)
    code = torch.where(x < 0, -a2, a2).to(torch.float8_e4m3fn)
    return code.view(-1), torch.where(none, torch.zeros_like(top), top / 448.0)[:, 0]


def _plain_adamw(s):
    g = s["g"].float()
    out = {}
    if s["clip"]:
        norm = g.square().sum(dtype=torch.float64).sqrt().float().view(1)
        out["norm"] = norm
        g = g * torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
    (b1, b2), lr, eps = HYPER["betas"], HYPER["lr"], HYPER["eps"]
    s["step"] += 1
    t = s["step"].double()
    c1, c2 = (1 - b1 ** t).float(), (1 - b2 ** t).float()
    if s["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        root = (s["s"].float().view(-1, BLOCK) * s["s_scale"][:, None]).view(-1)
        v = root * root
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * (g * g)
    w = s["master"] if s["master"] is not None else s["p"].float()
    shrink = 1 - lr * s["decay"]
    w = (w.view(-1, BLOCK) * shrink[:, None]).view(-1) - lr * (m / c1) / (torch.sqrt(v / c2) + eps)
    s["p"].copy_(w)
    out["p"] = s["p"]
    if s["master"] is not None:
        s["master"].copy_(w)
        out["master"] = s["master"]
    if s["bits"] == 8:
        r1, r2 = _random_bits(s["n"], s["step"])
        s["m"], s["m_scale"] = _plain_round8(m, r1, False)
        s["s"], s["s_scale"] = _plain_round8(torch.sqrt(v), r2, True)
        out.update(m=s["m"], m_scale=s["m_scale"], s=s["s"], s_scale=s["s_scale"])
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
        out.update(m=s["m"], v=s["v"])
    out["step"] = s["step"]
    return out


# ---------------------------------------------------------------------------- the package's calls
def _own_linear(s):
    import linear_cross_entropy_forward_gb300 as flce
    args = dict(bias=s["b"], activation=None if s["act"] == "none" else s["act"],
                residual=s["r"], weight_layout=s["layout"], out_dtype=DT[s["out"]])
    if s["op"] == "linear":
        return flce.flce_linear(s["x"], s["w"], **args)
    y = flce.linear(s["x"], s["w"], **args)
    leaves = {k: s[k] for k in ("x", "w", "b", "r") if s[k] is not None}
    grads = torch.autograd.grad(y, list(leaves.values()), s["gy"])
    out = {"d" + k: d for k, d in zip(leaves, grads)}
    out["y"] = y
    return out


def _own_logits(s):
    import linear_cross_entropy_forward_gb300 as flce
    args = dict(tokens=s["tokens"], prompt_lens=s["prompt_lens"], lengths=s["lengths"],
                bias_ids=s["bias_ids"], bias_values=s["bias_values"], allowed=s["allowed"])
    for k in ("repetition_penalty", "frequency_penalty", "presence_penalty", "temperature"):
        if s[k] is not None:
            args[k] = s[k]
    if s["op"] == "logits":
        out, lse = flce.flce_process_logits(s["logits"], need_lse=True, **args)
        return {"out": out, "lse": lse}
    logp, ent = flce.logits_logprob(s["logits"], s["labels"], **args)
    (d,) = torch.autograd.grad([logp, ent], [s["logits"]], [s["g_logp"], s["g_ent"]])
    return {"logp": logp, "entropy": ent, "dlogits": d}


def _own_adamw(s):
    opt = s["opt"]
    norm = opt.step(s["grads"])
    now = opt.state_dict()
    out = {"p": s["p"], "step": now["step"], "m": now["exp_avg"]}
    if s["clip"]:
        out["norm"] = norm
    if now["master"] is not None:
        out["master"] = now["master"]
    if s["bits"] == 8:
        out.update(m_scale=now["exp_avg_scale"], s=now["exp_rms"], s_scale=now["exp_rms_scale"])
    else:
        out["v"] = now["exp_avg_sq"]
    return out


def run(state):
    op = state["op"]
    if op in ("linear", "linear_train"):
        return _own_linear(state) if own else _plain_linear(state)
    if op in ("logits", "logprob"):
        return _own_logits(state) if own else _plain_logits(state)
    return _own_adamw(state) if own else _plain_adamw(state)


# ---------------------------------------------------------------------------- what cannot be avoided
def work(case):
    c = case
    if c["op"] in ("linear", "linear_train"):
        M, K, N, o = c["M"], c["K"], c["N"], SIZE[c["out"]]
        b = 2 * N if c["bias"] else 0
        data = 2 * (M * K + K * N) + b + M * N * o * (2 if c["res"] else 1)
        if c["op"] == "linear":
            return {"bytes": data, "flops": 2.0 * M * K * N}
        return {"bytes": data + M * N * o + 2 * (M * K + K * N) + b, "flops": 6.0 * M * K * N}
    if c["op"] in ("logits", "logprob"):
        R, V = c["R"], c["V"]
        mask = {"none": 0, "bits": R * V / 8, "bytes": R * V}[c["allowed"]]
        used = c["rep"] or c["freq"] or c["pres"]
        more = mask + R * c["bias"] * 12 + (4 * R * c["T"] if used else 0) + 40 * R
        return {"bytes": 2 * R * V * SIZE[c["dtype"]] + more, "flops": 10.0 * R * V}
    n = sum(_shapes(c))
    p, g = SIZE[c["dtype"]], SIZE[c["grad"]]
    state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    weight = p + 8 if c["master"] else 2 * p
    return {"bytes": n * (weight + g + state), "flops": 15.0 * n}


# ---------------------------------------------------------------------------- 64-bit values
def _exact_linear(s):
    w = s["w"].detach().double()
    if s["layout"] == "vh":
        w = w.T
    z = s["x"].detach().double().matmul(w)
    if s["b"] is not None:
        z += s["b"].detach().double()
    kind = s["act"]
    F = torch.nn.functional
    if s["op"] == "linear_train":
        z.requires_grad_(True)
    if kind == "relu":
        y = F.relu(z)
    elif kind == "silu":
        y = F.silu(z)
    elif kind in ("gelu", "gelu_tanh"):
        y = F.gelu(z, approximate="tanh" if kind == "gelu_tanh" else "none")
    else:
        y = z * 1.0
    dz = None
    if s["op"] == "linear_train":
        (dz,) = torch.autograd.grad(y, z, s["gy"].double())
    y = y.detach()
    if s["r"] is not None:
        y = y + s["r"].detach().double()
    if dz is None:
        return y
    out = {"y": y, "dx": dz.matmul(w.T)}
    x = s["x"].detach().double()
    out["dw"] = dz.T.matmul(x) if s["layout"] == "vh" else x.T.matmul(dz)
    if s["b"] is not None:
        out["db"] = dz.sum(0)
    if s["r"] is not None:
        out["dr"] = None
    return out


def _exact_logits(s):
    """Row by row: autograd in 64 bits over the definition."""
    outs = {"out": [], "lse": [], "logp": [], "entropy": [], "dlogits": []}
    R, V = s["logits"].shape
    for r in range(R):
        x = s["logits"][r].detach().double().requires_grad_(True)
        length, prompt = int(s["lengths"][r]), int(s["prompt_lens"][r])
        ids = s["tokens"][r]
        every = torch.bincount(ids[:length], minlength=V)
        made = torch.bincount(ids[prompt:length], minlength=V).double()
        z = x
        if s["repetition_penalty"] is not None:
            rp = s["repetition_penalty"][r].double()
            z = torch.where(every > 0, torch.where(z > 0, z / rp, z * rp), z)
        if s["frequency_penalty"] is not None:
            z = z - made * s["frequency_penalty"][r].double()
        if s["presence_penalty"] is not None:
            z = z - (made > 0).double() * s["presence_penalty"][r].double()
        if s["bias_ids"] is not None:
            ok = s["bias_ids"][r] >= 0
            z = z.index_add(0, s["bias_ids"][r][ok], s["bias_values"][r][ok].double())
        if s["allowed"] is not None:
            a = s["allowed"][r]
            if s["allowed_kind"] == "bits":
                a = ((a[:, None] >> torch.arange(32, device=a.device)) & 1).flatten()[:V] == 1
            z = z.masked_fill(~a, -math.inf)
        if s["temperature"] is not None:
            z = z / s["temperature"][r].double()
        lse = torch.logsumexp(z, 0)
        if s["op"] == "logits":
            outs["out"].append(z.detach())
            outs["lse"].append(lse.detach())
            continue
        y = int(s["labels"][r])
        if y == -100:
            outs["logp"].append(torch.zeros_like(lse.detach()))
            outs["entropy"].append(torch.zeros_like(lse.detach()))
            outs["dlogits"].append(torch.zeros_like(x.detach()))
            continue
        keep = torch.isfinite(z)
        logq = z[keep] - lse
        ent = -(logq.exp() * logq).sum()
        logp = z[y] - lse
        up = logp * s["g_logp"][r].double() + ent * s["g_ent"][r].double()
        (d,) = torch.autograd.grad(up, x)
        outs["logp"].append(logp.detach())
        outs["entropy"].append(ent.detach())
        outs["dlogits"].append(d)
    return {k: torch.stack(v) for k, v in outs.items() if v}


def _exact_round8(x, r, positive):
    x = x.reshape(-1, BLOCK)
    top = x.abs().max(1, keepdim=True).values
    scale = torch.where(top < 2.0 ** -110, torch.zeros_like(top), top / 448)
    a = torch.where(scale > 0, x.abs() / scale, torch.zeros_like(x)).clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    q = torch.floor(a / step + r.reshape(-1, BLOCK).double() / 2 ** 20) * step
    if positive:
        q = torch.where((a > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return (q * torch.sign(x)).reshape(-1), scale[:, 0]


def _exact_adamw(s):
    out = {}
    g = s["g"].double()
    if s["clip"]:
        norm = g.norm().reshape(1)
        out["norm"] = norm
        g *= (MAX_NORM / (norm + 1e-6)).clamp(max=1)
    beta1, beta2 = HYPER["betas"]
    t = STEPS_DONE + 1
    if s["bits"] == 8:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (s["s"].double() * s["s_scale"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = torch.lerp(g, m, beta1)
    v = torch.lerp(g * g, v, beta2)
    del g
    start = s["master"] if s["master"] is not None else s["p"]
    w = start.double() * (1 - HYPER["lr"] * s["decay"].double()).repeat_interleave(BLOCK)
    w -= HYPER["lr"] / (1 - beta1 ** t) * m / ((v / (1 - beta2 ** t)).sqrt() + HYPER["eps"])
    out["p"] = w
    if s["master"] is not None:
        out["master"] = w
    if s["bits"] == 8:
        r1, r2 = _random_bits(s["n"], torch.full((1,), t, dtype=torch.int64, device="cuda"))
        out["m"], out["m_scale"] = _exact_round8(m, r1, False)
        out["s"], out["s_scale"] = _exact_round8(v.sqrt(), r2, True)
    else:
        out["m"], out["v"] = m, v
    out["step"] = None
    return out


def exact(case, seed):
    c = dict(case)
    if c["op"] in ("linear", "linear_train"):
        return _exact_linear(_prepare_linear(c, seed))
    if c["op"] in ("logits", "logprob"):
        return _exact_logits(_prepare_logits(c, seed))
    return _exact_adamw(_adamw_inputs(c, seed))
