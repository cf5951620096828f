"""A rollout and an update of a small policy, with every operator around the LM head.

The model: a token's state is its embedding plus the one before it, a dense layer with SiLU is
added to it (its residual), and the logits are that times the same table (tied).  A rollout samples
from the processed logits:

    logits = linear(hidden, table)               fp32, no bias
    z, lse = flce_process_logits(...)            penalties, a mask of allowed tokens, temperature
    token ~ softmax(z),  old_logp = z[token] - lse

and an update scores the sampled tokens under the same distribution, takes the clipped policy loss
and steps all tensors at once:

    logp, entropy = logits_logprob(...)          the same penalties, row by row
    loss = policy_loss(logp, old_logp, ...)
    AdamW.step                                   clipped by the gradients' norm, moments in 8 bits

    python examples/rollout_and_update.py [--rounds 3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))

import linear_cross_entropy_forward_gb300 as flce  # noqa: E402

V, H, B, PROMPT, NEW = 1000, 128, 16, 8, 24
PENALTIES = dict(repetition_penalty=1.2, frequency_penalty=0.1, presence_penalty=0.1, temperature=0.8)


def hidden_states(ids, table, weight, bias):
    """[B * S, H] of [B, S] tokens."""
    x = flce.embedding(ids.contiguous(), table)
    x = torch.cat([x[:, :1], x[:, 1:] + x[:, :-1]], 1).reshape(-1, H)
    return flce.linear(x, weight, bias, "silu", x, weight_layout="vh")


def allowed_tokens(device):
    """Bits of the tokens that may be sampled: all but every seventh."""
    ok = torch.arange((V + 31) // 32 * 32, device=device) % 7 != 6
    word = (ok.view(-1, 32).long() << torch.arange(32, device=device)).sum(1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).int()[None]


@torch.no_grad()
def rollout(ids, table, weight, bias, allowed, gen):
    """NEW tokens behind each prompt; returns all tokens and the sampled ones' log-probabilities."""
    tokens = torch.full((B, PROMPT + NEW), -1, dtype=torch.int64, device=ids.device)
    tokens[:, :PROMPT] = ids
    old = []
    prompts = torch.full((B,), PROMPT, device=ids.device)
    for n in range(PROMPT, PROMPT + NEW):
        h = hidden_states(tokens[:, n - 2:n], table, weight, bias).view(B, 2, H)[:, 1].contiguous()
        logits = flce.flce_linear(h, table, weight_layout="vh", out_dtype=torch.float32)
        z, lse = flce.flce_process_logits(
            logits, tokens=tokens, prompt_lens=prompts, lengths=torch.full_like(prompts, n),
            allowed=allowed.expand(B, -1), need_lse=True, **PENALTIES)
        tokens[:, n] = torch.multinomial(torch.exp(z - lse[:, None]), 1, generator=gen)[:, 0]
        old.append(z.gather(1, tokens[:, n:n + 1])[:, 0] - lse)
    return tokens, torch.stack(old, 1)


def score(tokens, table, weight, bias, allowed):
    """[B, NEW] log-probabilities and entropies of the sampled tokens, each under the penalties of
    the tokens before it."""
    # the state of every position but the last, as the rollout saw it: a token and the one before
    pairs = torch.stack([tokens[:, PROMPT - 2:-2], tokens[:, PROMPT - 1:-1]], 2).view(-1, 2)
    h = hidden_states(pairs, table, weight, bias).view(-1, 2, H)[:, 1].contiguous()
    logits = flce.linear(h, table, weight_layout="vh", out_dtype=torch.float32)
    rows = tokens.repeat_interleave(NEW, 0)
    lengths = torch.arange(PROMPT, PROMPT + NEW, device=tokens.device).repeat(B)
    logp, entropy = flce.logits_logprob(
        logits, tokens[:, PROMPT:].reshape(-1), tokens=rows, lengths=lengths,
        prompt_lens=torch.full_like(lengths, PROMPT), allowed=allowed.expand(B * NEW, -1), **PENALTIES)
    return logp.view(B, NEW), entropy.view(B, NEW)


def main(rounds=3, seed=0, quiet=False):
    """Rollouts and updates; returns per round the loss, the gradients' norm and how far the scored
    log-probabilities of the unchanged policy are from the rollout's."""
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table = (torch.randn(V, H, generator=g) * 0.3).bfloat16().cuda().requires_grad_(True)
    weight = (torch.randn(H, H, generator=g) / H ** 0.5).bfloat16().cuda().requires_grad_(True)
    bias = torch.zeros(H).bfloat16().cuda().requires_grad_(True)
    allowed = allowed_tokens("cuda")
    opt = flce.AdamW([table, weight, bias], lr=2e-3, betas=(0.9, 0.98), weight_decay=[0.0, 0.1, 0.0],
                     state_bits=8, master=True, max_norm=1.0, seed=seed)
    out = []
    for _ in range(rounds):
        prompts = torch.randint(0, V, (B, PROMPT), generator=g).cuda()
        tokens, old = rollout(prompts, table, weight, bias, allowed, gen)
        rewards = (tokens[:, PROMPT:] % 2 == 0).float().mean(1)
        advantages = (rewards - rewards.mean()) / (rewards.std() + 1e-6)
        for epoch in range(2):
            logp, entropy = score(tokens, table, weight, bias, allowed)
            if epoch == 0:
                apart = float((logp.detach() - old).abs().max())
            loss, _, _ = flce.policy_loss(logp, old, advantages, entropy=entropy, entropy_coef=0.01)
            loss.sum().backward()
            norm = opt.step()
            for p in opt.params:
                p.grad = None
        out.append((float(loss), float(norm), apart))
        if not quiet:
            print("loss %.4f   norm %.4f   rollout and score apart by %.2g" % out[-1])
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=3)
    main(ap.parse_args().rounds)
