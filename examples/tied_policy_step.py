"""A fine-tuning step of a tied-table model, with every operator around the LM head.

The model is as small as one can be: a token's hidden state is its embedding (scaled by
sqrt(H)) plus the previous token's, and the logits are hidden @ table^T with the same
table [V, H].  A policy step forms, in three calls,

    the lookup                     flce_embedding
    loss, dhidden, dtable (head)   flce_policy_forward_backward
    dtable += lookup's gradient    flce_embedding_backward(accumulate=True)

and a preference step scores pairs of sequences under the policy and a frozen reference,
and sends the loss's gradient through the head and the table:

    python examples/tied_policy_step.py [--steps 20]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))

import linear_cross_entropy_forward_gb300 as flce  # noqa: E402

V, H, B, S = 2000, 128, 8, 96


def hidden_states(table, ids):
    """[B * S, H] hidden states of [B, S] tokens, and what their gradient is made of."""
    x = flce.flce_embedding(ids, table, scale=math.sqrt(H))
    h = x.clone()
    h[:, 1:] += x[:, :-1]
    return h.view(-1, H)


def add_lookup_gradient(dtable, dhidden, ids):
    """The lookup's gradient, added to the head's in place (one table, one gradient)."""
    d = dhidden.view(*ids.shape, H).clone()
    d[:, :-1] += dhidden.view(*ids.shape, H)[:, 1:]
    return flce.flce_embedding_backward(d, ids, V, scale=math.sqrt(H), dweight=dtable,
                                        accumulate=True)


def next_labels(ids, prompt):
    """Each position's label is the next token; the prompt and the last position do not count."""
    labels = torch.full_like(ids, flce.IGNORE_INDEX)
    labels[:, prompt - 1:-1] = ids[:, prompt:]
    return labels


def sequence_ends(device):
    return torch.arange(0, (B + 1) * S, S, dtype=torch.int32, device=device)


def policy_step(table, ids, prompt, advantages, old_logp, ref_logp, lr):
    """One update of `table`; returns the loss, the statistics and the counts."""
    labels = next_labels(ids, prompt).view(-1)
    hidden = hidden_states(table, ids)
    loss, stats, counts, _, _, dhidden, dtable = flce.flce_policy_forward_backward(
        hidden, table, labels, old_logp, advantages, ref_logp=ref_logp,
        cu_seqlens=sequence_ends(ids.device), clip_low=0.2, clip_high=0.28, kl_coef=0.01,
        entropy_coef=0.001, aggregate="seq_mean_token_mean", weight_layout="vh")
    add_lookup_gradient(dtable, dhidden, ids)
    table.sub_(dtable, alpha=lr)
    return loss, stats, counts


def log_probs(table, ids, prompt):
    """[B * S] log-probabilities of the labels (0 where none counts), without gradients."""
    nll, _, _, _ = flce.flce_forward(hidden_states(table, ids), table,
                                     next_labels(ids, prompt).view(-1), "none", weight_layout="vh")
    return -nll


def preference_step(table, reference, ids, prompt, lr):
    """One update on B / 2 pairs (the first half of the rows chosen, the second rejected)."""
    labels = next_labels(ids, prompt).view(-1)
    ref = log_probs(reference, ids, prompt).view(B, S)
    hidden = hidden_states(table, ids)
    nll, _, lse, ez = flce.flce_forward(hidden, table, labels, "none", weight_layout="vh")
    loss, rewards, dlogp = flce.flce_preference_loss(
        -nll.view(B, S), ref, mask=labels.view(B, S), beta=0.5)
    dhidden, dtable = flce.flce_backward(hidden, table, labels, lse, ez, -dlogp.view(-1), None,
                                         "none", weight_layout="vh")
    add_lookup_gradient(dtable, dhidden, ids)
    table.sub_(dtable, alpha=lr)
    return loss, rewards


def main(steps=20, seed=0, quiet=False):
    """Runs both kinds of step; returns the losses of each."""
    g = torch.Generator().manual_seed(seed)
    table = (torch.randn(V, H, generator=g) / H).to(torch.bfloat16).cuda()
    reference = table.clone()
    ids = torch.randint(0, V, (B, S), generator=g).cuda()
    prompt = 16
    old = ref = log_probs(reference, ids, prompt)
    advantages = torch.randn(B, generator=g).cuda()
    policy, preference = [], []
    for _ in range(steps):
        loss, stats, counts = policy_step(table, ids, prompt, advantages, old, ref, lr=0.2)
        policy.append(float(loss))
    if not quiet:
        print("policy     %.4f -> %.4f   KL %.4f   clipped %d of %d tokens"
              % (policy[0], policy[-1], float(stats[1]), int(counts[2]), int(counts[0])))
    table.copy_(reference)
    for _ in range(steps):
        loss, rewards = preference_step(table, reference, ids, prompt, lr=0.02)
        preference.append(float(loss))
    if not quiet:
        print("preference %.4f -> %.4f   rewards %.3f (chosen) %.3f (rejected)"
              % (preference[0], preference[-1], float(rewards[:B // 2].mean()),
                 float(rewards[B // 2:].mean())))
    return policy, preference


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    main(ap.parse_args().steps)
