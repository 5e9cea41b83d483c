"""A draft model learns from the target it is verified against: the operators
that score rows of logits, with the verify step before and after.

The target goes over the text once and the top logits of its rows are recorded
(`logprobs`, a few numbers a row instead of the vocabulary).  Then the draft is
trained on the record: `distill` gives the loss of its logits and their gradient,
autograd takes that on to its weights.  How many drafted tokens the target accepts
is what the verify step says.

    python examples/distill_draft.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_42_gb300 as sv  # noqa: E402

TEMPERATURE, TOP = 0.8, 64


class Bigrams:
    """Logits of the next token from the last one: an embedding and a head."""

    def __init__(self, vocab=2000, hidden=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab = vocab
        self.embed = torch.randn(vocab, hidden, generator=g, device="cuda")
        self.head = torch.randn(hidden, vocab, generator=g, device="cuda") * (3 * hidden ** -0.5)

    def __call__(self, tokens):
        return self.embed[tokens.long().clamp_min(0)] @ self.head


def text(target, batch=16, length=48):
    """Sequences [batch, length] of the target's tokens, ragged: -1 behind the last."""
    g = torch.Generator(device="cuda").manual_seed(7)
    out = [torch.randint(0, target.vocab, (batch,), generator=g, device="cuda")]
    for _ in range(length - 1):
        p = (target(out[-1]) / TEMPERATURE).softmax(-1)
        out.append(p.multinomial(1, generator=g)[:, 0])
    lens = torch.randint(length // 2, length + 1, (batch,), generator=g, device="cuda")
    return torch.stack(out, 1).masked_fill(torch.arange(length, device="cuda") >= lens[:, None], -1).int()


def record(target, tokens):
    """What the draft is to learn, per position: the target's likeliest tokens and their log
    probabilities (no entry where there is no token)."""
    top = sv.logprobs(target(tokens), temperature=TEMPERATURE, top_n=TOP)
    return top["top_ids"].masked_fill((tokens < 0)[..., None], -1), top["top_logprobs"]


def loss_and_gradients(draft, tokens, ids, logprobs):
    """Mean loss over the tokens; gradients are left with the draft's weights."""
    live = (tokens >= 0).float()
    logits = draft(tokens)
    got = sv.distill(logits.detach(), ids, logprobs, temperature=TEMPERATURE, teacher_temperature=1.0, tail=True,
                     grad_loss=live / live.sum())
    logits.backward(got["grad"])
    return got["loss"].sum() / live.sum(), got["accept"].sum() / live.sum()


def accepted(target, draft, tokens, k=4):
    """Mean number of k drafted tokens that the target accepts behind the given ones, [N]."""
    ver = sv.Verifier(vocab=target.vocab, max_batch=len(tokens), max_k=k, dtype="f32")
    last, q, x = tokens, [], []
    for j in range(k):
        q.append(draft(last)[:, None].detach())
        x.append(ver.draft_sample(q[-1], temperature=TEMPERATURE, seed=5 + j)[:, :1])
        last = x[-1][:, 0]
    x = torch.cat(x, 1).contiguous()
    rows = target(torch.cat([tokens[:, None], x], 1))
    out = ver.run(rows, torch.cat(q, 1), x, temperature=TEMPERATURE, seed=11, logprobs=1)
    ver.close()
    return float(out["num_accepted"].float().mean())


def train(steps=60, say=print):
    target, draft = Bigrams(seed=0), Bigrams(hidden=32, seed=1)
    weights = [draft.embed.requires_grad_(), draft.head.requires_grad_()]
    opt = torch.optim.Adam(weights, lr=0.05)
    tokens = text(target)
    ids, logprobs = record(target, tokens)
    start = tokens[:, 0].contiguous()
    say(f"accepted of 4 drafted tokens: {accepted(target, draft, start):.2f}")
    losses = []
    for i in range(steps):
        opt.zero_grad()
        loss, share = loss_and_gradients(draft, tokens, ids, logprobs)
        opt.step()
        losses.append(float(loss))
        if i % 20 == 0 or i == steps - 1:
            say(f"step {i}: loss {losses[-1]:.3f}, accept {float(share):.3f}")
    say(f"accepted of 4 drafted tokens: {accepted(target, draft, start):.2f}")
    return losses


if __name__ == "__main__":
    train()
