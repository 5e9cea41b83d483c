"""The example that trains a draft on the target's recorded top logits
(examples/distill_draft.py): it runs, and the gradients that reach the draft's
weights are those of the loss's formula in 64 bits."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_distillation_runs_with_the_formulas_gradients():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_42_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import distill_draft as ex
    said = []
    losses = ex.train(steps=3, say=said.append)
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses) and len(said) == 4

    target, draft = ex.Bigrams(vocab=501, seed=0), ex.Bigrams(vocab=501, hidden=32, seed=1)
    draft.embed.requires_grad_(), draft.head.requires_grad_()
    tokens = ex.text(target, batch=5, length=9)
    ids, logprobs = ex.record(target, tokens)
    loss, share = ex.loss_and_gradients(draft, tokens, ids, logprobs)
    # the logits as the operator had them, so that the matrix product's roundings are no part of the comparison
    rows = draft(tokens).detach().double().requires_grad_()
    live = tokens >= 0
    ln_p = (rows / ex.TEMPERATURE).log_softmax(-1)[live]
    at, ln_q = ids[live].long(), logprobs[live].double()
    q = ln_q.exp()
    q_rest = 1 - q.sum(-1)
    inside = torch.zeros_like(ln_p, dtype=torch.bool).scatter_(-1, at, True)
    rest = ln_p.masked_fill(inside, -math.inf).logsumexp(-1)
    want = ((q * (ln_q - ln_p.gather(-1, at))).sum(-1) + q_rest * (q_rest.log() - rest)).mean()
    want.backward()
    # fp32 sums of some tens of terms near 1 that are rounded a few times each, and logits up to 10 over 0.8 in the
    # exponents: 40 roundings of 2^-24 of what the loss is a difference of (ln q and ln p, below 32 here)
    assert abs(float(loss) - float(want)) < 40 * 2 ** -24 * 32
    assert 0 < float(share) <= 1
    with torch.no_grad():
        g = rows.grad
        grads = {"head": draft.embed[tokens.long().clamp_min(0)].double().flatten(0, 1).t() @ g.flatten(0, 1),
                 "embed": torch.zeros_like(draft.embed, dtype=torch.float64).index_add_(
                     0, tokens.long().clamp_min(0).flatten(), (g @ draft.head.double().t()).flatten(0, 1))}
    for name, mine in (("head", draft.head.grad), ("embed", draft.embed.grad)):
        # products in torch's fp32 (or TF32, 2^-11 an operand, should it be on): sums of up to 501 terms
        far = float((mine.double() - grads[name]).norm() / grads[name].norm())
        assert far < 2 ** -9, (name, far)
