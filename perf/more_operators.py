"""The operators that score rows of logits, as cases to be measured.

Beside a verify step: the log probabilities of given tokens with their ranks,
the entropy and the top alternatives of each row (logprobs), their gradient
(logprobs_grad), and the draft model's training loss, the divergence from a
teacher of which the top logits are recorded (distill), with its gradient
(distill_grad).

With ``own`` false a case runs in plain torch operations, in 32 bits; with
``own`` true through the package's ``logprobs`` and ``distill``.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------- #
# the cases                                                                    #
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one user of a small model: 5 verified positions, the 5 likeliest tokens of each
        dict(name="logprobs_b1_t5_v1000_f32", op="logprobs", b=1, t=5, v=1000, dtype="f32", top=5, temp=1.0,
             tokens=True, ragged=False),
        # one user's verify step: 9 positions, all emitted
        dict(name="logprobs_b1_t9_v128256", op="logprobs", b=1, t=9, v=128256, dtype="bf16", top=20, temp=1.0,
             tokens=True, ragged=False),
        # a verify batch: 64 requests, only the emitted positions are scored
        dict(name="logprobs_b64_t9_v128256", op="logprobs", b=64, t=9, v=128256, dtype="bf16", top=20, temp=0.7,
             tokens=True, ragged=True),
        # prompts scored for their likelihood; one token was added to the vocabulary, so rows start on odd elements
        dict(name="logprobs_b4_t600_v32001_f16", op="logprobs", b=4, t=600, v=32001, dtype="f16", top=0, temp=1.0,
             tokens=True, ragged=True),
        # a teacher's top logits are recorded for a draft to learn from
        dict(name="logprobs_b1000_t2_v152064_top64", op="logprobs", b=1000, t=2, v=152064, dtype="bf16", top=64,
             temp=1.0, tokens=False, ragged=False),
        # a small policy step in 32 bits, next-token positions of each sequence
        dict(name="logprobs_grad_b6_t50_v32000_f32", op="logprobs_grad", b=6, t=50, v=32000, dtype="f32", temp=1.0,
             ragged=True),
        # a policy step with an entropy bonus
        dict(name="logprobs_grad_b4_t500_v128256", op="logprobs_grad", b=4, t=500, v=128256, dtype="bf16", temp=1.0,
             ragged=True),
        # a draft's loss on a few held-out positions
        dict(name="distill_b4_t12_v32000", op="distill", b=4, t=12, v=32000, dtype="bf16", k=20, temp=1.0, tail=False,
             teacher="logits", ragged=False),
        # a draft's loss over a held-out batch, what the top 64 leave out as one more outcome
        dict(name="distill_b256_t8_v152064", op="distill", b=256, t=8, v=152064, dtype="bf16", k=64, temp=1.0,
             tail=True, teacher="logprobs", ragged=True),
        # a draft that learns while it serves: the positions of one verify batch, the target's top-k as it sampled
        dict(name="distill_grad_b64_t8_v128256", op="distill_grad", b=64, t=8, v=128256, dtype="bf16", k=50, temp=0.7,
             tail=False, teacher="logits", ragged=True),
        # a training batch in half precision, a vocabulary of odd size
        dict(name="distill_grad_b3_t500_v100003_f16", op="distill_grad", b=3, t=500, v=100003, dtype="f16", k=32,
             temp=2.0, tail=True, teacher="logprobs", ragged=True),
        # a training batch with logits in 32 bits
        dict(name="distill_grad_b7_t111_v128256_f32", op="distill_grad", b=7, t=111, v=128256, dtype="f32", k=128,
             temp=1.0, tail=True, teacher="logits", ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "distill", "distill_grad", "distill_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    v = rng.choice([32000, 32001, 100003, 128256, 152064, _log(rng, 1000, 200000), _log(rng, 1000, 200000)])
    # no more elements than the largest listed cases
    most = (80e6 if op.endswith("grad") else 100e6) if dtype == "f32" else (140e6 if op.endswith("grad") else 280e6)
    rows = max(1, min(_log(rng, 1, 4000), int(most / v)))
    b = _log(rng, 1, rows)
    t = max(1, rows // b)
    case = dict(op=op, b=b, t=t, v=v, dtype=dtype, temp=rng.choice([1.0, 1.0, 0.7, 2.0]), ragged=rng.random() < 0.6)
    if op == "logprobs":
        return dict(case, top=rng.choice([0, 1, 5, 20, 64, 128]), tokens=rng.random() < 0.7)
    if op == "logprobs_grad":
        return case
    return dict(case, k=_log(rng, 4, 128), tail=rng.random() < 0.5, teacher=rng.choice(["logits", "logprobs"]))


# --------------------------------------------------------------------------- #
# sizes a case fixes without its seed                                          #
# --------------------------------------------------------------------------- #
def _lens(case):
    """Positions of each sequence that count: all, or (ragged) from t down to about half of it."""
    t = case["t"]
    return t - (np.arange(case["b"]) % max(1, (t + 1) // 2) if case["ragged"] else np.zeros(case["b"], np.int64))


def work(case):
    rows, all_rows, v = int(_lens(case).sum()), case["b"] * case["t"], case["v"]
    s = 4 if case["dtype"] == "f32" else 2
    grad = case["op"].endswith("grad")
    if case["op"].startswith("logprobs"):
        # row_status, entropy, lse; token, log probability (and, in the forward, its rank); two upstream gradients
        small = all_rows * (12 + 8 * case.get("top", 0) + (16 if grad else 12 if case["tokens"] else 0))
        rows = rows if grad or case["tokens"] else all_rows
    else:
        width = 4 if case["teacher"] == "logprobs" or case["dtype"] == "f32" else 2
        # ids and values; loss, accept, row_status; the teacher's lse, the upstream gradient
        small = all_rows * (case["k"] * (4 + width) + 12 + (4 if case["tail"] and case["teacher"] == "logits" else 0)
                            + (4 if grad else 0))
    return dict(bytes=float(rows * v * s + (all_rows * v * s if grad else 0) + small),
                flops=float(rows * v * (12 if grad else 8)))


# --------------------------------------------------------------------------- #
# inputs                                                                       #
# --------------------------------------------------------------------------- #
def prepare(case, seed):
    dev = torch.device("cuda")
    rng = np.random.default_rng([seed, 78])
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    b, t, v, dt = case["b"], case["t"], case["v"], _DT[case["dtype"]]
    lens = torch.from_numpy(_lens(case)[rng.permutation(b)]).to(dev)
    live = torch.arange(t, device=dev)[None, :] < lens[:, None]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    # logits as the verify workloads have them: spread 3, some 20 likely tokens 8 above; the last tokens of a
    # vocabulary are padding of its matrix and masked
    x = randn(b, t, v).mul_(3.0)
    hot = torch.randint(0, v, (b, t, 20), generator=gen, device=dev)
    x.scatter_add_(2, hot, torch.full(hot.shape, 8.0, device=dev))
    x[..., v - v // 500:] = -math.inf
    st = dict(case=case)
    if case["op"].startswith("logprobs"):
        # tokens as they were sampled, by the largest of logits with Gumbel noise
        noise = torch.rand(b, t, v, generator=gen, device=dev).clamp_(1e-10, 1.0 - 1e-7).log_().neg_().log_().neg_()
        tok = (x / case["temp"] + noise).argmax(-1)
        st["tokens"] = torch.where(live, tok, -1).int() if case.get("tokens", True) else None
        st["logits"] = x.to(dt)
        if case["op"] == "logprobs_grad":
            # advantages, and the weight of the entropy bonus
            st["gl"] = torch.where(live, randn(b, t), 0.0)
            st["gh"] = torch.where(live, torch.full((b, t), 0.05, device=dev), 0.0)
        return st
    # the student's logits are the teacher's with noise, as a draft's are the target's
    k, temp = min(case["k"], v - v // 500), case["temp"]
    values, ids = x.topk(k, -1)
    st["ids"] = torch.where(live[..., None], ids, -1).int()
    st["lse"] = None
    if case["teacher"] == "logits":
        st["teacher"], st["teacher_temp"] = values.to(dt), temp
        if case["tail"]:
            st["lse"] = (x / temp).logsumexp(-1)
    else:
        st["teacher"] = values / temp - (x / temp).logsumexp(-1, keepdim=True)
        st["teacher_temp"] = 1.0
    st["student"] = x.add_(randn(b, t, v)).to(dt)
    st["gl"] = torch.rand(b, t, generator=gen, device=dev) + 0.5 if case["op"] == "distill_grad" else None
    return st


# --------------------------------------------------------------------------- #
# one pass                                                                     #
# --------------------------------------------------------------------------- #
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_logprobs(st):
    import speculative_decoding_verification_42_gb300 as sv
    c = st["case"]
    return sv.logprobs(st["logits"], st["tokens"], temperature=c["temp"], top_n=c["top"], rank=c["tokens"])


def _own_logprobs_grad(st):
    import speculative_decoding_verification_42_gb300 as sv
    return sv.logprobs(st["logits"], st["tokens"], temperature=st["case"]["temp"], grad_logprob=st["gl"],
                       grad_entropy=st["gh"])


def _own_distill(st):
    import speculative_decoding_verification_42_gb300 as sv
    c = st["case"]
    return sv.distill(st["student"], st["ids"], st["teacher"], temperature=c["temp"],
                      teacher_temperature=st["teacher_temp"], tail=c["tail"], teacher_lse=st["lse"],
                      grad_loss=st["gl"])


_own = dict(logprobs=_own_logprobs, logprobs_grad=_own_logprobs_grad, distill=_own_distill, distill_grad=_own_distill)


def _softmax(x, temp):
    """Of rows [.., v] in 32 bits: their largest element, the distances d from it over temp, and e^d."""
    x = x.float()
    top = x.amax(-1, keepdim=True)
    d = (x - top) / temp
    return top, d, torch.exp(d)


def _plain_logprobs(st, grad=False):
    c, tok = st["case"], st["tokens"]
    x = st["logits"]
    m, d, e = _softmax(x, c["temp"])
    z = e.sum(-1, keepdim=True)
    lp, p, lse = d - torch.log(z), e / z, (m / c["temp"] + torch.log(z)).squeeze(-1)
    live = tok >= 0 if tok is not None else torch.ones_like(lse, dtype=torch.bool)
    plp = torch.where(p > 0, p * lp, 0.0)
    ent = -plp.sum(-1)
    out = dict(entropy=torch.where(live, ent, 0.0), lse=torch.where(live, lse, 0.0),
               row_status=torch.zeros(lse.shape, dtype=torch.int32, device=x.device))
    ids = torch.arange(c["v"], device=x.device)
    if tok is not None:
        at = tok.clamp(min=0).long()[..., None]
        out["logprob"] = torch.where(live, lp.gather(-1, at).squeeze(-1), 0.0)
    if grad:
        g = (ids == at).float().sub_(p).mul_(st["gl"][..., None])
        g -= (plp + p * ent[..., None]) * st["gh"][..., None]
        out["grad"] = torch.where(live[..., None], g / c["temp"], 0.0).to(x.dtype)
        return out
    if tok is not None:
        xt = x.gather(-1, at)
        ahead = ((x > xt) | ((x == xt) & (ids < at))).sum(-1)
        out["rank"] = torch.where(live, ahead, -1).int()
    if c["top"]:
        # ordered by logit, the lowest id first among equals: one 64-bit number for both
        i = x.float().view(torch.int32).long()
        key = torch.where(i < 0, -(i & 0x7fffffff), i) * (1 << 20) + ((1 << 20) - 1 - ids)
        best = (1 << 20) - 1 - (key.topk(c["top"], -1).values & ((1 << 20) - 1))
        out["top_ids"] = torch.where(live[..., None], best, -1).int()
        out["top_logprobs"] = torch.where(live[..., None], lp.gather(-1, best), -math.inf)
    return out


def _plain_logprobs_grad(st):
    return _plain_logprobs(st, grad=True)


def _plain_distill(st):
    c, ids = st["case"], st["ids"].long()
    x = st["student"]
    _, d, e = _softmax(x, c["temp"])
    has = ids >= 0
    live = has.any(-1)
    # sums, and the k values of a row, in 64 bits: what they leave of 1 is a small difference, and near its minimum
    # the loss is one
    z = e.sum(-1, dtype=torch.float64)
    y = torch.where(has, st["teacher"].double() / st["teacher_temp"], -math.inf)
    if c["tail"]:
        lq = y - st["lse"].double()[..., None] if st["lse"] is not None else y
    else:
        lq = y - torch.where(live, y.logsumexp(-1), 0.0)[..., None]
    q = torch.exp(lq)
    at = torch.where(has, ids, 0)
    lpi = d.gather(-1, at).double() - torch.log(z)[..., None]
    loss = torch.where(q > 0, q * (lq - lpi), 0.0).sum(-1)
    inside = torch.zeros_like(d, dtype=torch.int8).scatter_add_(-1, at, has.to(torch.int8)) > 0
    mass = q.sum(-1)
    if c["tail"]:
        qr = (1.0 - mass).clamp(min=0.0)
        pr = torch.where(inside, 0.0, e).sum(-1, dtype=torch.float64) / z
        loss = loss + torch.where(qr > 0, qr * (torch.log(qr) - torch.log(pr)), 0.0)
        mass = mass + qr
    out = dict(loss=torch.where(live, loss, 0.0).float(),
               accept=torch.minimum(q, lpi.exp()).sum(-1).float(),
               row_status=torch.zeros(live.shape, dtype=torch.int32, device=x.device))
    if st["gl"] is None:
        return out
    g = e * (mass / z).float()[..., None]
    if c["tail"]:
        g -= torch.where(inside, 0.0, e * (qr / pr / z).float()[..., None])
    g.scatter_add_(-1, at, -q.float())
    g *= (st["gl"] / c["temp"])[..., None]
    return dict(out, grad=torch.where(live[..., None], g, 0.0).to(x.dtype))


_plain = dict(logprobs=_plain_logprobs, logprobs_grad=_plain_logprobs_grad, distill=_plain_distill,
              distill_grad=_plain_distill)


# --------------------------------------------------------------------------- #
# the definitions in 64 bits                                                   #
# --------------------------------------------------------------------------- #
def exact(case, seed):
    st = prepare(case, seed)
    one = _exact_logprobs if case["op"].startswith("logprobs") else _exact_distill
    rows, v = case["b"] * case["t"], case["v"]
    step = max(1, 40_000_000 // v)
    parts = [one(st, slice(r, min(rows, r + step))) for r in range(0, rows, step)]
    lead = (case["b"], case["t"])
    return {n: torch.cat([p[n] for p in parts]).unflatten(0, lead) for n in parts[0]}


def _exact_logprobs(st, sl):
    """Some rows, from logits to log probabilities by torch's log-sum-exp, the order by a stable sort."""
    c = st["case"]
    raw = st["logits"].flatten(0, 1)[sl]
    y = raw.double() / c["temp"]
    lse = torch.logsumexp(y, -1)
    lp = y - lse[:, None]
    p = lp.exp()
    ent = torch.special.entr(p).sum(-1)
    tok = st["tokens"].flatten()[sl].long() if st["tokens"] is not None else torch.zeros(len(y), device=y.device).long()
    dead = tok < 0
    r = torch.arange(len(y), device=y.device)
    out = dict(entropy=ent.masked_fill(dead, 0.0), lse=lse.masked_fill(dead, 0.0),
               row_status=torch.zeros(len(y), dtype=torch.int32, device=y.device))
    if st["tokens"] is not None:
        out["logprob"] = lp[r, tok].masked_fill(dead, 0.0)
    if c["op"] == "logprobs_grad":
        gl, gh = (st[n].flatten()[sl].double()[:, None] for n in ("gl", "gh"))
        # d logprob = 1[v = x] - p;  d H = entr(p) - p H
        g = -gl * p + gh * (torch.special.entr(p) - p * ent[:, None])
        g[r, tok] += gl[:, 0]
        out["grad"] = (g / c["temp"]).masked_fill(dead[:, None], 0.0)
        return out
    if st["tokens"] is not None or c["top"]:
        order = torch.sort(raw.float(), dim=-1, descending=True, stable=True).indices
    if st["tokens"] is not None:
        out["rank"] = (order == tok[:, None]).int().argmax(-1).masked_fill(dead, -1).int()
    if c["top"]:
        best = order[:, :c["top"]]
        out["top_ids"] = best.masked_fill(dead[:, None], -1).int()
        out["top_logprobs"] = lp.gather(-1, best).masked_fill(dead[:, None], -math.inf)
    return out


def _exact_distill(st, sl):
    """Some rows: the divergence of two distributions over the teacher's tokens and (tail) one outcome for the rest,
    and its gradient through that of the log-softmax."""
    c = st["case"]
    y = st["student"].flatten(0, 1)[sl].double() / c["temp"]
    lp = y - torch.logsumexp(y, -1, keepdim=True)
    ids = st["ids"].flatten(0, 1)[sl].long()
    t = st["teacher"].flatten(0, 1)[sl].double() / st["teacher_temp"]
    dead = ids[:, 0] < 0  # a row has all of its entries or none
    ids = ids.clamp(min=0)
    if c["tail"]:
        if st["lse"] is not None:
            t = t - st["lse"].flatten()[sl].double()[:, None]
        rest = (-torch.expm1(torch.logsumexp(t, -1))).clamp(min=0.0)
        t, lpi = torch.cat([t, rest.log()[:, None]], 1), lp.gather(-1, ids)
        left = lp.scatter(-1, ids, -math.inf)
        lps = torch.cat([lpi, torch.logsumexp(left, -1, keepdim=True)], 1)
    else:
        t, lps = torch.log_softmax(t, -1), lp.gather(-1, ids)
    q = t.exp()
    k = ids.shape[1]
    out = dict(loss=torch.where(q > 0, q * (t - lps), 0.0).sum(-1).masked_fill(dead, 0.0),
               accept=torch.minimum(q[:, :k], lps[:, :k].exp()).sum(-1).masked_fill(dead, 0.0),
               row_status=torch.zeros(len(y), dtype=torch.int32, device=y.device))
    if st["gl"] is None:
        return out
    # L = - sum_i q_i lps_i + ..., so the gradient reaches the log probabilities of the teacher's tokens as -q_i, and
    # those of the rest as -q_r times their share of the rest; from ln p to l: g - p sum(g)
    g = torch.zeros_like(lp)
    if c["tail"]:
        g = -q[:, k:] * (left - lps[:, k:]).exp()
    g.scatter_(-1, ids, -q[:, :k])
    g = g - lp.exp() * g.sum(-1, keepdim=True)
    g = g * (st["gl"].flatten()[sl].double() / c["temp"])[:, None]
    return dict(out, grad=g.masked_fill(dead[:, None], 0.0))
