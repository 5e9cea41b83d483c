"""Plain 64-bit implementations of the operators that score rows of logits
(numpy, row by row), and the error bounds the kernels have to keep."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}      # half a step of a type
LEAST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -28}  # an eighth of the smallest step, or what is flushed
NAN = float("nan")


def softmax(l, temp):
    """m, d = (l - m) / temp, ln Z, p of one row."""
    m = l.max()
    with np.errstate(invalid="ignore"):
        d = (l - m) / temp
    e = np.exp(d)
    z = e.sum()
    return m, d, np.log(z), e / z


def adds(V):
    """The longest chain of fp32 additions that a sum over a row may take: the 128
    threads of a CTA, with two sums each, share all of it at most, and tens join them."""
    return -(-V // 256) + 48


def logz_bound(V, p, d):
    """Of ln Z, absolute: a term 2^x is off by 2^-22 (the instruction's bound), its
    exponent by the difference's, the constant's and the product's rounding; the sum by
    its additions; ln and what is stored by a few more."""
    ed = float((p * np.abs(np.where(p > 0, d, 0))).sum())
    return U * (4 + 3 * ed + adds(V) + 8)


def logprobs(l, tok, temp, top_n, kind, gl=0.0, gh=0.0):
    """One row of float64 logits -> dict of results and dict of bounds."""
    V = len(l)
    none = dict(logprob=0.0, rank=-1, entropy=0.0, lse=0.0, row_status=0, top_ids=np.full(top_n, -1),
                top_logprobs=np.full(top_n, -np.inf), grad=np.zeros(V))
    zero = dict(logprob=0.0, entropy=0.0, lse=0.0, top_logprobs=np.zeros(top_n), grad=np.zeros(V))
    if tok == -1:
        return none, zero
    bad = tok is not None and not 0 <= tok < V
    if bad or not l.max() > -np.inf or not l.max() < np.inf:  # NaN is neither
        return dict(none, logprob=NAN, entropy=NAN, lse=NAN, row_status=1 if bad else 3,
                    top_logprobs=np.full(top_n, NAN)), zero
    m, d, lz, p = softmax(l, temp)
    live = p > 0
    lp = np.where(l > -np.inf, d - lz, -np.inf)
    plp = np.where(live, p * np.where(live, lp, 0), 0.0)
    ent = -plp.sum()
    order = np.lexsort((np.arange(V), -l))
    order = order[l[order] > -np.inf]
    top = np.full(top_n, -1)
    top[:min(top_n, len(order))] = order[:top_n]
    res = dict(entropy=ent, lse=m / temp + lz, row_status=0, top_ids=top,
               top_logprobs=np.where(top >= 0, lp[top], -np.inf))
    bz = logz_bound(V, p, d)
    ad = np.abs(np.where(live, d, 0))
    ed, ed2 = float((p * ad).sum()), float((p * ad * ad).sum())

    def lp_bound(v):
        return bz + U * (3 * np.abs(d[v]) + 2 * np.abs(lp[v]))

    bound = dict(lse=bz + U * (2 * abs(m / temp) + abs(lz) + abs(res["lse"])),
                 entropy=2 * bz + U * ((adds(V) + 16) * ed + 4 * ed2 + 2 * ent),
                 top_logprobs=np.where(top >= 0, lp_bound(top), 0.0))
    g = -gh * (plp + p * ent)
    if tok is not None:
        res["logprob"] = lp[tok]
        bound["logprob"] = lp_bound(tok) if lp[tok] > -np.inf else 0.0
        res["rank"] = int((l > l[tok]).sum() + ((l == l[tok]) & (np.arange(V) < tok) & (l > -np.inf)).sum())
        g = g + gl * ((np.arange(V) == tok) - p)
    res["grad"] = g / temp
    # p is off by ln Z's bound and its own exponent's, relative; ln p + H by theirs, absolute; the products by 8 U
    rel = bz + U * (12 + 3 * ad)
    off = p * (abs(gl) * rel + abs(gh) * (np.abs(np.where(live, lp + ent, 0)) * rel + bz + bound["entropy"]
                                          + U * (4 * ad + 4 * abs(lz) + 4 * ent)))
    # 2^x is 0 below 2^-126: of p (gl + gh (ln p + H)) that loses what it has at p = 2^-126 at most, as p |ln p| grows
    # with p there: 2^-126 (|gl| + |gh| (126 ln 2 + ln Z + H))
    off = off + 2.0 ** -126 * (abs(gl) + abs(gh) * (88 + abs(lz) + ent))
    off = off + 4 * U * (abs(gl) * (0 if tok is None else (np.arange(V) == tok)))
    bound["grad"] = off / temp * 1.01 + (np.abs(res["grad"]) + off / temp) * (HALF[kind] * 1.01 + 2 * U) + 8 * LEAST[kind]
    return res, bound


def distill(l, ids, t, temp, t_temp, tail, t_lse, w, kind):
    """One row -> dict of results and dict of bounds."""
    V = len(l)
    has = ids != -1
    none = dict(loss=0.0, accept=0.0, row_status=0, grad=np.zeros(V))
    zero = dict(loss=0.0, accept=0.0, grad=np.zeros(V))
    if not has.any():
        return none, zero
    ids, t = ids[has], t[has]
    fail = dict(none, loss=NAN, accept=NAN)
    if (ids < 0).any() or (ids >= V).any() or len(set(ids.tolist())) < len(ids):
        return dict(fail, row_status=1), zero
    if not l.max() > -np.inf or not l.max() < np.inf or not t.max() < np.inf or \
            (not tail and t.max() == -np.inf) or not np.isfinite(t_lse):
        return dict(fail, row_status=3), zero
    m, d, lz, p = softmax(l, temp)
    y = t / t_temp
    lq = y - (t_lse if tail else y.max() + np.log(np.exp(y - y.max()).sum()))
    q = np.exp(lq)
    inside = np.zeros(V, bool)
    inside[ids] = True
    pi, li = p[ids], d[ids] - lz
    with np.errstate(invalid="ignore", divide="ignore"):
        terms = np.where(q > 0, q * (lq - li), 0.0)
        loss, mass = terms.sum(), q.sum()
        # the rest in logarithms: its share of a confident student's row is too small for a number
        rest = np.where(inside, -np.inf, d)
        top = rest.max() if tail else -np.inf
        share = np.exp(rest - top) if top > -np.inf else np.zeros(V)
        lr = top + np.log(share.sum())
        share = share / max(share.sum(), 1.0)
        qr = 0.0
        if tail:
            qr = max(0.0, 1.0 - mass)
            if qr > 0:
                loss = loss + qr * (np.log(qr) - (lr - lz))
            mass = mass + qr
    g = mass * p - qr * share
    g[ids] -= q
    res = dict(loss=loss, accept=np.minimum(q, pi).sum(), row_status=0, grad=g * w / temp)
    bz = logz_bound(V, p, d)
    # q: the exponent in fp32 (its value, and the row's sum without tail), 2^x's and the product's roundings
    bq = U * (12 + np.abs(np.where(q > 0, lq, 0)) + (adds(0) if not tail else 0))
    dq = float((q * bq).sum()) + 2 * U  # of the sum of q, and so of q_r
    fin = np.isfinite(loss)
    with np.errstate(invalid="ignore", divide="ignore"):
        b = (q * bq * np.abs(np.where(q > 0, lq - li, 0))).sum() + mass * 2 * bz + U * abs(loss)
        if tail and top > -np.inf:
            # the rest's largest distance is rounded too
            b += dq * (2 + abs(np.log(max(qr, dq)) - lr + lz)) + qr * (2 * bz + 4 * U * abs(top))
    bound = dict(loss=b if fin else 0.0, accept=float((q * bq + pi * (2 * bz + U * (8 + 3 * np.abs(
        np.where(pi > 0, d[ids], 0))))).sum()) + U * 4)
    ad = np.abs(np.where(p > 0, d, 0))
    off = p * mass * (bz + dq + U * (12 + 3 * ad))
    off[ids] += q * (bq + 4 * U)
    far = np.abs(np.where(share > 0, rest, 0) - (top if top > -np.inf else 0))
    off += share * (dq + qr * (3 * bz + U * (12 + 3 * far)))
    off = off * abs(w) / temp
    bound["grad"] = off * 1.01 + (np.abs(res["grad"]) + off) * (HALF[kind] * 1.01 + 2 * U) + 8 * LEAST[kind]
    return res, bound
