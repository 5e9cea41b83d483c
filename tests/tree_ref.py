"""Plain 64-bit implementations of the operators around a verify step (numpy,
sequence by sequence), the trees and caches the tests use, and the error bounds
the kernels have to keep."""
import numpy as np


def to_f64(t):
    return t.detach().double().cpu().numpy()


def random_parents(rng, B, T, kind):
    """Parents before children: 'chain', 'star', 'random', 'forest' (several roots)."""
    p = np.full((B, T), -1, np.int32)
    for b in range(B):
        for j in range(1, T):
            p[b, j] = {"chain": j - 1, "star": 0}.get(kind, rng.integers(0, j) if kind == "random"
                                                      else rng.integers(-1, j))
    return p


def ancestors(parents, n):
    """[T] parents -> (bool [T, T] ancestor-or-self, depth [T]); rows j >= n empty."""
    T = len(parents)
    see, depth = np.zeros((T, T), bool), np.full(T, -1)
    for j in range(n):
        a = j
        while a >= 0:
            see[j, a] = True
            a = parents[a]
            depth[j] += 1
    return see, depth


def pack_mask(see):
    """bool [B, T, T] -> int32 words [B, T, ceil(T / 32)]"""
    B, T, _ = see.shape
    W = -(-T // 32)
    bits = np.zeros((B, T, W * 32), np.uint64)
    bits[:, :, :T] = see
    words = (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def plan(ctx, n, parents, held, ring, free, table, page, T):
    """The allocator as a host would write it; free and table are updated."""
    B, width, N = len(ctx), table.shape[1], len(free)
    head, tail = ring
    old = free.copy()
    W = -(-T // 32)
    out = dict(held=np.array(held, np.int32), slot_map=np.full((B, T), -1, np.int32),
               positions=np.full((B, T), -1, np.int32), row_status=np.zeros(B, np.int32))
    if parents is not None:
        out["tree_mask"] = np.zeros((B, T, W), np.int32)
    asked = took = gave = 0
    for b in range(B):
        if ctx[b] < 0 or not 0 <= n[b] <= T or not 0 <= held[b] <= width or ctx[b] + n[b] > width * page:
            out["row_status"][b] = 5
            continue
        need = -(-(int(ctx[b]) + int(n[b])) // page)
        if need > held[b]:
            asked += need - held[b]
            if asked > tail - head:
                out["row_status"][b] = 7
                continue
            for i in range(held[b], need):
                table[b, i] = old[(head + took) % N]
                took += 1
        for i in range(need, held[b]):
            free[(tail + gave) % N] = table[b, i]
            gave += 1
        out["held"][b] = need
        if parents is not None and any(not -1 <= parents[b, j] < j for j in range(n[b])):
            out["row_status"][b] = 6
            continue
        see, depth = ancestors(parents[b], n[b]) if parents is not None else (None, np.arange(T))
        for j in range(n[b]):
            at = int(ctx[b]) + j
            out["slot_map"][b, j] = table[b, at // page] * page + at % page
            out["positions"][b, j] = ctx[b] + depth[j]
        if parents is not None:
            out["tree_mask"][b] = pack_mask(see[None])[0]
    out["ring"] = np.array([head + took, tail + gave], np.int64)
    return out


def norm_rotate(x, w, eps, cs, pos, interleaved):
    """x [..., heads, D] of one token; returns (y, bound on the fp32 arithmetic's error)."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    mag = np.abs(y)
    if cs is not None:
        rot = cs.shape[1]
        h = rot // 2
        c, s = (cs[pos, :h], cs[pos, h:]) if 0 <= pos < len(cs) else (np.full(h, np.nan),) * 2
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        mag[..., a] = mag[..., b] = np.abs(ya) + np.abs(yb)
    # norm: D-term sum, square root, reciprocal, two products; rotation: two
    # products and a sum: about (log2-tree of 8 lanes-local + 32 lanes) 16
    # roundings of 2^-24 of the terms' magnitude, taken twice
    return y, mag * 32 * 2.0 ** -24


UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # unit roundoff of the 16-bit types
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the spacing of their subnormals


def attend(q, keys, vals, see, scale, dtype):
    """One (sequence, query head): q [n, D], keys / vals [N, D] fp64, see bool
    [n, N].  Returns (out, lse, tolerance of out, tolerance of lse); keys a row
    does not see are left out of every sum."""
    n, D = q.shape
    out, lse = np.zeros((n, D)), np.full(n, -np.inf)
    tol, tol_l = np.zeros((n, D)), np.zeros(n)
    for i in range(n):
        k, v = keys[see[i]], vals[see[i]]
        N = len(k)
        if N == 0:
            continue
        with np.errstate(all="ignore"):
            s = scale * (k @ q[i])
            top = s.max() if not np.isnan(s).any() else np.nan
            if top == -np.inf:
                continue
            p = np.exp(s - top)
            z = p.sum()
            lse[i] = top + np.log(z)
            out[i] = (p[:, None] * v).sum(0) / z
            # scores: a D-term fp32 sum (any order) and the scaling; the exponent's
            # argument reaches 2^7 log2 units before the exponential underflows to
            # nothing, and its approximation is good to 2^-21
            ds = (D + 8) * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q[i])).max() + 2.0 ** -17
            a = (p[:, None] * np.abs(v)).sum(0) / z
            # probabilities rounded to the 16-bit type (u a, and their subnormals),
            # N-term fp32 sums, the output's own rounding
            u = UNIT[dtype]
            tol[i] = (u + 2 * ds + 4 * (N + 8) * 2.0 ** -24) * a + u * np.abs(out[i]) * 1.01 + \
                TINY[dtype] * (1 + np.abs(v).sum(0))
            tol_l[i] = ds + (N + 8) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[i])
    return out, lse, tol, tol_l
