"""The operators around a verify step, as cases to be measured.

A round of speculative decoding on the target model's side, per layer: page
tables, slots, positions and ancestor masks for the drafted tokens (plan); the
per-head norm and rotation of the new queries and keys and the write of keys
and values into the paged cache (append); attention of the drafted tokens, a
tree or a chain, over the cache (attend); and, once the verify step has chosen
a path, the move of the accepted nodes' keys and values to the places the next
round reads (keep).

With ``own`` false a case runs in plain torch operations, in 32 bits; with
``own`` true through the package's ``TreeCache``.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-6


# --------------------------------------------------------------------------- #
# the cases                                                                    #
# --------------------------------------------------------------------------- #
def listed():
    heads = dict(hq=64, hkv=8, d=128, dtype="bf16")
    return [
        # one verify batch of chains turned trees: 64 requests, 9 nodes each
        dict(name="plan_b64_t9", op="plan", b=64, t=9, page=16, ctx_lo=40, ctx_hi=2000, tree=True),
        # a full server: 1000 requests with trees of 64 nodes
        dict(name="plan_b1000_t64", op="plan", b=1000, t=64, page=16, ctx_lo=1, ctx_hi=16000, tree=True),
        # a single user's single token
        dict(name="append_b1_t1", op="append", b=1, t=1, page=16, ctx_lo=500, ctx_hi=500, rot=128, inter=False,
             norm=True, **heads),
        # the verify batch: 64 requests, 9 tokens
        dict(name="append_b64_t9", op="append", b=64, t=9, page=16, ctx_lo=20, ctx_hi=300, rot=128, inter=False,
             norm=True, **heads),
        # wide trees of a smaller model: 7 query heads per key head, 80-element heads of which 32 are rotated
        dict(name="append_b100_t60_f16_d80", op="append", b=100, t=60, page=32, ctx_lo=5, ctx_hi=100, rot=32,
             inter=True, norm=True, hq=28, hkv=4, d=80, dtype="f16"),
        # one user, plain decoding of one token over a short context
        dict(name="attend_b1_t1_c500", op="attend", b=1, t=1, page=16, ctx_lo=500, ctx_hi=500, tree=False,
             hq=32, hkv=8, d=128, dtype="bf16"),
        # the verify batch: 64 requests of mixed lengths, trees of 9 nodes
        dict(name="attend_b64_t9_c4k", op="attend", b=64, t=9, page=16, ctx_lo=100, ctx_hi=4100, tree=True, **heads),
        # wide trees, few requests: 512 query rows per key head
        dict(name="attend_b16_t64_c8k", op="attend", b=16, t=64, page=64, ctx_lo=4000, ctx_hi=8191, tree=True, **heads),
        # one very long document
        dict(name="attend_b1_t32_c260k", op="attend", b=1, t=32, page=32, ctx_lo=260001, ctx_hi=260001, tree=True,
             **heads),
        # a smaller model in f16 that takes a chunk of its prompt: a chain of 333 tokens, 7 heads per key head
        dict(name="attend_b6_t333_f16_d80", op="attend", b=6, t=333, page=32, ctx_lo=0, ctx_hi=3001, tree=False,
             hq=28, hkv=4, d=80, dtype="f16"),
        # after the verify: the accepted paths of 64 requests, four layers
        dict(name="keep_b64_t9_l4", op="keep", b=64, t=9, page=16, ctx_lo=20, ctx_hi=300, layers=4, keep=5,
             hkv=8, d=128, dtype="bf16"),
        # many requests with wide trees, eight layers in one call
        dict(name="keep_b200_t64_l8", op="keep", b=200, t=64, page=16, ctx_lo=10, ctx_hi=100, layers=8, keep=9,
             hkv=4, d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "keep"])
    page = rng.choice([16, 32, 64])
    hq, hkv = rng.choice([(64, 8), (32, 8), (28, 4), (16, 16), (40, 8), (12, 1), (24, 8)])
    d = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "plan":
        tree = rng.random() < 0.7
        b = _log(rng, 1, 1000)
        t = _log(rng, 1, 64) if tree else _log(rng, 1, max(1, min(2000, 60000 // b)))
        hi = _log(rng, 20, 16000)
        return dict(op=op, b=b, t=t, page=page, ctx_lo=rng.randint(0, hi), ctx_hi=hi, tree=tree)
    if op == "append":
        b = _log(rng, 1, 120)
        t = _log(rng, 1, 60)
        while b * t * (hq + 2 * hkv) * d > 100 * 60 * 36 * 80 * 2:
            b = max(1, b // 2)
        hi = _log(rng, 2, 300)
        return dict(op=op, b=b, t=t, page=page, ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    rot=rng.choice([d, d, 32, 0]), inter=rng.random() < 0.3, norm=rng.random() < 0.8,
                    hq=hq, hkv=hkv, d=d, dtype=dtype)
    if op == "keep":
        b = _log(rng, 1, 200)
        t = _log(rng, 2, 64)
        hi = _log(rng, 2, 100)
        layers = rng.randint(1, 8)
        while b * (hi + t) * layers * hkv * d > 200 * 164 * 8 * 4 * 128:
            b = max(1, b // 2)
            if b == 1:
                break
        return dict(op=op, b=b, t=t, page=page, ctx_lo=rng.randint(0, hi), ctx_hi=hi, layers=layers,
                    keep=rng.randint(1, max(2, (t + 1) // 2)), hkv=hkv, d=d, dtype=dtype)
    tree = rng.random() < 0.75
    b = _log(rng, 1, 64)
    t = _log(rng, 1, 64) if tree else _log(rng, 1, 333)
    hi = _log(rng, 16, 131072)
    # no more keys and no more products than the largest listed cases
    while b > 1 and (b * (hi + t) * hkv * d > 16 * 8255 * 8 * 128 or
                     b * (hi + t) * t * hq * d > 16 * 8255 * 64 * 64 * 128):
        b //= 2
    while (hi + t) * t * hq * d > 260033 * 32 * 64 * 128 or (hi + t) * hkv * d > 260033 * 8 * 128:
        hi //= 2
    return dict(op=op, b=b, t=t, page=page, ctx_lo=rng.randint(0, hi), ctx_hi=hi, tree=tree, hq=hq, hkv=hkv, d=d,
                dtype=dtype)


# --------------------------------------------------------------------------- #
# sizes a case fixes without its seed                                          #
# --------------------------------------------------------------------------- #
def _ctx(case):
    """The context lengths of a case, spread evenly over its range (prepare orders them by the seed)."""
    return np.linspace(case["ctx_lo"], case["ctx_hi"], case["b"]).round().astype(np.int64)


def _nodes(case):
    """Drafted tokens per request, from t down to about half of it (ragged, as confidence-cut drafts are)."""
    t = case["t"]
    return t - (np.arange(case["b"]) % max(1, t // 2))


def _kept(case):
    return np.minimum(case["keep"] - np.arange(case["b"]) % case["keep"], (_nodes(case) + 1) // 2)


def _width(case):
    return -(-(case["ctx_hi"] + case["t"]) // case["page"])


def work(case):
    n, ctx = _nodes(case), _ctx(case)
    b, t = case["b"], case["t"]
    tok = int(n.sum())
    if case["op"] == "plan":
        pages = int((-(-(ctx + n) // case["page"])).sum())
        new = pages - int(_held(case, ctx, n).sum())
        words = -(-t // 32) if case["tree"] else 0
        # lengths, held pages, parents and new pages in; table entries, slots, positions, masks, held and status out
        return dict(bytes=float(16 * b + (4 * tok if case["tree"] else 0) + 8 * max(new, 0) + b * t * (8 + 4 * words)
                                + 8 * b), flops=float(tok))
    d = case["d"]
    if case["op"] == "append":
        el = tok * (case["hq"] + 2 * case["hkv"]) * d
        return dict(bytes=float(4 * el + tok * (8 + 4 * case["rot"])), flops=float(10 * el))
    if case["op"] == "keep":
        # of a path of k nodes the first f, 1 <= f <= k, are in place already (prepare): half of k - 1 move
        rows = float((_kept(case) - 1).sum()) / 2
        return dict(bytes=8 * case["layers"] * rows * case["hkv"] * d + 4.0 * int(_kept(case).sum()) + 16.0 * b,
                    flops=0.0)
    keys = int((ctx + n).sum())
    return dict(bytes=float(4 * keys * case["hkv"] * d + tok * case["hq"] * (4 * d + 4) + 4 * keys // case["page"]),
                flops=float(4 * d * case["hq"] * int((n * (ctx + 1)).sum())))


# --------------------------------------------------------------------------- #
# inputs                                                                       #
# --------------------------------------------------------------------------- #
def _held(case, ctx, n):
    """Pages each request holds before the call: its context's, those of its last round too for every third request
    (so that some give pages back), none for every seventh (a new request)."""
    page = case["page"]
    held = -(-ctx // page)
    i = np.arange(len(ctx))
    held = np.where(i % 3 == 1, np.minimum(held + 2, _width(case)), held)
    return np.where(i % 7 == 3, 0, held)


def _parents(rng, b, t):
    """Trees numbered level by level: the parents of nodes 1.. do not decrease; node 0 is the root."""
    j = np.arange(t)
    p = np.floor(j * rng.random((b, t)) ** 3).astype(np.int64)
    p = np.maximum.accumulate(p, axis=1)
    p[:, 0] = -1
    return p


def _pages(rng, b, width, extra=0):
    """A random assignment of pages: [b, width] of all different pages, and `extra` more."""
    perm = rng.permutation(b * width + extra)
    return perm[:b * width].reshape(b, width), perm[b * width:]


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = np.random.default_rng([seed, 77])
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    b, t, page = case["b"], case["t"], case["page"]
    order = rng.permutation(b)
    ctx, n, width = _ctx(case)[order], _nodes(case)[order], _width(case)

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)

    def randn(*shape, scale=1.0):
        x = torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)
        return (x * scale).to(_DT[case["dtype"]])

    st = dict(case=case, ctx=i32(ctx), n=i32(n), tc=None)
    if case["op"] == "plan":
        held = _held(case, _ctx(case), _nodes(case))[order]
        total = b * width + 64
        table, _ = _pages(rng, b, width)
        # the free ring holds every page that no request holds
        mask = np.zeros(total, bool)
        for r in range(b):
            mask[table[r, :held[r]]] = True
        free = rng.permutation(np.flatnonzero(~mask))
        head = int(rng.integers(0, 5 * total))
        ring = np.full(total, -1, np.int64)
        ring[(head + np.arange(len(free))) % total] = free
        tab = np.full((b, width), -1, np.int64)
        for r in range(b):
            tab[r, :held[r]] = table[r, :held[r]]
        st.update(held=i32(held), ring=torch.tensor([head, head + len(free)], dtype=torch.int64, device=dev),
                  free=i32(ring), table=i32(tab), pages=total,
                  parents=i32(_parents(rng, b, t)) if case["tree"] else None)
    else:
        hkv, d = case["hkv"], case["d"]
        table, _ = _pages(rng, b, width)
        pages = b * width
        st.update(pages=pages, table=i32(table))
        lead = (case["layers"],) if case["op"] == "keep" else ()
        st["kc"], st["vc"] = (randn(*lead, pages, page, hkv, d) for _ in range(2))
    if case["op"] == "append":
        hq, rot = case["hq"], case["rot"]
        # q, k and v as one projection leaves them: side by side in each token's row
        st["qkv"] = randn(b, t, (hq + 2 * hkv) * d, scale=1.7)
        st["qw"], st["kw"] = ((1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(_DT[case["dtype"]])
                              if case["norm"] else None for _ in range(2))
        pos = ctx[:, None] + np.minimum(np.arange(t)[None, :], rng.integers(0, 6, (b, t)))
        at = ctx[:, None] + np.arange(t)[None, :]
        slot = np.take_along_axis(table, at // page, 1) * page + at % page
        slot[np.arange(t)[None, :] >= n[:, None]] = -1
        st.update(pos=i32(pos), slot=i32(slot), cs=None)
        if rot:
            inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
            ang = np.arange(width * page)[:, None] * inv[None, :]
            st["cs"] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(dev)
    elif case["op"] == "attend":
        st["q"] = randn(b, t, case["hq"], d, scale=1.6)
        st["mask"] = None
        if case["tree"]:
            st["mask"] = _plain_mask(i32(_parents(rng, b, t)), st["n"])
    elif case["op"] == "keep":
        # accepted paths: strictly ascending nodes from the root whose moves overwrite no node another move
        # reads, so that a pass can be repeated on the same cache
        kept = _kept(case)[order]
        path = np.full((b, t), -1, np.int64)
        for r in range(b):
            k = int(kept[r])
            f = int(rng.integers(1, k + 1))
            path[r, :f] = np.arange(f)
            path[r, f:k] = np.sort(rng.choice(np.arange(k, n[r]), k - f, replace=False)) if k > f else []
        st.update(path=i32(path), kept=i32(kept))
    if own:
        import speculative_decoding_verification_42_gb300 as sv
        hkv, d = case.get("hkv", 8), case.get("d", 128)
        st["tc"] = sv.TreeCache(max_batch=b, max_tokens=t, q_heads=case.get("hq", hkv), kv_heads=hkv, head_dim=d,
                                dtype=case.get("dtype", "bf16"), page_size=page, num_pages=st["pages"],
                                table_width=width)
    return st


# --------------------------------------------------------------------------- #
# one pass                                                                     #
# --------------------------------------------------------------------------- #
def run(st):
    op = st["case"]["op"]
    return (_own if own else _plain)[op](st)


def _split(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    q, k, v = st["qkv"].split([hq * d, hkv * d, hkv * d], dim=-1)
    return (x.unflatten(-1, (-1, d)) for x in (q, k, v))


def _own_plan(st):
    out = st["tc"].plan(st["ctx"], st["n"], st["held"], st["ring"], st["free"], st["table"], parents=st["parents"],
                        max_tokens=st["case"]["t"])
    return dict(out, free=st["free"], table=st["table"])


def _own_append(st):
    q, k, v = _split(st)
    c = st["case"]
    out = st["tc"].append(q, k, v, st["kc"], st["vc"], st["slot"], st["pos"], st["n"], q_weight=st["qw"],
                          k_weight=st["kw"], eps=_EPS, cos_sin=st["cs"], interleaved=c["inter"])
    return dict(q=out, kc=st["kc"], vc=st["vc"])


def _own_attend(st):
    return st["tc"].attend(st["q"], st["kc"], st["vc"], st["table"], st["ctx"], st["n"], tree_mask=st["mask"])


def _own_keep(st):
    out = st["tc"].keep(st["kc"], st["vc"], st["table"], st["ctx"], st["n"], st["path"], st["kept"])
    return dict(out, kc=st["kc"], vc=st["vc"])


_own = dict(plan=_own_plan, append=_own_append, attend=_own_attend, keep=_own_keep)


def _plain_mask(parents, n):
    """Ancestor-or-self bits [b, t, ceil(t / 32)] (int32 words) of trees given by parents, by doubling the reach."""
    b, t = parents.shape
    idx = torch.arange(t, device=parents.device)
    m = torch.eye(t, device=parents.device).expand(b, t, t)
    hop = parents.long()
    for _ in range(max(1, (t - 1).bit_length())):
        src = hop.clamp(min=0)
        up = torch.gather(m, 1, src[:, :, None].expand(b, t, t)) * (hop >= 0)[:, :, None]
        m = ((m + up) > 0).float()
        hop = torch.where(hop >= 0, torch.gather(hop, 1, src), hop)
    m = (m > 0) & (idx[None, :, None] < n[:, None, None])
    words = -(-t // 32)
    m = torch.nn.functional.pad(m, (0, words * 32 - t)).view(b, t, words, 32).long()
    w = (m << torch.arange(32, device=parents.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def _bits(mask, t):
    """int32 words [.., w] -> booleans [.., t]"""
    m = (mask[..., None] >> torch.arange(32, device=mask.device)) & 1
    return m.flatten(-2)[..., :t] > 0


def _plain_plan(st):
    c = st["case"]
    page, width, total, t = c["page"], _width(c), st["pages"], c["t"]
    ctx, n, held = st["ctx"].long(), st["n"].long(), st["held"].long()
    dev = ctx.device
    ok = (ctx >= 0) & (n >= 0) & (n <= t) & (held >= 0) & (held <= width) & (ctx + n <= width * page)
    need = torch.where(ok, (ctx + n + page - 1) // page, held)
    want, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    head, tail = st["ring"][0], st["ring"][1]
    before, back_before = want.cumsum(0) - want, back.cumsum(0) - back
    short = (want > 0) & (before + want > tail - head)
    want = torch.where(short, torch.zeros_like(want), want)
    held_out = torch.where(short, held, need)
    col = torch.arange(width, device=dev)
    # new pages: from the head of the ring, in the order of the requests
    new = (col[None, :] >= held[:, None]) & (col[None, :] < (held + want)[:, None])
    at = (head + before[:, None] + col[None, :] - held[:, None]) % total
    old = st["table"].long()
    table = torch.where(new, st["free"].long()[at], old)
    # surplus pages: to the tail
    gone = (col[None, :] >= need[:, None]) & (col[None, :] < held[:, None])
    to = (tail + back_before[:, None] + col[None, :] - need[:, None]) % total
    dest = torch.where(gone, to, torch.full_like(to, total))
    free = torch.cat([st["free"], st["free"][:1]])
    free[dest.flatten()] = old.flatten().int()
    st["free"].copy_(free[:total])
    st["table"].copy_(table)
    j = torch.arange(t, device=dev)
    good = (ok & ~short)[:, None] & (j[None, :] < n[:, None])
    place = (ctx[:, None] + j[None, :]).clamp(0, width * page - 1)
    slot = torch.gather(table, 1, place // page) * page + place % page
    mask = None
    if st["parents"] is not None:
        mask = torch.where(good[:, :, None], _plain_mask(st["parents"], st["n"]), 0)
        depth = _bits(mask, t).sum(-1) - 1
    else:
        depth = j[None, :].expand(len(ctx), t)
    status = torch.where(ok, torch.where(short, 7, 0), 5).int()
    out = dict(held=held_out.int(), ring=torch.stack([head + want.sum(), tail + back.sum()]),
               slot_map=torch.where(good, slot, -1).int(),
               positions=torch.where(good, ctx[:, None] + depth, -1).int(), row_status=status)
    if mask is not None:
        out["tree_mask"] = mask
    return dict(out, free=st["free"], table=st["table"])


def _rotate(x, cs, pos, inter):
    """x [b, t, h, d] in 32 bits, the first rot elements rotated by the angles of cs [positions, rot] at pos"""
    rot = cs.shape[1]
    c, s = cs[pos.long()].unsqueeze(2).split(rot // 2, dim=-1)
    head, tail = x[..., :rot], x[..., rot:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, tail], -1)


def _plain_append(st):
    c = st["case"]
    q, k, v = _split(st)
    dt = q.dtype

    def norm(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w.float()
        return x if st["cs"] is None else _rotate(x, st["cs"], st["pos"], c["inter"])

    live = st["slot"] >= 0
    qo = torch.where(live[:, :, None, None], norm(q, st["qw"]), 0.0).to(dt)
    at = st["slot"][live].long()
    st["kc"].view(-1, c["hkv"], c["d"])[at] = norm(k, st["kw"]).to(dt)[live]
    st["vc"].view(-1, c["hkv"], c["d"])[at] = v[live]
    return dict(q=qo, kc=st["kc"], vc=st["vc"])


def _plain_attend(st):
    c = st["case"]
    b, t, hq, hkv, d, page = (c[x] for x in ("b", "t", "hq", "hkv", "d", "page"))
    g, dev = hq // hkv, st["q"].device
    keys = _width(c) * page
    # sequences at a time, so that the scores stay within some gigabytes
    step = max(1, min(b, 2 ** 30 // (keys * max(hq * t, 2 * hkv * d))))
    outs, lses = [], []
    pos, j = torch.arange(keys, device=dev), torch.arange(t, device=dev)
    for b0 in range(0, b, step):
        sl = slice(b0, min(b, b0 + step))
        ctx, n, tab = st["ctx"][sl].long(), st["n"][sl].long(), st["table"][sl].long()
        m = len(ctx)
        k, v = (x[tab].view(m, keys, hkv, d).permute(0, 2, 1, 3).float() for x in (st["kc"], st["vc"]))
        q = st["q"][sl].float().view(m, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(m, hkv, t * g, d)
        s = torch.matmul(q, k.transpose(-1, -2)).view(m, hkv, t, g, keys) * (d ** -0.5)
        tree = _bits(st["mask"][sl], t) if st["mask"] is not None else (j[:, None] >= j[None, :]).expand(m, t, t)
        node = pos[None, :] - ctx[:, None]
        inside = (node >= 0) & (node < n[:, None])
        vis = torch.gather(tree, 2, node.clamp(0, t - 1)[:, None, :].expand(m, t, keys))
        vis = (vis & inside[:, None, :]) | (node < 0)[:, None, :]
        vis = vis & (j[None, :] < n[:, None])[:, :, None]
        s = s.masked_fill(~vis[:, None, :, None, :], -math.inf)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = torch.exp(s - top)
        z = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(m, hkv, t * g, keys), v).view(m, hkv, t, g, d)
        o = torch.where(z > 0, o / z, 0.0)
        outs.append(o.permute(0, 2, 1, 3, 4).reshape(m, t, hq, d).to(st["q"].dtype))
        lses.append((top + torch.log(z)).permute(0, 2, 1, 3, 4).reshape(m, t, hq))
    return dict(out=torch.cat(outs), lse=torch.cat(lses))


def _plain_keep(st):
    c = st["case"]
    page, t = c["page"], c["t"]
    ctx, path = st["ctx"].long(), st["path"].long()
    i = torch.arange(t, device=ctx.device)
    live = i[None, :] < st["kept"][:, None]

    def slots(node):
        at = (ctx[:, None] + node.clamp(min=0))
        return (torch.gather(st["table"].long(), 1, at // page) * page + at % page)[live]

    src, dst = slots(path), slots(i[None, :].expand_as(path))
    for x in (st["kc"], st["vc"]):
        flat = x.view(c["layers"], -1, c["hkv"], c["d"])
        flat[:, dst] = flat[:, src]
    return dict(ctx_len=(st["ctx"] + st["kept"]).int(), row_status=torch.zeros_like(st["ctx"]), kc=st["kc"],
                vc=st["vc"])


_plain = dict(plan=_plain_plan, append=_plain_append, attend=_plain_attend, keep=_plain_keep)


# --------------------------------------------------------------------------- #
# the definitions in 64 bits                                                   #
# --------------------------------------------------------------------------- #
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return dict(plan=_exact_plan, append=_exact_append, attend=_exact_attend, keep=_exact_keep)[case["op"]](st)


def _exact_plan(st):
    """Request by request, as a host's allocator would: integers only."""
    c = st["case"]
    page, t, total = c["page"], c["t"], st["pages"]
    ctx, n, held = (st[x].tolist() for x in ("ctx", "n", "held"))
    head, tail = st["ring"].tolist()
    free, table = st["free"].cpu().numpy().copy(), st["table"].cpu().numpy().copy()
    old = free.copy()
    par = st["parents"].tolist() if st["parents"] is not None else None
    slot, posn = np.full((len(ctx), t), -1, np.int32), np.full((len(ctx), t), -1, np.int32)
    mask = np.zeros((len(ctx), t, -(-t // 32)), np.uint32)
    avail, status, took, gave = tail - head, [0] * len(ctx), 0, 0
    for r in range(len(ctx)):
        need = -(-(ctx[r] + n[r]) // page)
        if need > held[r] and took + need - held[r] > avail:
            status[r] = 7
            avail = -1  # those behind it that need a page wait too
            continue
        for col in range(held[r], need):
            table[r, col] = old[(head + took) % total]
            took += 1
        for col in range(need, held[r]):
            free[(tail + gave) % total] = table[r, col]
            gave += 1
        held[r] = need
        up = []
        for j in range(n[r]):
            p = par[r][j] if par else j - 1
            up.append((up[p] if p >= 0 else set()) | {j} if par else None)
            slot[r, j] = table[r, (ctx[r] + j) // page] * page + (ctx[r] + j) % page
            posn[r, j] = ctx[r] + (len(up[j]) - 1 if par else j)
            for a in up[j] or ():
                mask[r, j, a // 32] |= np.uint32(1 << (a % 32))
    out = dict(held=torch.tensor(held, dtype=torch.int32), ring=torch.tensor([head + took, tail + gave]),
               slot_map=torch.from_numpy(slot), positions=torch.from_numpy(posn),
               row_status=torch.tensor(status, dtype=torch.int32))
    if par:
        out["tree_mask"] = torch.from_numpy(mask.view(np.int32))
    return dict(out, free=torch.from_numpy(free), table=torch.from_numpy(table))


def _exact_append(st):
    c = st["case"]
    hq, hkv, d, rot = c["hq"], c["hkv"], c["d"], c["rot"]
    x = st["qkv"].double().cpu().numpy().reshape(c["b"], c["t"], hq + 2 * hkv, d)
    slot, pos = st["slot"].cpu().numpy(), st["pos"].cpu().numpy()

    def turn(y, w):
        if w is not None:
            y = y / np.sqrt((y ** 2).sum(-1, keepdims=True) / d + _EPS) * w.double().cpu().numpy()
        if rot:
            cs = st["cs"].double().cpu().numpy()[pos]
            z = cs[:, :, None, :rot // 2] + 1j * cs[:, :, None, rot // 2:]
            if c["inter"]:
                w2 = (y[..., 0:rot:2] + 1j * y[..., 1:rot:2]) * z
                y[..., 0:rot:2], y[..., 1:rot:2] = w2.real, w2.imag
            else:
                w2 = (y[..., :rot // 2] + 1j * y[..., rot // 2:rot]) * z
                y[..., :rot // 2], y[..., rot // 2:rot] = w2.real, w2.imag
        return y

    q = turn(x[:, :, :hq].copy(), st["qw"])
    k = turn(x[:, :, hq:hq + hkv].copy(), st["kw"])
    v = x[:, :, hq + hkv:]
    live = slot >= 0
    q[~live] = 0.0
    kc, vc = (y.double().cpu().numpy().reshape(-1, hkv, d) for y in (st["kc"], st["vc"]))
    kc[slot[live]], vc[slot[live]] = k[live], v[live]
    shape = tuple(st["kc"].shape)
    return dict(q=torch.from_numpy(q), kc=torch.from_numpy(kc.reshape(shape)), vc=torch.from_numpy(vc.reshape(shape)))


def _exact_attend(st):
    """Sequence by sequence, and only the keys that it has; scores in slices of its nodes."""
    c = st["case"]
    t, hq, hkv, d, page = (c[x] for x in ("t", "hq", "hkv", "d", "page"))
    g = hq // hkv
    ctx, n, dev = st["ctx"].tolist(), st["n"].tolist(), st["q"].device
    out = torch.zeros(c["b"], t, hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((c["b"], t, hq), -math.inf, dtype=torch.float64, device=dev)
    words = st["mask"].cpu().numpy().view(np.uint32) if st["mask"] is not None else None
    for r in range(c["b"]):
        keys = ctx[r] + n[r]
        tab = st["table"][r, :-(-keys // page)].long()
        k, v = (x[tab].reshape(-1, hkv, d)[:keys].double() for x in (st["kc"], st["vc"]))
        for j0 in range(0, n[r], 16):
            js = list(range(j0, min(n[r], j0 + 16)))
            see = np.ones((len(js), keys), bool)
            for i, j in enumerate(js):
                for a in range(n[r]):
                    see[i, ctx[r] + a] = bool(words[r, j, a // 32] >> np.uint32(a % 32) & 1) if words is not None \
                        else a <= j
            q = st["q"][r, js].double().view(len(js), hkv, g, d)
            s = torch.einsum("ihgd,khd->ihgk", q, k) / math.sqrt(d)
            s = torch.where(torch.from_numpy(see).to(dev)[:, None, None, :], s, -math.inf)
            lse[r, js] = torch.logsumexp(s, -1).reshape(len(js), hq)
            out[r, js] = torch.einsum("ihgk,khd->ihgd", torch.softmax(s, -1), v).reshape(len(js), hq, d)
    return dict(out=out, lse=lse)


def _exact_keep(st):
    c = st["case"]
    page = c["page"]
    tab, path = st["table"].cpu().numpy(), st["path"].cpu().numpy()
    ctx, kept = st["ctx"].tolist(), st["kept"].tolist()
    res = []
    for x in (st["kc"], st["vc"]):
        y = x.clone()
        for r in range(c["b"]):
            for i in range(kept[r]):
                a, z = ctx[r] + int(path[r, i]), ctx[r] + i
                y[:, tab[r, z // page], z % page] = x[:, tab[r, a // page], a % page]
        res.append(y.double())
    return dict(ctx_len=torch.tensor([a + k for a, k in zip(ctx, kept)], dtype=torch.int32),
                row_status=torch.zeros(c["b"], dtype=torch.int32), kc=res[0], vc=res[1])
