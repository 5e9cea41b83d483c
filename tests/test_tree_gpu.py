"""The operators around a verify step on the GPU, against the plain 64-bit
implementations of tree_ref.py, at the sizes, masks and layouts where they can
go wrong.  Bounds come from the roundings the operators make (tree_ref.py)."""
import numpy as np
import pytest

import tree_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_42_gb300 import build
    build.build()
    import speculative_decoding_verification_42_gb300 as m
    m.load_library()
    return m


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _rand(rng, shape, dtype, scale=1.0):
    import torch
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(_dt(dtype)).cuda()


def _tc(sv, B, T, Hq, Hkv, D, page, pages, width, dtype="bf16"):
    return sv.TreeCache(max_batch=B, max_tokens=T, q_heads=Hq, kv_heads=Hkv, head_dim=D, dtype=dtype,
                        page_size=page, num_pages=pages, table_width=width)


def _layout(rng, pages, page, Hkv, D, dtype, kind, fill=None):
    """K and V caches of one layout: 'tokens' [pages, page, H, D], 'heads'
    [pages, H, page, D] and 'pairs' [pages, 2, page, H, D] storage."""
    import torch
    if kind == "pairs":
        kv = _rand(rng, (pages, 2, page, Hkv, D), dtype)
        return kv[:, 0], kv[:, 1]
    if kind == "heads":
        return tuple(_rand(rng, (pages, Hkv, page, D), dtype).permute(0, 2, 1, 3) for _ in range(2))
    return tuple(_rand(rng, (pages, page, Hkv, D), dtype) for _ in range(2))


# --------------------------------------------------------------------------- #
# plan                                                                         #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("B,T,page,kind", [
    (1, 1, 8, "chain"), (1, 1, 16, None), (5, 9, 16, "random"), (3, 256, 16, "chain"), (4, 33, 64, "forest"),
    (700, 7, 16, "random"), (1300, 3, 8, None), (2, 2100, 32, None), (9, 64, 1024, "star"), (3, 32, 16, "random")])
def test_plan(sv, B, T, page, kind):
    import torch
    rng = np.random.default_rng(B * 1000 + T)
    width = max(2, -(-(T + 300) // page))
    N = B * width
    table, free = np.full((B, width), -1, np.int32), rng.permutation(N).astype(np.int32)
    at = int(rng.integers(0, 3 * N))
    free, ring, held = np.roll(free, at % N), (at, at + N), np.zeros(B, np.int32)
    tc = _tc(sv, B, T, 2, 1, 16, page, N, width)
    dev = dict(held=_i32(held), ring=torch.tensor(ring, dtype=torch.int64).cuda(), free=_i32(free), table=_i32(table))
    for _ in range(4):  # rounds: lengths come and go, some out of range
        ctx = rng.integers(0, 300, B)
        n = rng.integers(0, T + 1, B)
        ctx[rng.random(B) < 0.1] = 0
        n[rng.random(B) < 0.1] = 0
        if B > 3:
            ctx[1], n[2] = -5, T + 1
            ctx[3] = width * page
        par = ref.random_parents(rng, B, T, kind) if kind else None
        if kind == "random" and B > 4 and T > 2:
            par[4, 2] = 2
            n[4], ctx[4] = T, 3
        want = ref.plan(ctx, n, par, held, ring, free, table, page, T)
        for again in range(2):  # a call on unchanged inputs repeats its result
            got = tc.plan(_i32(ctx), _i32(n), dev["held"], dev["ring"], dev["free"], dev["table"],
                          parents=_i32(par) if kind else None, max_tokens=T)
            for name, w in want.items():
                assert (got[name].cpu().numpy() == w).all(), (name, again)
            assert set(got) == set(want)
            assert (dev["table"].cpu().numpy() == table).all()
            assert (dev["free"].cpu().numpy() == free).all()
        held, ring = want["held"], tuple(int(x) for x in want["ring"])
        dev["held"], dev["ring"] = got["held"], got["ring"]
    tc.close()


def test_plan_runs_out_of_pages(sv):
    """The sequences from the first that does not fit get none, those that need
    none are served, and pages returned are free from the next call on."""
    import torch
    B, T, page, width, N = 6, 4, 8, 4, 5
    tc = _tc(sv, B, T, 2, 1, 16, page, N, width)
    pool = tc.new_pool(B)
    table, free = pool["block_table"].cpu().numpy().copy(), pool["free_pages"].cpu().numpy().copy()
    held, ring = np.zeros(B, np.int32), (0, N)
    state = (pool["held"], pool["ring"])
    seen = set()
    for ctx, n in (([8, 0, 20, 0, 1, 0], [1, 0, 3, 0, 1, 0]), ([0, 0, 20, 4, 1, 0], [0, 0, 3, 4, 1, 1]),
                   ([0, 9, 20, 4, 1, 0], [0, 1, 3, 4, 1, 1]), ([0] * 6, [0] * 6)):
        want = ref.plan(ctx, n, None, held, ring, free, table, page, T)
        got = tc.plan(_i32(ctx), _i32(n), *state, pool["free_pages"], pool["block_table"], max_tokens=T)
        for name, w in want.items():
            assert (got[name].cpu().numpy() == w).all(), (name, got[name], w)
        assert (pool["block_table"].cpu().numpy() == table).all()
        assert (pool["free_pages"].cpu().numpy() == free).all()
        held, ring, state = want["held"], tuple(want["ring"]), (got["held"], got["ring"])
        seen |= set(want["row_status"].tolist())
    assert seen == {0, 7}
    assert sorted(free.tolist()) == list(range(N)) and ring[1] - ring[0] == N
    with pytest.raises(sv.SpecVerifyError):  # held in and out are two buffers
        tc.plan(_i32([0] * 6), _i32([0] * 6), *state, pool["free_pages"], pool["block_table"], max_tokens=T,
                out=dict(held=state[0]))
    torch.cuda.synchronize()
    tc.close()


# --------------------------------------------------------------------------- #
# append                                                                       #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,inter,norm,dtype,kind", [
    (1, 1, 8, 2, 128, 128, False, True, "bf16", "tokens"), (3, 9, 64, 8, 128, 128, False, True, "bf16", "tokens"),
    (2, 5, 7, 1, 80, 32, False, True, "f16", "heads"), (2, 5, 7, 1, 80, 80, True, True, "f16", "pairs"),
    (4, 3, 6, 3, 16, 16, False, False, "bf16", "tokens"), (2, 7, 5, 5, 64, 48, False, True, "bf16", "heads"),
    (2, 3, 4, 2, 256, 256, False, True, "f16", "pairs"), (2, 3, 4, 2, 192, 64, True, True, "bf16", "tokens"),
    (3, 4, 16, 1, 112, 0, False, True, "bf16", "tokens"), (3, 4, 3, 3, 96, 0, False, False, "f16", "heads")])
def test_append(sv, B, T, Hq, Hkv, D, rot, inter, norm, dtype, kind):
    import torch
    rng = np.random.default_rng(D + rot + B)
    page, pages, P = 8, 16, 40
    tc = _tc(sv, B, T, Hq, Hkv, D, page, pages, 4, dtype)
    qkv = _rand(rng, (B, T, (Hq + 2 * Hkv) * D), dtype, 2.0)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
    if T > 2:
        q[0, 1] = 0.0   # a zero head: norm of eps alone
        k[0, 2] *= 50.0
    kc, vc = _layout(rng, pages, page, Hkv, D, dtype, kind)
    slot = rng.permutation(pages * page)[:B * T].reshape(B, T)
    pos = rng.integers(0, P, (B, T))
    n = rng.integers(1, T + 1, B)
    n[0] = T
    if B > 1:
        slot[1, 0] = -1
    if B > 2:
        slot[2, 0] = pages * page
    qw, kw = ((1 + 0.3 * _rand(rng, (D,), dtype)).to(_dt(dtype)) if norm else None for _ in range(2))
    cs = rng.standard_normal((P, rot)).astype(np.float32) if rot else None
    if rot and B > 1 and T > 1:
        pos[B - 1, 1], n[B - 1] = P, T  # beyond the table
    want_k, want_v = ref.to_f64(kc), ref.to_f64(vc)
    tol_k = np.zeros_like(want_k)
    want_q, tol_q = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D))
    u = ref.UNIT[dtype]
    xq, xk, xv = (ref.to_f64(x) for x in (q, k, v))
    w64 = [ref.to_f64(w) if norm else None for w in (qw, kw)]
    cs64 = cs.astype(np.float64) if rot else None
    for b in range(B):
        for j in range(n[b]):
            s = slot[b, j]
            if not 0 <= s < pages * page:
                continue
            want_q[b, j], tol_q[b, j] = ref.norm_rotate(xq[b, j], w64[0], 1e-6, cs64, pos[b, j], inter)
            want_k[s // page, s % page], tol_k[s // page, s % page] = \
                ref.norm_rotate(xk[b, j], w64[1], 1e-6, cs64, pos[b, j], inter)
            want_v[s // page, s % page] = xv[b, j]
    got = tc.append(q, k, v, kc, vc, _i32(slot), _i32(pos), _i32(n), q_weight=qw, k_weight=kw,
                    cos_sin=torch.from_numpy(cs).cuda() if rot else None, interleaved=inter)
    torch.cuda.synchronize()

    def close(got, want, tol):
        got = ref.to_f64(got)
        assert (np.isnan(got) == np.isnan(want)).all()
        with np.errstate(invalid="ignore"):
            err = np.abs(got - want) - (tol + u * (np.abs(want) + tol) + ref.TINY[dtype])
        assert not (err > 0).any(), float(np.nanmax(err))

    close(got, want_q, tol_q)
    close(kc, want_k, tol_k)
    assert (ref.to_f64(vc) == want_v).all()
    tc.close()


# --------------------------------------------------------------------------- #
# attend                                                                       #
# --------------------------------------------------------------------------- #
def _attend_case(sv, rng, B, T, Hq, Hkv, D, page, ctx, n, dtype, kind="tokens", tree="random", std=1.5, scale=None,
                 see=None, touch=None, poison=True, stream=None):
    """Runs attend on random data (pages in random order, everything outside the
    sequences' tokens NaN or inf when poison) and compares with tree_ref."""
    import torch
    ctx, n = np.asarray(ctx), np.asarray(n)
    width = max(1, int(-(-(ctx + n).max() // page))) + 1
    pages = B * width + 3
    tc = _tc(sv, B, T, Hq, Hkv, D, page, pages, width, dtype)
    table = rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)
    kc, vc = _layout(rng, pages, page, Hkv, D, dtype, kind)
    q = _rand(rng, (B, T, Hq, D), dtype, std)
    if see is None and tree:
        par = ref.random_parents(rng, B, T, tree)
        see = np.stack([ref.ancestors(par[b], n[b])[0] for b in range(B)])
    node_see = see if see is not None else np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    if poison:
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b in range(B):
            for i in range(ctx[b] + n[b]):
                used[table[b, i // page], i % page] = True
        bad = [float("nan"), float("inf"), -float("inf")]
        for t in (kc, vc):
            t[~used.cuda()] = torch.tensor(bad, dtype=t.dtype, device="cuda")[rng.integers(0, 3)]
        table_dev = table.copy()
        for b in range(B):  # entries past a sequence's pages are never followed
            table_dev[b, -(-int(ctx[b] + n[b]) // page):] = rng.choice([-1, 2 ** 30, pages])
    else:
        table_dev = table
    if touch:
        touch(q, kc, vc, table)
    mask = _i32(ref.pack_mask(see)) if see is not None else None
    sc = D ** -0.5 if scale is None else scale
    got = tc.attend(q, kc, vc, _i32(table_dev), _i32(ctx), _i32(n), tree_mask=mask, scale=scale, stream=stream)
    torch.cuda.synchronize()
    assert tc.check() == sv.SPEC_OK
    tc.close()
    q64, k64, v64 = ref.to_f64(q), ref.to_f64(kc), ref.to_f64(vc)
    out, lse = ref.to_f64(got["out"]), ref.to_f64(got["lse"])
    worst = 0.0
    for b in range(B):
        N = int(ctx[b] + n[b])
        at = np.arange(N)
        k = k64[table[b, at // page], at % page]
        v = v64[table[b, at // page], at % page]
        vis = np.concatenate([np.ones((n[b], ctx[b]), bool), node_see[b][:n[b], :n[b]]], 1)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            o, l, to, tl = ref.attend(q64[b, :n[b], h], k[:, hk], v[:, hk], vis, sc, dtype)
            go, gl = out[b, :n[b], h], lse[b, :n[b], h]
            fin = np.isfinite(o)
            assert (np.isnan(go) == np.isnan(o)).all() and (go[np.isinf(o)] == o[np.isinf(o)]).all()
            assert not (np.abs(go - o)[fin] > to[fin]).any(), (b, h, float((np.abs(go - o)[fin] - to[fin]).max()))
            if fin.any():
                worst = max(worst, float((np.abs(go - o)[fin] / (to[fin] + 1e-300)).max()))
            finl = np.isfinite(l)
            assert (np.isnan(gl) == np.isnan(l)).all() and (gl[np.isinf(l)] == l[np.isinf(l)]).all()
            assert (np.abs(gl - l)[finl] <= tl[finl]).all(), (b, h, np.abs(gl - l)[finl].max())
        assert (out[b, n[b]:] == 0).all() and (lse[b, n[b]:] == -np.inf).all()
    return worst


@pytest.mark.parametrize("B,T,Hq,Hkv,D,page,ctx,n,dtype,kind,tree", [
    # one token: no context, one key, around a page's and a tile's end
    (1, 1, 8, 8, 64, 16, [0], [1], "bf16", "tokens", None),
    (5, 1, 8, 2, 128, 16, [1, 15, 16, 127, 128], [1] * 5, "bf16", "tokens", None),
    (4, 1, 32, 8, 128, 8, [500, 63, 64, 255], [1] * 4, "f16", "heads", "random"),
    # trees: rows below, at and above one row tile (T G = 8, 126, 128, 130, 256, 260, 520)
    (3, 9, 14, 2, 80, 32, [300, 0, 7], [9, 9, 3], "f16", "pairs", "random"),
    (2, 18, 7, 1, 128, 16, [200, 129], [18, 18], "bf16", "tokens", "random"),
    (2, 16, 8, 1, 128, 64, [130, 1000], [16, 15], "bf16", "tokens", "star"),
    (2, 65, 2, 1, 64, 16, [333, 90], [65, 33], "bf16", "heads", "forest"),
    (2, 32, 16, 2, 128, 16, [700, 64], [32, 31], "bf16", "tokens", "random"),
    (1, 26, 20, 2, 96, 16, [513], [26], "bf16", "pairs", "random"),
    (2, 40, 13, 1, 128, 128, [400, 260], [40, 17], "f16", "tokens", "random"),
    # a tree at the largest size, chains longer than a tile, heads of all sizes
    (1, 256, 2, 1, 64, 32, [77], [256], "bf16", "tokens", "random"),
    (2, 200, 4, 2, 128, 256, [10, 700], [200, 131], "bf16", "tokens", None),
    (1, 333, 7, 1, 80, 32, [100], [333], "f16", "tokens", None),
    (2, 5, 4, 1, 256, 16, [600, 31], [5, 4], "bf16", "tokens", "random"),
    (1, 70, 6, 2, 256, 64, [300], [70], "f16", "heads", None),
    (2, 12, 12, 1, 192, 16, [450, 64], [12, 12], "bf16", "pairs", "random"),
    (2, 3, 4, 4, 16, 8, [100, 9], [3, 3], "bf16", "tokens", "random"),
    (2, 4, 3, 1, 48, 1024, [1500, 1023], [4, 2], "f16", "tokens", "random"),
    (1, 2, 128, 1, 112, 16, [260], [2], "bf16", "tokens", "random"),
    # more sequences than SMs, and empty ones among them
    (170, 2, 2, 1, 64, 16, [i % 37 for i in range(170)], [i % 3 for i in range(170)], "bf16", "tokens", "random"),
    # one long sequence: split over many CTAs
    (1, 3, 2, 1, 64, 16, [20011], [3], "bf16", "tokens", "random"),
    (2, 8, 8, 1, 128, 64, [9000, 5], [8, 8], "bf16", "tokens", "random"),
    # more key tiles than SMs: ranges of several tiles and several items
    (24, 3, 16, 8, 128, 16, [(i * 97) % 1500 for i in range(24)], [1 + i % 3 for i in range(24)], "bf16", "tokens",
     "random"),
    (12, 70, 16, 8, 128, 16, [(i * 131) % 1300 for i in range(12)], [70 - i for i in range(12)], "bf16", "heads",
     "random"),
    (20, 4, 16, 8, 64, 32, [(i * 211) % 2100 for i in range(20)], [1 + i % 4 for i in range(20)], "f16", "tokens", None),
    (14, 5, 12, 6, 256, 16, [(i * 173) % 1100 for i in range(14)], [1 + i % 5 for i in range(14)], "bf16", "pairs",
     "random"),
    (6, 150, 8, 8, 80, 8, [(i * 311) % 900 for i in range(6)], [150 - 20 * i for i in range(6)], "f16", "tokens", None),
])
def test_attend(sv, B, T, Hq, Hkv, D, page, ctx, n, dtype, kind, tree):
    from parity_util import report
    rng = np.random.default_rng(B * 7 + T + D)
    worst = _attend_case(sv, rng, B, T, Hq, Hkv, D, page, ctx, n, dtype, kind, tree)
    report(f"attend B={B} T={T} heads {Hq}/{Hkv} D={D} {dtype}: worst error {worst:.2f} of its bound")


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16"), (256, "bf16")])
def test_attend_rows_that_see_nothing(sv, D, dtype):
    """Masks with empty rows (no context), with bits above the node and without
    the node itself; rows beyond n are zero."""
    rng = np.random.default_rng(D)
    B, T = 3, 37
    see = rng.random((B, T, T)) < 0.4
    see[:, ::3] = False
    n = [T, 20, 1]
    for b in range(B):
        see[b, :, n[b]:] = True  # bits of nodes that do not exist change nothing
    _attend_case(sv, rng, B, T, 4, 2, D, 16, [0, 150, 0], n, dtype, see=see)


@pytest.mark.parametrize("D,T,dtype", [(128, 20, "bf16"), (64, 70, "f16"), (256, 20, "bf16")])
def test_attend_non_finite_values(sv, D, T, dtype):
    """NaN and infinities in nodes' keys and values reach the rows that see the
    node, in their columns, and no other row; in the context they reach all."""
    rng = np.random.default_rng(D + T)
    B, page, ctx = 2, 16, [131, 40]

    def touch(q, kc, vc, table):
        def at(b, i):
            return table[b, i // page], i % page
        for b in range(B):
            for node, col, val in ((3, 5, float("nan")), (7, 9, float("inf")), (7, 10, -float("inf")),
                                   (11, D - 1, float("inf"))):
                p, o = at(b, ctx[b] + node)
                vc[p, o, 0, col] = val
            p, o = at(b, ctx[b] + 5)
            kc[p, o, 0] = float("nan")
        p, o = at(1, 17)
        vc[p, o, 1, 3] = float("inf")

    _attend_case(sv, rng, B, T, 4, 2, D, page, ctx, [T, T - 1], dtype, touch=touch, tree="random")
    _attend_case(sv, rng, B, T, 4, 2, D, page, ctx, [T, T - 1], dtype, touch=touch, tree=None)


@pytest.mark.parametrize("std,scale", [(30.0, None), (0.0, None), (1.0, 4.0)])
def test_attend_score_ranges(sv, std, scale):
    """Sharp rows (one key takes all), equal scores, a scale of one's own; the
    running maximum grows along the keys."""
    rng = np.random.default_rng(int(std) + 1)

    def touch(q, kc, vc, table):
        for b in range(2):
            for i in range(0, 600, 50):  # keys ever more like the first query
                kc[table[b, i // 16], i % 16, 0] = (q[b, 0, 0].float() * (i / 600.0)).to(kc.dtype)
    _attend_case(sv, rng, 2, 10, 4, 1, 128, 16, [610, 605], [10, 9], "bf16", std=std, scale=scale, touch=touch)


def test_attend_lengths_out_of_range(sv):
    """Lengths the table cannot hold: zero rows, nothing read."""
    import torch
    rng = np.random.default_rng(3)
    tc = _tc(sv, 4, 4, 4, 2, 64, 16, 8, 2)
    kc, vc = _layout(rng, 8, 16, 2, 64, "bf16", "tokens")
    q = _rand(rng, (4, 4, 4, 64), "bf16")
    table = _i32(np.arange(8).reshape(4, 2))
    got = tc.attend(q, kc, vc, table, _i32([-1, 30, 31, 3]), _i32([2, 2, 2, 5]))
    out, lse = got["out"].float().cpu().numpy(), got["lse"].cpu().numpy()
    assert (out[[0, 2, 3]] == 0).all() and (lse[[0, 2, 3]] == -np.inf).all()
    assert np.isfinite(out[1]).all() and (out[1, :2] != 0).any() and (out[1, 2:] == 0).all()
    torch.cuda.synchronize()
    tc.close()


def test_attend_is_deterministic_and_stream_ordered(sv):
    """The same call gives the same bits, on another stream and in a graph too."""
    import torch
    rng = np.random.default_rng(9)
    B, T, ctx = 3, 11, [3000, 40, 777]
    tc = _tc(sv, B, T, 16, 2, 128, 16, 3 * 190, 190)
    kc, vc = _layout(rng, 570, 16, 2, 128, "bf16", "tokens")
    q = _rand(rng, (B, T, 16, 128), "bf16")
    args = (q, kc, vc, _i32(rng.permutation(570).reshape(3, 190)), _i32(ctx), _i32([11, 7, 9]))
    first = tc.attend(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = tc.attend(*args)
    s.synchronize()
    third = {k: torch.full_like(x, float("nan")) for k, x in first.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tc.attend(*args, out=third)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], second[k]) and torch.equal(first[k], third[k])
    tc.close()


def test_outputs_of_another_stream_take_no_memory_in_use(sv):
    """Outputs of a call with stream= are not put where kernels in flight on the
    current stream still read."""
    import torch
    rng = np.random.default_rng(15)
    B, T, H, D = 2, 300, 16, 128
    tc = _tc(sv, B, T, H, 4, D, 16, 80, 40)
    kc, vc = _layout(rng, 80, 16, 4, D, "bf16", "tokens")
    q, k, v = (_rand(rng, (B, T, h, D), "bf16") for h in (H, 4, 4))
    table, ctx, slots = _i32(np.arange(80).reshape(2, 40)), _i32([300, 5]), _i32(np.full((B, T), -1))
    calls = (lambda s: tc.attend(q, kc, vc, table, ctx, stream=s)["out"],
             lambda s: tc.append(q, k, v, kc, vc, slots, stream=s))
    side, seen = torch.cuda.Stream(), torch.empty_like(q)
    for call in calls:
        first = call(None)
        torch.cuda.synchronize()
        x = torch.full_like(q, 3.0)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # some milliseconds
        torch.add(x, 0, out=seen)
        del x
        second = call(side)
        torch.cuda.synchronize()
        assert (seen == 3.0).all()
        assert torch.equal(first, second)
    tc.close()


def test_stalled_attend_reports_and_recovers(sv):
    import torch
    rng = np.random.default_rng(12)
    tc = _tc(sv, 1, 2, 4, 2, 64, 16, 8, 8)
    kc, vc = _layout(rng, 8, 16, 2, 64, "bf16", "tokens")
    args = (_rand(rng, (1, 2, 4, 64), "bf16"), kc, vc, _i32([np.arange(8)]), _i32([100]), _i32([2]))
    first = tc.attend(*args)
    assert tc.check() == sv.SPEC_OK
    sv.spec_tree_inject_fault(tc.h, sv.SPEC_FAULT_STALL_STREAM)
    tc.attend(*args)
    assert tc.check() == sv.SPEC_ERR_TIMEOUT and tc.check() == sv.SPEC_OK
    second = tc.attend(*args)
    assert tc.check() == sv.SPEC_OK
    assert torch.equal(first["out"], second["out"]) and torch.equal(first["lse"], second["lse"])
    tc.close()


# --------------------------------------------------------------------------- #
# keep                                                                         #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("B,T,Hkv,D,page,layers,kind", [
    (1, 1, 1, 16, 8, 1, "tokens"), (5, 9, 8, 128, 16, 3, "tokens"), (4, 40, 3, 80, 8, 2, "heads"),
    (3, 64, 2, 256, 32, 1, "pairs"), (2, 256, 1, 64, 16, 2, "tokens")])
def test_keep(sv, B, T, Hkv, D, page, layers, kind):
    import torch
    rng = np.random.default_rng(T + D)
    width = -(-(50 + T) // page)
    pages = B * width
    tc = _tc(sv, B, T, Hkv, Hkv, D, page, pages, width)
    made = [_layout(rng, pages, page, Hkv, D, "bf16", kind) for _ in range(layers)]
    if layers == 1:
        kc, vc = made[0]
    elif kind == "heads":
        kc, vc = (torch.stack([m[i].permute(0, 2, 1, 3) for m in made]).permute(0, 1, 3, 2, 4) for i in range(2))
    else:
        kc, vc = (torch.stack([m[i] for m in made]) for i in range(2))
    table = rng.permutation(pages).reshape(B, width)
    ctx, n = rng.integers(0, 50, B), rng.integers(1, T + 1, B)
    path, plen = np.full((B, T), -7), np.zeros(B, int)
    for b in range(B):
        plen[b] = rng.integers(0, n[b] + 1)
        path[b, :plen[b]] = np.sort(rng.choice(n[b], plen[b], replace=False))
    status = np.zeros(B, int)
    if B > 3:
        n[2] = max(n[2], 2)
        path[2, :2], plen[2], status[2] = 1, 2, 6    # not ascending
        plen[3], status[3] = n[3] + 1, 5             # longer than the tree
    if B > 4:
        path[4, 0], plen[4], status[4] = n[4], 1, 6  # a node that does not exist
    want = [x.clone() for x in (kc, vc)]
    for src, dst in zip((kc, vc), want):
        s4, d4 = (x if x.dim() == 5 else x[None] for x in (src, dst))
        for b in range(B):
            for i in range(plen[b] if status[b] == 0 else 0):
                a, z = int(ctx[b] + path[b, i]), int(ctx[b] + i)
                d4[:, table[b, z // page], z % page] = s4[:, table[b, a // page], a % page]
    got = tc.keep(kc, vc, _i32(table), _i32(ctx), _i32(n), _i32(path), _i32(plen))
    torch.cuda.synchronize()
    assert (got["row_status"].cpu().numpy() == status).all()
    assert (got["ctx_len"].cpu().numpy() == ctx + np.where(status == 0, plen, 0)).all()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    tc.close()


# --------------------------------------------------------------------------- #
# the whole cache range, refusals                                              #
# --------------------------------------------------------------------------- #
def test_offsets_beyond_32_bits(sv):
    """Pages whose elements lie past 2^32: append, attend and keep reach them."""
    import torch
    Hkv, D, page, pages = 8, 256, 64, 33000  # 4.3e9 elements each
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 18 GB for the cache")
    rng = np.random.default_rng(1)
    tc = _tc(sv, 1, 8, 8, Hkv, D, page, pages, 4)
    kc, vc = (torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = _tc(sv, 1, 8, 8, Hkv, D, page, 4, 4)
    far, near = np.array([[32999, 32900, 5, 32998]]), np.array([[3, 0, 1, 2]])
    ks, vs = _layout(rng, 4, page, Hkv, D, "bf16", "tokens")
    for a, z in zip(far[0], near[0]):
        kc[a], vc[a] = ks[z], vs[z]
    q, k, v = (_rand(rng, (1, 8, 8, D), "bf16") for _ in range(3))
    ctx, n = 150, _i32([8])
    at = ctx + np.arange(8)
    outs = []
    for t, kk, vv, tab in ((tc, kc, vc, far), (small, ks, vs, near)):
        slot = _i32([tab[0][at // page] * page + at % page])
        qo = t.append(q, k, v, kk, vv, slot, n_tokens=n)
        r = t.attend(qo, kk, vv, _i32(tab), _i32([ctx]), n)
        t.keep(kk, vv, _i32(tab), _i32([ctx]), n, _i32([[0, 2, 5, 7, 0, 0, 0, 0]]), _i32([4]))
        outs.append((r["out"], r["lse"], torch.cat([kk[i] for i in tab[0]]), torch.cat([vv[i] for i in tab[0]])))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    tc.close()
    small.close()


def test_refusals(sv):
    """Wrong shapes, types, devices and alignments are refused on the host."""
    import torch
    B, T, Hq, Hkv, D, page, pages, width = 2, 3, 4, 2, 64, 16, 8, 4
    tc = _tc(sv, B, T, Hq, Hkv, D, page, pages, width)
    rng = np.random.default_rng(0)
    kc, vc = _layout(rng, pages, page, Hkv, D, "bf16", "tokens")
    q, k, v = (_rand(rng, (B, T, h, D), "bf16") for h in (Hq, Hkv, Hkv))
    table, ctx, n = _i32(np.arange(8).reshape(2, 4)), _i32([5, 6]), _i32([3, 3])
    slot = _i32([[5, 6, 7], [70, 71, 72]])
    good = dict(q=q, k_cache=kc, v_cache=vc, block_table=table, ctx_len=ctx, n_tokens=n)
    tc.attend(**good)
    for change in (dict(q=q.float()), dict(q=q[:, :, :2]), dict(q=q.cpu()), dict(k_cache=kc[:4]),
                   dict(v_cache=vc.half()), dict(block_table=table.long()), dict(block_table=table[:, :2]),
                   dict(ctx_len=ctx[:1]), dict(n_tokens=n.float()),
                   dict(tree_mask=torch.zeros(B, T, 2, dtype=torch.int32, device="cuda")),
                   dict(v_cache=vc.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)),
                   dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            tc.attend(**dict(good, **change))
    flat = torch.zeros(B * T * Hq * D + 8, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:1 + B * T * Hq * D].view(B, T, Hq, D)
    wide = torch.zeros(B, T, Hq, D + 4, dtype=torch.bfloat16, device="cuda")[..., :D]
    for bad_q in (odd, wide):
        with pytest.raises(sv.SpecVerifyError) as e:
            tc.attend(**dict(good, q=bad_q))
        assert e.value.code == sv.SPEC_ERR_UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(sv.SpecVerifyError) as e:
            tc.attend(**good, scale=scale)
        assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    cs = torch.zeros(16, 64, device="cuda")
    with pytest.raises(ValueError):
        tc.append(q, k, v, kc, vc, slot, cos_sin=cs)           # no positions
    with pytest.raises(ValueError):
        tc.append(q, k, v[:1], kc, vc, slot)
    with pytest.raises(ValueError):
        tc.append(q, k, v, kc, vc, slot, q_weight=torch.ones(D, device="cuda"))
    for bad in (dict(cos_sin=cs[:, :24].contiguous()), dict(cos_sin=torch.zeros(16, 80, device="cuda"))):
        with pytest.raises(sv.SpecVerifyError) as e:
            tc.append(q, k, v, kc, vc, slot, slot, **bad)
        assert e.value.code == sv.SPEC_ERR_UNSUPPORTED
    with pytest.raises(sv.SpecVerifyError) as e:
        tc.append(q, k, v, kc, vc, slot, eps=-1.0)
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    big = _rand(rng, (B, T + 1, Hq, D), "bf16")
    with pytest.raises(sv.SpecVerifyError) as e:
        tc.attend(**dict(good, q=big))
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    with pytest.raises(sv.SpecVerifyError) as e:
        tc.keep(kc, vc, table, ctx, n, _i32([[0, 1, 2]] * 2), _i32([1, 1]), out=dict(ctx_len=ctx))
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    torch.cuda.synchronize()
    tc.close()
