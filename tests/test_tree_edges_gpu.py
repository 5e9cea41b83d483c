"""The operators around a verify step where other parts of a program meet them:
page shortages, non-finite values, other streams, layouts that are refused, the
ends of the ranges.  Against the plain 64-bit implementations of tree_ref.py."""
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


def test_a_sequence_without_pages_touches_nothing(sv):
    """Sequence 0 gave two pages back, sequence 1 holds them now, and sequence 0
    finds the ring empty: its table row no longer leads to them, append and keep
    leave the cache alone, and its length stays."""
    import torch
    rng = np.random.default_rng(21)
    B, T, H, D, page, width, N = 2, 4, 2, 64, 8, 3, 4
    tc = _tc(sv, B, T, 2 * H, H, D, page, N, width)
    pool = tc.new_pool(B)
    kc, vc = (_rand(rng, (N, page, H, D), "bf16") for _ in range(2))
    for ctx, n in (([20, 0], [4, 0]), ([5, 0], [0, 0]), ([5, 16], [0, 4])):
        plan = tc.plan(_i32(ctx), _i32(n), pool["held"], pool["ring"], pool["free_pages"], pool["block_table"],
                       max_tokens=T)
        pool["held"], pool["ring"] = plan["held"], plan["ring"]
        assert plan["row_status"].tolist() == [0, 0]
    rows = pool["block_table"].tolist()
    assert sorted(rows[0][:1] + rows[1]) == list(range(N)) and rows[0][1] in rows[1]
    ctx, n = _i32([5, 16]), _i32([4, 4])
    for _ in range(2):  # repeatable
        plan = tc.plan(ctx, n, pool["held"], pool["ring"], pool["free_pages"], pool["block_table"], max_tokens=T)
        assert plan["row_status"].tolist() == [sv.SPEC_ROW_NO_PAGES, 0] and plan["held"].tolist() == [1, 3]
        assert pool["block_table"].tolist() == [[rows[0][0], -1, rows[0][2]], rows[1]]
        assert plan["slot_map"][0].tolist() == [-1] * T
    q, k, v = (_rand(rng, (B, T, h, D), "bf16") for h in (2 * H, H, H))
    before = kc.clone(), vc.clone()
    qo = tc.append(q, k, v, kc, vc, plan["slot_map"], n_tokens=n)
    own = [int(p) for p in rows[1]]
    for x, y in zip((kc, vc), before):
        assert torch.equal(x[rows[0][0]], y[rows[0][0]])
    out = tc.attend(qo, kc, vc, pool["block_table"], ctx, n)["out"]
    alone = _tc(sv, 1, T, 2 * H, H, D, page, N, width)
    assert torch.equal(out[1:], alone.attend(qo[1:], kc, vc, _i32([own]), _i32([16]), _i32([4]))["out"])
    # what the row can still see is its first page; its other keys and values are zeros
    zk, zv = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (kc, vc))
    wide = _tc(sv, 1, T, 2 * H, H, D, page, N + 1, width)
    assert torch.equal(out[:1], wide.attend(qo[:1], zk, zv, _i32([[rows[0][0], N, N]]), _i32([5]), _i32([4]))["out"])
    before = kc.clone(), vc.clone()
    path, plen = _i32([[0, 2, 3, 0], [0, 1, 2, 3]]), _i32([3, 4])
    for status in (plan["row_status"], None):
        got = tc.keep(kc, vc, pool["block_table"], ctx, n, path, plen,
                      **({} if status is None else dict(plan_status=status)))
        assert got["ctx_len"].tolist() == [5, 20] and got["row_status"].tolist() == [sv.SPEC_ROW_NO_PAGES, 0]
        assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    torch.cuda.synchronize()
    for t in (tc, alone, wide):
        t.close()


def test_keep_leaves_what_plan_refused(sv):
    """A status of the plan stops the keep, also where the path would fit a page that the sequence holds."""
    import torch
    rng = np.random.default_rng(22)
    tc = _tc(sv, 4, 4, 1, 1, 32, 8, 8, 2)
    kc, vc = (_rand(rng, (8, 8, 1, 32), "bf16") for _ in range(2))
    before = kc.clone(), vc.clone()
    table, ctx, n = _i32(np.arange(8).reshape(4, 2)), _i32([1, 2, 3, 0]), _i32([4] * 4)
    path, plen, status = _i32([[1, 3, 0, 0]] * 4), _i32([2, 2, 2, 2]), _i32([5, 6, 7, 0])
    got = tc.keep(kc, vc, table, ctx, n, path, plen, plan_status=status)
    assert got["ctx_len"].tolist() == [1, 2, 3, 2] and got["row_status"].tolist() == [5, 6, 7, 0]
    for x, y in zip((kc, vc), before):
        assert torch.equal(x[:6], y[:6]) and torch.equal(x[6, 0], y[6, 1]) and torch.equal(x[6, 1], y[6, 3])
    tc.close()


@pytest.mark.parametrize("D,rot,inter,norm,dtype", [
    (64, 32, True, False, "bf16"), (64, 32, False, False, "bf16"), (80, 16, True, True, "f16"),
    (80, 48, False, True, "f16"), (256, 64, True, False, "f16"), (128, 96, False, False, "bf16")])
def test_append_non_finite_elements(sv, D, rot, inter, norm, dtype):
    """Infinities and NaN reach what the formula says: their pair in the rotated
    part, themselves past it, the whole head through a norm."""
    import torch
    rng = np.random.default_rng(D + rot)
    B, T, Hq, Hkv, page, pages, P = 1, 6, 4, 2, 8, 2, 16
    tc = _tc(sv, B, T, Hq, Hkv, D, page, pages, 2, dtype)
    q, k, v = (_rand(rng, (B, T, h, D), dtype, 2.0) for h in (Hq, Hkv, Hkv))
    inf, nan = float("inf"), float("nan")
    for x in (q, k):
        for j, (e, val) in enumerate(((rot, inf), (rot + 1, -inf), (D - 1, nan), (1, inf), (rot // 2, nan))):
            x[0, j, j % x.shape[2], e] = val
    v[0, 1, 0, 0], v[0, 2, 1, D - 1] = inf, nan
    kc, vc = (_rand(rng, (pages, page, Hkv, D), dtype) for _ in range(2))
    w = (1 + 0.3 * _rand(rng, (D,), dtype)).to(_dt(dtype)) if norm else None
    cs, pos, slot = rng.standard_normal((P, rot)).astype(np.float32), rng.integers(0, P, (B, T)), np.arange(T)[None]
    got = tc.append(q, k, v, kc, vc, _i32(slot), _i32(pos), q_weight=w, k_weight=w,
                    cos_sin=torch.from_numpy(cs).cuda(), interleaved=inter)
    torch.cuda.synchronize()
    u, w64 = ref.UNIT[dtype], ref.to_f64(w) if norm else None
    for j in range(T):
        for x, y in ((q[0, j], got[0, j]), (k[0, j], kc[0, j])):
            with np.errstate(invalid="ignore"):
                want, tol = ref.norm_rotate(ref.to_f64(x), w64, 1e-6, cs.astype(np.float64), int(pos[0, j]), inter)
            y, fin = ref.to_f64(y), np.isfinite(want)
            assert (np.isnan(y) == np.isnan(want)).all(), j
            assert (y[np.isinf(want)] == want[np.isinf(want)]).all(), j
            err = np.abs(y[fin] - want[fin]) - (tol + u * (np.abs(want) + tol) + ref.TINY[dtype])[fin]
            assert not (err > 0).any(), (j, err.max())
    assert torch.equal(vc[0, :T].isnan(), v[0].isnan()) and torch.equal(vc[0, :T].nan_to_num(), v[0].nan_to_num())
    tc.close()


def test_inputs_of_another_stream_may_be_dropped(sv):
    """Tensors given to a call with stream= stay whole until that stream has read
    them, although the caller drops them and allocates anew; the outputs take no
    memory that the current stream still uses."""
    import torch
    rng = np.random.default_rng(25)
    B, T, H, D = 2, 300, 16, 128
    tc = _tc(sv, B, T, H, 4, D, 16, 80, 40)
    kc, vc = (_rand(rng, (80, 16, 4, D), "bf16") for _ in range(2))
    q, k, v = (_rand(rng, (B, T, h, D), "bf16") for h in (H, 4, 4))
    table, ctx, slots = _i32(np.arange(80).reshape(2, 40)), _i32([300, 5]), _i32(np.full((B, T), -1))
    path, plen = _i32(np.arange(T)[None].repeat(B, 0)), _i32([7, 9])
    pool = tc.new_pool(B)
    K, V = 4, 50000
    ver = sv.Verifier(vocab=V, max_batch=8, max_k=K, dtype="bf16")
    target, draft, probs = (_rand(rng, (8, n, V), "bf16", 3.0) for n in (K + 1, K, K))
    drafted = _i32(rng.integers(0, V, (8, K)))
    copy = lambda *ts: [t.clone() for t in ts]  # noqa: E731
    calls = dict(
        attend=lambda s: tc.attend(*copy(q, kc, vc, table, ctx), stream=s)["out"],
        append=lambda s: tc.append(*copy(q, k, v), kc, vc, *copy(slots), stream=s),
        plan=lambda s: tc.plan(*copy(ctx), None, *copy(pool["held"], pool["ring"], pool["free_pages"],
                                                       pool["block_table"]), stream=s)["slot_map"],
        keep=lambda s: tc.keep(kc, vc, *copy(table, ctx), None, *copy(path, plen), stream=s)["ctx_len"],
        run=lambda s: ver.run(*copy(target, draft, drafted), temperature=0.9, top_k=50, stream=s)["target_lse"],
        draft_sample=lambda s: ver.draft_sample(*copy(probs), temperature=0.9, probs=True, stream=s)[1])
    side = torch.cuda.Stream()
    for name, call in calls.items():
        first = call(None)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()  # what the call frees is the only memory of its size
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(60_000_000)  # some 30 ms: the copies are made and dropped meanwhile
        second = call(side)
        over = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in [x.numel() * x.element_size() for x in (q, k, v, kc, vc, table, ctx, slots, path, target, draft,
                                                                 drafted, probs, pool["free_pages"])] * 2]
        torch.cuda.synchronize()
        assert torch.equal(first, second), name
        del over
    tc.close()
    ver.close()


def test_caches_with_shared_elements_are_refused(sv):
    """A stride of 0 where there are several pages, tokens, heads or layers: append and keep write there."""
    import torch
    B, T, H, D, page, pages, layers = 1, 2, 2, 32, 8, 4, 3
    tc = _tc(sv, B, T, H, H, D, page, pages, 2)
    q = torch.zeros(B, T, H, D, dtype=torch.bfloat16, device="cuda")
    table, ctx, n, at = _i32([[0, 1]]), _i32([3]), _i32([2]), _i32([[3, 4]])
    whole = (layers, pages, page, H, D)
    for dim in range(4):
        k, v = (torch.zeros([1 if i == dim else x for i, x in enumerate(whole)], dtype=torch.bfloat16,
                            device="cuda").expand(whole) for _ in range(2))
        calls = [lambda: tc.keep(k, v, table, ctx, n, _i32([[0, 1]]), _i32([2]))]
        if dim:
            calls += [lambda: tc.append(q, q, q, k[0], v[0], at),
                      lambda: tc.attend(q, k[0], v[0], table, ctx, n)]
        for call in calls:
            with pytest.raises(sv.SpecVerifyError) as e:
                call()
            assert e.value.code == sv.SPEC_ERR_UNSUPPORTED
    # inputs may be broadcast: they are only read
    k, v = (torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    one = torch.ones(1, 1, 1, D, dtype=torch.bfloat16, device="cuda").expand(B, T, H, D)
    out = tc.append(one, one, one, k, v, at)
    assert (out == 1).all() and float(k.sum()) == float(v.sum()) == T * H * D and (k[0, 3:5] == 1).all()
    tc.close()


def test_plan_entries_outside_the_cache(sv):
    """A node whose page a table row does not give has no slot, no position and no mask."""
    import torch
    tc = _tc(sv, 2, 4, 2, 1, 32, 8, 4, 2)
    table = _i32([[4, 1], [2, -1]])  # of 4 pages
    parents, ring = _i32([[-1, 0, 0, 1]] * 2), torch.tensor([0, 0], dtype=torch.int64, device="cuda")
    for par in (parents, None):
        got = tc.plan(_i32([6, 6]), _i32([4, 4]), _i32([2, 2]), ring, _i32([0, 0, 0, 0]), table, parents=par,
                      max_tokens=4)
        assert got["row_status"].tolist() == [0, 0]
        assert got["slot_map"].tolist() == [[-1, -1, 8, 9], [22, 23, -1, -1]]
        assert got["positions"].tolist() == ([[-1, -1, 7, 8], [6, 7, -1, -1]] if par is not None else
                                             [[-1, -1, 8, 9], [6, 7, -1, -1]])
        if par is not None:
            assert got["tree_mask"][:, :, 0].tolist() == [[0, 0, 5, 11], [1, 3, 0, 0]]
    tc.close()


@pytest.mark.parametrize("D,T,tree", [(64, 1, False), (128, 3, True), (256, 2, True)])
def test_attend_f16_many_small_probabilities(sv, D, T, tree):
    """Many keys whose probabilities are far below the largest still count: each of 2^-25.5 of it, less
    than the smallest f16.  So many sequences (of the same pages) that most are not cut."""
    import torch
    B, ctx, page = 400, 100000, 64
    pages = ctx // page + 2
    tc = _tc(sv, B, T, 2, 1, D, page, pages, pages, "f16")
    q = torch.zeros(B, T, 2, D, dtype=torch.float16, device="cuda")
    kc, vc = (torch.zeros(pages, page, 1, D, dtype=torch.float16, device="cuda") for _ in range(2))
    q[..., 0] = 4.0
    kc[0, 3, 0, 0] = 25.5 * np.log(2.0) / 4.0
    vc[...] = 1.0
    vc[0, 3] = 0.0
    mask = _i32(ref.pack_mask(np.eye(T, dtype=bool)[None].repeat(B, 0))) if tree else None
    got = tc.attend(q, kc, vc, _i32(np.arange(pages)[None].repeat(B, 0)), _i32([ctx] * B),
                    _i32([T] * B), tree_mask=mask, scale=1.0)
    assert tc.check() == sv.SPEC_OK
    p = np.exp(-4.0 * float(kc[0, 3, 0, 0]))
    N = ctx  # keys but the one: the context's others and the node itself
    z = 1.0 + N * p
    want, lse = N * p / z, 4.0 * float(kc[0, 3, 0, 0]) + np.log(z)
    # each probability rounded to f16 in units of 2^7 of the largest or finer (2^-11 of itself, or half the
    # subnormals' spacing), fp32 sums of N terms in some hundred parts of a thousand, the output's rounding
    u = ref.UNIT["f16"]
    tol = u * want + N * 2.0 ** -25 * 2.0 ** -7 / z + 2.0 ** -13 * want + u * want
    assert float((got["out"].double() - want).abs().max()) <= tol, (float(got["out"].double().min()), want, tol)
    assert float((got["lse"].double() - lse).abs().max()) <= 2.0 ** -17 * abs(lse)
    tc.close()


@pytest.mark.parametrize("D", [64, 256])
def test_attend_f16_largest_probabilities(sv, D):
    """Scores just below the growth that moves the running maximum: the largest probabilities stay finite."""
    rng = np.random.default_rng(D)
    B, ctx, page = 400, 1500, 64
    pages = ctx // page + 2
    tc = _tc(sv, B, 1, 1, 1, D, page, pages, pages, "f16")
    q, kc, vc = (_rand(rng, s, "f16") for s in ((1, 1, 1, D), (pages, page, 1, D), (pages, page, 1, D)))
    q[...] = 0
    q[..., 0] = 1
    kc[...] = 0
    kc[6:, :, 0, 0] = 7.99 * np.log(2.0)  # from the fourth tile of 128 keys on
    got = tc.attend(q.expand(B, 1, 1, D).contiguous(), kc, vc, _i32(np.arange(pages)[None].repeat(B, 0)),
                    _i32([ctx] * B), _i32([1] * B), scale=1.0)
    assert tc.check() == sv.SPEC_OK
    at = np.arange(ctx + 1)
    k, v = (ref.to_f64(x)[at // page, at % page, 0] for x in (kc, vc))
    out, lse, tol, tol_l = ref.attend(ref.to_f64(q)[0, 0], k, v, np.ones((1, ctx + 1), bool), 1.0, "f16")
    assert (np.abs(ref.to_f64(got["out"])[:, 0, 0] - out[0]) <= tol[0]).all()
    assert (np.abs(ref.to_f64(got["lse"])[:, 0, 0] - lse[0]) <= tol_l[0]).all()
    tc.close()


def _parts(ctx, n, G, D, Hkv, sms):
    """How sv_tree_attend.cu cuts a call without many row tiles: (may its first joining form be used, the
    number of parts of every item that is cut)."""
    KT, cost_of = (128 if D <= 128 else 64), 4
    group = (2 if D <= 128 else 1) * (128 // G)
    assert all(x <= group for x in n)
    cost = [-(-(c + x) // KT) + cost_of if x else 0 for c, x in zip(ctx, n)]
    total = sum(cost) * Hkv
    ctas = min(sms, total)
    q, r = total // ctas, total % ctas
    owner = lambda x: x // (q + 1) if x < r * (q + 1) else r + (x - r * (q + 1)) // q  # noqa: E731
    parts, at = [], 0
    for _ in range(Hkv):
        for c in cost:
            if c:
                first, last = owner(at + cost_of), owner(at + c - 1)
                if last > first:
                    parts.append(last - first + 1)
            at += c
    q_rows = -(-min(128 // G, max(n)) * G // 8) * 8
    rows = q_rows * (2 if D <= 128 else 1)
    tasks = len(ctx) * Hkv * (-(-rows // 32)) * (D // 8)
    return tasks > 2 * sms, parts


@pytest.mark.parametrize("Hkv,G,D,dtype,ctx,n", [
    (4, 8, 128, "bf16", [40011], [32]), (4, 8, 128, "f16", [40011, 3000, 2000], [32, 32, 9]),
    (6, 8, 64, "bf16", [30, 50000, 0, 2300], [32, 31, 0, 32]), (8, 4, 256, "f16", [30001, 1700, 1500], [32, 20, 32]),
    (4, 7, 80, "bf16", [1500, 60001, 2900], [36, 33, 35])])
def test_attend_joins_in_both_forms(sv, Hkv, G, D, dtype, ctx, n):
    """Items in many parts and items in few, joined by one launch whose CTAs go
    from tasks of the one form to tasks of the other."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    first_form, parts = _parts(ctx, n, G, D, Hkv, sms)
    assert first_form and max(parts) > 8, parts
    if len(ctx) > 1:
        assert min(parts) <= 8, parts
    rng = np.random.default_rng(D + Hkv)
    B, T, Hq, page = len(ctx), max(n), Hkv * G, 32
    width = -(-(max(ctx) + T) // page)
    pages = sum(-(-(c + x) // page) for c, x in zip(ctx, n))
    tc = _tc(sv, B, T, Hq, Hkv, D, page, pages, width, dtype)
    q, kc, vc = (_rand(rng, s, dtype, 1.3) for s in ((B, T, Hq, D), (pages, page, Hkv, D), (pages, page, Hkv, D)))
    free, table = rng.permutation(pages).tolist(), np.full((B, width), -1, np.int32)
    see = np.zeros((B, T, T), bool)
    par = ref.random_parents(rng, B, T, "random")
    for b in range(B):
        for i in range(-(-(ctx[b] + n[b]) // page)):
            table[b, i] = free.pop()
            # values that change along the context: a part that is lost or taken twice shows
            vc[int(table[b, i])] += 3 * np.cos(6.3 * i * page / (ctx[b] + n[b]))
        see[b] = ref.ancestors(par[b], n[b])[0]
    got = tc.attend(q, kc, vc, _i32(table), _i32(ctx), _i32(n), tree_mask=_i32(ref.pack_mask(see)))
    assert tc.check() == sv.SPEC_OK
    u, scale, worst = ref.UNIT[dtype], D ** -0.5, 0.0
    for b in range(B):
        N = ctx[b] + n[b]
        assert (got["out"][b, n[b]:] == 0).all() and (got["lse"][b, n[b]:] == -np.inf).all()
        if not N or not n[b]:
            continue
        at = np.arange(N)
        pg, off = (torch.from_numpy(x).cuda() for x in (table[b, at // page].astype(np.int64), at % page))
        vis = np.concatenate([np.ones((n[b], ctx[b]), bool), see[b][:n[b], :n[b]]], 1)
        vis = torch.from_numpy(vis).cuda()[:, None, :]
        for hk in range(Hkv):
            k, v = kc[pg, off, hk].double(), vc[pg, off, hk].double()
            x = q[b, :n[b], hk * G:(hk + 1) * G].double()
            s = torch.where(vis, (x @ k.T) * scale, -np.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[..., None])
            want, a = p @ v, p @ v.abs()
            # scores: D-term fp32 sums, the exponent as in tree_ref; sums: 128 keys of a tile, the tiles of a
            # part, the parts: far fewer than 1000 additions one after another; p and the output rounded
            ds = (D + 8) * 2.0 ** -24 * scale * (x.abs() @ k.abs().T).amax(-1, keepdim=True) + 2.0 ** -17
            sums = 1000 * 2.0 ** -24
            tol = (u + 2 * ds + 4 * sums) * a + u * want.abs() * 1.01 + \
                ref.TINY[dtype] * (1 + v.abs().sum(0) * (2.0 ** -7 if dtype == "f16" else 1.0))
            err = (got["out"][b, :n[b], hk * G:(hk + 1) * G].double() - want).abs()
            worst = max(worst, float((err / tol).max()))
            assert (err <= tol).all(), (b, hk, worst)
            el = (got["lse"][b, :n[b], hk * G:(hk + 1) * G].double() - lse).abs()
            assert (el <= ds[..., 0] + sums + 2.0 ** -22 * lse.abs()).all(), (b, hk, float(el.max()))
    tc.close()
    from parity_util import report
    report(f"joins, heads {Hq}/{Hkv} D={D} {dtype}: parts {min(parts)} to {max(parts)}, worst error {worst:.2f} of "
           "its bound")


@pytest.mark.parametrize("D,T", [(16, 1), (256, 2)])
def test_attend_over_almost_two_to_the_31_keys(sv, D, T):
    """The longest context a table may describe (pages may repeat in it), to its last key."""
    import torch
    page, pages, width = 64, 1001, (1 << 25) - 1
    N = page * width
    tc = _tc(sv, 1, T, 1, 1, D, page, pages, width)
    table = (torch.arange(width, device="cuda", dtype=torch.int32) % (pages - 1))[None].contiguous()
    table[0, -1] = pages - 1
    kc, vc = (torch.zeros(pages, page, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    vc[...] = 1.0
    vc[-1] = 2.0 ** 24  # the last page counts for a third
    q = torch.ones(1, T, 1, D, dtype=torch.bfloat16, device="cuda")
    got = tc.attend(q, kc, vc, table, _i32([N - T]), _i32([T]), tree_mask=_i32([[[(1 << T) - 1]] * T]))
    assert tc.check() == sv.SPEC_OK
    want = (N - page + page * 2.0 ** 24) / N
    # probabilities of 1, sums of whole numbers in parts of 2^24 keys, the output's rounding
    assert float((got["out"].double() - want).abs().max()) <= want * (2.0 ** -8 + 2.0 ** -14)
    assert float((got["lse"].double() - np.log(N)).abs().max()) <= 2.0 ** -14
    # a shorter one beside the end of the range: nothing is read past it
    got = tc.attend(q, kc, vc, table, _i32([N - T + 1]), _i32([T]))
    assert (got["out"] == 0).all() and (got["lse"] == -np.inf).all()
    tc.close()


def test_plan_of_a_very_long_chain(sv):
    """More chunks of tokens than a grid's second dimension has CTAs."""
    import torch
    T, page = 68_000_003, 1024
    width = T // page + 2
    tc = _tc(sv, 1, T, 1, 1, 16, page, width, width)
    pool = tc.new_pool(1)
    got = tc.plan(_i32([700]), None, pool["held"], pool["ring"], pool["free_pages"], pool["block_table"])
    assert got["row_status"].tolist() == [0] and got["held"].tolist() == [-(-(T + 700) // page)]
    want = torch.arange(700, 700 + T, dtype=torch.int32, device="cuda")[None]
    assert torch.equal(got["positions"], want) and torch.equal(got["slot_map"], want)
    tc.close()


def test_plan_of_no_tokens_is_refused(sv):
    import torch
    tc = _tc(sv, 2, 4, 2, 1, 32, 8, 4, 2)
    pool = tc.new_pool(2)
    with pytest.raises(sv.SpecVerifyError) as e:
        tc.plan(_i32([0, 0]), None, pool["held"], pool["ring"], pool["free_pages"], pool["block_table"], max_tokens=0)
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    torch.cuda.synchronize()
    tc.close()
