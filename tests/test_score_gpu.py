"""The operators that score rows of logits on the GPU, against the plain 64-bit
implementations of score_ref.py, at the sizes, values and layouts where they can
go wrong.  Bounds come from the roundings the operators make (score_ref.py)."""
import os

import numpy as np
import pytest

import score_ref as ref

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


def _dt(kind):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[kind]


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, want, bound, what):
    got, want, bound = np.asarray(got, np.float64), np.asarray(want, np.float64), np.asarray(bound)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    with np.errstate(invalid="ignore"):
        over = np.where(fine, np.abs(got - want) - bound, -1.0)
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert not over.size or over[at] <= 0, (what, at, got[at], want[at], np.broadcast_to(bound, over.shape)[at])


def _check_logprobs(got, logits, tok, temp, top_n, kind, gl=None, gh=None):
    """Every row of a result against the plain one; logits [N, V] as the kernel saw them."""
    N = len(logits)
    got = {n: (t.reshape(N, -1) if n in ("grad", "top_ids", "top_logprobs") else t.reshape(N)).cpu()
           for n, t in got.items()}
    for r in range(N):
        want, bound = ref.logprobs(logits[r], None if tok is None else int(tok[r]), temp, top_n, kind,
                                   0.0 if gl is None else float(gl[r]), 0.0 if gh is None else float(gh[r]))
        for n, t in got.items():
            if n in ("row_status", "rank", "top_ids"):
                assert np.array_equal(t[r].numpy(), want[n]), (n, r, t[r], want[n])
            else:
                _close(_f64(t[r]), want[n], bound[n], (n, r))


def _check_distill(got, logits, ids, teacher, temp, t_temp, tail, t_lse, w, kind):
    N = len(logits)
    got = {n: (t.reshape(N, -1) if n == "grad" else t.reshape(N)).cpu() for n, t in got.items()}
    for r in range(N):
        want, bound = ref.distill(logits[r], ids[r], teacher[r], temp, t_temp, tail,
                                  0.0 if t_lse is None else float(t_lse[r]), 1.0 if w is None else float(w[r]), kind)
        for n, t in got.items():
            if n == "row_status":
                assert int(t[r]) == want[n], (n, r, t[r], want[n])
            else:
                _close(_f64(t[r]), want[n], bound[n], (n, r))


def _logits(rng, N, V, kind, how="peaks"):
    x = rng.standard_normal((N, V)) * 3
    if how == "peaks":
        for r in range(N):
            x[r, rng.integers(0, V, 20)] += 8
    elif how == "ties":
        x = rng.integers(-2, 3, (N, V)).astype(np.float64)
    elif how == "equal":
        x = np.full((N, V), 1.5)
    elif how == "zeros":  # of both signs: equal values
        x = np.where(rng.random((N, V)) < 0.5, -0.0, 0.0)
    elif how == "masked":  # a grammar leaves few tokens
        x[rng.random((N, V)) > 0.01] = -np.inf
        x[np.arange(N), rng.integers(0, V, N)] = 0.5
    elif how == "block":  # unmasked tokens side by side
        lo = rng.integers(0, max(1, V // 2))
        keep = np.zeros(V, bool)
        keep[lo:lo + max(1, V // 5)] = True
        x[:, ~keep] = -np.inf
    elif how == "one":
        x[:] = -np.inf
        x[np.arange(N), rng.integers(0, V, N)] = -7.0
    elif how == "lowest":  # masks of the type's lowest value
        import torch
        x[rng.random((N, V)) > 0.3] = torch.finfo(_dt(kind)).min
    elif how == "all_lowest":
        import torch
        x[:] = torch.finfo(_dt(kind)).min
        x[:, ::3] = -np.inf
    elif how == "far":  # a far offset
        x = x + 30000.0
    elif how == "steep":
        x = x * 100
    return _dev(x.astype(np.float32), _dt(kind))


SIZES = [("f32", 1), ("bf16", 2), ("f16", 7), ("f32", 31), ("bf16", 255), ("bf16", 1000), ("f16", 4097), ("f32", 4097),
         ("bf16", 32001), ("f32", 32000), ("f16", 50001), ("bf16", 128256), ("f32", 128257), ("bf16", 152064)]


@pytest.mark.parametrize("kind,V", SIZES)
@pytest.mark.parametrize("top_n", [0, 1, 20, 128])
def test_logprobs(sv, kind, V, top_n):
    rng = np.random.default_rng(V + top_n)
    N = 5
    x = _logits(rng, N, V, kind)
    tok = rng.integers(0, V, N)
    tok[-1] = -1
    temp = [1.0, 0.7, 2.5][V % 3]
    got = sv.logprobs(x, _dev(tok.astype(np.int32)), temperature=temp, top_n=top_n, rank=True)
    assert set(got) == {"logprob", "rank", "entropy", "lse", "row_status"} | ({"top_ids", "top_logprobs"} if top_n else set())
    _check_logprobs(got, _f64(x), tok, temp, top_n, kind)


@pytest.mark.parametrize("how", ["ties", "equal", "zeros", "masked", "block", "one", "lowest", "all_lowest", "far", "steep"])
@pytest.mark.parametrize("kind,V", [("bf16", 1003), ("f16", 20000), ("f32", 20001), ("bf16", 128256), ("f32", 66)])
def test_logprobs_of_unusual_rows(sv, kind, V, how):
    rng = np.random.default_rng(V)
    N = 4
    x = _logits(rng, N, V, kind, how)
    tok = rng.integers(0, V, N)
    tok[0] = int(_f64(x)[0].argmax())  # a token that no mask hides
    gl, gh = rng.standard_normal(N), rng.standard_normal(N)
    f = np.float32
    for top_n in (0, 5, 100):
        got = sv.logprobs(x, _dev(tok.astype(np.int32)), top_n=top_n, rank=True)
        _check_logprobs(got, _f64(x), tok, 1.0, top_n, kind)
    got = sv.logprobs(x, _dev(tok.astype(np.int32)), top_n=3, grad_logprob=_dev(gl.astype(f)), grad_entropy=_dev(gh.astype(f)))
    _check_logprobs(got, _f64(x), tok, 1.0, 3, kind, gl.astype(f), gh.astype(f))


@pytest.mark.parametrize("kind,V", [(k, v) for k, v in SIZES if v > 1])
def test_logprobs_gradient(sv, kind, V):
    rng = np.random.default_rng(V)
    N, temp = 4, [1.0, 0.6, 3.0][V % 3]
    x = _logits(rng, N, V, kind)
    tok = rng.integers(0, V, N)
    tok[2] = -1
    gl, gh = (rng.standard_normal(N).astype(np.float32) for _ in range(2))
    toks = _dev(tok.astype(np.int32))
    both = sv.logprobs(x, toks, temperature=temp, grad_logprob=_dev(gl), grad_entropy=_dev(gh))
    _check_logprobs(both, _f64(x), tok, temp, 0, kind, gl, gh)
    _check_logprobs(sv.logprobs(x, toks, temperature=temp, grad_logprob=_dev(gl)), _f64(x), tok, temp, 0, kind, gl)
    alone = sv.logprobs(x, temperature=temp, grad_entropy=_dev(gh))
    _check_logprobs(alone, _f64(x), None, temp, 0, kind, None, gh)


@pytest.mark.parametrize("kind,V", [("bf16", 13), ("f32", 13), ("bf16", 5003), ("f32", 40001)])
@pytest.mark.parametrize("temp", [1.46, 3.0, 40.0])
def test_entropy_gradient_of_masks_of_the_lowest_value(sv, kind, V, temp):
    """The distance of such a token over the temperature is in range, its product with an upstream gradient is not."""
    rng = np.random.default_rng(V)
    N, temp = 6, float(np.float32(temp))
    x = _logits(rng, N, V, kind, "lowest")
    tok = rng.integers(0, V, N)
    gh = np.array([2.9, -7, 300, -1e4, 1e6, 0.1], np.float32)
    gl = np.array([0, 1, -2, 0, 5, 1], np.float32)
    got = sv.logprobs(x, _dev(tok.astype(np.int32)), temperature=temp, grad_logprob=_dev(gl), grad_entropy=_dev(gh))
    assert not got["grad"].isnan().any()
    _check_logprobs(got, _f64(x), tok, temp, 0, kind, gl, gh)


def test_logprobs_without_tokens_and_row_statuses(sv):
    import torch
    rng = np.random.default_rng(3)
    V = 777
    for kind in ("f32", "bf16", "f16"):
        x = _logits(rng, 8, V, kind)
        x[1, 5] = float("nan")
        x[2, V - 1] = float("inf")
        x[3] = float("-inf")
        x[4, 0] = float("nan")  # not scored: not read
        tok = np.array([4, 3, 2, 1, -1, V, -2, 2 ** 31 - 1])
        ones = torch.ones(8, device="cuda")
        got = sv.logprobs(x, _dev(tok.astype(np.int32)), top_n=4, rank=True, grad_logprob=ones, grad_entropy=ones)
        assert got["row_status"].tolist() == [0, 3, 3, 3, 0, 1, 1, 1]
        _check_logprobs(got, _f64(x), tok, 1.0, 4, kind, np.ones(8), np.ones(8))
        got = sv.logprobs(x, top_n=4)
        assert got["row_status"].tolist() == [0, 3, 3, 3, 3, 0, 0, 0] and "logprob" not in got
        _check_logprobs(got, _f64(x), None, 1.0, 4, kind)


def _layout(x, how):
    """The values of x [B, T, V] in another layout."""
    import torch
    B, T, V = x.shape
    if how == "shifted":      # next-token positions of a batch
        big = torch.zeros(B, T + 1, V, dtype=x.dtype, device=x.device)
        big[:, :T] = x
        return big[:, :-1]
    if how == "transposed":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    if how == "padded":       # rows behind another matrix's, on an odd element
        big = torch.full((B, T, V + 13), float("nan"), dtype=x.dtype, device=x.device)
        big[..., 5:5 + V] = x
        return big[..., 5:5 + V]
    if how == "offset":
        big = torch.full((B * T * V + 3,), float("nan"), dtype=x.dtype, device=x.device)
        big[3:] = x.flatten()
        return big[3:].view(B, T, V)
    return x


@pytest.mark.parametrize("how", ["contiguous", "shifted", "transposed", "padded", "offset"])
@pytest.mark.parametrize("kind,V", [("bf16", 1000), ("f16", 9999), ("f32", 4099), ("bf16", 70001), ("f32", 60000)])
def test_layouts(sv, kind, V, how):
    import torch
    rng = np.random.default_rng(V)
    B, T, k = 2, 3, 9
    x = _layout(_logits(rng, B * T, V, kind).view(B, T, V), how)
    flat = _f64(x).reshape(B * T, V)
    tok = rng.integers(0, V, (B, T))
    gl, gh = (rng.standard_normal((B, T)).astype(np.float32) for _ in range(2))
    args = (x, _dev(tok.astype(np.int32)))
    kw = dict(temperature=0.9, top_n=6, rank=True, grad_logprob=_dev(gl), grad_entropy=_dev(gh))
    got = sv.logprobs(*args, **kw)
    assert got["grad"].is_contiguous() and got["top_ids"].shape == (B, T, 6) and got["lse"].shape == (B, T)
    _check_logprobs(got, flat, tok.ravel(), 0.9, 6, kind, gl.ravel(), gh.ravel())
    # a gradient of another layout than the logits', and one over them: the same values, nothing beside them
    for other in ("padded", "transposed", "offset"):
        g = _layout(torch.zeros(B, T, V, dtype=x.dtype, device="cuda"), other)
        sv.logprobs(*args, **kw, out={"grad": g})
        assert torch.equal(g, got["grad"])
        if other == "padded":
            whole = torch.as_strided(g, (B, T, V + 13), (T * (V + 13), V + 13, 1), g.storage_offset() - 5)
            assert int(whole.isnan().sum()) == B * T * 13
    ids = np.stack([rng.permutation(V)[:k] for _ in range(B * T)]).reshape(B, T, k).astype(np.int32)
    t = rng.standard_normal((B, T, k)).astype(np.float32) - 3
    dargs = (x, _dev(ids), _dev(t))
    dkw = dict(temperature=0.9, teacher_temperature=1.0, tail=True, grad_loss=_dev(gl))
    dgot = sv.distill(*dargs, **dkw)
    _check_distill(dgot, flat, ids.reshape(-1, k), t.reshape(-1, k).astype(np.float64), 0.9, 1.0, True, None,
                   gl.ravel(), kind)
    mine = _layout(x.clone(), how)
    over = sv.distill(mine, *dargs[1:], **dkw, out={"grad": mine})
    assert over["grad"] is mine
    for n in dgot:
        assert torch.equal(over[n], dgot[n]), n
    mine = _layout(x.clone(), how)
    over = sv.logprobs(mine, args[1], **kw, out={"grad": mine})
    for n in got:
        assert torch.equal(over[n], got[n]), n


def test_broadcast_rows_and_one_row_forms(sv):
    import torch
    rng = np.random.default_rng(9)
    V = 5003
    x = _logits(rng, 1, V, "bf16")
    tok = rng.integers(0, V, 6)
    wide = x.expand(6, V)
    got = sv.logprobs(wide, _dev(tok.astype(np.int32)), rank=True, grad_logprob=torch.ones(6, device="cuda"))
    assert got["grad"].shape == (6, V)
    _check_logprobs(got, np.repeat(_f64(x), 6, 0), tok, 1.0, 0, "bf16", np.ones(6))
    with pytest.raises(sv.SpecVerifyError):
        sv.logprobs(wide, _dev(tok.astype(np.int32)), grad_logprob=torch.ones(6, device="cuda"), out={"grad": wide})
    one = sv.logprobs(x[:, None], _dev(tok[:1, None].astype(np.int32)))
    assert one["logprob"].shape == (1, 1) and float(one["logprob"]) == float(got["logprob"][0])
    for shape in ((0, V), (3, 0, V), (0, 4, V)):
        e = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        t = torch.empty(shape[:-1], dtype=torch.int32, device="cuda")
        w = torch.empty(shape[:-1], device="cuda")
        got = sv.logprobs(e, t, top_n=3, rank=True, grad_logprob=w)
        assert got["grad"].shape == shape and got["top_ids"].shape == (*shape[:-1], 3)
        ids = torch.empty(*shape[:-1], 4, dtype=torch.int32, device="cuda")
        got = sv.distill(e, ids, ids.float(), grad_loss=w)
        assert got["loss"].shape == shape[:-1] and got["grad"].shape == shape


def _teacher(rng, logits, k, kind):
    """Entries of a teacher near the student: ids in no order, and values."""
    N, V = logits.shape
    t = logits + rng.standard_normal((N, V))
    ids = np.argsort(-t, -1)[:, :k]
    ids = np.stack([rng.permutation(i) for i in ids]).astype(np.int32)
    v = np.take_along_axis(t, ids.astype(np.int64), -1)
    m = t.max(-1)
    lse = (m + np.log(np.exp(t - m[:, None]).sum(-1))).astype(np.float32)
    return ids, _dev(v.astype(np.float32), _dt(kind)), lse


@pytest.mark.parametrize("kind,V", SIZES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("k,t_kind", [(1, "f32"), (20, "bf16"), (129, "f16"), (256, "f32")])
def test_distill(sv, kind, V, tail, k, t_kind):
    rng = np.random.default_rng(V + k)
    N, k = 4, min(k, V)
    x = _logits(rng, N, V, kind)
    ids, t, lse = _teacher(rng, _f64(x), k, t_kind)
    ids[2] = -1
    w = rng.standard_normal(N).astype(np.float32)
    temp = [1.0, 0.7, 2.0][V % 3]
    args = (x, _dev(ids), t)
    kw = dict(temperature=temp, teacher_temperature=1.0, tail=tail, teacher_lse=_dev(lse) if tail else None)
    only = sv.distill(*args, **kw)
    assert set(only) == {"loss", "accept", "row_status"}
    got = sv.distill(*args, **kw, grad_loss=_dev(w))
    _check_distill(got, _f64(x), ids, _f64(t), temp, 1.0, tail, lse, w, kind)
    # the forward pass alone adds in another order: each form is held to the formula, not to the other's last bit
    _check_distill(only, _f64(x), ids, _f64(t), temp, 1.0, tail, lse, w, kind)


@pytest.mark.parametrize("how", ["ties", "equal", "masked", "block", "one", "lowest", "all_lowest", "far", "steep"])
@pytest.mark.parametrize("kind,V", [("bf16", 1003), ("f32", 20001), ("f16", 66), ("bf16", 128256)])
def test_distill_of_unusual_rows(sv, kind, V, how):
    """Masked student tokens among the teacher's, tails without mass."""
    rng = np.random.default_rng(V)
    N, k = 4, 11
    x = _logits(rng, N, V, kind, how)
    ids = np.stack([rng.permutation(V)[:k] for _ in range(N)]).astype(np.int32)
    lx = _f64(x)
    ids[0, 0] = lx[0].argmax()
    ids[0, 1:] = [v for v in ids[0, 1:] if v != ids[0, 0]][:k - 1] + [-1] * int((ids[0, 1:] == ids[0, 0]).sum())
    seen = np.argsort(-lx[1], kind="stable")[:k]
    ids[1] = seen  # with few unmasked tokens, all of them: nothing is left for the tail
    t = (rng.standard_normal((N, k)) - 3).astype(np.float32)
    t[3, 4] = -np.inf
    w = rng.standard_normal(N).astype(np.float32)
    for tail in (False, True):
        got = sv.distill(x, _dev(ids), _dev(t), tail=tail, grad_loss=_dev(w))
        _check_distill(got, lx, ids, t.astype(np.float64), 1.0, 1.0, tail, None, w, kind)
        assert not got["grad"].isnan().any()


def test_distill_row_statuses(sv):
    import torch
    rng = np.random.default_rng(4)
    V, k, N = 500, 6, 13
    for kind in ("f32", "bf16"):
        x = _logits(rng, N, V, kind)
        ids, t, lse = _teacher(rng, _f64(x), k, "f32")
        t = t.cpu().numpy()
        ids[0, 3] = ids[0, 1]                      # a token twice
        ids[1, 5] = V
        ids[2, 0] = -2
        ids[3, 2], t[3, 2] = -1, np.nan            # no entry: its value does not count
        t[4, 0] = np.nan
        t[5, 1] = np.inf
        x[6, 7] = float("nan")
        x[7, 7] = float("inf")
        x[8] = float("-inf")
        ids[9], x[9] = -1, float("nan")            # no entries: not read
        t[10] = -np.inf                            # without tail no finite value
        ids[11, 1:] = -1
        lse[12] = np.inf
        for tail in (False, True):
            got = sv.distill(x, _dev(ids), _dev(t), tail=tail, teacher_lse=_dev(lse) if tail else None,
                             grad_loss=torch.ones(N, device="cuda"))
            assert got["row_status"].tolist() == [1, 1, 1, 0, 3, 3, 3, 3, 3, 0, 0 if tail else 3, 0, 3 if tail else 0]
            _check_distill(got, _f64(x), ids, t.astype(np.float64), 1.0, 1.0, tail, lse if tail else None,
                           None, kind)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_is_the_slope(sv, tail):
    """Differences of the loss in 32 bits: of h^2 / 6 times a third derivative (below 1) and
    of the loss's rounding over h."""
    import torch
    rng = np.random.default_rng(5)
    V, k, h = 40, 5, 2.0 ** -5
    x = _logits(rng, 1, V, "f32", "plain")
    ids, t, lse = _teacher(rng, _f64(x), k, "f32")
    kw = dict(temperature=1.3, teacher_temperature=1.0, tail=tail, teacher_lse=_dev(lse) if tail else None)
    n = 2 * V
    rows = x.expand(n, V).clone()
    rows[torch.arange(V), torch.arange(V)] += h
    rows[V + torch.arange(V), torch.arange(V)] -= h
    ids_n, t_n = _dev(ids).expand(n, k).contiguous(), t.expand(n, k).contiguous()
    if tail:
        kw["teacher_lse"] = kw["teacher_lse"].expand(n).contiguous()
    loss = sv.distill(rows, ids_n, t_n, **kw)["loss"].double()
    slope = (loss[:V] - loss[V:]) / (2 * h)
    if tail:
        kw["teacher_lse"] = kw["teacher_lse"][:1]
    got = sv.distill(x, _dev(ids), t, **kw, grad_loss=torch.ones(1, device="cuda"))
    assert float((slope - got["grad"][0].double()).abs().max()) < h * h / 6 + 40 * ref.U * (1 + float(loss.max())) / h


def test_logprobs_gradient_is_the_slope(sv):
    import torch
    rng = np.random.default_rng(6)
    V, h, temp = 33, 2.0 ** -5, 1.3
    x = _logits(rng, 1, V, "f32", "plain")
    n = 2 * V
    rows = x.expand(n, V).clone()
    rows[torch.arange(V), torch.arange(V)] += h
    rows[V + torch.arange(V), torch.arange(V)] -= h
    tok = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    got = sv.logprobs(rows, tok, temperature=temp)
    f = 0.7 * got["logprob"].double() - 0.4 * got["entropy"].double()
    slope = (f[:V] - f[V:]) / (2 * h)
    g = sv.logprobs(x, tok[:1], temperature=temp, grad_logprob=torch.full((1,), 0.7, device="cuda"),
                    grad_entropy=torch.full((1,), -0.4, device="cuda"))["grad"][0].double()
    # the third derivative of ln p and of H over a logit is below 4 for entropies below 3
    assert float(got["entropy"].max()) < 3
    assert float((slope - g).abs().max()) < 4 * h * h / 6 + 40 * ref.U * 8 / h


@pytest.mark.parametrize("kind,V", [("bf16", 128256), ("f32", 30000), ("f16", 777)])
def test_repeatable_on_any_stream_and_captured(sv, kind, V):
    """The same bits on two streams at once, and from a graph replayed on new values."""
    import torch
    rng = np.random.default_rng(V)
    N, k = 40, 30
    xs = [_logits(rng, N, V, kind) for _ in range(2)]
    tok = _dev(rng.integers(0, V, N).astype(np.int32))
    ids, t, _ = _teacher(rng, _f64(xs[0]), k, "f32")
    ids = _dev(ids)
    ones = torch.ones(N, device="cuda")

    def both(x, stream=None):
        return {**sv.logprobs(x, tok, top_n=20, rank=True, grad_logprob=ones, grad_entropy=ones, stream=stream),
                **{"d" + n: y for n, y in sv.distill(x, ids, t, grad_loss=ones, stream=stream).items()}}

    want = [{n: y.clone() for n, y in both(x).items()} for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[both(xs[i], s) for _ in range(3)] for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for n in want[i]:
                assert torch.equal(g[n], want[i][n]), n
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(x)
    for i in (1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        for n in want[i]:
            assert torch.equal(held[n], want[i][n]), n


def test_first_calls_of_a_process_may_be_captured(sv):
    import subprocess
    import sys
    code = """
import torch
import speculative_decoding_verification_42_gb300 as sv
x = torch.randn(6, 5000, device="cuda")
tok, w = torch.arange(6, device="cuda", dtype=torch.int32), torch.ones(6, device="cuda")
def calls():
    a = sv.logprobs(x, tok, top_n=4, rank=True, grad_logprob=w, grad_entropy=w)
    return {**a, **sv.distill(x, a["top_ids"], a["top_logprobs"], tail=True, grad_loss=w)}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = calls()
graph.replay()
torch.cuda.synchronize()
now = calls()
assert all(torch.equal(held[n], now[n]) for n in now)
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.stdout.strip() == "ok", r.stderr[-2000:]


def test_rows_beyond_two_to_the_31(sv):
    """Offsets of more than 32 bits, in elements and in bytes."""
    import torch
    V, step = 1001, 2 ** 31 + 24
    big = torch.empty(step + V, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(8)
    x = torch.as_strided(big, (2, 1, V), (step, V, 1))
    x.copy_(_logits(rng, 2, V, "bf16").view(2, 1, V))
    tok = rng.integers(0, V, 2)
    ones = torch.ones(2, 1, device="cuda")
    got = sv.logprobs(x, _dev(tok[:, None].astype(np.int32)), top_n=3, rank=True, grad_logprob=ones)
    flat = _f64(x).reshape(2, V)
    _check_logprobs(got, flat, tok, 1.0, 3, "bf16", np.ones(2))
    over = sv.logprobs(x, _dev(tok[:, None].astype(np.int32)), grad_logprob=ones, out={"grad": x})
    assert torch.equal(over["grad"].contiguous(), got["grad"])
    del big, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind,V", [("f32", 425984), ("bf16", 851968)])
def test_the_largest_vocabulary(sv, kind, V):
    import torch
    rng = np.random.default_rng(V)
    N = 3
    x = _logits(rng, N, V, kind)
    tok = rng.integers(0, V, N)
    ones = np.ones(N, np.float32)
    got = sv.logprobs(x, _dev(tok.astype(np.int32)), top_n=128, rank=True, grad_logprob=_dev(ones), grad_entropy=_dev(ones))
    _check_logprobs(got, _f64(x), tok, 1.0, 128, kind, ones, ones)
    ids, t, lse = _teacher(rng, _f64(x), 256, "f32")
    got = sv.distill(x, _dev(ids), t, tail=True, teacher_lse=_dev(lse), grad_loss=_dev(ones))
    _check_distill(got, _f64(x), ids, _f64(t), 1.0, 1.0, True, lse, ones, kind)
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.logprobs(torch.zeros(1, V + 1, dtype=x.dtype, device="cuda"))
    assert e.value.code == sv.SPEC_ERR_UNSUPPORTED


def test_refusals(sv):
    import torch
    V = 64
    x = torch.zeros(2, 3, V, dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    w = torch.ones(2, 3, device="cuda")
    ids = torch.zeros(2, 3, 4, dtype=torch.int32, device="cuda")
    val = torch.zeros(2, 3, 4, device="cuda")
    bad = [
        (ValueError, lambda: sv.logprobs(x[0, 0], tok[0, 0])), (ValueError, lambda: sv.logprobs(x.cpu(), tok.cpu())),
        (TypeError, lambda: sv.logprobs(x.double(), tok)), (ValueError, lambda: sv.logprobs(x, tok.long())),
        (ValueError, lambda: sv.logprobs(x, tok[:, :2])), (ValueError, lambda: sv.logprobs(x.transpose(1, 2), tok)),
        (ValueError, lambda: sv.logprobs(x, rank=True)), (ValueError, lambda: sv.logprobs(x, grad_logprob=w)),
        (ValueError, lambda: sv.logprobs(x, tok, grad_logprob=w.bfloat16())),
        (ValueError, lambda: sv.logprobs(x, tok, grad_logprob=w, out={"grad": x.float()})),
        (ValueError, lambda: sv.logprobs(x, tok, out={"lse": w.double()})),
        (ValueError, lambda: sv.logprobs(x, tok.cpu())),
        (ValueError, lambda: sv.distill(x, ids[..., :2], val)), (TypeError, lambda: sv.distill(x, ids, val.int())),
        (ValueError, lambda: sv.distill(x, ids, val[..., ::2])), (ValueError, lambda: sv.distill(x, ids, val, grad_loss=w[0])),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
    refused = [
        (1, lambda: sv.logprobs(x, tok, temperature=0.0)), (1, lambda: sv.logprobs(x, tok, temperature=float("nan"))),
        (1, lambda: sv.logprobs(x, tok, temperature=-1.0)), (1, lambda: sv.logprobs(x, tok, temperature=float("inf"))),
        (1, lambda: sv.logprobs(x, tok, top_n=-1)), (2, lambda: sv.logprobs(x, tok, top_n=129)),
        (1, lambda: sv.logprobs(x[..., :0], tok)),
        (1, lambda: sv.distill(x, ids[..., :0], val[..., :0])), (1, lambda: sv.distill(x, ids, val, teacher_lse=w)),
        (1, lambda: sv.distill(x, ids, val, teacher_temperature=0.0)),
        (2, lambda: sv.distill(x, ids.repeat(1, 1, 65), val.repeat(1, 1, 65))),
        (1, lambda: sv.distill(x, ids, val, grad_loss=w, out={"grad": x[:, :1].expand(2, 3, V)})),
    ]
    for code, call in refused:
        with pytest.raises(sv.SpecVerifyError) as e:
            call()
        assert e.value.code == code
    torch.cuda.synchronize()


def test_numbers_out_of_range(sv):
    """Numbers that a record of the library cannot hold are refused like its other bad ones, before anything is
    allocated for them."""
    import torch
    x = torch.zeros(2, 8, device="cuda")
    ids, val = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for code, call in [
        (1, lambda: sv.logprobs(x, temperature=1e300)), (1, lambda: sv.distill(x, ids, val, temperature=1e300)),
        (1, lambda: sv.distill(x, ids, val, teacher_temperature=-1e39)),
        (2, lambda: sv.logprobs(x, top_n=2 ** 40)), (1, lambda: sv.logprobs(x, top_n=-2 ** 40)),
    ]:
        with pytest.raises(sv.SpecVerifyError) as e:
            call()
        assert e.value.code == code
    for call in (lambda: sv.logprobs(x[:1].expand(2 ** 33, 8)),
                 lambda: sv.distill(x[:1].expand(2 ** 33, 8), ids[:1].expand(2 ** 33, 1), val[:1].expand(2 ** 33, 1))):
        with pytest.raises(ValueError):
            call()
    assert torch.cuda.max_memory_allocated() - before < 2 ** 20  # a few results of two rows


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("temp", [0.8, 0.25])
def test_distill_losses_next_to_the_end_of_fp32(sv, kind, temp):
    """Entries on tokens masked with the type's lowest value: their distance over the temperature is beyond fp32, the
    teacher's small share of it is not."""
    import torch
    rng = np.random.default_rng(6)
    N, V, k = 3, 500, 2
    x = _logits(rng, N, V, kind)
    ids = np.stack([rng.permutation(V)[:k] for _ in range(N)]).astype(np.int32)
    for r in range(N):
        x[r, ids[r].tolist()] = torch.finfo(x.dtype).min
    t = (rng.standard_normal((N, k)) * 0.1 - 5).astype(np.float32)
    got = sv.distill(x, _dev(ids), _dev(t), temperature=temp, teacher_temperature=1.0, tail=True)
    assert got["loss"].isfinite().all() and (got["loss"] > 1e36).all()
    _check_distill(got, _f64(x), ids, t.astype(np.float64), float(np.float32(temp)), 1.0, True, None, None, kind)


def test_verify_then_score_then_distill(sv):
    """The operators as they are used together: a verify step with the log probabilities of
    what it emitted, the target's top logits recorded, and the draft's loss against them, whose
    accept is the verify step's alpha under the same knobs."""
    import torch
    rng = np.random.default_rng(11)
    B, K, V, k, temp = 6, 4, 4001, 50, 0.8
    target = _logits(rng, B * (K + 1), V, "f32").view(B, K + 1, V)
    draft = (target[:, :K] + 0.7 * _logits(rng, B * K, V, "f32", "plain").view(B, K, V) / 3).contiguous()
    kpr = torch.tensor([4, 3, 0, 4, 1, 4], dtype=torch.int32, device="cuda")
    ver = sv.Verifier(vocab=V, max_batch=B, max_k=K, dtype="f32")
    x = ver.draft_sample(draft, kpr, temperature=temp, seed=3)
    out = ver.run(target, draft, x, kpr, temperature=temp, seed=3, logprobs=5)
    score = out["logprobs"]
    _check_logprobs(score, _f64(target).reshape(-1, V), out["tokens"].flatten().cpu().numpy(), 1.0, 5, "f32")
    assert (score["logprob"][out["tokens"] < 0] == 0).all()
    with pytest.raises(ValueError):
        ver.run(target, draft, x, kpr, w_vocab=target, logprobs=5)
    top = sv.logprobs(target[:, :K], temperature=temp, top_n=k)
    loss = sv.distill(draft, top["top_ids"], top["top_logprobs"], temperature=temp, teacher_temperature=1.0,
                      tail=True, grad_loss=torch.ones(B, K, device="cuda"))
    _check_distill(loss, _f64(draft).reshape(-1, V), top["top_ids"].cpu().numpy().reshape(-1, k),
                   _f64(top["top_logprobs"]).reshape(-1, k), temp, 1.0, True, None, None, "f32")
    # with top-k on the target alone (its rows masked to their top k) alpha is the sum of min(q, p)
    masked = torch.full_like(target, float("-inf"))
    ids = sv.logprobs(target, top_n=k)["top_ids"].long()
    masked.scatter_(-1, ids, target.gather(-1, ids))
    alpha = ver.run(masked, draft, x, kpr, temperature=temp, seed=3, alpha=True)["alpha"]
    sharp = sv.distill(draft, ids[:, :K].int().contiguous(), target.gather(-1, ids)[:, :K].contiguous(), temperature=temp)
    live = torch.arange(K, device="cuda")[None] < kpr[:, None]
    assert float((alpha - sharp["accept"])[live].abs().max()) < 2e-5  # alpha is held to 1e-5, accept below that
    ver.close()
