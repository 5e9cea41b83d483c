"""The operators that score rows of logits: refusals the host makes without a
GPU, and the plain implementations the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest

import score_ref as ref


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_42_gb300 import build
    path = build.build()
    import speculative_decoding_verification_42_gb300 as sv
    return sv, sv.load_library(path)


P = 1 << 20  # an address that is never used: every call here is refused on the host, or a no-op


def _rows(sv, ptr=P, seq=0, tok=64):
    return sv.spec_score_rows(ptr, seq, tok)


def _logprobs(sv, **change):
    a = dict(device=0, dtype=1, batch=1, tokens=3, vocab=64, top_n=0, temperature=1.0, logits=_rows(sv), row_status=P)
    a.update(change)
    return sv.spec_score_logprobs_args(**a)


def _distill(sv, **change):
    a = dict(device=0, dtype=1, teacher_dtype=0, batch=1, tokens=3, vocab=64, entries=4, tail=0, temperature=1.0,
             teacher_temperature=1.0, student=_rows(sv), ids=P, teacher=P, row_status=P)
    a.update(change)
    return sv.spec_score_distill_args(**a)


COMMON = [
    (dict(device=-1), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(batch=-1), 1), (dict(tokens=-1), 1),
    (dict(vocab=0), 1), (dict(temperature=0.0), 1), (dict(temperature=float("nan")), 1),
    (dict(temperature=float("inf")), 1), (dict(temperature=1e-39), 1), (dict(row_status=None), 1),
    (dict(row_status=P + 2), 2), (dict(batch=1 << 15, tokens=1 << 14), 2), (dict(dtype=0, vocab=425985), 2),
    (dict(vocab=851969), 2), (dict(batch=0), 0), (dict(tokens=0), 0)]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(top_n=-1), 1), (dict(top_n=2), 1), (dict(top_n=129, top_ids=P, top_logprobs=P), 2), (dict(logprob=P), 1),
    (dict(rank=P), 1), (dict(grad_entropy=P), 1), (dict(ids=P + 1), 2), (dict(entropy=P + 2), 2)])
def test_logprobs_refuses(lib, change, code):
    sv, L = lib
    assert L.spec_score_logprobs(C.byref(_logprobs(sv, **change)), None) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(teacher_dtype=4), 1), (dict(entries=0), 1), (dict(entries=257), 2), (dict(teacher_temperature=0.0), 1),
    (dict(ids=None), 1), (dict(teacher=None), 1), (dict(teacher_lse=P), 1), (dict(grad_loss=P), 1),
    (dict(teacher=P + 2), 2), (dict(loss=P + 1), 2)])
def test_distill_refuses(lib, change, code):
    sv, L = lib
    assert L.spec_score_distill(C.byref(_distill(sv, **change)), None) == code


@pytest.mark.parametrize("logits,grad,shape,code", [
    ((None, 0, 64), None, (1, 3), 1), ((P, -1, 64), None, (2, 3), 1), ((P, 0, -64), None, (1, 3), 1),
    ((P + 1, 0, 64), None, (1, 3), 2), ((P, 1 << 34, 64), None, (2, 3), 2),
    ((P, 192, 64), (P * 2, 0, 64), (2, 3), 1), ((P, 192, 64), (P * 2, 192, 0), (2, 3), 1),
    ((P, 192, 64), (P * 2, 128, 64), (2, 3), 1), ((P, 192, 64), (P * 2, 64, 64), (2, 3), 1),
    ((P, 192, 64), (P * 2, 192, 63), (2, 3), 1), ((P, 192, 64), (P, 256, 64), (2, 3), 1),
    ((P, 192, 64), (P, 64, 128), (2, 3), 1), ((P, 0, 63), (P, 0, 63), (1, 3), 1)])
def test_rows_refused(lib, logits, grad, shape, code):
    """Negative and huge strides, gradients whose rows share elements, and gradients over the logits in another layout."""
    sv, L = lib
    kw = dict(batch=shape[0], tokens=shape[1])
    g = {} if grad is None else dict(grad=_rows(sv, *grad))
    a = _logprobs(sv, logits=_rows(sv, *logits), **kw, **g, **({} if grad is None else dict(grad_entropy=P)))
    assert L.spec_score_logprobs(C.byref(a), None) == code
    assert L.spec_score_distill(C.byref(_distill(sv, student=_rows(sv, *logits), **kw, **g)), None) == code


def test_null_arguments(lib):
    sv, L = lib
    assert L.spec_score_logprobs(None, None) == sv.SPEC_ERR_INVALID_ARG
    assert L.spec_score_distill(None, None) == sv.SPEC_ERR_INVALID_ARG


def test_reference_gradients_are_slopes():
    """The plain gradients against differences in 64 bits: (h^2 / 6) f''' and 2^-53 / h."""
    rng = np.random.default_rng(0)
    V, h = 12, 1e-4
    l = rng.standard_normal(V) * 2
    l[5] = -np.inf
    ids, t = np.array([3, -1, 7, 0]), np.array([0.2, np.nan, -1.0, -0.3])

    def scores(x):
        a, _ = ref.logprobs(x, 2, 1.4, 0, "f32")
        return (0.3 * a["logprob"] - 0.8 * a["entropy"],
                ref.distill(x, ids, t, 1.4, 0.9, False, 0.0, 1.0, "f32")[0]["loss"],
                ref.distill(x, ids, t, 1.4, 0.9, True, 1.5, 1.0, "f32")[0]["loss"])

    g = (ref.logprobs(l, 2, 1.4, 0, "f32", 0.3, -0.8)[0]["grad"],
         ref.distill(l, ids, t, 1.4, 0.9, False, 0.0, 1.0, "f32")[0]["grad"],
         ref.distill(l, ids, t, 1.4, 0.9, True, 1.5, 1.0, "f32")[0]["grad"])
    for v in range(V):
        up, down = l.copy(), l.copy()
        up[v] += h
        down[v] -= h
        for i, (a, b) in enumerate(zip(scores(up), scores(down))):
            assert abs((a - b) / (2 * h) - g[i][v]) < 1e-7


def test_reference_rows():
    """Two tokens: the logistic function; equal logits rank by id; a mask hides a token."""
    r, _ = ref.logprobs(np.array([1.0, 3.0]), 0, 2.0, 2, "f32")
    p = 1 / (1 + np.exp(1.0))
    assert np.isclose(r["logprob"], np.log(p)) and r["rank"] == 1 and r["top_ids"].tolist() == [1, 0]
    assert np.isclose(r["entropy"], -(p * np.log(p) + (1 - p) * np.log(1 - p)))
    r, _ = ref.logprobs(np.array([2.0, -np.inf, 2.0, 2.0]), 2, 1.0, 4, "f32")
    assert r["rank"] == 1 and r["top_ids"].tolist() == [0, 2, 3, -1] and np.isclose(r["entropy"], np.log(3))
    r, _ = ref.logprobs(np.array([2.0, -np.inf, 2.0, -np.inf]), 3, 1.0, 0, "f32")
    assert r["rank"] == 2 and r["logprob"] == -np.inf
    d, _ = ref.distill(np.log(np.array([0.5, 0.2, 0.3])), np.array([1, 0]), np.log(np.array([0.2, 0.5])), 1.0, 1.0, True,
                       0.0, 1.0, "f32")
    assert abs(d["loss"]) < 1e-15 and np.isclose(d["accept"], 0.7) and np.abs(d["grad"]).max() < 1e-15


def test_packed_records_have_the_structures_layout():
    """The wrapper packs its arguments at once: sizes and places are those of the declared structures."""
    import struct
    import speculative_decoding_verification_42_gb300.score as sc
    for cls, packed in ((sc.spec_score_logprobs_args, sc._LOGPROBS_ARGS), (sc.spec_score_distill_args, sc._DISTILL_ARGS)):
        fields = []
        for name, kind in cls._fields_:
            fields += [(name, n) for n, _ in kind._fields_] if kind is sc.spec_score_rows else [(name, None)]
        assert C.sizeof(cls) == packed.size
        values = [i + 1 for i in range(len(fields))]
        rec = cls.from_buffer_copy(packed.pack(*values))
        for (name, sub), v in zip(fields, values):
            got = getattr(rec, name) if sub is None else getattr(getattr(rec, name), sub)
            assert got == v, (name, sub)
    assert struct.calcsize("P") == 8
