"""The operators around a verify step: refusals the host makes without a GPU,
and the plain implementations the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest

import tree_ref as ref


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_42_gb300 import build
    path = build.build()
    import speculative_decoding_verification_42_gb300 as sv
    return sv, sv.load_library(path)


GOOD = dict(device=0, max_batch=4, max_tokens=8, q_heads=8, kv_heads=2, head_dim=64, dtype=1,
            page_size=16, num_pages=32, table_width=8)


@pytest.mark.parametrize("change,code", [
    (dict(max_batch=0), 1), (dict(max_tokens=0), 1), (dict(q_heads=0), 1), (dict(kv_heads=0), 1),
    (dict(q_heads=7), 1), (dict(head_dim=0), 1), (dict(num_pages=0), 1), (dict(table_width=0), 1),
    (dict(device=-1), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1),
    (dict(num_pages=1 << 28), 1), (dict(table_width=1 << 28), 1),
    (dict(dtype=0), 2), (dict(head_dim=24), 2), (dict(head_dim=272), 2), (dict(page_size=4), 2),
    (dict(page_size=24), 2), (dict(page_size=2048), 2), (dict(q_heads=258, kv_heads=2), 2)])
def test_create_refuses(lib, change, code):
    sv, L = lib
    h = C.c_void_p()
    cfg = sv.spec_tree_config(**dict(GOOD, **change))
    assert L.spec_tree_create(C.byref(cfg), C.byref(h)) == code
    assert not h.value


def test_null_arguments(lib):
    sv, L = lib
    h = C.c_void_p()
    assert L.spec_tree_create(None, C.byref(h)) == sv.SPEC_ERR_INVALID_ARG
    assert L.spec_tree_create(C.byref(sv.spec_tree_config(**GOOD)), None) == sv.SPEC_ERR_INVALID_ARG
    assert L.spec_tree_destroy(None) == sv.SPEC_ERR_INVALID_ARG
    assert L.spec_tree_check(None, None) == sv.SPEC_ERR_INVALID_ARG
    assert L.spec_tree_inject_fault(None, 0) == sv.SPEC_ERR_INVALID_ARG
    for name, args in (("plan", sv.spec_tree_plan_args), ("append", sv.spec_tree_append_args),
                       ("attend", sv.spec_tree_attend_args), ("keep", sv.spec_tree_keep_args)):
        assert getattr(L, "spec_tree_" + name)(None, C.byref(args()), None) == sv.SPEC_ERR_INVALID_ARG


def test_reference_attention_is_a_softmax():
    """The plain attention against the closed form of two keys, and its rows
    that see nothing."""
    q = np.array([[1.0, 0.0], [0.0, 2.0]])
    k, v = np.eye(2), np.array([[1.0, 5.0], [3.0, -1.0]])
    out, lse, _, _ = ref.attend(q, k, v, np.array([[True, True], [False, False]]), 0.5, "bf16")
    w = 1.0 / (1.0 + np.exp(-0.5))
    assert np.allclose(out[0], w * v[0] + (1 - w) * v[1], atol=1e-15)
    assert np.isclose(lse[0], np.log(np.exp(0.5) + 1.0))
    assert (out[1] == 0).all() and lse[1] == -np.inf


def test_reference_plan_moves_every_page_once():
    """Over random rounds every page is held by one sequence or free, once."""
    rng = np.random.default_rng(5)
    B, T, page, width, N = 7, 5, 8, 6, 30
    table, free = np.full((B, width), -1, np.int32), rng.permutation(N).astype(np.int32)
    held, ring = np.zeros(B, np.int32), (11, 11 + N)
    free = np.roll(free, 11 % N)
    seen = set()
    for _ in range(40):
        ctx, n = rng.integers(-1, width * page, B), rng.integers(0, T + 1, B)
        out = ref.plan(ctx, n, None, held, ring, free, table, page, T)
        held, ring = out["held"], tuple(out["ring"])
        seen |= set(out["row_status"].tolist())
        pages = [int(table[b, i]) for b in range(B) for i in range(held[b])] + \
            [int(free[i % N]) for i in range(*ring)]
        assert sorted(pages) == list(range(N))
    assert seen == {0, 5, 7}


def test_ancestors():
    see, depth = ref.ancestors([-1, 0, 0, 1, -1], 5)
    assert depth.tolist() == [0, 1, 1, 2, 0]
    assert see.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0],
                                        [1, 1, 0, 1, 0], [0, 0, 0, 0, 1]]
    assert ref.pack_mask(see[None])[0, :, 0].tolist() == [1, 3, 5, 11, 16]
