"""Binding of include/spec_tree.h: the operators around a verify step.

The C entry points under their own names (argument marshalling only), and
``TreeCache``, which takes torch tensors.  Every step runs in the library's
CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes as C

SPEC_F16 = 2
SPEC_ROW_BAD_LEN, SPEC_ROW_BAD_TREE, SPEC_ROW_NO_PAGES = 5, 6, 7
SPEC_TREE_MAX_NODES = 256

TREE_FUNCTIONS = ("spec_tree_create", "spec_tree_destroy", "spec_tree_check",
                  "spec_tree_inject_fault", "spec_tree_plan", "spec_tree_append",
                  "spec_tree_attend", "spec_tree_keep")


class spec_tree_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("device", "max_batch", "max_tokens", "q_heads", "kv_heads",
                                         "head_dim", "dtype", "page_size", "num_pages",
                                         "table_width")]


class spec_tree_plan_args(C.Structure):
    _fields_ = [("ctx_len", C.c_void_p), ("n_tokens", C.c_void_p), ("parents", C.c_void_p),
                ("held", C.c_void_p), ("ring", C.c_void_p), ("free_pages", C.c_void_p),
                ("block_table", C.c_void_p), ("batch", C.c_int32), ("tokens", C.c_int32),
                ("held_out", C.c_void_p), ("ring_out", C.c_void_p), ("slot_map", C.c_void_p),
                ("positions", C.c_void_p), ("tree_mask", C.c_void_p), ("row_status", C.c_void_p)]


class spec_tree_rows(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("seq_stride", C.c_int64), ("token_stride", C.c_int64),
                ("head_stride", C.c_int64)]


class spec_tree_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64),
                ("token_stride", C.c_int64), ("head_stride", C.c_int64),
                ("layer_stride", C.c_int64), ("layers", C.c_int32)]


class spec_tree_append_args(C.Structure):
    _fields_ = [("q", spec_tree_rows), ("k", spec_tree_rows), ("v", spec_tree_rows),
                ("cache", spec_tree_cache), ("slot_map", C.c_void_p), ("positions", C.c_void_p),
                ("n_tokens", C.c_void_p), ("q_weight", C.c_void_p), ("k_weight", C.c_void_p),
                ("cos_sin", C.c_void_p), ("table_len", C.c_int32), ("rot_dim", C.c_int32),
                ("interleaved", C.c_int32), ("eps", C.c_float), ("batch", C.c_int32),
                ("tokens", C.c_int32), ("q_out", C.c_void_p)]


class spec_tree_attend_args(C.Structure):
    _fields_ = [("q", spec_tree_rows), ("cache", spec_tree_cache), ("block_table", C.c_void_p),
                ("ctx_len", C.c_void_p), ("n_tokens", C.c_void_p), ("tree_mask", C.c_void_p),
                ("scale", C.c_float), ("batch", C.c_int32), ("tokens", C.c_int32),
                ("out", C.c_void_p), ("lse", C.c_void_p)]


class spec_tree_keep_args(C.Structure):
    _fields_ = [("cache", spec_tree_cache), ("block_table", C.c_void_p), ("ctx_len", C.c_void_p),
                ("n_tokens", C.c_void_p), ("path", C.c_void_p), ("path_len", C.c_void_p),
                ("batch", C.c_int32), ("tokens", C.c_int32), ("ctx_out", C.c_void_p),
                ("row_status", C.c_void_p), ("plan_status", C.c_void_p)]


def bind(L: C.CDLL) -> None:
    """Declare the argument types of this header's functions on the library."""
    L.spec_tree_create.argtypes = [C.POINTER(spec_tree_config), C.POINTER(C.c_void_p)]
    L.spec_tree_destroy.argtypes = [C.c_void_p]
    L.spec_tree_check.argtypes = [C.c_void_p, C.c_void_p]
    L.spec_tree_inject_fault.argtypes = [C.c_void_p, C.c_int32]
    for name, args in (("plan", spec_tree_plan_args), ("append", spec_tree_append_args),
                       ("attend", spec_tree_attend_args), ("keep", spec_tree_keep_args)):
        getattr(L, "spec_tree_" + name).argtypes = [C.c_void_p, C.POINTER(args), C.c_void_p]
    for name in TREE_FUNCTIONS:
        getattr(L, name).restype = C.c_int


# --------------------------------------------------------------------------- #
# the C entry points, same names                                              #
# --------------------------------------------------------------------------- #
def _lib():
    from . import load_library
    return load_library()


def _check(code: int, what: str) -> None:
    if code:
        from . import SpecVerifyError
        raise SpecVerifyError(code, what)


def spec_tree_create(cfg: spec_tree_config) -> C.c_void_p:
    h = C.c_void_p()
    _check(_lib().spec_tree_create(C.byref(cfg), C.byref(h)), "spec_tree_create")
    return h


def spec_tree_destroy(h) -> None:
    _check(_lib().spec_tree_destroy(h), "spec_tree_destroy")


def spec_tree_check(h, stream: int = 0) -> int:
    """Wait for `stream`, then read and clear the handle's record of waits that
    ran out: SPEC_OK or SPEC_ERR_TIMEOUT (returned; other errors raise)."""
    from . import SPEC_ERR_TIMEOUT
    code = _lib().spec_tree_check(h, C.c_void_p(stream))
    if code != SPEC_ERR_TIMEOUT:
        _check(code, "spec_tree_check")
    return code


def spec_tree_inject_fault(h, fault: int) -> None:
    _check(_lib().spec_tree_inject_fault(h, int(fault)), "spec_tree_inject_fault")


def spec_tree_plan(h, args: spec_tree_plan_args, stream: int = 0) -> None:
    _check(_lib().spec_tree_plan(h, C.byref(args), C.c_void_p(stream)), "spec_tree_plan")


def spec_tree_append(h, args: spec_tree_append_args, stream: int = 0) -> None:
    _check(_lib().spec_tree_append(h, C.byref(args), C.c_void_p(stream)), "spec_tree_append")


def spec_tree_attend(h, args: spec_tree_attend_args, stream: int = 0) -> None:
    _check(_lib().spec_tree_attend(h, C.byref(args), C.c_void_p(stream)), "spec_tree_attend")


def spec_tree_keep(h, args: spec_tree_keep_args, stream: int = 0) -> None:
    _check(_lib().spec_tree_keep(h, C.byref(args), C.c_void_p(stream)), "spec_tree_keep")


# --------------------------------------------------------------------------- #
# torch wrapper                                                               #
# --------------------------------------------------------------------------- #
def _tensors(values):
    import torch
    for t in values:
        if isinstance(t, torch.Tensor):
            if t.is_cuda:
                yield t
        elif isinstance(t, dict):
            yield from _tensors(t.values())
        elif isinstance(t, tuple):
            yield from _tensors(t)


def on_stream(stream, device, op, *args, **kw):
    """op(*args, **kw) with ``stream`` current.  Its new outputs come from that
    stream's memory (the current stream's may still be read by kernels in flight
    there), and are noted as used by the current stream, which the caller is likely
    to read them on; the tensors it is given are noted as used by ``stream``, so that
    the caller may drop them at once.  It orders nothing: ``stream`` has to wait for
    the work that fills the inputs."""
    import torch
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        res = op(*args, **kw)
    for t in _tensors((args, kw)):
        t.record_stream(stream)
    for t in _tensors((res,)):
        t.record_stream(here)
    return res


class TreeCache:
    """One handle of the operators around a verify step, for one cache shape.

    ``plan`` once a round, ``append`` and ``attend`` once per layer, ``keep``
    once the verify step has chosen a path.  The tensors (block table, ring of
    free pages, caches) are the caller's; the cache of a layer is a pair of
    tensors [num_pages, page_size, kv_heads, head_dim] of one layout, any
    strides with a contiguous last dimension.  ``new_pool`` makes the state of
    an empty pool.  Small calls are bound by the host, so the checks here are
    kept short: plain attributes, one pass over each tensor."""

    def __init__(self, *, max_batch: int, max_tokens: int, q_heads: int, kv_heads: int,
                 head_dim: int, dtype, page_size: int, num_pages: int, table_width: int,
                 device: int | None = None):
        import torch
        from . import SPEC_BF16, SPEC_F32, load_library
        self.h = None
        types = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
        self.dtype = types.get(dtype, dtype)
        code = {torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16,
                torch.float32: SPEC_F32}.get(self.dtype)
        if code is None:
            raise TypeError(f"dtype must be 'bf16' or 'f16', got {dtype}")
        self.device = torch.cuda.current_device() if device is None else int(device)
        self.cfg = spec_tree_config(self.device, max_batch, max_tokens, q_heads, kv_heads,
                                    head_dim, code, page_size, num_pages, table_width)
        self.h = spec_tree_create(self.cfg)
        self._lib = load_library()
        self._dev = torch.device("cuda", self.device)
        self._hq, self._hkv, self._d = q_heads, kv_heads, head_dim
        self._pages, self._width, self._max_tokens = num_pages, table_width, max_tokens
        self._cache_shape = (num_pages, page_size, kv_heads, head_dim)
        self._scale = head_dim ** -0.5
        self._current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
        # the argument records of the calls, filled anew by each (one handle, one caller at a time)
        self._plan_args, self._append_args = spec_tree_plan_args(), spec_tree_append_args()
        self._attend_args, self._keep_args = spec_tree_attend_args(), spec_tree_keep_args()

    def close(self):
        if self.h is not None and self.h.value:
            spec_tree_destroy(self.h)
        self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- argument checks --------------------------------------------------- #
    def _tensor(self, t, shape, dtype, what):
        """The address of a contiguous tensor of this shape and type on the handle's device."""
        if t.shape != shape or t.dtype is not dtype or t.device != self._dev or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {shape} on "
                             f"{self._dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _rows(self, rec, t, shape, what):
        """Fill a spec_tree_rows with a [B, T, heads, head_dim] tensor of any strides."""
        if t.shape != shape or t.dtype is not self.dtype or t.device != self._dev:
            raise ValueError(f"{what} must be {self.dtype} {shape} on {self._dev}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        st = t.stride()
        if st[3] != 1:
            raise ValueError(f"the last dimension of {what} must be contiguous")
        rec.ptr = t.data_ptr()
        # the stride of a dimension of size 1 is never used
        rec.seq_stride = st[0] if shape[0] > 1 else 0
        rec.token_stride = st[1] if shape[1] > 1 else 0
        rec.head_stride = st[2] if shape[2] > 1 else 0

    def _cache(self, rec, k, v, layered=False):
        """Fill a spec_tree_cache with the K and V tensors of one layer or (layered) of several."""
        shape, st = k.shape, k.stride()
        if v.shape != shape or (v.stride() != st and
                                any(a != b for a, b, n in zip(st, v.stride(), shape) if n > 1)):
            raise ValueError("k_cache and v_cache must have the same shape and strides")
        many = layered and len(shape) == 5
        if (shape[1:] if many else shape) != self._cache_shape or k.dtype is not self.dtype or \
                v.dtype is not self.dtype or k.device != self._dev or v.device != self._dev:
            raise ValueError(f"the caches must be {self.dtype} {self._cache_shape} on {self._dev}, "
                             f"got {k.dtype} and {v.dtype} {tuple(shape)} on {k.device}")
        if st[-1] != 1:
            raise ValueError("the last dimension of the caches must be contiguous")
        size = self._cache_shape
        rec.k, rec.v = k.data_ptr(), v.data_ptr()
        rec.page_stride = st[-4] if size[0] > 1 else 0
        rec.token_stride = st[-3] if size[1] > 1 else 0
        rec.head_stride = st[-2] if size[2] > 1 else 0
        rec.layers = shape[0] if many else 1
        rec.layer_stride = st[0] if many and shape[0] > 1 else 0

    def _stream(self):
        # the address of the current stream, without an object for it where torch can tell
        return self._current_stream(self.device)

    def _on(self, stream, op, *args, **kw):
        return on_stream(stream, self.device, op, *args, **kw)

    def _out(self, out, key, shape, dtype, like=None):
        """The caller's output tensor (checked), or a new one (like `like`, a contiguous
        tensor of that shape and type, when given)."""
        if out is None or key not in out:
            import torch
            if like is not None:
                return torch.empty_like(like)
            return torch.empty(shape, dtype=dtype, device=self._dev)
        self._tensor(out[key], shape, dtype, f"out['{key}']")
        return out[key]

    # ---- the operators ------------------------------------------------------ #
    def new_pool(self, batch: int) -> dict:
        """The plan's state of an empty cache: block_table, held, ring and
        free_pages, every page free."""
        import torch
        i32, dev = torch.int32, self._dev
        return dict(block_table=torch.full((batch, self._width), -1, dtype=i32, device=dev),
                    held=torch.zeros(batch, dtype=i32, device=dev),
                    ring=torch.tensor([0, self._pages], dtype=torch.int64, device=dev),
                    free_pages=torch.arange(self._pages, dtype=i32, device=dev))

    def plan(self, ctx_len, n_tokens, held, ring, free_pages, block_table, *, parents=None,
             max_tokens: int | None = None, out: dict | None = None, stream=None) -> dict:
        """Pages, slots, positions and ancestor masks of a round (see
        include/spec_tree.h); updates free_pages and block_table in place and
        returns held, ring, slot_map, positions, row_status (and tree_mask with
        parents).  T is parents.shape[1], or max_tokens for chains."""
        if stream is not None:
            return self._on(stream, self.plan, ctx_len, n_tokens, held, ring, free_pages, block_table,
                            parents=parents, max_tokens=max_tokens, out=out)
        import torch
        i32, a = torch.int32, self._plan_args
        B = ctx_len.shape[0]
        T = parents.shape[1] if parents is not None else \
            self._max_tokens if max_tokens is None else int(max_tokens)
        b, bt = (B,), (B, T)
        a.ctx_len = self._tensor(ctx_len, b, i32, "ctx_len")
        a.n_tokens = None if n_tokens is None else self._tensor(n_tokens, b, i32, "n_tokens")
        a.held = self._tensor(held, b, i32, "held")
        a.ring = self._tensor(ring, (2,), torch.int64, "ring")
        a.free_pages = self._tensor(free_pages, (self._pages,), i32, "free_pages")
        a.block_table = self._tensor(block_table, (B, self._width), i32, "block_table")
        a.parents = a.tree_mask = None
        if parents is not None:
            a.parents = self._tensor(parents, bt, i32, "parents")
        res = {"held": self._out(out, "held", b, i32, held),
               "ring": self._out(out, "ring", (2,), torch.int64, ring),
               "slot_map": self._out(out, "slot_map", bt, i32, parents),
               "positions": self._out(out, "positions", bt, i32, parents),
               "row_status": self._out(out, "row_status", b, i32, held)}
        if parents is not None:
            mask = res["tree_mask"] = self._out(out, "tree_mask", (B, T, (T + 31) // 32), i32)
            a.tree_mask = mask.data_ptr()
        a.batch, a.tokens = B, T
        a.held_out, a.ring_out = res["held"].data_ptr(), res["ring"].data_ptr()
        a.slot_map, a.positions = res["slot_map"].data_ptr(), res["positions"].data_ptr()
        a.row_status = res["row_status"].data_ptr()
        _check(self._lib.spec_tree_plan(self.h, a, self._stream()), "spec_tree_plan")
        return res

    def append(self, q, k, v, k_cache, v_cache, slot_map, positions=None, n_tokens=None, *,
               q_weight=None, k_weight=None, eps: float = 1e-6, cos_sin=None,
               interleaved: bool = False, out=None, stream=None):
        """Norm and rotation of q and k, k and v into the cache; returns the
        new q [B, T, q_heads, head_dim].  cos_sin: float32 [positions, rot_dim],
        rot_dim / 2 cosines, then as many sines."""
        if stream is not None:
            return self._on(stream, self.append, q, k, v, k_cache, v_cache, slot_map, positions, n_tokens,
                            q_weight=q_weight, k_weight=k_weight, eps=eps, cos_sin=cos_sin,
                            interleaved=interleaved, out=out)
        import torch
        i32, a, d, hkv = torch.int32, self._append_args, self._d, self._hkv
        B, T = q.shape[:2]
        shape, bt = (B, T, self._hq, d), (B, T)
        self._rows(a.q, q, shape, "q")
        self._rows(a.k, k, (B, T, hkv, d), "k")
        self._rows(a.v, v, (B, T, hkv, d), "v")
        self._cache(a.cache, k_cache, v_cache)
        a.slot_map = self._tensor(slot_map, bt, i32, "slot_map")
        a.positions = None if positions is None else self._tensor(positions, bt, i32, "positions")
        a.n_tokens = None if n_tokens is None else self._tensor(n_tokens, (B,), i32, "n_tokens")
        a.q_weight = None if q_weight is None else self._tensor(q_weight, (d,), self.dtype, "q_weight")
        a.k_weight = None if k_weight is None else self._tensor(k_weight, (d,), self.dtype, "k_weight")
        a.cos_sin, a.table_len, a.rot_dim = None, 0, 0
        if cos_sin is not None:
            if cos_sin.dim() != 2 or positions is None:
                raise ValueError("cos_sin must be a float32 tensor [positions, rot_dim], with "
                                 "positions given")
            a.cos_sin = self._tensor(cos_sin, cos_sin.shape, torch.float32, "cos_sin")
            a.table_len, a.rot_dim = cos_sin.shape
        a.interleaved, a.eps, a.batch, a.tokens = bool(interleaved), eps, B, T
        if out is None:
            out = torch.empty(shape, dtype=self.dtype, device=self._dev)
            a.q_out = out.data_ptr()
        else:
            a.q_out = self._tensor(out, shape, self.dtype, "out")
        _check(self._lib.spec_tree_append(self.h, a, self._stream()), "spec_tree_append")
        return out

    def attend(self, q, k_cache, v_cache, block_table, ctx_len, n_tokens=None, *, tree_mask=None,
               scale: float | None = None, out: dict | None = None, lse: bool = True,
               stream=None) -> dict:
        """Attention of the nodes over context and tree (or, without tree_mask,
        over context and chain); scale defaults to head_dim ** -0.5.  Returns
        out [B, T, q_heads, head_dim] and, with lse, lse [B, T, q_heads]."""
        if stream is not None:
            return self._on(stream, self.attend, q, k_cache, v_cache, block_table, ctx_len, n_tokens,
                            tree_mask=tree_mask, scale=scale, out=out, lse=lse)
        import torch
        i32, a = torch.int32, self._attend_args
        B, T = q.shape[:2]
        shape = (B, T, self._hq, self._d)
        self._rows(a.q, q, shape, "q")
        self._cache(a.cache, k_cache, v_cache)
        a.block_table = self._tensor(block_table, (B, self._width), i32, "block_table")
        a.ctx_len = self._tensor(ctx_len, (B,), i32, "ctx_len")
        a.n_tokens = None if n_tokens is None else self._tensor(n_tokens, (B,), i32, "n_tokens")
        a.tree_mask = None if tree_mask is None else \
            self._tensor(tree_mask, (B, T, (T + 31) // 32), i32, "tree_mask")
        a.scale, a.batch, a.tokens = self._scale if scale is None else scale, B, T
        o = self._out(out, "out", shape, self.dtype)
        res = {"out": o}
        a.out, a.lse = o.data_ptr(), None
        if lse:
            e = res["lse"] = self._out(out, "lse", shape[:3], torch.float32)
            a.lse = e.data_ptr()
        _check(self._lib.spec_tree_attend(self.h, a, self._stream()), "spec_tree_attend")
        return res

    def keep(self, k_cache, v_cache, block_table, ctx_len, n_tokens, path, path_len, *,
             plan_status=None, out: dict | None = None, stream=None) -> dict:
        """Move the accepted nodes' keys and values behind the context, in all
        layers of [layers, num_pages, page_size, kv_heads, head_dim] caches (or
        in one layer's); returns the new ctx_len and row_status.  plan_status is
        the row_status of the round's plan: where it is not 0 nothing moves and
        the length stays."""
        if stream is not None:
            return self._on(stream, self.keep, k_cache, v_cache, block_table, ctx_len, n_tokens, path,
                            path_len, plan_status=plan_status, out=out)
        import torch
        i32, a = torch.int32, self._keep_args
        B, T = path.shape
        b = (B,)
        self._cache(a.cache, k_cache, v_cache, True)
        a.block_table = self._tensor(block_table, (B, self._width), i32, "block_table")
        a.ctx_len = self._tensor(ctx_len, b, i32, "ctx_len")
        a.n_tokens = None if n_tokens is None else self._tensor(n_tokens, b, i32, "n_tokens")
        a.path = self._tensor(path, (B, T), i32, "path")
        a.path_len = self._tensor(path_len, b, i32, "path_len")
        a.plan_status = None if plan_status is None else \
            self._tensor(plan_status, b, i32, "plan_status")
        a.batch, a.tokens = B, T
        res = {"ctx_len": self._out(out, "ctx_len", b, i32, ctx_len),
               "row_status": self._out(out, "row_status", b, i32, ctx_len)}
        a.ctx_out, a.row_status = res["ctx_len"].data_ptr(), res["row_status"].data_ptr()
        _check(self._lib.spec_tree_keep(self.h, a, self._stream()), "spec_tree_keep")
        return res

    def check(self, stream=None) -> int:
        """SPEC_OK, or SPEC_ERR_TIMEOUT when a wait of an attend ran out."""
        return spec_tree_check(self.h, self._stream() if stream is None else stream.cuda_stream)


__all__ = [n for n in dir() if n.startswith("spec_tree_") or n.startswith("SPEC_")] + ["TreeCache"]
