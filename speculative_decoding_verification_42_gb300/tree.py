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
                ("row_status", C.c_void_p)]


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
class TreeCache:
    """One handle of the operators around a verify step, for one cache shape.

    ``plan`` once a round, ``append`` and ``attend`` once per layer, ``keep``
    once the verify step has chosen a path.  The tensors (block table, ring of
    free pages, caches) are the caller's; the cache of a layer is a pair of
    tensors [num_pages, page_size, kv_heads, head_dim] of one layout, any
    strides with a contiguous last dimension.  ``new_pool`` makes the state of
    an empty pool."""

    def __init__(self, *, max_batch: int, max_tokens: int, q_heads: int, kv_heads: int,
                 head_dim: int, dtype, page_size: int, num_pages: int, table_width: int,
                 device: int | None = None):
        import torch
        from . import SPEC_BF16, SPEC_F32
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
    def _ints(self, t, shape, what, dtype=None):
        import torch
        if t is None:
            return None
        if t.dtype != (dtype or torch.int32) or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype or torch.int32} tensor of shape "
                             f"{shape}, got {t.dtype} {tuple(t.shape)}")
        self._on_device(t, what)
        return t.data_ptr()

    def _on_device(self, t, what):
        if t.device.type != "cuda" or t.device.index != self.device:
            raise ValueError(f"{what} is on {t.device}, the handle on cuda:{self.device}")

    def _rows(self, t, heads, what):
        if t.dtype != self.dtype or t.dim() != 4 or t.shape[2] != heads or \
                t.shape[3] != self.cfg.head_dim:
            raise ValueError(f"{what} must be {self.dtype} [B, T, {heads}, {self.cfg.head_dim}], "
                             f"got {t.dtype} {tuple(t.shape)}")
        self._on_device(t, what)
        return spec_tree_rows(t.data_ptr(), *self._strides(t, (0, 1, 2), what))

    @staticmethod
    def _strides(t, dims, what):
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"the last dimension of {what} must be contiguous")
        # the stride of a dimension of size 1 is never used
        return [t.stride(d) if t.shape[d] > 1 else 0 for d in dims]

    def _cache(self, k, v, layered):
        c = self.cfg
        want = (c.num_pages, c.page_size, c.kv_heads, c.head_dim)
        for t, what in ((k, "k_cache"), (v, "v_cache")):
            if t.dtype != self.dtype or tuple(t.shape[-4:]) != want or t.dim() not in (4, 4 + layered):
                raise ValueError(f"{what} must be {self.dtype} {want}, got {t.dtype} {tuple(t.shape)}")
            self._on_device(t, what)
        strides = self._strides(k, (-4, -3, -2), "k_cache")
        layer = k.stride(0) if k.dim() == 5 and k.shape[0] > 1 else 0
        if self._strides(v, (-4, -3, -2), "v_cache") != strides or v.shape != k.shape or \
                (layer and v.stride(0) != layer):
            raise ValueError("k_cache and v_cache must have the same shape and strides")
        return spec_tree_cache(k.data_ptr(), v.data_ptr(), *strides, layer,
                               k.shape[0] if k.dim() == 5 else 1)

    def _stream(self, stream):
        import torch
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        return s.cuda_stream

    def _out(self, t, shape, dtype, what):
        import torch
        if t is None:
            return torch.empty(shape, dtype=dtype, device=f"cuda:{self.device}")
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
        self._on_device(t, what)
        return t

    # ---- the operators ------------------------------------------------------ #
    def new_pool(self, batch: int) -> dict:
        """The plan's state of an empty cache: block_table, held, ring and
        free_pages, every page free."""
        import torch
        c, dev = self.cfg, f"cuda:{self.device}"
        return dict(block_table=torch.full((batch, c.table_width), -1, dtype=torch.int32, device=dev),
                    held=torch.zeros(batch, dtype=torch.int32, device=dev),
                    ring=torch.tensor([0, c.num_pages], dtype=torch.int64, device=dev),
                    free_pages=torch.arange(c.num_pages, dtype=torch.int32, device=dev))

    def plan(self, ctx_len, n_tokens, held, ring, free_pages, block_table, *, parents=None,
             max_tokens: int | None = None, out: dict | None = None, stream=None) -> dict:
        """Pages, slots, positions and ancestor masks of a round (see
        include/spec_tree.h); updates free_pages and block_table in place and
        returns held, ring, slot_map, positions, row_status (and tree_mask with
        parents).  T is parents.shape[1], or max_tokens for chains."""
        import torch
        B = ctx_len.shape[0]
        T = parents.shape[1] if parents is not None else int(max_tokens or self.cfg.max_tokens)
        out = out or {}
        i32 = torch.int32
        res = dict(held=self._out(out.get("held"), (B,), i32, "out['held']"),
                   ring=self._out(out.get("ring"), (2,), torch.int64, "out['ring']"),
                   slot_map=self._out(out.get("slot_map"), (B, T), i32, "out['slot_map']"),
                   positions=self._out(out.get("positions"), (B, T), i32, "out['positions']"),
                   row_status=self._out(out.get("row_status"), (B,), i32, "out['row_status']"))
        if parents is not None:
            res["tree_mask"] = self._out(out.get("tree_mask"), (B, T, -(-T // 32)), i32,
                                         "out['tree_mask']")
        c = self.cfg
        args = spec_tree_plan_args(
            self._ints(ctx_len, (B,), "ctx_len"), self._ints(n_tokens, (B,), "n_tokens"),
            self._ints(parents, (B, T), "parents"), self._ints(held, (B,), "held"),
            self._ints(ring, (2,), "ring", torch.int64),
            self._ints(free_pages, (c.num_pages,), "free_pages"),
            self._ints(block_table, (B, c.table_width), "block_table"), B, T,
            res["held"].data_ptr(), res["ring"].data_ptr(), res["slot_map"].data_ptr(),
            res["positions"].data_ptr(),
            res["tree_mask"].data_ptr() if parents is not None else None,
            res["row_status"].data_ptr())
        spec_tree_plan(self.h, args, self._stream(stream))
        return res

    def append(self, q, k, v, k_cache, v_cache, slot_map, positions=None, n_tokens=None, *,
               q_weight=None, k_weight=None, eps: float = 1e-6, cos_sin=None,
               interleaved: bool = False, out=None, stream=None):
        """Norm and rotation of q and k, k and v into the cache; returns the
        new q [B, T, q_heads, head_dim].  cos_sin: float32 [positions, rot_dim],
        rot_dim / 2 cosines, then as many sines."""
        import torch
        c = self.cfg
        B, T = q.shape[:2]
        if tuple(k.shape[:2]) != (B, T) or tuple(v.shape[:2]) != (B, T):
            raise ValueError("q, k and v must have the same batch and tokens")
        for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None and (w.dtype != self.dtype or tuple(w.shape) != (c.head_dim,) or
                                  not w.is_contiguous()):
                raise ValueError(f"{what} must be a contiguous {self.dtype} tensor [{c.head_dim}]")
        if cos_sin is not None and (cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or
                                    not cos_sin.is_contiguous() or positions is None):
            raise ValueError("cos_sin must be a contiguous float32 tensor [positions, rot_dim], "
                             "with positions given")
        for t, what in ((q_weight, "q_weight"), (k_weight, "k_weight"), (cos_sin, "cos_sin")):
            if t is not None:
                self._on_device(t, what)
        out = self._out(out, (B, T, c.q_heads, c.head_dim), self.dtype, "out")
        table_len, rot = cos_sin.shape if cos_sin is not None else (0, 0)
        args = spec_tree_append_args(
            self._rows(q, c.q_heads, "q"), self._rows(k, c.kv_heads, "k"),
            self._rows(v, c.kv_heads, "v"), self._cache(k_cache, v_cache, False),
            self._ints(slot_map, (B, T), "slot_map"), self._ints(positions, (B, T), "positions"),
            self._ints(n_tokens, (B,), "n_tokens"),
            q_weight.data_ptr() if q_weight is not None else None,
            k_weight.data_ptr() if k_weight is not None else None,
            cos_sin.data_ptr() if cos_sin is not None else None, table_len, rot,
            int(interleaved), float(eps), B, T, out.data_ptr())
        spec_tree_append(self.h, args, self._stream(stream))
        return out

    def attend(self, q, k_cache, v_cache, block_table, ctx_len, n_tokens=None, *, tree_mask=None,
               scale: float | None = None, out: dict | None = None, lse: bool = True,
               stream=None) -> dict:
        """Attention of the nodes over context and tree (or, without tree_mask,
        over context and chain); scale defaults to head_dim ** -0.5.  Returns
        out [B, T, q_heads, head_dim] and, with lse, lse [B, T, q_heads]."""
        import torch
        c = self.cfg
        B, T = q.shape[:2]
        out = out or {}
        res = dict(out=self._out(out.get("out"), (B, T, c.q_heads, c.head_dim), self.dtype,
                                 "out['out']"))
        if lse:
            res["lse"] = self._out(out.get("lse"), (B, T, c.q_heads), torch.float32, "out['lse']")
        args = spec_tree_attend_args(
            self._rows(q, c.q_heads, "q"), self._cache(k_cache, v_cache, False),
            self._ints(block_table, (B, c.table_width), "block_table"),
            self._ints(ctx_len, (B,), "ctx_len"), self._ints(n_tokens, (B,), "n_tokens"),
            self._ints(tree_mask, (B, T, -(-T // 32)), "tree_mask"),
            float(c.head_dim ** -0.5 if scale is None else scale), B, T, res["out"].data_ptr(),
            res["lse"].data_ptr() if lse else None)
        spec_tree_attend(self.h, args, self._stream(stream))
        return res

    def keep(self, k_cache, v_cache, block_table, ctx_len, n_tokens, path, path_len, *,
             out: dict | None = None, stream=None) -> dict:
        """Move the accepted nodes' keys and values behind the context, in all
        layers of [layers, num_pages, page_size, kv_heads, head_dim] caches (or
        in one layer's); returns the new ctx_len and row_status."""
        import torch
        B, T = path.shape
        out = out or {}
        res = dict(ctx_len=self._out(out.get("ctx_len"), (B,), torch.int32, "out['ctx_len']"),
                   row_status=self._out(out.get("row_status"), (B,), torch.int32,
                                        "out['row_status']"))
        args = spec_tree_keep_args(
            self._cache(k_cache, v_cache, True),
            self._ints(block_table, (B, self.cfg.table_width), "block_table"),
            self._ints(ctx_len, (B,), "ctx_len"), self._ints(n_tokens, (B,), "n_tokens"),
            self._ints(path, (B, T), "path"), self._ints(path_len, (B,), "path_len"), B, T,
            res["ctx_len"].data_ptr(), res["row_status"].data_ptr())
        spec_tree_keep(self.h, args, self._stream(stream))
        return res

    def check(self, stream=None) -> int:
        """SPEC_OK, or SPEC_ERR_TIMEOUT when a wait of an attend ran out."""
        return spec_tree_check(self.h, self._stream(stream))


__all__ = [n for n in dir() if n.startswith("spec_tree_") or n.startswith("SPEC_")] + ["TreeCache"]
