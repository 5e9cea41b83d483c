"""Binding of include/spec_score.h: the operators that score rows of logits.

The C entry points under their own names (argument marshalling only), and
``logprobs`` and ``distill``, which take torch tensors.  Every step runs in the
library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import struct

from .tree import SPEC_F16, on_stream

SPEC_SCORE_MAX_TOP, SPEC_SCORE_MAX_ENTRIES = 128, 256

SCORE_FUNCTIONS = ("spec_score_logprobs", "spec_score_distill")


class spec_score_rows(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("seq_stride", C.c_int64), ("token_stride", C.c_int64)]


class spec_score_logprobs_args(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("device", "dtype", "batch", "tokens", "vocab", "top_n")] + \
        [("temperature", C.c_float), ("logits", spec_score_rows)] + \
        [(n, C.c_void_p) for n in ("ids", "grad_logprob", "grad_entropy", "logprob", "rank", "entropy",
                                   "lse", "top_ids", "top_logprobs", "row_status")] + \
        [("grad", spec_score_rows)]


class spec_score_distill_args(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("device", "dtype", "teacher_dtype", "batch", "tokens", "vocab",
                                         "entries", "tail")] + \
        [("temperature", C.c_float), ("teacher_temperature", C.c_float), ("student", spec_score_rows)] + \
        [(n, C.c_void_p) for n in ("ids", "teacher", "teacher_lse", "grad_loss", "loss", "accept",
                                   "row_status")] + \
        [("grad", spec_score_rows)]


def bind(L: C.CDLL) -> None:
    """Declare the argument types of this header's functions on the library."""
    L.spec_score_logprobs.argtypes = [C.POINTER(spec_score_logprobs_args), C.c_void_p]
    L.spec_score_distill.argtypes = [C.POINTER(spec_score_distill_args), C.c_void_p]
    for name in SCORE_FUNCTIONS:
        getattr(L, name).restype = C.c_int


# --------------------------------------------------------------------------- #
# the C entry points, same names                                              #
# --------------------------------------------------------------------------- #
def _call(name: str, args, stream: int) -> None:
    from . import SpecVerifyError, load_library
    code = getattr(load_library(), name)(C.byref(args), C.c_void_p(stream))
    if code:
        raise SpecVerifyError(code, name)


def spec_score_logprobs(args: spec_score_logprobs_args, stream: int = 0) -> None:
    _call("spec_score_logprobs", args, stream)


def spec_score_distill(args: spec_score_distill_args, stream: int = 0) -> None:
    _call("spec_score_distill", args, stream)


# --------------------------------------------------------------------------- #
# torch wrapper                                                               #
# --------------------------------------------------------------------------- #
# Small calls are bound by the host, so the wrapper is kept short: the argument records are packed at once
# (the layouts of the two structures above).
_LOGPROBS_ARGS, _DISTILL_ARGS = struct.Struct("@6ifPqq10PPqq"), struct.Struct("@8i2fPqq7PPqq")
_bound: dict = {}


def _bind_wrapper() -> dict:
    """What the wrapper looks up once: torch, the type codes, and the library's functions taking packed records."""
    import torch
    from . import SPEC_BF16, SPEC_F32, load_library
    L, known = load_library(), {"torch": torch}
    for name in SCORE_FUNCTIONS:
        f = L[name]  # a function object of its own: the library's keeps its declared types
        f.argtypes, f.restype = [C.c_char_p, C.c_void_p], C.c_int
        known[name] = f
    known["codes"] = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}
    known["stream"] = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _bound.update(known)  # at once, as another thread may look
    return _bound


def _code(dtype, what) -> int:
    code = _bound["codes"].get(dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32, got {dtype}")
    return code


def _rows(t, what):
    """(address, stride of a sequence, of a position) of a [B, T, V] or [N, V] tensor of any strides."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    return t.data_ptr(), st[0] if len(st) == 3 else 0, st[-2]


def _shape(t, what):
    """(B, T, V) of a tensor of rows on a CUDA device."""
    shape = t.shape
    if len(shape) == 2:
        shape = (1, *shape)
    elif len(shape) != 3:
        raise ValueError(f"{what} must be [B, T, V] or [N, V], got {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device, got {t.device}")
    if max(shape) > 0x7FFFFFFF:  # (an expanded tensor may well be)
        raise ValueError(f"{what} must have sizes below 2^31, got {tuple(shape)}")
    return shape


def _temperature(t) -> float:
    """A number that fp32 holds, where there is one; the library refuses the others."""
    t = float(t)
    return t if -1e38 < t < 1e38 else float("nan")


def _tensor(t, shape, dtype, device, what):
    """The address of a contiguous tensor of this shape and type."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _result(res, out, name, shape, dtype, device):
    """A result into res, the caller's tensor or a new one; its address."""
    t = None if out is None else out.get(name)
    if t is None:
        t = res[name] = _bound["torch"].empty(shape, dtype=dtype, device=device)
        return t.data_ptr()
    res[name] = t
    return _tensor(t, shape, dtype, device, f"out['{name}']")


def _grad(out, like, res):
    """The caller's gradient tensor (checked; the logits themselves may be given), or a new one."""
    g = None if out is None else out.get("grad")
    if g is None:
        g = _bound["torch"].empty(like.shape, dtype=like.dtype, device=like.device)
    elif g.shape != like.shape or g.dtype is not like.dtype or g.device != like.device:
        raise ValueError(f"out['grad'] must be {like.dtype} {tuple(like.shape)} on {like.device}, got "
                         f"{g.dtype} {tuple(g.shape)} on {g.device}")
    res["grad"] = g
    return _rows(g, "out['grad']")


def _run(name, args, device) -> None:
    code = _bound[name](args, _bound["stream"](device.index))
    if code:
        from . import SpecVerifyError
        raise SpecVerifyError(code, name)


def logprobs(logits, tokens=None, *, temperature: float = 1.0, top_n: int = 0, rank: bool = False,
             grad_logprob=None, grad_entropy=None, out: dict | None = None, stream=None) -> dict:
    """Log probabilities of given tokens, with entropy and top alternatives.

    logits [B, T, V] or [N, V] (bf16, f16 or fp32; any strides, the last dimension
    contiguous); tokens int32 [B, T] or [N], -1 where a row is not to be scored, or
    None.  Returns entropy, lse and row_status of every row, logprob of its token
    (and, with rank, how many tokens are likelier), and with top_n top_ids and
    top_logprobs [.., top_n] in order.  With grad_logprob or grad_entropy (fp32,
    [B, T] or [N]) also grad, the gradient with respect to the logits, as for
    ``logits.backward(grad)``; ``out={"grad": logits}`` writes it over them.
    See include/spec_score.h.  stream: as in ``Verifier.run``."""
    if stream is not None:
        return on_stream(stream, logits.device, logprobs, logits, tokens, temperature=temperature, top_n=top_n,
                         rank=rank, grad_logprob=grad_logprob, grad_entropy=grad_entropy, out=out)
    torch = (_bound or _bind_wrapper())["torch"]
    B, T, V = _shape(logits, "logits")
    lead, dev, f32, i32 = logits.shape[:-1], logits.device, torch.float32, torch.int32
    if tokens is None and (rank or grad_logprob is not None):
        raise ValueError("rank and grad_logprob need tokens")
    code, rows = _code(logits.dtype, "logits"), _rows(logits, "logits")
    ids = _tensor(tokens, lead, i32, dev, "tokens")
    up = _tensor(grad_logprob, lead, f32, dev, "grad_logprob"), _tensor(grad_entropy, lead, f32, dev, "grad_entropy")
    res, lp, rk, ti, tl, grad = {}, 0, 0, 0, 0, (0, 0, 0)
    if tokens is not None:
        lp = _result(res, out, "logprob", lead, f32, dev)
        if rank:
            rk = _result(res, out, "rank", lead, i32, dev)
    ent, lse = _result(res, out, "entropy", lead, f32, dev), _result(res, out, "lse", lead, f32, dev)
    status = _result(res, out, "row_status", lead, i32, dev)
    top_n = max(-1, min(top_n, SPEC_SCORE_MAX_TOP + 1))  # the library refuses both, and nothing is allocated for them
    if 0 < top_n <= SPEC_SCORE_MAX_TOP:
        ti = _result(res, out, "top_ids", (*lead, top_n), i32, dev)
        tl = _result(res, out, "top_logprobs", (*lead, top_n), f32, dev)
    if grad_logprob is not None or grad_entropy is not None:
        grad = _grad(out, logits, res)
    _run("spec_score_logprobs", _LOGPROBS_ARGS.pack(dev.index, code, B, T, V, top_n, _temperature(temperature), *rows,
                                                    ids, *up, lp, rk, ent, lse, ti, tl, status, *grad), dev)
    return res


def distill(student, top_ids, teacher, *, temperature: float = 1.0, teacher_temperature: float | None = None,
            tail: bool = False, teacher_lse=None, grad_loss=None, out: dict | None = None, stream=None) -> dict:
    """Divergence of a student's rows from a teacher's top logits.

    student [B, T, V] or [N, V] as in ``logprobs``; top_ids int32 [.., k] the
    tokens of the teacher's entries (-1: no entry) and teacher [.., k] their
    logits, in bf16, f16 or fp32, which are divided by teacher_temperature
    (default: temperature).  Without tail they are renormalised; with tail what
    they leave of the teacher's mass is one more outcome, and they are log
    probabilities unless teacher_lse gives the teacher's log-sum-exp (at its
    temperature).  ``logprobs(target, top_n=k, temperature=t)`` records them:
    top_ids, and top_logprobs with teacher_temperature=1.
    Returns loss, accept (the sum of min(q, p) over the entries) and row_status,
    and with grad_loss (fp32, one per row) grad, the gradient of sum(grad_loss *
    loss), as for ``student.backward(grad)``; ``out={"grad": student}`` writes it
    over the logits.  See include/spec_score.h.  stream: as in ``Verifier.run``."""
    if stream is not None:
        return on_stream(stream, student.device, distill, student, top_ids, teacher, temperature=temperature,
                         teacher_temperature=teacher_temperature, tail=tail, teacher_lse=teacher_lse,
                         grad_loss=grad_loss, out=out)
    torch = (_bound or _bind_wrapper())["torch"]
    B, T, V = _shape(student, "student")
    lead, dev, f32 = student.shape[:-1], student.device, torch.float32
    k = top_ids.shape[-1] if top_ids.dim() else 0
    code, t_code, rows = _code(student.dtype, "student"), _code(teacher.dtype, "teacher"), _rows(student, "student")
    ins = (_tensor(top_ids, (*lead, k), torch.int32, dev, "top_ids"),
           _tensor(teacher, (*lead, k), teacher.dtype, dev, "teacher"),
           _tensor(teacher_lse, lead, f32, dev, "teacher_lse"), _tensor(grad_loss, lead, f32, dev, "grad_loss"))
    res, grad = {}, (0, 0, 0)
    outs = (_result(res, out, "loss", lead, f32, dev), _result(res, out, "accept", lead, f32, dev),
            _result(res, out, "row_status", lead, torch.int32, dev))
    if grad_loss is not None:
        grad = _grad(out, student, res)
    temp = _temperature(temperature)
    t_temp = temp if teacher_temperature is None else _temperature(teacher_temperature)
    _run("spec_score_distill", _DISTILL_ARGS.pack(dev.index, code, t_code, B, T, V, k, bool(tail), temp, t_temp,
                                                  *rows, *ins, *outs, *grad), dev)
    return res


__all__ = [n for n in dir() if n.startswith("spec_score_") or n.startswith("SPEC_SCORE_")] + \
    ["logprobs", "distill"]
