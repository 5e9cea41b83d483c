"""Binding of include/spec_score.h: the operators that score rows of logits.

The C entry points under their own names (argument marshalling only), and
``logprobs`` and ``distill``, which take torch tensors.  Every step runs in the
library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes as C

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
_CODES: dict = {}


def _code(dtype, what) -> int:
    if not _CODES:
        import torch
        from . import SPEC_BF16, SPEC_F32
        _CODES.update({torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16})
    if dtype not in _CODES:
        raise TypeError(f"{what} must be bfloat16, float16 or float32, got {dtype}")
    return _CODES[dtype]


def _rows(rec, t, what):
    """Fill a spec_score_rows with a [B, T, V] or [N, V] tensor of any strides."""
    st = t.stride()
    if t.shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    rec.ptr = t.data_ptr()
    rec.token_stride = st[-2]
    rec.seq_stride = st[0] if len(st) == 3 else 0


def _logits(t, what):
    """(leading shape, B, T, V) of a tensor of rows on a CUDA device."""
    shape = t.shape
    if len(shape) == 3:
        B, T, V = shape
    elif len(shape) == 2:
        (T, V), B = shape, 1
    else:
        raise ValueError(f"{what} must be [B, T, V] or [N, V], got {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device, got {t.device}")
    return shape[:-1], B, T, V


def _tensor(t, shape, dtype, device, what):
    """The address of a contiguous tensor of this shape and type."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _grad(rec, out, like, res):
    """The caller's gradient tensor (checked; the logits themselves may be given), or a new one."""
    g = None if out is None else out.get("grad")
    if g is None:
        import torch
        g = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    elif g.shape != like.shape or g.dtype is not like.dtype or g.device != like.device:
        raise ValueError(f"out['grad'] must be {like.dtype} {tuple(like.shape)} on {like.device}, got "
                         f"{g.dtype} {tuple(g.shape)} on {g.device}")
    _rows(rec, g, "out['grad']")
    res["grad"] = g


def _stream(device) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


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
    import torch
    a, dev, f32, i32 = spec_score_logprobs_args(), logits.device, torch.float32, torch.int32
    lead, a.batch, a.tokens, a.vocab = _logits(logits, "logits")
    a.device, a.dtype, a.top_n, a.temperature = dev.index, _code(logits.dtype, "logits"), top_n, temperature
    _rows(a.logits, logits, "logits")
    if tokens is None and (rank or grad_logprob is not None):
        raise ValueError("rank and grad_logprob need tokens")
    a.ids = _tensor(tokens, lead, i32, dev, "tokens")
    a.grad_logprob = _tensor(grad_logprob, lead, f32, dev, "grad_logprob")
    a.grad_entropy = _tensor(grad_entropy, lead, f32, dev, "grad_entropy")
    res = {}

    def result(name, shape, dtype):
        t = None if out is None else out.get(name)
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
            setattr(a, name, t.data_ptr())
        else:
            setattr(a, name, _tensor(t, shape, dtype, dev, f"out['{name}']"))
        res[name] = t

    if tokens is not None:
        result("logprob", lead, f32)
        if rank:
            result("rank", lead, i32)
    result("entropy", lead, f32)
    result("lse", lead, f32)
    result("row_status", lead, i32)
    if top_n > 0:
        result("top_ids", (*lead, top_n), i32)
        result("top_logprobs", (*lead, top_n), f32)
    if grad_logprob is not None or grad_entropy is not None:
        _grad(a.grad, out, logits, res)
    spec_score_logprobs(a, _stream(dev))
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
    import torch
    a, dev, f32 = spec_score_distill_args(), student.device, torch.float32
    lead, a.batch, a.tokens, a.vocab = _logits(student, "student")
    k = top_ids.shape[-1] if top_ids.dim() else 0
    a.device, a.dtype, a.teacher_dtype = dev.index, _code(student.dtype, "student"), _code(teacher.dtype, "teacher")
    a.entries, a.tail, a.temperature = k, bool(tail), temperature
    a.teacher_temperature = temperature if teacher_temperature is None else teacher_temperature
    _rows(a.student, student, "student")
    a.ids = _tensor(top_ids, (*lead, k), torch.int32, dev, "top_ids")
    a.teacher = _tensor(teacher, (*lead, k), teacher.dtype, dev, "teacher")
    a.teacher_lse = _tensor(teacher_lse, lead, f32, dev, "teacher_lse")
    a.grad_loss = _tensor(grad_loss, lead, f32, dev, "grad_loss")
    res = {}
    for name, dtype in (("loss", f32), ("accept", f32), ("row_status", torch.int32)):
        t = None if out is None else out.get(name)
        if t is None:
            t = torch.empty(lead, dtype=dtype, device=dev)
            setattr(a, name, t.data_ptr())
        else:
            setattr(a, name, _tensor(t, lead, dtype, dev, f"out['{name}']"))
        res[name] = t
    if grad_loss is not None:
        _grad(a.grad, out, student, res)
    spec_score_distill(a, _stream(dev))
    return res


__all__ = [n for n in dir() if n.startswith("spec_score_") or n.startswith("SPEC_SCORE_")] + \
    ["logprobs", "distill"]
