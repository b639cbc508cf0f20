"""The operators around the selection in a language model.

A router's top-k picks each token's experts: ``sort_ids`` lists the slots
expert by expert, ``dispatch`` copies the tokens into that order, ``combine``
brings the experts' results back with the gate weights applied.  A sampler's
top-k picks the next token: ``embedding`` looks it up, ``policy_loss`` scores
sampled tokens under the model's logits.  The gradients are calls of their own
(``*_backward``, ``policy_loss_grad``); none of them records an autograd graph.

Like ``batched_topk`` these only marshal arguments: tensor metadata is checked
before anything is queued, outputs not given and workspaces are allocated with
torch, and the work runs in the library's HIP kernels, on ``stream`` or the
current stream.  With ``stream`` given, what is allocated or copied here belongs
to that stream too; inputs made on another one must be ready for it, as for
any torch call under ``torch.cuda.stream``.  Matrices need a unit stride along
their rows' elements and non-overlapping rows; others are copied first.
All calls may be captured into a graph.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import KEY_TYPES, SegTopKError, _device_tensor, _raw_stream, library

_FLOAT = {torch.float32: KEY_TYPES["f32"], torch.bfloat16: KEY_TYPES["bf16"],
          torch.float16: KEY_TYPES["f16"]}
_INDEX = {torch.int32: KEY_TYPES["i32"], torch.int64: KEY_TYPES["i64"]}


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("type", ctypes.c_int32)]


class _PolicyLossArgs(ctypes.Structure):
    _fields_ = [("logits", _Rows), ("dlogits", _Rows), ("token_ids", ctypes.c_void_p),
                ("id_type", ctypes.c_int32), ("clip_low", ctypes.c_double),
                ("clip_high", ctypes.c_double), ("kl_coef", ctypes.c_double),
                ("temperature", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("tokens", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("num_segments", ctypes.c_int64), ("segment_offsets", ctypes.c_void_p),
                ("old_logp", ctypes.c_void_p), ("ref_logp", ctypes.c_void_p),
                ("advantages", ctypes.c_void_p), ("loss", ctypes.c_void_p),
                ("logp", ctypes.c_void_p)]


_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_R = ctypes.POINTER(_Rows)
_SIGNATURES = {
    "segtopk_sort_ids_workspace": (_I64, [_I64, _I64]),
    "segtopk_sort_ids": (_I32, [_P, _I32, _I64, _I64, _P, _P, _P, _P, _I64, _P]),
    "segtopk_dispatch_rows": (_I32, [_R, _R, _I64, _I64, _I64, _P, _P, _P]),
    "segtopk_combine_rows": (_I32, [_R, _R, _P, _I32, _I64, _I64, _I64, _P, _P, _P]),
    "segtopk_combine_rows_backward": (_I32, [_R, _R, _R, _P, _P, _I32, _I64, _I64, _I64, _P, _P,
                                             _P]),
    "segtopk_embedding_rows": (_I32, [_R, _R, _P, _I32, _I64, _I64, _I64, _F32, _P]),
    "segtopk_embedding_backward_workspace": (_I64, [_I64, _I64, _I64]),
    "segtopk_embedding_backward": (_I32, [_R, _R, _P, _I32, _I64, _I64, _I64, _F32, _I64, _I32,
                                          _P, _I64, _P]),
    "segtopk_policy_loss_workspace": (_I64, [_I64, _I64, _I64]),
    "segtopk_policy_loss": (_I32, [ctypes.POINTER(_PolicyLossArgs), _P, _I64, _P]),
}


_NO_ROWS = _Rows()
_entries = {}


def entry(name: str):
    """The library's function of that name, with its argument types set."""
    fn = _entries.get(name)
    if fn is None:
        fn = getattr(library(), name)
        fn.restype, fn.argtypes = _SIGNATURES[name]
        _entries[name] = fn
    return fn


def _call(name, *args):
    rc = (_entries.get(name) or entry(name))(*args)
    if rc:
        raise SegTopKError(rc, name)


# Sizes are pure functions of the arguments, and programs repeat few of them.
@functools.lru_cache(maxsize=256)
def _sort_workspace(n, num_segments):
    return entry("segtopk_sort_ids_workspace")(n, num_segments)


@functools.lru_cache(maxsize=256)
def _grad_workspace(n, num_rows, width):
    return entry("segtopk_embedding_backward_workspace")(n, num_rows, width)


@functools.lru_cache(maxsize=256)
def _loss_workspace(tokens, vocab, num_segments):
    return entry("segtopk_policy_loss_workspace")(tokens, vocab, num_segments)


# The current device without torch.cuda's checks; a device tensor is at hand
# where it is asked for.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

# A decode step calls these for microseconds of work each, so what the host does
# counts: names that every call uses are the module's own, a tensor's metadata is
# read once, and the checks of the usual case come before their messages.
_Tensor, _I32T, _I64T, _F32T = torch.Tensor, torch.int32, torch.int64, torch.float32
_empty = torch.empty_strided  # torch.empty takes a third longer to say the same


def _on_its_stream(fn):
    """Runs fn on the device of its first tensor and on the stream asked for."""
    @functools.wraps(fn)
    def wrapped(first, *args, stream=None, **kw):
        if isinstance(first, _Tensor) and first.is_cuda and (
                stream is not None or first.get_device() != _current_device()):
            if stream is not None and stream.device != first.device:
                raise ValueError(f"stream is on {stream.device}, the tensors are on {first.device}")
            with torch.cuda.device(first.device), torch.cuda.stream(stream):
                return fn(first, *args, **kw)
        return fn(first, *args, **kw)
    return wrapped


def _stream(dev):
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _device_of(name, t):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    return t.device


def _there(name, t, dev):
    if not isinstance(t, _Tensor) or t.device != dev:
        _device_tensor(name, t, dev)


def _overlaps(t):
    """Whether a matrix is other than rows with a unit inner stride, apart from each other."""
    return (t.stride(1) != 1 and t.shape[1] > 1) or (t.stride(0) < t.shape[1] and t.shape[0] > 1)


def _matrix(name, t, dev):
    """t as rows with a unit inner stride that do not overlap: (t, number of
    rows, width, the library's view of it)."""
    _there(name, t, dev)
    code, shape = _FLOAT.get(t.dtype), t.shape
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16 (got {t.dtype})")
    if len(shape) != 2:
        raise ValueError(f"{name} must have shape (rows, width) (got {tuple(shape)})")
    rows, width = shape
    if width < 1:
        raise ValueError(f"{name} must be at least one element wide")
    if t.is_contiguous():
        return t, rows, width, _Rows(t.data_ptr(), width, code)
    if _overlaps(t):
        t = t.contiguous()
    return t, rows, width, _rows(t)


def _rows(t):
    # The stride of a single row is never used, and torch may say anything.
    stride, width = t.stride(0), t.shape[1]
    return _Rows(t.data_ptr(), stride if stride > width else width, _FLOAT[t.dtype])


def _result(name, t, dev, rows, width, dtype):
    """An output matrix that the caller gave, checked, or a new one: (t, the
    library's view of it)."""
    if t is None:
        t = _empty((rows, width), (width, 1), dtype=dtype, device=dev)
        return t, _Rows(t.data_ptr(), width, _FLOAT[dtype])
    _there(name, t, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != (rows, width):
        raise ValueError(f"{name} must have shape {(rows, width)} (got {tuple(t.shape)})")
    if _overlaps(t):
        raise ValueError(f"{name} must have a unit inner stride and rows that do not overlap")
    return t, _rows(t)


def _ids(name, t, dev):
    """(t contiguous, the library's code of its type)"""
    _there(name, t, dev)
    code = _INDEX.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be int32 or int64 (got {t.dtype})")
    return (t if t.is_contiguous() else t.contiguous()), code


def _vector(name, t, dev, n):
    _there(name, t, dev)
    if t.dtype != _F32T:
        raise TypeError(f"{name} must be {_F32T} (got {t.dtype})")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},) (got {tuple(t.shape)})")
    return t if t.is_contiguous() else t.contiguous()


def _new(n, dtype, dev):
    return _empty((n,), (1,), dtype=dtype, device=dev)


def _workspace(n, dev):
    # torch's blocks are aligned to 512 bytes.
    return _new(n, torch.uint8, dev) if n else None


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _offsets(name, t, dev):
    """(t contiguous, number of segments)"""
    _there(name, t, dev)
    if t.dtype != _I64T:
        raise TypeError(f"{name} must be int64 (got {t.dtype})")
    shape = t.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError(f"{name} must be 1-D with num_segments + 1 entries")
    return (t if t.is_contiguous() else t.contiguous()), shape[0] - 1


def _slots(position, offsets, dev):
    """(position, offsets, tokens, k, pointer to the number of slots kept)."""
    _there("position", position, dev)
    if position.dtype != _I32T:
        raise TypeError(f"position must be int32 (got {position.dtype})")
    shape = position.shape
    if len(shape) not in (1, 2):
        raise ValueError("position must have shape (tokens, k) or (tokens,)")
    tokens, k = shape if len(shape) == 2 else (shape[0], 1)
    if k < 1:
        raise ValueError("position needs at least one slot a token")
    if not position.is_contiguous():
        position = position.contiguous()
    if offsets is None:
        return position, None, tokens, k, None
    offsets, segments = _offsets("offsets", offsets, dev)
    return position, offsets, tokens, k, offsets.data_ptr() + 8 * segments


def _weights(weights, dev, position, dtype):
    """(weights contiguous, the library's code of their type)"""
    if weights is None:
        return None, _FLOAT[_F32T]
    _there("weights", weights, dev)
    wtype = weights.dtype
    if wtype != _F32T and wtype != dtype:
        raise TypeError(f"weights must be float32 or {dtype} (got {wtype})")
    if weights.shape != position.shape:
        raise ValueError(f"weights must have position's shape {tuple(position.shape)} "
                         f"(got {tuple(weights.shape)})")
    return (weights if weights.is_contiguous() else weights.contiguous()), _FLOAT[wtype]


@_on_its_stream
def sort_ids(ids: torch.Tensor, num_segments: int):
    """The stable sort of ids (int32 or int64, any shape) into num_segments.

    Returns (order, position, offsets):
      order     int32 (n,): the slots by id, equal ids by slot; slots whose id is
                outside [0, num_segments) come last, they are dropped
      position  int32, ids' shape: where each slot went, order's inverse
      offsets   int64 (num_segments + 1,): segment s is
                order[offsets[s]:offsets[s + 1]]; offsets[-1] slots are kept.
                They are batched_topk's segment_offsets.
    """
    dev = _device_of("ids", ids)
    ids, code = _ids("ids", ids, dev)
    n, num_segments = ids.numel(), int(num_segments)
    if num_segments < 0:
        raise ValueError("num_segments must be >= 0")
    order = _new(n, _I32T, dev)
    position = torch.empty_like(ids, dtype=_I32T)
    offsets = _new(num_segments + 1, _I64T, dev)
    need = _sort_workspace(n, num_segments)
    ws = _workspace(need, dev)
    _call("segtopk_sort_ids", ids.data_ptr(), code, n, num_segments, order.data_ptr(),
          position.data_ptr(), offsets.data_ptr(), _ptr(ws), need, _stream(dev))
    return order, position, offsets


@_on_its_stream
def dispatch(x: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor | None = None, *,
             out: torch.Tensor | None = None):
    """Tokens in expert order: out[position[t, j]] = x[t].

    x         (tokens, width)
    position  int32 (tokens, k) from sort_ids, or (tokens,) for k = 1
    offsets   from sort_ids: rows from offsets[-1] on belong to dropped slots
              and are zero; None: every slot is kept
    Returns (tokens * k, width).
    """
    dev = _device_of("x", x)
    x, rows, width, xr = _matrix("x", x, dev)
    position, offsets, tokens, k, kept = _slots(position, offsets, dev)
    if rows != tokens:
        raise ValueError(f"position is for {tokens} tokens, x has {rows} rows")
    out, outr = _result("out", out, dev, tokens * k, width, x.dtype)
    _call("segtopk_dispatch_rows", xr, outr, tokens, k, width, position.data_ptr(), kept,
          _stream(dev))
    return out


@_on_its_stream
def combine(rows: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor | None = None,
            weights: torch.Tensor | None = None, *, out: torch.Tensor | None = None):
    """Rows in expert order summed into their tokens:
    out[t] = sum_j weights[t, j] rows[position[t, j]] over the slots kept.

    rows      (tokens * k, width); rows of dropped slots are not read
    weights   position's shape, float32 or rows' dtype; None: all one
    The sum is held in 32 bits and rounded once.  Returns (tokens, width).
    """
    dev = _device_of("rows", rows)
    position, offsets, tokens, k, kept = _slots(position, offsets, dev)
    rows, n, width, rr = _matrix("rows", rows, dev)
    if n != tokens * k:
        raise ValueError(f"rows must have tokens * k = {tokens * k} rows (got {n})")
    weights, code = _weights(weights, dev, position, rows.dtype)
    out, outr = _result("out", out, dev, tokens, width, rows.dtype)
    _call("segtopk_combine_rows", rr, outr, _ptr(weights), code, tokens, k, width,
          position.data_ptr(), kept, _stream(dev))
    return out


def dispatch_backward(drows: torch.Tensor, position: torch.Tensor,
                      offsets: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
                      stream=None):
    """The gradient of dispatch: dx[t] = sum_j drows[position[t, j]] over the
    slots kept.  Returns (tokens, width)."""
    return combine(drows, position, offsets, out=out, stream=stream)


@_on_its_stream
def combine_backward(dout: torch.Tensor, rows: torch.Tensor | None, position: torch.Tensor,
                     offsets: torch.Tensor | None = None, weights: torch.Tensor | None = None, *,
                     out: torch.Tensor | None = None):
    """The gradients of combine, (drows, dweights):
    drows[position[t, j]] = weights[t, j] dout[t] and
    dweights[t, j] = <dout[t], rows[position[t, j]]>, zero for dropped slots.

    dweights has the weights' dtype and position's shape (float32 without
    weights).  rows None: dweights is not computed, and None.
    """
    dev = _device_of("dout", dout)
    position, offsets, tokens, k, kept = _slots(position, offsets, dev)
    dout, n, width, dr = _matrix("dout", dout, dev)
    if n != tokens:
        raise ValueError(f"position is for {tokens} tokens, dout has {n} rows")
    dtype = dout.dtype
    weights, code = _weights(weights, dev, position, dtype)
    dweights = rr = None
    if rows is not None:
        rows, n, wide, rr = _matrix("rows", rows, dev)
        if rows.dtype != dtype:
            raise TypeError(f"rows must be {dtype} (got {rows.dtype})")
        if n != tokens * k or wide != width:
            raise ValueError(f"rows must have shape {(tokens * k, width)} (got {(n, wide)})")
        dweights = torch.empty_like(position, dtype=_F32T if weights is None else weights.dtype)
    out, outr = _result("out", out, dev, tokens * k, width, dtype)
    _call("segtopk_combine_rows_backward", dr, rr, outr, _ptr(weights), _ptr(dweights), code, tokens,
          k, width, position.data_ptr(), kept, _stream(dev))
    return out, dweights


@_on_its_stream
def embedding(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
              out: torch.Tensor | None = None):
    """out[i] = scale * table[ids[i]], rounded once; zero where ids[i] is outside
    the table.  ids: int32 or int64, any shape.  Returns ids' shape + (width,);
    ``out``, if given, is (number of ids, width) and is returned as it is."""
    dev = _device_of("table", table)
    table, num_rows, width, tr = _matrix("table", table, dev)
    ids, code = _ids("ids", ids, dev)
    n = ids.numel()
    res, rr = _result("out", out, dev, n, width, table.dtype)
    _call("segtopk_embedding_rows", tr, rr, ids.data_ptr(), code, n, num_rows, width, float(scale),
          _stream(dev))
    return res if out is not None or ids.dim() == 1 else res.view(*ids.shape, width)


@_on_its_stream
def embedding_backward(dout: torch.Tensor, ids: torch.Tensor, num_rows: int, *,
                       scale: float = 1.0, padding_id: int | None = None,
                       dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                       accumulate: bool = False):
    """The gradient of embedding in its table, (num_rows, width):
    row v is scale * sum over ids[i] == v of dout[i].

    dout        ids' shape + (width,), or (number of ids, width)
    padding_id  a row without gradient
    dtype       dout's (default) or float32
    accumulate  add to ``out``, which is then required; rows of ids that do not
                occur are left alone
    Sums are held in 32 bits, in the order of the tokens within fixed chunks.
    """
    dev = _device_of("dout", dout)
    ids, code = _ids("ids", ids, dev)
    n, num_rows = ids.numel(), int(num_rows)
    if num_rows < 0:
        raise ValueError("num_rows must be >= 0")
    if dout.dim() != 2 and tuple(dout.shape[:-1]) == tuple(ids.shape):
        dout = dout.reshape(n, dout.shape[-1])
    dout, rows, width, dr = _matrix("dout", dout, dev)
    if rows != n:
        raise ValueError(f"dout must have one row an id ({n}; got {rows})")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if dtype is None:
        dtype = out.dtype if out is not None else dout.dtype
    if dtype != dout.dtype and dtype != _F32T:
        raise TypeError(f"the gradient must be float32 or {dout.dtype} (got {dtype})")
    out, outr = _result("out", out, dev, num_rows, width, dtype)
    need = _grad_workspace(n, num_rows, width)
    ws = _workspace(need, dev)
    _call("segtopk_embedding_backward", dr, outr, ids.data_ptr(), code, n, num_rows, width,
          float(scale), -1 if padding_id is None else int(padding_id), int(bool(accumulate)),
          _ptr(ws), need, _stream(dev))
    return out


def _policy(logits, token_ids, old_logp, advantages, segment_offsets, ref_logp, kl_coef, clip_low,
            clip_high, temperature, grad_scale, dlogits, want_grad):
    dev = _device_of("logits", logits)
    given = logits
    logits, tokens, vocab, lr = _matrix("logits", logits, dev)
    token_ids, code = _ids("token_ids", token_ids, dev)
    if token_ids.shape != (tokens,):
        raise ValueError(f"token_ids must have shape ({tokens},) (got {tuple(token_ids.shape)})")
    old_logp = _vector("old_logp", old_logp, dev, tokens)
    advantages = _vector("advantages", advantages, dev, tokens)
    if ref_logp is not None:
        ref_logp = _vector("ref_logp", ref_logp, dev, tokens)
    elif kl_coef:
        raise ValueError("kl_coef needs ref_logp")
    offsets, segments = _offsets("segment_offsets", segment_offsets, dev)
    loss = _empty((), (), dtype=_F32T, device=dev)
    logp = _new(tokens, _F32T, dev)
    dr = _NO_ROWS
    if want_grad:
        if dlogits is given:
            if logits is not given:
                raise ValueError("dlogits may be the logits only where these have a unit inner "
                                 "stride and rows that do not overlap")
            dr = lr
        else:
            dlogits, dr = _result("dlogits", dlogits, dev, tokens, vocab, logits.dtype)
    a = _PolicyLossArgs(lr, dr, token_ids.data_ptr(), code, clip_low, clip_high, kl_coef,
                        temperature, grad_scale, tokens, vocab, segments, offsets.data_ptr(),
                        old_logp.data_ptr(), _ptr(ref_logp), advantages.data_ptr(),
                        loss.data_ptr(), logp.data_ptr())
    need = _loss_workspace(tokens, vocab, segments)
    ws = _workspace(need, dev)
    _call("segtopk_policy_loss", a, _ptr(ws), need, _stream(dev))
    return loss, logp, dlogits


@_on_its_stream
def policy_loss(logits: torch.Tensor, token_ids: torch.Tensor, old_logp: torch.Tensor,
                advantages: torch.Tensor, segment_offsets: torch.Tensor, *,
                ref_logp: torch.Tensor | None = None, kl_coef: float = 0.0,
                clip_low: float = 0.2, clip_high: float = 0.2, temperature: float = 1.0):
    """The clipped policy loss of sampled tokens, (loss, logp).

    logits           (tokens, vocab): row t is what token_ids[t] was drawn from
    token_ids        int32 or int64 (tokens,); a row whose id is outside
                     [0, vocab) is left out (prompt, padding)
    old_logp         float32 (tokens,), log-probabilities at sampling time
    advantages       float32 (tokens,)
    segment_offsets  int64 (answers + 1,): answer s is rows offsets[s] to
                     offsets[s + 1]; rows outside every answer are left out
    ref_logp         float32 (tokens,), for the KL term of weight kl_coef
    With r = exp(logp - old_logp), a row's term is
      -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
      + kl_coef (exp(ref_logp - logp) - (ref_logp - logp) - 1)
    and the loss is the mean over answers of each answer's mean over its rows.
    Returns the loss (float32, 0-D) and logp (float32, 0 for rows left out).
    """
    return _policy(logits, token_ids, old_logp, advantages, segment_offsets, ref_logp, kl_coef,
                   clip_low, clip_high, temperature, 1.0, None, False)[:2]


@_on_its_stream
def policy_loss_grad(logits: torch.Tensor, token_ids: torch.Tensor, old_logp: torch.Tensor,
                     advantages: torch.Tensor, segment_offsets: torch.Tensor, *,
                     ref_logp: torch.Tensor | None = None, kl_coef: float = 0.0,
                     clip_low: float = 0.2, clip_high: float = 0.2, temperature: float = 1.0,
                     grad_scale: float = 1.0, dlogits: torch.Tensor | None = None):
    """policy_loss and its gradient, (loss, logp, dlogits).

    dlogits is grad_scale * d loss / d logits, of the logits' dtype; it may be
    ``logits`` itself, which is then overwritten.  The other arguments are
    policy_loss's.
    """
    return _policy(logits, token_ids, old_logp, advantages, segment_offsets, ref_logp, kl_coef,
                   clip_low, clip_high, temperature, grad_scale, dlogits, True)
