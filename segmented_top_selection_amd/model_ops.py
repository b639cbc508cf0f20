"""The operators around the selection in a language model.

A router's top-k picks each token's experts: ``sort_ids`` lists the slots
expert by expert, ``dispatch`` copies the tokens into that order, ``combine``
brings the experts' results back with the gate weights applied.  A sampler's
top-k picks the next token: ``embedding`` looks it up, ``policy_loss`` scores
sampled tokens under the model's logits.  The gradients are calls of their own
(``*_backward``, ``policy_loss_grad``); none of them records an autograd graph.

Like ``batched_topk`` these only marshal arguments, in ``_binding`` (built from
csrc_ops/binding.cpp): tensor metadata is checked before anything is queued,
outputs not given and workspaces are allocated with torch, and the work runs in
the library's HIP kernels, on ``stream`` or the current stream.  With ``stream``
given, what is allocated or copied here belongs to that stream too; inputs made
on another one must be ready for it, as for any torch call under
``torch.cuda.stream``, and are kept until that stream has used them.  Matrices
need a unit stride along their rows' elements and non-overlapping rows; others
are copied first.  All calls may be captured into a graph.  Tensors that a call
writes into (``out``, ``dlogits``) count as modified in place for autograd.
"""
from __future__ import annotations

import ctypes

import torch

from . import LIB_PATH, SegTopKError, library


# The C interface for callers with raw pointers: `entry` gives its functions.
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


_entries = {}


def entry(name: str):
    """The library's function of that name, with its argument types set."""
    fn = _entries.get(name)
    if fn is None:
        fn = getattr(library(), name)
        fn.restype, fn.argtypes = _SIGNATURES[name]
        _entries[name] = fn
    return fn


class _NotLoaded:
    """Stands for the compiled binding until the first call, which loads it and the library."""

    def __getattr__(self, name):
        global _native
        library()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the operators' binding is not built; run `python -c 'import "
                               "__graft_entry__; __graft_entry__.build()'` first") from e
        _binding.load(LIB_PATH, SegTopKError)
        _native = _binding
        return getattr(_binding, name)


_native = _NotLoaded()


def _on(stream, name, *args):
    """The call on a stream of the caller's."""
    first = args[0]
    if isinstance(first, torch.Tensor) and first.is_cuda:
        if stream.device != first.device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {first.device}")
        with torch.cuda.stream(stream):
            out = getattr(_native, name)(*args)
        # What the caller may free before that stream has come to it.
        for t in args:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        return out
    return getattr(_native, name)(*args)


def sort_ids(ids: torch.Tensor, num_segments: int, *, stream=None):
    """The stable sort of ids (int32 or int64, any shape) into num_segments.

    Returns (order, position, offsets):
      order     int32 (n,): the slots by id, equal ids by slot; slots whose id is
                outside [0, num_segments) come last, they are dropped
      position  int32, ids' shape: where each slot went, order's inverse
      offsets   int64 (num_segments + 1,): segment s is
                order[offsets[s]:offsets[s + 1]]; offsets[-1] slots are kept.
                They are batched_topk's segment_offsets.
    """
    if stream is not None:
        return _on(stream, "sort_ids", ids, num_segments)
    return _native.sort_ids(ids, num_segments)


def dispatch(x: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor | None = None, *,
             out: torch.Tensor | None = None, stream=None):
    """Tokens in expert order: out[position[t, j]] = x[t].

    x         (tokens, width)
    position  int32 (tokens, k) from sort_ids, or (tokens,) for k = 1
    offsets   from sort_ids: rows from offsets[-1] on belong to dropped slots
              and are zero; None: every slot is kept
    Returns (tokens * k, width).
    """
    if stream is not None:
        return _on(stream, "dispatch", x, position, offsets, out)
    return _native.dispatch(x, position, offsets, out)


def combine(rows: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor | None = None,
            weights: torch.Tensor | None = None, *, out: torch.Tensor | None = None, stream=None):
    """Rows in expert order summed into their tokens:
    out[t] = sum_j weights[t, j] rows[position[t, j]] over the slots kept.

    rows      (tokens * k, width); rows of dropped slots are not read
    weights   position's shape, float32 or rows' dtype; None: all one
    The sum is held in 32 bits and rounded once.  Returns (tokens, width).
    """
    if stream is not None:
        return _on(stream, "combine", rows, position, offsets, weights, out)
    return _native.combine(rows, position, offsets, weights, out)


def dispatch_backward(drows: torch.Tensor, position: torch.Tensor,
                      offsets: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
                      stream=None):
    """The gradient of dispatch: dx[t] = sum_j drows[position[t, j]] over the
    slots kept.  Returns (tokens, width)."""
    return combine(drows, position, offsets, out=out, stream=stream)


def combine_backward(dout: torch.Tensor, rows: torch.Tensor | None, position: torch.Tensor,
                     offsets: torch.Tensor | None = None, weights: torch.Tensor | None = None, *,
                     out: torch.Tensor | None = None, stream=None):
    """The gradients of combine, (drows, dweights):
    drows[position[t, j]] = weights[t, j] dout[t] and
    dweights[t, j] = <dout[t], rows[position[t, j]]>, zero for dropped slots.

    dweights has the weights' dtype and position's shape (float32 without
    weights).  rows None: dweights is not computed, and None.
    """
    if stream is not None:
        return _on(stream, "combine_backward", dout, rows, position, offsets, weights, out)
    return _native.combine_backward(dout, rows, position, offsets, weights, out)


def embedding(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
              out: torch.Tensor | None = None, stream=None):
    """out[i] = scale * table[ids[i]], rounded once; zero where ids[i] is outside
    the table.  ids: int32 or int64, any shape.  Returns ids' shape + (width,);
    ``out``, if given, is (number of ids, width) and is returned as it is."""
    if stream is not None:
        return _on(stream, "embedding", table, ids, scale, out)
    return _native.embedding(table, ids, scale, out)


def embedding_backward(dout: torch.Tensor, ids: torch.Tensor, num_rows: int, *,
                       scale: float = 1.0, padding_id: int | None = None,
                       dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                       accumulate: bool = False, stream=None):
    """The gradient of embedding in its table, (num_rows, width):
    row v is scale * sum over ids[i] == v of dout[i].

    dout        ids' shape + (width,), or (number of ids, width)
    padding_id  a row without gradient
    dtype       dout's (default) or float32
    accumulate  add to ``out``, which is then required; rows of ids that do not
                occur are left alone
    Sums are held in 32 bits, in the order of the tokens within fixed chunks.
    """
    args = dout, ids, num_rows, scale, padding_id, dtype, out, accumulate
    if stream is not None:
        return _on(stream, "embedding_backward", *args)
    return _native.embedding_backward(*args)


def policy_loss(logits: torch.Tensor, token_ids: torch.Tensor, old_logp: torch.Tensor,
                advantages: torch.Tensor, segment_offsets: torch.Tensor, *,
                ref_logp: torch.Tensor | None = None, kl_coef: float = 0.0,
                clip_low: float = 0.2, clip_high: float = 0.2, temperature: float = 1.0, stream=None):
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
    Rows left out may hold anything; NaN or a logit of +inf in any other row
    makes the loss, and that row's gradient, NaN.
    """
    args = (logits, token_ids, old_logp, advantages, segment_offsets, ref_logp, kl_coef, clip_low,
            clip_high, temperature, 1.0, None, False)
    if stream is not None:
        return _on(stream, "policy_loss", *args)
    return _native.policy_loss(*args)


def policy_loss_grad(logits: torch.Tensor, token_ids: torch.Tensor, old_logp: torch.Tensor,
                     advantages: torch.Tensor, segment_offsets: torch.Tensor, *,
                     ref_logp: torch.Tensor | None = None, kl_coef: float = 0.0,
                     clip_low: float = 0.2, clip_high: float = 0.2, temperature: float = 1.0,
                     grad_scale: float = 1.0, dlogits: torch.Tensor | None = None, stream=None):
    """policy_loss and its gradient, (loss, logp, dlogits).

    dlogits is grad_scale * d loss / d logits, of the logits' dtype; it may be
    ``logits`` itself, which is then overwritten.  The other arguments are
    policy_loss's.
    """
    args = (logits, token_ids, old_logp, advantages, segment_offsets, ref_logp, kl_coef, clip_low,
            clip_high, temperature, grad_scale, dlogits, True)
    if stream is not None:
        return _on(stream, "policy_loss", *args)
    return _native.policy_loss(*args)
