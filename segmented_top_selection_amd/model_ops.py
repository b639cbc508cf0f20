"""The operators around the selection in a language model.

A router's top-k picks each token's experts: ``sort_ids`` lists the slots
expert by expert, ``dispatch`` copies the tokens into that order, ``combine``
brings the experts' results back with the gate weights applied.  A sampler's
top-k picks the next token: ``embedding`` looks it up, ``policy_loss`` scores
sampled tokens under the model's logits.  ``route`` is a router's whole selection, from
scores to gate weights; ``dispatch_quantized`` and ``expert_matmul`` are the experts'
products in 8 bits; ``verify_drafts`` says which tokens of a draft model stand.  The
gradients are calls of their own (``*_backward``, ``policy_loss_grad``,
``expert_matmul_dweights``); none of them records an autograd graph.

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


class _Matrices(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("matrix_stride", ctypes.c_int64),
                ("stride", ctypes.c_int64), ("type", ctypes.c_int32)]


class _RouteArgs(ctypes.Structure):
    _fields_ = [("logits", _Rows), ("tokens", ctypes.c_int64), ("num_experts", ctypes.c_int64),
                ("k", ctypes.c_int64), ("scoring", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_double), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int64),
                ("kept_groups", ctypes.c_int64), ("group_best", ctypes.c_int32),
                ("weights", ctypes.c_void_p), ("experts", ctypes.c_void_p)]


class _ExpertMatmulArgs(ctypes.Structure):
    _fields_ = [("rows", _Rows), ("out", _Rows), ("weights", _Matrices),
                ("row_scales", ctypes.c_void_p), ("weight_scales", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("num_rows", ctypes.c_int64),
                ("num_experts", ctypes.c_int64), ("width", ctypes.c_int64),
                ("depth", ctypes.c_int64)]


class _ExpertDweightsArgs(ctypes.Structure):
    _fields_ = [("dout", _Rows), ("rows", _Rows), ("dweights", _Matrices),
                ("offsets", ctypes.c_void_p), ("num_rows", ctypes.c_int64),
                ("num_experts", ctypes.c_int64), ("width", ctypes.c_int64),
                ("depth", ctypes.c_int64), ("accumulate", ctypes.c_int32)]


class _VerifyArgs(ctypes.Structure):
    _fields_ = [("target", _Rows), ("draft", _Rows), ("draft_tokens", ctypes.c_void_p),
                ("id_type", ctypes.c_int32), ("draft_offsets", ctypes.c_void_p),
                ("num_drafts", ctypes.c_int64), ("num_requests", ctypes.c_int64),
                ("vocab", ctypes.c_int64), ("temperature", ctypes.c_double),
                ("temperatures", ctypes.c_void_p), ("accept", ctypes.c_void_p),
                ("sample", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("counts", ctypes.c_void_p)]


_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_F64 = ctypes.c_double
_R = ctypes.POINTER(_Rows)
_M = ctypes.POINTER(_Matrices)
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
    "segtopk_route": (_I32, [ctypes.POINTER(_RouteArgs), _P]),
    "segtopk_route_backward": (_I32, [_R, _R, _P, _P, _I64, _I64, _I64, _I32, _I32, _F64, _P]),
    "segtopk_quantize_rows": (_I32, [_R, _R, _P, _I64, _I64, _I64, _P, _P, _P]),
    "segtopk_quantize_blocks": (_I32, [_M, _M, _P, _I64, _I64, _I64, _P]),
    "segtopk_expert_matmul": (_I32, [ctypes.POINTER(_ExpertMatmulArgs), _P]),
    "segtopk_expert_dweights_workspace": (_I64, [_I64, _I64, _I64, _I64]),
    "segtopk_expert_dweights": (_I32, [ctypes.POINTER(_ExpertDweightsArgs), _P, _I64, _P]),
    "segtopk_verify_workspace": (_I64, [_I64, _I64, _I64]),
    "segtopk_verify_drafts": (_I32, [ctypes.POINTER(_VerifyArgs), _P, _I64, _P]),
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


_SCORING = {"softmax": 0, "sigmoid": 1}


def _scoring(name: str) -> int:
    if name not in _SCORING:
        raise ValueError(f"scoring must be one of {', '.join(_SCORING)} (got {name!r})")
    return _SCORING[name]


def route(logits: torch.Tensor, k: int, *, scoring: str = "softmax",
          bias: torch.Tensor | None = None, groups: int = 1, kept_groups: int | None = None,
          group_best: int = 2, renormalize: bool = True, scale: float = 1.0, stream=None):
    """A router's selection, from logits to gate weights: (weights, experts).

    logits       (tokens, experts)
    scoring      p = "softmax" of a token's logits, or their "sigmoid"
    bias         float32 (experts,), added to p for the choice alone
    groups       experts form this many groups of neighbours; the kept_groups
                 (default: all) best of them, by the sum of their group_best (1
                 or 2) best p + bias, stay in the choice
    renormalize  the chosen p are divided by their sum
    Returns
      weights  float32 (tokens, k): scale p of the chosen
      experts  int32 (tokens, k): the k best by p + bias, best first, ties to the
               lower index; -1, with weight 0, where none is left
    A logit (or bias) of -inf rules an expert out.  Scores are compared in 64 bits.
    ``experts`` is what sort_ids takes, which drops the -1; ``weights`` is combine's.
    At most 1024 experts, 64 groups and k = 64.
    """
    args = (logits, k, _scoring(scoring), bias, groups, kept_groups, group_best, renormalize, scale)
    if stream is not None:
        return _on(stream, "route", *args)
    return _native.route(*args)


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *,
                   scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   out: torch.Tensor | None = None, stream=None):
    """The gradient of route in its logits, of their shape and dtype.

    dweights  float32 (tokens, k), the gradient of route's weights
    experts   int32 (tokens, k), the experts that it chose
    The other arguments are route's; the choice, and with it the bias, has no gradient.
    """
    args = dweights, logits, experts, _scoring(scoring), renormalize, scale, out
    if stream is not None:
        return _on(stream, "route_backward", *args)
    return _native.route_backward(*args)


def quantize_rows(x: torch.Tensor, *, stream=None):
    """Rows in 8 bits with a scale for each 128 columns: (rows, scales).

    x is (rows, width).  Returns float8_e4m3fn of x's shape, its rows 128-byte
    aligned, and float32 (rows, ceil(width / 128)):
    scale = max |x| / 448 over the block (at least 2^-96 / 448), and
    rows = x * (448 / max |x|) rounded to nearest even, so that x is about
    rows * scale.
    """
    if stream is not None:
        return _on(stream, "quantize_rows", x, None, None)
    return _native.quantize_rows(x, None, None)


def quantize_blocks(x: torch.Tensor, *, stream=None):
    """Matrices in 8 bits with a scale for each block of 128 x 128: (matrices, scales).

    x is (rows, width) or (matrices, rows, width), weights for instance; the scales
    are float32 (..., ceil(rows / 128), ceil(width / 128)), made as by quantize_rows.
    """
    if stream is not None:
        return _on(stream, "quantize_blocks", x)
    return _native.quantize_blocks(x)


def dispatch_quantized(x: torch.Tensor, position: torch.Tensor,
                       offsets: torch.Tensor | None = None, *, stream=None):
    """dispatch and quantize_rows in one: tokens in expert order, in 8 bits.

    Takes dispatch's arguments; returns quantize_rows' (rows, scales) with
    tokens * k rows.  Rows of dropped slots, and their scales, are zero.
    """
    if position is None:
        raise TypeError("position must be a torch tensor")
    if stream is not None:
        return _on(stream, "quantize_rows", x, position, offsets)
    return _native.quantize_rows(x, position, offsets)


def expert_matmul(rows: torch.Tensor, row_scales: torch.Tensor, weights: torch.Tensor,
                  weight_scales: torch.Tensor, offsets: torch.Tensor, *,
                  dtype: torch.dtype | None = None, out: torch.Tensor | None = None, stream=None):
    """Each row times its expert's transposed weights, both in 8 bits with scales.

    rows           float8_e4m3fn (rows, depth) in expert order, and
    row_scales     float32 (rows, ceil(depth / 128)): dispatch_quantized's, or
                   quantize_rows' of rows that are in expert order
    weights        float8_e4m3fn (experts, width, depth), and
    weight_scales  float32 (experts, ceil(width / 128), ceil(depth / 128)):
                   quantize_blocks'
    offsets        int64 (experts + 1,) from sort_ids: expert e has the rows
                   offsets[e] to offsets[e + 1]
    dtype          of the result: bfloat16 (default), float16 or float32
    Sums are held in 32 bits; for a result of 16 each eight products are added up with
    the smaller cut off at 2^-13 of the largest, as the 8-bit matrix instruction does.
    Returns (rows, width); rows from offsets[-1] on are zero, those before offsets[0]
    are not written.  Operands whose rows do not begin at multiples of 16 bytes are
    copied first.

    The gradient of the rows is the same call on quantize_rows' of the result's
    gradient, and the weights transposed:
      weights.transpose(1, 2).contiguous(), weight_scales.transpose(1, 2).contiguous()
    """
    args = rows, row_scales, weights, weight_scales, offsets, dtype, out
    if stream is not None:
        return _on(stream, "expert_matmul", *args)
    return _native.expert_matmul(*args)


def expert_matmul_dweights(dout: torch.Tensor, rows: torch.Tensor, offsets: torch.Tensor, *,
                           dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                           accumulate: bool = False, stream=None):
    """The gradient of expert_matmul in its weights, (experts, width, depth):
    for each expert the sum over its rows r of dout[r]^T rows[r].

    dout        (rows, width), the gradient of the result
    rows        (rows, depth) in expert order, of dout's dtype; dispatch's, before
                they are taken to 8 bits
    dtype       dout's (default) or float32
    accumulate  add to ``out``, which is then required
    Both are taken to 8 bits with a scale for each column and 128 rows of an expert;
    sums are expert_matmul's.  Rows from offsets[-1] on are not read.
    """
    args = dout, rows, offsets, dtype, out, accumulate
    if stream is not None:
        return _on(stream, "expert_dweights", *args)
    return _native.expert_dweights(*args)


def verify_drafts(target_logits: torch.Tensor, draft_tokens: torch.Tensor,
                  draft_offsets: torch.Tensor, accept: torch.Tensor, sample: torch.Tensor, *,
                  draft_logits: torch.Tensor | None = None,
                  temperature: float | torch.Tensor = 1.0, stream=None):
    """Which drafted tokens stand, and the token behind them: (tokens, counts).

    target_logits  (drafts + requests, vocab): each request's rows one behind the
                   other, one for each of its drafted tokens and one more
    draft_tokens   int32 or int64 (drafts,)
    draft_offsets  int64 (requests + 1,), from 0 to drafts: request r drafted
                   draft_tokens[draft_offsets[r]:draft_offsets[r + 1]]
    accept         float32 (drafts,), and
    sample         float32 (requests,): uniform numbers in [0, 1)
    draft_logits   (drafts, vocab), what the drafted tokens were drawn from; None:
                   they were certain
    temperature    of both: a number or float32 (requests,); 0: the largest logit
    With p and q the target's and the draft's probabilities, token t stands if
    accept q(t) < p(t).  Behind the last that stands comes one more: drawn from
    max(p - q, 0) at the first that does not, or from p behind all drafts, as the
    lowest index whose running sum passes sample times the whole.
    Returns
      tokens  draft_tokens' dtype (drafts + requests,): request r's from
              draft_offsets[r] + r on, -1 behind its last
      counts  int32 (requests,): how many it gets
    A logit of -inf is a token ruled out.  A row with NaN or +inf, or nothing but
    -inf, has no distribution: its draft does not stand, and no token is drawn (-1).
    """
    args = (target_logits, draft_tokens, draft_offsets, accept, sample, draft_logits, temperature)
    if stream is not None:
        return _on(stream, "verify_drafts", *args)
    return _native.verify_drafts(*args)
