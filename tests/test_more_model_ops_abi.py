"""CPU-side checks of the routing, 8-bit and verification operators: every refusal fires
before a HIP call or a dereference (the pointers below are not real), empty requests are
no-ops, and workspaces are checked."""
import ctypes

import pytest
import torch

import segmented_top_selection_amd as st
from segmented_top_selection_amd import model_ops as mo

A, B, C, D, WS = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
F32, BF16, I32, F16, I64, E4M3 = 0, 1, 3, 4, 8, 32
OK, INVALID, NOT_SUPPORTED, TOO_SMALL = 0, 1, 2, 4
NAN, INF = float("nan"), float("inf")


def rows(data=A, stride=64, type=BF16):
    return mo._Rows(data, stride, type)


def rows8(data=A, stride=64, type=E4M3):
    return mo._Rows(data, stride, type)


def matrices(data=A, matrix_stride=64 * 32, stride=64, type=E4M3):
    return mo._Matrices(data, matrix_stride, stride, type)


def filled(cls, base, kw):
    a = cls()
    for name, v in {**base, **kw}.items():
        setattr(a, name, v)
    return a


def route(**kw):
    base = dict(logits=rows(), tokens=10, num_experts=64, k=8, scoring=0, renormalize=1, scale=1.0, bias=C,
                groups=4, kept_groups=2, group_best=2, weights=B, experts=D)
    return mo.entry("segtopk_route")(ctypes.byref(filled(mo._RouteArgs, base, kw)), None)


@pytest.mark.parametrize("kw", [
    dict(logits=rows(None)), dict(logits=rows(A + 1)), dict(logits=rows(stride=63)), dict(logits=rows(type=E4M3)),
    dict(tokens=-1), dict(tokens=2 ** 31 - 1), dict(num_experts=0), dict(num_experts=1025), dict(k=0), dict(k=65),
    dict(k=33), dict(scoring=2), dict(scoring=-1), dict(scale=NAN), dict(scale=INF), dict(bias=C + 2),
    dict(groups=0), dict(groups=65), dict(groups=5), dict(kept_groups=0), dict(kept_groups=5), dict(group_best=0),
    dict(group_best=3), dict(weights=None), dict(weights=B + 2), dict(experts=None), dict(experts=D + 1)])
def test_route_refusals(kw):
    assert route(**kw) == INVALID


def test_route_of_nothing():
    assert route(tokens=0) == route(tokens=0, logits=rows(None)) == OK
    assert mo.entry("segtopk_route")(None, None) == INVALID


def route_backward(logits=None, dlogits=None, experts=C, dweights=D, tokens=10, num_experts=64, k=8, scoring=0,
                   scale=1.0):
    return mo.entry("segtopk_route_backward")(logits or rows(), dlogits or rows(B), experts, dweights, tokens,
                                              num_experts, k, scoring, 1, scale, None)


@pytest.mark.parametrize("kw", [
    dict(logits=rows(None)), dict(logits=rows(stride=63)), dict(dlogits=rows(None)), dict(dlogits=rows(B + 1)),
    dict(dlogits=rows(B, type=F16)), dict(dlogits=rows(B, stride=60)), dict(experts=None), dict(experts=C + 2),
    dict(dweights=None), dict(dweights=D + 1), dict(tokens=-1), dict(num_experts=0), dict(num_experts=2000),
    dict(k=0), dict(k=65), dict(scoring=7), dict(scale=NAN)])
def test_route_backward_refusals(kw):
    assert route_backward(**kw) == INVALID
    assert route_backward(tokens=0) == OK


def test_routing_of_more_than_one_launch_holds():
    for tokens in (2 ** 26 - 3, 2 ** 31 - 2):
        assert route(tokens=tokens) == route_backward(tokens=tokens) == NOT_SUPPORTED


def quantize(x=None, q=None, scales=C, tokens=10, k=2, width=64, position=D, kept=WS):
    return mo.entry("segtopk_quantize_rows")(x or rows(), q or rows8(B), scales, tokens, k, width, position, kept,
                                             None)


@pytest.mark.parametrize("kw", [
    dict(x=rows(None)), dict(x=rows(A + 1)), dict(x=rows(stride=63)), dict(x=rows8()), dict(q=rows(B)),
    dict(q=rows8(None)), dict(q=rows8(B + 8)), dict(q=rows8(B, stride=72)), dict(q=rows8(B, stride=48)),
    dict(scales=None), dict(scales=C + 2), dict(tokens=-1), dict(tokens=2 ** 30, k=2), dict(k=0), dict(width=0),
    dict(width=2 ** 31), dict(position=None), dict(position=D + 2), dict(kept=WS + 4),
    dict(position=None, k=1)])
def test_quantize_rows_refusals(kw):
    assert quantize(**kw) == INVALID


def quantize_blocks(x=None, q=None, scales=C, count=2, rows=32, width=64):
    return mo.entry("segtopk_quantize_blocks")(x or matrices(type=BF16), q or matrices(B), scales, count, rows, width,
                                               None)


@pytest.mark.parametrize("kw", [
    dict(x=matrices(None, type=F32)), dict(x=matrices(A + 2, type=F32)), dict(x=matrices(stride=63, type=F32)),
    dict(x=matrices(-1, type=F32)), dict(x=matrices()), dict(q=matrices(None)), dict(q=matrices(B + 8)),
    dict(q=matrices(B, stride=65)), dict(q=matrices(B, matrix_stride=2050)), dict(q=matrices(B, type=BF16)),
    dict(scales=None), dict(scales=C + 1), dict(count=-1), dict(rows=-1), dict(width=0), dict(width=2 ** 31)])
def test_quantize_blocks_refusals(kw):
    assert quantize_blocks(**kw) == INVALID


def test_quantizers_of_nothing_and_of_too_much():
    assert quantize(tokens=0) == quantize(tokens=0, x=rows(None), position=None) == OK
    assert quantize_blocks(count=0) == quantize_blocks(rows=0) == OK
    # More workgroups than one launch holds.
    wide = 2 ** 31 - 256
    assert quantize(x=rows(stride=wide), q=rows8(B, stride=wide), tokens=1000, width=wide) == NOT_SUPPORTED
    big = dict(x=matrices(matrix_stride=0, stride=wide, type=BF16), q=matrices(B, matrix_stride=0, stride=wide))
    assert quantize_blocks(**big, rows=200, width=wide) == NOT_SUPPORTED


def matmul(**kw):
    base = dict(rows=rows8(), out=rows(B, stride=32), weights=matrices(), row_scales=C, weight_scales=D, offsets=WS,
                num_rows=100, num_experts=4, width=32, depth=64)
    return mo.entry("segtopk_expert_matmul")(ctypes.byref(filled(mo._ExpertMatmulArgs, base, kw)), None)


@pytest.mark.parametrize("kw", [
    dict(rows=rows()), dict(rows=rows8(None)), dict(rows=rows8(A + 8)), dict(rows=rows8(stride=72)),
    dict(rows=rows8(stride=48)), dict(out=rows(None)), dict(out=rows(B + 1)), dict(out=rows(B, stride=31)),
    dict(out=rows8(B)), dict(weights=matrices(None)), dict(weights=matrices(A + 4)),
    dict(weights=matrices(stride=40)), dict(weights=matrices(matrix_stride=100)), dict(weights=matrices(type=F16)),
    dict(row_scales=None), dict(row_scales=C + 2), dict(weight_scales=None), dict(weight_scales=D + 1),
    dict(offsets=None), dict(offsets=WS + 4), dict(num_rows=-1), dict(num_rows=2 ** 31 - 1), dict(num_experts=0),
    dict(num_experts=65536), dict(width=0), dict(width=2 ** 31), dict(depth=0), dict(depth=2 ** 31)])
def test_expert_matmul_refusals(kw):
    assert matmul(**kw) == INVALID


def test_expert_matmul_of_nothing_and_of_too_much():
    assert matmul(num_rows=0) == matmul(num_rows=0, rows=rows8(None)) == OK
    assert mo.entry("segtopk_expert_matmul")(None, None) == INVALID
    most = 2 ** 31 - 2048
    assert matmul(num_rows=most, width=most, out=rows(B, stride=most)) == NOT_SUPPORTED


def dweights(ws=WS, ws_bytes=1 << 40, **kw):
    base = dict(dout=rows(stride=32), rows=rows(B), dweights=matrices(C, type=F32), offsets=D, num_rows=100,
                num_experts=4, width=32, depth=64, accumulate=0)
    return mo.entry("segtopk_expert_dweights")(ctypes.byref(filled(mo._ExpertDweightsArgs, base, kw)), ws, ws_bytes,
                                               None)


@pytest.mark.parametrize("kw", [
    dict(dout=rows(None)), dict(dout=rows(stride=31)), dict(dout=rows(type=E4M3)), dict(rows=rows(None)),
    dict(rows=rows(B, type=F16)), dict(rows=rows(B, stride=63)), dict(dweights=matrices(None, type=F32)),
    dict(dweights=matrices(C + 2, type=F32)), dict(dweights=matrices(C, stride=63, type=F32)),
    dict(dweights=matrices(C, -1, type=F32)), dict(dweights=matrices(C, type=F16)), dict(dweights=matrices(C)),
    dict(offsets=None), dict(offsets=D + 4), dict(num_rows=-1), dict(num_rows=2 ** 31), dict(num_experts=0),
    dict(num_experts=65536), dict(width=0), dict(depth=0), dict(ws=None), dict(ws=WS + 8)])
def test_dweights_refusals(kw):
    assert dweights(**kw) == INVALID


def test_dweights_workspace():
    need = mo.entry("segtopk_expert_dweights_workspace")
    assert need(-1, 4, 32, 64) == need(100, 0, 32, 64) == need(100, 4, 0, 64) == need(100, 4, 32, 2 ** 31) == 0
    assert need(0, 4, 32, 64) == 0
    # Each expert's rows padded to 128, both operands in 8 bits, a scale a column and 128 rows.
    assert need(100, 4, 32, 64) >= 4 * 128 * 96 + 4 * 96 * 4
    assert dweights(ws_bytes=need(100, 4, 32, 64) - 1) == dweights(ws_bytes=-1) == TOO_SMALL
    assert mo.entry("segtopk_expert_dweights")(None, None, 0, None) == INVALID
    most = 2 ** 31 - 2048
    assert dweights(width=most, dout=rows(stride=most), num_experts=65535, ws_bytes=2 ** 62) == NOT_SUPPORTED


def verify(ws=WS, ws_bytes=1 << 40, **kw):
    base = dict(target=rows(), draft=rows(B), draft_tokens=C, id_type=I64, draft_offsets=D, num_drafts=10,
                num_requests=3, vocab=64, temperature=1.0, temperatures=None, accept=A, sample=B, tokens=C, counts=D)
    return mo.entry("segtopk_verify_drafts")(ctypes.byref(filled(mo._VerifyArgs, base, kw)), ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(target=rows(None)), dict(target=rows(A + 1)), dict(target=rows(stride=63)), dict(target=rows(type=E4M3)),
    dict(draft=rows(B + 1)), dict(draft=rows(B, stride=10)), dict(draft=rows(B, type=F32)), dict(draft_tokens=None),
    dict(draft_tokens=C + 4), dict(id_type=F32), dict(draft_offsets=None), dict(draft_offsets=D + 4),
    dict(num_drafts=-1), dict(num_drafts=2 ** 22), dict(num_requests=-1), dict(num_requests=0),
    dict(num_requests=2 ** 22), dict(vocab=0), dict(vocab=2 ** 31), dict(temperature=-0.5), dict(temperature=NAN),
    dict(temperature=INF), dict(temperatures=A + 2), dict(accept=None), dict(accept=A + 1), dict(sample=None),
    dict(sample=B + 2), dict(tokens=None), dict(tokens=C + 4), dict(counts=None), dict(counts=D + 2), dict(ws=None),
    dict(ws=WS + 8)])
def test_verify_refusals(kw):
    assert verify(**kw) == INVALID


def test_verify_workspace():
    need = mo.entry("segtopk_verify_workspace")
    assert need(10, 3, 64) > 0
    assert need(-1, 3, 64) == need(10, -3, 64) == need(10, 3, 0) == need(2 ** 22, 3, 64) == need(0, 0, 64) == 0
    assert verify(ws_bytes=need(10, 3, 64) - 1) == verify(ws_bytes=-1) == TOO_SMALL
    assert verify(num_drafts=0, num_requests=0, ws=None, ws_bytes=0) == OK
    assert mo.entry("segtopk_verify_drafts")(None, None, 0, None) == INVALID
    assert verify(num_drafts=2 ** 21, vocab=2 ** 31 - 1, target=rows(stride=2 ** 31), draft=rows(B, stride=2 ** 31),
                  ws_bytes=2 ** 62) == NOT_SUPPORTED


def test_binding_refuses_host_tensors_and_other_types():
    x, f = torch.zeros(4, 8), torch.zeros(4)
    i32, off = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    x8 = x.to(torch.float8_e4m3fn)
    for call in (lambda: st.route(x, 2), lambda: st.route_backward(x, x, i32), lambda: st.quantize_rows(x),
                 lambda: st.quantize_blocks(x), lambda: st.dispatch_quantized(x, i32),
                 lambda: st.expert_matmul(x8, x, x8[None], x, off), lambda: st.expert_matmul_dweights(x, x, off),
                 lambda: st.verify_drafts(x, off, off, f, f)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: st.route(None, 2), lambda: st.route_backward([1], x, i32), lambda: st.quantize_rows(3),
                 lambda: st.quantize_blocks("t"), lambda: st.dispatch_quantized(x, None),
                 lambda: st.expert_matmul(None, x, x8, x, off), lambda: st.expert_matmul_dweights(None, x, off),
                 lambda: st.verify_drafts(None, off, off, f, f)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        st.route(x, 2, scoring="relu")
