"""What the block-scaled entry points refuse, before anything reaches a device (CPU).

Pointers are never dereferenced: every refused call returns from the host
checks.  Calls that pass them stop at the device check where there is no GPU.
"""
import ctypes

import pytest
import torch

from bit_quantized_b200 import build as q8build

q8build.build()
from bit_quantized_b200 import q8  # noqa: E402

L = q8.lib()
P, MIS = 0x10000, 0x10008
NO_GPU = not torch.cuda.is_available()
PASSED = (q8.Q8_ERR_CUDA, q8.Q8_ERR_UNSUPPORTED_ARCH)
BIG = 65535 * 128


def W(n=256, k=256, ld=None, codes=P, scale=P):
    return ctypes.byref(q8.CWeightBlock(codes, scale, n, k, k if ld is None else ld))


def A(m=4, k=256, ld=None, codes=P, scale=P):
    return ctypes.byref(q8.CActBlock(codes, scale, m, k, k if ld is None else ld))


def act(X=P, dt=q8.Q8_BF16, m=4, k=256, ld=256, codes=P, scale=P):
    return L.q8_quantize_act_block(X, dt, m, k, ld, codes, scale, None)


def weight(X=P, dt=q8.Q8_BF16, e=1, n=256, k=256, ld=256, codes=P, scale=P):
    return L.q8_quantize_weight_block(X, dt, e, n, k, ld, codes, scale, None)


def linear(x=None, w=None, bias=None, y=P, ldy=256):
    return L.q8_linear_fp8_block(A() if x is None else x, W() if w is None else w, bias, y, ldy, None)


def dynamic(X=P, dt=q8.Q8_BF16, m=4, k=256, ld=256, w=None, bias=None, y=P, ldy=256, ws=None, wsb=0):
    return L.q8_linear_fp8_block_dynamic(X, dt, m, k, ld, W() if w is None else w, bias, y, ldy, ws, wsb, None)


def grouped(x=None, w=None, e=2, off=P, bias=None, y=P, ldy=128):
    return L.q8_linear_fp8_block_grouped(A() if x is None else x, W() if w is None else w, e, off, bias, y, ldy, None)


def route(logits=P, dt=q8.Q8_F32, m=4, e=16, ld=16, k=2, scoring=0, ids=P, w=P):
    return L.q8_moe_route(logits, dt, m, e, ld, k, scoring, 1, ids, w, None)


WS = q8.q8_moe_workspace_size(4, 2, 8, 256, 128)


def moe(X=P, dt=q8.Q8_BF16, m=4, h=256, ld=256, ids=P, wt=P, k=2, w13=None, w2=None, e=8, y=P, ldy=256, ws=P, wsb=WS):
    return L.q8_moe_fp8_block(X, dt, m, h, ld, ids, wt, k, W(8 * 256, 256) if w13 is None else w13,
                              W(8 * 256, 128) if w2 is None else w2, e, y, ldy, ws, wsb, None)


NULL, SHAPE, ALIGN, DTYPE, SCHEME, WORK = (q8.Q8_ERR_NULL, q8.Q8_ERR_SHAPE, q8.Q8_ERR_ALIGN, q8.Q8_ERR_DTYPE, q8.Q8_ERR_SCHEME,
                                           q8.Q8_ERR_WORKSPACE)


@pytest.mark.parametrize("fn,bad,status", [
    (act, dict(X=None), NULL), (act, dict(codes=None), NULL), (act, dict(scale=None), NULL),
    (act, dict(k=16, ld=16), SHAPE), (act, dict(k=0), SHAPE), (act, dict(m=-1), SHAPE), (act, dict(ld=128), SHAPE),
    (act, dict(m=BIG + 1), SHAPE), (act, dict(k=BIG + 128, ld=BIG + 128), SHAPE),
    (act, dict(dt=q8.Q8_E4M3), DTYPE), (act, dict(dt=-1), DTYPE), (act, dict(X=MIS), ALIGN), (act, dict(ld=260), ALIGN),
    (act, dict(codes=MIS), ALIGN),
    (weight, dict(X=None), NULL), (weight, dict(n=24), SHAPE), (weight, dict(k=48, ld=48), SHAPE), (weight, dict(ld=255), SHAPE),
    (weight, dict(e=-1), SHAPE), (weight, dict(e=65536), SHAPE), (weight, dict(e=65535, n=65536), SHAPE),
    (weight, dict(dt=q8.Q8_S8), DTYPE), (weight, dict(scale=MIS), ALIGN),
    (linear, dict(x=A(k=128)), SHAPE), (linear, dict(x=A(ld=128)), SHAPE), (linear, dict(w=W(n=24)), SHAPE),
    (linear, dict(w=W(k=16)), SHAPE), (linear, dict(ldy=128), SHAPE), (linear, dict(x=A(m=-1)), SHAPE),
    (linear, dict(x=A(m=BIG), w=W(n=BIG), ldy=BIG), SHAPE),
    (linear, dict(x=A(codes=None)), NULL), (linear, dict(x=A(scale=None)), NULL), (linear, dict(w=W(scale=None)), NULL),
    (linear, dict(y=None), NULL), (linear, dict(y=MIS), ALIGN), (linear, dict(ldy=260), ALIGN), (linear, dict(bias=MIS), ALIGN),
    (linear, dict(w=W(ld=264)), ALIGN), (linear, dict(x=A(ld=264)), ALIGN),
    (dynamic, dict(X=None), NULL), (dynamic, dict(k=128), SHAPE), (dynamic, dict(dt=q8.Q8_E4M3), DTYPE),
    (dynamic, dict(ld=128), SHAPE), (dynamic, dict(m=17), WORK), (dynamic, dict(m=17, ws=P, wsb=17 * 256), WORK),
    (dynamic, dict(m=17, ws=0x10010, wsb=1 << 20), ALIGN), (dynamic, dict(X=MIS), ALIGN),
    (grouped, dict(e=0), SHAPE), (grouped, dict(e=513), SHAPE), (grouped, dict(e=3), SHAPE), (grouped, dict(w=W(n=48)), SHAPE),
    (grouped, dict(off=None), NULL), (grouped, dict(off=0x10002), ALIGN), (grouped, dict(ldy=64), SHAPE),
    (grouped, dict(y=None), NULL), (grouped, dict(bias=MIS), ALIGN),
    (route, dict(logits=None), NULL), (route, dict(ids=None), NULL), (route, dict(w=None), NULL), (route, dict(k=0), SHAPE),
    (route, dict(k=17, e=32, ld=32), SHAPE), (route, dict(k=16, e=8), SHAPE), (route, dict(e=513, ld=513), SHAPE),
    (route, dict(e=0), SHAPE), (route, dict(ld=15), SHAPE), (route, dict(m=-1), SHAPE), (route, dict(scoring=2), SCHEME),
    (route, dict(dt=q8.Q8_S32), DTYPE), (route, dict(logits=0x10002), ALIGN), (route, dict(ids=0x10001), ALIGN),
    (moe, dict(X=None), NULL), (moe, dict(ids=None), NULL), (moe, dict(wt=None), NULL), (moe, dict(y=None), NULL),
    (moe, dict(m=65), SHAPE), (moe, dict(m=-1), SHAPE), (moe, dict(k=0), SHAPE), (moe, dict(k=17), SHAPE), (moe, dict(e=0), SHAPE),
    (moe, dict(e=513), SHAPE), (moe, dict(e=4), SHAPE), (moe, dict(h=128), SHAPE), (moe, dict(ld=128), SHAPE),
    (moe, dict(ldy=128), SHAPE), (moe, dict(w2=W(8 * 256, 160), w13=W(8 * 320, 256)), SHAPE),
    (moe, dict(w13=W(8 * 128, 256)), SHAPE), (moe, dict(dt=q8.Q8_S8), DTYPE), (moe, dict(ws=None), WORK), (moe, dict(wsb=WS - 1), WORK),
    (moe, dict(ws=0x10080), ALIGN), (moe, dict(X=MIS), ALIGN), (moe, dict(ldy=260), ALIGN), (moe, dict(ids=0x10002), ALIGN),
])
def test_refused(fn, bad, status):
    assert fn(**bad) == status


@pytest.mark.parametrize("fn", [act, weight, linear, dynamic, grouped, route, moe])
def test_valid_calls_reach_the_device_check(fn):
    if NO_GPU:
        assert fn() in PASSED


def test_injected_failures_reach_the_new_calls():
    for fn in (act, weight, linear, dynamic, grouped, route, moe):
        q8.q8_inject_failure(q8.Q8_ERR_LAUNCH)
        assert fn() == q8.Q8_ERR_LAUNCH


def test_null_structs():
    assert L.q8_linear_fp8_block(None, W(), None, P, 256, None) == NULL
    assert L.q8_linear_fp8_block(A(), None, None, P, 256, None) == NULL
    assert L.q8_moe_fp8_block(P, q8.Q8_BF16, 4, 256, 256, P, P, 2, None, W(), 8, P, 256, P, WS, None) == NULL


def test_empty_calls_are_valid():
    assert act(m=0) == 0 and weight(n=0) == 0 and weight(e=0) == 0 and linear(x=A(m=0)) == 0
    assert dynamic(m=0) == 0 and grouped(x=A(m=0)) == 0 and route(m=0) == 0 and moe(m=0) == 0


def test_workspace_sizes():
    f = q8.q8_workspace_size
    assert f(q8.Q8_OP_LINEAR_FP8_BLOCK, 16, 4096, 4096) == 0
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    assert f(q8.Q8_OP_LINEAR_FP8_BLOCK, 333, 4112, 2080) == up(333 * 2080) + up(4 * 333 * 17)
    assert f(q8.Q8_OP_LINEAR_FP8_BLOCK, BIG + 1, 16, 32) == 2**64 - 1 and f(q8.Q8_OP_LINEAR_FP8_BLOCK, -1, 16, 32) == 0
    g = q8.q8_moe_workspace_size
    assert g(65, 2, 8, 256, 128) == 2**64 - 1 and g(4, 17, 8, 256, 128) == 2**64 - 1 and g(4, 2, 8, 65568, 128) == 2**64 - 1
    assert g(-1, 2, 8, 256, 128) == 0 and 0 < g(1, 1, 1, 32, 128) <= g(1, 2, 8, 32, 128) <= g(64, 16, 512, 4096, 4096)


def test_python_refusals():
    X = torch.zeros(4, 256)
    w = q8.QWeightBlock(torch.zeros(256, 256, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(2, 2))
    for call in (lambda: q8.q8_quantize_act_block(X), lambda: q8.q8_quantize_weight_block(X),
                 lambda: q8.q8_linear_fp8_block_dynamic(X, w), lambda: w.c(), lambda: q8.q8_moe_route(X, 2),
                 lambda: q8.QActBlock(w.codes, w.scale).c(), lambda: q8.q8_moe_fp8_block(X, X, X, w, w)):
        with pytest.raises(ValueError):
            call()


def test_a_stack_is_no_single_weight():
    q = torch.zeros(2, 256, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    w = q8.QWeightBlock(q, torch.zeros(2, 2, 2))
    with pytest.raises(ValueError, match="stack of experts"):
        q8._one_weight(w)
