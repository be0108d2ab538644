"""Block-scaled FP8 on the GPU where its kernels' orders and ranges end."""
import threading

import pytest
import torch

import workloads
from tests import block_reference as R

pytestmark = pytest.mark.gpu

from bit_quantized_b200 import q8  # noqa: E402

DEV = "cuda:0"


def _operands(m, n, k, seed, dtype=torch.bfloat16):
    X = workloads.random_matrix(m, k, torch.float32, seed)
    X.view(-1)[::97] *= 50.0
    W = workloads.random_matrix(n, k, torch.bfloat16, seed + 1, std=0.02)
    return X.to(dtype).to(DEV), q8.q8_quantize_weight_block(W.to(DEV))


@pytest.mark.parametrize("m,n,k", [(1, 128, 1024), (16, 272, 1024), (16, 16, 512), (20, 400, 1024), (50, 128, 896), (100, 256, 256)])
def test_one_group_per_cta_of_a_cluster(m, n, k):
    # a CTA pushes its sums to the others after a single K group, launch upon launch
    X, w = _operands(m, n, k, m + n)
    a = q8.q8_quantize_act_block(X)
    y, mag = R.linear(R.act_value(a.codes, a.scale), R.weight_value(w.codes, w.scale))
    want = q8.q8_linear_fp8_block(a, w)
    R.check(want, y, mag, k, f"{m}x{n}x{k}")
    outs = [f(*args) for _ in range(25) for f, args in ((q8.q8_linear_fp8_block, (a, w)), (q8.q8_linear_fp8_block_dynamic, (X, w)))]
    assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in outs)
    assert q8.q8_get_device_status() == 0


def test_calls_from_two_host_threads():
    # one kernel with several ring lengths, and with them shared-memory sizes
    cases = [_operands(m, n, k, 5) for m, n, k in ((20, 128, 256), (20, 16, 4096), (24, 4096, 512), (30, 272, 8192))]
    want = [q8.q8_linear_fp8_block_dynamic(X, w) for X, w in cases]
    torch.cuda.synchronize()
    bad = []

    def work(order, stream):
        with torch.cuda.stream(stream):
            for i in order * 20:
                Y = q8.q8_linear_fp8_block_dynamic(*cases[i])
                if not torch.equal(Y.view(torch.int16), want[i].view(torch.int16)):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(order, torch.cuda.Stream())) for order in ([0, 1, 2, 3], [3, 2, 1, 0])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and q8.q8_get_device_status() == 0


def test_one_token_with_an_odd_row_stride():
    X, w = _operands(1, 272, 288, 3)
    want = q8.q8_linear_fp8_block_dynamic(X, w)
    odd = torch.as_strided(torch.cat([X[0], X[0, :5]]), (1, 288), (289, 1))
    out = torch.as_strided(torch.zeros(300, dtype=torch.bfloat16, device=DEV), (1, 272), (277, 1))
    a = q8.q8_quantize_act_block(odd)
    ids, p = q8.q8_moe_route(torch.as_strided(X[0], (1, 16), (17, 1)), 2)
    assert ids.tolist() == [torch.sort(X[0, :16].float(), descending=True, stable=True).indices[:2].tolist()]
    for Y in (q8.q8_linear_fp8_block_dynamic(odd, w, out=out), q8.q8_linear_fp8_block(a, w)):
        assert torch.equal(Y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantizers_over_the_whole_range_of_a_type(dtype):
    # group maxima from the type's largest value, where the low part of 1 / S is subnormal, down to the
    # scale's floor and below; within a group, values down to the type's smallest
    big = float(torch.finfo(dtype).max)
    m, k = 128, 1024
    g = torch.Generator().manual_seed(11)
    top = torch.logspace(0, -40, m, base=10.0, dtype=torch.float64)[:, None] * big
    X = top * torch.exp2(-40.0 * torch.rand(m, k, generator=g, dtype=torch.float64) ** 2)
    X[:, ::128] = top                                          # every group's absmax
    X[:, 1::64] = top * (torch.randint(0, 449, (m, 16), generator=g) / 448.0)
    X = (X * torch.where(torch.rand(m, k, generator=g) < 0.5, -1.0, 1.0)).to(dtype)
    assert torch.isfinite(X.float()).all()
    Q, S = R.quant_act(X)
    a = q8.q8_quantize_act_block(X.to(DEV))
    assert torch.equal(a.scale.cpu().double(), S)
    assert torch.equal(a.codes.cpu().float().double(), Q) and torch.equal(torch.signbit(a.codes.cpu().float()), torch.signbit(Q))
    for W in (X, X.flip(0)[:16], X[:16]):                      # 128 x 128 blocks of both ends of the range
        Q, S = R.quant_weight(W)
        w = q8.q8_quantize_weight_block(W.to(DEV).contiguous())
        assert torch.equal(w.scale.cpu().double(), S)
        assert torch.equal(w.codes.cpu().float().double(), Q) and torch.equal(torch.signbit(w.codes.cpu().float()), torch.signbit(Q))


@pytest.mark.parametrize("m,n,k", [(5, 272, 288), (20, 272, 416), (50, 400, 288), (100, 256, 544), (48, 9216, 96), (300, 784, 416)])
def test_activation_codes_with_a_row_stride(m, n, k):
    X, w = _operands(m, n, k, m)
    a = q8.q8_quantize_act_block(X)
    y, mag = R.linear(R.act_value(a.codes, a.scale), R.weight_value(w.codes, w.scale))
    wide = torch.full((m, k + 48), 0x7E, dtype=torch.uint8, device=DEV)     # 448 beside every row
    wide[:, :k] = a.codes.view(torch.uint8)
    s = q8.QActBlock(wide.view(R.F8)[:, :k], a.scale)
    Y = q8.q8_linear_fp8_block(s, w)
    R.check(Y, y, mag, k, f"strided codes {m}x{n}x{k}")
    assert torch.equal(Y.view(torch.int16), q8.q8_linear_fp8_block(a, w).view(torch.int16))


def test_grouped_activation_codes_with_a_row_stride():
    counts, n, k = (33, 0, 140, 7), 272, 416
    m, E = sum(counts), len(counts)
    X = _operands(m, 16, k, 9)[0]
    w = q8.q8_quantize_weight_block(workloads.random_matrix(E * n, k, torch.bfloat16, 3, std=0.02).view(E, n, k).to(DEV))
    a = q8.q8_quantize_act_block(X)
    wide = torch.full((m, k + 16), 0x7E, dtype=torch.uint8, device=DEV)
    wide[:, :k] = a.codes.view(torch.uint8)
    off = torch.tensor([0, 33, 33, 173, 180], dtype=torch.int32, device=DEV)
    Y = q8.q8_linear_fp8_block_grouped(q8.QActBlock(wide.view(R.F8)[:, :k], a.scale), w, off)
    x, lo = R.act_value(a.codes, a.scale), 0
    for e, c in enumerate(counts):
        y, mag = R.linear(x[lo:lo + c], R.weight_value(w.codes[e], w.scale[e]))
        R.check(Y[lo:lo + c], y, mag, k, f"expert {e}")
        lo += c


@pytest.mark.parametrize("offsets,spans", [
    ([-5, 40, 30, 900], [(0, 0, 40), (2, 40, 150)]),           # below 0, falling, past the last row
    ([10, 60, 60, 149], [(0, 10, 60), (2, 60, 149)]),          # rows before the first expert and after the last
    ([200, 300, 400, 500], []), ([0, 0, 0, -7], [])])
def test_grouped_offsets_are_clamped(offsets, spans):
    n, k, m = 144, 256, 150
    X = _operands(m, 16, k, 1)[0]
    w = q8.q8_quantize_weight_block(workloads.random_matrix(3 * n, k, torch.bfloat16, 2, std=0.02).view(3, n, k).to(DEV))
    a = q8.q8_quantize_act_block(X)
    Y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV)
    q8.q8_linear_fp8_block_grouped(a, w, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=Y)
    x, stays = R.act_value(a.codes, a.scale), torch.ones(m, dtype=torch.bool)
    for e, lo, hi in spans:
        y, mag = R.linear(x[lo:hi], R.weight_value(w.codes[e], w.scale[e]))
        R.check(Y[lo:hi], y, mag, k, f"expert {e}")
        stays[lo:hi] = False
    assert (Y[stays.to(DEV)] == 7.0).all()
