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
