"""The expert layer at the sizes of large checkpoints and where its steps meet, within the bound of tests/test_gpu_moe_block.py."""
import pytest
import torch

import workloads
from tests.test_gpu_moe_block import DEV, _check, _choice, _weights

pytestmark = pytest.mark.gpu

from bit_quantized_b200 import q8  # noqa: E402


@pytest.mark.parametrize("m,E,k,hidden,inter", [(1, 8, 4, 7168, 512), (9, 6, 2, 4096, 1408), (40, 4, 2, 7168, 256),
                                                (64, 3, 1, 8192, 128), (2, 3, 2, 512, 8192)])
def test_layer_of_large_hidden_sizes(m, E, k, hidden, inter):
    X = workloads.random_matrix(m, hidden, torch.bfloat16, m + 1)
    w13, w2 = _weights(E, inter, hidden, 5)
    ids, w = _choice(m, E, k, 6)
    Y = q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2)
    _check(Y, X, ids, w, w13, w2, f"{m} {E} {k} {hidden} {inter}")
    for _ in range(5):
        assert torch.equal(q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2).view(torch.int16), Y.view(torch.int16))


def test_padding_rows_of_anything_change_nothing():
    # rows without an expert may hold what a buffer held before
    m, E, k, hidden, inter = 30, 6, 2, 416, 256
    X = workloads.random_matrix(m, hidden, torch.bfloat16, 2)
    w13, w2 = _weights(E, inter, hidden, 7)
    ids, w = _choice(m, E, k, 8)
    ids[::3] = -1
    want = q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2)
    for junk in (float("nan"), float("inf"), -3e38):
        P, pw = X.clone(), w.clone()
        P[::3] = junk
        pw[::3] = junk
        Y = q8.q8_moe_fp8_block(P.to(DEV), ids, pw, w13, w2)
        assert torch.equal(Y.view(torch.int16), want.view(torch.int16)) and (Y[::3] == 0).all()
