"""Block-scaled FP8 on the GPU: quantizers bit for bit, linears within the bound of tests/block_reference.py."""
import pytest
import torch

import workloads
from tests import block_reference as R

pytestmark = pytest.mark.gpu

from bit_quantized_b200 import q8  # noqa: E402

DEV = "cuda:0"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _spiky(m, k, dtype, seed):
    X = workloads.random_matrix(m, k, torch.float32, seed)
    X.view(-1)[::97] *= 50.0
    return X.to(dtype)


def _weight(n, k, seed, experts=None):
    e = 1 if experts is None else experts
    W = workloads.random_matrix(e * n, k, torch.bfloat16, seed, std=0.02)
    return W if experts is None else W.view(e, n, k)


def _same_codes(q, ref):
    assert torch.equal(q.cpu().float().double(), ref)
    assert torch.equal(torch.signbit(q.cpu().float()), torch.signbit(ref))   # -0 keeps its sign


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k", [(1, 32), (1, 4096), (33, 128), (70, 160), (5, 416), (257, 1056)])
def test_act_quantizer(m, k, dtype):
    X = _spiky(m, k, dtype, m + k)
    X[0, :4] = torch.tensor([0.0, -0.0, 1e-30, -1e-12]).to(dtype)
    if m > 2:
        X[1] = 0.0
        X[2] = (X[2].float() * 1e-7).to(dtype)          # below the scale's floor
    big = torch.full((m, k + 16), 9.0, dtype=dtype, device=DEV)
    big[:, :k] = X.to(DEV)
    Q, S = R.quant_act(X)
    for src in (X.to(DEV), big[:, :k]):
        a = q8.q8_quantize_act_block(src)
        _same_codes(a.codes, Q)
        assert torch.equal(a.scale.cpu().double(), S)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e,n,k", [(None, 16, 32), (None, 144, 288), (None, 512, 640), (3, 208, 160)])
def test_weight_quantizer(e, n, k, dtype):
    W = (_weight(n, k, n + k, e).float() * 3).to(dtype)
    W.view(-1, k)[0, :2] = torch.tensor([-0.0, 1e-20]).to(dtype)
    w = q8.q8_quantize_weight_block(W.to(DEV))
    for i in range(1 if e is None else e):
        Q, S = R.quant_weight(W if e is None else W[i])
        _same_codes(w.codes if e is None else w.codes[i], Q)
        assert torch.equal((w.scale if e is None else w.scale[i]).cpu().double(), S)


def _linear_case(m, n, k, dtype, bias, seed=0):
    X = _spiky(m, k, dtype, m + n + k + seed).to(DEV)
    w = q8.q8_quantize_weight_block(_weight(n, k, n + seed).to(DEV))
    b = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(DEV) if bias else None
    a = q8.q8_quantize_act_block(X)
    y, mag = R.linear(R.act_value(a.codes, a.scale), R.weight_value(w.codes, w.scale), b)
    return X, w, b, a, y, mag


LINEAR = [(1, 16, 32), (1, 4096, 1056), (3, 144, 128), (16, 272, 160), (17, 528, 416), (33, 128, 2048), (64, 400, 1312),
          (65, 144, 288), (128, 1040, 544), (129, 256, 1024), (200, 4112, 2080), (256, 528, 96), (257, 128, 1152),
          (300, 272, 800), (515, 784, 416), (640, 4096, 512)]


@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear(m, n, k):
    X, w, b, a, y, mag = _linear_case(m, n, k, DTYPES[(m + n // 16) % 3], bias=m % 2 == 0)
    big = torch.full((m + 3, n + 24), -5.0, dtype=torch.bfloat16, device=DEV)
    Y = q8.q8_linear_fp8_block(a, w, b, out=big[:m, :n])
    R.check(Y, y, mag, k, f"linear {m}x{n}x{k}")
    assert (big[:m, n:] == -5.0).all() and (big[m:] == -5.0).all()
    again = q8.q8_linear_fp8_block(a, w, b)
    assert torch.equal(again.view(torch.int16), Y.contiguous().view(torch.int16))
    D = q8.q8_linear_fp8_block_dynamic(X, w, b)     # quantized inside the call: the same result, bit for bit
    assert torch.equal(D.view(torch.int16), again.view(torch.int16))
    assert q8.q8_get_device_status() == 0


@pytest.mark.parametrize("m", [1, 20, 50])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dynamic_types_and_strides(m, dtype):
    n, k = 272, 1184
    X, w, b, a, y, mag = _linear_case(m, n, k, dtype, True)
    big = torch.full((m, k + 32), 300.0, dtype=dtype, device=DEV)
    big[:, :k] = X
    Y = q8.q8_linear_fp8_block_dynamic(big[:, :k], w, b)
    R.check(Y, y, mag, k, "dynamic")


def test_weight_with_row_stride():
    n, k = 272, 416
    X, w, b, a, y, mag = _linear_case(40, n, k, torch.bfloat16, False)
    wide = torch.zeros(n, k + 48, dtype=torch.uint8, device=DEV)
    wide[:, :k] = w.codes.view(torch.uint8)
    ws = q8.QWeightBlock(wide.view(R.F8)[:, :k], w.scale)
    for x in (a, q8.QActBlock(a.codes, a.scale)):
        R.check(q8.q8_linear_fp8_block(x, ws), y, mag, k, "strided weight")


def test_long_reduction():
    X, w, b, a, y, mag = _linear_case(24, 128, 28672, torch.bfloat16, False)
    R.check(q8.q8_linear_fp8_block(a, w), y, mag, 28672, "long")
    X, w, b, a, y, mag = _linear_case(300, 128, 14336, torch.bfloat16, False)
    R.check(q8.q8_linear_fp8_block(a, w), y, mag, 14336, "long")


def test_many_tiles_per_cta():
    # more tiles than CTA pairs: the persistent loop, its barriers' phases and the store buffers wrap
    X, w, b, a, y, mag = _linear_case(2600, 2064, 416, torch.bfloat16, True)
    R.check(q8.q8_linear_fp8_block(a, w, b), y, mag, 416, "many tiles")


@pytest.mark.parametrize("counts,n,k", [
    ((130, 0, 7, 300), 256, 512), ((1,), 128, 256), ((64,) * 8, 144, 1024), ((3, 250, 0, 0, 129), 528, 160),
    ((0, 0, 5), 16, 32), ((700, 1, 257, 256), 1040, 416)])
@pytest.mark.parametrize("bias", [False, True])
def test_grouped(counts, n, k, bias):
    E, m = len(counts), sum(counts)
    X = _spiky(m, k, torch.bfloat16, m + n).to(DEV)
    w = q8.q8_quantize_weight_block(_weight(n, k, n, E).to(DEV))
    b = torch.randn(E * n, generator=torch.Generator().manual_seed(3)).to(DEV) if bias else None
    off = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device=DEV)
    a = q8.q8_quantize_act_block(X)
    x = R.act_value(a.codes, a.scale)
    big = torch.full((m + 2, n + 24), -5.0, dtype=torch.bfloat16, device=DEV)
    Y = q8.q8_linear_fp8_block_grouped(a, w, off, b, out=big[:m, :n])
    lo = 0
    for e, c in enumerate(counts):
        be = None if b is None else b[e * n:(e + 1) * n]
        y, mag = R.linear(x[lo:lo + c], R.weight_value(w.codes[e], w.scale[e]), be)
        R.check(Y[lo:lo + c], y, mag, k, f"expert {e}")
        lo += c
    assert (big[:m, n:] == -5.0).all() and (big[m:] == -5.0).all()


def test_grouped_uncovered_rows_stay():
    n, k = 144, 256
    X = _spiky(150, k, torch.bfloat16, 1).to(DEV)
    w = q8.q8_quantize_weight_block(_weight(n, k, 2, 3).to(DEV))
    a = q8.q8_quantize_act_block(X)
    Y = torch.full((150, n), 7.0, dtype=torch.bfloat16, device=DEV)
    q8.q8_linear_fp8_block_grouped(a, w, torch.tensor([0, 40, 100, 100], dtype=torch.int32, device=DEV), out=Y)
    assert (Y[100:] == 7.0).all() and (Y[:100] != 7.0).any()
    # offsets out of range are clamped, as the rowwise grouped linear does
    Z = torch.full((150, n), 7.0, dtype=torch.bfloat16, device=DEV)
    q8.q8_linear_fp8_block_grouped(a, w, torch.tensor([-5, 40, 30, 900], dtype=torch.int32, device=DEV), out=Z)
    assert torch.equal(Z[:40], Y[:40]) and torch.isfinite(Z.float()).all()


def test_grouped_many_experts():
    E, n, k = 300, 128, 160
    counts = torch.randint(0, 6, (E,), generator=torch.Generator().manual_seed(8))
    m = int(counts.sum())
    X = _spiky(m, k, torch.float16, 3).to(DEV)
    w = q8.q8_quantize_weight_block(_weight(n, k, 2, E).to(DEV))
    a = q8.q8_quantize_act_block(X)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).to(DEV)
    Y = q8.q8_linear_fp8_block_grouped(a, w, off)
    x = R.act_value(a.codes, a.scale)
    for e in range(0, E, 17):
        lo, hi = int(off[e]), int(off[e + 1])
        y, mag = R.linear(x[lo:hi], R.weight_value(w.codes[e], w.scale[e]))
        R.check(Y[lo:hi], y, mag, k, f"expert {e}")


@pytest.mark.parametrize("m", [8, 100, 400])
def test_captured_and_replayed_on_another_stream(m):
    n, k = 272, 1056
    X, w, b, a, y, mag = _linear_case(m, n, k, torch.bfloat16, True)
    X2 = _spiky(m, k, torch.bfloat16, 77).to(DEV)
    want = q8.q8_linear_fp8_block_dynamic(X2, w, b)
    s = torch.cuda.Stream()
    src, Y = X.clone(), torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(1, q8.q8_workspace_size(q8.Q8_OP_LINEAR_FP8_BLOCK, m, n, k)), dtype=torch.uint8, device=DEV)
    q8.q8_linear_fp8_block_dynamic(src, w, b, out=Y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q8.q8_linear_fp8_block_dynamic(src, w, b, out=Y, workspace=ws)
        q8.q8_linear_fp8_block_dynamic(src, w, b, out=Y, workspace=ws)
    src.copy_(X2)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y.view(torch.int16), want.view(torch.int16))
    # called on a stream that is not the current one, with outputs made by the call
    outs = [q8.q8_linear_fp8_block_dynamic(X2, w, b, stream=s) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in outs)


@pytest.mark.parametrize("m", [16, 100, 640])
def test_weight_requantized_in_place_before_linear(m):
    n, k = 1280, 2048
    X = _spiky(m, k, torch.bfloat16, m).to(DEV)
    Wa, Wb = _weight(n, k, 1).to(DEV), (_weight(n, k, 2).float() * 2).bfloat16().to(DEV)
    ref = q8.q8_linear_fp8_block_dynamic(X, q8.q8_quantize_weight_block(Wb))
    w = q8.q8_quantize_weight_block(Wa)
    for _ in range(3):
        for W in (Wa, Wb):
            st = q8.lib().q8_quantize_weight_block(W.data_ptr(), q8.Q8_BF16, 1, n, k, k, w.codes.data_ptr(),
                                                   w.scale.data_ptr(), torch.cuda.current_stream().cuda_stream)
            assert st == 0
            Y = q8.q8_linear_fp8_block_dynamic(X, w)
        assert torch.equal(Y.view(torch.int16), ref.view(torch.int16))


def test_empty_calls():
    w = q8.q8_quantize_weight_block(_weight(64, 128, 0).to(DEV))
    X = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    assert q8.q8_linear_fp8_block_dynamic(X, w).shape == (0, 64)
    a = q8.q8_quantize_act_block(X)
    assert q8.q8_linear_fp8_block(a, w).shape == (0, 64)


@pytest.mark.parametrize("m,n,k", [
    (5, 19200, 96), (16, 19216, 160),        # more 128-channel tiles than SMs, quantized inside
    (24, 8192, 288), (48, 19200, 64),        # the two-team decode GEMM, split and not
    (96, 4608, 96), (250, 4112, 160),        # tiles with fewer than 257 tokens
    (130, 2048, 1056), (70, 4096, 32)])      # 128-token decode GEMM; one K group
def test_linear_where_the_kernels_change(m, n, k):
    X, w, b, a, y, mag = _linear_case(m, n, k, torch.bfloat16, bias=True, seed=5)
    Y = q8.q8_linear_fp8_block(a, w, b)
    R.check(Y, y, mag, k, f"linear {m}x{n}x{k}")
    D = q8.q8_linear_fp8_block_dynamic(X, w, b)
    assert torch.equal(D.view(torch.int16), Y.view(torch.int16))


def test_calls_that_overlap_on_two_streams():
    cases = [_linear_case(m, n, 1056, torch.bfloat16, True, seed=m) for m, n in ((3, 528), (60, 528), (300, 784), (100, 4608))]
    want = [q8.q8_linear_fp8_block_dynamic(X, w, b) for X, w, b, *_ in cases]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for r in range(10):
        for i, s in enumerate(streams):
            c = (r + 2 * i) % len(cases)
            outs.append((c, q8.q8_linear_fp8_block_dynamic(*cases[c][:3], stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(o.view(torch.int16), want[c].view(torch.int16)) for c, o in outs)
    assert q8.q8_get_device_status() == 0


def test_stack_of_one_and_wrong_stack():
    X, w, b, a, y, mag = _linear_case(40, 272, 288, torch.bfloat16, False)
    one = q8.QWeightBlock(w.codes[None], w.scale[None])
    R.check(q8.q8_linear_fp8_block(a, one), y, mag, 288, "stack of one")
    two = q8.q8_quantize_weight_block(_weight(272, 288, 1, 2).to(DEV))
    for call in (lambda: q8.q8_linear_fp8_block(a, two), lambda: q8.q8_linear_fp8_block_dynamic(X, two)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("m", [1, 2, 4, 5, 9, 16])
@pytest.mark.parametrize("n,k", [(19200, 4096), (14336, 4128), (4096, 14336), (128, 28672)])
def test_few_tokens_over_many_groups(m, n, k):
    # many more K groups per CTA than stages, and with few tokens fewer pieces of a group
    # than quantizing warps: each warp then skips several uses of a stage
    X = _spiky(m, k, torch.bfloat16, m).to(DEV)
    w = q8.q8_quantize_weight_block(_weight(n, k, 3).to(DEV))
    a = q8.q8_quantize_act_block(X)
    want = q8.q8_linear_fp8_block(a, w)
    cols = torch.arange(0, n, max(1, n // 96))
    y, mag = R.linear(R.act_value(a.codes, a.scale), R.weight_value(w.codes, w.scale)[cols])
    R.check(want[:, cols.to(DEV)], y, mag, k, f"{m}x{n}x{k}")
    for _ in range(4):
        assert torch.equal(q8.q8_linear_fp8_block_dynamic(X, w).view(torch.int16), want.view(torch.int16))
    assert q8.q8_get_device_status() == 0
