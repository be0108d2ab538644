"""The router's choice and the expert layer for a few tokens, against 64-bit statements of both.

Bound of the layer.  G and U carry the bound of tests/block_reference.py, dG and
dU.  silu has a slope of at most 1.1, and h = silu(G) U takes expf (2 ulp), an
addition, a division (half an ulp each) and a product in fp32: less than
2^-20 |h| together, so
    dh = 1.1 dG (|U| + dU) + |silu(G)| dU + 2^-20 |h|.
The scale of h's group moves by at most the largest dh over the group's absmax
(rho, plus 2^-23).  A code of h may then be any e4m3 value between the codes of
the ends of its interval; most intervals hold no border and leave it as it is.
The deviation of each h, times |w2|, plus the bound of the second product, times
the weights' magnitudes, bounds y (one more rounding per expert: the weighted
sum), and bf16 adds 2^-8 |y|.  The router's weights are off by expf and two
roundings: 2^-20 relative.
"""
import pytest
import torch

import workloads
from tests import block_reference as R

pytestmark = pytest.mark.gpu

from bit_quantized_b200 import q8  # noqa: E402

DEV = "cuda:0"


def _route_ref(logits, top_k, scoring, renormalize):
    L = logits.double().cpu()
    m, E = L.shape
    ids = torch.full((m, top_k), -1, dtype=torch.int32)
    w = torch.zeros(m, top_k, dtype=torch.float64)
    for t in range(m):
        order = sorted((e for e in range(E) if L[t, e] > -float("inf")), key=lambda e: (-float(L[t, e]), e))
        if not order:
            continue
        ex = torch.exp(L[t] - L[t, order[0]]) if scoring == "softmax" else 1.0 / (1.0 + torch.exp(-L[t]))
        ex[torch.isnan(L[t])] = 0.0
        total = ex.sum()
        pick = order[:top_k]
        ids[t, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
        v = ex[pick]
        if renormalize:
            v = v / v.sum()
        elif scoring == "softmax":
            v = v / total
        w[t, :len(pick)] = v
    return ids, w


@pytest.mark.parametrize("m,E,k", [(1, 1, 1), (1, 16, 2), (7, 33, 5), (64, 128, 8), (130, 512, 16), (3, 4, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scoring,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route(m, E, k, dtype, scoring, renormalize):
    L = (workloads.random_matrix(m, E, torch.float32, m + E) * 2).to(dtype)
    if m > 2:
        L[0] = 0.5                                   # all equal: the lowest indexes
        L[1, ::2] = -float("inf")                    # masked experts
        L[2] = -float("inf")                         # a padding row
        if E > 2:
            L[1, 1] = float("nan")
    wide = torch.zeros(m, E + 3, dtype=dtype, device=DEV)
    wide[:, :E] = L.to(DEV)
    ids, w = q8.q8_moe_route(wide[:, :E], k, scoring, renormalize)
    ref_ids, ref_w = _route_ref(L, k, scoring, renormalize)
    assert torch.equal(ids.cpu(), ref_ids)
    assert ((w.double().cpu() - ref_w).abs() <= 2.0 ** -20 * ref_w).all()


def test_route_extremes():
    big = float(torch.finfo(torch.float32).max)
    L = torch.tensor([[float("inf"), 1.0, big, -big], [-0.0, 0.0, -1e-38, 1e-45], [-200.0, -200.0, -200.0, -200.0]], device=DEV)
    ids, w = q8.q8_moe_route(L, 2)
    assert ids.tolist() == [[0, 2], [3, 0], [0, 1]] and w[0].tolist() == [0.5, 0.5] and w[2].tolist() == [0.5, 0.5]
    ids, w = q8.q8_moe_route(L, 2, scoring="sigmoid")
    assert ids.tolist() == [[0, 2], [3, 0], [0, 1]] and w[2].tolist() == [0.0, 0.0]   # both sigmoids are 0 in fp32


def _bound(k):
    return (18 + R.up(k)) * 2.0 ** -24 * (1 + 2.0 ** -8)


def _layer_ref(X, ids, weights, w13, w2):
    """(y, dy) in float64: the layer and how far the kernel may be from it before bf16's rounding."""
    x = R.act_value(*R.quant_act(X))
    m, hidden = x.shape
    E, _, inter = w2.codes.shape
    ids, weights = ids.cpu().tolist(), weights.double().cpu().tolist()
    y, dy = torch.zeros(m, hidden, dtype=torch.float64), torch.zeros(m, hidden, dtype=torch.float64)
    for e in range(E):
        pairs = [(t, sum(w for i, w in zip(ids[t], weights[t]) if i == e)) for t in range(m) if e in ids[t]]
        if not pairs:
            continue
        rows, wt = torch.tensor([p[0] for p in pairs]), torch.tensor([[p[1]] for p in pairs], dtype=torch.float64)
        gu, mag = R.linear(x[rows], R.weight_value(w13.codes[e], w13.scale[e]))
        G, U, dG, dU = gu[:, :inter], gu[:, inter:], _bound(hidden) * mag[:, :inter], _bound(hidden) * mag[:, inter:]
        silu = G / (1.0 + torch.exp(-G))
        h = silu * U
        dh = 1.1 * dG * (U.abs() + dU) + silu.abs() * dU + 2.0 ** -20 * h.abs() + 1e-40
        Q, S = R.quant_act(h)          # fl32 of h's quotients; h itself is within dh
        Sv = S.T.repeat_interleave(R.BLOCK, 1)[:, :inter]
        group = lambda v: v.reshape(len(pairs), -1, R.BLOCK).amax(2).repeat_interleave(R.BLOCK, 1)  # noqa: E731
        rho = group(dh) / group(h.abs()).clamp_min(448e-8) + 2.0 ** -23
        v = h / Sv
        dv = dh / Sv + v.abs() * 2 * rho + 2.0 ** -24 * v.abs()
        lo, hi = R.e4m3((v - dv).clamp(-448, 448)), R.e4m3((v + dv).clamp(-448, 448))
        dev = torch.maximum((hi - Q).abs(), (lo - Q).abs()) * Sv * (1 + rho) + Q.abs() * Sv * rho
        W = R.weight_value(w2.codes[e], w2.scale[e])
        ye, mag = R.linear(Q * Sv, W)
        de = (dev @ W.abs().T) + _bound(inter) * (mag + dev @ W.abs().T)
        y[rows] += wt * ye
        dy[rows] += wt.abs() * (de + 2.0 ** -22 * (ye.abs() + de)) + 2.0 ** -23 * y[rows].abs()
    return y, dy


def _weights(E, inter, hidden, seed):
    w13 = q8.q8_quantize_weight_block(workloads.random_matrix(E * 2 * inter, hidden, torch.bfloat16, seed, 0.05).view(E, 2 * inter, hidden).to(DEV))
    w2 = q8.q8_quantize_weight_block(workloads.random_matrix(E * hidden, inter, torch.bfloat16, seed + 1, 0.05).view(E, hidden, inter).to(DEV))
    return w13, w2


def _check(Y, X, ids, weights, w13, w2, what=""):
    y, dy = _layer_ref(X, ids, weights, w13, w2)
    err = (Y.double().cpu() - y).abs()
    bad = ~(err <= 2.0 ** -8 * (y.abs() + dy) + dy + 2.0 ** -133)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst {float((err - dy).max())}"
    # the bound is not vacuous: the whole output is near the reference
    assert float(err.norm()) <= 0.01 * float(y.norm()) + 1e-30


def _choice(m, E, k, seed):
    return q8.q8_moe_route((workloads.random_matrix(m, E, torch.float32, seed) * 1.5).to(DEV), k)


CASES = [(1, 4, 1, 128, 128), (1, 16, 2, 1056, 256), (2, 8, 3, 160, 384), (5, 40, 8, 544, 128), (16, 8, 2, 416, 256),
         (17, 6, 2, 288, 128), (31, 64, 4, 256, 256), (33, 4, 4, 1440, 128), (64, 16, 4, 320, 384), (64, 3, 2, 2080, 128),
         (48, 130, 8, 96, 128), (1, 2, 2, 32, 128), (3, 300, 16, 128, 128)]


@pytest.mark.parametrize("m,E,k,hidden,inter", CASES)
def test_layer(m, E, k, hidden, inter):
    dtype = [torch.bfloat16, torch.float16, torch.float32][(m + E) % 3]
    X = workloads.random_matrix(m, hidden, torch.float32, m + hidden)
    X.view(-1)[::61] *= 20.0
    X = X.to(dtype)
    w13, w2 = _weights(E, inter, hidden, E + inter)
    ids, w = _choice(m, E, k, m + 7)
    wide = torch.full((m, hidden + 16), 50.0, dtype=dtype, device=DEV)
    wide[:, :hidden] = X.to(DEV)
    big = torch.full((m + 2, hidden + 8), -5.0, dtype=torch.bfloat16, device=DEV)
    Y = q8.q8_moe_fp8_block(wide[:, :hidden], ids, w, w13, w2, out=big[:m, :hidden])
    assert q8.q8_get_device_status() == 0
    _check(Y, X, ids, w, w13, w2, f"moe {m} {E} {k} {hidden} {inter}")
    assert (big[:m, hidden:] == -5.0).all() and (big[m:] == -5.0).all()
    again = q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2)
    assert torch.equal(again.view(torch.int16), Y.contiguous().view(torch.int16))


def test_layer_skips_and_repeats():
    m, E, hidden, inter = 20, 5, 256, 256
    X = workloads.random_matrix(m, hidden, torch.bfloat16, 3)
    w13, w2 = _weights(E, inter, hidden, 4)
    ids = torch.randint(-2, E + 2, (m, 4), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    ids[0] = -1                                                  # no expert
    ids[1] = torch.tensor([2, 2, 2, 2])                          # the same one four times
    ids[2] = torch.tensor([2**31 - 1, -2**31, E, 0])             # ids of nothing
    w = torch.rand(m, 4, generator=torch.Generator().manual_seed(2))
    w[3, 0] = 0.0
    ids, w = ids.to(DEV), w.to(DEV)
    Y = q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2)
    ok = (ids >= 0) & (ids < E)
    _check(Y, X, torch.where(ok, ids, -1), torch.where(ok, w, 0.0), w13, w2)
    assert (Y[0] == 0).all()
    none = torch.full((m, 4), -1, dtype=torch.int32, device=DEV)
    assert (q8.q8_moe_fp8_block(X.to(DEV), none, w, w13, w2) == 0).all()


def test_layer_every_token_on_one_expert():
    m, E, hidden, inter = 64, 4, 416, 256
    X = workloads.random_matrix(m, hidden, torch.bfloat16, 3)
    X[5] = 0.0
    w13, w2 = _weights(E, inter, hidden, 4)
    ids = torch.full((m, 1), 3, dtype=torch.int32, device=DEV)
    w = torch.ones(m, 1, device=DEV)
    Y = q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2)
    _check(Y, X, ids, w, w13, w2)
    assert (Y[5] == 0).all()


def test_layer_agrees_with_the_grouped_linear():
    # decode and prefill of the same weights: the grouped products with torch's SwiGLU between them
    m, E, k, hidden, inter = 40, 8, 2, 512, 384
    X = workloads.random_matrix(m, hidden, torch.bfloat16, 9).to(DEV)
    w13, w2 = _weights(E, inter, hidden, 10)
    ids, w = _choice(m, E, k, 11)
    Y = q8.q8_moe_fp8_block(X, ids, w, w13, w2)
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
    a = q8.q8_quantize_act_block(X[order // k])
    gu = q8.q8_linear_fp8_block_grouped(a, w13, off).float()
    h = torch.nn.functional.silu(gu[:, :inter]) * gu[:, inter:]
    ye = q8.q8_linear_fp8_block_grouped(q8.q8_quantize_act_block(h), w2, off).float()
    ref = torch.zeros(m, hidden, device=DEV).index_add_(0, order // k, ye * w.flatten()[order][:, None])
    # the grouped path rounds G, U and each expert's output to bf16 on the way (2^-8 each), and those
    # roundings move codes of h (up to 2^-4 of a value): the two agree to a few percent of the output's size
    assert float((Y.float() - ref).norm() / ref.norm()) < 0.05


@pytest.mark.parametrize("m", [1, 24, 64])
def test_captured_with_the_router_and_on_two_streams(m):
    E, k, hidden, inter = 24, 3, 544, 256
    w13, w2 = _weights(E, inter, hidden, 20)
    Xs = [workloads.random_matrix(m, hidden, torch.bfloat16, s).to(DEV) for s in (1, 2, 3)]
    Ls = [(workloads.random_matrix(m, E, torch.float32, s + 50) * 1.5).to(DEV) for s in (1, 2, 3)]

    def step(X, L, out=None, ws=None, stream=None):
        ids, w = q8.q8_moe_route(L, k, stream=stream)
        return q8.q8_moe_fp8_block(X, ids, w, w13, w2, out=out, workspace=ws, stream=stream)

    want = [step(X, L) for X, L in zip(Xs, Ls)]
    torch.cuda.synchronize()
    X, L = Xs[0].clone(), Ls[0].clone()
    ids, w = q8.q8_moe_route(L, k)
    Y = torch.empty_like(want[0])
    ws = torch.full((q8.q8_moe_workspace_size(m, k, E, hidden, inter),), 0xA5, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q8.q8_moe_route(L, k, out=(ids, w))
        q8.q8_moe_fp8_block(X, ids, w, w13, w2, out=Y, workspace=ws)
        q8.q8_moe_route(L, k, out=(ids, w))
        q8.q8_moe_fp8_block(X, ids, w, w13, w2, out=Y, workspace=ws)
    for i in (1, 2, 0, 1):
        X.copy_(Xs[i])
        L.copy_(Ls[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y.view(torch.int16), want[i].view(torch.int16))
    # calls that overlap on two streams, each with what it allocates
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for r in range(12):
        for i, s in ((r % 3, a), ((r + 1) % 3, b)):
            with torch.cuda.stream(s):
                outs.append((i, step(Xs[i], Ls[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(o.view(torch.int16), want[i].view(torch.int16)) for i, o in outs)
    assert q8.q8_get_device_status() == 0


def test_weights_requantized_in_place_before_the_layer():
    m, E, k, hidden, inter = 4, 6, 2, 1024, 512
    X = workloads.random_matrix(m, hidden, torch.bfloat16, 1).to(DEV)
    ids, w = _choice(m, E, k, 2)
    Wa = [workloads.random_matrix(E * 2 * inter, hidden, torch.bfloat16, s, 0.05).to(DEV) for s in (1, 2)]
    Wb = [workloads.random_matrix(E * hidden, inter, torch.bfloat16, s, 0.05).to(DEV) for s in (3, 4)]
    quant = lambda W, n: q8.q8_quantize_weight_block(W.view(E, n, -1))  # noqa: E731
    want = [q8.q8_moe_fp8_block(X, ids, w, quant(Wa[i], 2 * inter), quant(Wb[i], hidden)) for i in (0, 1)]
    w13, w2 = quant(Wa[0], 2 * inter), quant(Wb[0], hidden)
    s = torch.cuda.current_stream().cuda_stream
    for r in range(4):
        i = r % 2
        for W, d, n, kk in ((Wa[i], w13, 2 * inter, hidden), (Wb[i], w2, hidden, inter)):
            assert q8.lib().q8_quantize_weight_block(W.data_ptr(), q8.Q8_BF16, E, n, kk, kk, d.codes.data_ptr(), d.scale.data_ptr(), s) == 0
        Y = q8.q8_moe_fp8_block(X, ids, w, w13, w2)
        assert torch.equal(Y.view(torch.int16), want[i].view(torch.int16))


@pytest.mark.parametrize("m,E,k,hidden,inter", [(16, 64, 8, 1024, 640), (64, 24, 6, 1568, 384), (30, 12, 4, 2048, 512)])
def test_layer_with_tiles_shared_by_several_ctas(m, E, k, hidden, inter):
    # several tiles per CTA, most of them whole, the first and the last shared
    X = workloads.random_matrix(m, hidden, torch.bfloat16, m)
    w13, w2 = _weights(E, inter, hidden, 31)
    ids, w = _choice(m, E, k, 8)
    Y = q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2)
    _check(Y, X, ids, w, w13, w2)
    for _ in range(5):
        assert torch.equal(q8.q8_moe_fp8_block(X.to(DEV), ids, w, w13, w2).view(torch.int16), Y.view(torch.int16))
