"""The block-scaled FP8 operators stated plainly on the CPU, in 64 bits, for the tests.

Rounding steps that the definition has (fl32 of the scale and of the quotient,
e4m3 codes) are taken in 64 bits and rounded once; everything else is exact to
64 bits.

Bounds.  The kernels sum a group of 128 products in four tensor-core steps of
32, each off by at most 2 x 2^-24 of the magnitudes summed (one rounding of the
running sum, as much again inside the step), round the product of the two
scales (2^-24), and add the groups with one FMA rounding each; up to eight
split sums and the bias add one rounding each.  With mag the sum of the
magnitudes of all products, scaled,
    |y - ref| <= (8 + 1 + groups + 8 + 1) 2^-24 (mag + |bias|),
and bf16's rounding adds 2^-8 |y|.
"""
import numpy as np
import torch

BLOCK = 128
F8 = torch.float8_e4m3fn


def up(v, b=BLOCK):
    return -(-v // b)


def e4m3(v):
    """v (float64) to the nearest e4m3 value: 4 significant bits, ties to even, subnormal step 2^-9, at most 448."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 4).clamp_min(-9))
    return torch.copysign((torch.round(v / step) * step).clamp(-448.0, 448.0), v)


def scale_of(amax):
    s = (amax.double() / 448.0).float()
    return torch.maximum(s, torch.tensor(1e-8, dtype=torch.float32)).double()


def quant_act(X):
    """(code values m x k, scales ceil(k/128) x m), both float64."""
    X = X.double().cpu()
    m, k = X.shape
    Q, S = torch.empty_like(X), torch.empty(up(k), m, dtype=torch.float64)
    for j in range(up(k)):
        g = X[:, j * BLOCK:(j + 1) * BLOCK]
        S[j] = scale_of(g.abs().amax(1))
        Q[:, j * BLOCK:(j + 1) * BLOCK] = e4m3((g / S[j][:, None]).float().double())
    return Q, S


def quant_weight(W):
    """(code values n x k, scales ceil(n/128) x ceil(k/128)), both float64."""
    W = W.double().cpu()
    n, k = W.shape
    Q, S = torch.empty_like(W), torch.empty(up(n), up(k), dtype=torch.float64)
    for i in range(up(n)):
        for j in range(up(k)):
            b = W[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            S[i, j] = scale_of(b.abs().max())
            Q[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = e4m3((b / S[i, j]).float().double())
    return Q, S


def act_value(Q, S):
    return Q.double().cpu() * S.double().cpu().T.repeat_interleave(BLOCK, 1)[:, :Q.shape[1]]


def weight_value(Q, S):
    n, k = Q.shape
    return Q.double().cpu() * S.double().cpu().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def linear(x, w, bias=None):
    """(y, mag) in float64 of dequantized operands."""
    y, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        y, mag = y + bias.double().cpu(), mag + bias.double().cpu().abs()
    return y, mag


def check(Y, y, mag, k, what=""):
    """The bound of the module docstring on a bf16 output."""
    got = Y.double().cpu()
    err = (got - y).abs()
    bound = 2.0 ** -8 * y.abs() + (18 + up(k)) * 2.0 ** -24 * (1 + 2.0 ** -8) * mag + 2.0 ** -133
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad.numpy())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outputs outside the bound; first at {i}: "
                             f"got {got[i].item()!r} ref {y[i].item()!r} bound {bound[i].item()!r}")
