"""The plain block-scaled reference against torch's own e4m3 casts and hand-made values (CPU)."""
import torch

from tests import block_reference as R


def test_e4m3_matches_torch_cast():
    g = torch.Generator().manual_seed(1)
    v = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 9, (20000,), generator=g).float(),
                   torch.arange(-448, 449).float(), torch.arange(-64, 65).float() * 2.0 ** -10]).clamp(-448, 448)
    assert torch.equal(R.e4m3(v.double()), v.to(R.F8).double())


def test_quantizers_on_known_values():
    X = torch.zeros(2, 160)
    X[0, 3], X[0, 150] = 448.0, -0.5
    Q, S = R.quant_act(X)
    assert S.shape == (2, 2) and S[0, 0] == 1.0 and Q[0, 3] == 448.0
    assert S[1, 0] == torch.tensor(0.5 / 448.0).double() and Q[0, 150] == -448.0
    assert (S[:, 1] == torch.tensor(1e-8).double()).all() and (Q[1] == 0).all()
    Qw, Sw = R.quant_weight(X)
    assert Sw.shape == (1, 2) and Sw[0, 0] == 1.0
    y, mag = R.linear(R.act_value(Q, S), R.weight_value(Qw, Sw))
    assert abs(float(y[0, 0]) - 448.0 ** 2 - 0.25) < 1e-3 and float(mag[1, 1]) == 0.0
