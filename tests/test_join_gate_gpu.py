"""The join's gate element by element, relative to each element, over gates from -80 to 80.

With x = 0, no second norm, RMS norms without parameters and fp32 throughout, r = act(gate) n and
dGate = act'(gate) n (dR = 1). Bounds, relative: n is a sum of 64 squares, all positive and added by
pairs and eights (10 roundings at most), its root and two products: 12 * 2^-24. The sigmoid s and its
complement are 1 / (1 + e) and e / (1 + e) with e = exp(-|gate|): e is off by (2 + 1.173 |gate|) 2^-23,
the reciprocal by 2^-22, both are products of at most one more rounding; s (1 - s) has the
reciprocal twice; 4 products more: 4 * 2^-24. Together (2 + 1.173 |gate|) 2^-23 + 2 * 2^-22 + 18 * 2^-24.
NaN passes no comparison. The derivative of SiLU, s (1 + gate (1 - s)), has a root near -1.28: its
error is taken relative to s (1 + |gate| (1 - s)). exp(-80) is 1.8e-35, a normal number."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("far", [20, 80])
@pytest.mark.parametrize("H", [1, 12, 32])
def test_gate_and_its_derivative(act, far, H):
    T, d = 50, 64
    gen = torch.Generator().manual_seed(far + H)
    gate = torch.linspace(-far, far, T * H * d)[torch.randperm(T * H * d, generator=gen)]
    gate = gate.reshape(1, T, H * d).cuda()
    Z = torch.randn(1, H, T, d, generator=gen).cuda()
    x = torch.zeros_like(gate)
    R, _ = ttt.join_fwd(x, Z, gate, rms=True, act=act, want_h=False)
    got = ttt.join_bwd(R, Z, gate, None, None, None, None, None, torch.ones_like(x), None, rms=True,
                       act=act)["gate"]
    g, z = gate.double(), Z.double()
    n = (z / (z.square().mean(-1, keepdim=True) + 1e-5).sqrt()).transpose(1, 2).flatten(2)
    e = torch.exp(-g.abs())
    s, rest = (torch.where(g < 0, p, q) for p, q in ((e / (1 + e), 1 / (1 + e)),
                                                     (1 / (1 + e), e / (1 + e))))
    if act == "silu":
        val, der, size = g * s, s * (1 + g * rest), s * (1 + g.abs() * rest)
    else:
        val, der, size = s, s * rest, s * rest
    tol = (2 + 1.173 * g.abs()) * 2.0 ** -23 + 2 * 2.0 ** -22 + 18 * 2.0 ** -24
    assert ((R.double() - val * n).abs() <= tol * (val * n).abs()).all()
    assert ((got.double() - der * n).abs() <= tol * (size * n).abs()).all()
