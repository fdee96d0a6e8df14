"""The oracle of the gated delta rule and of the join, pinned on the CPU: against
the C oracle of the linear layer, numbers worked by hand, and differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import delta as od

F64 = torch.float64


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def case(B=2, Hk=1, H=2, T=5, dk=3, dv=2, N=None):
    r = lambda i, *s: rand(*s, seed=i)  # noqa: E731
    return dict(Q=r(1, B, Hk, T, dk), K=r(2, B, Hk, T, dk), V=r(3, B, H, T, dv),
                eta=torch.sigmoid(r(4, B, H, T)), g=-torch.exp(r(5, B, H, T)),
                W0=r(6, N or B, H, dk, dv))


def test_two_tokens_by_hand():
    one = torch.ones(1, 1, 2, 1, dtype=F64)
    # W = 2; token 1: Wd = 1, rho = 3 - 1 = 2, W = 1 + 0.5 * 2 = 2; token 2: Wd = 1, rho = 2, W = 2
    half = torch.full((1, 1, 2), 0.5, dtype=F64)
    Z, W = od.delta(one, one, 3 * one, half, half.log(), torch.full((1, 1, 1), 2.0, dtype=F64),
                    q_scale=10.0)
    assert Z.flatten().tolist() == [20.0, 20.0] and float(W) == 2.0


def test_forgetting_everything_starts_again():
    x = case()
    x["g"][:, :, 2] = -float("inf")
    Z, W = od.delta(**x, w0_per_seq=True)
    later = {n: t[:, :, 2:] for n, t in x.items() if n not in ("W0", "g")}
    Z2, W2 = od.delta(**later, g=x["g"][:, :, 2:])
    assert torch.equal(Z[:, :, 2:], Z2) and torch.equal(W, W2)


def test_packed_sequences_are_separate_ones():
    x = case(B=1, T=7, N=3)
    Z, W = od.delta(**x, w0_per_seq=True, seq_start=[0, 2, 2, 6])
    part = lambda a, b: {n: t[:, :, a:b] for n, t in x.items() if n != "W0"}  # noqa: E731
    Za, Wa = od.delta(**part(0, 2), W0=x["W0"][:1], w0_per_seq=True)
    Zb, Wb = od.delta(**part(2, 6), W0=x["W0"][2:], w0_per_seq=True)
    assert torch.equal(Z[:, :, :2], Za) and torch.equal(Z[:, :, 2:6], Zb)
    assert not Z[:, :, 6:].any() and torch.equal(W, torch.cat([Wa, x["W0"][1:2], Wb]))


def test_without_gate_it_is_the_online_linear_layer():
    B, H, T, d = 1, 2, 9, 16
    r = lambda i, *s: rand(*s, seed=i).float().numpy()  # noqa: E731
    Q, K, V = r(1, B, H, T, d), 0.3 * r(2, B, H, T, d), r(3, B, H, T, d)
    eta, W0 = np.abs(0.3 * r(4, B, H, T)), 0.2 * r(5, H, d, d)
    Zr, Wr = oracle.linear_primal(Q, K, V, eta, W0, b=1, ln=False)[:2]
    Z, W = od.delta_f64(*(torch.from_numpy(t) for t in (Q, K, V, eta)), None, torch.from_numpy(W0))
    # both in float64: 9 tokens of 16 terms added up in another order, 144 * 2^-53 = 2e-14
    assert np.abs(Z.numpy() - Zr).max() <= 1e-13 * np.abs(Zr).max()
    assert np.abs(W.numpy() - Wr).max() <= 1e-13 * np.abs(Wr).max()


@pytest.mark.parametrize("starts", [None, [0, 2, 2, 5]])
def test_gradients_against_differences(starts):
    """Central differences in float64 with e = 1e-5: the cubic term is e^2 = 1e-10 of the third
    derivative's size, a rounding 2^-53 / e = 1e-11 of the loss's; 1e-7 covers both."""
    x = case(B=2 if starts is None else 1, N=None if starts is None else 3)
    kw = dict(w0_per_seq=True, seq_start=starts, q_scale=0.5)
    Z, W = od.delta(**x, **kw)
    dZ, dW = rand(*Z.shape, seed=11), rand(*W.shape, seed=12)
    g = od.delta_grads(**x, dZ=dZ, dW_out=dW, **kw)

    def loss(y):
        Z, W = od.delta(**y, **kw)
        return float((Z * dZ).sum() + (W * dW).sum())
    for n in x:
        d = rand(*x[n].shape, seed=13)
        num = (loss({**x, n: x[n] + 1e-5 * d}) - loss({**x, n: x[n] - 1e-5 * d})) / 2e-5
        assert abs(num - float((g[n] * d).sum())) <= 1e-7 * (1 + abs(num)), n


@pytest.mark.parametrize("rms,act", [(False, "silu"), (True, "sigmoid")])
def test_join_gradients_against_differences(rms, act):
    B, H, T, d = 1, 2, 3, 4
    D = H * d
    r = lambda i, *s: rand(*s, seed=i)  # noqa: E731
    x = dict(Z=r(2, B, H, T, d), gate=r(3, B, T, D), scale=r(4, D), gamma1=r(5, H, d),
             beta1=r(6, H, d))
    X, g2, b2, dR, dH = r(1, B, T, D), r(7, D), r(8, D), r(9, B, T, D), r(10, B, T, D)
    order = lambda y: (y["Z"], y["gate"], y["scale"], y["gamma1"], y["beta1"])  # noqa: E731

    def loss(y, X=X, g2=g2, b2=b2):
        R = od.join(X, *order(y), rms=rms, act=act)
        return float((R * dR).sum() + (od.norm(R, g2, b2, rms=rms) * dH).sum())
    R = od.join(X, *order(x), rms=rms, act=act)
    g = od.join_grads(R, *order(x), g2, b2, dR, dH, rms=rms, act=act)
    e = 1e-5
    for n in x:
        v = rand(*x[n].shape, seed=13)
        num = (loss({**x, n: x[n] + e * v}) - loss({**x, n: x[n] - e * v})) / (2 * e)
        assert abs(num - float((g[n] * v).sum())) <= 1e-7 * (1 + abs(num)), n
    for n, base, kw in (("X", X, "X"), ("gamma2", g2, "g2"), ("beta2", b2, "b2")):
        v = rand(*base.shape, seed=14)
        num = (loss(x, **{kw: base + e * v}) - loss(x, **{kw: base - e * v})) / (2 * e)
        assert abs(num - float((g[n] * v).sum())) <= 1e-7 * (1 + abs(num)), n


def test_norms_by_hand():
    x = torch.tensor([[1.0, 3.0]], dtype=F64)
    assert torch.allclose(od.norm(x, eps=0.0), torch.tensor([[-1.0, 1.0]], dtype=F64))
    assert torch.allclose(od.norm(x, rms=True, eps=0.0), x / 5.0 ** 0.5)
    # a gate of 0 opens SiLU by nothing and the sigmoid by half
    Z, zero = torch.tensor([[[[1.0, 3.0]]]], dtype=F64), torch.zeros(1, 1, 2, dtype=F64)
    assert not od.join(zero, Z, zero, eps=0.0).any()
    assert torch.allclose(od.join(zero, Z, zero, act="sigmoid", eps=0.0),
                          torch.tensor([[[-0.5, 0.5]]], dtype=F64))
