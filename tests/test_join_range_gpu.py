"""The join at the ends of its range. A row (or head) of finite values whose squares leave fp32 has an
infinite norm: its normed values are 0, so the outputs are the betas and no gradient passes through
the norm, in the kernel as in the formula taken in fp32 (1 / sqrt(inf) = 0). Nothing of it reaches
another row. Equalities are exact: 0 times a finite value is 0, and adding it changes nothing."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from test_join_gpu import make

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("H,d", [(1, 72), (12, 64), (24, 128), (16, 256)])
@pytest.mark.parametrize("size", [1e20, 1e30])
def test_rows_whose_squares_overflow(dt, rms, H, d, size):
    B, T, t = 2, 5, 3
    x = make(B, H, T, d, dt, False, seed=H)
    plain = {n: v.clone() for n, v in x.items()}
    x["X"][1, t] = (x["X"][1, t].float() * size).to(DT[dt])
    x["Z"][0, 0, t] *= size
    names = ("Z", "gate", "scale", "gamma1", "beta1", "gamma2", "beta2")
    kw = dict(rms=rms, act="silu")
    R, Hn = ttt.join_fwd(x["X"], *[x[n] for n in names], **kw)
    R0, H0 = ttt.join_fwd(plain["X"], *[plain[n] for n in names], **kw)
    assert torch.isfinite(R.float()).all() and torch.isfinite(Hn.float()).all()
    # the row of x: h is beta; all others are what they were
    assert torch.equal(Hn[1, t], x["beta2"].to(DT[dt]))
    rest = torch.ones(B, T, dtype=torch.bool, device="cuda")
    rest[1, t] = rest[0, t] = False
    assert torch.equal(R[rest], R0[rest]) and torch.equal(Hn[rest], H0[rest])
    # the head of z: as a head of zeros with the same beta
    zero = {**plain, "Z": plain["Z"].clone()}
    zero["Z"][0, 0, t] = 0
    Rz, Hz = ttt.join_fwd(zero["X"], *[zero[n] for n in names], **kw)
    assert torch.equal(R[0, t], Rz[0, t]) and torch.equal(Hn[0, t], Hz[0, t])

    g = ttt.join_bwd(R, *[x[n] for n in names], x["dR"], x["dH"], **kw)
    assert all(torch.isfinite(v).all() for v in g.values())
    assert torch.equal(g["X"][1, t], x["dR"][1, t]) and (g["Z"][0, 0, t] == 0).all()
    g0 = ttt.join_bwd(R0, *[plain[n] for n in names], x["dR"], x["dH"], **kw)
    assert torch.equal(g["X"][rest], g0["X"][rest]) and torch.equal(g["gate"][rest], g0["gate"][rest])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_alone_of_rows_whose_squares_overflow(dt, rms):
    x = make(2, 1, 3, 768, dt, False, seed=3)
    x["X"][1, 1] = (x["X"][1, 1].float() * 1e25).to(DT[dt])
    _, h = ttt.join_fwd(x["X"], None, pre_gamma=x["gamma2"], pre_beta=x["beta2"], rms=rms)
    assert torch.isfinite(h.float()).all() and torch.equal(h[1, 1], x["beta2"].to(DT[dt]))


def test_nan_and_infinity_stay_in_their_row():
    x = make(2, 4, 3, 64, "fp32", False, seed=4)
    names = ("Z", "gate", "scale", "gamma1", "beta1", "gamma2", "beta2")
    R0, H0 = ttt.join_fwd(x["X"], *[x[n] for n in names])
    x["X"][0, 1, 5] = float("nan")
    x["Z"][1, 2, 0, 7] = float("inf")
    R, Hn = ttt.join_fwd(x["X"], *[x[n] for n in names])
    assert torch.isnan(Hn[0, 1]).all() and torch.isnan(Hn[1, 0]).all()
    rest = torch.ones(2, 3, dtype=torch.bool, device="cuda")
    rest[0, 1] = rest[1, 0] = False
    assert torch.equal(R[rest], R0[rest]) and torch.equal(Hn[rest], H0[rest])
