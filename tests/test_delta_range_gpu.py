"""Tokens behind a full forgetting, each measured against its own row. A start weight of 1e8, or one
outlying value, makes the tokens in front of the forgetting 1e8 times those behind it in one chunk:
their sizes must not reach the others' bits through a scale that they share (16 tokens share one).

Keys, queries, values and gradients have a common direction, so that rows are not sums that cancel
by chance; what is left is rho = v - k W, which shrinks as W learns: its terms' sizes are up to
8 times itself (0.3 of v is not common). Tolerance: 8 times the relative bound of the other tests,
5e-5 for gradients and 2e-5 for Z."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from oracle import delta as od
from test_delta_gpu import make

pytestmark = pytest.mark.gpu

T = 150


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


def case(dt, dk, dv, at, big, outlier=None):
    x = make(1, 1, 2, T, dk, dv, dt, seed=1, decay=0.2)
    gen = torch.Generator().manual_seed(at)
    rn = lambda n: torch.randn(x[n].shape, generator=gen)  # noqa: E731
    unit = lambda v: v / v.norm(dim=-1, keepdim=True)  # noqa: E731
    for n in ("Q", "K"):
        x[n] = unit(rn(n) + 1).to(x[n].dtype).cuda()
    x["V"] = (1 + 0.3 * rn("V")).to(x["V"].dtype).cuda()
    x["W0"] = (big * (1 + 0.3 * rn("W0"))).cuda()
    if outlier is not None:
        x["V"][:, :, outlier] *= 1e8
    x["g"][:, :, at] = -300.0
    return x, (1 + 0.3 * rn("V")).cuda()


def off(got, ref, first):
    """Largest error of a token from `first` on, relative to its own largest element."""
    g = got.double().cpu()
    assert torch.isfinite(g).all()
    if g.dim() == 3:
        g, ref = g.unsqueeze(-1), ref.unsqueeze(-1)
    e = (g - ref).abs().amax(-1) / ref.abs().amax(-1)
    return float(e[:, :, first:].max())


# first token behind, start weight, outlying value
PLACES = [(32, 1e8, None), (16, 1e8, None), (48, 1e8, None), (112, 1.0, 97), (40, 1e3, None)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("at,big,outlier", PLACES)
def test_gradients_behind_a_forgetting(dt, dk, dv, at, big, outlier):
    x, dZ = case(dt, dk, dv, at, big, outlier)
    args = [x[n] for n in ("Q", "K", "V", "eta", "g", "W0")]
    got = ttt.delta_bwd(*args, dZ, None, w0_per_seq=True)
    ref = od.delta_grads(*args, dZ, None, w0_per_seq=True)
    for n in ("Q", "K", "V", "eta"):
        assert off(got[n], ref[n], at) <= 4e-4, n


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64)])
@pytest.mark.parametrize("at,big,outlier", PLACES)
def test_read_out_behind_a_forgetting(dt, dk, dv, at, big, outlier):
    x, _ = case(dt, dk, dv, at, big, outlier)
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
    assert off(Z, Zr, at) <= 1.6e-4


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("at,big,outlier", PLACES)
def test_gradient_of_the_decays_behind_a_forgetting(dt, dk, dv, at, big, outlier):
    """A pair of tokens on one side of t counts nothing for g_t: it has left the running sum to the
    last bit of 53, however large it was. At the forgetting itself nothing passes (exp(-300) of it)."""
    x, dZ = case(dt, dk, dv, at, big, outlier)
    args = [x[n] for n in ("Q", "K", "V", "eta", "g", "W0")]
    got = ttt.delta_bwd(*args, dZ, None, w0_per_seq=True)["g"]
    ref = od.delta_grads(*args, dZ, None, w0_per_seq=True)["g"]
    assert off(got, ref, at + 1) <= 4e-4
    assert float(got[:, :, at].abs().max()) <= 1e-12 * float(got.abs().max())
