"""The gated delta rule's backward on the GPU: against float64 autograd through
the token-by-token oracle, and against differences of the forward.

Metric max |gpu - ref| / max |ref| per tensor. Tolerance 5e-5: a gradient passes
the forward's products (at most 128 + 64 terms rounded to fp32 one after the other,
192 * 2^-24 = 1.2e-5 of the sum of their sizes), the reverse scan's (the same) and the
chunk's own (128 + 64 terms more): 3.5e-5 at the worst, and two fp16 terms an
operand, 2^-22 each."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from oracle import delta as od
from test_delta_gpu import err, make, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


TOL = 5e-5


def grads(x, seed=0, dW=True, **kw):
    gen = torch.Generator().manual_seed(1000 + seed)
    dZ = torch.randn(x["V"].shape, generator=gen).cuda()
    dW_out = None
    if dW:
        n = kw["seq_start"].numel() - 1 if kw.get("seq_start") is not None else x["V"].shape[0]
        dW_out = torch.randn((n, x["V"].shape[1], x["Q"].shape[3], x["V"].shape[3]),
                             generator=gen).cuda()
    return ttt.delta_bwd(x["Q"], x["K"], x["V"], x["eta"], x.get("g"), x.get("W0"), dZ, dW_out,
                         **kw), dZ, dW_out


def check(x, tol=TOL, **kw):
    got, dZ, dW_out = grads(x, **kw)
    starts = kw.pop("seq_start", None)
    kw.pop("dW", None), kw.pop("seed", None)
    ref = od.delta_grads(x["Q"], x["K"], x["V"], x["eta"], x.get("g"), x.get("W0"), dZ, dW_out,
                         seq_start=None if starts is None else starts.tolist(), **kw)
    assert set(got) == set(ref)
    for n, r in ref.items():
        assert got[n].dtype == torch.float32 and got[n].shape == r.shape
        assert err(got[n], r) <= tol, n
    return got


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 150])
def test_backward_lengths(dt, T):
    check(make(2, 2, 2, T, 64, 64, dt, seed=T), w0_per_seq=True, q_scale=0.125)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_backward_widths(dk, dv, dt):
    check(make(1, 2, 4, 140, dk, dv, dt, seed=dk + dv), w0_per_seq=True)


def test_backward_shared_weight_and_keys():
    """One key head for three value heads, one start weight for three sequences."""
    x = make(3, 1, 3, 100, 64, 64, seed=3)
    x["W0"] = x["W0"][0].contiguous()
    check(x)


@pytest.mark.parametrize("absent", [("g",), ("W0",), ("g", "W0")])
@pytest.mark.parametrize("dW", [False, True])
def test_backward_missing_inputs(absent, dW):
    x = make(1, 2, 2, 90, 64, 64, seed=4)
    for n in absent:
        del x[n]
    check(x, w0_per_seq="W0" in x, dW=dW)


@pytest.mark.parametrize("starts", [[0, 3, 70, 70, 199, 210], [5, 64, 128], [0, 0, 1, 1, 180],
                                    [10, 10]])
def test_backward_packed(starts):
    x = make(1, 2, 4, 210, 64, 64, seed=len(starts), N=len(starts) - 1)
    got = check(x, w0_per_seq=True, seq_start=offsets(starts))
    outside = torch.ones(210, dtype=torch.bool)
    outside[starts[0]:starts[-1]] = False
    for n in ("Q", "K", "V", "eta", "g"):
        assert (got[n][:, :, outside.cuda()] == 0).all(), n


def test_backward_gates_at_their_ends():
    """Full forgetting, very strong decay, no step, zero keys, queries and gradients."""
    x = make(1, 1, 2, 150, 128, 64, seed=6)
    x["g"][:, :, 7] = -300.0          # exp(g) is 0 in fp32 and in float64's gradients 1e-130
    x["g"][:, 0, 80:96] = -90.0
    x["eta"][:, :, 30:40] = 0
    x["K"][:, :, 35:45] = 0
    x["Q"][:, :, 100:110] = 0
    check(x, w0_per_seq=True)


@pytest.mark.parametrize("size", [1e-12, 1e8])
def test_backward_sizes_of_values(size):
    x = make(1, 1, 1, 100, 64, 64, seed=7)
    x["V"], x["W0"] = (x["V"].float() * size).bfloat16(), x["W0"] * size
    x["K"] = (x["K"].float() * 2e-2).bfloat16()
    check(x, w0_per_seq=True)


def test_backward_against_differences():
    """Along random directions: (L(x + e d) - L(x - e d)) / 2e of the float32 forward. The forward
    is off by 2e-5 of its size at most, so with e = 1e-2 the difference is off by about 2e-3 of the
    sum's terms, and the cubic term by e^2. For a random direction <g, d> is of the size
    |g| |d| / sqrt(n); a fifth of that is allowed, which a gradient that lacks one of its terms
    misses. (The tolerance proper is that of the comparison with autograd above.)"""
    x = make(1, 2, 2, 130, 64, 64, "fp32", seed=8)
    g, dZ, dW_out = grads(x, w0_per_seq=True)
    loss = lambda y: sum((a.double() * b.double()).sum() for a, b in  # noqa: E731
                         zip(ttt.delta_fwd(**y, w0_per_seq=True), (dZ, dW_out)))
    gen = torch.Generator().manual_seed(5)
    for n in g:
        d = torch.randn(x[n].shape, generator=gen).cuda()
        d = d / d.norm() * x[n].norm()
        e = 1e-2
        num = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        assert abs(float(num - (g[n].double() * d.double()).sum())) <= 2e-2 * float(
            g[n].norm() * d.norm()) / x[n].numel() ** 0.5 * 10, n


def test_backward_same_bits_other_stream_and_graph():
    x = make(2, 1, 2, 200, 64, 128, seed=9)
    a, _, _ = grads(x, w0_per_seq=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, dZ, dW_out = grads(x, w0_per_seq=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a[n], b[n]) for n in a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = ttt.delta_bwd(x["Q"], x["K"], x["V"], x["eta"], x["g"], x["W0"], dZ, dW_out,
                          w0_per_seq=True)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], c[n]) for n in a)


def test_backward_refusals():
    x = make(1, 1, 1, 20, 64, 64, seed=10)
    dZ = torch.zeros_like(x["V"], dtype=torch.float32)
    args = [x[n] for n in ("Q", "K", "V", "eta", "g", "W0")]
    with pytest.raises(ValueError, match="dZ"):
        ttt.delta_bwd(*args, dZ.bfloat16(), w0_per_seq=True)
    with pytest.raises(ValueError, match="dW_out"):
        ttt.delta_bwd(*args, dZ, x["W0"][:, :, :32].contiguous(), w0_per_seq=True)
    with pytest.raises(ttt.TTTError):
        ttt.delta_bwd(*args, dZ, w0_per_seq=True, workspace=torch.empty(256, dtype=torch.uint8,
                                                                        device="cuda"))
