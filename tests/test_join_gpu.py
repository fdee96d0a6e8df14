"""The join between two blocks (norm after, gate, residual scale, residual, norm
before) and its backward on the GPU against the float64 oracle.

Metric: max |gpu - ref| / max |ref| per tensor. fp32 outputs: a row's sums of D
terms, added pairwise by threads and warps and 8 in a thread, are off by less
than 32 roundings, 32 * 2^-24 = 2e-6; the norm's backward subtracts two means,
which are smaller than the largest value; 1e-5 leaves a factor for that. Sums
over rows, up to 500 here, are added one after the other: 500 * 2^-24 = 3e-5 at
worst of the sum of sizes. Stored bf16 adds half a step, 2^-8; h is the norm of
the stored r, and r may differ by one step where the exact r lies next to the
middle of two values: two half steps more for h."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from oracle import delta as od

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL, SUM_TOL = 1e-5, 3e-5
PARAMS = ("scale", "gamma1", "beta1", "gamma2", "beta2")


def make(B, H, T, d, dt, z_bf16, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    D = H * d
    x = dict(X=(2 * rn(B, T, D)).to(DT[dt]), Z=(0.5 * rn(B, H, T, d) + 0.3), gate=rn(B, T, D).to(DT[dt]),
             scale=1 + 0.3 * rn(D), gamma1=1 + 0.1 * rn(H, d), beta1=0.1 * rn(H, d),
             gamma2=1 + 0.1 * rn(D), beta2=0.1 * rn(D), dR=rn(B, T, D), dH=rn(B, T, D))
    x["Z"] = x["Z"].bfloat16() if z_bf16 else x["Z"]
    return {n: t.cuda() for n, t in x.items()}


def err(got, ref):
    got = got.double().cpu().reshape(ref.shape)
    assert torch.isfinite(got).all()
    return float((got - ref).abs().max() / ref.abs().max().clamp_min(1e-30))


def check(x, dt, *, rms, act, eps=1e-5):
    f = lambda n: None if x[n] is None else x[n].double().cpu()  # noqa: E731
    args = [x[n] for n in ("Z", "gate", "scale", "gamma1", "beta1", "gamma2", "beta2")]
    R, Hn = ttt.join_fwd(x["X"], *args, rms=rms, act=act, eps=eps)
    r = od.join(f("X"), f("Z"), f("gate"), f("scale"), f("gamma1"), f("beta1"), rms=rms, act=act,
                eps=eps)
    h = od.norm(R.double().cpu(), f("gamma2"), f("beta2"), rms=rms, eps=eps)
    half = 2.0 ** -8 if dt == "bf16" else 0.0
    assert R.dtype == Hn.dtype == DT[dt]
    assert err(R, r) <= TOL + half and err(Hn, h) <= TOL + half
    g = ttt.join_bwd(R, *args, x["dR"], x["dH"], rms=rms, act=act, eps=eps)
    ref = od.join_grads(R, *args, x["dR"], x["dH"], rms=rms, act=act, eps=eps)
    assert set(g) == set(ref)
    for n, y in ref.items():
        assert g[n].dtype == torch.float32
        assert err(g[n], y) <= (SUM_TOL if n in PARAMS else TOL), n
    return R, Hn, g


@pytest.mark.parametrize("dt,z_bf16", [("bf16", False), ("bf16", True), ("fp32", False),
                                       ("fp32", True)])
@pytest.mark.parametrize("rms,act", [(False, "silu"), (True, "sigmoid")])
@pytest.mark.parametrize("B,H,T,d", [(1, 1, 1, 8), (2, 3, 5, 16), (1, 12, 33, 64), (3, 8, 7, 128),
                                     (1, 16, 3, 256), (2, 1, 4, 1000), (1, 1, 2, 4096),
                                     (1, 40, 500, 32)])
def test_join(B, H, T, d, dt, z_bf16, rms, act):
    check(make(B, H, T, d, dt, z_bf16, seed=H * d + T), dt, rms=rms, act=act)


@pytest.mark.parametrize("dt,z_bf16", [("bf16", False), ("fp32", True)])
@pytest.mark.parametrize("rms,act", [(False, "sigmoid"), (True, "silu")])
@pytest.mark.parametrize("B,H,T,d", [(1, 24, 500, 64), (2, 16, 150, 128), (1, 20, 333, 128),
                                     (1, 1, 190, 2056), (1, 30, 170, 128)])
def test_join_wide_rows(B, H, T, d, dt, z_bf16, rms, act):
    """Rows of more than 1024 channels, in every size of block; more rows than blocks."""
    check(make(B, H, T, d, dt, z_bf16, seed=H + T), dt, rms=rms, act=act)


@pytest.mark.parametrize("absent", [("gate",), ("scale",), ("gamma1", "beta1"), ("beta1", "beta2"),
                                    ("gamma2", "beta2"), ("gate",) + PARAMS])
def test_join_optional_inputs(absent):
    x = make(2, 2, 9, 64, "bf16", False, seed=3)
    for n in absent:
        x[n] = None
    check(x, "bf16", rms=False, act="silu")


def test_norm_alone_and_join_alone():
    x = make(2, 2, 9, 64, "fp32", False, seed=4)
    R, Hn = ttt.join_fwd(x["X"], None, pre_gamma=x["gamma2"], pre_beta=x["beta2"])
    assert R is x["X"]
    f = {n: t.double().cpu() for n, t in x.items()}
    assert err(Hn, od.norm(f["X"], f["gamma2"], f["beta2"])) <= TOL
    g = ttt.join_bwd(x["X"], None, None, None, None, None, x["gamma2"], x["beta2"], None, x["dH"])
    ref = od.join_grads(x["X"], None, None, None, None, None, x["gamma2"], x["beta2"], None, x["dH"])
    assert set(g) == set(ref) and all(err(g[n], ref[n]) <= SUM_TOL for n in ref)
    R, Hn = ttt.join_fwd(x["X"], x["Z"], x["gate"], want_h=False)
    assert Hn is None and err(R, od.join(f["X"], f["Z"], f["gate"])) <= TOL
    g = ttt.join_bwd(R, x["Z"], x["gate"], None, None, None, None, None, x["dR"], None)
    ref = od.join_grads(R, x["Z"], x["gate"], None, None, None, None, None, x["dR"], None)
    assert set(g) == set(ref) and all(err(g[n], ref[n]) <= TOL for n in ref)


def test_rows_without_variance_and_gates_at_their_ends():
    """A constant head (its variance is 0, eps alone is left), zero rows, gates far out."""
    x = make(1, 2, 6, 64, "fp32", False, seed=5)
    x["Z"][:, :, 1] = 3.0
    x["Z"][:, :, 2] = 0.0
    x["gate"][:, 3] = 200.0
    x["gate"][:, 4] = -200.0
    check(x, "fp32", rms=False, act="silu")
    check(x, "fp32", rms=True, act="sigmoid")


def test_repeated_calls_give_the_same_bits():
    x = make(4, 8, 1100, 128, "bf16", False, seed=6)
    args = [x[n] for n in ("Z", "gate", "scale", "gamma1", "beta1", "gamma2", "beta2")]
    a = ttt.join_bwd(x["X"], *args, x["dR"], x["dH"])
    b = ttt.join_bwd(x["X"], *args, x["dR"], x["dH"])
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_join_other_stream_and_graph():
    x = make(2, 2, 50, 64, "bf16", False, seed=7)
    args = [x[n] for n in ("Z", "gate", "scale", "gamma1", "beta1", "gamma2", "beta2")]
    R, Hn = ttt.join_fwd(x["X"], *args)
    g = ttt.join_bwd(R, *args, x["dR"], x["dH"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g2 = ttt.join_bwd(R, *args, x["dR"], x["dH"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g[n], g2[n]) for n in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R3, H3 = ttt.join_fwd(x["X"], *args)
        g3 = ttt.join_bwd(R3, *args, x["dR"], x["dH"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(R3, R) and torch.equal(H3, Hn) and all(torch.equal(g[n], g3[n]) for n in g)


def test_join_refusals():
    x = make(2, 2, 5, 64, "bf16", False, seed=8)
    with pytest.raises(ValueError, match="is not D"):
        ttt.join_fwd(x["X"], x["Z"][:, :1].contiguous())
    with pytest.raises(ValueError, match="act"):
        ttt.join_fwd(x["X"], x["Z"], x["gate"], act="tanh")
    with pytest.raises(ValueError, match="contiguous"):
        ttt.join_fwd(x["X"], x["Z"].transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError, match="shape"):
        ttt.join_fwd(x["X"], x["Z"], scale=x["scale"][:8])
    with pytest.raises(ValueError, match="expected"):
        ttt.join_bwd(x["X"], x["Z"], None, None, None, None, None, None, x["dR"].bfloat16(), None)
    with pytest.raises(ttt.TTTError):
        ttt.join_bwd(x["X"], x["Z"], None, None, None, None, None, None, None, None)  # no gradient
    with pytest.raises(ttt.TTTError):
        y = make(1, 2, 3, 24, "bf16", False)                 # heads of 24 channels
        ttt.join_fwd(y["X"], y["Z"])
