"""The operators one after the other, as a layer uses them: delta rule, join, their
backwards; prompts into a pool of states, and decode from it. Each stage is compared
with the float64 oracle on the inputs that the stage before really stored, so that every
tolerance is the operator's own: 2e-5 for the forward rule and 5e-5 for its
gradients (128 + 64 products rounded to fp32 one after the other, 2^-24 each, three times
over for a gradient), 1e-5 for the join and 3e-5 for its sums over rows; a stored bf16
adds half a step, 2^-8. Calls that must agree in every bit are compared for that."""
import threading

import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from oracle import delta as od
from test_delta_gpu import BF16_TOL, err, make, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


FWD, BWD, JOIN, SUMS, HALF = 2e-5, 5e-5, 1e-5, 3e-5, 2.0 ** -8
RULE = ("Q", "K", "V", "eta", "g", "W0")


def block(B, Hk, H, T, d, dt, seed, N=None):
    x = make(B, Hk, H, T, d, d, dt, seed=seed, N=N)
    gen = torch.Generator().manual_seed(seed + 1)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    D, t = H * d, x["Q"].dtype
    y = dict(X=rn(B, T, D).to(t), gate=rn(B, T, D).to(t), scale=1 + 0.2 * rn(D),
             gamma1=1 + 0.1 * rn(H, d), beta1=0.1 * rn(H, d), gamma2=1 + 0.1 * rn(D),
             beta2=0.1 * rn(D), dR=rn(B, T, D), dH=rn(B, T, D))
    return {**x, **{n: v.cuda() for n, v in y.items()}}


def train(x, rms, act, **kw):
    """Forward and backward of the block: everything that it stores."""
    rule = [x[n] for n in RULE]
    Z, W = ttt.delta_fwd(*rule, w0_per_seq=True, **kw)
    tail = [x["gate"], x["scale"], x["gamma1"], x["beta1"], x["gamma2"], x["beta2"]]
    R, Hn = ttt.join_fwd(x["X"], Z, *tail, rms=rms, act=act)
    gj = ttt.join_bwd(R, Z, *tail, x["dR"], x["dH"], rms=rms, act=act)
    gd = ttt.delta_bwd(*rule, gj["Z"], None, w0_per_seq=True, **kw)
    return Z, W, R, Hn, gj, gd


def flatten(out):
    return [*out[:4], *out[4].values(), *out[5].values()]


@pytest.mark.parametrize("B,Hk,H,T,d,dt,starts,rms,act", [
    (2, 2, 2, 100, 64, "bf16", None, False, "silu"),
    (1, 1, 2, 150, 128, "fp32", None, True, "sigmoid"),
    (1, 2, 4, 210, 64, "bf16", [0, 3, 70, 70, 210], True, "silu"),
    (1, 1, 2, 20, 64, "fp32", [0, 1, 20], False, "silu"),
])
def test_a_block_forward_and_backward(B, Hk, H, T, d, dt, starts, rms, act):
    x = block(B, Hk, H, T, d, dt, seed=T, N=None if starts is None else len(starts) - 1)
    kw = {} if starts is None else dict(seq_start=offsets(starts))
    Z, W, R, Hn, gj, gd = train(x, rms, act, **kw)
    f = lambda t: t.double().cpu()  # noqa: E731
    okw = dict(w0_per_seq=True, seq_start=starts)
    Zr, Wr = od.delta_f64(*(x[n] for n in RULE), **okw)
    assert err(Z, Zr) <= FWD and err(W, Wr) <= FWD
    half = HALF if dt == "bf16" else 0.0
    args = [x[n] for n in ("gate", "scale", "gamma1", "beta1", "gamma2", "beta2")]
    r = od.join(f(x["X"]), f(Z), *map(f, args[:4]), rms=rms, act=act)
    h = od.norm(f(R), *map(f, args[4:]), rms=rms)
    assert err(R, r) <= JOIN + half and err(Hn, h) <= JOIN + half
    ref = od.join_grads(R, Z, *args, x["dR"], x["dH"], rms=rms, act=act)
    assert set(ref) == set(gj)
    for n, t in ref.items():
        tol = JOIN if n in ("X", "Z", "gate") else SUMS
        assert err(gj[n].reshape(t.shape), t) <= tol, n
    ref = od.delta_grads(*(x[n] for n in RULE), gj["Z"], None, **okw)
    for n, t in ref.items():
        assert err(gd[n], t) <= BWD, n


@pytest.mark.parametrize("T", [20, 100])
def test_a_block_captured_and_replayed(T):
    """A training step in a graph, while what it is compared with is computed eagerly."""
    x = block(2, 1, 2, T, 64, "bf16", seed=5)
    train(x, True, "silu")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train(x, True, "silu")
    for n in ("V", "X", "dH"):
        x[n].mul_(0.5)
    x["g"].sub_(0.1)
    graph.replay()
    for a, b in zip(flatten(out), flatten(train(x, True, "silu"))):
        assert torch.equal(a, b)
    graph.replay()
    for a, b in zip(flatten(out), flatten(train(x, True, "silu"))):
        assert torch.equal(a, b)


def test_two_graphs_with_a_workspace_each_run_at_once():
    x, y = block(1, 2, 4, 300, 64, "bf16", seed=6), block(1, 2, 4, 300, 64, "bf16", seed=7)
    want = [train(v, True, "silu") for v in (x, y)]
    got, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for v in (x, y):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):  # its own pool, so its own workspaces
            got.append(train(v, True, "silu"))
    for _ in range(5):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(flatten(a), flatten(b)))


def test_two_threads_and_streams_at_once():
    xs = [block(1, 1, 2, 260, 64, "bf16", seed=8 + i) for i in range(4)]
    want = [flatten(train(x, False, "silu")) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream() if i < 2 else torch.cuda.default_stream()  # 2 and 3 share one
        with torch.cuda.stream(s):
            for _ in range(10):
                got = flatten(train(xs[i], False, "silu"))
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_memory_of_a_call_on_another_stream_is_not_reused_early():
    """The call waits on its stream behind a long one; what the caller drops meanwhile must not be
    given to the current stream's next tensors."""
    x = block(2, 2, 2, 200, 64, "bf16", seed=12)
    want = flatten(train(x, True, "silu"))
    side, n = torch.cuda.Stream(), 8192
    slow = torch.randn(n, n, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            slow = slow @ slow * 1e-4
    y = {k: t.clone() for k, t in x.items()}
    rule = [y[k] for k in RULE]
    Z, W = ttt.delta_fwd(*rule, w0_per_seq=True, stream=side)
    del rule, y
    junk = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(64)]
    side.synchronize()
    assert torch.equal(Z, want[0]) and torch.equal(W, want[1])
    del junk


@pytest.mark.parametrize("T", [7, 24, 25, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_then_decode_from_the_pool(T, d):
    """A ragged batch of prompts into a pool, then tokens one by one, against the whole."""
    more, H = 5, 2
    x = make(1, 1, H, 3 * (T + more), d, d, "bf16", seed=T + d, N=3)
    at = [0, T, T + 1, T + 1 + (T + 3) // 2]                       # prompts of T, 1, ..
    take = lambda spans: {n: torch.cat([x[n][:, :, a:b] for a, b in spans], 2).contiguous()  # noqa: E731
                          for n in RULE[:5]}
    whole = [(n * (T + more), n * (T + more) + at[n + 1] - at[n] + more) for n in range(3)]
    y = take([(a, b - more) for a, b in whole])
    Z, W = ttt.delta_fwd(**y, W0=x["W0"], w0_per_seq=True, seq_start=offsets(at))
    pool = torch.zeros(6, H, d, d, device="cuda")
    index = torch.tensor([4, 0, -1, 2], dtype=torch.int32, device="cuda")  # row 2: padding
    pool[[4, 0, 2]] = W
    kept = pool[[1, 3, 5]].clone()
    rows = [0, 1, None, 2]
    zs = []
    for t in range(more):
        step = {n: torch.stack([x[n][0, :, (whole[r][1] - more + t) if r is not None else 0]
                                for r in rows]).contiguous() for n in RULE[:5]}
        for n in RULE[:5]:
            step[n][2] = float("nan")                              # nothing of padding is used
        z = torch.full((4, H, d), 7.0, device="cuda")
        ttt.delta_decode(*(step[k] for k in ("Q", "K", "V", "eta", "g")), pool, state_index=index,
                         z=z)
        assert bool((z[2] == 7).all())
        zs.append(z[[0, 1, 3]])
    assert torch.equal(pool[[1, 3, 5]], kept)
    full = take(whole)
    starts = [0]
    for a, b in whole:
        starts.append(starts[-1] + b - a)
    Zr, Wr = od.delta_f64(*(full[n] for n in RULE[:5]), x["W0"], w0_per_seq=True, seq_start=starts)
    # the prompts' weights are off by FWD, the tokens after them by as much again
    assert err(pool[[4, 0, 2]], Wr) <= 2 * FWD
    for n in range(3):
        ref = Zr[0, :, starts[n + 1] - more:starts[n + 1]].transpose(0, 1)
        got = torch.stack([z[n] for z in zs])
        assert float((got.double().cpu() - ref).abs().max()) <= 2 * FWD * float(Zr.abs().max())


@pytest.mark.parametrize("T,starts", [(20, [2, 2, 9, 17]), (190, [3, 3, 70, 171])])
def test_what_lies_outside_the_sequences_is_not_read(T, starts):
    x = make(1, 1, 2, T, 64, 64, "bf16", seed=T, N=3)
    out = [*range(starts[0]), *range(starts[-1], T)]
    dZ = torch.randn(x["V"].shape, generator=torch.Generator().manual_seed(1)).cuda()
    clean = [t.clone() for t in (*(x[n] for n in RULE[:5]), dZ)]
    kw = dict(w0_per_seq=True, seq_start=offsets(starts))
    Z0, W0 = ttt.delta_fwd(*clean[:5], x["W0"], **kw)
    g0 = ttt.delta_bwd(*clean[:5], x["W0"], clean[5], **kw)
    for bad in (float("nan"), float("inf")):
        dirty = [t.clone() for t in clean]
        for t in dirty:
            t[:, :, out] = bad
        Z = torch.full(x["V"].shape, 7.0, device="cuda")
        _, W = ttt.delta_fwd(*dirty[:5], x["W0"], Z=Z, **kw)
        inside = slice(starts[0], starts[-1])
        assert torch.equal(Z[:, :, inside], Z0[:, :, inside]) and torch.equal(W, W0)
        assert bool((Z[:, :, out] == 7).all())
        g = ttt.delta_bwd(*dirty[:5], x["W0"], dirty[5], **kw)
        for n in g:
            assert torch.equal(g[n], g0[n]), n
            if n != "W0":
                assert not g[n][:, :, out].any(), n


@pytest.mark.parametrize("T", [24, 25])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64), (128, 128)])
def test_the_longest_short_call_and_the_shortest_long_one(T, dt, dk, dv):
    x = make(2, 1, 2, T, dk, dv, dt, seed=T + dk)
    for z_bf16 in (False, True):
        Z, W = ttt.delta_fwd(**x, w0_per_seq=True, z_bf16=z_bf16)
        Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
        assert err(Z, Zr) <= (BF16_TOL if z_bf16 else FWD) and err(W, Wr) <= FWD
    shared = x["W0"][0].contiguous()
    Z, W = ttt.delta_fwd(*(x[n] for n in RULE[:5]), shared)
    Zr, Wr = od.delta_f64(*(x[n] for n in RULE[:5]), shared)
    assert err(Z, Zr) <= FWD and err(W, Wr) <= FWD
    Z, W = ttt.delta_fwd(x["Q"], x["K"], x["V"], x["eta"])
    Zr, Wr = od.delta_f64(x["Q"], x["K"], x["V"], x["eta"])
    assert err(Z, Zr) <= FWD and err(W, Wr) <= FWD


@pytest.mark.parametrize("T", [20, 100])
def test_a_value_that_is_not_a_number_stays_in_its_sequence_and_head(T):
    x = make(2, 2, 2, T, 64, 64, "bf16", seed=T)
    Z0, W0 = ttt.delta_fwd(**x, w0_per_seq=True)
    for name in ("V", "eta", "g"):
        y = {n: t.clone() for n, t in x.items()}
        y[name][1, 0, 11] = float("nan")
        Z, W = ttt.delta_fwd(**y, w0_per_seq=True)
        assert torch.isnan(Z[1, 0, 11:]).any() and torch.isnan(W[1, 0]).any(), name
        assert torch.equal(Z[0], Z0[0]) and torch.equal(W[0], W0[0])
        assert torch.equal(Z[1, 1], Z0[1, 1]) and torch.equal(W[1, 1], W0[1, 1])


@pytest.mark.parametrize("dk,dv,dt,H", [(64, 64, "bf16", 38), (64, 128, "fp32", 19),
                                        (128, 128, "bf16", 19), (128, 64, "fp32", 38)])
@pytest.mark.parametrize("z_bf16", [False, True])
def test_more_heads_than_one_round_of_blocks(dk, dv, dt, H, z_bf16):
    """Just more blocks of 16 columns than SMs, where the scan may take 32 columns a block."""
    x = make(1, 1, H, 130, dk, dv, dt, seed=H + dk)
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True, z_bf16=z_bf16)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
    assert err(Z, Zr) <= (BF16_TOL if z_bf16 else FWD) and err(W, Wr) <= FWD
    kw = dict(w0_per_seq=True, z_bf16=z_bf16, seq_start=offsets([0, 0, 65, 120]))
    x["W0"] = torch.cat([x["W0"], 2 * x["W0"], -x["W0"]])
    Z = torch.full(x["V"].shape, 7.0, device="cuda", dtype=Z.dtype)
    _, W = ttt.delta_fwd(**x, Z=Z, **kw)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True, seq_start=[0, 0, 65, 120])
    assert bool((Z[:, :, 120:] == 7).all()) and err(W, Wr) <= FWD
    assert err(Z[:, :, :120], Zr[:, :, :120]) <= (BF16_TOL if z_bf16 else FWD)


@pytest.mark.parametrize("T", [20, 150])
def test_gates_above_zero(T):
    """Log decays of both signs: the weight grows by up to e^0.1 a token."""
    x = make(1, 2, 2, T, 64, 64, "fp32", seed=T + 3)
    x["g"] = 0.1 * torch.tanh(x["V"][..., 0]).contiguous()
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
    assert err(Z, Zr) <= FWD and err(W, Wr) <= FWD
    dZ = torch.randn(x["V"].shape, generator=torch.Generator().manual_seed(2)).cuda()
    g = ttt.delta_bwd(*(x[n] for n in RULE), dZ, None, w0_per_seq=True)
    ref = od.delta_grads(*(x[n] for n in RULE), dZ, None, w0_per_seq=True)
    for n, r in ref.items():
        assert err(g[n], r) <= BWD, n


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,starts", [(1, None), (10, list(range(11))), (150, [0, 1, 70, 150])])
def test_a_decay_of_nothing_has_no_gradient(T, starts, dt):
    """Without a start weight the first token's decay scales zero: its gradient is exactly 0."""
    N = 1 if starts is None else len(starts) - 1
    x = make(1, 2, 4, T, 128, 64, dt, seed=T, N=N)
    gen = torch.Generator().manual_seed(3)
    dZ, dW = torch.randn(x["V"].shape, generator=gen), torch.randn((N, 4, 128, 64), generator=gen)
    kw = {} if starts is None else dict(seq_start=offsets(starts))
    g = ttt.delta_bwd(*(x[n] for n in RULE[:5]), None, dZ.cuda(), dW.cuda(), **kw)["g"]
    first = [0] if starts is None else starts[:-1]
    assert not g[:, :, first].any()
    ref = od.delta_grads(*(x[n] for n in RULE[:5]), None, dZ, dW, seq_start=starts)["g"]
    assert float((g.double().cpu() - ref).abs().max()) <= BWD * float(ref.abs().max())
