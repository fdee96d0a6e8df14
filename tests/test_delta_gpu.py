"""The gated delta rule on the GPU against the float64 token-by-token oracle.

Error metric of the other parity tests: max |gpu - ref| / max |ref| per tensor.
Tolerance of fp32 outputs, 2e-5: a product over dk = 128 terms rounded to fp32
at every term is off by at most 128 * 2^-24 = 7.6e-6 of the sum of its terms'
sizes, a sum over a chunk's 64 tokens by 64 * 2^-24 = 3.8e-6 more, two fp16 terms
of an operand by 2^-22 = 2.4e-7 each; with unit keys and step sizes below 1 the
recurrence does not amplify what came before. A bf16 Z adds half a step, 2^-8 of
the value; its products of one fp16 term are off by 2^-11 of the sum of their
terms' sizes, which for the sums here (random signs, at most 192 terms) stays
below another 2^-9 of the largest value."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from oracle import delta as od

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


F32_TOL = 2e-5
BF16_TOL = 2.0 ** -8 + 2.0 ** -9
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(B, Hk, H, T, dk, dv, dt="bf16", seed=0, N=None, decay=1.0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(Q=unit(rn(B, Hk, T, dk)).to(DT[dt]), K=unit(rn(B, Hk, T, dk) + 0.3).to(DT[dt]),
             V=rn(B, H, T, dv).to(DT[dt]), eta=torch.sigmoid(rn(B, H, T)),
             g=-decay * torch.nn.functional.softplus(rn(B, H, T) - 1),
             W0=0.2 * rn(N or B, H, dk, dv))
    return {n: t.cuda() for n, t in x.items()}


def err(got, ref):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    return float((got - ref).abs().max() / ref.abs().max().clamp_min(1e-30))


def offsets(starts):
    return torch.tensor(starts, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 15, 63, 64, 65, 200])
def test_forward_lengths(dt, T):
    x = make(2, 2, 2, T, 64, 64, dt, seed=T)
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True, q_scale=0.125)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True, q_scale=0.125)
    assert err(Z, Zr) <= F32_TOL and err(W, Wr) <= F32_TOL


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("z_bf16", [False, True])
def test_forward_widths_and_types(dk, dv, dt, z_bf16):
    x = make(1, 2, 4, 150, dk, dv, dt, seed=dk + dv)
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True, z_bf16=z_bf16)
    assert Z.dtype == (torch.bfloat16 if z_bf16 else torch.float32)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
    assert err(Z, Zr) <= (BF16_TOL if z_bf16 else F32_TOL)
    assert err(W, Wr) <= F32_TOL


def test_forward_shared_and_missing_inputs():
    x = make(2, 1, 3, 130, 64, 64, seed=4)
    shared = x["W0"][0].contiguous()
    Z, W = ttt.delta_fwd(x["Q"], x["K"], x["V"], x["eta"], x["g"], shared)
    Zr, Wr = od.delta_f64(x["Q"], x["K"], x["V"], x["eta"], x["g"], shared)
    assert err(Z, Zr) <= F32_TOL and err(W, Wr) <= F32_TOL
    Z, W = ttt.delta_fwd(x["Q"], x["K"], x["V"], x["eta"], want_w=False)
    assert W is None
    assert err(Z, od.delta_f64(x["Q"], x["K"], x["V"], x["eta"])[0]) <= F32_TOL


def test_forward_without_gate_is_the_online_linear_layer():
    """g = 0 and q_scale = 1: ttt_linear_fwd with b = 1 and no LayerNorm."""
    x = make(2, 3, 3, 100, 64, 64, "fp32", seed=5)
    Z, W = ttt.delta_fwd(x["Q"], x["K"], x["V"], x["eta"], None, x["W0"], w0_per_seq=True)
    Zl, Wl = ttt.linear_fwd(x["Q"], x["K"], x["V"], x["eta"], x["W0"], b=1, ln=False,
                            w0_per_seq=True)
    assert err(Z, Zl.double().cpu()) <= 2 * F32_TOL and err(W, Wl.double().cpu()) <= 2 * F32_TOL


@pytest.mark.parametrize("z_bf16", [False, True])
@pytest.mark.parametrize("starts", [[0, 3, 70, 70, 199, 263], [5, 64, 128], [0, 0, 1, 1, 300],
                                    [10, 10]])
def test_forward_packed(starts, z_bf16):
    """Sequences of no, one and many tokens, rows in front of the first and behind the last."""
    T, N = 300, len(starts) - 1
    x = make(1, 2, 4, T, 64, 128, seed=len(starts), N=N)
    Z = torch.full((1, 4, T, 128), 7.0, dtype=torch.bfloat16 if z_bf16 else torch.float32,
                   device="cuda")
    _, W = ttt.delta_fwd(**x, w0_per_seq=True, seq_start=offsets(starts), Z=Z, z_bf16=z_bf16)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True, seq_start=starts)
    inside = torch.zeros(T, dtype=torch.bool)
    for a, b in zip(starts, starts[1:]):
        inside[a:b] = True
    assert (Z[:, :, ~inside.cuda()] == 7).all()
    if inside.any():
        assert err(Z[:, :, inside.cuda()], Zr[:, :, inside]) <= (BF16_TOL if z_bf16 else F32_TOL)
    assert err(W, Wr) <= F32_TOL


def test_packed_offsets_out_of_range_are_clamped():
    """Offsets that decrease or leave [0, T] reach no memory outside the arrays."""
    T = 130
    x = make(1, 1, 1, T, 64, 64, seed=9, N=3)
    Z = torch.zeros((1, 1, T, 64), device="cuda")
    _, W = ttt.delta_fwd(**x, w0_per_seq=True, seq_start=offsets([-5, 40, 20, 9999]), Z=Z)
    x2 = dict(x)
    W0 = x2.pop("W0")
    _, W1 = ttt.delta_fwd(**x2, W0=W0[:1].contiguous(), w0_per_seq=True, seq_start=offsets([0, 40]))
    assert torch.equal(W[0], W1[0])
    assert torch.equal(W[1], W0[1])            # 40 .. 20: no tokens
    assert torch.isfinite(W[2]).all() and torch.isfinite(Z).all()


@pytest.mark.parametrize("T", [100, 300])
def test_forward_gates_at_their_ends(T):
    """Full forgetting (g = -inf), very strong decay, no step (eta = 0), zero keys."""
    x = make(1, 1, 2, T, 128, 64, seed=11)
    x["g"][:, :, 7] = float("-inf")
    x["g"][:, :, 70:74] = float("-inf")
    x["g"][:, 0, 80:96] = -90.0
    x["g"][:, 1, 20:24] = torch.finfo(torch.float32).min
    x["eta"][:, :, 30:40] = 0
    x["K"][:, :, 35:45] = 0
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
    assert err(Z, Zr) <= F32_TOL and err(W, Wr) <= F32_TOL


@pytest.mark.parametrize("size", [1e-18, 1e-6, 1e4, 1e12])
def test_forward_sizes_of_values(size):
    """Values far from 1, and keys of small norm: no intermediate leaves its type's range."""
    x = make(1, 1, 1, 140, 64, 64, seed=12)
    x["V"], x["W0"] = (x["V"].float() * size).to(torch.bfloat16), x["W0"] * size
    x["K"] = (x["K"].float() * 1e-3).to(torch.bfloat16)
    x["Q"] = (x["Q"].float() * 1e5).to(torch.bfloat16)
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
    assert err(Z, Zr) <= F32_TOL and err(W, Wr) <= F32_TOL


def test_forward_in_two_calls_and_in_place():
    """A sequence resumed from W_out, written over W0, equals one call."""
    x = make(2, 2, 2, 200, 64, 64, seed=13)
    Zr, Wr = ttt.delta_fwd(**x, w0_per_seq=True)
    W = x["W0"].clone()
    part = lambda a, b: {n: x[n][:, :, a:b].contiguous() for n in ("Q", "K", "V", "eta", "g")}  # noqa: E731
    for a, b in ((0, 77), (77, 200)):
        p = part(a, b)
        Z = torch.empty((2, 2, b - a, 64), device="cuda")
        need = ttt.ttt_delta_workspace_bytes(2, 2, 2, b - a, 64, 64, 0, ttt.TTT_BF16)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        ttt.ttt_delta_fwd(p["Q"], p["K"], p["V"], p["eta"], p["g"], W, Z, W, None, 0, 1.0, 2, 2, 2,
                          b - a, 64, 64, ttt.TTT_BF16, ttt.TTT_F_W0_PER_SEQ, ws, need)
        assert err(Z, Zr[:, :, a:b].double().cpu()) <= 2 * F32_TOL
    assert err(W, Wr.double().cpu()) <= 2 * F32_TOL


@pytest.mark.parametrize("dk,dv,dt,n", [(64, 64, "bf16", 1), (128, 128, "bf16", 1),
                                        (128, 64, "fp32", 3), (64, 128, "bf16", 5)])
def test_decode_pool(dk, dv, dt, n):
    B, slots = 7, 9
    x = make(B, 2, 4, n, dk, dv, dt, seed=n + dk)
    pool = 0.2 * torch.randn(slots, 4, dk, dv, device="cuda")
    index = torch.tensor([8, 0, -1, 3, 9, 2, 5], dtype=torch.int32, device="cuda")
    live = torch.tensor([0, 1, 3, 5, 6], device="cuda")
    W, Z = pool.clone(), torch.full((B, 4, n, dv), 7.0, device="cuda")
    del x["W0"]
    ttt.delta_decode_tokens(**x, W=W, state_index=index, Z=Z, q_scale=dk ** -0.5)
    Zr, Wr = od.delta_f64(**{k: t[live] for k, t in x.items()}, W0=pool[index[live].long()],
                          w0_per_seq=True, q_scale=dk ** -0.5)
    assert err(Z[live], Zr) <= F32_TOL and err(W[index[live].long()], Wr) <= F32_TOL
    assert (Z[[2, 4]] == 7).all()              # padding rows
    untouched = [i for i in range(slots) if i not in index[live].tolist()]
    assert torch.equal(W[untouched], pool[untouched])


def test_decode_tokens_equal_single_tokens_and_the_forward():
    x = make(3, 1, 2, 12, 128, 128, seed=21)
    W0 = x.pop("W0")
    Wa, Wb = W0.clone(), W0.clone()
    Za = ttt.delta_decode_tokens(**x, W=Wa)
    Zb = torch.stack([ttt.delta_decode(*(x[k][:, :, t].contiguous() for k in ("Q", "K", "V", "eta",
                                                                             "g")), Wb)
                      for t in range(12)], 2)
    assert torch.equal(Za, Zb) and torch.equal(Wa, Wb)
    Zf, Wf = ttt.delta_fwd(**x, W0=W0, w0_per_seq=True)
    assert err(Za, Zf.double().cpu()) <= 2 * F32_TOL and err(Wa, Wf.double().cpu()) <= 2 * F32_TOL


def test_decode_large_pool_offsets_past_32_bits():
    """The last state of a pool of more than 2^31 elements."""
    H, d = 16, 128
    slots = 2 ** 31 // (H * d * d) + 3
    pool = torch.zeros(slots, H, d, d, device="cuda")
    x = make(1, 4, H, 1, d, d, seed=23)
    pool[-1] = x.pop("W0")[0]
    W0 = pool[-1:].clone()
    Z = ttt.delta_decode_tokens(**x, W=pool, state_index=offsets([slots - 1]))
    Zr, Wr = od.delta_f64(**x, W0=W0, w0_per_seq=True)
    assert err(Z, Zr) <= F32_TOL and err(pool[-1:], Wr) <= F32_TOL


def test_other_stream_and_graph_replay():
    x = make(2, 2, 2, 150, 64, 64, seed=31)
    Zr, Wr = ttt.delta_fwd(**x, w0_per_seq=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Z, Zr) and torch.equal(W, Wr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z, W = ttt.delta_fwd(**x, w0_per_seq=True)
    x["V"].mul_(2)
    x["W0"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Z, 2 * Zr) and torch.equal(W, 2 * Wr)  # the rule is linear in (v, W0)


def test_refusals():
    x = make(2, 2, 2, 20, 64, 64, seed=41)
    with pytest.raises(ValueError, match="not contiguous"):
        ttt.delta_fwd(**{**x, "Q": x["Q"].transpose(2, 3).contiguous().transpose(2, 3)},
                      w0_per_seq=True)
    with pytest.raises(ValueError, match="shape"):
        ttt.delta_fwd(**{**x, "eta": x["eta"][:1]}, w0_per_seq=True)
    with pytest.raises(ValueError, match="shape"):
        ttt.delta_fwd(**x)                                   # W0 per sequence without its flag
    with pytest.raises(ValueError, match="is on"):
        ttt.delta_fwd(**{**x, "g": x["g"].cpu()}, w0_per_seq=True)
    with pytest.raises(ValueError, match="expected"):
        ttt.delta_fwd(**{**x, "V": x["V"].float()}, w0_per_seq=True)
    with pytest.raises(ValueError, match="B = 1"):
        ttt.delta_fwd(**x, w0_per_seq=True, seq_start=offsets([0, 5, 20]))
    with pytest.raises(TypeError):
        ttt.delta_fwd(**{k: t.half() if k in "QKV" else t for k, t in x.items()}, w0_per_seq=True)
    with pytest.raises(ttt.TTTError):                        # heads that do not divide
        y = make(1, 2, 3, 20, 64, 64, seed=42)
        ttt.delta_fwd(**y, w0_per_seq=True)
    with pytest.raises(ttt.TTTError):                        # a pool smaller than the rows
        ttt.delta_decode_tokens(*(x[k] for k in ("Q", "K", "V", "eta", "g")), x["W0"][:1])
