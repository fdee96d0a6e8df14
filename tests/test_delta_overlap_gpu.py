"""Outputs of the gated delta rule's calls over their inputs: what the header allows gives the bits of
separate arrays; everything else is refused before a launch, and leaves the arrays as they were."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from test_delta_gpu import make, offsets

pytestmark = pytest.mark.gpu

ARG = -1


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


def lay_over(a, over, what):
    """Both arrays from the start of one buffer that holds the larger: a call that were not refused
    would mix them up, and would not leave them."""
    n, m = a[over].numel(), a[what].numel()
    buf = torch.zeros(max(n, m), device="cuda")
    assert a[over].element_size() == a[what].element_size() == 4
    buf[:m] = a[what].flatten().view(torch.float32)
    a[what] = buf[:m].view(a[what].dtype).view(a[what].shape)
    a[over] = buf[:n].view(a[over].shape)


def call(fn, a, *tail):
    return fn(*a.values(), *tail, check=False)


def fwd_args(x, dt, z_bf16=False, n_seq=0):
    B, Hk, T, dk = x["Q"].shape
    H, dv = x["V"].shape[1], x["V"].shape[3]
    N = n_seq or B
    need = ttt.ttt_delta_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, dt)
    a = dict(x, Z=torch.zeros(B, H, T, dv, dtype=torch.bfloat16 if z_bf16 else torch.float32, device="cuda"),
             W_out=torch.zeros(N, H, dk, dv, device="cuda"),
             seq_start=None)
    ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    shape = (n_seq, 0.5, B, Hk, H, T, dk, dv, dt,
             ttt.TTT_F_W0_PER_SEQ | (ttt.TTT_F_Z_BF16 if z_bf16 else 0))
    return a, shape, ws


def run_fwd(a, shape, ws):
    return call(ttt.ttt_delta_fwd, a, *shape, ws, ws.numel())


@pytest.mark.parametrize("T", [20, 200])
@pytest.mark.parametrize("dt,z_bf16", [("fp32", False), ("bf16", True)])
@pytest.mark.parametrize("dk", [64, 128])
def test_forward_in_place(T, dt, z_bf16, dk):
    code = ttt.TTT_BF16 if dt == "bf16" else ttt.TTT_FP32
    x = make(2, 3, 3, T, dk, 128, dt, seed=T)
    a, shape, ws = fwd_args(x, code, z_bf16)
    assert run_fwd(a, shape, ws) == 0
    b, _, _ = fwd_args({n: t.clone() for n, t in x.items()}, code, z_bf16)
    b["Z"], b["W_out"] = b["V"], b["W0"]
    assert run_fwd(b, shape, ws) == 0
    assert torch.equal(a["Z"], b["Z"]) and torch.equal(a["W_out"], b["W_out"])


@pytest.mark.parametrize("T", [20, 200])
@pytest.mark.parametrize("over,what", [("Z", "Q"), ("Z", "K"), ("Z", "W_out"), ("Z", "eta"), ("Z", "g"),
                                       ("W_out", "V"), ("W_out", "g"), ("W_out", "seq_start")])
def test_forward_refuses_overlaps(T, over, what):
    x = make(1, 2, 2, T, 64, 64, "fp32", seed=1)
    a, shape, ws = fwd_args(x, ttt.TTT_FP32)
    if what == "seq_start":
        shape = (1, *shape[1:])
        a["seq_start"] = offsets([0, T])
    lay_over(a, over, what)
    before = {n: t.clone() for n, t in a.items() if t is not None}
    assert run_fwd(a, shape, ws) == ARG
    assert all(torch.equal(a[n], t) for n, t in before.items())


def test_forward_refuses_shifted_arrays_and_workspaces():
    x = make(1, 2, 2, 100, 64, 64, "fp32", seed=2)
    a, shape, ws = fwd_args(x, ttt.TTT_FP32)
    n = x["V"].numel()
    buf = torch.zeros(n + 64, device="cuda")
    buf[:n] = x["V"].flatten()
    a["V"], z = buf[:n].view(x["V"].shape), buf[64:].view(x["V"].shape)
    assert run_fwd(dict(a, Z=z), shape, ws) == ARG
    need = ttt.ttt_delta_workspace_bytes(1, 2, 2, 100, 64, 64, 0, ttt.TTT_FP32)
    whole = torch.zeros(need + 4 * n, dtype=torch.uint8, device="cuda")
    z = whole[need:].view(torch.float32).view(x["V"].shape)
    assert call(ttt.ttt_delta_fwd, dict(a, Z=z), *shape, whole, whole.numel()) == 0  # behind it
    z = whole[need - 256:need - 256 + 4 * n].view(torch.float32).view(x["V"].shape)
    assert call(ttt.ttt_delta_fwd, dict(a, Z=z), *shape, whole, whole.numel()) == ARG
    with pytest.raises(ttt.TTTError):
        ttt.delta_fwd(**x, w0_per_seq=True, Z=x["Q"])


def bwd_args(x, packed=False):
    gen = torch.Generator().manual_seed(7)
    B, Hk, T, dk = x["Q"].shape
    H, dv = x["V"].shape[1], x["V"].shape[3]
    N = x["W0"].shape[0]
    a = dict(x, dZ=torch.randn(B, H, T, dv, generator=gen).cuda(),
             dW_out=torch.randn(N, H, dk, dv, generator=gen).cuda())
    a.update({"d" + n: torch.zeros_like(x[n], dtype=torch.float32) for n in ("Q", "K", "V", "eta", "g", "W0")})
    a["seq_start"] = offsets([3, 40, 41, T - 5]) if packed else None
    n_seq = 3 if packed else 0
    need = ttt.ttt_delta_bwd_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, ttt.TTT_FP32)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return a, (n_seq, 0.5, B, Hk, H, T, dk, dv, ttt.TTT_FP32, ttt.TTT_F_W0_PER_SEQ, ws, need)


GRADS = ("Q", "K", "V", "eta", "g", "W0")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64)])
def test_backward_in_place(packed, dk, dv):
    x = make(1, 2, 4, 150, dk, dv, "fp32", seed=3, N=3 if packed else 1)
    a, tail = bwd_args(x, packed)
    assert call(ttt.ttt_delta_bwd, a, *tail) == 0
    b, tail = bwd_args({n: t.clone() for n, t in x.items()}, packed)
    b.update({"d" + n: b[n] for n in GRADS})
    assert call(ttt.ttt_delta_bwd, b, *tail) == 0
    for n in GRADS:
        assert torch.equal(a["d" + n], b["d" + n]), n
    c, tail = bwd_args(x, packed)
    c["dW0"] = c["dW_out"]
    assert call(ttt.ttt_delta_bwd, c, *tail) == 0
    assert torch.equal(a["dW0"], c["dW0"])


@pytest.mark.parametrize("over,what", [("dV", "dZ"), ("dQ", "dZ"), ("dK", "dZ"), ("dQ", "K"), ("dK", "dQ"),
                                       ("dV", "dQ"), ("deta", "g"), ("dg", "deta"), ("dg", "eta"),
                                       ("dQ", "V"), ("dW0", "dZ"), ("dW0", "Q")])
def test_backward_refuses_overlaps(over, what):
    x = make(1, 2, 2, 130, 64, 64, "fp32", seed=4)
    a, tail = bwd_args(x)
    lay_over(a, over, what)
    before = {n: t.clone() for n, t in a.items() if t is not None}
    assert call(ttt.ttt_delta_bwd, a, *tail) == ARG
    assert all(torch.equal(a[n], t) for n, t in before.items())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 3])
def test_decode_over_v_and_refusals(dt, n):
    x = make(5, 4, 4, n, 128, 128, dt, seed=5)
    W0 = x.pop("W0")
    Wa, Wb = W0.clone(), W0.clone()
    Za = ttt.delta_decode_tokens(**x, W=Wa, z_bf16=dt == "bf16")
    v = x["V"].clone()
    Zb = ttt.delta_decode_tokens(**{**x, "V": v}, W=Wb, z_bf16=dt == "bf16", Z=v)
    assert Zb is v and torch.equal(Za, Zb) and torch.equal(Wa, Wb)
    for over in ("Q", "K"):
        with pytest.raises(ttt.TTTError):
            ttt.delta_decode_tokens(**x, W=W0, z_bf16=dt == "bf16", Z=x[over])
    if dt == "fp32":
        with pytest.raises(ttt.TTTError):
            ttt.delta_decode_tokens(**x, W=W0, Z=W0.flatten()[:Za.numel()].view(Za.shape))
    assert torch.equal(W0, make(5, 4, 4, n, 128, 128, dt, seed=5)["W0"])
