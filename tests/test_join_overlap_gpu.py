"""Outputs of the join's calls over their inputs: what the header allows gives the bits of separate
arrays, everything else is refused before a launch and leaves the arrays as they were. Pairs of
unequal sizes stand in one buffer that holds the larger."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from test_join_gpu import make

pytestmark = pytest.mark.gpu

ARG = -1
FWD = ("X", "Z", "gate", "scale", "gamma1", "beta1", "gamma2", "beta2", "R", "Hn")
BWD = ("R", "Z", "gate", "scale", "gamma1", "beta1", "gamma2", "dR", "dH", "dX", "dZ", "dGate",
       "dscale", "dgamma1", "dbeta1", "dgamma2", "dbeta2")


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


def fwd(a, H, d):
    B, T, _ = a["X"].shape
    code = ttt.TTT_BF16 if a["X"].dtype == torch.bfloat16 else ttt.TTT_FP32
    flags = ttt.TTT_F_Z_BF16 if a["Z"].dtype == torch.bfloat16 else 0
    return ttt.ttt_join_fwd(*[a[n] for n in FWD], 1e-5, B, H, T, d, code, flags, check=False)


def bwd(a, H, d):
    B, T, _ = a["R"].shape
    need = ttt.ttt_join_bwd_workspace_bytes(B, H, T, d)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return ttt.ttt_join_bwd(*[a[n] for n in BWD], 1e-5, B, H, T, d, ttt.TTT_FP32, 0, ws, need,
                            check=False)


def fwd_args(B, H, T, d, dt, z_bf16):
    a = make(B, H, T, d, dt, z_bf16, seed=H)
    return {**a, "R": torch.zeros_like(a["X"]), "Hn": torch.zeros_like(a["X"])}


def bwd_args(B, H, T, d):
    a = make(B, H, T, d, "fp32", False, seed=H + 1)
    a["R"] = a.pop("X")
    like = dict(dX="R", dZ="Z", dGate="gate", dscale="scale", dgamma1="gamma1", dbeta1="beta1",
                dgamma2="gamma2", dbeta2="beta2")
    return {**a, **{n: torch.zeros_like(a[m]) for n, m in like.items()}}


def lay_over(a, over, what):
    n, m = a[over].numel(), a[what].numel()
    buf = torch.zeros(max(n, m), device="cuda")
    assert a[over].dtype == a[what].dtype == torch.float32
    buf[:m] = a[what].flatten()
    a[what], a[over] = buf[:m].view(a[what].shape), buf[:n].view(a[over].shape)


@pytest.mark.parametrize("dt,z_bf16", [("bf16", True), ("fp32", False)])
@pytest.mark.parametrize("H,d,pairs", [
    (12, 64, [{"R": "X"}, {"R": "gate"}, {"Hn": "gate"}, {"R": "X", "Hn": "gate"}]),
    (1, 776, [{"R": "Z"}, {"Hn": "Z"}, {"R": "X", "Hn": "Z"}])])
def test_forward_in_place(dt, z_bf16, H, d, pairs):
    a = fwd_args(2, H, 301, d, dt, z_bf16)
    assert fwd(a, H, d) == 0
    for pair in pairs:
        b = fwd_args(2, H, 301, d, dt, z_bf16)
        b.update({n: b[m].view(b[n].shape) for n, m in pair.items()})
        assert fwd(b, H, d) == 0
        assert torch.equal(a["R"], b["R"]) and torch.equal(a["Hn"], b["Hn"]), pair


@pytest.mark.parametrize("H,d,pairs", [
    (12, 64, [{"dX": "R"}, {"dX": "gate"}, {"dX": "dR", "dGate": "gate", "dZ": "Z"},
              {"dGate": "R", "dX": "dR"}, {"dGate": "dR"}, {"dGate": "dH"},
              {"dscale": "scale", "dgamma1": "gamma1", "dbeta1": "beta1", "dgamma2": "gamma2"},
              {"dscale": "gamma2", "dbeta2": "scale"}]),
    (40, 64, [{"dscale": "scale", "dgamma1": "gamma1", "dbeta1": "beta1", "dgamma2": "gamma2"}]),
    (1, 776, [{"dX": "Z"}, {"dZ": "R"}, {"dZ": "dH", "dX": "Z", "dGate": "R"}])])
def test_backward_in_place(H, d, pairs):
    a = bwd_args(2, H, 301, d)
    assert bwd(a, H, d) == 0
    for pair in pairs:
        b = bwd_args(2, H, 301, d)
        b.update({n: b[m].view(b[n].shape) for n, m in pair.items()})
        assert bwd(b, H, d) == 0
        for n in BWD[9:]:
            assert torch.equal(a[n], b[n]), (pair, n)


def refused(call, a, H, d):
    before = {n: t.clone() for n, t in a.items()}
    assert call(a, H, d) == ARG
    assert all(torch.equal(a[n], t) for n, t in before.items())


@pytest.mark.parametrize("over,what", [("R", "Z"), ("Hn", "Z"), ("Hn", "R"), ("Hn", "X"), ("R", "scale"),
                                       ("Hn", "beta2")])
def test_forward_refuses(over, what):
    a = fwd_args(2, 3, 40, 64, "fp32", False)
    lay_over(a, over, what)
    refused(fwd, a, 3, 64)


@pytest.mark.parametrize("over,what", [("dX", "Z"), ("dZ", "R"), ("dZ", "dR"), ("dZ", "gate"), ("dGate", "Z"),
                                       ("dX", "dH"), ("dX", "dZ"), ("dGate", "dX"), ("dscale", "dbeta2"),
                                       ("dscale", "R"), ("dX", "gamma1")])
def test_backward_refuses(over, what):
    a = bwd_args(2, 3, 40, 64)
    lay_over(a, over, what)
    refused(bwd, a, 3, 64)


def test_refuses_arrays_shifted_by_a_row():
    a = fwd_args(2, 3, 40, 64, "fp32", False)
    n, D = a["X"].numel(), 192
    buf = torch.zeros(n + D, device="cuda")
    buf[:n] = a["X"].flatten()
    a["X"], a["R"] = buf[:n].view(2, 40, D), buf[D:].view(2, 40, D)
    refused(fwd, a, 3, 64)
    b = bwd_args(2, 3, 40, 64)
    buf = torch.zeros(n + D, device="cuda")
    buf[D:] = b["dR"].flatten()
    b["dR"], b["dX"] = buf[D:].view(2, 40, D), buf[:n].view(2, 40, D)
    refused(bwd, b, 3, 64)
