"""A forward of at most 24 tokens runs token by token and takes no workspace: its size is 0, a call
without one passes the host's checks, and the convenience allocates none."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from test_delta_join_abi_cpu import PASSED, WS, fwd


@pytest.mark.parametrize("dt", [ttt.TTT_BF16, ttt.TTT_FP32])
def test_size_is_zero_exactly_for_short_calls(dt):
    size = ttt.ttt_delta_workspace_bytes
    for T in (1, 2, 16, 24):
        assert size(256, 8, 16, T, 128, 128, 0, dt) == 0 and size(1, 2, 4, T, 64, 128, 3, dt) == 0
    assert size(256, 8, 16, 25, 128, 128, 0, dt) > 0 and size(1, 2, 4, 25, 64, 128, 3, dt) > 0
    assert ttt.ttt_delta_bwd_workspace_bytes(2, 2, 4, 1, 64, 64, 0, dt) > 0  # always by chunks


def test_short_calls_pass_without_a_workspace():
    none = dict(workspace=None, workspace_bytes=0)
    for kw in (dict(T=24), dict(T=1), dict(T=20, B=1, seq_start=1 << 20, n_seq=5)):
        assert fwd(**kw, **none) in PASSED
    assert fwd(T=25, **none) == WS


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_a_short_call_allocates_its_outputs_alone(packed):
    from test_delta_gpu import make, offsets
    B, T = (1, 24) if packed else (64, 24)
    x = make(B, 4, 8, T, 128, 128, seed=1, N=3 if packed else B)
    kw = dict(w0_per_seq=True, seq_start=offsets([0, 5, 5, 24]) if packed else None)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    Z, W = ttt.delta_fwd(**x, **kw)
    outputs = Z.numel() * 4 + W.numel() * 4
    assert torch.cuda.max_memory_allocated() - before <= outputs + 1024
    # and, with memory that a caller gives all the same, the same bits
    Z2, W2 = ttt.delta_fwd(**x, **kw, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    assert torch.equal(Z, Z2) and torch.equal(W, W2)
