"""Loops of the gated delta rule's kernels past their first turns, against the float64 oracle: rings of
stages refilled more than once (11 chunks and more: the third stage, both parities of a stage's use),
the sum of a shared start weight's gradient over sixteen sequences at a time and the rest, zeros
outside packed sequences by more than one block a head. Tolerances are those of the shorter
calls: with unit keys and steps below 1 an error of a chunk does not grow over those behind it."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from oracle import delta as od
from test_delta_bwd_gpu import check, grads
from test_delta_gpu import F32_TOL, err, make, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_forward_and_backward_of_eleven_chunks(dk, dv, dt):
    x = make(1, 1, 1, 650, dk, dv, dt, seed=dk + dv + 1, decay=0.1)
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True)
    Zr, Wr = od.delta_f64(**x, w0_per_seq=True)
    assert err(Z, Zr) <= F32_TOL and err(W, Wr) <= F32_TOL
    check(x, w0_per_seq=True)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_forward_of_forty_chunks_with_32_columns_a_block(dt):
    """256 blocks of 16 columns: 32 a block. Two of the heads against the oracle."""
    x = make(4, 8, 8, 2500, 128, 128, dt, seed=2, decay=0.05)
    Z, W = ttt.delta_fwd(**x, w0_per_seq=True)
    for b, h in ((0, 0), (3, 7)):
        one = {n: t[b:b + 1, h:h + 1] for n, t in x.items()}
        Zr, Wr = od.delta_f64(**one, w0_per_seq=True)
        assert err(Z[b:b + 1, h:h + 1], Zr) <= F32_TOL and err(W[b:b + 1, h:h + 1], Wr) <= F32_TOL


@pytest.mark.parametrize("N", [15, 16, 17, 33])
@pytest.mark.parametrize("packed", [False, True])
def test_shared_start_weight_of_many_sequences(N, packed):
    if packed:
        starts = [0]
        for i in range(N):
            starts.append(starts[-1] + (i * 7) % 5)  # lengths 0 .. 4
        x = make(1, 2, 2, starts[-1], 64, 64, seed=N, N=1)
    else:
        x = make(N, 2, 2, 3, 64, 64, seed=N)
    x["W0"] = x["W0"][0].contiguous()
    check(x, seq_start=offsets(starts) if packed else None)


@pytest.mark.parametrize("starts", [[700, 820, 831], [0, 11, 131], [640, 640, 760]])
def test_many_tokens_outside_the_packed_sequences(starts):
    T = 1500
    x = make(1, 1, 2, T, 64, 128, seed=starts[0] + 3, N=2)
    outside = torch.ones(T, dtype=torch.bool)
    outside[starts[0]:starts[-1]] = False
    for n in x:
        if n != "W0":
            x[n][:, :, outside.cuda()] = float("nan")  # not read
    # the oracle takes the inside alone
    inside = {n: t if n == "W0" else t[:, :, starts[0]:starts[-1]].contiguous() for n, t in x.items()}
    got, dZ, dW_out = grads(x, seq_start=offsets(starts), w0_per_seq=True)
    ref = od.delta_grads(*[inside[n] for n in ("Q", "K", "V", "eta", "g", "W0")],
                         dZ[:, :, starts[0]:starts[-1]], dW_out,
                         seq_start=[s - starts[0] for s in starts], w0_per_seq=True)
    for n, r in ref.items():
        g = got[n]
        if n != "W0":
            assert (g[:, :, outside.cuda()] == 0).all(), n
            g = g[:, :, starts[0]:starts[-1]]
        assert err(g, r) <= 5e-5, n
