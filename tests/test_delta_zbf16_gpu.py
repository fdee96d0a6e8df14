"""A bf16 Z of the gated delta rule is its fp32 Z rounded, bit for bit, as it is for the library's
other forwards: every product that Z depends on is formed as for fp32, and rounded once. Covered:
the token-by-token calls (up to 24 tokens, decode), the chunked scan with 16 columns a block and
with 32 (256 blocks of 16 columns), packed sequences, resumed states."""
import pytest
import torch

import test_sequence_layers_layer_b200 as ttt
from test_delta_gpu import make, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert ttt.ttt_device_status() == 0


def same(x, **kw):
    Z, W = ttt.delta_fwd(**x, z_bf16=False, **kw)
    Zb, Wb = ttt.delta_fwd(**x, z_bf16=True, **kw)
    assert Zb.dtype == torch.bfloat16
    assert torch.equal(Zb, Z.to(torch.bfloat16)) and torch.equal(W, Wb)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 24, 25, 64, 333])
def test_bf16_z_is_the_rounded_fp32_z(dk, dv, dt, T):
    same(make(1, 2, 4, T, dk, dv, dt, seed=T + dk), w0_per_seq=True, q_scale=dk ** -0.5)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_bf16_z_with_many_heads(dk, dt):
    same(make(4, 4, 8, 200, dk, 128, dt, seed=dk), w0_per_seq=True)


def test_bf16_z_of_packed_sequences():
    starts = [0, 3, 70, 70, 199, 300]
    x = make(1, 2, 4, 300, 128, 128, seed=6, N=5)
    same(x, w0_per_seq=True, seq_start=offsets(starts))


def test_bf16_z_of_decode():
    x = make(5, 2, 4, 3, 128, 64, seed=7)
    W0 = x.pop("W0")
    Wa, Wb = W0.clone(), W0.clone()
    Za = ttt.delta_decode_tokens(**x, W=Wa)
    Zb = ttt.delta_decode_tokens(**x, W=Wb, z_bf16=True)
    assert torch.equal(Zb, Za.to(torch.bfloat16)) and torch.equal(Wa, Wb)
