"""The gated delta rule and the join without a GPU: every argument the C entry
points refuse on the host, the workspace sizes, and that what passes the host
checks stops at the check of the device."""
import ctypes
import gc
import weakref

import pytest
import torch

import test_sequence_layers_layer_b200 as ttt

P = 1 << 20  # a fake, 256-byte aligned "device" address; never dereferenced
ARG, SHAPE, DTYPE, ALIGN, PTR, ARCH, WS = -1, -2, -3, -4, -5, -8, -9
BIG = 1 << 40
# what a call that passes the host checks answers here: no sm_100 device, or a
# pointer that is not device memory
PASSED = (ARCH, PTR)


def fwd(**kw):
    a = dict(Q=P, K=P, V=P, eta=P, g=P, W0=P, Z=P, W_out=2 * P, seq_start=None, n_seq=0,
             q_scale=1.0, B=2, Hk=2, H=4, T=100, dk=64, dv=128, dt=ttt.TTT_BF16,
             flags=ttt.TTT_F_W0_PER_SEQ, workspace=P, workspace_bytes=BIG, stream=0)
    a.update(kw)
    return ttt.ttt_delta_fwd(**a, check=False)


def bwd(**kw):
    a = dict(Q=P, K=P, V=P, eta=P, g=P, W0=P, dZ=P, dW_out=P, dQ=P, dK=P, dV=P, deta=P, dg=P,
             dW0=P, seq_start=None, n_seq=0, q_scale=1.0, B=2, Hk=2, H=4, T=100, dk=64, dv=128,
             dt=ttt.TTT_BF16, flags=0, workspace=P, workspace_bytes=BIG, stream=0)
    a.update(kw)
    return ttt.ttt_delta_bwd(**a, check=False)


def dec(**kw):
    a = dict(Q=P, K=P, V=P, eta=P, g=P, W=P, Z=P, state_index=P, n_slots=3, q_scale=1.0, B=4, Hk=2,
             H=4, n=1, dk=64, dv=128, dt=ttt.TTT_BF16, flags=0, stream=0)
    a.update(kw)
    return ttt.ttt_delta_decode(**a, check=False)


def jf(**kw):
    a = dict(X=P, Z=P, gate=P, scale=P, post_gamma=P, post_beta=P, pre_gamma=P, pre_beta=P,
             R=2 * P, Hn=3 * P, eps=1e-5, B=2, H=3, T=5, d=64, dt=ttt.TTT_BF16, flags=0, stream=0)
    a.update(kw)
    return ttt.ttt_join_fwd(**a, check=False)


def jb(**kw):
    a = dict(R=P, Z=P, gate=P, scale=P, post_gamma=P, post_beta=P, pre_gamma=P, dR=P, dH=2 * P,
             dX=3 * P, dZ=4 * P, dGate=5 * P, dscale=P, dpost_gamma=P, dpost_beta=P, dpre_gamma=P,
             dpre_beta=P, eps=1e-5, B=2, H=3, T=5, d=64, dt=ttt.TTT_BF16, flags=0, workspace=P,
             workspace_bytes=BIG, stream=0)
    a.update(kw)
    return ttt.ttt_join_bwd(**a, check=False)


DELTA_SHAPES = [dict(B=0), dict(Hk=0), dict(H=0), dict(H=3), dict(dk=32), dict(dk=256), dict(dv=96),
                dict(B=1 << 24), dict(B=-1)]


@pytest.mark.parametrize("kw,code", [
    *[(k, SHAPE) for k in DELTA_SHAPES], (dict(T=0), SHAPE), (dict(T=(1 << 30) + 1), SHAPE),
    *[({n: None}, PTR) for n in ("Q", "K", "V", "eta", "Z")],
    *[({n: P + 8}, ALIGN) for n in ("Q", "K", "V", "W0", "Z", "W_out")],
    (dict(dt=7), DTYPE), (dict(flags=ttt.TTT_F_LN), ARG), (dict(flags=1 << 20), ARG),
    (dict(n_seq=1), ARG), (dict(seq_start=P, n_seq=0, B=1), ARG),
    (dict(seq_start=P, n_seq=-1, B=1), ARG), (dict(seq_start=P, n_seq=2), ARG),  # packed: B = 1
    (dict(W_out=P, flags=0), ARG),                                   # over a shared W0
    (dict(workspace=None), WS), (dict(workspace=P + 16), WS), (dict(workspace_bytes=64), WS),
])
def test_forward_refuses(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw", [{}, dict(T=1), dict(g=None, W0=None), dict(W_out=None),
                                dict(W_out=P), dict(seq_start=P, n_seq=3, B=1),
                                dict(flags=ttt.TTT_F_Z_BF16), dict(dt=ttt.TTT_FP32)])
def test_forward_passes_to_the_device_check(kw):
    assert fwd(**kw) in PASSED


@pytest.mark.parametrize("kw,code", [
    *[(k, SHAPE) for k in DELTA_SHAPES], (dict(T=0), SHAPE),
    *[({n: None}, PTR) for n in ("Q", "K", "V", "eta", "dZ", "dQ", "dK", "dV", "deta", "dg",
                                 "dW0")],
    (dict(g=None), ARG), (dict(W0=None), ARG),                       # a gradient of nothing
    *[({n: P + 4}, ALIGN) for n in ("Q", "K", "V", "W0", "dZ", "dW_out", "dQ", "dK", "dV", "dW0")],
    (dict(dt=7), DTYPE), (dict(flags=ttt.TTT_F_Z_BF16), ARG),
    (dict(n_seq=1), ARG), (dict(seq_start=P, n_seq=2), ARG),
    (dict(workspace=None), WS), (dict(workspace=P + 128), WS), (dict(workspace_bytes=64), WS),
])
def test_backward_refuses(kw, code):
    assert bwd(**kw) == code


@pytest.mark.parametrize("kw", [{}, dict(g=None, dg=None, W0=None, dW0=None, dW_out=None),
                                dict(seq_start=P, n_seq=3, B=1), dict(T=1)])
def test_backward_passes_to_the_device_check(kw):
    assert bwd(**kw) in PASSED


@pytest.mark.parametrize("kw,code", [
    *[(k, SHAPE) for k in DELTA_SHAPES], (dict(n=0), SHAPE), (dict(n_slots=0), SHAPE),
    (dict(state_index=None), SHAPE),                                 # 4 rows, 3 states
    *[({n: None}, PTR) for n in ("Q", "K", "V", "eta", "W", "Z")],
    *[({n: P + 8}, ALIGN) for n in ("Q", "K", "V", "W", "Z")],
    (dict(dt=7), DTYPE), (dict(flags=ttt.TTT_F_W0_PER_SEQ), ARG),
])
def test_decode_refuses(kw, code):
    assert dec(**kw) == code


def test_decode_passes_to_the_device_check():
    assert dec() in PASSED and dec(state_index=None, n_slots=4, n=7, g=None) in PASSED


JOIN_SHAPES = [dict(B=0), dict(H=0), dict(T=0), dict(d=0), dict(d=48), dict(H=1, d=12),
               dict(H=17, d=256), dict(H=1, d=4104)]


@pytest.mark.parametrize("kw,code", [
    *[(k, SHAPE) for k in JOIN_SHAPES],
    (dict(X=None), PTR), (dict(R=None), PTR),
    *[({n: P + 8}, ALIGN) for n in ("X", "Z", "gate", "scale", "post_gamma", "post_beta",
                                    "pre_gamma", "pre_beta", "R", "Hn")],
    (dict(Z=None), ARG), (dict(Hn=None), ARG),                       # parameters of no norm
    (dict(Z=None, gate=None, scale=None, post_gamma=None, post_beta=None), ARG),  # R without Z
    (dict(Z=None, gate=None, scale=None, post_gamma=None, post_beta=None, R=None, Hn=None), PTR),
    (dict(Hn=2 * P), ARG), (dict(Hn=P), ARG),                        # Hn over R, over X
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(dt=7), DTYPE), (dict(flags=ttt.TTT_F_LN), ARG),
])
def test_join_refuses(kw, code):
    assert jf(**kw) == code


@pytest.mark.parametrize("kw", [
    {}, dict(R=P), dict(Hn=None, pre_gamma=None, pre_beta=None), dict(H=1, d=4096),
    dict(H=1, d=8), dict(H=16, d=256), dict(flags=ttt.TTT_F_RMS | ttt.TTT_F_GATE_SIGMOID),
    dict(Z=None, gate=None, scale=None, post_gamma=None, post_beta=None, R=None)])
def test_join_passes_to_the_device_check(kw):
    assert jf(**kw) in PASSED


@pytest.mark.parametrize("kw,code", [
    *[(k, SHAPE) for k in JOIN_SHAPES],
    (dict(dX=None), PTR), (dict(dR=None, dH=None), PTR), (dict(R=None), PTR), (dict(dZ=None), PTR),
    (dict(dGate=None), PTR), (dict(gate=None), ARG), (dict(Z=None), ARG),
    (dict(dH=None), ARG),                                            # a norm's gradients without dH
    (dict(dX=2 * P), ARG),                                           # dX over dH
    *[({n: P + 8}, ALIGN) for n in ("R", "Z", "gate", "scale", "post_gamma", "post_beta",
                                    "pre_gamma", "dR", "dH", "dX", "dZ", "dGate")],
    (dict(eps=0.0), ARG), (dict(dt=7), DTYPE), (dict(flags=1 << 9), ARG),
    (dict(workspace=None), WS), (dict(workspace=P + 16), WS), (dict(workspace_bytes=4), WS),
])
def test_join_backward_refuses(kw, code):
    assert jb(**kw) == code


@pytest.mark.parametrize("kw", [
    {}, dict(dX=P, dR=P), dict(dH=None, dpre_gamma=None, dpre_beta=None),
    dict(dR=None), dict(dscale=None, dpost_gamma=None, dpost_beta=None)])
def test_join_backward_passes_to_the_device_check(kw):
    assert jb(**kw) in PASSED


def test_workspace_sizes():
    bf, f32 = ttt.TTT_BF16, ttt.TTT_FP32
    size, back = ttt.ttt_delta_workspace_bytes, ttt.ttt_delta_bwd_workspace_bytes
    for q in (size, back):
        assert q(2, 2, 4, 100, 64, 64, 0, bf) > 0
        assert q(2, 2, 4, 100, 64, 64, 0, f32) >= q(2, 2, 4, 100, 64, 64, 0, bf)
        # packed: every sequence may leave a partial chunk
        assert q(1, 2, 4, 1000, 64, 64, 10, bf) > q(1, 2, 4, 1000, 64, 64, 0, bf)
        # no size for what the call refuses
        assert q(2, 2, 3, 100, 64, 64, 0, bf) == 0 and q(2, 2, 4, 100, 48, 64, 0, bf) == 0
        assert q(2, 2, 4, 100, 64, 64, 3, bf) == 0 and q(2, 2, 4, 0, 64, 64, 0, bf) == 0
        assert q(2, 2, 4, 100, 64, 64, 0, 9) == 0
        # past 32 bits
        assert q(8, 8, 8, 1 << 20, 128, 128, 0, f32) > 1 << 33
    assert back(2, 2, 4, 100, 64, 64, 0, bf) > size(2, 2, 4, 100, 64, 64, 0, bf)
    assert ttt.ttt_join_bwd_workspace_bytes(2, 3, 5, 64) > 0
    assert ttt.ttt_join_bwd_workspace_bytes(2, 3, 5, 48) == 0


def test_conveniences_refuse_host_tensors():
    t = torch.zeros(1, 1, 4, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        ttt.delta_fwd(t, t, t, t[..., 0])
    with pytest.raises(ValueError, match="CUDA device"):
        ttt.delta_decode_tokens(t, t, t, t[..., 0], None, torch.zeros(1, 1, 64, 64))
    with pytest.raises(ValueError, match="CUDA device"):
        ttt.join_fwd(torch.zeros(1, 4, 64), t)


def test_a_call_holds_its_own_workspace():
    """The memory a call takes for itself outlives the address it passes on."""
    class Memory:
        def data_ptr(self):
            return 7 * 256
    refs = []

    class Sub(ttt._On):
        def empty(self, shape, dtype):
            m = Memory()
            refs.append(weakref.ref(m))
            return m
    on = object.__new__(Sub)
    on.torch, on.side = torch, None
    assert on.workspace(None, 1000) == (7 * 256, 1000)
    gc.collect()
    assert refs[0]() is not None


def test_the_library_exports_what_the_header_declares():
    L = ttt.lib()
    for s in ("ttt_delta_fwd", "ttt_delta_bwd", "ttt_delta_decode", "ttt_join_fwd", "ttt_join_bwd"):
        assert s in ttt.header_symbols() and isinstance(getattr(L, s), ctypes._CFuncPtr)
