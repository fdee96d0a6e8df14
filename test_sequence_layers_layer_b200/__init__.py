"""Python binding of libttt.so, the B200 library for a Test-Time-Training (TTT)
layer: its forward passes (TTT-Linear, TTT-MLP, large chunk), the backward
passes of TTT-Linear and large-chunk TTT, the affine-map calls behind the
sequence-parallel large-chunk forward (seqpar.py), the gated delta rule
(forward, backward, decode from a pool of states) and the join between two
blocks (norm, gate, residual, norm; forward and backward).

The functions named like the C ABI (ttt_linear_fwd, ttt_mlp_fwd,
ttt_chunk_fwd, ...) take exactly the C arguments; a pointer argument may be a
torch tensor (its data_ptr() is passed), an int address, or None. They only
marshal arguments: every step of the computation runs in the library's CUDA
kernels. linear_fwd / mlp_fwd / chunk_fwd / linear_bwd / chunk_bwd /
chunk_map / affine_prefix / delta_fwd / delta_bwd / delta_decode /
delta_decode_tokens / join_fwd / join_bwd are conveniences that read the shapes
off torch tensors and allocate the outputs (and workspaces) with torch.

There is no fallback: if libttt.so is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libttt.so")
HEADER_PATH = os.path.join(os.path.dirname(HERE), "include", "ttt.h")

TTT_OK = 0
TTT_BF16, TTT_FP32 = 0, 1
TTT_F_LN = 1
TTT_F_W0_PER_SEQ = 2
TTT_F_Z_BF16 = 4
TTT_F_L2_KEYS = 8
TTT_F_RMS = 16
TTT_F_GATE_SIGMOID = 32

_P = ctypes.c_void_p
_I = ctypes.c_int
_lib = None


class TTTError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {status}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """Load libttt.so (built in-tree by build.py). Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libttt.so not built at {LIB_PATH}; run build.py")
        L = ctypes.CDLL(LIB_PATH)
        L.ttt_abi_version.restype = _I
        L.ttt_abi_version.argtypes = []
        L.ttt_status_string.restype = ctypes.c_char_p
        L.ttt_status_string.argtypes = [_I]
        L.ttt_linear_fwd.restype = _I
        L.ttt_linear_fwd.argtypes = [_P] * 9 + [_I] * 6 + [ctypes.c_uint, _P]
        L.ttt_mlp_decode.restype = _I
        L.ttt_mlp_decode.argtypes = [_P] * 9 + [_I] * 5 + [ctypes.c_uint, _P]
        L.ttt_linear_decode.restype = _I
        L.ttt_linear_decode.argtypes = [_P] * 8 + [_I] * 4 + [ctypes.c_uint, _P]
        L.ttt_linear_fwd_steps.restype = _I
        L.ttt_linear_fwd_steps.argtypes = [_P] * 9 + [_I] * 6 + [ctypes.c_uint, _P]
        L.ttt_linear_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_linear_bwd_workspace_bytes.argtypes = [_I] * 5
        L.ttt_linear_bwd.restype = _I
        L.ttt_linear_bwd.argtypes = [_P] * 16 + [_I] * 6 + [ctypes.c_uint, _P, ctypes.c_size_t, _P]
        L.ttt_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_chunk_bwd_workspace_bytes.argtypes = [_I] * 5
        L.ttt_chunk_bwd.restype = _I
        L.ttt_chunk_bwd.argtypes = [_P] * 12 + [_I] * 6 + [ctypes.c_uint, _P, ctypes.c_size_t, _P]
        L.ttt_mlp_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_mlp_bwd_workspace_bytes.argtypes = [_I] * 6
        L.ttt_mlp_bwd.restype = _I
        L.ttt_mlp_bwd.argtypes = [_P] * 19 + [_I] * 7 + [ctypes.c_uint, _P, ctypes.c_size_t, _P]
        L.ttt_mlp_fwd.restype = _I
        L.ttt_mlp_fwd.argtypes = [_P] * 11 + [_I] * 7 + [ctypes.c_uint, _P]
        L.ttt_chunk_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_chunk_workspace_bytes.argtypes = [_I] * 5
        L.ttt_chunk_fwd.restype = _I
        L.ttt_chunk_fwd.argtypes = [_P] * 7 + [_I] * 6 + [ctypes.c_uint, _P, ctypes.c_size_t, _P]
        L.ttt_chunk_fwd_noalloc.restype = _I
        L.ttt_chunk_fwd_noalloc.argtypes = [_P] * 7 + [_I] * 6 + [ctypes.c_uint, _P]
        L.ttt_chunk_map_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_chunk_map_workspace_bytes.argtypes = [_I] * 6
        L.ttt_chunk_map.restype = _I
        L.ttt_chunk_map.argtypes = [_P] * 5 + [_I] * 6 + [_P, ctypes.c_size_t, _P]
        L.ttt_linear_map_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_linear_map_workspace_bytes.argtypes = [_I] * 6
        L.ttt_linear_map.restype = _I
        L.ttt_linear_map.argtypes = [_P] * 5 + [_I] * 6 + [_P, ctypes.c_size_t, _P]
        L.ttt_affine_prefix.restype = _I
        L.ttt_affine_prefix.argtypes = ([_P] * 5 + [_I] * 4 + [ctypes.c_longlong] * 2
                                        + [ctypes.c_uint, _P])
        L.ttt_delta_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_delta_workspace_bytes.argtypes = [_I] * 8
        L.ttt_delta_fwd.restype = _I
        L.ttt_delta_fwd.argtypes = ([_P] * 9 + [_I, ctypes.c_float] + [_I] * 7
                                    + [ctypes.c_uint, _P, ctypes.c_size_t, _P])
        L.ttt_delta_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_delta_bwd_workspace_bytes.argtypes = [_I] * 8
        L.ttt_delta_bwd.restype = _I
        L.ttt_delta_bwd.argtypes = ([_P] * 15 + [_I, ctypes.c_float] + [_I] * 7
                                    + [ctypes.c_uint, _P, ctypes.c_size_t, _P])
        L.ttt_delta_decode.restype = _I
        L.ttt_delta_decode.argtypes = ([_P] * 8 + [_I, ctypes.c_float] + [_I] * 7
                                       + [ctypes.c_uint, _P])
        L.ttt_join_fwd.restype = _I
        L.ttt_join_fwd.argtypes = [_P] * 10 + [ctypes.c_float] + [_I] * 5 + [ctypes.c_uint, _P]
        L.ttt_join_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ttt_join_bwd_workspace_bytes.argtypes = [_I] * 4
        L.ttt_join_bwd.restype = _I
        L.ttt_join_bwd.argtypes = ([_P] * 17 + [ctypes.c_float] + [_I] * 5
                                   + [ctypes.c_uint, _P, ctypes.c_size_t, _P])
        L.ttt_device_status.restype = _I
        L.ttt_device_status.argtypes = [_P]
        L.ttt_launch_count.restype = ctypes.c_ulonglong
        L.ttt_launch_count.argtypes = []
        L.ttt_diag_kernel_timing.restype = _I
        L.ttt_diag_kernel_timing.argtypes = [_I]
        L.ttt_diag_kernel_times.restype = _I
        L.ttt_diag_kernel_times.argtypes = [ctypes.POINTER(ctypes.c_float), _I]
        L.ttt_selftest_umma.restype = _I
        L.ttt_selftest_umma.argtypes = [_I] * 5 + [_P, _P, _P, _P]
        L.ttt_diag_gelu.restype = _I
        L.ttt_diag_gelu.argtypes = [_P, _P, _P, _I, _P]
        L.ttt_diag_wait_timeout.restype = _I
        L.ttt_diag_wait_timeout.argtypes = [ctypes.c_uint, _P]
        L.ttt_linear_decode_tokens.restype = _I
        L.ttt_linear_decode_tokens.argtypes = [_P] * 8 + [_I] * 5 + [ctypes.c_uint, _P]
        L.ttt_mlp_decode_tokens.restype = _I
        L.ttt_mlp_decode_tokens.argtypes = [_P] * 9 + [_I] * 6 + [ctypes.c_uint, _P]
        L.ttt_diag_mlp_fwd_tcgen05.restype = _I
        L.ttt_diag_mlp_fwd_tcgen05.argtypes = [_P] * 11 + [_I] * 7 + [ctypes.c_uint, _P]
        L.ttt_diag_umma_issue_cycles.restype = _I
        L.ttt_diag_umma_issue_cycles.argtypes = [_I] * 4 + [_P, _P]
        _lib = L
    return _lib


def header_symbols() -> list[str]:
    """Names of the functions the public headers (include/*.h) declare."""
    import glob
    names = []
    for path in sorted(glob.glob(os.path.join(os.path.dirname(HEADER_PATH), "*.h"))):
        names += re.findall(r"TTT_API\s+[\w\s\*]*?\b(ttt_\w+)\s*\(", open(path).read())
    return names


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn, rc):
    if rc != TTT_OK:
        raise TTTError(fn, rc)
    return rc


def status_string(status: int) -> str:
    return lib().ttt_status_string(int(status)).decode()


def abi_version() -> int:
    return lib().ttt_abi_version()


# ----------------------------------------------------------------- C-ABI calls

def ttt_linear_fwd(Q, K, V, eta, W0, ln_gamma, ln_beta, Z, W_out, B, H, T, d, b, dt, flags,
                   stream=None, check=True):
    rc = lib().ttt_linear_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W0), _ptr(ln_gamma),
                              _ptr(ln_beta), _ptr(Z), _ptr(W_out), B, H, T, d, b, dt, flags,
                              _stream(stream))
    return _check("ttt_linear_fwd", rc) if check else rc


def ttt_mlp_decode(q, k, v, eta, W1, W2, ln_gamma, ln_beta, z, B, H, d, dh, dt, flags,
                   stream=None, check=True):
    rc = lib().ttt_mlp_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(W1), _ptr(W2),
                              _ptr(ln_gamma), _ptr(ln_beta), _ptr(z), B, H, d, dh, dt, flags,
                              _stream(stream))
    return _check("ttt_mlp_decode", rc) if check else rc


def ttt_linear_decode(q, k, v, eta, W, ln_gamma, ln_beta, z, B, H, d, dt, flags, stream=None,
                      check=True):
    rc = lib().ttt_linear_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(W), _ptr(ln_gamma),
                                 _ptr(ln_beta), _ptr(z), B, H, d, dt, flags, _stream(stream))
    return _check("ttt_linear_decode", rc) if check else rc


def ttt_linear_decode_tokens(q, k, v, eta, W, ln_gamma, ln_beta, z, B, H, n, d, dt, flags,
                             stream=None, check=True):
    rc = lib().ttt_linear_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(W),
                                        _ptr(ln_gamma), _ptr(ln_beta), _ptr(z), B, H, n, d, dt,
                                        flags, _stream(stream))
    return _check("ttt_linear_decode_tokens", rc) if check else rc


def ttt_mlp_decode_tokens(q, k, v, eta, W1, W2, ln_gamma, ln_beta, z, B, H, n, d, dh, dt, flags,
                          stream=None, check=True):
    rc = lib().ttt_mlp_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(W1), _ptr(W2),
                                     _ptr(ln_gamma), _ptr(ln_beta), _ptr(z), B, H, n, d, dh, dt,
                                     flags, _stream(stream))
    return _check("ttt_mlp_decode_tokens", rc) if check else rc


def ttt_linear_fwd_steps(Q, K, V, eta, W0, ln_gamma, ln_beta, Z, W_out, B, H, T, d, n_steps, dt,
                         flags, stream=None, check=True):
    rc = lib().ttt_linear_fwd_steps(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W0),
                                    _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(W_out), B, H, T,
                                    d, n_steps, dt, flags, _stream(stream))
    return _check("ttt_linear_fwd_steps", rc) if check else rc


def ttt_linear_bwd_workspace_bytes(B, H, T, d, b) -> int:
    return int(lib().ttt_linear_bwd_workspace_bytes(B, H, T, d, b))


def ttt_linear_bwd(Q, K, V, eta, W0, ln_gamma, ln_beta, dZ, dW_out, dQ, dK, dV, deta, dW0, dgamma,
                   dbeta, B, H, T, d, b, dt, flags, workspace, workspace_bytes, stream=None,
                   check=True):
    rc = lib().ttt_linear_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W0), _ptr(ln_gamma),
                              _ptr(ln_beta), _ptr(dZ), _ptr(dW_out), _ptr(dQ), _ptr(dK), _ptr(dV),
                              _ptr(deta), _ptr(dW0), _ptr(dgamma), _ptr(dbeta), B, H, T, d, b, dt,
                              flags, _ptr(workspace), workspace_bytes, _stream(stream))
    return _check("ttt_linear_bwd", rc) if check else rc


def ttt_chunk_bwd_workspace_bytes(B, H, T, d, chunk) -> int:
    return int(lib().ttt_chunk_bwd_workspace_bytes(B, H, T, d, chunk))


def ttt_chunk_bwd(Q, K, V, eta, W0, dZ, dW_out, dQ, dK, dV, deta, dW0, B, H, T, d, chunk, dt, flags,
                  workspace, workspace_bytes, stream=None, check=True):
    rc = lib().ttt_chunk_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W0), _ptr(dZ),
                             _ptr(dW_out), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(deta), _ptr(dW0), B,
                             H, T, d, chunk, dt, flags, _ptr(workspace), workspace_bytes,
                             _stream(stream))
    return _check("ttt_chunk_bwd", rc) if check else rc


def ttt_mlp_bwd_workspace_bytes(B, H, T, d, dh, b) -> int:
    return int(lib().ttt_mlp_bwd_workspace_bytes(B, H, T, d, dh, b))


def ttt_mlp_bwd(Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, dZ, dW1_out, dW2_out, dQ, dK, dV,
                deta, dW1_0, dW2_0, dgamma, dbeta, B, H, T, d, dh, b, dt, flags, workspace,
                workspace_bytes, stream=None, check=True):
    rc = lib().ttt_mlp_bwd(*[_ptr(x) for x in (Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, dZ,
                                               dW1_out, dW2_out, dQ, dK, dV, deta, dW1_0, dW2_0,
                                               dgamma, dbeta)],
                           B, H, T, d, dh, b, dt, flags, _ptr(workspace), workspace_bytes,
                           _stream(stream))
    return _check("ttt_mlp_bwd", rc) if check else rc


def ttt_mlp_fwd(Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, Z, W1_out, W2_out, B, H, T, d, dh,
                b, dt, flags, stream=None, check=True):
    rc = lib().ttt_mlp_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W1_0), _ptr(W2_0),
                           _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(W1_out), _ptr(W2_out),
                           B, H, T, d, dh, b, dt, flags, _stream(stream))
    return _check("ttt_mlp_fwd", rc) if check else rc


def ttt_diag_mlp_fwd_tcgen05(Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, Z, W1_out, W2_out, B, H,
                             T, d, dh, b, dt, flags, stream=None, check=True):
    rc = lib().ttt_diag_mlp_fwd_tcgen05(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W1_0),
                                        _ptr(W2_0), _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z),
                                        _ptr(W1_out), _ptr(W2_out), B, H, T, d, dh, b, dt, flags,
                                        _stream(stream))
    return _check("ttt_diag_mlp_fwd_tcgen05", rc) if check else rc


def ttt_diag_umma_issue_cycles(M, N, count, nacc, cycles, stream=None, check=True):
    rc = lib().ttt_diag_umma_issue_cycles(M, N, count, nacc, _ptr(cycles), _stream(stream))
    return _check("ttt_diag_umma_issue_cycles", rc) if check else rc


def ttt_chunk_workspace_bytes(B, H, T, d, chunk) -> int:
    return int(lib().ttt_chunk_workspace_bytes(B, H, T, d, chunk))


def ttt_chunk_fwd(Q, K, V, eta, W0, Z, W_out, B, H, T, d, chunk, dt, flags, workspace,
                  workspace_bytes, stream=None, check=True):
    rc = lib().ttt_chunk_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W0), _ptr(Z),
                             _ptr(W_out), B, H, T, d, chunk, dt, flags, _ptr(workspace),
                             workspace_bytes, _stream(stream))
    return _check("ttt_chunk_fwd", rc) if check else rc


def ttt_chunk_fwd_noalloc(Q, K, V, eta, W0, Z, W_out, B, H, T, d, chunk, dt, flags, stream=None,
                          check=True):
    """ttt_chunk_fwd with the library's static scratch instead of a workspace,
    for callers that cannot allocate device memory (see include/ttt.h)."""
    rc = lib().ttt_chunk_fwd_noalloc(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(W0), _ptr(Z),
                                     _ptr(W_out), B, H, T, d, chunk, dt, flags, _stream(stream))
    return _check("ttt_chunk_fwd_noalloc", rc) if check else rc


def ttt_chunk_map_workspace_bytes(B, H, T, d, chunk, dt) -> int:
    return int(lib().ttt_chunk_map_workspace_bytes(B, H, T, d, chunk, dt))


def ttt_chunk_map(K, V, eta, M, N, B, H, T, d, chunk, dt, workspace, workspace_bytes, stream=None,
                  check=True):
    rc = lib().ttt_chunk_map(_ptr(K), _ptr(V), _ptr(eta), _ptr(M), _ptr(N), B, H, T, d, chunk, dt,
                             _ptr(workspace), workspace_bytes, _stream(stream))
    return _check("ttt_chunk_map", rc) if check else rc


def ttt_linear_map_workspace_bytes(B, H, T, d, b, dt) -> int:
    return int(lib().ttt_linear_map_workspace_bytes(B, H, T, d, b, dt))


def ttt_linear_map(K, V, eta, M, N, B, H, T, d, b, dt, workspace, workspace_bytes, stream=None,
                   check=True):
    rc = lib().ttt_linear_map(_ptr(K), _ptr(V), _ptr(eta), _ptr(M), _ptr(N), B, H, T, d, b, dt,
                              _ptr(workspace), workspace_bytes, _stream(stream))
    return _check("ttt_linear_map", rc) if check else rc


def ttt_affine_prefix(M, N, W0, W_in, W_end, S, H, nseg, d, seq_stride, seg_stride, flags,
                      stream=None, check=True):
    rc = lib().ttt_affine_prefix(_ptr(M), _ptr(N), _ptr(W0), _ptr(W_in), _ptr(W_end), S, H, nseg,
                                 d, seq_stride, seg_stride, flags, _stream(stream))
    return _check("ttt_affine_prefix", rc) if check else rc


def ttt_delta_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, dt) -> int:
    return int(lib().ttt_delta_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, dt))


def ttt_delta_fwd(Q, K, V, eta, g, W0, Z, W_out, seq_start, n_seq, q_scale, B, Hk, H, T, dk, dv,
                  dt, flags, workspace, workspace_bytes, stream=None, check=True):
    rc = lib().ttt_delta_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(g), _ptr(W0), _ptr(Z),
                             _ptr(W_out), _ptr(seq_start), n_seq, q_scale, B, Hk, H, T, dk, dv,
                             dt, flags, _ptr(workspace), workspace_bytes, _stream(stream))
    return _check("ttt_delta_fwd", rc) if check else rc


def ttt_delta_bwd_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, dt) -> int:
    return int(lib().ttt_delta_bwd_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, dt))


def ttt_delta_bwd(Q, K, V, eta, g, W0, dZ, dW_out, dQ, dK, dV, deta, dg, dW0, seq_start, n_seq,
                  q_scale, B, Hk, H, T, dk, dv, dt, flags, workspace, workspace_bytes, stream=None,
                  check=True):
    rc = lib().ttt_delta_bwd(*[_ptr(x) for x in (Q, K, V, eta, g, W0, dZ, dW_out, dQ, dK, dV, deta,
                                                 dg, dW0, seq_start)],
                             n_seq, q_scale, B, Hk, H, T, dk, dv, dt, flags, _ptr(workspace),
                             workspace_bytes, _stream(stream))
    return _check("ttt_delta_bwd", rc) if check else rc


def ttt_delta_decode(Q, K, V, eta, g, W, Z, state_index, n_slots, q_scale, B, Hk, H, n, dk, dv,
                     dt, flags, stream=None, check=True):
    rc = lib().ttt_delta_decode(_ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _ptr(g), _ptr(W), _ptr(Z),
                                _ptr(state_index), n_slots, q_scale, B, Hk, H, n, dk, dv, dt,
                                flags, _stream(stream))
    return _check("ttt_delta_decode", rc) if check else rc


def ttt_join_fwd(X, Z, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta, R, Hn, eps, B, H,
                 T, d, dt, flags, stream=None, check=True):
    rc = lib().ttt_join_fwd(*[_ptr(x) for x in (X, Z, gate, scale, post_gamma, post_beta,
                                                pre_gamma, pre_beta, R, Hn)],
                            eps, B, H, T, d, dt, flags, _stream(stream))
    return _check("ttt_join_fwd", rc) if check else rc


def ttt_join_bwd_workspace_bytes(B, H, T, d) -> int:
    return int(lib().ttt_join_bwd_workspace_bytes(B, H, T, d))


def ttt_join_bwd(R, Z, gate, scale, post_gamma, post_beta, pre_gamma, dR, dH, dX, dZ, dGate,
                 dscale, dpost_gamma, dpost_beta, dpre_gamma, dpre_beta, eps, B, H, T, d, dt,
                 flags, workspace, workspace_bytes, stream=None, check=True):
    rc = lib().ttt_join_bwd(*[_ptr(x) for x in (R, Z, gate, scale, post_gamma, post_beta,
                                                pre_gamma, dR, dH, dX, dZ, dGate, dscale,
                                                dpost_gamma, dpost_beta, dpre_gamma, dpre_beta)],
                            eps, B, H, T, d, dt, flags, _ptr(workspace), workspace_bytes,
                            _stream(stream))
    return _check("ttt_join_bwd", rc) if check else rc


def ttt_device_status(stream=None) -> int:
    return lib().ttt_device_status(_stream(stream))


def ttt_launch_count() -> int:
    return int(lib().ttt_launch_count())


def ttt_diag_kernel_timing(enable: bool) -> int:
    return lib().ttt_diag_kernel_timing(int(bool(enable)))


def ttt_diag_kernel_times(max_kernels: int = 8) -> list[float]:
    """Per kernel position, the summed duration (ms) over the calls recorded since
    timing was enabled (diagnostic)."""
    buf = (ctypes.c_float * max_kernels)()
    n = lib().ttt_diag_kernel_times(buf, max_kernels)
    if n < 0:
        raise TTTError("ttt_diag_kernel_times", n)
    return [buf[i] for i in range(min(n, max_kernels))]


def ttt_selftest_umma(M, N, K, a_layout, b_layout, A, B, D, stream=None, check=True):
    """Diagnostic (include/ttt_diag.h): D = A @ B through one tcgen05 MMA chain."""
    rc = lib().ttt_selftest_umma(M, N, K, a_layout, b_layout, _ptr(A), _ptr(B), _ptr(D),
                                 _stream(stream))
    return _check("ttt_selftest_umma", rc) if check else rc


def ttt_diag_wait_timeout(limit_us, stream=None, check=True):
    """Diagnostic (include/ttt_diag.h): a bounded on-chip wait that runs out."""
    rc = lib().ttt_diag_wait_timeout(limit_us, _stream(stream))
    return _check("ttt_diag_wait_timeout", rc) if check else rc


def ttt_diag_gelu(h, gelu, gelu_prime, n, stream=None, check=True):
    """Diagnostic (include/ttt_diag.h): the MLP kernel's GELU and GELU'."""
    rc = lib().ttt_diag_gelu(_ptr(h), _ptr(gelu), _ptr(gelu_prime), n, _stream(stream))
    return _check("ttt_diag_gelu", rc) if check else rc


# ----------------------------------------------------------------- conveniences

def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return TTT_BF16
    if t.dtype == torch.float32:
        return TTT_FP32
    raise TypeError(f"Q/K/V must be bf16 or fp32, got {t.dtype}")


def linear_fwd(Q, K, V, eta, W0, ln_gamma=None, ln_beta=None, *, b, ln, w0_per_seq=False,
               stream=None, want_w=True, z_bf16=False, l2_keys=False):
    """TTT-Linear forward. Q, K, V: [B,H,T,d] cuda tensors (bf16 or fp32).
    l2_keys: normalise every key to unit length (TTT_F_L2_KEYS).
    Returns (Z fp32 [B,H,T,d], W_out fp32 [B,H,d,d] or None)."""
    import torch
    B, H, T, d = Q.shape
    Z = torch.empty((B, H, T, d), dtype=torch.bfloat16 if z_bf16 else torch.float32, device=Q.device)
    W_out = torch.empty((B, H, d, d), dtype=torch.float32, device=Q.device) if want_w else None
    flags = (TTT_F_LN if ln else 0) | (TTT_F_W0_PER_SEQ if w0_per_seq else 0) | \
        (TTT_F_Z_BF16 if z_bf16 else 0) | (TTT_F_L2_KEYS if l2_keys else 0)
    ttt_linear_fwd(Q, K, V, eta, W0, ln_gamma, ln_beta, Z, W_out, B, H, T, d, b,
                   _dtype_code(Q), flags, stream)
    return Z, W_out


def mlp_decode(q, k, v, eta, W1, W2, ln_gamma, ln_beta, *, z=None, z_bf16=False, stream=None):
    """One TTT-MLP token per sequence, d = 64, dh = 256: q, k, v [B, H, 64], eta
    [B, H], W1 [B, H, 64, 256] and W2 [B, H, 256, 64] fp32 updated in place
    (ttt_mlp_decode). Returns z."""
    import torch
    B, H, d = q.shape
    if z is None:
        z = torch.empty((B, H, d), dtype=torch.bfloat16 if z_bf16 else torch.float32,
                        device=q.device)
    ttt_mlp_decode(q, k, v, eta, W1, W2, ln_gamma, ln_beta, z, B, H, d, W1.shape[-1],
                   _dtype_code(q), TTT_F_LN | (TTT_F_Z_BF16 if z_bf16 else 0), stream)
    return z


def linear_decode(q, k, v, eta, W, ln_gamma=None, ln_beta=None, *, ln, z=None, z_bf16=False,
                  l2_keys=False, stream=None):
    """One TTT-Linear token per sequence, d = 64: q, k, v [B, H, 64], eta [B, H],
    W [B, H, 64, 64] fp32 updated in place (ttt_linear_decode). Returns z."""
    import torch
    B, H, d = q.shape
    if z is None:
        z = torch.empty((B, H, d), dtype=torch.bfloat16 if z_bf16 else torch.float32,
                        device=q.device)
    flags = (TTT_F_LN if ln else 0) | (TTT_F_Z_BF16 if z_bf16 else 0) | \
        (TTT_F_L2_KEYS if l2_keys else 0)
    ttt_linear_decode(q, k, v, eta, W, ln_gamma, ln_beta, z, B, H, d, _dtype_code(q), flags,
                      stream)
    return z


def linear_decode_tokens(Q, K, V, eta, W, ln_gamma=None, ln_beta=None, *, ln, z_bf16=False,
                         l2_keys=False, stream=None):
    """n TTT-Linear tokens per sequence in one call, d = 64: Q, K, V [B, H, n, 64],
    eta [B, H, n], W [B, H, 64, 64] fp32 updated in place, the weight on chip
    across the tokens (ttt_linear_decode_tokens). Returns Z [B, H, n, 64]."""
    import torch
    B, H, n, d = Q.shape
    Z = torch.empty((B, H, n, d), dtype=torch.bfloat16 if z_bf16 else torch.float32,
                    device=Q.device)
    flags = (TTT_F_LN if ln else 0) | (TTT_F_Z_BF16 if z_bf16 else 0) | \
        (TTT_F_L2_KEYS if l2_keys else 0)
    ttt_linear_decode_tokens(Q, K, V, eta, W, ln_gamma, ln_beta, Z, B, H, n, d, _dtype_code(Q),
                             flags, stream)
    return Z


def mlp_decode_tokens(Q, K, V, eta, W1, W2, ln_gamma, ln_beta, *, z_bf16=False, stream=None):
    """n TTT-MLP tokens per sequence in one call, d = 64, dh = 256: Q, K, V
    [B, H, n, 64], eta [B, H, n], W1 [B, H, 64, 256] and W2 [B, H, 256, 64] fp32
    updated in place, both on chip across the tokens (ttt_mlp_decode_tokens).
    Returns Z [B, H, n, 64]."""
    import torch
    B, H, n, d = Q.shape
    Z = torch.empty((B, H, n, d), dtype=torch.bfloat16 if z_bf16 else torch.float32,
                    device=Q.device)
    ttt_mlp_decode_tokens(Q, K, V, eta, W1, W2, ln_gamma, ln_beta, Z, B, H, n, d, W1.shape[-1],
                          _dtype_code(Q), TTT_F_LN | (TTT_F_Z_BF16 if z_bf16 else 0), stream)
    return Z


def linear_fwd_steps(Q, K, V, eta, W0, ln_gamma=None, ln_beta=None, *, n_steps, ln,
                     w0_per_seq=False, stream=None, want_w=True, z_bf16=False, l2_keys=False):
    """TTT-Linear forward, online, n_steps gradient steps per token before its
    read-out (ttt_linear_fwd_steps). Returns (Z, W_out) like linear_fwd."""
    import torch
    B, H, T, d = Q.shape
    Z = torch.empty((B, H, T, d), dtype=torch.bfloat16 if z_bf16 else torch.float32, device=Q.device)
    W_out = torch.empty((B, H, d, d), dtype=torch.float32, device=Q.device) if want_w else None
    flags = (TTT_F_LN if ln else 0) | (TTT_F_W0_PER_SEQ if w0_per_seq else 0) | \
        (TTT_F_Z_BF16 if z_bf16 else 0) | (TTT_F_L2_KEYS if l2_keys else 0)
    ttt_linear_fwd_steps(Q, K, V, eta, W0, ln_gamma, ln_beta, Z, W_out, B, H, T, d, n_steps,
                         _dtype_code(Q), flags, stream)
    return Z, W_out


def linear_bwd(Q, K, V, eta, W0, ln_gamma, ln_beta, dZ, dW_out=None, *, b, ln, w0_per_seq=False,
               workspace=None, stream=None):
    """TTT-Linear backward. Returns a dict of fp32 cuda tensors: Q, K, V, eta,
    W0 and (with ln) gamma, beta -- the gradients of sum(Z * dZ) +
    sum(W_out * dW_out). Allocates the workspace with torch unless one is given."""
    import torch
    B, H, T, d = Q.shape
    dev = Q.device
    f32 = dict(dtype=torch.float32, device=dev)
    need = ttt_linear_bwd_workspace_bytes(B, H, T, d, b)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    g = dict(Q=torch.empty((B, H, T, d), **f32), K=torch.empty((B, H, T, d), **f32),
             V=torch.empty((B, H, T, d), **f32), eta=torch.empty((B, H, T), **f32),
             W0=torch.empty(tuple(W0.shape), **f32))
    if ln:
        g["gamma"] = torch.empty((H, d), **f32)
        g["beta"] = torch.empty((H, d), **f32)
    flags = (TTT_F_LN if ln else 0) | (TTT_F_W0_PER_SEQ if w0_per_seq else 0)
    ttt_linear_bwd(Q, K, V, eta, W0, ln_gamma, ln_beta, dZ, dW_out, g["Q"], g["K"], g["V"],
                   g["eta"], g["W0"], g.get("gamma"), g.get("beta"), B, H, T, d, b, _dtype_code(Q),
                   flags, workspace, workspace.numel() * workspace.element_size(), stream)
    return g


def mlp_bwd(Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, dZ, dW1_out=None, dW2_out=None, *, b,
            w0_per_seq=False, workspace=None, stream=None):
    """TTT-MLP backward. Returns a dict of fp32 gradients with keys Q, K, V,
    eta, W1, W2, gamma, beta (W1/W2 shaped like W1_0/W2_0)."""
    import torch
    B, H, T, d = Q.shape
    dh = W1_0.shape[-1]
    f = dict(device=Q.device, dtype=torch.float32)
    g = {"Q": torch.empty((B, H, T, d), **f), "K": torch.empty((B, H, T, d), **f),
         "V": torch.empty((B, H, T, d), **f), "eta": torch.empty((B, H, T), **f),
         "W1": torch.empty(tuple(W1_0.shape), **f), "W2": torch.empty(tuple(W2_0.shape), **f),
         "gamma": torch.empty((H, d), **f), "beta": torch.empty((H, d), **f)}
    need = ttt_mlp_bwd_workspace_bytes(B, H, T, d, dh, b)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=Q.device)
    flags = TTT_F_LN | (TTT_F_W0_PER_SEQ if w0_per_seq else 0)
    ttt_mlp_bwd(Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, dZ, dW1_out, dW2_out, g["Q"], g["K"],
                g["V"], g["eta"], g["W1"], g["W2"], g["gamma"], g["beta"], B, H, T, d, dh, b,
                _dtype_code(Q), flags, workspace, workspace.numel() * workspace.element_size(),
                stream)
    return g


def chunk_bwd(Q, K, V, eta, W0, dZ, dW_out=None, *, chunk, w0_per_seq=False, workspace=None,
              stream=None):
    """Large-chunk TTT backward. Returns a dict of fp32 cuda tensors Q, K, V,
    eta, W0: the gradients of sum(Z * dZ) + sum(W_out * dW_out)."""
    import torch
    B, H, T, d = Q.shape
    f32 = dict(dtype=torch.float32, device=Q.device)
    need = ttt_chunk_bwd_workspace_bytes(B, H, T, d, chunk)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=Q.device)
    g = dict(Q=torch.empty((B, H, T, d), **f32), K=torch.empty((B, H, T, d), **f32),
             V=torch.empty((B, H, T, d), **f32), eta=torch.empty((B, H, T), **f32),
             W0=torch.empty(tuple(W0.shape), **f32))
    ttt_chunk_bwd(Q, K, V, eta, W0, dZ, dW_out, g["Q"], g["K"], g["V"], g["eta"], g["W0"], B, H, T,
                  d, chunk, _dtype_code(Q), TTT_F_W0_PER_SEQ if w0_per_seq else 0, workspace,
                  workspace.numel() * workspace.element_size(), stream)
    return g


def mlp_fwd(Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, *, b, w0_per_seq=False, stream=None,
            want_w=True, z_bf16=False, kernel="default"):
    """TTT-MLP forward. Returns (Z, W1_out, W2_out). kernel="tcgen05" runs the
    diagnostic single-issuer tensor-core kernel (ttt_diag_mlp_fwd_tcgen05)."""
    import torch
    B, H, T, d = Q.shape
    dh = W1_0.shape[-1]
    Z = torch.empty((B, H, T, d), dtype=torch.bfloat16 if z_bf16 else torch.float32, device=Q.device)
    W1o = torch.empty((B, H, d, dh), dtype=torch.float32, device=Q.device) if want_w else None
    W2o = torch.empty((B, H, dh, d), dtype=torch.float32, device=Q.device) if want_w else None
    flags = TTT_F_LN | (TTT_F_W0_PER_SEQ if w0_per_seq else 0) | (TTT_F_Z_BF16 if z_bf16 else 0)
    fn = ttt_diag_mlp_fwd_tcgen05 if kernel == "tcgen05" else ttt_mlp_fwd
    fn(Q, K, V, eta, W1_0, W2_0, ln_gamma, ln_beta, Z, W1o, W2o, B, H, T, d, dh, b,
       _dtype_code(Q), flags, stream)
    return Z, W1o, W2o


def chunk_fwd(Q, K, V, eta, W0, *, chunk, w0_per_seq=False, workspace=None, stream=None,
              want_w=True, z_bf16=False):
    """Large-chunk TTT forward (apply-then-update). Allocates the workspace
    with torch unless one is given. Returns (Z, W_out)."""
    import torch
    B, H, T, d = Q.shape
    Z = torch.empty((B, H, T, d), dtype=torch.bfloat16 if z_bf16 else torch.float32, device=Q.device)
    W_out = torch.empty((B, H, d, d), dtype=torch.float32, device=Q.device) if want_w else None
    need = ttt_chunk_workspace_bytes(B, H, T, d, chunk)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    flags = (TTT_F_W0_PER_SEQ if w0_per_seq else 0) | (TTT_F_Z_BF16 if z_bf16 else 0)
    ttt_chunk_fwd(Q, K, V, eta, W0, Z, W_out, B, H, T, d, chunk, _dtype_code(Q), flags,
                  workspace, need, stream)
    return Z, W_out


def chunk_map(K, V, eta, *, chunk, workspace=None, stream=None):
    """Affine map W -> M W + N of each sequence's chunks (see ttt_chunk_map).
    Returns (M, N), each [B, H, d, d] fp32."""
    import torch
    B, H, T, d = K.shape
    M = torch.empty((B, H, d, d), dtype=torch.float32, device=K.device)
    N = torch.empty_like(M)
    dt = _dtype_code(K)
    need = ttt_chunk_map_workspace_bytes(B, H, T, d, chunk, dt)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=K.device)
    ttt_chunk_map(K, V, eta, M, N, B, H, T, d, chunk, dt, workspace,
                  workspace.numel() * workspace.element_size(), stream)
    return M, N


def linear_map(K, V, eta, *, b, workspace=None, stream=None):
    """Affine map W -> M W + N of each sequence's mini-batches of TTT-Linear
    without LayerNorm (see ttt_linear_map). Returns (M, N), each [B, H, d, d]."""
    import torch
    B, H, T, d = K.shape
    M = torch.empty((B, H, d, d), dtype=torch.float32, device=K.device)
    N = torch.empty_like(M)
    dt = _dtype_code(K)
    need = ttt_linear_map_workspace_bytes(B, H, T, d, b, dt)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=K.device)
    ttt_linear_map(K, V, eta, M, N, B, H, T, d, b, dt, workspace,
                   workspace.numel() * workspace.element_size(), stream)
    return M, N


def affine_prefix(M, N, W0, W_in, W_end=None, *, S, H, nseg, seq_stride, seg_stride,
                  w0_per_seq=False, stream=None):
    """Fold segment maps into starting weights (see ttt_affine_prefix); writes
    W_in and, if given, W_end."""
    d = M.shape[-1]
    ttt_affine_prefix(M, N, W0, W_in, W_end, S, H, nseg, d, seq_stride, seg_stride,
                      TTT_F_W0_PER_SEQ if w0_per_seq else 0, stream)


# The calls below read their shapes off the tensors, check every tensor
# (device, type, shape, contiguous) and run on the tensors' own device, on
# `stream` or that device's current stream; what they allocate belongs to the
# stream that uses it. They are written for calls of a few microseconds: plain
# attribute reads and one C call, no context managers unless the device differs.

def _tensors(fn, index, **want):
    """want: name=(tensor or None, dtypes, shape). Raises ValueError on the first that is off."""
    for name, (t, dtypes, shape) in want.items():
        if t is None or (t.get_device() == index and t.dtype in dtypes and t.shape == shape
                         and t.is_contiguous()):
            continue
        if t.get_device() != index:
            raise ValueError(f"{fn}: {name} is on {t.device}, expected cuda:{index}")
        if t.dtype not in dtypes:
            raise ValueError(f"{fn}: {name} is {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if t.shape != shape:
            raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{fn}: {name} is not contiguous")


class _On:
    """The device and the stream of a call: empty() allocates for it, run() makes it."""

    __slots__ = ("fn", "index", "handle", "side", "torch", "held")

    def __init__(self, fn, first, stream):
        import torch
        index = first.get_device()
        if index < 0:
            raise ValueError(f"{fn}: tensors must be on a CUDA device, got {first.device}")
        self.torch, self.fn, self.index, self.side = torch, fn, index, None
        if stream is None:  # the address alone: a Stream object costs a microsecond
            self.handle = torch._C._cuda_getCurrentRawStream(index)
            return
        current = torch.cuda.current_stream(index)
        self.handle = current.cuda_stream
        if isinstance(stream, int):
            # 0 is the legacy default stream, which torch knows as its default stream
            stream = torch.cuda.ExternalStream(stream, device=first.device) if stream else \
                torch.cuda.default_stream(first.device)
        if stream.device != first.device:
            raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on {first.device}")
        if stream != current:
            self.handle, self.side = stream.cuda_stream, stream

    def uses(self, *tensors):
        """The call reads or writes these (None: nothing): on another stream than the current one
        their memory is not handed out again before the call is done."""
        if self.side is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.side)

    def empty(self, shape, dtype):
        t = self.torch.empty(shape, dtype=dtype, device=self.index)
        if self.side is not None:
            # memory the current stream may still be using: the call waits for
            # that, and the block is not handed out again before the call is done
            self.side.wait_stream(self.torch.cuda.current_stream(self.index))
            t.record_stream(self.side)
        return t

    def like(self, t, dtype):
        """An uninitialised tensor of t's (contiguous) shape."""
        if self.side is not None:
            return self.empty(t.shape, dtype)
        return self.torch.empty_like(t, dtype=dtype)

    def workspace(self, given, need):
        """A workspace of `need` bytes (a given one is checked): its address and size."""
        if given is None:
            if need == 0:  # none is used, or the call refuses its shapes
                return None, 0
            # held to the end of the call: freed before the launch, another
            # thread's allocation on this stream could be put in its place
            self.held = self.empty(max(need, 256), self.torch.uint8)
            return self.held.data_ptr(), max(need, 256)
        if given.get_device() != self.index or not given.is_contiguous():
            raise ValueError(f"{self.fn}: workspace must be contiguous and on cuda:{self.index}")
        self.uses(given)
        return given.data_ptr(), given.numel() * given.element_size()

    def run(self, name, f, *args):
        if self.torch.cuda.current_device() == self.index:
            rc = f(*args, self.handle)
        else:
            with self.torch.cuda.device(self.index):
                rc = f(*args, self.handle)
        if rc != TTT_OK:
            raise TTTError(name, rc)


def _p(t):
    return None if t is None else t.data_ptr()


def _delta_shapes(fn, index, Q, K, V, eta, g, W0, w0_per_seq, seq_start):
    """Checks the inputs of the gated delta rule; returns B, Hk, H, T, dk, dv, n_seq, N, dtype code."""
    import torch
    if Q.dim() != 4 or V.dim() != 4:
        raise ValueError(f"{fn}: Q, K, V must be [B, heads, T, d]")
    B, Hk, T, dk = Q.shape
    _, H, _, dv = V.shape
    n_seq = 0
    if seq_start is not None:
        if seq_start.dim() != 1 or seq_start.numel() < 2:
            raise ValueError(f"{fn}: seq_start must hold n_seq + 1 >= 2 offsets")
        if B != 1:
            raise ValueError(f"{fn}: packed sequences need B = 1, got {B}")
        n_seq = seq_start.numel() - 1
    N = n_seq or B
    code = _dtype_code(Q)
    f32, same = (torch.float32,), (Q.dtype,)
    _tensors(fn, index, Q=(Q, same, (B, Hk, T, dk)), K=(K, same, (B, Hk, T, dk)),
             V=(V, same, (B, H, T, dv)), eta=(eta, f32, (B, H, T)), g=(g, f32, (B, H, T)),
             W0=(W0, f32, (N, H, dk, dv) if w0_per_seq else (H, dk, dv)),
             seq_start=(seq_start, (torch.int32,), (n_seq + 1,)))
    return B, Hk, H, T, dk, dv, n_seq, N, code


def delta_fwd(Q, K, V, eta, g=None, W0=None, *, w0_per_seq=False, seq_start=None, q_scale=1.0,
              z_bf16=False, want_w=True, Z=None, workspace=None, stream=None):
    """Gated delta rule forward (ttt_delta_fwd). Q, K [B, Hk, T, dk], V [B, H, T, dv] (bf16 or
    fp32), eta and g (log decays; None: no decay) [B, H, T] fp32, W0 [H, dk, dv] or, with
    w0_per_seq, [N, H, dk, dv] (None: zero). seq_start: int32 offsets of N packed sequences along
    T (B = 1). Returns (Z [B, H, T, dv], W_out [N, H, dk, dv] or None). Z may be given; its rows
    outside every sequence are left as they are (in a new Z they are undefined)."""
    import torch
    on = _On("delta_fwd", Q, stream)
    B, Hk, H, T, dk, dv, n_seq, N, code = _delta_shapes("delta_fwd", on.index, Q, K, V, eta, g, W0,
                                                        w0_per_seq, seq_start)
    zt = torch.bfloat16 if z_bf16 else torch.float32
    if Z is None:
        Z = on.like(V, zt)
    else:
        _tensors("delta_fwd", on.index, Z=(Z, (zt,), (B, H, T, dv)))
    W_out = on.empty((N, H, dk, dv), torch.float32) if want_w else None
    L = lib()
    ws, nbytes = on.workspace(workspace,
                              L.ttt_delta_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, code))
    on.uses(Q, K, V, eta, g, W0, Z, seq_start)
    on.run("ttt_delta_fwd", L.ttt_delta_fwd, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
           eta.data_ptr(), _p(g), _p(W0), Z.data_ptr(), _p(W_out), _p(seq_start), n_seq, q_scale,
           B, Hk, H, T, dk, dv, code,
           (TTT_F_W0_PER_SEQ if w0_per_seq else 0) | (TTT_F_Z_BF16 if z_bf16 else 0), ws, nbytes)
    return Z, W_out


def delta_bwd(Q, K, V, eta, g, W0, dZ, dW_out=None, *, w0_per_seq=False, seq_start=None,
              q_scale=1.0, workspace=None, stream=None):
    """Gated delta rule backward (ttt_delta_bwd): the gradients of sum(Z dZ) + sum(W_out dW_out)
    for delta_fwd's inputs, as a dict of fp32 tensors Q, K, V, eta and, for what was given, g and
    W0. dZ [B, H, T, dv] and dW_out [N, H, dk, dv] (or None) are fp32."""
    import torch
    on = _On("delta_bwd", Q, stream)
    B, Hk, H, T, dk, dv, n_seq, N, code = _delta_shapes("delta_bwd", on.index, Q, K, V, eta, g, W0,
                                                        w0_per_seq, seq_start)
    f32 = torch.float32
    _tensors("delta_bwd", on.index, dZ=(dZ, (f32,), (B, H, T, dv)),
             dW_out=(dW_out, (f32,), (N, H, dk, dv)))
    grads = {n: on.like(t, f32) for n, t in
             dict(Q=Q, K=K, V=V, eta=eta, g=g, W0=W0).items() if t is not None}
    L = lib()
    ws, nbytes = on.workspace(workspace,
                              L.ttt_delta_bwd_workspace_bytes(B, Hk, H, T, dk, dv, n_seq, code))
    on.uses(Q, K, V, eta, g, W0, dZ, dW_out, seq_start)
    on.run("ttt_delta_bwd", L.ttt_delta_bwd, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
           eta.data_ptr(), _p(g), _p(W0), dZ.data_ptr(), _p(dW_out), grads["Q"].data_ptr(),
           grads["K"].data_ptr(), grads["V"].data_ptr(), grads["eta"].data_ptr(),
           _p(grads.get("g")), _p(grads.get("W0")), _p(seq_start), n_seq, q_scale, B, Hk, H, T, dk,
           dv, code, TTT_F_W0_PER_SEQ if w0_per_seq else 0, ws, nbytes)
    return grads


def _delta_decode(on, Q, K, V, eta, g, W, state_index, q_scale, z_bf16, Z, B, Hk, H, n, dk, dv):
    """The decode call, Q, K, V, eta and g being checked already."""
    torch = on.torch
    zt = torch.bfloat16 if z_bf16 else torch.float32
    if W.dim() != 4:
        raise ValueError("delta_decode: W must be [slots, H, dk, dv]")
    slots = W.shape[0]
    if Z is None:
        Z = on.like(V, zt)
    else:
        _tensors("delta_decode", on.index, Z=(Z, (zt,), V.shape))
    _tensors("delta_decode", on.index, W=(W, (torch.float32,), (slots, H, dk, dv)),
             state_index=(state_index, (torch.int32,), (B,)))
    on.uses(Q, K, V, eta, g, W, Z, state_index)
    on.run("ttt_delta_decode", lib().ttt_delta_decode, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
           eta.data_ptr(), _p(g), W.data_ptr(), Z.data_ptr(), _p(state_index), slots, q_scale, B,
           Hk, H, n, dk, dv, _dtype_code(Q), TTT_F_Z_BF16 if z_bf16 else 0)
    return Z


def delta_decode_tokens(Q, K, V, eta, g, W, *, state_index=None, q_scale=1.0, z_bf16=False, Z=None,
                        stream=None):
    """n tokens of the gated delta rule per row, the states updated in place (ttt_delta_decode).
    Q, K [B, Hk, n, dk], V [B, H, n, dv], eta and g (or None) [B, H, n] fp32, W
    [slots, H, dk, dv] fp32; row b continues state state_index[b] (int32 [B]; None: state b).
    Rows whose index is outside the pool are padding: their Z is left as it is (undefined in a
    new Z). The other rows' indices must be distinct. Returns Z [B, H, n, dv]."""
    on = _On("delta_decode", Q, stream)
    B, Hk, H, n, dk, dv, _, _, _ = _delta_shapes("delta_decode", on.index, Q, K, V, eta, g, None,
                                                 False, None)
    return _delta_decode(on, Q, K, V, eta, g, W, state_index, q_scale, z_bf16, Z, B, Hk, H, n, dk,
                         dv)


def delta_decode(q, k, v, eta, g, W, *, state_index=None, q_scale=1.0, z_bf16=False, z=None,
                 stream=None):
    """delta_decode_tokens for one token per row: q, k [B, Hk, dk], v [B, H, dv], eta and g (or
    None) [B, H]. Returns z [B, H, dv]."""
    on = _On("delta_decode", q, stream)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("delta_decode: q, k, v must be [B, heads, d]")
    B, Hk, dk = q.shape
    _, H, dv = v.shape
    f32, same = (on.torch.float32,), (q.dtype,)
    _tensors("delta_decode", on.index, q=(q, same, (B, Hk, dk)), k=(k, same, (B, Hk, dk)),
             v=(v, same, (B, H, dv)), eta=(eta, f32, (B, H)), g=(g, f32, (B, H)))
    return _delta_decode(on, q, k, v, eta, g, W, state_index, q_scale, z_bf16, z, B, Hk, H, 1, dk,
                         dv)


_ACTS = {"silu": 0, "sigmoid": TTT_F_GATE_SIGMOID}


def _join_shapes(fn, index, X, Z, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta, rms,
                 act):
    """Checks the inputs of the join; returns B, H, T, d, the flags and the dtype code."""
    import torch
    if X.dim() != 3 or (Z is not None and Z.dim() != 4):
        raise ValueError(f"{fn}: expected [B, T, D] and Z [B, H, T, d]")
    if act not in _ACTS:
        raise ValueError(f"{fn}: act must be one of {sorted(_ACTS)}, got {act!r}")
    B, T, D = X.shape
    H, d = (1, D) if Z is None else (Z.shape[1], Z.shape[3])
    if H * d != D:
        raise ValueError(f"{fn}: H * d = {H * d} is not D = {D}")
    code = _dtype_code(X)
    same, f32 = (X.dtype,), (torch.float32,)
    flat = lambda p: (p, f32, (D,) if p is None or p.dim() == 1 else (H, d))  # noqa: E731
    _tensors(fn, index, X=(X, same, (B, T, D)), gate=(gate, same, (B, T, D)),
             Z=(Z, (torch.float32, torch.bfloat16), (B, H, T, d)), scale=flat(scale),
             post_gamma=flat(post_gamma), post_beta=flat(post_beta), pre_gamma=flat(pre_gamma),
             pre_beta=flat(pre_beta))
    flags = (TTT_F_RMS if rms else 0) | _ACTS[act]
    if Z is not None and Z.dtype == torch.bfloat16:
        flags |= TTT_F_Z_BF16
    return B, H, T, d, flags, code


def join_fwd(X, Z, gate=None, scale=None, post_gamma=None, post_beta=None, pre_gamma=None,
             pre_beta=None, *, rms=False, act="silu", eps=1e-5, want_h=True, stream=None):
    """The join between two blocks (ttt_join_fwd): r = x + scale act(gate) (Norm(z) post_gamma +
    post_beta), h = Norm(r) pre_gamma + pre_beta. X, gate [B, T, H d] (bf16 or fp32), Z
    [B, H, T, d] (fp32 or bf16; its norm is per head), the parameters [D] or [H, d] fp32, each
    optional. Returns (R, Hn); Hn is None without want_h. With Z None only Hn = Norm(X) is
    computed, and R is X."""
    on = _On("join_fwd", X, stream)
    B, H, T, d, flags, code = _join_shapes("join_fwd", on.index, X, Z, gate, scale, post_gamma,
                                           post_beta, pre_gamma, pre_beta, rms, act)
    R = None if Z is None else on.like(X, X.dtype)
    Hn = on.like(X, X.dtype) if want_h else None
    on.uses(X, Z, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta)
    on.run("ttt_join_fwd", lib().ttt_join_fwd, X.data_ptr(), _p(Z), _p(gate), _p(scale),
           _p(post_gamma), _p(post_beta), _p(pre_gamma), _p(pre_beta), _p(R), _p(Hn), eps, B, H, T,
           d, code, flags)
    return (X if Z is None else R), Hn


def join_bwd(R, Z, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta, dR, dH, *, rms=False,
             act="silu", eps=1e-5, workspace=None, stream=None):
    """Backward of join_fwd from the stored R (with Z None: X) and the gradients dR and dH
    [B, T, D] fp32 of R and Hn (either may be None: zero). Returns a dict of fp32 gradients: X, and
    for what was given Z, gate, scale, gamma1, beta1 (post_*), gamma2, beta2 (pre_*; not without
    dH)."""
    import torch
    on = _On("join_bwd", R, stream)
    B, H, T, d, flags, code = _join_shapes("join_bwd", on.index, R, Z, gate, scale, post_gamma,
                                           post_beta, pre_gamma, pre_beta, rms, act)
    f32 = torch.float32
    _tensors("join_bwd", on.index, dR=(dR, (f32,), R.shape), dH=(dH, (f32,), R.shape))
    want = dict(X=R, Z=Z, gate=gate, scale=scale, gamma1=post_gamma, beta1=post_beta)
    if dH is not None:
        want.update(gamma2=pre_gamma, beta2=pre_beta)
    g = {n: on.like(t, f32) for n, t in want.items() if t is not None}
    L = lib()
    ws, nbytes = on.workspace(workspace, L.ttt_join_bwd_workspace_bytes(B, H, T, d))
    at = lambda n: _p(g.get(n))  # noqa: E731
    on.uses(R, Z, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta, dR, dH)
    on.run("ttt_join_bwd", L.ttt_join_bwd, R.data_ptr(), _p(Z), _p(gate), _p(scale),
           _p(post_gamma), _p(post_beta), _p(pre_gamma), _p(dR), _p(dH), at("X"), at("Z"),
           at("gate"), at("scale"), at("gamma1"), at("beta1"), at("gamma2"), at("beta2"), eps, B,
           H, T, d, code, flags, ws, nbytes)
    return g
