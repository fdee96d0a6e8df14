"""Oracle of the gated delta rule and of the join between two blocks: float64,
token by token, straight from the definitions; gradients by autograd through
them. Independent of the library's chunked forms."""
from __future__ import annotations

import torch


def _f64(x):
    return None if x is None else torch.as_tensor(x).detach().cpu().double()


def delta(Q, K, V, eta, g=None, W0=None, *, seq_start=None, w0_per_seq=False, q_scale=1.0):
    """Z [B, H, T, dv] (zero outside the sequences) and W_out [N, H, dk, dv], differentiable.
    Per token: Wd = exp(g) W, rho = v - k Wd, W = Wd + eta k^T rho, z = q_scale q W."""
    B, Hk, T, dk = Q.shape
    H, dv = V.shape[1], V.shape[3]
    spans = [(0, 0, T)] * B if seq_start is None else \
        [(0, int(a), int(b)) for a, b in zip(seq_start[:-1], seq_start[1:])]
    rep = H // Hk
    rows = {}
    W_out = []
    for n, (_, a, b) in enumerate(spans):
        batch = n if seq_start is None else 0
        if W0 is None:
            W = torch.zeros(H, dk, dv, dtype=torch.float64)
        else:
            W = W0[n] if w0_per_seq else W0
        for t in range(a, b):
            q = Q[batch, :, t].repeat_interleave(rep, 0)
            k = K[batch, :, t].repeat_interleave(rep, 0)
            if g is not None:
                W = torch.exp(g[batch, :, t])[:, None, None] * W
            rho = V[batch, :, t] - torch.einsum("hk,hkv->hv", k, W)
            W = W + torch.einsum("hk,hv->hkv", k, eta[batch, :, t, None] * rho)
            rows[batch, t] = q_scale * torch.einsum("hk,hkv->hv", q, W)
        W_out.append(W)
    zero = torch.zeros(H, dv, dtype=torch.float64)
    Z = torch.stack([torch.stack([rows.get((b, t), zero) for t in range(T)], 1) for b in range(B)])
    return Z, torch.stack(W_out)


def delta_f64(Q, K, V, eta, g=None, W0=None, **kw):
    """delta() of any tensors, in float64."""
    return delta(*(_f64(x) for x in (Q, K, V, eta, g, W0)), **kw)


def delta_grads(Q, K, V, eta, g, W0, dZ, dW_out=None, **kw):
    """Gradients of sum(Z dZ) + sum(W_out dW_out): dict Q, K, V, eta and, if given, g, W0."""
    x = {n: _f64(t).requires_grad_() for n, t in
         dict(Q=Q, K=K, V=V, eta=eta, g=g, W0=W0).items() if t is not None}
    Z, W = delta(x["Q"], x["K"], x["V"], x["eta"], x.get("g"), x.get("W0"), **kw)
    loss = (Z * _f64(dZ)).sum()
    if dW_out is not None:
        loss = loss + (W * _f64(dW_out)).sum()
    got = torch.autograd.grad(loss, list(x.values()), allow_unused=True)
    return {n: torch.zeros_like(x[n]) if y is None else y for n, y in zip(x, got)}


def _norm(x, gamma, beta, rms, eps):
    if not rms:
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if gamma is not None:
        y = y * gamma
    return y if beta is None else y + beta


def join(X, Z, gate=None, scale=None, post_gamma=None, post_beta=None, *, rms=False, act="silu",
         eps=1e-5):
    """r of the join: [B, T, D], Z [B, H, T, d], differentiable."""
    B, H, T, d = Z.shape
    head = lambda p: None if p is None else p.reshape(H, 1, d)  # noqa: E731
    y = _norm(Z, head(post_gamma), head(post_beta), rms, eps).transpose(1, 2).reshape(B, T, H * d)
    if gate is not None:
        y = y * torch.sigmoid(gate) * (gate if act == "silu" else 1)
    if scale is not None:
        y = y * scale.reshape(-1)
    return X + y


def norm(R, pre_gamma=None, pre_beta=None, *, rms=False, eps=1e-5):
    flat = lambda p: None if p is None else p.reshape(-1)  # noqa: E731
    return _norm(R, flat(pre_gamma), flat(pre_beta), rms, eps)


def join_grads(R, Z, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta, dR, dH, *,
               rms=False, act="silu", eps=1e-5):
    """Gradients of sum(r dR) + sum(h dH) at the stored r: dict X, and for what is given Z, gate,
    scale, gamma1, beta1, gamma2, beta2."""
    leaf = lambda t: None if t is None else _f64(t).requires_grad_()  # noqa: E731
    r, g2, b2 = leaf(R), leaf(pre_gamma), leaf(pre_beta)
    dX = torch.zeros_like(r) if dR is None else _f64(dR)
    got = {}
    if dH is not None:
        wrt = [t for t in (r, g2, b2) if t is not None]
        gr = torch.autograd.grad(norm(r, g2, b2, rms=rms, eps=eps), wrt, _f64(dH))
        dX = dX + gr[0]
        got.update(zip([n for n, t in (("gamma2", g2), ("beta2", b2)) if t is not None], gr[1:]))
    got["X"] = dX.detach()
    if Z is not None:
        x = {n: leaf(t) for n, t in dict(Z=Z, gate=gate, scale=scale, gamma1=post_gamma,
                                         beta1=post_beta).items() if t is not None}
        y = join(torch.zeros_like(r), x["Z"], x.get("gate"), x.get("scale"), x.get("gamma1"),
                 x.get("beta1"), rms=rms, act=act, eps=eps)
        got.update(zip(x, torch.autograd.grad(y, list(x.values()), got["X"])))
    return got
