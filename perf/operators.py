"""The gated delta rule (forward, backward, decode) and the join between two
blocks (norm after, gate, residual scale, residual, norm before; forward and
backward): cases, inputs, a plain form in elementary torch operations, and the
calls of the library.

Gated delta rule, per sequence and value head, W [dk][dv]:
    Wd = exp(g_t) W;  rho = v_t - k_t Wd;  W = Wd + eta_t k_t^T rho;  z_t = c q_t W
Join, per token, D = H d channels:
    n = Norm_d(z) gamma1 + beta1;  r = x + s act(gate) n;  h = Norm_D(r) gamma2 + beta2
"""
import math
import random

import torch

own = False

CHUNK = 64  # tokens per step of the plain forms' recurrence
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    fwd, dec, bwd = "delta_fwd", "delta_decode", "delta_bwd"
    return [
        # a short prompt on a small layer, inputs in fp32: latency
        dict(name="fwd_short_fp32_d64", op=fwd, B=1, T=77, Hk=4, H=4, dk=64, dv=64, seqs=0, dt="fp32", z_bf16=False, w0=False),
        # a training batch of 2,048 tokens, 12 heads
        dict(name="fwd_b8h12_t2048_d64", op=fwd, B=8, T=2048, Hk=12, H=12, dk=64, dv=64, seqs=0, dt="bf16", z_bf16=False, w0=True),
        # prompts of different lengths packed behind one another, keys shared by pairs of value heads, states resumed
        dict(name="fwd_packed_d128", op=fwd, B=1, T=10007, Hk=8, H=16, dk=128, dv=128, seqs=13, dt="bf16", z_bf16=True, w0=True),
        # long context, wide heads
        dict(name="fwd_b4h8_t32768_d128", op=fwd, B=4, T=32768, Hk=8, H=8, dk=128, dv=128, seqs=0, dt="bf16", z_bf16=True, w0=False),
        # one user's next token on a small layer: latency
        dict(name="decode_b1_d64", op=dec, B=1, n=1, Hk=12, H=12, dk=64, dv=64, slots=1, dt="bf16", z_bf16=True),
        # a serving batch whose states live in a pool, one token each
        dict(name="decode_b256_pool_d128", op=dec, B=256, n=1, Hk=8, H=16, dk=128, dv=128, slots=300, dt="bf16", z_bf16=True),
        # a packed training batch with short and long pieces
        dict(name="bwd_packed_d64", op=bwd, B=1, T=1999, Hk=6, H=12, dk=64, dv=64, seqs=5, dt="bf16", w0=True),
        # a training batch of longer sequences, wide heads
        dict(name="bwd_b2h8_t8192_d128", op=bwd, B=2, T=8192, Hk=8, H=8, dk=128, dv=128, seqs=0, dt="bf16", w0=False),
        # one token of a serving batch between two blocks: latency
        dict(name="join_fwd_b33_d768", op="join_fwd", B=33, T=1, H=12, d=64, dt="bf16", z_bf16=True, rms=False, act="silu"),
        # a training batch between two blocks, the read-out in fp32
        dict(name="join_fwd_t32768_d1024", op="join_fwd", B=4, T=8192, H=8, d=128, dt="bf16", z_bf16=False, rms=True, act="silu"),
        # its gradient
        dict(name="join_bwd_t32768_d1024", op="join_bwd", B=4, T=8192, H=8, d=128, dt="bf16", z_bf16=False, rms=True, act="silu"),
        # the gradient over an odd number of tokens, 12 narrow heads, LayerNorm, all in fp32
        dict(name="join_bwd_t2047_fp32_d768", op="join_bwd", B=1, T=2047, H=12, d=64, dt="fp32", z_bf16=False, rms=False, act="sigmoid"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["delta_fwd", "delta_fwd", "delta_decode", "delta_bwd", "join_fwd", "join_bwd"])
    dt = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("join"):
        d = rng.choice([64, 128])
        H = rng.randint(1, 1536 // d)
        B = log(1, 8)
        return dict(op=op, B=B, T=log(1, 20000 // B), H=H, d=d, dt=dt, z_bf16=rng.random() < 0.5, rms=rng.random() < 0.5, act=rng.choice(["silu", "sigmoid"]))
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
    Hk = rng.randint(1, 8)
    H = Hk * rng.choice([1, 1, 2])
    if op == "delta_decode":
        B = log(1, 160)
        return dict(op=op, B=B, n=rng.choice([1, 1, 1, 2, 3, 5]), Hk=Hk, H=H, dk=dk, dv=dv, slots=B + rng.randint(0, 20), dt=dt, z_bf16=rng.random() < 0.5)
    seqs = rng.choice([0, 0, rng.randint(1, 20)])
    B = 1 if seqs else log(1, 4)
    most = 12000 if op == "delta_fwd" else 6000
    c = dict(op=op, B=B, T=max(seqs, log(1, most // B)), Hk=Hk, H=H, dk=dk, dv=dv, seqs=seqs, dt=dt, w0=rng.random() < 0.5)
    if op == "delta_fwd":
        c["z_bf16"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _keys(gen, *shape):
    """Unit keys with a common direction, as projections of real tokens have."""
    x = _normal(gen, *shape) + 0.4 * _normal(gen, *([1] * (len(shape) - 1)), shape[-1])
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _gates(gen, H, *shape):
    """Step sizes in (0, 1), and log decays of heads that forget at different speeds."""
    eta = torch.sigmoid(_normal(gen, *shape))
    rate = torch.logspace(-2, 0.7, H, device="cuda").view([1, H] + [1] * (len(shape) - 2))
    g = -rate * torch.log1p(torch.exp(_normal(gen, *shape) - 2))
    return eta, g


def _lengths(case, seed):
    """Offsets of the packed sequences: uneven, each of one token at least."""
    rng = random.Random(seed * 7919 + case["T"])
    cuts = sorted(rng.sample(range(1, case["T"]), case["seqs"] - 1)) if case["seqs"] > 1 else []
    return [0] + cuts + [case["T"]]


def prepare(case, seed):
    gen, dt, s = _gen(seed), DT[case["dt"]], dict(case=case)
    B, H = case["B"], case["H"]
    if case["op"].startswith("join"):
        T, d = case["T"], case["d"]
        D = H * d
        zt = torch.bfloat16 if case["z_bf16"] else torch.float32
        s.update(X=(2 * _normal(gen, B, T, D)).to(dt), Z=(0.3 * _normal(gen, B, H, T, d) + 0.1).to(zt),
                 gate=_normal(gen, B, T, D).to(dt), scale=0.1 + 0.05 * _normal(gen, D),
                 gamma1=1 + 0.02 * _normal(gen, H, d), beta1=None if case["rms"] else 0.02 * _normal(gen, H, d),
                 gamma2=1 + 0.02 * _normal(gen, D), beta2=None if case["rms"] else 0.02 * _normal(gen, D))
        if case["op"] == "join_bwd":
            s.update(R=(2 * _normal(gen, B, T, D)).to(dt), dR=_normal(gen, B, T, D), dH=_normal(gen, B, T, D))
        return s
    n = case["n"] if case["op"] == "delta_decode" else case["T"]
    Hk, dk, dv = case["Hk"], case["dk"], case["dv"]
    eta, g = _gates(gen, H, B, H, n)
    s.update(Q=_keys(gen, B, Hk, n, dk).to(dt), K=_keys(gen, B, Hk, n, dk).to(dt), V=_normal(gen, B, H, n, dv).to(dt),
             eta=eta, g=g, c=dk ** -0.5)
    if case["op"] == "delta_decode":
        s["W"] = 0.1 * _normal(gen, case["slots"], H, dk, dv)
        s["slot"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        return s
    s["N"] = case["seqs"] or B
    s["W0"] = 0.1 * _normal(gen, s["N"], H, dk, dv) if case["w0"] else None
    s["starts"] = _lengths(case, seed) if case["seqs"] else None
    s["seq_start"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda") if case["seqs"] else None
    if case["op"] == "delta_bwd":
        s["dZ"] = _normal(gen, B, H, n, dv)
        s["dW_out"] = 0.1 * _normal(gen, s["N"], H, dk, dv) if case["w0"] else None
    return s


# ------------------------------------------------------------------ the library's calls

def _run_own(s):
    import test_sequence_layers_layer_b200 as ttt
    c, op = s["case"], s["case"]["op"]
    if op == "delta_fwd":
        return ttt.delta_fwd(s["Q"], s["K"], s["V"], s["eta"], s["g"], s["W0"], w0_per_seq=c["w0"], seq_start=s["seq_start"],
                             q_scale=s["c"], z_bf16=c["z_bf16"])
    if op == "delta_bwd":
        return ttt.delta_bwd(s["Q"], s["K"], s["V"], s["eta"], s["g"], s["W0"], s["dZ"], s["dW_out"], w0_per_seq=c["w0"],
                             seq_start=s["seq_start"], q_scale=s["c"])
    if op == "delta_decode":
        Z = ttt.delta_decode_tokens(s["Q"], s["K"], s["V"], s["eta"], s["g"], s["W"], state_index=s["slot"], q_scale=s["c"],
                                    z_bf16=c["z_bf16"])
        return Z, s["W"]
    norms = (s["gamma1"], s["beta1"], s["gamma2"], s["beta2"])
    if op == "join_fwd":
        return ttt.join_fwd(s["X"], s["Z"], s["gate"], s["scale"], *norms, rms=c["rms"], act=c["act"])
    return ttt.join_bwd(s["R"], s["Z"], s["gate"], s["scale"], *norms, s["dR"], s["dH"], rms=c["rms"], act=c["act"])


# ------------------------------------------------------------------ the plain forms

def _padded(starts, x, length):
    """[1, H, T, ...] packed -> [N, H, length, ...], zeros behind each sequence, and the places of the tokens in it."""
    lens = torch.tensor([b - a for a, b in zip(starts, starts[1:])], device=x.device)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=x.device), lens)
    pos = torch.arange(x.shape[2], device=x.device) - torch.tensor(starts[:-1], device=x.device)[seq]
    y = x.new_zeros((len(lens), x.shape[1], length) + tuple(x.shape[3:]))
    y = y.transpose(1, 2).index_put((seq, pos), x[0].transpose(0, 1)).transpose(1, 2)
    return y, (seq, pos)


def _dense(s, *names):
    """The named inputs in 32 bits, [N, H, L, ...] with L a multiple of CHUNK (padding: zeros), heads repeated for shared keys."""
    starts, T = s["starts"], s["case"]["T"]
    longest = max(b - a for a, b in zip(starts, starts[1:])) if starts else T
    L = -(-longest // CHUNK) * CHUNK
    out, at = [], None
    for name in names:
        x = s[name].float() if torch.is_tensor(s[name]) else s[name]
        if name in ("Q", "K"):
            x = x.repeat_interleave(s["case"]["H"] // s["case"]["Hk"], 1)
        if starts:
            x, at = _padded(starts, x, L)
        else:
            x = torch.cat([x, x.new_zeros(x.shape[:2] + (L - T,) + x.shape[3:])], 2)
        out.append(x)
    return out, at


def _packed(s, x, at):
    """The way back from _dense for an output [N, H, L, ...]."""
    if at is None:
        return x[:, :, :s["case"]["T"]]
    return x.transpose(1, 2)[at].transpose(0, 1).unsqueeze(0)


def _plain_chunks(q, k, v, eta, g, W, c):
    N, H, L, _ = q.shape
    cut = lambda x: x.unflatten(2, (L // CHUNK, CHUNK))  # noqa: E731
    q, k, v, eta, g = (cut(x) for x in (q, k, v, eta, g))
    G = g.double().cumsum(-1)  # sums of decays, and their differences, in 64 bits
    low = torch.ones(CHUNK, CHUNK, device=q.device).tril().bool()
    gam = torch.exp((G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(~low, float("-inf"))).float()
    A = ((k @ k.mT) * gam * eta.unsqueeze(-2)).tril(-1).double()
    P = c * (q @ k.mT) * gam * eta.unsqueeze(-2)
    eye = torch.eye(CHUNK, dtype=torch.double, device=q.device)
    T, sq = eye - A, A
    for _ in range(5):  # (I + A)^-1 = (I - A)(I + A^2)(I + A^4)...: A^64 = 0
        sq = sq @ sq
        T = T @ (eye + sq)
    T = T.float()
    D = torch.exp(G).float().unsqueeze(-1)
    last = torch.exp(G[..., -1]).float()[..., None, None]
    kb = (k * (torch.exp(G[..., -1:] - G).float() * eta).unsqueeze(-1)).mT
    qd, kd = c * q * D, k * D
    z = []
    for i in range(L // CHUNK):  # the recurrence itself
        rho = T[:, :, i] @ (v[:, :, i] - kd[:, :, i] @ W)
        z.append(qd[:, :, i] @ W + P[:, :, i] @ rho)
        W = last[:, :, i] * W + kb[:, :, i] @ rho
    return torch.cat(z, 2), W


def _start_state(s):
    c = s["case"]
    return s["W0"] if s["W0"] is not None else torch.zeros(s["N"], c["H"], c["dk"], c["dv"], device="cuda")


def _plain_fwd(s):
    x, at = _dense(s, "Q", "K", "V", "eta", "g")
    z, W = _plain_chunks(*x, _start_state(s), s["c"])
    z = _packed(s, z, at)
    return (z.bfloat16() if s["case"]["z_bf16"] else z.contiguous()), W


def _plain_bwd(s):
    leaf = dict(s, **{n: s[n].float().requires_grad_() for n in ("Q", "K", "V", "eta", "g")})
    W0 = _start_state(s).clone().requires_grad_()
    x, at = _dense(leaf, "Q", "K", "V", "eta", "g")
    z, W = _plain_chunks(*x, W0, s["c"])
    loss = (_packed(s, z, at) * s["dZ"]).sum()
    if s["dW_out"] is not None:
        loss = loss + (W * s["dW_out"]).sum()
    names = ["Q", "K", "V", "eta", "g"] + (["W0"] if s["W0"] is not None else [])
    grads = torch.autograd.grad(loss, [leaf[n] for n in names[:5]] + [W0][: len(names) - 5])
    return dict(zip(names, grads))


def _plain_decode(s):
    c, slot = s["case"], s["slot"].long()
    q, k = (s[n].float().repeat_interleave(c["H"] // c["Hk"], 1) for n in ("Q", "K"))
    v, W, z = s["V"].float(), s["W"][slot], []
    for t in range(c["n"]):
        W = W * torch.exp(s["g"][:, :, t])[..., None, None]
        rho = v[:, :, t] - (k[:, :, t].unsqueeze(-2) @ W).squeeze(-2)
        W = W + k[:, :, t].unsqueeze(-1) * (s["eta"][:, :, t].unsqueeze(-1) * rho).unsqueeze(-2)
        z.append(s["c"] * (q[:, :, t].unsqueeze(-2) @ W).squeeze(-2))
    s["W"][slot] = W
    return torch.stack(z, 2).to(torch.bfloat16 if c["z_bf16"] else torch.float32), s["W"]


def _norm(x, gamma, beta, rms):
    if not rms:
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma
    return y if beta is None else y + beta


def _branch(s, z, gate, scale, gamma1, beta1):
    c = s["case"]
    n = _norm(z.transpose(1, 2), gamma1, beta1, c["rms"]).flatten(2)
    a = torch.sigmoid(gate)
    return scale * (gate * a if c["act"] == "silu" else a) * n


def _plain_join_fwd(s):
    dt = DT[s["case"]["dt"]]
    r = (s["X"].float() + _branch(s, s["Z"].float(), s["gate"].float(), s["scale"], s["gamma1"], s["beta1"])).to(dt)
    return r, _norm(r.float(), s["gamma2"], s["beta2"], s["case"]["rms"]).to(dt)


def _plain_join_bwd(s, to=torch.float32):
    leaf = {n: s[n].to(to).requires_grad_() for n in ("R", "Z", "gate", "scale", "gamma1", "beta1", "gamma2", "beta2") if s[n] is not None}
    get = leaf.get
    h = _norm(leaf["R"], leaf["gamma2"], get("beta2"), s["case"]["rms"])
    names2 = [n for n in ("gamma2", "beta2") if n in leaf]
    g2 = torch.autograd.grad(h, [leaf["R"]] + [leaf[n] for n in names2], s["dH"].to(to))
    dX = s["dR"].to(to) + g2[0]
    y = _branch(s, leaf["Z"], leaf["gate"], leaf["scale"], leaf["gamma1"], get("beta1"))
    names1 = [n for n in ("Z", "gate", "scale", "gamma1", "beta1") if n in leaf]
    g1 = torch.autograd.grad(y, [leaf[n] for n in names1], dX)
    return dict(zip(["X"] + names2 + names1, (dX,) + g2[1:] + g1))


def run(state):
    if own:
        return _run_own(state)
    return {"delta_fwd": _plain_fwd, "delta_bwd": _plain_bwd, "delta_decode": _plain_decode, "join_fwd": _plain_join_fwd,
            "join_bwd": _plain_join_bwd}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = 2 if case["dt"] == "bf16" else 4
    B, H = case["B"], case["H"]
    if case["op"].startswith("join"):
        n = B * case["T"] * H * case["d"]
        z = 2 if case["z_bf16"] else 4
        if case["op"] == "join_fwd":
            return {"bytes": n * (4 * e + z), "flops": 20 * n}
        return {"bytes": n * (2 * e + z + 8 + 12), "flops": 50 * n}
    dk, dv, Hk = case["dk"], case["dv"], case["Hk"]
    n = B * (case["n"] if case["op"] == "delta_decode" else case["T"])
    io = n * (2 * Hk * dk * e + H * dv * e + 8 * H)
    one = n * H * dk * dv
    if case["op"] == "delta_decode":
        return {"bytes": io + n * H * dv * (2 if case["z_bf16"] else 4) + 8 * B * H * dk * dv, "flops": 7 * one}
    states = 4 * (case["seqs"] or B) * H * dk * dv
    if case["op"] == "delta_fwd":
        return {"bytes": io + n * H * dv * (2 if case["z_bf16"] else 4) + states * (2 if case["w0"] else 1), "flops": 7 * one}
    grads = n * (4 * (2 * Hk * dk + 2 * H * dv) + 8 * H)
    return {"bytes": io + grads + states * (3 if case["w0"] else 0), "flops": 20 * one}


# ------------------------------------------------------------------ 64 bits, token by token

def _exact_heads(s):
    """Q, K, V, eta, g in 64 bits as [S, L, ...] (S sequences x heads, padded with tokens that change nothing), and the lengths."""
    c = s["case"]
    starts = s["starts"] or [0, c["T"]]
    spans = list(zip(starts, starts[1:]))
    L = max(b - a for a, b in spans)
    out = []
    for name in ("Q", "K", "V", "eta", "g") + (("dZ",) if "dZ" in s else ()):
        x = s[name].double()
        if name in ("Q", "K"):
            x = x.unsqueeze(2).expand(-1, -1, c["H"] // c["Hk"], *[-1] * (x.dim() - 2)).flatten(1, 2)
        rows = [x[:, :, a:b] for a, b in spans]
        rows = [torch.cat([r, r.new_zeros(r.shape[:2] + (L - r.shape[2],) + r.shape[3:])], 2) for r in rows]
        out.append(torch.cat(rows, 0).flatten(0, 1))
    return out, spans, L


def _exact_back(s, x, spans):
    """[S, L, ...] -> [B, H, T, ...]."""
    c = s["case"]
    x = x.unflatten(0, (-1, c["H"]))
    if s["starts"] is None:
        return x
    return torch.cat([x[i:i + 1, :, :b - a] for i, (a, b) in enumerate(spans)], 2)


def _exact_step(W, k, v, eta, g):
    W = W * g.exp()[:, None, None]
    rho = v - torch.bmm(k[:, None], W)[:, 0]
    return W, rho, torch.baddbmm(W, k[:, :, None], (eta[:, None] * rho)[:, None])


def _exact_fwd(s):
    (q, k, v, eta, g), spans, L = _exact_heads(s)
    W = _start_state(s).double().flatten(0, 1)
    z = torch.empty_like(v)
    for t in range(L):
        W = _exact_step(W, k[:, t], v[:, t], eta[:, t], g[:, t])[2]
        z[:, t] = s["c"] * torch.bmm(q[:, t, None], W)[:, 0]
    return _exact_back(s, z, spans), W.unflatten(0, (s["N"], -1))


def _exact_bwd(s):
    (q, k, v, eta, g, dz), spans, L = _exact_heads(s)
    W = _start_state(s).double().flatten(0, 1)
    saved = []
    for t in range(L):
        if t % 64 == 0:
            saved.append(W)
        W = _exact_step(W, k[:, t], v[:, t], eta[:, t], g[:, t])[2]
    O = torch.zeros_like(W) if s["dW_out"] is None else s["dW_out"].double().flatten(0, 1)  # noqa: E741
    dq, dk, dv, de, dg = (torch.empty_like(x) for x in (q, k, v, eta, g))
    for c0 in reversed(range(0, L, 64)):
        W, steps = saved[c0 // 64], []
        for t in range(c0, min(c0 + 64, L)):
            Wd, rho, W = _exact_step(W, k[:, t], v[:, t], eta[:, t], g[:, t])
            steps.append((Wd, rho, W))
        for t in reversed(range(c0, min(c0 + 64, L))):
            Wd, rho, W = steps[t - c0]
            dq[:, t] = s["c"] * torch.bmm(W, dz[:, t, :, None])[..., 0]
            O = torch.baddbmm(O, s["c"] * q[:, t, :, None], dz[:, t, None])  # noqa: E741
            kO = torch.bmm(k[:, t, None], O)[:, 0]
            de[:, t] = (kO * rho).sum(-1)
            dv[:, t] = eta[:, t, None] * kO
            dk[:, t] = torch.bmm(O, (eta[:, t, None] * rho)[..., None])[..., 0] - torch.bmm(Wd, dv[:, t, :, None])[..., 0]
            O = torch.baddbmm(O, k[:, t, :, None], dv[:, t, None], alpha=-1)  # noqa: E741
            dg[:, t] = (Wd * O).sum((-1, -2))
            O = O * g[:, t].exp()[:, None, None]  # noqa: E741
    group = lambda x: x.unflatten(1, (s["case"]["Hk"], -1)).sum(2)  # noqa: E731
    back = [_exact_back(s, x, spans) for x in (dq, dk, dv, de, dg)]
    got = dict(Q=group(back[0]), K=group(back[1]), V=back[2], eta=back[3], g=back[4])
    if s["W0"] is not None:
        got["W0"] = O.unflatten(0, (s["N"], -1))
    return got


def _exact_decode(s):
    c = s["case"]
    heads = lambda x: x.double().repeat_interleave(c["H"] // x.shape[1], 1).flatten(0, 1)  # noqa: E731
    q, k, v, eta, g = (heads(s[n]) for n in ("Q", "K", "V", "eta", "g"))
    pool = s["W"].double()
    W, z = pool[s["slot"].long()].flatten(0, 1), torch.empty_like(v)
    for t in range(c["n"]):
        W = _exact_step(W, k[:, t], v[:, t], eta[:, t], g[:, t])[2]
        z[:, t] = s["c"] * torch.bmm(q[:, t, None], W)[:, 0]
    pool[s["slot"].long()] = W.unflatten(0, (c["B"], -1))
    return z.unflatten(0, (c["B"], -1)), pool


def _exact_norm(x, rms):
    """xhat, 1 / sqrt(mean square + eps) of the last axis."""
    m = 0.0 if rms else x.sum(-1, keepdim=True) / x.shape[-1]
    i = 1 / torch.sqrt(((x - m) ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return (x - m) * i, i


def _exact_join(s, bwd):
    c = s["case"]
    x = {n: s[n].double() for n in ("X", "Z", "gate", "scale", "gamma1", "gamma2")}
    add1, add2 = (0.0 if s[n] is None else s[n].double() for n in ("beta1", "beta2"))
    zh, zi = _exact_norm(x["Z"].permute(0, 2, 1, 3), c["rms"])
    n = (zh * x["gamma1"] + add1).flatten(2)
    sg = 1 / (1 + torch.exp(-x["gate"]))
    silu = c["act"] == "silu"
    a = x["gate"] * sg if silu else sg
    if not bwd:
        r = x["X"] + x["scale"] * a * n
        # h is the norm of r as it is stored
        return r, _exact_norm(r.float().to(DT[c["dt"]]).double(), c["rms"])[0] * x["gamma2"] + add2

    def through(dy, xh, i):
        return i * (dy - (0.0 if c["rms"] else dy.mean(-1, keepdim=True)) - xh * (dy * xh).mean(-1, keepdim=True))

    dH = s["dH"].double()
    rh, ri = _exact_norm(s["R"].double(), c["rms"])
    dX = s["dR"].double() + through(dH * x["gamma2"], rh, ri)
    dn = (dX * x["scale"] * a).unflatten(2, (c["H"], c["d"]))
    got = dict(X=dX, gamma2=(dH * rh).sum((0, 1)), scale=(dX * a * n).sum((0, 1)), gamma1=(dn * zh).sum((0, 1)),
               gate=dX * x["scale"] * n * (sg * (1 + x["gate"] * (1 - sg)) if silu else sg * (1 - sg)),
               Z=through(dn * x["gamma1"], zh, zi).permute(0, 2, 1, 3))
    if s["beta1"] is not None:
        got.update(beta1=dn.sum((0, 1)), beta2=dH.sum((0, 1)))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("join"):
        return _exact_join(s, op == "join_bwd")
    return {"delta_fwd": _exact_fwd, "delta_bwd": _exact_bwd, "delta_decode": _exact_decode}[op](s)
