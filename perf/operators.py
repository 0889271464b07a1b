"""The gated delta rule (chunked forward, its training step, the decode step) and layer norm (forward, training step):
the calls a user makes of them, their plain forms in elementary torch operations, and their definitions in 64 bits.

Gated delta rule, per batch row and head, state S (P, N), decay a_t = exp(g_t), write strength beta_t:
    S_t = a_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   o_t = scale S_t q_t,   scale = 1 / sqrt(N)
q, k (batch, L, G, N), shared by the H / G heads of a group; v, o (batch, L, H, P); g, beta (batch, L, H); S (batch, H, P, N).

Layer norm of the rows of x (rows, cols), with an optional gate z:
    y = ((x - mean) rstd w + b) silu(z),   rstd = 1 / sqrt(var + eps);   rms: mean = 0, var = the mean square.
"""
import math

import torch

own = False

CHUNK = 64          # steps the plain form takes at once
EPS = 1e-5


def listed():
    return [
        # One short prompt of a chat request, continued from a cached state: latency.
        dict(name="prompt_short", op="gdr_fwd", batch=1, seqlen=61, heads=32, headdim=128, dstate=128, groups=16, carry=True),
        # Prefill at the sizes of this repository's chunked-scan benchmark: 32 heads of 64 share one group.
        dict(name="prompt_batch", op="gdr_fwd", batch=4, seqlen=4096, heads=32, headdim=64, dstate=128, groups=1, carry=False),
        # One long document, a length that is no multiple of anything.
        dict(name="prompt_long", op="gdr_fwd", batch=1, seqlen=16397, heads=32, headdim=128, dstate=128, groups=16, carry=False),
        # Training step of a small model, forward and backward.
        dict(name="train_small", op="gdr_train", batch=2, seqlen=1000, heads=8, headdim=64, dstate=64, groups=8, carry=False),
        # Training step with a query and key of its own for every head.
        dict(name="train", op="gdr_train", batch=4, seqlen=2048, heads=16, headdim=128, dstate=128, groups=16, carry=False),
        # Training step with queries and keys shared by four heads each, odd length.
        dict(name="train_shared", op="gdr_train", batch=2, seqlen=4099, heads=32, headdim=64, dstate=128, groups=8, carry=False),
        # Decoding for one request: latency.
        dict(name="step_one", op="gdr_step", batch=1, heads=32, headdim=128, dstate=128, groups=16, io="bf16"),
        # Decoding for the 512 requests of this repository's decode benchmark.
        dict(name="step_512", op="gdr_step", batch=512, heads=32, headdim=64, dstate=128, groups=1, io="bf16"),
        # The norm before a layer while decoding for a few requests: latency.
        dict(name="norm_decode", op="norm_fwd", rows=37, cols=2048, io="bf16", gate=False, rms=False),
        # The norm over (batch 4, L 2048) tokens of 1536 channels in fp32.
        dict(name="norm_tokens", op="norm_fwd", rows=8192, cols=1536, io="f32", gate=False, rms=False),
        # The gated norm of every head's output, as it follows the delta rule in a layer; training step.
        dict(name="norm_heads_train", op="norm_train", rows=524288, cols=64, io="bf16", gate=True, rms=True),
        # The norm over (batch 8, L 4096) tokens of 2048 channels in bf16; training step.
        dict(name="norm_train", op="norm_train", rows=32768, cols=2048, io="bf16", gate=False, rms=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gdr_fwd", "gdr_train", "gdr_step", "norm_fwd", "norm_train"))
    if op in ("gdr_fwd", "gdr_train"):
        P, N = rng.choice((64, 128)), rng.choice((64, 128))
        batch = rng.choice((1, 2, 3, 4))
        groups = rng.choice((1, 2, 3, 4, 8))
        heads = groups * rng.choice((1, 2, 4))
        longest = min(16397 if op == "gdr_fwd" else 4099, 4 * 4096 * 32 // (2 * batch * heads))
        return dict(op=op, batch=batch, seqlen=_spread(rng, 1, longest), heads=heads, headdim=P, dstate=N, groups=groups,
                    carry=op == "gdr_fwd" and rng.random() < 0.5)
    if op == "gdr_step":
        groups = rng.choice((1, 2, 5, 16))
        return dict(op=op, batch=_spread(rng, 1, 512), heads=groups * rng.choice((1, 2)), headdim=rng.choice((32, 64, 96, 128)),
                    dstate=rng.choice((32, 64, 96, 128)), groups=groups, io=rng.choice(("bf16", "f32")))
    cols = _spread(rng, 3, 12289)
    return dict(op=op, rows=_spread(rng, 1, max(2, 2 ** 25 // cols)), cols=cols, io=rng.choice(("bf16", "f32")),
                gate=rng.random() < 0.5, rms=rng.random() < 0.5)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    io = torch.float32 if case.get("io") == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = (normal(rows, cols) * (0.5 + uniform(rows, 1)) + 0.5 * normal(rows, 1)).to(io)
        s["weight"] = 1 + 0.1 * normal(cols)
        s["bias"] = None if case["rms"] else 0.1 * normal(cols)
        s["z"] = normal(rows, cols).to(io) if case["gate"] else None
        s["dy"] = normal(rows, cols).to(io) if case["op"] == "norm_train" else None
        return s
    lead = (case["batch"],) if case["op"] == "gdr_step" else (case["batch"], case["seqlen"])
    H, G, P, N = case["heads"], case["groups"], case["headdim"], case["dstate"]
    q, k = normal(*lead, G, N), normal(*lead, G, N)
    s["q"] = (q / q.square().sum(-1, keepdim=True).sqrt()).to(io)
    s["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).to(io)
    s["v"] = normal(*lead, H, P).to(io)
    # the step sizes and decay rates of this repository's chunked-scan benchmark
    step = torch.exp(math.log(1e-3) + math.log(100.0) * uniform(*lead, H))
    s["g"] = (-step * (1 + 15 * uniform(H))).to(io)
    s["beta"] = (1 / (1 + torch.exp(-normal(*lead, H)))).to(io)
    if case["op"] == "gdr_step":
        s["h"] = 0.3 * normal(case["batch"], H, P, N)
    else:
        s["h0"] = 0.3 * normal(case["batch"], H, P, N) if case["carry"] else None
    s["do"] = normal(*lead, H, P).to(io) if case["op"] == "gdr_train" else None
    return s


# ------------------------------------------------------------ plain forms ----
def _chunked(x, heads):
    """(batch, L, heads or groups, ...) to (batch, heads, chunks, CHUNK, ...) in 32 bits, zeros past L."""
    x = x.float().repeat_interleave(heads // x.shape[2], dim=2).movedim(2, 1)
    short = -x.shape[2] % CHUNK
    if short:
        x = torch.cat([x, x.new_zeros(x.shape[:2] + (short,) + x.shape[3:])], dim=2)
    return x.reshape(x.shape[:2] + (-1, CHUNK) + x.shape[3:])


def _steps(x, like):
    """The inverse of _chunked, rounded to the type of `like`; groups' values are the sums over their heads."""
    x = x.flatten(2, 3)[:, :, :like.shape[1]].movedim(1, 2)
    if x.shape[2] != like.shape[2]:
        x = x.reshape(x.shape[:2] + (like.shape[2], -1) + x.shape[3:]).sum(3)
    return x.to(like.dtype)


def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower A: inverses of diagonal blocks of 1, 2, 4, ... joined."""
    T = torch.eye(CHUNK, device=A.device).expand(A.shape).clone()
    for s in (1, 2, 4, 8, 16, 32):
        for i in range(0, CHUNK, 2 * s):
            a, b = slice(i, i + s), slice(i + s, i + 2 * s)
            T[..., b, a] = -T[..., b, b] @ A[..., b, a] @ T[..., a, a]
    return T


def _gdr_chunks(s):
    """What both directions share: the chunks' operands, masks and the states at their starts."""
    H, N = s["v"].shape[2], s["k"].shape[3]
    q, k, v = (_chunked(s[n], H) for n in ("q", "k", "v"))
    g, beta = (_chunked(s[n], H)[..., None] for n in ("g", "beta"))
    q = q / math.sqrt(N)
    c = g.double().cumsum(-2)                                 # 64 bits: differences of long sums
    low = torch.ones(CHUNK, CHUNK, device=q.device, dtype=torch.bool).tril()
    D = torch.where(low, torch.exp((c - c.mT).masked_fill(~low, 0.0)).float(), 0.0)
    eg, tail, last = torch.exp(c).float(), torch.exp(c[..., -1:, :] - c).float(), torch.exp(c[..., -1:, :]).float()
    A = beta * D * (k @ k.mT)
    A = A - torch.diag_embed(A.diagonal(dim1=-2, dim2=-1))
    T, P = _unit_lower_inverse(A), D * (q @ k.mT)
    S = q.new_zeros(q.shape[:2] + (v.shape[-1], N)) if s["h0"] is None else s["h0"].clone()
    starts, new = [], []
    for i in range(q.shape[2]):
        starts.append(S)
        kS = k[:, :, i] @ S.mT
        u = T[:, :, i] @ (beta[:, :, i] * (v[:, :, i] - eg[:, :, i] * kS))
        S = last[:, :, i] * S + (tail[:, :, i] * u).mT @ k[:, :, i]
        new.append(u)
    return q, k, v, beta, D, eg, tail, last, A, T, P, torch.stack(starts, 2), torch.stack(new, 2), S


def _plain_gdr_fwd(s):
    q, k, v, beta, D, eg, tail, last, A, T, P, S, u, hT = _gdr_chunks(s)
    return {"o": _steps(eg * (q @ S.mT) + P @ u, s["v"]), "hT": hT}


def _plain_gdr_train(s):
    q, k, v, beta, D, eg, tail, last, A, T, P, S, u, hT = _gdr_chunks(s)
    do = _chunked(s["do"], v.shape[1])
    du, dSs, dr = P.mT @ do, [], []
    dS = torch.zeros_like(hT)                                 # the gradient reaching the state after the chunk
    for i in reversed(range(q.shape[2])):
        dSs.append(dS)
        r = T[:, :, i].mT @ (du[:, :, i] + tail[:, :, i] * (k[:, :, i] @ dS.mT))
        dS = last[:, :, i] * dS + (eg[:, :, i] * do[:, :, i]).mT @ q[:, :, i] - (beta[:, :, i] * eg[:, :, i] * r).mT @ k[:, :, i]
        dr.append(r)
    dS, dr = torch.stack(dSs[::-1], 2), torch.stack(dr[::-1], 2)
    dP, dA = do @ u.mT, -(dr @ u.mT)
    qS, kS, kdS = eg * (do @ S), eg * (dr @ S), tail * (u @ dS)
    pd, ad = dP * D, (dA * beta * D).tril(-1)
    dq = pd @ k + qS
    dk = pd.mT @ q + (ad + ad.mT) @ k + kdS - beta * kS
    own_k, own_w = (k * kdS).sum(-1), (k * kS).sum(-1)
    dbeta = (dr * v).sum(-1) - own_w + (dA * D * (k @ k.mT)).tril(-1).sum(-1)
    PP, AA = (dP * P).double(), (dA * A).double()
    dc = PP.sum(-1) - PP.sum(-2) + AA.sum(-1) - AA.sum(-2) + (q * qS).sum(-1) - beta[..., 0] * own_w - own_k
    dc[..., -1] += last[..., 0, 0] * (S * dS).sum((-1, -2)) + own_k.sum(-1)
    dg = dc.flip(-1).cumsum(-1).flip(-1)
    return {"o": _steps(eg * (q @ S.mT) + P @ u, s["v"]), "dq": _steps(dq / math.sqrt(q.shape[-1]), s["q"]), "dk": _steps(dk, s["k"]),
            "dv": _steps(beta * dr, s["v"]), "dg": _steps(dg, s["g"]), "dbeta": _steps(dbeta, s["beta"])}


def _plain_gdr_step(s):
    H, N = s["v"].shape[1], s["k"].shape[2]
    q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], dim=1) for n in ("q", "k"))
    h = s["h"].mul_(torch.exp(s["g"].float())[..., None, None])
    u = s["beta"].float()[..., None] * (s["v"].float() - (h * k[:, :, None]).sum(-1))
    h.add_(u[..., None] * k[:, :, None])
    return {"o": ((h * q[:, :, None]).sum(-1) / math.sqrt(N)).to(s["v"].dtype), "h": h}


def _plain_norm(s):
    rms, x = s["case"]["rms"], s["x"].float()
    mean = x.new_zeros(x.shape[0]) if rms else x.mean(-1)
    x = x - mean[:, None]
    rstd = 1 / torch.sqrt(x.square().mean(-1) + EPS)
    xh = x * rstd[:, None]
    n = xh * s["weight"] + (0 if s["bias"] is None else s["bias"])
    if s["z"] is None:
        return xh, n, n, mean, rstd
    z = s["z"].float()
    return xh, n, n * (z / (1 + torch.exp(-z))), mean, rstd


def _plain_norm_fwd(s):
    xh, n, y, mean, rstd = _plain_norm(s)
    out = {"y": y.to(s["x"].dtype), "rstd": rstd}
    return out if s["case"]["rms"] else {**out, "mean": mean}


def _plain_norm_train(s):
    xh, n, y, mean, rstd = _plain_norm(s)
    dy, out = s["dy"].float(), {"y": y.to(s["x"].dtype)}
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1 / (1 + torch.exp(-z))
        out["dz"] = (dy * n * sig * (1 + z * (1 - sig))).to(s["z"].dtype)
        dy = dy * z * sig
    d = dy * s["weight"]
    dx = d - xh * (d * xh).mean(-1, keepdim=True)
    if not s["case"]["rms"]:
        dx = dx - d.mean(-1, keepdim=True)
    out["dx"] = (dx * rstd[:, None]).to(s["x"].dtype)
    out["dweight"] = (dy * xh).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


# ------------------------------------------------------- the user's calls ----
def _own(s):
    import selective_state_space_momentum_b200 as mm

    op = s["case"]["op"]
    if op == "gdr_fwd":
        o, hT = mm.gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["h0"])
        return {"o": o, "hT": hT}
    if op == "gdr_train":
        o, _, ckpt = mm.gdr_fwd_train(s["q"], s["k"], s["v"], s["g"], s["beta"])
        return {"o": o, **mm.gdr_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], ckpt, s["do"])}
    if op == "gdr_step":
        return {"o": mm.gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h"]), "h": s["h"]}
    rms = s["case"]["rms"]
    y, mean, rstd = mm.layer_norm_fwd(s["x"], s["weight"], s["bias"], z=s["z"], eps=EPS, rms=rms)
    if op == "norm_fwd":
        return {"y": y, "rstd": rstd} if rms else {"y": y, "rstd": rstd, "mean": mean}
    return {"y": y, **mm.layer_norm_bwd(s["x"], s["weight"], s["bias"], mean, rstd, s["dy"], z=s["z"], rms=rms)}


_PLAIN = {"gdr_fwd": _plain_gdr_fwd, "gdr_train": _plain_gdr_train, "gdr_step": _plain_gdr_step,
          "norm_fwd": _plain_norm_fwd, "norm_train": _plain_norm_train}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


def work(case):
    eb = 4 if case.get("io") == "f32" else 2
    if case["op"].startswith("norm"):
        n = case["rows"] * case["cols"]
        gate, train = int(case["gate"]), case["op"] == "norm_train"
        # forward x, z, y; a training step also reads dy and writes dx, dz
        tensors = 2 + gate + (2 + gate if train else 0)
        rows = (1 if case["rms"] else 2) * case["rows"] * 4
        return {"bytes": tensors * n * eb + (0 if train else rows) + (2 if train else 1) * case["cols"] * (4 if case["rms"] else 8),
                "flops": n * (8 + 4 * gate + (14 + 8 * gate if train else 0))}
    H, G, P, N = case["heads"], case["groups"], case["headdim"], case["dstate"]
    tokens = case["batch"] * case.get("seqlen", 1)
    into, state = tokens * (2 * G * N + H * P + 2 * H) * eb, case["batch"] * H * P * N * 4
    o = tokens * H * P * eb
    if case["op"] == "gdr_train":            # q, k, v, g, beta, do in; o and the five gradients out
        return {"bytes": 2 * into + 2 * o, "flops": tokens * H * (6 + 14) * P * N}
    states = 2 if case["op"] == "gdr_step" or case["carry"] else 1
    return {"bytes": into + o + states * state, "flops": tokens * H * 6 * P * N}


# ------------------------------------------------- the definition, 64 bits ----
def _exact_norm(s, train):
    rms, eps, x, w = s["case"]["rms"], EPS, s["x"].double(), s["weight"].double()
    cols = x.shape[1]
    mean = torch.zeros_like(x[:, :1]) if rms else x.sum(1, keepdim=True) / cols
    rstd = ((x - mean).pow(2).sum(1, keepdim=True) / cols + eps).pow(-0.5)
    xh = (x - mean) * rstd
    n = xh * w if s["bias"] is None else xh * w + s["bias"].double()
    z = None if s["z"] is None else s["z"].double()
    gate = 1.0 if z is None else z * torch.sigmoid(z)
    out = {"y": n * gate}
    if not train:
        out["rstd"] = rstd[:, 0]
        if not rms:
            out["mean"] = mean[:, 0]
        return out
    dy = s["dy"].double()
    if z is not None:
        out["dz"] = dy * n * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
    dn = dy * gate
    dxh = dn * w
    # xh = (x - mean) rstd: through the mean, and through rstd by d rstd / dx = -rstd^2 xh / cols
    drstd = (dxh * (x - mean)).sum(1, keepdim=True)
    dx = dxh * rstd - drstd * rstd.pow(2) * xh / cols
    if not rms:
        dx = dx - (dxh * rstd).sum(1, keepdim=True) / cols
    out["dx"], out["dweight"] = dx, (dn * xh).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dn.sum(0)
    return out


def _exact_steps(s):
    """The operands of the recurrence by step, heads apart: lists of (batch, H, ...) in 64 bits."""
    H = s["v"].shape[2]
    wide = {n: s[n].double().repeat_interleave(H // s[n].shape[2], dim=2) for n in ("q", "k")}
    return [t.unbind(1) for t in (wide["q"], wide["k"], s["v"].double(), s["g"].double().exp(), s["beta"].double())]


def _exact_advance(S, k, v, a, beta):
    decayed = S * a[..., None, None]
    write = v - torch.einsum("bhpn,bhn->bhp", decayed, k)
    return decayed, write, decayed + torch.einsum("bhp,bhn->bhpn", beta[..., None] * write, k)


def _exact_gdr(s, train):
    q, k, v, a, beta = _exact_steps(s)
    B, L, H, P = s["v"].shape
    N = s["k"].shape[3]
    scale, every = N ** -0.5, 64
    S = torch.zeros(B, H, P, N, device=s["v"].device, dtype=torch.float64) if s["h0"] is None else s["h0"].double()
    kept, o = [], []
    for t in range(L):
        if t % every == 0:
            kept.append(S)
        S = _exact_advance(S, k[t], v[t], a[t], beta[t])[2]
        o.append(scale * torch.einsum("bhpn,bhn->bhp", S, q[t]))
    o = torch.stack(o, 1)
    if not train:
        return {"o": o, "hT": S}
    do = s["do"].double().unbind(1)
    grads = {n: [None] * L for n in ("dq", "dk", "dv", "dg", "dbeta")}
    G = torch.zeros_like(S)
    for first in reversed(range(0, L, every)):
        S, path = kept.pop(), []
        for t in range(first, min(L, first + every)):
            decayed, write, S = _exact_advance(S, k[t], v[t], a[t], beta[t])
            path.append((decayed, write, S))
        for t in reversed(range(first, min(L, first + every))):
            decayed, write, S = path.pop()
            G = G + scale * torch.einsum("bhp,bhn->bhpn", do[t], q[t])
            grads["dq"][t] = scale * torch.einsum("bhpn,bhp->bhn", S, do[t])
            Gk = torch.einsum("bhpn,bhn->bhp", G, k[t])
            dwrite = beta[t][..., None] * Gk
            grads["dbeta"][t] = (write * Gk).sum(-1)
            grads["dv"][t] = dwrite
            grads["dk"][t] = torch.einsum("bhpn,bhp->bhn", G, beta[t][..., None] * write) - torch.einsum("bhpn,bhp->bhn", decayed, dwrite)
            G = G - torch.einsum("bhp,bhn->bhpn", dwrite, k[t])
            grads["dg"][t] = (G * decayed).sum((-1, -2))
            G = G * a[t][..., None, None]
    out = {n: torch.stack(t, 1) for n, t in grads.items()}
    for n in ("dq", "dk"):
        out[n] = out[n].reshape(B, L, s["k"].shape[2], -1, N).sum(3)
    return {"o": o, **out}


def _exact_step(s):
    H, N = s["v"].shape[1], s["k"].shape[2]
    q, k = (s[n].double().repeat_interleave(H // s[n].shape[1], dim=1) for n in ("q", "k"))
    S = _exact_advance(s["h"].double(), k, s["v"].double(), s["g"].double().exp(), s["beta"].double())[2]
    return {"o": N ** -0.5 * torch.einsum("bhpn,bhn->bhp", S, q), "h": S}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s, case["op"] == "norm_train")
    if case["op"] == "gdr_step":
        return _exact_step(s)
    return _exact_gdr(s, case["op"] == "gdr_train")
