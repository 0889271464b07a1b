"""The gated delta rule and layer norm in 64 bits, step by step and element by
element, for the tests: the recurrence as it is defined, its gradients by
walking the steps back, and the inputs the tests share."""
import math

import torch


def inputs(batch, L, H, G, P, N, seed=0, dtype=torch.bfloat16, device="cpu", kind="random", carry=False):
    """Inputs of a call: `kind` picks the decays and keys that make it hard."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    q, k, v = rnd(batch, L, G, N), rnd(batch, L, G, N), rnd(batch, L, H, P)
    q = q / q.norm(dim=-1, keepdim=True)
    k = k / k.norm(dim=-1, keepdim=True)
    g = -torch.exp(math.log(1e-3) + math.log(1e3) * torch.rand(batch, L, H, generator=gen))
    beta = torch.rand(batch, L, H, generator=gen)
    if kind == "no_decay":
        g = torch.zeros_like(g)
    elif kind == "strong_decay":                     # whole chunks decay past fp32's range
        g = 20 * g - 1
    elif kind == "resets":                           # some steps forget everything
        hit = torch.rand(g.shape, generator=gen) < 0.15
        g = torch.where(hit, torch.where(torch.rand(g.shape, generator=gen) < 0.5, -1e5, -math.inf), g)
    elif kind == "same_keys":                        # k_i.k_j = 1: the triangular system at its worst
        k = k[:, :1].expand_as(k).contiguous()
        beta = torch.ones_like(beta)
        g = 0.01 * g
    elif kind == "beta_edges":
        beta = torch.randint(0, 3, beta.shape, generator=gen).float()      # 0, 1 and 2
    elif kind == "zero_keys":
        k[:, ::3] = 0
    h0 = 0.3 * rnd(batch, H, P, N) if carry else None
    put = lambda t: t.to(device).to(dtype).contiguous()
    return put(q), put(k), put(v), put(g), put(beta), None if h0 is None else h0.to(device)


def _heads(x, H):
    return x.double().repeat_interleave(H // x.shape[2], dim=2)


def forward(q, k, v, g, beta, h0=None, scale=None):
    """(o, hT) in 64 bits."""
    B, L, H, P = v.shape
    N = k.shape[3]
    scale = N ** -0.5 if scale is None else scale
    q, k, v, a, beta = _heads(q, H), _heads(k, H), v.double(), g.double().exp(), beta.double()
    S = v.new_zeros(B, H, P, N) if h0 is None else h0.double()
    o = []
    for t in range(L):
        S = a[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None]
        o.append(scale * (S * q[:, t, :, None]).sum(-1))
    return torch.stack(o, 1), S


def backward(q, k, v, g, beta, do, h0=None, dhT=None, scale=None):
    """dict of dq, dk, dv, dg, dbeta, dh0 in 64 bits, the steps walked back."""
    B, L, H, P = v.shape
    G, N = k.shape[2:]
    scale = N ** -0.5 if scale is None else scale
    q, k, v, a, beta, do = _heads(q, H), _heads(k, H), v.double(), g.double().exp(), beta.double(), do.double()
    S = v.new_zeros(B, H, P, N) if h0 is None else h0.double()
    kept = []
    for t in range(L):
        D = a[:, t, :, None, None] * S
        w = v[:, t] - (D * k[:, t, :, None]).sum(-1)
        S = D + (beta[:, t, :, None] * w)[..., None] * k[:, t, :, None]
        kept.append((D, w, S))
    grads = {n: [None] * L for n in ("dq", "dk", "dv", "dg", "dbeta")}
    dS = torch.zeros_like(S) if dhT is None else dhT.double()
    for t in reversed(range(L)):
        D, w, S = kept[t]
        dS = dS + scale * do[:, t, :, :, None] * q[:, t, :, None]
        grads["dq"][t] = scale * (S * do[:, t, :, :, None]).sum(2)
        dSk = (dS * k[:, t, :, None]).sum(-1)
        dw = beta[:, t, :, None] * dSk
        grads["dbeta"][t] = (w * dSk).sum(-1)
        grads["dv"][t] = dw
        grads["dk"][t] = (dS * (beta[:, t, :, None] * w)[..., None]).sum(2) - (D * dw[..., None]).sum(2)
        dS = dS - dw[..., None] * k[:, t, :, None]
        grads["dg"][t] = (dS * D).sum((-1, -2))
        dS = a[:, t, :, None, None] * dS
    out = {n: torch.stack(x, 1) for n, x in grads.items()}
    for n in ("dq", "dk"):
        out[n] = out[n].reshape(B, L, G, H // G, N).sum(3)
    return {**out, "dh0": dS}


def step(q, k, v, g, beta, h, scale=None):
    o, S = forward(q[:, None], k[:, None], v[:, None], g[:, None], beta[:, None], h, scale)
    return o[:, 0], S


def norm(x, weight=None, bias=None, z=None, eps=1e-5, rms=False):
    """(y, mean, rstd) in 64 bits."""
    x = x.double()
    mean = torch.zeros_like(x[..., 0]) if rms else x.mean(-1)
    c = x - mean[..., None]
    rstd = 1 / torch.sqrt((c * c).mean(-1) + eps)
    n = c * rstd[..., None]
    if weight is not None:
        n = n * weight.double()
    if bias is not None:
        n = n + bias.double()
    if z is not None:
        n = n * z.double() * torch.sigmoid(z.double())
    return n, mean, rstd


def norm_grads(x, weight, bias, z, dy, eps=1e-5, rms=False):
    """Gradients of norm() by the elementary derivatives of its 64-bit form."""
    leaves = {n: t.detach().double().requires_grad_() for n, t in (("dx", x), ("dweight", weight), ("dbias", bias), ("dz", z)) if t is not None}
    y = norm(leaves["dx"], leaves.get("dweight"), leaves.get("dbias"), leaves.get("dz"), eps, rms)[0]
    return dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), dy.double())))
