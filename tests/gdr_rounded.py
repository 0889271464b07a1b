"""The chunked gated delta rule in 64 bits with the roundings to bf16 that the
kernels make, at the places where they make them, for the tests: how far from
the definition those roundings alone take a result.

`single`: names of values that are to be rounded to one bf16 term where the
kernels keep two ("S", "T", "x", "w": the decayed rows u), for tests that such a
loss is noticed.
"""
import math

import torch

from tests.gdr_plain import _heads

CHUNK = 64


def bf(x):
    return x.to(torch.bfloat16).double()


def _two(x, one=False):
    hi = bf(x)
    return (hi, torch.zeros_like(hi)) if one else (hi, bf(x - hi))


def _chunks(x, n):
    """(B, L, H, ...) to (B, H, n, CHUNK, ...), zeros past L."""
    pad = n * CHUNK - x.shape[1]
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
    return x.movedim(2, 1).reshape(x.shape[0], x.shape[2], n, CHUNK, *x.shape[3:])


def _steps(x, L):
    return x.flatten(2, 3)[:, :, :L].movedim(1, 2)


def _product(a, b):
    """a b of values in two terms each, without the product of the two low ones."""
    return a[0] @ (b[0] + b[1]) + a[1] @ b[0]


def _inverse(A):
    """(I + A)^-1 in blocks of 16: those on the diagonal by substitution, the others
    T_ij = -T_ii sum_{j<=m<i} A_im T_mj with every operand in two terms; in two terms itself."""
    blk = lambda i: slice(16 * i, 16 * i + 16)
    eye = torch.eye(16, dtype=A.dtype, device=A.device)
    Th, Tl = torch.zeros_like(A), torch.zeros_like(A)
    for i in range(4):
        t = torch.linalg.solve_triangular(eye + A[..., blk(i), blk(i)], eye.expand(*A.shape[:-2], 16, 16), upper=False)
        Th[..., blk(i), blk(i)], Tl[..., blk(i), blk(i)] = _two(t)
    part = lambda x, i, j: (x[0][..., blk(i), blk(j)], x[1][..., blk(i), blk(j)])
    a = _two(A)
    for j in range(4):
        for i in range(j + 1, 4):
            s = sum(_product(part(a, i, m), part((Th, Tl), m, j)) for m in range(j, i))
            Th[..., blk(i), blk(j)], Tl[..., blk(i), blk(j)] = _two(-_product(part((Th, Tl), i, i), _two(s)))
    return Th, Tl


def forward(q, k, v, g, beta, h0=None, scale=None, single=()):
    """(o, hT, kept): kept is what backward() needs."""
    L, H, N = v.shape[1], v.shape[2], k.shape[3]
    n = -(-L // CHUNK)
    scale = N ** -0.5 if scale is None else scale
    q, k, v = (_chunks(t, n) for t in (_heads(q, H), _heads(k, H), v.double()))
    g, beta = _chunks(g.double().clamp(min=-1e4), n), _chunks(beta.double(), n)[..., None]
    c = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=c.device).tril()
    D = torch.where(low, torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~low, 0.0)), 0.0)
    eg, tail, last = c.exp()[..., None], torch.exp(c[..., -1:] - c)[..., None], c[..., -1:].exp()[..., None]
    kk = k @ k.mT
    A = (beta * D * kk).tril(-1)
    Th, Tl = _inverse(A)
    if "T" in single:
        Tl = torch.zeros_like(Tl)
    Pm = scale * D * (q @ k.mT)
    S = v.new_zeros(*v.shape[:2], v.shape[-1], N) if h0 is None else h0.double()
    starts, us, os = [], [], []
    for i in range(n):
        starts.append(S)
        Sh, Sl = _two(S, "S" in single)
        x = beta[:, :, i] * (v[:, :, i] - eg[:, :, i] * (k[:, :, i] @ (Sh + Sl).mT))
        xh, xl = _two(x, "x" in single)
        u = Th[:, :, i] @ (xh + xl) + Tl[:, :, i] @ xh
        os.append(scale * eg[:, :, i] * (q[:, :, i] @ (Sh + Sl).mT) + bf(Pm[:, :, i]) @ bf(u))
        wh, wl = _two(tail[:, :, i] * u, "w" in single)
        S = last[:, :, i] * S + (wh + wl).mT @ k[:, :, i]
        us.append(u)
    kept = dict(q=q, k=k, v=v, beta=beta, D=D, eg=eg, tail=tail, last=last, kk=kk, Th=Th, Pm=Pm, S=torch.stack(starts, 2),
                u=torch.stack(us, 2), L=L, scale=scale)
    return bf(_steps(torch.stack(os, 2), L)), S, kept


def backward(kept, do, groups, dhT=None):
    """dict of dq, dk, dv, dg, dbeta, dh0."""
    f = kept
    q, k, v, beta, D, eg, tail, last, scale, L = (f[x] for x in ("q", "k", "v", "beta", "D", "eg", "tail", "last", "scale", "L"))
    n = q.shape[2]
    do = _chunks(do.double(), n)
    S, u, Pm = bf(f["S"]), bf(f["u"]), bf(f["Pm"])
    dS = torch.zeros_like(f["S"][:, :, 0]) if dhT is None else dhT.double()
    ends, rs = [], []
    for i in reversed(range(n)):
        dSb = bf(dS)
        ends.append(dSb)
        x = tail[:, :, i] * (k[:, :, i] @ dSb.mT) + Pm[:, :, i].mT @ do[:, :, i]
        r = f["Th"][:, :, i].mT @ bf(x)
        rs.append(r)
        dS = (last[:, :, i] * dS + bf(-beta[:, :, i] * eg[:, :, i] * r).mT @ k[:, :, i]
              + bf(scale * eg[:, :, i] * do[:, :, i]).mT @ q[:, :, i])
    dSe, r = torch.stack(ends[::-1], 2), torch.stack(rs[::-1], 2)
    rb = bf(r)
    ru, dou = rb @ u.mT, do @ u.mT
    pd, ad = scale * D * dou, -(beta * D * ru).tril(-1)
    Y, Z = rb @ S, u @ dSe
    doS = do @ S
    dq = bf(pd) @ k + scale * eg * doS
    dk = bf(pd).mT @ q + (bf(ad) + bf(ad).mT) @ k + tail * Z - beta * eg * Y
    kY, kZ, qS = (k * Y).sum(-1), (k * Z).sum(-1), (q * doS).sum(-1)
    e, t, b = eg[..., 0], tail[..., 0], beta[..., 0]
    dbeta = (rb * v).sum(-1) - e * kY - (D * f["kk"] * ru).tril(-1).sum(-1)
    W = (pd * (q @ k.mT) + ad * f["kk"]).tril(-1)
    dc = W.sum(-1) - W.sum(-2) + scale * e * qS - b * e * kY - t * kZ
    dc[..., -1] += last[..., 0, 0] * (S * dSe).sum((-1, -2)) + (t * kZ).sum(-1)
    dg = dc.flip(-1).cumsum(-1).flip(-1)
    out = dict(dq=_steps(dq, L), dk=_steps(dk, L), dv=_steps(beta * r, L), dg=_steps(dg, L), dbeta=_steps(dbeta, L))
    for name in ("dq", "dk"):
        x = out[name]
        out[name] = x.reshape(x.shape[0], L, groups, -1, x.shape[-1]).sum(3)
    return {**{name: bf(x) for name, x in out.items()}, "dh0": dS}


# ------------------------------------------------------------- the bounds ----
# hT: every value on its way is kept in two bf16 terms.  A rounding to bf16 is off
# by 0.41 2^-8 of the value in the mean square (uniform in half a step of 2^-8 at
# the bottom of a binade), two terms by the square of that, 2.5e-6; S, x, T (with
# the product of the two low terms left out, in T's own formation too) and the
# rows decayed are five such values, whose errors add in squares: 5.7e-6, under
# 1e-5.  (With nearly equal keys T and the rows written are differences of larger
# sums; the emulated error says by how much more.)  And a chunk adds to the state
# in 8 steps of fp32 (two terms, 64 rows in steps of 16), each off by 2^-24 of it
# on average.
def state_tol(L):
    return 1e-5 + -(-L // CHUNK) * 2.0 ** -21


# o and the gradients: the kernels make the roundings of this file at the values
# of this file, up to sums of fp32 that tip a rounding now and then, so their
# error has the size of the emulated one.  A quarter more, and what the two-term
# values leave (2^-16 of what is summed up).
MARGIN, REST = 1.25, 2.0 ** -16


def check(got, want, emulated, L, what=""):
    """Relative to the norm of the whole tensor.  `got`, `want`, `emulated`: dicts with any of o, hT, dq ... dh0."""
    for name, w in want.items():
        off = float((got[name].double() - w).norm())
        if name == "hT":
            bound = state_tol(L) * float(w.norm()) + MARGIN * max(0.0, float((emulated[name] - w).norm()) - 1e-5 * float(w.norm()))
        else:
            size = float(w.norm())
            if name in ("dg", "dbeta"):              # sums over the products of a step's gradients, which may cancel
                size = max(size, float(want["dv"].norm()) + float(want["dk"].norm()))
            bound = MARGIN * float((emulated[name] - w).norm()) + REST * size
        assert off <= bound + 1e-30, f"{what} {name}: off by {off:.3e}, bound {bound:.3e}, norm {float(w.norm()):.3e}"
    return True


def wrong(got, want, emulated, L, name):
    """Whether check() refuses tensor `name` of `got`."""
    try:
        keep = {name: want[name]} if name not in ("dg", "dbeta") else {n: want[n] for n in (name, "dv", "dk")}
        check({**emulated, name: got}, keep, emulated, L)
    except AssertionError:
        return True
    return False
