"""GPU parity of the gated delta rule (mm_gdr_fwd, mm_gdr_bwd, mm_gdr_step)
against the 64-bit recurrence of tests/gdr_plain.py, through the binding.

Tolerances, from the roundings a value passes (bf16: at most 2^-8 of it, a value
split in two bf16 terms: 2^-16):
* o: its own rounding, and those of Pm and u in sum_j Pm_ij u_j, so element by
  element 2^-8 |o| + 2 2^-8 sum_j |Pm_ij| |u_j|, plus what the state is off;
* the state: a written row u = T x is off by at most 2^-16 for each of x, T,
  S k and the split of tail u, that is 2^-14 of the magnitudes summed (M);
* gradients: up to eight roundings to bf16 on the longest path (dS, Pm, x, T, r,
  u or S, pd or ad, the output); they are independent and the norm of a whole
  tensor adds them in squares: sqrt(8) 2^-8 of its norm.  With equal keys sums
  of 64 terms of alternating sign are what cancels: sqrt(64) of it.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import selective_state_space_momentum_b200 as mm  # noqa: E402
from tests import gdr_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8
GRAD_TOL = math.sqrt(8) * BF16
KINDS = ["random", "no_decay", "strong_decay", "resets", "same_keys", "beta_edges", "zero_keys"]
# batch, L, H, G, P, N: a step, odd lengths, the chunk's edges, several chunks, every width, shared and own keys
SHAPES = [(1, 1, 1, 1, 64, 64), (2, 2, 2, 1, 64, 128), (1, 63, 3, 3, 128, 64), (2, 64, 4, 2, 128, 128), (1, 65, 8, 1, 64, 128),
          (3, 130, 2, 2, 128, 128), (1, 257, 6, 3, 64, 64), (2, 192, 5, 5, 128, 64)]


def _magnitudes(q, k, v, g, beta, h0):
    """(sum_j |Pm_ij| |u_j|, M): the magnitudes o's and the state's sums run over."""
    B, L, H, P = v.shape
    N = k.shape[3]
    q, k, v, g, beta = plain._heads(q, H), plain._heads(k, H), v.double(), g.double().clamp(min=-1e4), beta.double()
    S = v.new_zeros(B, H, P, N) if h0 is None else h0.double()
    M, sums = S.abs(), torch.zeros_like(v)
    for t0 in range(0, L, 64):
        s = slice(t0, min(L, t0 + 64))
        qc, kc, vc, bc = (x[:, s].transpose(1, 2) for x in (q, k, v, beta))
        c = g[:, s].transpose(1, 2).cumsum(-1)
        D = torch.exp((c[..., :, None] - c[..., None, :]).tril()).tril()
        A = bc[..., None] * D * (kc @ kc.mT)
        T = torch.linalg.inv(torch.eye(A.shape[-1], dtype=torch.float64, device=A.device) + A.tril(-1))
        Sk = kc @ S.mT
        x = bc[..., None] * (vc - c.exp()[..., None] * Sk)
        xm = bc[..., None].abs() * (vc.abs() + c.exp()[..., None] * (kc.abs() @ M.mT))
        u, um = T @ x, T.abs() @ xm
        Pm = N ** -0.5 * D * (qc @ kc.mT)
        sums[:, s] = (Pm.abs() @ u.abs()).transpose(1, 2)
        tail = torch.exp(c[..., -1:] - c)[..., None]
        last = torch.exp(c[..., -1])[..., None, None]
        S = last * S + (tail * u).mT @ kc
        M = last * M + (tail * um).mT @ kc.abs()
    return sums, M


def _check_o(o, want, sums, M, k, q, what):
    off = 2 ** -14 * k.shape[3] ** -0.5 * M.abs().amax(-1)[:, None] * q.double().abs().amax()     # the state's part
    bound = BF16 * want.abs() + 2 * BF16 * sums + math.sqrt(k.shape[3]) * off + 1e-30
    bad = ((o.double() - want).abs() > bound).sum()
    assert int(bad) == 0, f"{what}: {int(bad)} of {o.numel()} outside the bound"
    rel = float((o.double() - want).norm() / want.norm().clamp(min=1e-30))
    return rel


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, kind):
    args = plain.inputs(*shape, seed=len(kind) + shape[1], device="cuda", kind=kind,
                        carry=shape[1] % 2 == 0)
    *qkvgb, h0 = args
    o, hT = mm.gdr_fwd(*qkvgb, h0=h0)
    mm.mm_device_status()
    want_o, want_h = plain.forward(*qkvgb, h0)
    sums, M = _magnitudes(*qkvgb, h0)
    _check_o(o, want_o, sums, M, qkvgb[1], qkvgb[0], f"{shape} {kind}")
    assert bool(((hT.double() - want_h).abs() <= 2 ** -14 * M.amax() + 1e-30).all()), f"{shape} {kind} hT"
    assert o.dtype == torch.bfloat16 and hT.dtype == torch.float32


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, kind):
    *qkvgb, h0 = plain.inputs(*shape, seed=7 + shape[1], device="cuda", kind=kind, carry=shape[1] % 2 == 0)
    gen = torch.Generator().manual_seed(shape[1])
    do = torch.randn(qkvgb[2].shape, generator=gen).cuda().to(torch.bfloat16)
    dhT = torch.randn(shape[0], shape[2], shape[4], shape[5], generator=gen).cuda() if shape[1] % 2 == 0 else None
    o, hT, ckpt = mm.gdr_fwd_train(*qkvgb, h0=h0, return_last_state=True)
    got = mm.gdr_bwd(*qkvgb, ckpt, do, dhT=dhT, return_dh0=True)
    mm.mm_device_status()
    o2, hT2 = mm.gdr_fwd(*qkvgb, h0=h0)
    assert torch.equal(o, o2) and torch.equal(hT, hT2)          # keeping the checkpoint changes nothing
    want = plain.backward(*qkvgb, do, h0=h0, dhT=dhT)
    tol = GRAD_TOL * (math.sqrt(64) if kind == "same_keys" else 1)
    for name, w in want.items():
        assert got[name].shape == w.shape
        off = float((got[name].double() - w).norm())
        # dg and dbeta are sums over P x N terms that cancel: of the size of the largest gradient a step can have
        size = float(w.norm())
        if name in ("dg", "dbeta"):
            size = max(size, float((want["dv"].norm() + want["dk"].norm()) * (w.numel() / want["dv"].numel()) ** 0.5))
        assert off <= tol * size + 1e-6, f"{shape} {kind} {name}: {off / max(size, 1e-30):.2e}"


def test_long_sequence_many_heads():
    """More chunks and CTAs than fit at once, on sampled heads."""
    *qkvgb, h0 = plain.inputs(2, 1500, 40, 8, 128, 128, seed=5, device="cuda", carry=True)
    o, hT = mm.gdr_fwd(*qkvgb, h0=h0)
    mm.mm_device_status()
    for h in (0, 7, 39):
        part = [qkvgb[0][:, :, h // 5:h // 5 + 1], qkvgb[1][:, :, h // 5:h // 5 + 1]] + [t[:, :, h:h + 1] for t in qkvgb[2:]]
        want_o, want_h = plain.forward(*part, h0[:, h:h + 1])
        sums, M = _magnitudes(*part, h0[:, h:h + 1])
        assert bool(((hT[:, h:h + 1].double() - want_h).abs() <= 2 ** -14 * M.amax()).all())
        assert float((o[:, :, h:h + 1].double() - want_o).norm() / want_o.norm()) <= math.sqrt(3) * BF16


def test_streaming_is_bit_identical_and_in_place():
    *qkvgb, h0 = plain.inputs(2, 300, 4, 2, 64, 128, seed=1, device="cuda", carry=True)
    o, hT = mm.gdr_fwd(*qkvgb, h0=h0)
    cut = lambda a, b: [t[:, a:b].contiguous() for t in qkvgb]
    first = cut(0, 128)
    o1, h1 = mm.gdr_fwd(*first, h0=h0)
    rest = cut(128, 300)
    o2 = torch.empty_like(rest[2])
    ws = torch.empty(mm.mm_gdr_fwd_workspace_size(2, 172, 4, 64, 128, 2), device="cuda", dtype=torch.uint8)
    mm.mm_gdr_fwd(*rest, h1, 128 ** -0.5, o2, h1, None, ws)      # the state updated in place
    assert torch.equal(torch.cat([o1, o2], 1), o) and torch.equal(h1, hT)


def test_padding_keeps_the_state_and_other_rows():
    """Steps with beta = 0 and g = 0 at a row's end leave its state; a batch row
    of NaN and infinity reaches no other."""
    *qkvgb, h0 = plain.inputs(3, 100, 2, 1, 64, 64, seed=2, device="cuda", carry=True)
    q, k, v, g, beta = (t.clone() for t in qkvgb)
    o_short, h_short = mm.gdr_fwd(*(t[:1, :70].contiguous() for t in (q, k, v, g, beta)), h0=h0[:1].contiguous())
    g[0, 70:], beta[0, 70:] = 0, 0
    for t in (q, k, v):
        t[1] = math.nan
    v[1, ::2] = math.inf
    o, hT = mm.gdr_fwd(q, k, v, g, beta, h0=h0)
    assert torch.equal(hT[0], h_short[0]) and torch.equal(o[0, :70], o_short[0])
    clean_o, clean_h = mm.gdr_fwd(*qkvgb, h0=h0)
    assert torch.equal(o[2], clean_o[2]) and torch.equal(hT[2], clean_h[2])
    assert not bool(torch.isfinite(o[1].float()).any())
    _, _, ckpt = mm.gdr_fwd_train(q, k, v, g, beta, h0=h0)
    do = torch.randn(v.shape, device="cuda").to(v.dtype)
    grads = mm.gdr_bwd(q, k, v, g, beta, ckpt, do)
    assert all(bool(torch.isfinite(t[[0, 2]].float()).all()) for t in grads.values())


def test_nan_stays_in_its_chunk_and_head():
    """A NaN at a step reaches its chunk and what follows, no chunk before it and, in v, no other head."""
    q, k, v, g, beta, _ = plain.inputs(2, 200, 4, 2, 64, 128, seed=4, device="cuda")
    clean, _ = mm.gdr_fwd(q, k, v, g, beta)
    bad = v.clone()
    bad[0, 100, 1, 3] = math.nan
    o, hT = mm.gdr_fwd(q, k, bad, g, beta)
    assert torch.equal(o[:, :64], clean[:, :64]) and torch.equal(o[1], clean[1])
    assert torch.equal(o[0, :, [0, 2, 3]], clean[0, :, [0, 2, 3]])
    assert bool(torch.isnan(o[0, 100:, 1, 3].float()).all()) and bool(torch.isnan(hT[0, 1, 3]).all())
    bad = k.clone()
    bad[0, 100, 1, 3] = math.inf
    o, _ = mm.gdr_fwd(q, bad, v, g, beta)
    assert torch.equal(o[:, :64], clean[:, :64]) and torch.equal(o[1], clean[1]) and torch.equal(o[0, :, :2], clean[0, :, :2])
    assert not bool(torch.isfinite(o[0, 101:, 2:].float()).any())


@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("N", [64, 128])
def test_state_tiles_of_32_and_64_rows(P, N):
    """Calls with fewer and with more tiles of 32 state rows than the GPU has SMs, and the
    checkpointing call: the same bits."""
    *qkvgb, h0 = plain.inputs(6, 150, 40, 8, P, N, seed=P + N, device="cuda", carry=True)
    o, hT = mm.gdr_fwd(*qkvgb, h0=h0)
    kept = mm.gdr_fwd_train(*qkvgb, h0=h0, return_last_state=True)
    assert torch.equal(o, kept[0]) and torch.equal(hT, kept[1])
    few = [t[:, :, h:h + n].contiguous() for t, h, n in zip(qkvgb, (2, 2, 10, 10, 10), (1, 1, 5, 5, 5))]
    few_o, few_h = mm.gdr_fwd(*(t[4:5] for t in few), h0=h0[4:5, 10:15].contiguous())
    assert torch.equal(o[4:5, :, 10:15], few_o) and torch.equal(hT[4:5, 10:15], few_h)


def test_runs_are_bit_identical():
    *qkvgb, h0 = plain.inputs(2, 200, 8, 2, 128, 128, seed=3, device="cuda", carry=True)
    do = torch.randn(qkvgb[2].shape, device="cuda").to(torch.bfloat16)

    def run():
        o, hT, ckpt = mm.gdr_fwd_train(*qkvgb, h0=h0, return_last_state=True)
        return [o, hT, *mm.gdr_bwd(*qkvgb, ckpt, do, return_dh0=True).values()]
    first = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


def test_other_stream_and_graphs_with_one_workspace():
    """A call on a side stream; two captured graphs that share a workspace,
    replayed in turn on new inputs; a captured backward."""
    shape = (1, 150, 4, 4, 64, 64)
    sets = [plain.inputs(*shape, seed=s, device="cuda")[:5] for s in (1, 2, 3)]
    do = torch.randn(sets[0][2].shape, device="cuda").to(torch.bfloat16)
    want = []
    for s in sets:
        o, hT, ckpt = mm.gdr_fwd_train(*s, return_last_state=True)
        want.append((o, hT, mm.gdr_bwd(*s, ckpt, do)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, hT = mm.gdr_fwd(*sets[0], stream=side)
    side.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(hT, want[0][1])

    sizes = (1, 150, 4, 64, 64, 4)
    ws = torch.empty(mm.mm_gdr_fwd_workspace_size(*sizes), device="cuda", dtype=torch.uint8)
    ins = [[t.clone() for t in sets[0]] for _ in range(2)]
    outs = [(torch.empty_like(sets[0][2]), torch.empty(1, 4, 64, 64, device="cuda")) for _ in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mm.mm_gdr_fwd(*ins[i], None, 64 ** -0.5, outs[i][0], outs[i][1], None, ws)
        graphs.append(g)
    for s in (1, 2):
        for i in range(2):
            for dst, src in zip(ins[i], sets[s]):
                dst.copy_(src)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for o, hT in outs:
            assert torch.equal(o, want[s][0]) and torch.equal(hT, want[s][1])

    train = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, _, ckpt = mm.gdr_fwd_train(*train)
        grads = mm.gdr_bwd(*train, ckpt, do)
    eager = mm.gdr_bwd(*sets[0], mm.gdr_fwd_train(*sets[0])[2], do)
    for dst, src in zip(train, sets[2]):
        dst.copy_(src)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(grads[n], want[2][2][n]) for n in grads)
    assert all(torch.equal(eager[n], want[0][2][n]) for n in eager)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 4), (3, 4, 2, 64, 128), (2, 6, 3, 37, 100), (5, 2, 1, 128, 256), (1, 3, 3, 7, 12), (33, 8, 8, 96, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step(shape, io):
    """fp32 arithmetic: sums of up to 256 products, log2(256) + 2 roundings of 2^-24 each way of the magnitudes."""
    B, H, G, P, N = shape
    q, k, v, g, beta, h = plain.inputs(B, 1, H, G, P, N, seed=P, dtype=io, device="cuda", carry=True)
    q, k, v, g, beta = (t[:, 0].contiguous() for t in (q, k, v, g, beta))
    want_o, want_h = plain.step(q, k, v, g, beta, h)
    mags = (h.double().abs().sum(-1).amax() + v.double().abs().amax())
    o = mm.gdr_step(q, k, v, g, beta, h)
    assert bool(((h.double() - want_h).abs() <= 16 * 2 ** -24 * mags).all())
    bound = (BF16 * want_o.abs() if io == torch.bfloat16 else 0) + 32 * 2 ** -24 * mags
    assert bool(((o.double() - want_o).abs() <= bound).all())


def test_step_clears_on_minus_infinity():
    q, k, v, g, beta, h = plain.inputs(2, 1, 2, 2, 8, 16, seed=1, device="cuda", carry=True)
    q, k, v, g, beta = (t[:, 0].contiguous() for t in (q, k, v, g, beta))
    g[0] = -math.inf
    want_o, want_h = plain.step(q, k, v, g, beta, h)
    o = mm.gdr_step(q, k, v, g, beta, h)
    assert bool(((h.double() - want_h).abs() <= 1e-6).all()) and bool(torch.isfinite(o.float()).all())


def test_prefill_then_decode():
    """A prompt, then single steps, against the recurrence over all of it."""
    *qkvgb, _ = plain.inputs(2, 90, 4, 2, 64, 128, seed=6, device="cuda")
    head = [t[:, :70].contiguous() for t in qkvgb]
    o, h = mm.gdr_fwd(*head)
    outs = [o]
    for t in range(70, 90):
        outs.append(mm.gdr_step(*(x[:, t].contiguous() for x in qkvgb), h)[:, None])
    want_o, want_h = plain.forward(*qkvgb)
    sums, M = _magnitudes(*qkvgb, None)
    _check_o(torch.cat(outs, 1), want_o, sums, M, qkvgb[1], qkvgb[0], "prefill and decode")
    assert bool(((h.double() - want_h).abs() <= 2 ** -14 * M.amax()).all())


def test_layer_forward_and_backward():
    """The delta rule and the gated norm of its heads as a layer uses them: the
    output and the gradients reaching the layer's inputs."""
    shape = (2, 140, 4, 2, 64, 64)
    *qkvgb, _ = plain.inputs(*shape, seed=8, device="cuda")
    gen = torch.Generator().manual_seed(1)
    z = torch.randn(qkvgb[2].shape, generator=gen).cuda().to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(64, generator=gen)).cuda()
    dy = torch.randn(z.shape, generator=gen).cuda().to(torch.bfloat16)
    o, _, ckpt = mm.gdr_fwd_train(*qkvgb)
    y, _, rstd = mm.layer_norm_fwd(o, w, z=z, rms=True)
    ng = mm.layer_norm_bwd(o, w, None, None, rstd, dy, z=z, rms=True)
    grads = mm.gdr_bwd(*qkvgb, ckpt, ng["dx"])
    want_o, _ = plain.forward(*qkvgb)
    want_y = plain.norm(want_o, w, None, z, rms=True)[0]
    want_ng = plain.norm_grads(want_o, w, None, z, dy, rms=True)
    want = plain.backward(*qkvgb, want_ng["dx"])
    # o's three roundings, then y's; dx adds o's rounding inside the norm and its own to the chain's eight.
    # The norm divides rows of small o by their size: the relative error of a row is that of o's row, whatever its size.
    rows = (o.double() - want_o).norm(dim=-1) / want_o.norm(dim=-1).clamp(min=1e-30)
    assert float((y.double() - want_y).norm() / want_y.norm()) <= 2 * float(rows.square().mean().sqrt()) + 2 * BF16
    assert float((ng["dweight"].double() - want_ng["dweight"]).norm() / want_ng["dweight"].norm()) <= 2 * float(rows.square().mean().sqrt()) + BF16
    row_tol = 4 * float(rows.square().mean().sqrt()) + 4 * BF16
    for name, t in grads.items():
        assert float((t.double() - want[name]).norm() / want[name].norm()) <= GRAD_TOL + row_tol, name


def test_two_calls_at_once():
    """Two streams, each its own call with its own workspace, many times over."""
    sets = [plain.inputs(2, 200, 4, 2, 128, 64, seed=s, device="cuda", carry=True) for s in (11, 12)]
    want = [mm.gdr_fwd(*s[:5], h0=s[5]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[mm.gdr_fwd(*s[:5], h0=s[5], stream=st) for s, st in zip(sets, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    mm.mm_device_status()
    for pair in got:
        assert all(torch.equal(a, b) for one, ref in zip(pair, want) for a, b in zip(one, ref))


def test_offsets_past_32_bits():
    """v of more than 2^31 elements: the last batch row as in a call of its own."""
    B, L, H, P, N = 9, 65600, 32, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)
    q, k = (torch.nn.functional.normalize(rnd(B, L, 1, N).float(), dim=-1).to(torch.bfloat16) for _ in range(2))
    v, do = rnd(B, L, H, P), rnd(B, L, H, P)
    g, beta = -rnd(B, L, H).abs(), rnd(B, L, H).sigmoid()
    assert v.numel() > 2 ** 31
    o, hT, ckpt = mm.gdr_fwd_train(q, k, v, g, beta, return_last_state=True)
    grads = mm.gdr_bwd(q, k, v, g, beta, ckpt, do)
    mm.mm_device_status()
    del ckpt
    last = [t[-1:] for t in (q, k, v, g, beta)]
    o1, h1 = mm.gdr_fwd(*last)
    assert torch.equal(o[-1:], o1) and torch.equal(hT[-1:], h1)
    _, _, ckpt = mm.gdr_fwd_train(*last)
    assert all(torch.equal(grads[n][-1:], t) for n, t in mm.gdr_bwd(*last, ckpt, do[-1:]).items())


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
def test_wait_runs_out(monkeypatch, backward):
    """Nothing staged (no copy is in flight): the bounded waits give up, the status says so
    once, and the next call is right."""
    *qkvgb, h0 = plain.inputs(2, 130, 4, 2, 64, 128, seed=9, device="cuda", carry=True)
    do = torch.randn(qkvgb[2].shape, device="cuda").to(torch.bfloat16)
    call = lambda: mm.gdr_bwd(*qkvgb, ckpt, do, return_dh0=True).values() if backward else mm.gdr_fwd(*qkvgb, h0=h0)
    _, _, ckpt = mm.gdr_fwd_train(*qkvgb, h0=h0)
    want = [t.clone() for t in call()]
    monkeypatch.setenv("MMSCAN_FAULT_INJECT", "stall")
    call()
    monkeypatch.delenv("MMSCAN_FAULT_INJECT")
    with pytest.raises(mm.MMError) as ei:
        mm.mm_device_status()
    assert ei.value.name == "MM_ERR_DEVICE_TIMEOUT", str(ei.value)
    mm.mm_device_status()
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    mm.mm_device_status()
