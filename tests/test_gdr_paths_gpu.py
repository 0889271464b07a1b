"""GPU parity of the gated delta rule against the 64-bit recurrence, relative to
whole tensors' norms: the bounds of tests/gdr_rounded.py, which do not grow over
chunks (tests/test_gdr_rounded.py shows on the CPU what they refuse).  Up to 32
chunks, with and without decay; calls large enough for every way the kernels
share work: CTAs of the preparing kernel that take two and four heads, CTAs of
the gradients' kernel that go on to further items.
"""
import pytest

torch = pytest.importorskip("torch")

import selective_state_space_momentum_b200 as mm  # noqa: E402
from tests import gdr_plain as plain  # noqa: E402
from tests import gdr_rounded as rounded  # noqa: E402

pytestmark = pytest.mark.gpu

KINDS = ["random", "no_decay", "strong_decay", "resets", "same_keys", "beta_edges", "zero_keys"]
# batch, L, H, G, P, N: 1, 3, 8 and 32 chunks, every width
SHAPES = [(2, 60, 4, 2, 64, 64), (1, 190, 4, 1, 128, 64), (2, 512, 2, 2, 64, 128), (1, 2040, 2, 1, 128, 128)]


def _reference(q, k, v, g, beta, do, h0, dhT, scale=None):
    o, hT = plain.forward(q, k, v, g, beta, h0, scale)
    want = {"o": o, "hT": hT, **plain.backward(q, k, v, g, beta, do, h0=h0, dhT=dhT, scale=scale)}
    o, hT, kept = rounded.forward(q, k, v, g, beta, h0, scale)
    return want, {"o": o, "hT": hT, **rounded.backward(kept, do, q.shape[2], dhT)}


def _run(q, k, v, g, beta, do, h0, dhT, scale=None):
    o, hT, ckpt = mm.gdr_fwd_train(q, k, v, g, beta, h0=h0, scale=scale, return_last_state=True)
    got = {"o": o, "hT": hT, **mm.gdr_bwd(q, k, v, g, beta, ckpt, do, dhT=dhT, scale=scale, return_dh0=True)}
    mm.mm_device_status()
    return got


def _call(shape, kind, seed):
    *qkvgb, h0 = plain.inputs(*shape, seed=seed, device="cuda", kind=kind, carry=True)
    gen = torch.Generator().manual_seed(seed)
    do = torch.randn(qkvgb[2].shape, generator=gen).cuda().to(torch.bfloat16)
    dhT = torch.randn(h0.shape, generator=gen).cuda()
    return [*qkvgb, do, h0, dhT]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_the_definition(shape, kind):
    args = _call(shape, kind, seed=31 + shape[1])
    got = _run(*args)
    o, hT = mm.gdr_fwd(*args[:5], h0=args[6])
    assert torch.equal(o, got["o"]) and torch.equal(hT, got["hT"])
    rounded.check(got, *_reference(*args), shape[1], f"{shape} {kind}")


@pytest.mark.parametrize("scale", [0.75, -2.0, 0.0])
def test_scale(scale):
    args = _call((1, 150, 4, 2, 64, 128), "random", seed=77)
    got = _run(*args, scale=scale)
    rounded.check(got, *_reference(*args, scale=scale), 150, f"scale {scale}")


@pytest.mark.parametrize("near", [0.9, 0.99, 1.0])
def test_correlated_keys(near):
    """Keys of one direction but for a part: k_i.k_j = near on average, beta = 1, little decay.  The
    rows written are then small differences, and the roundings to bf16 weigh more."""
    q, k, v, g, beta, do, h0, dhT = _call((2, 500, 4, 4, 64, 128), "random", seed=13)
    k = near ** 0.5 * k[:, :1].double() + (1 - near) ** 0.5 * k.double()
    k = (k / k.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    args = [q, k, v, (0.01 * g.double()).to(torch.bfloat16), torch.ones_like(beta), do, h0, dhT]
    rounded.check(_run(*args), *_reference(*args), 500, f"keys {near}")


def test_step_offsets_past_32_bits():
    """A state of more than 2^31 elements: the last requests as in a call of their own."""
    B, H, P, N = 4200, 64, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v, g, beta = r(B, 2, N), r(B, 2, N), r(B, H, P), -r(B, H).abs(), r(B, H).sigmoid()
    h = torch.randn(B, H, P, N, generator=gen, device="cuda")
    assert h.numel() > 2 ** 31
    few = [t[-3:].clone() for t in (q, k, v, g, beta, h)]
    o = mm.gdr_step(q, k, v, g, beta, h)
    assert torch.equal(mm.gdr_step(*few), o[-3:]) and torch.equal(few[5], h[-3:])


def _heads(x, b, h, n):
    return x[b:b + 1, :, h:h + n].contiguous()


# heads of a group: 2 and 4 (as many to a CTA of the preparing kernel), 3 (one each)
@pytest.mark.parametrize("per_group, H", [(2, 32), (4, 64), (3, 12)])
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("N", [64, 128])
def test_large_calls(P, N, per_group, H):
    """38 chunks, the last of 5 steps: 1216 (304 at three heads) items of batch row, group and
    chunk, eight (two) rounds of 148 and a part of one.  Sampled groups against the definition, and
    the same bits as in a call of their own, which is small."""
    L, G = 2373, H // per_group
    chunks, items = 2 * H * 38, 2 * G * 38
    assert items > 2 * 148 and items % 148 and (per_group == 3 or 2 * 4 * 148 * per_group <= chunks)
    q, k, v, g, beta, do, h0, dhT = _call((2, L, H, G, P, N), "random", seed=P + N + H)
    got = _run(q, k, v, g, beta, do, h0, dhT)
    for b, grp in ((0, 0), (1, G - 1), (0, G // 2)):
        h, n = grp * per_group, per_group
        part = [_heads(q, b, grp, 1), _heads(k, b, grp, 1), *(_heads(t, b, h, n) for t in (v, g, beta, do)),
                h0[b:b + 1, h:h + n].contiguous(), dhT[b:b + 1, h:h + n].contiguous()]
        mine = {x: _heads(t, b, *((grp, 1) if x in ("dq", "dk") else (h, n))) for x, t in got.items() if x not in ("hT", "dh0")}
        mine.update({x: got[x][b:b + 1, h:h + n] for x in ("hT", "dh0")})
        alone = _run(*part)
        assert all(torch.equal(mine[x], alone[x]) for x in mine), [x for x in mine if not torch.equal(mine[x], alone[x])]
        rounded.check(mine, *_reference(*part), L, f"{P} {N} {per_group} batch row {b} group {grp}")


@pytest.mark.parametrize("where, value", [("g", float("nan")), ("beta", float("nan")), ("beta", float("inf"))])
@pytest.mark.parametrize("H", [4, 64])
def test_bad_decay_or_strength_stays_in_its_chunk_and_head(where, value, H):
    """As for v: nothing before the chunk, no other batch row, no other head, also where a CTA of the
    preparing kernel takes four heads (64 heads in 16 groups)."""
    L, G = (200, 2) if H == 4 else (2373, 16)
    q, k, v, g, beta, _, _, _ = _call((2, L, H, G, 64, 128), "random", seed=5)
    clean, clean_h = mm.gdr_fwd(q, k, v, g, beta)
    bad = {"g": g.clone(), "beta": beta.clone()}
    bad[where][0, 100, 1] = value
    o, hT = mm.gdr_fwd(q, k, v, bad["g"], bad["beta"])
    mm.mm_device_status()
    others = [h for h in range(H) if h != 1]
    assert torch.equal(o[:, :64], clean[:, :64]) and torch.equal(o[1], clean[1]) and torch.equal(hT[1], clean_h[1])
    assert torch.equal(o[0][:, others], clean[0][:, others]) and torch.equal(hT[0, others], clean_h[0, others])
    assert not bool(torch.isfinite(o[0, 101:, 1].float()).any()) and not bool(torch.isfinite(hT[0, 1]).any())


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
def test_wait_runs_out_after_a_start(monkeypatch, backward):
    """Only the first two chunks (heads) of a CTA staged: the bounded waits give up behind copies and
    products that were issued and are complete, the status says so once, and the next call is right."""
    args = _call((2, 330, 4, 1, 64, 128), "random", seed=9)
    _, _, ckpt = mm.gdr_fwd_train(*args[:5], h0=args[6])
    call = lambda: list(mm.gdr_bwd(*args[:5], ckpt, args[5], return_dh0=True).values()) if backward else list(mm.gdr_fwd(*args[:5], h0=args[6]))
    want = [t.clone() for t in call()]
    monkeypatch.setenv("MMSCAN_FAULT_INJECT", "stall-late")
    call()
    monkeypatch.delenv("MMSCAN_FAULT_INJECT")
    with pytest.raises(mm.MMError) as ei:
        mm.mm_device_status()
    assert ei.value.name == "MM_ERR_DEVICE_TIMEOUT", str(ei.value)
    mm.mm_device_status()
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    mm.mm_device_status()
