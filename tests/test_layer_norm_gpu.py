"""GPU parity of layer norm (mm_layer_norm_fwd, mm_layer_norm_bwd) against its
64-bit form in tests/gdr_plain.py.

Tolerances: the statistics and sums are fp32 (2^-24 a rounding) over sums of at
most 16384 terms, formed per thread (16 in turn) and then as a tree (10 levels):
under 32 roundings of the magnitudes summed, and the few operations around them.
bf16 outputs add their own rounding, 2^-8 of the value.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import selective_state_space_momentum_b200 as mm  # noqa: E402
from tests import gdr_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu

F32 = 40 * 2.0 ** -24
BF16 = 2.0 ** -8
COLS = [1, 2, 3, 7, 8, 9, 16, 31, 64, 65, 100, 128, 129, 256, 257, 384, 513, 1000, 1024, 1025, 1536, 2048, 2049, 4096, 4097, 8192, 8193, 12289, 16384]
VARIANTS = {"plain": (False, False, False), "wb": (True, True, False), "wbz": (True, True, True), "z": (False, False, True), "b": (False, True, False)}


def _inputs(rows, cols, io, seed, weight, bias, gate, offset=0.0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    x = (rnd(rows, cols) * (0.2 + torch.rand(rows, 1, generator=gen)) + offset + rnd(rows, 1)).cuda().to(io)
    return (x, (1 + 0.2 * rnd(cols)).cuda() if weight else None, rnd(cols).cuda() if bias else None,
            rnd(rows, cols).cuda().to(io) if gate else None, rnd(rows, cols).cuda().to(io))


def _close(got, want, tol, io, size=None, what=""):
    size = want.abs().amax() if size is None else size
    bound = tol * size + (BF16 * want.abs() if io == torch.bfloat16 else 0) + 1e-30
    worst = ((got.double() - want).abs() - bound).amax()
    assert float(worst) <= 0, f"{what}: past the bound by {float(worst):.2e} (size {float(size):.2e})"


def _check(rows, cols, io, variant, rms, seed=0, offset=0.0, eps=1e-5):
    x, w, b, z, dy = _inputs(rows, cols, io, seed + cols, *VARIANTS[variant], offset=offset)
    y, mean, rstd = mm.layer_norm_fwd(x, w, b, z=z, eps=eps, rms=rms)
    grads = mm.layer_norm_bwd(x, w, b, mean, rstd, dy, z=z, rms=rms)
    want_y, want_mean, want_rstd = plain.norm(x, w, b, z, eps, rms)
    what = f"{rows}x{cols} {io} {variant} rms={rms}"
    # a mean far from zero leaves x - mean with the mean's own rounding
    far = F32 * (1 + float((x.double().abs().mean(-1) * want_rstd).amax()))
    if rms:
        assert mean is None
    else:
        _close(mean, want_mean, F32, None, what=what + " mean")
    assert float(((rstd.double() - want_rstd) / want_rstd).abs().amax()) <= far, what + " rstd"
    _close(y, want_y, far, io, what=what + " y")
    want = plain.norm_grads(x, w, b, z, dy, eps, rms)
    assert set(grads) == set(want)
    for name, g in want.items():
        size = None
        if name in ("dweight", "dbias"):
            # sums over rows: each thread a share of them in turn, then the blocks' in 32 turns and a tree
            size = (dy.double().abs().sum(0) * (1 if z is None else 4)).amax() * (1 if name == "dbias" else float(cols) ** 0.5)
            # (dweight sums dy xh, and xh carries the saved mean's rounding: 2^-24 |mean| rstd, which `far` bounds)
            _close(grads[name], g, 2 * far if name == "dweight" else 2 * F32, None, size, what + " " + name)
            continue
        if name == "dx":
            size = (dy.double().abs().amax() * (1 if w is None else w.abs().amax()) * (1 if z is None else z.double().abs().amax()) * want_rstd.amax()) * 4
        _close(grads[name], g, far, io, size, what + " " + name)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_sizes(cols, io):
    for rows in (1, 5, 67):
        _check(rows, cols, io, "wbz" if cols % 2 else "wb", rms=False)
        _check(rows, cols, io, "wb" if cols % 2 else "wbz", rms=True)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("cols", [24, 33, 640, 1001])
def test_optional_operands(cols, variant):
    for io in (torch.bfloat16, torch.float32):
        for rms in (False, True):
            _check(19, cols, io, variant, rms)


def test_many_rows():
    """More rows than the grid holds at once, every row group of a block in use."""
    _check(40001, 64, torch.bfloat16, "wbz", rms=True)
    _check(9001, 257, torch.float32, "wb", rms=False)
    _check(3001, 2048, torch.bfloat16, "wb", rms=False)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [8, 16, 24, 64, 200, 512, 1000, 1536, 2048, 2056, 4096])
def test_several_rows_a_block(cols, io):
    """Every thread layout with several rows to a block, the last round of them not full; a
    row's results are those of a call of a few rows."""
    rows = 6_000_000 // cols | 1
    _check(rows, cols, io, "wbz", rms=False)
    _check(rows, cols, io, "wb", rms=True)
    x, w, b, z, _ = _inputs(rows, cols, io, 5, True, True, True)
    for gate in (None, z):
        every = mm.layer_norm_fwd(x, w, b, z=gate)
        few = mm.layer_norm_fwd(x[-7:], w, b, z=None if gate is None else gate[-7:])
        assert all(torch.equal(m[-7:], f) for m, f in zip(every, few))


def test_mean_far_from_zero_and_constant_rows():
    _check(9, 1024, torch.float32, "wb", rms=False, offset=3e3)
    _check(9, 1536, torch.bfloat16, "wb", rms=False, offset=50.0)
    x = torch.full((4, 300), 2.5, device="cuda")
    y, mean, rstd = mm.layer_norm_fwd(x, None, None, eps=1e-5)
    assert torch.equal(y, torch.zeros_like(x)) and torch.equal(mean, torch.full((4,), 2.5, device="cuda"))
    assert bool(torch.isfinite(rstd).all())


def test_leading_dimensions_and_skipped_outputs():
    x, w, b, z, dy = _inputs(24, 40, torch.bfloat16, 3, True, True, True)
    y, mean, rstd = mm.layer_norm_fwd(x, w, b, z=z)
    y4, mean4, rstd4 = mm.layer_norm_fwd(x.view(2, 3, 4, 40), w, b, z=z.view(2, 3, 4, 40))
    assert torch.equal(y4.view(24, 40), y) and torch.equal(mean4.view(-1), mean) and rstd4.shape == (2, 3, 4)
    y2 = torch.empty_like(x)
    mm.mm_layer_norm_fwd(x, w, b, z, 1e-5, False, y2, None, None)
    assert torch.equal(y2, y)
    dx = torch.empty_like(x)
    mm.mm_layer_norm_bwd(x, w, b, z, False, mean, rstd, dy, dx, None, None, None, None)
    assert torch.equal(dx, mm.layer_norm_bwd(x, w, b, mean, rstd, dy, z=z)["dx"])


def test_bits_streams_and_graphs():
    x, w, b, z, dy = _inputs(3000, 192, torch.bfloat16, 5, True, True, True)
    y, mean, rstd = mm.layer_norm_fwd(x, w, b, z=z)
    first = mm.layer_norm_bwd(x, w, b, mean, rstd, dy, z=z)
    for _ in range(3):
        again = mm.layer_norm_bwd(x, w, b, mean, rstd, dy, z=z)
        assert all(torch.equal(first[n], again[n]) for n in first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys, ms, rs = mm.layer_norm_fwd(x, w, b, z=z, stream=side)
    gs = mm.layer_norm_bwd(x, w, b, ms, rs, dy, z=z, stream=side)
    side.synchronize()
    assert torch.equal(ys, y) and all(torch.equal(first[n], gs[n]) for n in first)
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, mg, rg = mm.layer_norm_fwd(xs, w, b, z=z)
        gg = mm.layer_norm_bwd(xs, w, b, mg, rg, dy, z=z)
    xs.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yg, mm.layer_norm_fwd(xs, w, b, z=z)[0])
    want = mm.layer_norm_bwd(xs, w, b, mg, rg, dy, z=z)
    assert all(torch.equal(gg[n], want[n]) for n in want)


def test_nan_stays_in_its_row():
    x, w, b, z, dy = _inputs(6, 520, torch.float32, 7, True, True, False)
    clean = mm.layer_norm_fwd(x, w, b)[0]
    x[2, 17] = math.nan
    x[4, 3] = math.inf
    y = mm.layer_norm_fwd(x, w, b)[0]
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[2]).all())
