"""Layer norm of more than 2^31 elements: the last rows as in a call of their own,
and the weight's and the bias's gradients against sums over the pieces."""
import pytest

torch = pytest.importorskip("torch")

import selective_state_space_momentum_b200 as mm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [2048, 2049], ids=["pieces of 16 bytes", "by element"])
def test_offsets_past_32_bits(cols):
    rows = 2 ** 31 // cols + 1000
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    dy = torch.empty_like(x).normal_(generator=gen)
    w = 1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")
    b = 0.1 * torch.randn(cols, generator=gen, device="cuda")
    assert x.numel() > 2 ** 31
    y, mean, rstd = mm.layer_norm_fwd(x, w, b)
    grads = mm.layer_norm_bwd(x, w, b, mean, rstd, dy)
    tail = slice(rows - 8, rows)                              # (8 rows of any width start on 16 bytes where all rows are even)
    part = [t[tail].clone() for t in (x, dy, mean, rstd)]
    yt, mt, rt = mm.layer_norm_fwd(part[0], w, b)
    assert torch.equal(yt, y[tail]) and torch.equal(mt, mean[tail]) and torch.equal(rt, rstd[tail])
    assert torch.equal(mm.layer_norm_bwd(part[0], w, b, mt, rt, part[1])["dx"], grads["dx"][tail])
    del y, yt
    dw, db = torch.zeros(cols, device="cuda", dtype=torch.float64), torch.zeros(cols, device="cuda", dtype=torch.float64)
    for r in range(0, rows, 1 << 17):
        s = slice(r, min(rows, r + (1 << 17)))
        d = dy[s].double()
        dw += (d * ((x[s].double() - mean[s, None]) * rstd[s, None])).sum(0)
        db += d.sum(0)
    # rows a thread adds in turn (a million over 592 blocks at most, so 2000), 32 blocks in turn and 5 levels: 2^-24
    # of the running sum each, whose size grows as the root of the rows; added in squares under 2^-24 sqrt(rows) sqrt(2000)
    bound = 2.0 ** -24 * rows ** 0.5 * 2000 ** 0.5 * 4
    assert float((grads["dbias"].double() - db).abs().max()) <= bound
    assert float((grads["dweight"].double() - dw).abs().max()) <= bound + rows ** 0.5 * 2.0 ** -20
