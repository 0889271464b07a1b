"""The allocating wrappers on a side stream while work on a block that was just
freed is still queued on the current stream: that work keeps its data, and the
call its results.  Nothing orders the side stream behind the current one."""
import pytest

torch = pytest.importorskip("torch")

import selective_state_space_momentum_b200 as mm  # noqa: E402
from tests import gdr_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu


def _gdr():
    *qkvgb, _ = plain.inputs(2, 200, 4, 2, 64, 128, seed=21, device="cuda")
    return qkvgb


def _gdr_fwd():
    a = _gdr()
    return lambda s: mm.gdr_fwd(*a, stream=s)


def _gdr_fwd_train():
    a = _gdr()
    return lambda s: mm.gdr_fwd_train(*a, return_last_state=True, stream=s)[:2]


def _gdr_bwd():
    a = _gdr()
    ckpt = mm.gdr_fwd_train(*a)[2]
    return lambda s: mm.gdr_bwd(*a, ckpt, a[2], return_dh0=True, stream=s)


def _gdr_step():
    a = [t[:, 0].contiguous() for t in _gdr()]
    h = torch.randn(2, 4, 64, 128, device="cuda")
    return lambda s: mm.gdr_step(*a, h.clone() if s is None else _cloned(h, s), stream=s)


def _cloned(t, stream):
    with torch.cuda.stream(stream):
        return t.clone()


def _rows():
    gen = torch.Generator().manual_seed(4)
    x, z, dy = (torch.randn(3000, 192, generator=gen).cuda().to(torch.bfloat16) for _ in range(3))
    w, b = (torch.randn(192, generator=gen).cuda() for _ in range(2))
    return x, z, dy, w, b


def _layer_norm_fwd():
    x, z, _, w, b = _rows()
    return lambda s: mm.layer_norm_fwd(x, w, b, z=z, stream=s)


def _layer_norm_bwd():
    x, z, dy, w, b = _rows()
    _, mean, rstd = mm.layer_norm_fwd(x, w, b, z=z)
    return lambda s: mm.layer_norm_bwd(x, w, b, mean, rstd, dy, z=z, stream=s)


def _scan_args():
    gen = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    return [r(2, 64, 200), r(2, 64, 200).abs() * 0.1, -r(64, 16).abs(), r(2, 16, 200), r(2, 16, 200)]


def _scan_fwd():
    a = _scan_args()
    return lambda s: mm.scan_fwd(*a, stream=s)


def _scan_fwd_train():
    a = _scan_args()
    return lambda s: mm.scan_fwd_train(*a, stream=s)


def _scan_fwd_split():
    a = _scan_args()
    return lambda s: mm.scan_fwd_split(*a, 64, 200, stream=s)


def _ssd(fn, **kw):
    gen = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    x, B, C = (r(1, 512, n, w).to(torch.bfloat16) for n, w in ((2, 64), (1, 128), (1, 128)))
    delta, A = r(1, 512, 2).abs() * 0.1, -r(2).abs()
    return lambda s: fn(x, delta, A, B, C, stream=s, **kw)


def _ssd_fwd():
    return _ssd(mm.ssd_fwd)


def _ssd_fwd_momentum():
    return _ssd(mm.ssd_fwd_momentum)


CALLS = {f.__name__[1:]: f for f in (_gdr_fwd, _gdr_fwd_train, _gdr_bwd, _gdr_step, _layer_norm_fwd, _layer_norm_bwd,
                                     _scan_fwd, _scan_fwd_train, _scan_fwd_split, _ssd_fwd, _ssd_fwd_momentum)}


def _values(out):
    return list(out.values()) if isinstance(out, dict) else list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("name", CALLS)
def test_freed_blocks_keep_their_data(name):
    call = CALLS[name]()
    side = torch.cuda.Stream()
    want = [t.clone() for t in _values(call(None))]
    torch.cuda.empty_cache()
    blocks = [torch.ones(n, device="cuda") for n in (1 << 10, 1 << 15, 1 << 19, 1 << 23)]
    kept = [torch.zeros_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                           # some 50 ms on the current stream
    for b, k in zip(blocks, kept):
        k.copy_(b)
    del blocks, b
    got = _values(call(side))
    torch.cuda.current_stream().wait_stream(side)
    same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert all(same) and len(got) == len(want)
    assert all(bool((k == 1).all()) for k in kept)
    mm.mm_device_status()
