"""CPU checks of the gated delta rule's and layer norm's C entry points and
binding: sizes, refusals and their statuses.  Pointers are fake, aligned
integers; every call fails a host-side check or takes the fault-injection path
that launches nothing.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

import selective_state_space_momentum_b200 as mm
from selective_state_space_momentum_b200 import build as mmbuild

torch = pytest.importorskip("torch")
HERE = os.path.dirname(os.path.abspath(__file__))
NULL, DIMS, SCALAR, DTYPE, ALIGN, UNSUPPORTED, CUDA, ALIAS = 1, 2, 3, 4, 5, 6, 7, 9
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    mmbuild.build()
    return mm.load_library()


def _p(k, off=0):
    return (k + 1) * (1 << 36) + off


def G(batch=1, L=64, H=2, P=64, N=64, Gr=1, io=mm.MM_BF16):
    return mm.GDRDims(batch, L, H, P, N, Gr, io)


def _fwd(lib, dims=None, scale=0.1, ws=BIG, **over):
    a = dict(q=_p(0), k=_p(1), v=_p(2), g=_p(3), beta=_p(4), h0=None, o=_p(5), hT=None, ckpt=None, w=_p(6))
    a.update(over)
    return lib.mm_gdr_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], a["h0"], scale, a["o"], a["hT"], a["ckpt"], a["w"], ws,
                          ctypes.byref(dims) if dims is not None else None, None)


def _bwd(lib, dims, scale=0.1, ws=BIG, **over):
    names = ("q", "k", "v", "g", "beta", "ckpt", "dout", "dhT", "dq", "dk", "dv", "dg", "dbeta", "dh0", "w")
    a = {n: _p(i) for i, n in enumerate(names)}
    a.update(over)
    return lib.mm_gdr_bwd(a["q"], a["k"], a["v"], a["g"], a["beta"], scale, *(a[n] for n in names[5:]), ws, ctypes.byref(dims), None)


def _step(lib, dims, scale=0.1, **over):
    names = ("q", "k", "v", "g", "beta", "h", "o")
    a = {n: _p(i) for i, n in enumerate(names)}
    a.update(over)
    return lib.mm_gdr_step(*(a[n] for n in names[:6]), scale, a["o"], ctypes.byref(dims), None)


def test_fwd_refusals(lib):
    assert _fwd(lib) == NULL                                             # dims
    for name in ("q", "k", "v", "g", "beta", "o", "w"):
        assert _fwd(lib, G(), **{name: None}) == NULL, name
        assert _fwd(lib, G(), **{name: _p(20, 8)}) == ALIGN, name
    for bad in (dict(batch=0), dict(L=0), dict(H=0), dict(P=0), dict(N=0), dict(Gr=0), dict(H=3, Gr=2), dict(batch=-1)):
        assert _fwd(lib, G(**bad)) == DIMS, bad
    for bad in (dict(P=32), dict(P=65), dict(N=16), dict(N=256), dict(L=(1 << 30) + 1), dict(batch=1 << 31),
                dict(batch=1 << 20, H=1 << 12)):
        assert _fwd(lib, G(**bad)) == UNSUPPORTED, bad
    assert _fwd(lib, G(io=mm.MM_F32)) == DTYPE and _fwd(lib, G(io=7)) == DTYPE
    assert _fwd(lib, G(), scale=float("nan")) == SCALAR and _fwd(lib, G(), scale=float("inf")) == SCALAR
    assert _fwd(lib, G(), ws=10) == DIMS
    for name in ("q", "k", "v", "g", "beta"):
        assert _fwd(lib, G(), o=_p({"q": 0, "k": 1, "v": 2, "g": 3, "beta": 4}[name])) == ALIAS, name
    assert _fwd(lib, G(), hT=_p(5)) == ALIAS and _fwd(lib, G(), ckpt=_p(6)) == ALIAS and _fwd(lib, G(), w=_p(1)) == ALIAS
    assert _fwd(lib, G(), h0=_p(9), hT=_p(9, 256)) == ALIAS              # overlapping, not the same
    assert _fwd(lib, G(batch=1 << 30, L=1 << 30, H=1 << 30)) in (DIMS, UNSUPPORTED)


def test_bwd_refusals(lib):
    for name in ("q", "k", "v", "g", "beta", "ckpt", "dout", "dq", "dk", "dv", "dg", "dbeta", "w"):
        assert _bwd(lib, G(), **{name: None}) == NULL, name
        assert _bwd(lib, G(), **{name: _p(40, 4)}) == ALIGN, name
    for out in ("dq", "dk", "dv", "dg", "dbeta", "dh0", "w"):
        assert _bwd(lib, G(), **{out: _p(0)}) == ALIAS, out              # over q
        assert _bwd(lib, G(), **{out: _p(5)}) == ALIAS, out              # over ckpt
    assert _bwd(lib, G(), dk=_p(8)) == ALIAS                              # over dq
    assert _bwd(lib, G(), ws=1000) == DIMS and _bwd(lib, G(N=32)) == UNSUPPORTED and _bwd(lib, G(io=mm.MM_F32)) == DTYPE


def test_step_refusals(lib):
    one = dict(L=1)
    assert _step(lib, G(L=2)) == DIMS
    for name in ("q", "k", "v", "g", "beta", "h", "o"):
        assert _step(lib, G(**one), **{name: None}) == NULL, name
    for N in (2, 6, 260, 1):
        assert _step(lib, G(N=N, **one)) == UNSUPPORTED, N
    assert _step(lib, G(io=3, **one)) == DTYPE and _step(lib, G(**one), scale=float("inf")) == SCALAR
    assert _step(lib, G(**one), o=_p(5)) == ALIAS and _step(lib, G(**one), h=_p(2)) == ALIAS
    assert _step(lib, G(batch=1 << 30, H=1 << 10, P=1 << 10, N=4, **one)) in (UNSUPPORTED, DIMS)


def _norm(lib, fwd, rows=4, cols=32, io=0, eps=1e-5, rms=0, ws=BIG, **over):
    names = ("x", "weight", "bias", "z", "y", "mean", "rstd") if fwd else \
        ("x", "weight", "bias", "z", "mean", "rstd", "dy", "dx", "dweight", "dbias", "dz", "w")
    a = {n: _p(i) for i, n in enumerate(names)}
    a.update(over)
    dims = ctypes.byref(mm.NormDims(rows, cols, io))
    if fwd:
        return lib.mm_layer_norm_fwd(a["x"], a["weight"], a["bias"], a["z"], eps, rms, a["y"], a["mean"], a["rstd"], dims, None)
    return lib.mm_layer_norm_bwd(a["x"], a["weight"], a["bias"], a["z"], rms, *(a[n] for n in names[4:]), ws, dims, None)


def test_norm_refusals(lib):
    for name in ("x", "y"):
        assert _norm(lib, True, **{name: None}) == NULL
    for name in ("x", "rstd", "dy", "dx", "mean", "w", "z"):             # z: dz without it
        assert _norm(lib, False, **{name: None}) == NULL, name
    for fwd in (True, False):
        assert _norm(lib, fwd, rows=0) == DIMS and _norm(lib, fwd, cols=-1) == DIMS
        assert _norm(lib, fwd, cols=16385) == UNSUPPORTED and _norm(lib, fwd, rows=1 << 31) == UNSUPPORTED
        assert _norm(lib, fwd, io=9) == DTYPE
        assert _norm(lib, fwd, weight=_p(30, 4)) == ALIGN
    assert _norm(lib, True, eps=float("nan")) == SCALAR and _norm(lib, True, eps=-1.0) == SCALAR
    assert _norm(lib, True, y=_p(0)) == ALIAS and _norm(lib, True, rstd=_p(5)) == ALIAS
    assert _norm(lib, False, dx=_p(6)) == ALIAS and _norm(lib, False, dz=_p(7)) == ALIAS and _norm(lib, False, w=_p(0)) == ALIAS
    assert _norm(lib, False, ws=16) == DIMS


def test_calls_that_pass_their_checks_reach_the_launch(lib, monkeypatch):
    monkeypatch.setenv("MMSCAN_FAULT_INJECT", "launch")
    assert _fwd(lib, G()) == CUDA and _fwd(lib, G(), h0=_p(9), hT=_p(9), ckpt=_p(12)) == CUDA
    assert _bwd(lib, G()) == CUDA and _bwd(lib, G(), dhT=None, dh0=None) == CUDA
    assert _step(lib, G(L=1, N=12, P=7, io=0)) == CUDA
    assert _norm(lib, True) == CUDA and _norm(lib, True, weight=None, bias=None, z=None, mean=None, rstd=None) == CUDA
    assert _norm(lib, False) == CUDA and _norm(lib, False, rms=1, mean=None, dz=None) == CUDA
    assert _norm(lib, False, dweight=None, dbias=None, w=None) == CUDA   # no workspace needed then
    assert "injected" in mm.mm_last_error()


def test_sizes(lib):
    # two heads of 64 rows and 64 states, 130 steps: 3 chunks, 6 records
    rec, tlo = 2 * 64 * 64 * 2 + 3 * 64 * 4, 64 * 64 * 2
    assert mm.mm_gdr_fwd_workspace_size(1, 130, 2, 64, 64, 1) == 6 * (rec + tlo)
    assert mm.mm_gdr_fwd_workspace_size(1, 130, 2, 64, 64, 1, True) == 6 * tlo
    assert mm.mm_gdr_ckpt_size(1, 130, 2, 64, 64, 1) == 6 * (rec + 64 * 64 * 2 + 64 * 64 * 2)
    assert mm.mm_gdr_bwd_workspace_size(1, 130, 2, 64, 64, 1) == 6 * (64 * 64 * 2 + 64 * 64 * 2)
    assert mm.mm_layer_norm_bwd_workspace_size(5, 2048) == 5 * 2 * 2048 * 4
    with pytest.raises(mm.MMError):
        mm.mm_gdr_ckpt_size(1, 130, 3, 64, 64, 2)
    assert lib.mm_gdr_ckpt_size(ctypes.byref(G()), None) == NULL


def _tensors(B=2, L=70, H=4, Gr=2, P=64, N=128, dt=torch.bfloat16):
    q, v, g = torch.zeros(B, L, Gr, N, dtype=dt), torch.zeros(B, L, H, P, dtype=dt), torch.zeros(B, L, H, dtype=dt)
    return dict(q=q, k=q.clone(), v=v, g=g, beta=g.clone())


def test_binding_refuses_before_any_call():
    t = _tensors()
    with pytest.raises(ValueError, match="CUDA"):
        mm.gdr_fwd(**t)
    with pytest.raises(TypeError, match="bf16"):
        mm.gdr_fwd(**_tensors(dt=torch.float32))
    with pytest.raises(ValueError, match="k has shape"):
        mm.gdr_fwd(**{**t, "k": t["k"][:, :60].contiguous()})
    with pytest.raises(TypeError, match="beta"):
        mm.gdr_fwd(**{**t, "beta": t["beta"].float()})
    with pytest.raises(ValueError, match="contiguous"):
        mm.gdr_fwd(**{**t, "v": torch.zeros(2, 4, 70, 64, dtype=torch.bfloat16).transpose(1, 2)})
    with pytest.raises(ValueError, match="h0"):
        mm.gdr_fwd(**t, h0=torch.zeros(2, 4, 128, 64))
    with pytest.raises(mm.MMError, match="ngroups"):
        mm.gdr_fwd(**_tensors(H=3))
    with pytest.raises(TypeError, match="q"):
        mm.gdr_fwd(None, t["k"], t["v"], t["g"], t["beta"])
    with pytest.raises(ValueError, match="dimensions"):
        mm.gdr_fwd(t["q"][0], t["k"], t["v"], t["g"], t["beta"])
    with pytest.raises(TypeError, match="ckpt"):
        mm.gdr_bwd(**t, ckpt=torch.zeros(8), dout=t["v"]) if torch.cuda.is_available() else mm._require_bytes("ckpt", torch.zeros(8), 8, -1)
    s = {n: x[:, 0].contiguous() for n, x in t.items()}
    with pytest.raises(ValueError, match="h has shape"):
        mm.gdr_step(**s, h=torch.zeros(2, 4, 64, 64))
    with pytest.raises(TypeError, match="h has dtype"):
        mm.gdr_step(**s, h=torch.zeros(2, 4, 64, 128, dtype=torch.bfloat16))


def test_norm_binding_refuses_before_any_call():
    x = torch.zeros(3, 40)
    with pytest.raises(ValueError, match="CUDA"):
        mm.layer_norm_fwd(x)
    with pytest.raises(TypeError):
        mm.layer_norm_fwd(x.half())
    with pytest.raises(ValueError, match="weight"):
        mm.layer_norm_fwd(x, torch.zeros(39))
    with pytest.raises(TypeError, match="weight"):
        mm.layer_norm_fwd(x, torch.zeros(40, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="z has shape"):
        mm.layer_norm_fwd(x, z=torch.zeros(3, 41))
    with pytest.raises(ValueError, match="contiguous"):
        mm.layer_norm_fwd(torch.zeros(40, 3).t())
    with pytest.raises(TypeError, match="mean"):
        mm.layer_norm_bwd(x, None, None, None, torch.zeros(3), x)
    with pytest.raises(TypeError, match="Tensor"):
        mm.layer_norm_fwd([1.0])


def test_checks_under_sanitizers(tmp_path):
    """mm_layer_api.cpp with AddressSanitizer and UndefinedBehaviorSanitizer
    against a stand-in runtime and counting launchers, at sizes at and past
    every limit."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    root = os.path.dirname(HERE)
    csrc = os.path.join(root, "selective_state_space_momentum_b200", "csrc")
    exe = tmp_path / "layer_checks"
    r = subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                        "-I", os.path.join(HERE, "c", "stub_cuda"), "-I", os.path.join(root, "include"), "-I", csrc,
                        os.path.join(HERE, "c", "layer_checks_sanitized.cpp"), os.path.join(csrc, "mm_layer_api.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    if r.returncode != 0 and "sanitize" in r.stderr and "cannot find" in r.stderr:
        pytest.skip("gcc sanitizer runtimes not available")
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and "layer checks ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
