"""On which stream the allocating wrappers take their memory (no GPU).

A block that was freed on a stream goes back to that stream's pool at once: the
work queued there before it may still be using it.  So what a wrapper's kernels
touch on ``stream`` has to come from the pool of ``stream``, not from that of
the caller's current stream, which ``stream`` is not ordered behind; and what
the wrapper returns has to be recorded for the current stream, on which the
caller goes on with it.  Streams, allocations and launches are stood in for
here; the tensors are host tensors.
"""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import selective_state_space_momentum_b200 as mm  # noqa: E402

HERE = torch.device("cpu")


class _Stream:
    def __init__(self, handle, device=HERE):
        self.cuda_stream, self.device = handle, device

    def wait_stream(self, other):
        pass


class _Lib:
    """The library with its launches counted and not made."""

    def __init__(self, real, log):
        self._real, self._log = real, log

    def __getattr__(self, name):
        if name.endswith("_size") or name == "mm_last_error":
            return getattr(self._real, name)

        def launch(*args):
            handle = args[-1]
            self._log.append((name, getattr(handle, "value", handle) or 0))
            return 0
        return launch


@pytest.fixture
def stage(monkeypatch):
    """current: the caller's stream; made: storage -> stream it was allocated on; recorded: (storage, handle)."""
    class Stage:
        pass
    st = Stage()
    st.current, st.default = _Stream(11), _Stream(0)
    st.made, st.recorded, st.launched, st.external, st.alive = {}, set(), [], [], []

    @contextlib.contextmanager
    def on(stream):
        before, st.current = st.current, stream
        yield
        st.current = before

    def external(handle, device=None):
        st.external.append((handle, device))
        return _Stream(handle, HERE if device is None else torch.device(device))

    def recording(fn):
        def make(*args, **kwargs):
            kwargs.pop("device", None)
            t = fn(*args, **kwargs)
            st.made[t.data_ptr()] = st.current.cuda_stream
            st.alive.append(t)
            return t
        return make
    real = mm.load_library()
    lib = _Lib(real, st.launched)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: st.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: st.default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch, "empty", recording(torch.empty))
    monkeypatch.setattr(torch, "empty_like", recording(torch.empty_like))
    monkeypatch.setattr(torch.Tensor, "new_empty", recording(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: st.recorded.add((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(mm, "_on_cuda", lambda device: None)
    monkeypatch.setattr(mm, "load_library", lambda path=None: lib)
    monkeypatch.setattr(mm, "_run", lambda index, stream, fn, *args: fn(*args, stream if isinstance(stream, int) else
                                                                        (stream or st.current).cuda_stream))
    return st


def _gdr(ndim=4):
    lead = (2, 70) if ndim == 4 else (2,)
    z = lambda *s: torch.zeros(*lead, *s, dtype=torch.bfloat16)
    return [z(2, 64), z(2, 64), z(4, 64), z(4), z(4)]


def _ckpt():
    return torch.zeros(mm.mm_gdr_ckpt_size(2, 70, 4, 64, 64, 2), dtype=torch.uint8)


X = torch.zeros(6, 40)
NEW = {
    "gdr_fwd": lambda s: mm.gdr_fwd(*_gdr(), stream=s),
    "gdr_fwd_train": lambda s: mm.gdr_fwd_train(*_gdr(), return_last_state=True, stream=s),
    "gdr_bwd": lambda s: mm.gdr_bwd(*_gdr(), _ckpt(), _gdr()[2], return_dh0=True, stream=s),
    "gdr_step": lambda s: mm.gdr_step(*_gdr(3), torch.zeros(2, 4, 64, 64), stream=s),
    "layer_norm_fwd": lambda s: mm.layer_norm_fwd(X, stream=s),
    "layer_norm_bwd": lambda s: mm.layer_norm_bwd(X, torch.zeros(40), torch.zeros(40), torch.zeros(6), torch.zeros(6), X, z=X, stream=s),
}


def _scan():
    x = torch.zeros(2, 8, 64)
    bc = torch.zeros(2, 16, 64)
    return [x, x, torch.zeros(8, 16), bc, bc]


def _ssd():
    x, bc = torch.zeros(1, 256, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 256, 1, 128, dtype=torch.bfloat16)
    return [x, torch.zeros(1, 256, 2), torch.zeros(2), bc, bc]


class _Peers:
    """One rank's record buffers, without the device."""
    rank, world = 0, 1

    def next(self):
        return torch.zeros(1, dtype=torch.int64), torch.zeros(mm.mm_scan_split_maps_size(2, 64, 8, 16, 2), dtype=torch.uint8)

    def barrier(self, stream=None):
        assert stream is None or stream.cuda_stream in (77, 0)


SCAN_CKPT = torch.zeros(2, 8, 4, 2, 16)
EARLIER = {
    "scan_fwd": lambda s: mm.scan_fwd(*_scan(), stream=s),
    "scan_fwd_gated": lambda s: mm.scan_fwd(*_scan(), stream=s, D=torch.zeros(8), z=_scan()[0]),
    "scan_fwd_train": lambda s: mm.scan_fwd_train(*_scan(), stream=s),
    "scan_bwd": lambda s: mm.scan_bwd(*_scan(), SCAN_CKPT, _scan()[0], stream=s),
    "scan_bwd_gated": lambda s: mm.scan_bwd(*_scan(), SCAN_CKPT, _scan()[0], stream=s, D=torch.zeros(8), z=_scan()[0]),
    "ssd_fwd": lambda s: mm.ssd_fwd(*_ssd(), stream=s),
    "ssd_fwd_momentum": lambda s: mm.ssd_fwd_momentum(*_ssd(), stream=s),
    "scan_fwd_split": lambda s: mm.scan_fwd_split(*_scan(), 32, 64, stream=s),
    "scan_fwd_split_peers": lambda s: mm.scan_fwd_split_peers(*_scan(), 32, 64, _Peers(), stream=s),
}


def _tensors(out):
    values = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else [out]
    return [t for t in values if t is not None]


def _check(st, call, stream, handle):
    out = _tensors(call(stream))
    assert st.made and set(st.made.values()) == {handle}, st.made
    assert st.launched and {h for _, h in st.launched} == {handle}
    assert out
    for t in out:
        recorded = (t.data_ptr(), st.current.cuda_stream) in st.recorded
        assert recorded == (handle != st.current.cuda_stream)


@pytest.mark.parametrize("name", NEW)
def test_memory_belongs_to_the_stream_that_uses_it(stage, name):
    _check(stage, NEW[name], _Stream(77), 77)


@pytest.mark.parametrize("name", NEW)
def test_current_stream_by_default_and_by_name(stage, name):
    _check(stage, NEW[name], None, 11)
    _check(stage, NEW[name], stage.current, 11)


@pytest.mark.parametrize("name", NEW)
def test_stream_handles(stage, name):
    """An integer handle: a stream of the operands' device; 0 is the default stream."""
    _check(stage, NEW[name], 77, 77)
    assert set(stage.external) == {(77, HERE)}
    stage.made.clear(), stage.launched.clear(), stage.external.clear()
    _check(stage, NEW[name], 0, 0)
    assert stage.external == []


@pytest.mark.parametrize("name", NEW)
def test_a_stream_of_another_device_is_refused(stage, name):
    with pytest.raises(ValueError, match="stream"):
        NEW[name](_Stream(77, torch.device("meta")))
    assert stage.launched == []


@pytest.mark.parametrize("name", EARLIER)
def test_earlier_wrappers(stage, name):
    _check(stage, EARLIER[name], _Stream(77), 77)
    stage.made.clear(), stage.launched.clear()
    _check(stage, EARLIER[name], None, 11)
    stage.made.clear(), stage.launched.clear()
    _check(stage, EARLIER[name], 0, 0)


def test_split_over_ranks_orders_the_collective(stage, monkeypatch):
    """The gathered records come from the current stream's pool and are read on the call's."""
    order = []
    monkeypatch.setattr(_Stream, "wait_stream", lambda self, other: order.append((self.cuda_stream, other.cuda_stream)))
    monkeypatch.setattr(torch.distributed, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.distributed, "get_rank", lambda group=None: 0)
    monkeypatch.setattr(torch.distributed, "get_world_size", lambda group=None: 2)
    gathered = []

    def gather(local, world, group):
        order.append("gather")
        gathered.append(torch.cat([local, local]))
        return gathered[0]
    monkeypatch.setattr(mm, "_all_gather_bytes", gather)
    mm.scan_fwd_split(*_scan(), 32, 128, stream=_Stream(77))
    assert order == [(11, 77), "gather", (77, 11)]
    assert (gathered[0].data_ptr(), 77) in stage.recorded and set(stage.made.values()) == {77}


def test_an_object_that_only_has_a_handle(stage):
    class Foreign:
        cuda_stream = 77
    _check(stage, NEW["gdr_step"], Foreign(), 77)
    _check(stage, EARLIER["scan_fwd"], Foreign(), 77)
