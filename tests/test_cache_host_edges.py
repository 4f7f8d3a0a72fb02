"""The 4-bit cache's binding and C entries, on the host alone: where tensors are
made and how long they are kept when a call runs on another stream, and the
refusals at the edges of the contract.  Devices, streams and the library are
stood in for where a call would otherwise launch."""
import ctypes as C
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from tests.test_cache_host import FAKE, _attn, _cache, _evict, _rows, sv  # noqa: F401


class Streams:
    """Streams by name, the current one, and what was done on which."""

    class One:
        def __init__(self, log, n):
            self.log, self.cuda_stream = log, n

        def wait_event(self, e):
            self.log.append(("wait", self.cuda_stream, e.on))

    def __init__(self):
        self.log = []
        self.here, self.side, self.third = (self.One(self.log, n) for n in (1, 2, 3))
        self.current = self.here

    def enter(self, s):
        streams = self

        class Under:
            def __enter__(self):
                self.before, streams.current = streams.current, s or streams.current

            def __exit__(self, *a):
                streams.current = self.before
        return Under()


@pytest.fixture
def faked(sv, monkeypatch):  # noqa: F811
    """The binding over tensors of a device that is not there: (sv, streams)."""
    import speculative_decoding_verification_ragged_gb300.cache as mod
    st = Streams()

    class Library:
        def __getattr__(self, name):
            if name == "spec_cache_workspace_bytes":
                return lambda *a: 4096
            return lambda *a: st.log.append(("launch", a[-1], name)) or 0

    class Event:
        def record(self):
            self.on = st.current.cuda_stream

    def made(f):
        def g(*a, **kw):
            st.log.append(("made", st.current.cuda_stream, f.__name__))
            return f(*a, **kw)
        return g

    monkeypatch.setattr(mod, "load_library", lambda path=None: Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: st.current)
    monkeypatch.setattr(torch.cuda, "stream", st.enter)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: st.log.append(("lent", s.cuda_stream, tuple(t.shape))))
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")
        z = lambda *s, d=torch.int32, dev="cuda:0": torch.zeros(*s, dtype=d, device=dev)
        st.cache = lambda **kw: sv.PagedCache(z(3, 1, 1, 36 * 64, d=torch.uint8), **kw)
        st.z = z
        st.args = (z(4, 2, 64, d=torch.float32), z(2), z(1), z(1, 3))
        st.made = lambda: (monkeypatch.setattr(torch, "zeros", made(torch.zeros)), monkeypatch.setattr(torch, "empty", made(torch.empty)))
        yield sv, st


def test_a_call_on_another_stream_makes_its_tensors_there(faked):
    """Workspace zeros and results on the stream of the launch; the inputs kept for
    it, the results for the caller's."""
    sv, st = faked
    cache, score = st.cache(), st.z(3, 32, d=torch.float32)
    st.made()
    sv.cache_attend(cache, *st.args, B=1, k_max=3, stream=st.side)
    assert {x[1] for x in st.log if x[0] == "made"} == {2} and sum(x[0] == "made" for x in st.log) >= 3
    lent = [x for x in st.log if x[0] == "lent"]
    assert {(2, (3, 1, 1, 36 * 64)), (2, (4, 2, 64)), (2, (1, 3)), (2, (4096,)), (1, (4, 2, 64)), (1, (4, 2))} <= {x[1:] for x in lent}
    launch = st.log.index(("launch", 2, "spec_cache_attend"))
    assert all(st.log.index(x) < launch for x in lent if x[1] == 2)
    for call in (lambda: sv.cache_read(cache, st.args[1], st.args[2], st.args[3], B=1, max_rows=4, stream=st.side),
                 lambda: sv.cache_evict(cache, score, st.args[2], st.args[3], st.args[3], B=1, budget=4, stream=st.side)):
        del st.log[:]
        call()
        assert {x[1] for x in st.log if x[0] == "made"} == {2}
        assert {x[1] for x in st.log if x[0] == "lent"} == {1, 2}


def test_a_handle_orders_its_workspace_before_another_stream(faked):
    sv, st = faked
    call = sv.cache_attend(st.cache(), *st.args, B=1, k_max=3, prepared=True)
    del st.log[:]
    call()
    assert st.log == [("launch", 1, "spec_cache_attend")]           # its own stream: nothing to do
    for stream in (st.side, st.third):
        del st.log[:]
        call(stream)
        n = stream.cuda_stream
        assert st.log[0] == ("wait", n, 1) and st.log[-1] == ("launch", n, "spec_cache_attend")
        assert sum(x[0] == "lent" for x in st.log) == len(st.log) - 2 >= 7
        del st.log[:]
        with st.enter(stream):
            call()
        assert st.log == [("launch", n, "spec_cache_attend")]       # from then on neither
    # prepared for another stream than the current one: the current one waits too
    call = sv.cache_attend(st.cache(), *st.args, B=1, k_max=3, prepared=True, stream=st.side)
    del st.log[:]
    call()
    assert st.log[0] == ("wait", 1, 2)


def test_a_handle_over_the_callers_workspace_waits_for_nothing(faked):
    sv, st = faked
    call = sv.cache_attend(st.cache(), *st.args, B=1, k_max=3, workspace=st.z(4096, d=torch.uint8), prepared=True)
    del st.log[:]
    call(st.side)
    assert all(x[0] != "wait" for x in st.log)


def test_a_captured_call_is_left_to_its_graph(faked, monkeypatch):
    sv, st = faked
    call = sv.cache_attend(st.cache(), *st.args, B=1, k_max=3, prepared=True)
    del st.log[:]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: st.current is st.side)
    call(st.side)
    assert st.log == [("launch", 2, "spec_cache_attend")]


# ---------------------------------------------------------------- refusals ---

def test_tensors_of_another_device_are_refused(faked):
    """... whichever argument they are: a pointer of another GPU must not reach a kernel."""
    sv, st = faked
    z, (q, cu, ln, tab) = st.z, st.args
    f32, there = torch.float32, dict(dev="cuda:1")
    kv, score, pos = z(4, 1, 64, d=f32), z(3, 32, d=f32), z(3, 32)
    lse, ws = z(4, 2, d=f32), z(4096, d=torch.uint8)
    call = dict(B=1)
    attend = lambda c=None, q=q, cu=cu, ln=ln, tab=tab, **kw: sv.cache_attend(c or st.cache(), q, cu, ln, tab, k_max=3, **call, **kw)
    weights = lambda c=None, q=q, lse=lse, tab=tab, score=score, **kw: sv.cache_weights(
        c or st.cache(), q, lse, cu, ln, tab, score, k_max=3, **call, **kw)
    append = lambda c=None, k=kv, v=kv, tab=tab, **kw: sv.cache_append(c or st.cache(), k, v, cu, ln, tab, max_rows=4, **call, **kw)
    read = lambda c=None, cu=cu, tab=tab, **kw: sv.cache_read(c or st.cache(), cu, ln, tab, max_rows=4, **call, **kw)
    evict = lambda c=None, score=score, tab=tab, dst=tab, **kw: sv.cache_evict(c or st.cache(), score, ln, tab, dst, budget=4, **call, **kw)
    for f in (attend, weights, append, read, evict):
        f()                                                          # all on one device: accepted
        for kw in (dict(k_scale=z(1, d=f32, **there)), dict(v_scale=z(1, d=f32, **there))):
            with pytest.raises(sv.SpecError, match="different devices"):
                f(st.cache(**kw))
        with pytest.raises(sv.SpecError, match="different devices"):
            f(tab=z(1, 3, **there))
        with pytest.raises(sv.SpecError, match="different devices"):
            f(status=z(1, **there))
    for f, kw in [(attend, dict(workspace=z(4096, d=torch.uint8, **there))), (attend, dict(q=z(4, 2, 64, d=f32, **there))),
                  (attend, dict(slopes=z(2, d=f32, **there))), (attend, dict(slot_pos=z(3, 32, **there))),
                  (weights, dict(lse=z(4, 2, d=f32, **there))), (weights, dict(score=z(3, 32, d=f32, **there))),
                  (append, dict(v=z(4, 1, 64, d=f32, **there))), (append, dict(score=z(3, 32, d=f32, **there))),
                  (append, dict(pos0=z(1, **there))), (read, dict(cu=z(2, **there))),
                  (evict, dict(score=z(3, 32, d=f32, **there))), (evict, dict(dst=z(1, 3, **there))),
                  (evict, dict(slot_pos=z(3, 32, **there)))]:
        with pytest.raises(sv.SpecError, match="different devices"):
            f(**kw)
    attend(workspace=ws)

ODD, HALF = C.c_void_p(0x10001), C.c_void_p(0x10002)


def test_arrays_off_their_words_are_refused(sv):  # noqa: F811
    """Device arrays of 32-bit values anywhere else, and a workspace off 16 bytes
    (its parts are read by vectors): refused before a launch would touch them."""
    L, n = sv.load_library(), 1 << 30
    rows = lambda f, c, r: f(C.byref(c), C.byref(r), None)
    attend = lambda c, a, lse=FAKE, ws=FAKE: L.spec_cache_attend(C.byref(c), C.byref(a), FAKE, lse, ws, n, None)
    weights = lambda c, a, lse=FAKE, score=FAKE: L.spec_cache_weights(C.byref(c), C.byref(a), lse, score, None)
    evict = lambda c, e: L.spec_cache_evict(C.byref(c), C.byref(e), None)
    for off in (ODD, HALF):
        for name in ("k_scale", "v_scale", "page_table"):
            c = _cache(**{name: off})
            assert rows(L.spec_cache_append, c, _rows()) == 1 and rows(L.spec_cache_read, c, _rows()) == 1, name
            assert attend(c, _attn()) == 1 and weights(c, _attn()) == 1 and evict(c, _evict()) == 1, name
        for name in ("cu_rows", "start", "score", "slot_pos", "pos0", "status"):
            assert rows(L.spec_cache_append, _cache(), _rows(**{name: off})) == 1, name
        for name in ("cu_rows", "len", "slopes", "slot_pos", "status"):
            assert attend(_cache(), _attn(**{name: off})) == 1 and weights(_cache(), _attn(**{name: off})) == 1, name
        assert attend(_cache(), _attn(), lse=off) == 1
        assert weights(_cache(), _attn(), lse=off) == 1 and weights(_cache(), _attn(), score=off) == 1
        for name in ("score", "slot_pos", "len", "dst_table", "kept", "new_len", "status"):
            assert evict(_cache(), _evict(**{name: off})) == 1, name
    for at in (0x10001, 0x10004, 0x10008):
        assert attend(_cache(), _attn(), ws=C.c_void_p(at)) == 1


def test_workspace_sizes_at_the_limits(sv):  # noqa: F811
    """Every size that a call would accept has one, near that of the same grid of
    blocks; sizes that no call accepts have none, with no sum wrapped on the way."""
    L = sv.load_library()
    full = L.spec_cache_workspace_bytes(4, 31, 64, 4, 128, 1 << 20)
    assert 0 < full < 1 << 28
    for ok in [(4, 31, 64, 4, 128, 1 << 30), (65535, 31, 64, 4, 128, 1 << 10), (4, 31, 65535, 65535, 128, 1 << 20)]:
        assert 0 < L.spec_cache_workspace_bytes(*ok) <= full, ok
    # one kv head for all: more columns, the widest tile
    assert 0 < L.spec_cache_workspace_bytes(65535, 31, 65535, 1, 64, 1 << 20) < 1 << 28
    for bad in [(4, 31, 64, 4, 128, 2 ** 31 - 1), (4, 31, 64, 4, 128, (1 << 30) + 1), (65536, 31, 64, 4, 128, 1024),
                (4, 31, 2 ** 31 - 1, 1, 128, 1024), (4, 31, 65536, 4, 128, 1024), (4, 31, 2 ** 31 - 1, 2 ** 31 - 1, 128, 1024)]:
        assert L.spec_cache_workspace_bytes(*bad) == 0, bad
