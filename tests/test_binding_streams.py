"""verify_* and draft_confidence on another stream than the current one: their
workspace and results made there, their memory kept.  On the host with stand-ins for
streams, devices and the library; on a GPU while the current stream is busy."""
import warnings

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from tests.test_cache_host import sv  # noqa: F401
from tests.test_cache_host_edges import Streams


@pytest.fixture
def faked(sv, monkeypatch):  # noqa: F811
    import speculative_decoding_verification_ragged_gb300.binding as mod
    st = Streams()

    class Library:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096
            return lambda *a: st.log.append(("launch", a[-1], name)) or 0

    def made(f):
        def g(*a, **kw):
            st.log.append(("made", st.current.cuda_stream, f.__name__))
            return f(*a, **kw)
        return g

    monkeypatch.setattr(mod, "load_library", lambda path=None: Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: st.current)
    monkeypatch.setattr(torch.cuda, "stream", st.enter)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: st.log.append(("lent", s.cuda_stream, tuple(t.shape))))
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")
        z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda:0")
        f32 = torch.float32
        rows = (z(6, 100, d=f32), z(3), z(6))
        kw = dict(V=100, B=2, k_max=2)
        per = lambda d: z(2, d=d)
        sample = (*rows, per(f32), per(torch.int32), per(f32), per(f32), per(torch.int64))
        calls = {
            "verify_greedy": lambda **s: sv.verify_greedy(*rows, **kw, **s),
            "verify_greedy_noalloc": lambda **s: sv.verify_greedy_noalloc(*rows, **kw, **s),
            "verify_relaxed_topk": lambda **s: sv.verify_relaxed_topk(*rows, per(torch.int32), **kw, **s),
            "verify_greedy_active": lambda **s: sv.verify_greedy_active(*rows, z(100), **kw, **s),
            "verify_greedy_margin": lambda **s: sv.verify_greedy_margin(*rows, per(f32), **kw, **s),
            "verify_sample": lambda **s: sv.verify_sample(*sample, **kw, **s),
            "draft_confidence": lambda **s: sv.draft_confidence(z(4, 100, d=f32), V=100, B=2, k=2, **s)}
        st.watch = lambda: (monkeypatch.setattr(torch, "zeros", made(torch.zeros)), monkeypatch.setattr(torch, "empty", made(torch.empty)))
        yield calls, st


NAMES = ["verify_greedy", "verify_greedy_noalloc", "verify_relaxed_topk", "verify_greedy_active", "verify_greedy_margin",
         "verify_sample", "draft_confidence"]


@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_another_stream_makes_its_tensors_there(faked, name):
    calls, st = faked
    call = calls[name]
    res = call()
    assert all(x[0] != "lent" and x[1] == 1 for x in st.log)         # none asked for: as it was
    st.watch()
    del st.log[:]
    got = call(stream=st.side)
    launch = next(i for i, x in enumerate(st.log) if x[0] == "launch")
    assert st.log[launch][1:] == (2, "spec_" + name)
    # (what the test itself makes for the call is made on stream 1, as its inputs are)
    mine = [x for x in st.log[:launch] if x[0] == "made" and x[1] == 2]
    assert len(mine) >= (1 if name.endswith("noalloc") else 2)
    lent = {x[1:] for x in st.log if x[0] == "lent"}
    assert {(1, tuple(t.shape)) for t in got.values()} <= lent       # results: kept for the caller's stream
    assert ((2, (6, 100)) in lent) or ((2, (4, 100)) in lent)        # inputs: for the call's
    assert res.keys() == got.keys()


def test_a_stream_that_is_the_current_one_needs_nothing(faked):
    calls, st = faked
    for name in NAMES:
        del st.log[:]
        calls[name](stream=st.here)
        assert all(x[0] != "lent" for x in st.log)


@pytest.mark.gpu
def test_verification_on_another_stream_while_the_current_one_is_busy():
    from tests._gpu import need_gpu
    sv = need_gpu()
    rng = np.random.default_rng(50)
    B, k, V = 16, 4, 40000
    logits = torch.from_numpy(rng.standard_normal((B * (k + 1), V)).astype(np.float32)).cuda()
    cu = torch.arange(0, B * (k + 1) + 1, k + 1, dtype=torch.int32, device="cuda")
    draft = logits.argmax(1).int()
    draft[::7] = 0
    f = lambda x, d: torch.tensor(x, dtype=d, device="cuda")
    par = (f([0.7] * B, torch.float32), f([40] * B, torch.int32), f([0.9] * B, torch.float32), f([0.0] * B, torch.float32),
           f(list(range(B)), torch.int64))
    calls = [lambda **s: sv.verify_greedy(logits, cu, draft, V=V, B=B, k_max=k, **s),
             lambda **s: sv.verify_sample(logits, cu, draft, *par, V=V, B=B, k_max=k, **s)]
    n = max(sv.workspace_bytes(B * (k + 1), B, V, 0, True), 1)
    side = torch.cuda.Stream()
    for call in calls:
        want = {x: y.clone() for x, y in call().items()}
        for _ in range(3):
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
            torch.cuda.synchronize()
            del junk
            torch.cuda._sleep(20_000_000)
            got = call(stream=side)
            late = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
            side.synchronize()
            assert all(torch.equal(want[x].cpu(), got[x].cpu()) for x in want)
            del late
