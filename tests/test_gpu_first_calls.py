"""The first calls of a process from several threads at once: what each kernel looks up once a device (how many clusters run
together, which decides in how many parts a prompt is split) is there for all of them, and so all get the same bits."""
import subprocess
import sys

import pytest

from tests._gpu import need_gpu
from tests.conftest import ROOT

pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

CODE = """
import threading
import torch
import speculative_decoding_verification_ragged_gb300 as sv

sv.build()
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
cu, cuk = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 5], [0, 9000]))
for D in (64, 128, 256):
    q, k, v = (torch.randn(n, h, D, generator=gen, device="cuda").to(torch.bfloat16) for n, h in ((5, 4), (9000, 2), (9000, 2)))
    for cap in (0.0, 30.0):
        call = lambda: sv.prompt_attend(q, k, v, cu, B=1, cu_keys=cuk, cap=cap)
        start, got = threading.Barrier(12), [None] * 12

        def first(i):
            start.wait()
            got[i] = call()

        torch.cuda.synchronize()
        threads = [threading.Thread(target=first, args=(i,)) for i in range(12)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        later = call()
        for x in got:
            assert torch.equal(x["out"], later["out"]) and torch.equal(x["lse"], later["lse"]), (D, cap)
print("same")
"""


def test_threads_that_call_first_split_as_later_calls_do():
    need_gpu()
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


FIRST = """
import hashlib
import sys
import torch
import speculative_decoding_verification_ragged_gb300 as sv

sv.build()
gen = torch.Generator(device="cuda")
gen.manual_seed(2)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
calls = []
for D in (64, 128, 256):
    q, k, v = rand(7, 4, D), rand(9000, 2, D), rand(9000, 2, D)
    for cap in (0.0, 30.0):
        for a, ws in ((lambda x: x, torch.bfloat16), (lambda x: x.float(), torch.float32)):
            for keys in (9000, 300):
                calls.append(sv.prompt_attend(a(q), a(k), a(v), i32([0, 7]), B=1, cu_keys=i32([0, keys]), cap=cap, prepared=True,
                                              workspace=sv.new_prompt_workspace(4, 2, D, ws)))
cache, table = sv.new_cache(6, 2, 64, 64), i32([[5, 1, 0, 3]])
cache.pages.zero_()
ws = sv.new_cache_workspace(cache, table, B=1, k_max=3, Hq=4)
q, parent = rand(4, 4, 64), i32([-1, 0, 0, 2])
for opt in (dict(), dict(window=50)):
    calls.append(sv.cache_attend_tree(cache, q, i32([0, 4]), i32([200]), table, parent, B=1, k_max=3, workspace=ws, prepared=True, **opt))
logits = rand(4, 5000)
calls.append(sv.adjust_logits(logits, i32([0, 4]), V=5000, B=1, k_max=3, history=i32([list(range(90))]), n_tokens=i32([90]),
                              repetition=torch.tensor([1.3], device="cuda"), prepared=True))
calls.append(sv.tree_accept(i32([5, 6, 7, 8]), i32([0, 4, 5, 7]), parent, i32([0, 4]), B=1, k_max=3, prepared=True))
torch.cuda.synchronize()
if sys.argv[1] == "captured":
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = [c() for c in calls]
    g.replay()
else:
    res = [c() for c in calls]
torch.cuda.synchronize()
h = hashlib.sha256()
for r in res:
    for x in r.values():
        h.update(x.contiguous().view(torch.uint8).cpu().numpy().tobytes())
print(h.hexdigest())
"""


def test_first_calls_can_be_captured():
    """Nothing of a first call's preparation is in a capture's way, and it finds the same things there."""
    need_gpu()
    got = []
    for how in ("eager", "captured"):
        r = subprocess.run([sys.executable, "-c", FIRST, how], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(r.stdout.split()[-1])
    assert got[0] == got[1]
