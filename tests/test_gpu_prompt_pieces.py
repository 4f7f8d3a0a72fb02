"""A prompt that comes in pieces over the 4-bit cache: each piece attends over what the cache holds, read back, and is appended
itself.  Tolerances: those of tests/test_gpu_prompt.py, whose definition gets the values read back."""
import numpy as np
import pytest

from tests._gpu import need_gpu
from tests.test_gpu_prompt import check, i32, offsets, rand

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    need_gpu()
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


@pytest.mark.parametrize("opt", [dict(), dict(window=90, prefix=4)])
def test_pieces_over_what_the_cache_holds(sv, opt):
    rng = np.random.default_rng(51)
    B, Hq, H, D, page = 3, 4, 2, 64, 64
    cache, table = sv.new_cache(B * 8, H, D, page), i32(rng.permutation(B * 8).reshape(B, 8))
    ws, length = sv.new_prompt_workspace(Hq, H, D), np.zeros(B, np.int64)
    for rows in ([150, 1, 40], [100, 200, 0], [3, 64, 260]):
        cu = i32(offsets(rows))
        q, k, v = (rand(rng, sum(rows), h, D) for h in (Hq, H, H))
        sv.cache_append(cache, k, v, cu, i32(length), table, B=B, max_rows=max(rows))
        length += rows
        cuk = offsets(length)
        kv = sv.cache_read(cache, i32(cuk), i32([0] * B), table, B=B, max_rows=int(length.max()), R_cap=int(cuk[-1]), dtype=torch.bfloat16)
        got = sv.prompt_attend(q, kv["k"], kv["v"], cu, B=B, cu_keys=i32(cuk), workspace=ws, **opt)
        check(sv, q, kv["k"], kv["v"], rows, list(length), got=got, **opt)
