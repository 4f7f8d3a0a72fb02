"""Scores under caps up to the largest fp32, which change nothing of scores as small as these: against the definitions
without a cap, where the next term of the tanh, (s / cap)^2 / 3, is far below 2^-64.

Tolerances: those of tests/test_gpu_prompt.py and tests/test_gpu_cache.py with the tanh's 2^-20, relative to the score itself
(|s| <= S) and not to the cap, and one rounding more of the score on either side of it (2u S): ds = (2 D u + 8u + 2^-20) S."""
import numpy as np
import pytest

from tests import _cache_ref, _step_ref
from tests._gpu import need_gpu
from tests.test_gpu_cache import dev, gpu_cache, queries, quick_pool
from tests.test_gpu_prompt import DT, HALF, i32, offsets, rand

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
CAPS = [2.0 ** 100, 2.0 ** 120, 1e37, 2.0 ** 127, 2.5e38, float(np.finfo(np.float32).max)]


@pytest.fixture(scope="module")
def sv():
    need_gpu()
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


def compare(got, R, out, lse, A, ds, keys, weights, half):
    rel = 2 * ds + 2.0 ** -20 + 2.0 ** -23 * (keys / 16 + 16)
    gl, go = got["lse"][:R].double().cpu().numpy(), got["out"][:R].double().cpu().numpy()
    assert (np.abs(gl - lse) <= rel + 4 * U * np.abs(lse)).all()
    assert (np.abs(go - out) <= 1.01 * (A * (rel + weights)[..., None] + half * np.abs(out)) + 1e-30).all()


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_prompts(sv, dtype, D, cap):
    rng = np.random.default_rng(3)
    rows, Hq, H = [150, 1, 40], 4, 2
    q, k, v = (rand(rng, sum(rows), h, D, dtype=dtype) for h in (Hq, H, H))
    out, lse, A, S = _step_ref.prompt(*(x.double().cpu().numpy() for x in (q, k, v)), offsets(rows))
    got = sv.prompt_attend(q, k, v, i32(offsets(rows)), B=len(rows), cap=cap)
    compare(got, sum(rows), out, lse, A, (2 * D * U + 8 * U + 2.0 ** -20) * S, 150, 2.0 ** -8 if dtype == "bf16" else 0.0, HALF[dtype])


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache(sv, dtype, cap):
    rng = np.random.default_rng(4)
    rows, lens, D = [3, 1, 6], [200, 1, 77], 64
    c = quick_pool(rng, B=3, H=2, D=D, page=64, lens=lens)
    q = queries(rng, sum(rows), 4, D, dtype)
    cu, cu_, len_, tab = offsets(rows), i32(offsets(rows)), i32(lens), dev(c.table)
    chain = np.concatenate([np.arange(n) - 1 for n in rows])
    opt = dict(B=3, k_max=5, cap=cap)
    weights, half = (2.0 ** -11, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -20, 2.0 ** -23)
    out, lse, A, S, w = _cache_ref.attention(c, q.float().cpu().numpy(), cu, lens)
    ds = (2 * D * U + 8 * U + 2.0 ** -20) * S
    got = sv.cache_attend(gpu_cache(sv, c), q, cu_, len_, tab, **opt)
    compare(got, sum(rows), out, lse, A, ds, 200, weights, half)
    tree = sv.cache_attend_tree(gpu_cache(sv, c), q, cu_, len_, tab, i32(chain), **opt)
    compare(tree, sum(rows), out, lse, A, ds, 200, weights, half)
    score = torch.zeros(c.n_pages, c.page, device="cuda")
    sv.cache_weights(gpu_cache(sv, c), q, torch.tensor(lse, dtype=torch.float32, device="cuda"), cu_, len_, tab, score, **opt)
    worst = float((2 * ds + 4 * U * np.abs(lse)).max()) + 2.0 ** -18
    for b, n in enumerate(lens):
        i = np.arange(n)
        have = score[dev(c.table[b, i // c.page]).long(), dev(i % c.page).long()].double().cpu().numpy()
        assert (np.abs(have - w[b]) <= worst * w[b] + 1e-30).all()
