"""Distance biases so steep that a row's own key decides alone: its bias is 0, whatever its neighbours' are.

Tolerances: those of tests/test_gpu_prompt.py, where the bias of a key is off by two roundings of itself (slope times log2 e, times
the distance) and counts where the key's weight does: among keys whose weight is above 2^-40 (the others stay below keys * 2^-39 of
the sum with twice that error)."""
import numpy as np
import pytest

from tests import _step_ref
from tests._gpu import need_gpu
from tests.test_gpu_prompt import HALF, i32, offsets, rand

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    need_gpu()
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


@pytest.mark.parametrize("opt", [dict(), dict(cap=20.0), dict(window=50, prefix=3)])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_prompts(sv, dtype, D, opt):
    rng = np.random.default_rng(6)
    rows, slopes = [150, 1, 140], np.array([1000.0, 3.0, 1e7, 1e34], np.float32)
    q, k, v = (rand(rng, sum(rows), h, D, dtype=dtype) for h in (4, 2, 2))
    cu = offsets(rows)
    out, lse, A, S = _step_ref.prompt(*(x.double().cpu().numpy() for x in (q, k, v)), cu, slopes=slopes, **opt)
    got = sv.prompt_attend(q, k, v, i32(cu), B=3, slopes=torch.tensor(slopes, device="cuda"), **opt)
    # weights above 2^-40: biases up to 40 ln 2 and the scores' range
    bias = np.where(slopes < 40 * np.log(2) + 2 * S, 40 * np.log(2) + 2 * S, 0.0)
    ds = (2 * D * U + 6 * U) * S + 2.0 ** -20 * opt.get("cap", 0.0) + 4 * U * bias
    rel = 2 * ds + 2.0 ** -20 + 2.0 ** -23 * (150 / 16 + 16)
    gl, go = got["lse"].double().cpu().numpy(), got["out"].double().cpu().numpy()
    err = np.abs(gl - lse) / (rel + 4 * U * np.abs(lse))
    assert (err <= 1).all(), err.max((0,))
    w = rel + (2.0 ** -8 if dtype == "bf16" else 0.0)
    assert (np.abs(go - out) <= 1.01 * (A * w[..., None] + HALF[dtype] * np.abs(out)) + 1e-30).all()
