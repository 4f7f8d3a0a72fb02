"""Prompt attention over many keys whose weights and values are alike, so that roundings of the sums go one way: against sums
in 64 bits.

Tolerances, from the operations (u = 2^-24).  Queries and keys have one channel that is not 0, so that a score is one
product, exact for these numbers, times a constant rounded twice; its distance to the row's reference is below 2^3 in log2 units, rounded to
within 8u; the exponential is within 2^-20.  A weight is then off by WEIGHT = 2^-20 + 16u, relative.
fp32 arithmetic: 64 terms of a tile are added one after another, tiles with their error kept (2u), references move by factors
of 2 or more (a rounding each, halved with every further one: 2u): SUMS = 70u, for weights and for values.
Tensor cores: weights of a row are added in pairs, 64 of them a step, the two halves (1), steps with their error kept (2u), up to 16
parts joined: 90u; the values' sums are truncated, up to 2^-13 of themselves, and weights rounded to bf16 before them (2^-8).
An output is the quotient of two sums (3u more), rounded once."""
import numpy as np
import pytest

from tests._gpu import need_gpu

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
WEIGHT = 2.0 ** -20 + 16 * U
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def sv():
    need_gpu()
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def inputs(scores, D, n, dtype, odd=False):
    """q [n, 1, D], k, v [m, 1, D] whose row i has the scores given (scale 1); values between 0.5 and 1.5 that rise slowly.
    odd: strides that TMA cannot take."""
    m = len(scores)
    new = lambda rows: torch.zeros(rows, 1, D + (1 if odd else 0), dtype=dtype, device="cuda")[..., :D]
    q, k, v = new(n), new(m), new(m)
    q[:, 0, 0] = 1
    k[:, 0, 0] = scores.to(dtype)
    rise = 1 + 0.2 * torch.arange(m, device="cuda", dtype=torch.float64) / m
    v[:, 0] = (rise[:, None] * torch.linspace(0.5, 1.25, D, device="cuda", dtype=torch.float64)).to(dtype)
    return q, k, v


def check(got, k, v, rows, n, sums, weights=0.0):
    """The rows given (of n, which are the last of the keys)."""
    m = len(k)
    s = k[:, 0, 0].double()
    w, top = torch.exp(s - s.max()), float(s.max())
    worst = 0.0
    for i in rows:
        upto = m - n + i + 1
        total = float(w[:upto].sum())
        lse = top + np.log(total)
        out = sum((w[a:b, None] * v[a:b, 0].double()).sum(0) for a, b in
                  ((a, min(a + (1 << 20), upto)) for a in range(0, upto, 1 << 20))) / total
        tol = WEIGHT + sums + 4 * U * abs(lse)
        err = abs(float(got["lse"][i, 0]) - lse)
        assert err <= tol, ("lse", i, err / tol)
        # (the values are positive: sum p |v| is the output itself)
        err = ((got["out"][i, 0].double() - out).abs() / out).max()
        tol = 2 * (WEIGHT + sums) + 3 * U + weights + 1.01 * HALF[v.dtype]
        assert float(err) <= tol, ("out", i, float(err) / tol)
        worst = max(worst, float(err) / tol)
    return worst


def scores_of(kind, m):
    j = torch.arange(m, device="cuda", dtype=torch.float64)
    if kind == "first":                                    # the first key above the others, which are equal
        return torch.where(j == 0, 0.375, 0.0)
    if kind == "creeping":                                 # each key a little above the one before
        return j * 2.0 ** -20
    return torch.where(j % 4096 == 4095, (j // 4096) % 5 * 0.25, -0.625)


FP32 = [("first", 64, 1048583), ("creeping", 64, 1048583), ("waves", 64, 600011), ("first", 128, 262147), ("creeping", 256, 65541)]


@pytest.mark.parametrize("kind,D,m", FP32)
def test_sums_of_fp32_prompts(sv, kind, D, m):
    q, k, v = inputs(scores_of(kind, m), D, 3, torch.float32)
    got = sv.prompt_attend(q, k, v, i32([0, 3]), B=1, cu_keys=i32([0, m]), scale=1.0)
    check(got, k, v, [0, 1, 2], 3, 70 * U)


@pytest.mark.parametrize("kind,D,m", [("first", 64, 1048583), ("waves", 128, 262147)])
def test_sums_of_bf16_prompts_that_tma_cannot_fetch(sv, kind, D, m):
    q, k, v = inputs(scores_of(kind, m), D, 3, torch.bfloat16, odd=True)
    got = sv.prompt_attend(q, k, v, i32([0, 3]), B=1, cu_keys=i32([0, m]), scale=1.0)
    check(got, k, v, [0, 2], 3, 70 * U)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_key_many_times(sv, dtype):
    """A row of keys and values read over and over (strides of 0): the output is the value, the lse the number's logarithm."""
    m = 1 << 22
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    q = torch.randn(2, 2, 64, generator=gen, device="cuda").to(dtype)
    v = (0.7 + 0.5 * torch.rand(1, 1, 64, generator=gen, device="cuda")).to(dtype)
    got = sv.prompt_attend(q, torch.zeros_like(v).expand(m, 1, 64), v.expand(m, 1, 64), i32([0, 2]), B=1, cu_keys=i32([0, m]))
    for i in range(2):
        lse = np.log(m - 1.0 + i)
        assert (got["lse"][i].double() - lse).abs().max() <= WEIGHT + 70 * U + 4 * U * lse
        err = ((got["out"][i].double() - v[0].double()).abs() / v[0].double()).max()
        assert float(err) <= 2 * (WEIGHT + 70 * U) + 3 * U + 1.01 * HALF[dtype], float(err)


@pytest.mark.parametrize("kind,D", [("first", 64), ("first", 128), ("waves", 64), ("first", 256)])
def test_sums_of_prompts_on_the_tensor_cores(sv, kind, D):
    """So many rows that their keys are not split."""
    m, n = 1048583, 77 * (128 if D == 256 else 256)
    q, k, v = inputs(scores_of(kind, m), D, n, torch.bfloat16)
    got = sv.prompt_attend(q, k, v, i32([0, n]), B=1, cu_keys=i32([0, m]), scale=1.0)
    check(got, k, v, [0, 1, n - 1], n, 90 * U, 2.0 ** -8 + 2.0 ** -13)
