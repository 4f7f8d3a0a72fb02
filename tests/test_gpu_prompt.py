"""Attention of whole prompts on the GPU against the 64-bit definition in tests/_step_ref.py.

Tolerances, from the operations (u = 2^-24, half an ulp of fp32).  A score is a sum of D products
in fp32 (each product of two bf16 is exact; at most 2 roundings or truncations of 2u a term), scaled by a constant rounded
twice, capped (the tanh within 2^-20 of the result), biased (slope, distance and difference rounded once each) and
taken less the row's reference: ds = (2 D u + 6 u) S + 2^-20 cap + 4 u bias, S = scale * sum |q k|.
exp turns ds into a relative error of 2 ds at most, its own is within 2^-20.  bf16: a weight is rounded to bf16
(half a step, 2^-8 at most, relative).  Sums run over `keys` terms, 16 a step, each step truncated by 2^-23 of what
it has.  An output is rounded once, by half a step of its type."""
import numpy as np
import pytest

from tests import _step_ref as ref
from tests._gpu import need_gpu

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def sv():
    need_gpu()
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


def rand(rng, *shape, dtype="bf16", scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(DT[dtype]).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def offsets(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)


def check(sv, q, k, v, rows, keys=None, *, got=None, **kw):
    """Outputs and lse of every row against the definition."""
    cu, cuk = offsets(rows), None if keys is None else offsets(keys)
    R = int(cu[-1])
    opt = dict(kw)
    if opt.get("slopes") is not None:
        opt["slopes"] = torch.tensor(np.asarray(opt["slopes"], np.float32), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if got is None:
        got = sv.prompt_attend(q, k, v, i32(cu), B=len(rows), cu_keys=None if keys is None else i32(cuk), status=status, **opt)
    torch.cuda.synchronize()
    assert int(status) == 0
    dtype = "f32" if q.dtype == torch.float32 else "bf16"
    out, lse, A, S = ref.prompt(q[:R].double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(), cu, cuk, **kw)
    u, D, most = 2.0 ** -24, q.shape[2], max(keys or rows)
    bias = 0.0 if kw.get("slopes") is None else float(np.max(np.abs(kw["slopes"]))) * most
    ds = (2 * D * u + 6 * u) * S + 2.0 ** -20 * kw.get("cap", 0.0) + 4 * u * bias
    sums = 2.0 ** -23 * (most / 16 + 16)
    rel = 2 * ds + 2.0 ** -20 + sums
    seen = np.isfinite(lse)
    gl, go = got["lse"][:R].double().cpu().numpy(), got["out"][:R].double().cpu().numpy()
    assert np.array_equal(np.isfinite(gl), seen)
    err = np.abs(np.where(seen, gl, 0) - np.where(seen, lse, 0))
    tol = rel + 4 * u * np.abs(np.where(seen, lse, 0))
    assert (err <= tol).all(), float((err / tol).max())
    w = rel + (2.0 ** -8 if dtype == "bf16" else 0.0)
    err, tol = np.abs(go - out), 1.01 * (A * w[..., None] + HALF[dtype] * np.abs(out)) + 1e-30
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere((err > tol).any(-1))[:5])
    assert (go[~seen] == 0).all()
    return got


# rows, heads, kv heads, D: one row, odd ones, groups that do not divide a tile, tiles that end within a request
SHAPES = [([1], 1, 1, 64), ([1, 1, 1], 8, 2, 128), ([5], 4, 4, 256), ([37], 32, 8, 128), ([64, 1, 65], 5, 1, 64),
          ([129, 3, 127, 0, 2], 7, 1, 128), ([200], 6, 2, 256), ([300, 17], 12, 12, 64), ([257], 40, 8, 128),
          ([33, 70], 48, 1, 64), ([10], 128, 1, 128), ([520], 4, 4, 128), ([390, 140], 16, 2, 256), ([7, 9], 150, 1, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,Hq,H,D", SHAPES)
def test_shapes(sv, rows, Hq, H, D, dtype):
    rng = np.random.default_rng(sum(rows) + Hq)
    R = sum(rows)
    check(sv, rand(rng, R, Hq, D, dtype=dtype), rand(rng, R, H, D, dtype=dtype), rand(rng, R, H, D, dtype=dtype), rows)


OPTIONS = [dict(cap=20.0), dict(slopes=[0.5, 0.25, 0.03, 0.0]), dict(window=1), dict(window=40), dict(window=130, prefix=3),
           dict(window=2 ** 31 - 1), dict(scale=-0.3), dict(scale=0.0), dict(cap=1e-3), dict(cap=1e30),
           dict(window=100, prefix=2 ** 31 - 1), dict(cap=30.0, slopes=[0.1, 0.2, 0.3, 0.4], window=150, prefix=70, scale=0.2)]


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("f32", 64)])
@pytest.mark.parametrize("opt", OPTIONS)
def test_options(sv, opt, dtype, D):
    rng = np.random.default_rng(7)
    rows = [310, 5, 140]
    R = sum(rows)
    check(sv, rand(rng, R, 4, D, dtype=dtype), rand(rng, R, 2, D, dtype=dtype), rand(rng, R, 2, D, dtype=dtype), rows, **opt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("opt", [dict(), dict(window=200, prefix=5), dict(cap=15.0, slopes=[0.01, 0.02])])
def test_pieces_over_what_came_before(sv, opt, dtype):
    """More keys than rows, as many, fewer (rows that see nothing), none; a request without rows."""
    rng = np.random.default_rng(9)
    rows, keys = [3, 130, 40, 17, 0, 12, 1], [700, 130, 25, 0, 90, 13, 515]
    check(sv, rand(rng, sum(rows), 2, 128, dtype=dtype), rand(rng, sum(keys), 1, 128, dtype=dtype),
          rand(rng, sum(keys), 1, 128, dtype=dtype), rows, keys, **opt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_addresses(sv, dtype):
    """Queries, keys and values side by side in one product; heads before rows; rows that start anywhere."""
    rng = np.random.default_rng(11)
    rows, Hq, H, D = [100, 60], 6, 2, 64
    R = sum(rows)
    qkv = rand(rng, R, Hq + 2 * H, D, dtype=dtype)
    a = check(sv, qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], rows)
    q, k, v = (x.contiguous() for x in (qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]))
    b = check(sv, q, k, v, rows)
    turned = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    c = check(sv, *turned, rows)
    assert torch.equal(a["out"], b["out"]) and torch.equal(b["out"], c["out"]) and torch.equal(b["lse"], c["lse"])
    wide = [torch.zeros(R * x.shape[1] * (D + 3) + 1, dtype=x.dtype, device="cuda")[1:].view(R, x.shape[1], D + 3)[..., :D] for x in (q, k, v)]
    for w, x in zip(wide, (q, k, v)):
        w.copy_(x)
    check(sv, *wide, rows)
    one = k[:, :1].expand(R, 2, D)                              # two kv heads that are one
    check(sv, q, one, one, rows)


def test_rows_and_keys_of_no_request(sv):
    """Rows behind the last sequence stay as they were; keys that no row sees may hold anything."""
    rng = np.random.default_rng(13)
    rows, R, K = [70, 3], 90, 120
    for dtype in ("bf16", "f32"):
        q, k, v = rand(rng, R, 4, 128, dtype=dtype), rand(rng, K, 2, 128, dtype=dtype), rand(rng, K, 2, 128, dtype=dtype)
        k[73:], v[73:], q[73:] = float("nan"), float("inf"), float("nan")
        want = check(sv, q, k, v, rows)
        call = sv.prompt_attend(q, k, v, i32(offsets(rows)), B=2, prepared=True)
        res = call()
        for name in ("out", "lse"):
            res[name].fill_(7)
        call()
        torch.cuda.synchronize()
        assert torch.equal(res["out"][:73], want["out"][:73]) and bool((res["out"][73:] == 7).all())
        assert bool((res["lse"][73:] == 7).all())
        # a window hides all but the last keys of a long context from a short piece
        rows2, keys2 = [2, 5], [60, 60]
        q2, k2, v2 = q[:7], k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0)
        hidden = torch.zeros(120, dtype=torch.bool, device="cuda")
        for b, n in enumerate(rows2):
            hidden[60 * b + 2:60 * b + 60 - n - 9] = True      # window 10, prefix 2
        kk, vv = k2.clone(), v2.clone()
        kk[hidden], vv[hidden] = float("nan"), float("nan")
        a = check(sv, q2, k2, v2, rows2, keys2, window=10, prefix=2)
        b = sv.prompt_attend(q2, kk, vv, i32(offsets(rows2)), B=2, cu_keys=i32(offsets(keys2)), window=10, prefix=2)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_one_requests_numbers_do_not_reach_another(sv):
    rng = np.random.default_rng(15)
    rows = [50, 200, 61]
    for dtype in ("bf16", "f32"):
        q, k, v = (rand(rng, sum(rows), h, 64, dtype=dtype) for h in (4, 2, 2))
        a = check(sv, q, k, v, rows)
        for x in (q, k, v):
            x[50:250] = float("nan")
        b = sv.prompt_attend(q, k, v, i32(offsets(rows)), B=3)
        for name in ("out", "lse"):
            assert torch.equal(a[name][:50], b[name][:50]) and torch.equal(a[name][250:], b[name][250:])


def test_peaked_and_large_scores(sv):
    """Rows whose largest score comes late, moves by hundreds, or leaves the rest far behind."""
    rng = np.random.default_rng(17)
    for dtype in ("bf16", "f32"):
        q, k, v = rand(rng, 400, 2, 128, dtype=dtype, scale=4.0), rand(rng, 400, 1, 128, dtype=dtype), rand(rng, 400, 1, 128, dtype=dtype)
        k *= torch.linspace(0.1, 9, 400, device="cuda")[:, None, None].to(k.dtype)
        check(sv, q, k, v, [400])
        check(sv, q, k.flip(0).contiguous(), v, [150, 250])


def test_malformed_offsets(sv):
    rng = np.random.default_rng(19)
    for dtype in ("bf16", "f32"):
        q, k, v = rand(rng, 60, 2, 64, dtype=dtype), rand(rng, 60, 1, 64, dtype=dtype), rand(rng, 60, 1, 64, dtype=dtype)
        good = check(sv, q, k, v, [20, 40])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call = sv.prompt_attend(q, k, v, i32([0, 20, 61]), B=2, status=status, prepared=True)
        res = call()
        res["out"].fill_(3)
        call()
        assert int(status) == 0x10 and torch.equal(res["out"][:20], good["out"][:20]) and bool((res["out"][20:] == 3).all())
        for bad in ([0, 20, 61], [0, 30, 20], [-5, 20, 60], [2 ** 31 - 1, -2 ** 31, 5]):
            status.zero_()
            sv.prompt_attend(q, k, v, i32(bad), B=2, status=status)
            assert int(status) & 0x10
        for bad, ok in [([0, 20, 61], 1), ([20, 0, 40], 1), ([-1, 19, 59], 1)]:
            status.zero_()
            got = sv.prompt_attend(q, k, v, i32([0, 20, 60]), B=2, cu_keys=i32(bad), status=status)
            assert int(status) == 0x800
            b = 1 if bad[2] == 61 else 0
            part = slice(0, 20) if b == 0 else slice(20, 60)
            assert bool((got["out"][part] == 0).all()) and bool((got["lse"][part] == float("-inf")).all())


def test_many_requests(sv):
    """More requests than a CTA has threads, empty ones among them."""
    rng = np.random.default_rng(21)
    rows = [int(x) for x in rng.integers(0, 6, 1300)]
    for dtype in ("bf16", "f32"):
        R = sum(rows)
        check(sv, rand(rng, R, 2, 64, dtype=dtype), rand(rng, R, 1, 64, dtype=dtype), rand(rng, R, 1, 64, dtype=dtype), rows)


def test_streams_graphs_and_shared_workspaces(sv):
    rng = np.random.default_rng(23)
    cases = []
    for rows, Hq, H in [([300, 20], 8, 2), ([1], 8, 2), ([700], 4, 1), ([40] * 9, 8, 8)]:
        R = sum(rows)
        x = [rand(rng, R, h, 128) for h in (Hq, H, H)]
        cases.append((x, i32(offsets(rows)), len(rows), sv.prompt_attend(*x, i32(offsets(rows)), B=len(rows))))
    ws = torch.zeros(max(sv.prompt_workspace_bytes(8, h, 128) for h in (1, 2, 8)) * 2, dtype=torch.uint8, device="cuda")
    calls = [sv.prompt_attend(*x, cu, B=B, workspace=ws, prepared=True) for x, cu, B, _ in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for c in calls:
        with torch.cuda.stream(side):
            c()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for _ in range(3):
        for c, g, (_, _, _, want) in zip(calls, graphs, cases):
            res = c()
            for name in ("out", "lse"):
                res[name].fill_(0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(res["out"], want["out"]) and torch.equal(res["lse"], want["lse"])
    for x, cu, B, want in cases:
        got = sv.prompt_attend(*x, cu, B=B, stream=side)
        side.synchronize()
        assert torch.equal(got["out"], want["out"])


@pytest.mark.parametrize("opt,D", [(dict(), 128), (dict(window=3000, prefix=4), 128), (dict(), 64), (dict(), 256),
                                   (dict(cap=20.0, window=20000), 64), (dict(cap=20.0, slopes=[1e-4, 0.0, 1e-5, 1e-3]), 256)])
def test_long_prompts_by_samples_of_their_rows(sv, opt, D):
    """A long prompt and a piece over a long context (longer than tensor memory adds up at once): some rows against the
    definition."""
    rng = np.random.default_rng(25)
    n, m, Hq, H = 5003, 36011, 4, 1
    given = {**opt, "slopes": torch.tensor(opt["slopes"], device="cuda")} if "slopes" in opt else opt
    q, k, v = rand(rng, n, Hq, D), rand(rng, m, H, D), rand(rng, m, H, D)
    got = sv.prompt_attend(q, k, v, i32([0, n]), B=1, cu_keys=i32([0, m]), **given)
    own = sv.prompt_attend(q, k[-n:], v[-n:], i32([0, n]), B=1, **given)
    for i in [0, 1, 127, 2048, 4095, 5002]:
        upto = m - n + i + 1
        res = {x: got[x][i:i + 1] for x in got}
        check(sv, q[i:i + 1], k[:upto], v[:upto], [1], [upto], got=res, **opt)
        check(sv, q[i:i + 1], k[m - n:upto], v[m - n:upto], [1], [i + 1], got={x: own[x][i:i + 1] for x in own}, **opt)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("opt", [dict(), dict(window=900, prefix=70), dict(cap=15.0, slopes=[0.01, 0.02, 0.0, 0.003], window=3000)])
def test_few_rows_over_long_contexts(sv, opt, D):
    """So few rows that they are split along the keys: one row, a group that does not divide a tile, tiles whose first sees fewer
    keys than its second, rows that see nothing, a request whose keys are too few to split."""
    rng = np.random.default_rng(27)
    for rows, keys, Hq, H in [([1], [9001], 4, 1), ([140], [2600], 4, 4), ([70, 3, 0, 5], [5000, 90, 700, 2], 4, 2)]:
        check(sv, rand(rng, sum(rows), Hq, D), rand(rng, sum(keys), H, D), rand(rng, sum(keys), H, D), rows, keys, **opt)
    if "slopes" not in opt:
        check(sv, rand(rng, 300, 3, D), rand(rng, 2500, 1, D), rand(rng, 2500, 1, D), [300], [2500], **opt)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_split_prompts_repeat_and_share_a_workspace(sv, D):
    """The same bits every time, next to calls that are not split, captured and on another stream."""
    rng = np.random.default_rng(29)
    ws = sv.new_prompt_workspace(4, 1, D)
    calls = []
    for rows, keys in [([5], [30000]), ([900] * 30, [900] * 30), ([200], [4000]), ([2, 2], [40000, 300]), ([4], [16])]:
        q, k, v = rand(rng, sum(rows), 4, D), rand(rng, sum(keys), 1, D), rand(rng, sum(keys), 1, D)
        args = (q, k, v, i32(offsets(rows)))
        want = sv.prompt_attend(*args, B=len(rows), cu_keys=i32(offsets(keys)))
        calls.append((sv.prompt_attend(*args, B=len(rows), cu_keys=i32(offsets(keys)), workspace=ws, prepared=True), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call, _ in calls:
        call(stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = [call() for call, _ in calls]
    for _ in range(5):
        for res in held:
            for x in res.values():
                x.fill_(0)
        g.replay()
        for res, (_, want) in zip(held, calls):
            assert torch.equal(res["out"], want["out"]) and torch.equal(res["lse"], want["lse"])
    long = [sv.prompt_attend(q[:1], k, v, i32([0, 1]), B=1, cu_keys=i32([0, 300])) for _ in range(20)]
    assert all(torch.equal(x["out"], long[0]["out"]) for x in long)


def test_malformed_offsets_of_split_prompts(sv):
    rng = np.random.default_rng(31)
    q, k, v = rand(rng, 60, 2, 64), rand(rng, 5000, 1, 64), rand(rng, 5000, 1, 64)
    good = check(sv, q, k, v, [20, 40], [2500, 2500])
    for cu, cuk, is_status in [([0, 20, 61], [0, 2500, 5000], 0x10), ([0, 20, 60], [0, 2500, 5001], 0x800), ([0, 20, 10], [0, 2500, 5000], 0x10)]:
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = sv.prompt_attend(q, k, v, i32(cu), B=2, cu_keys=i32(cuk), status=status)
        assert int(status) == is_status and torch.equal(got["out"][:20], good["out"][:20])
        if is_status == 0x800:
            assert bool((got["out"][20:] == 0).all()) and bool((got["lse"][20:] == float("-inf")).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_split_prompts_with_fewer_items_than_could_be(sv, D):
    """Requests and rows of a padded batch leave whole groups of CTAs without an item."""
    rng = np.random.default_rng(33)
    rows, keys, R = [1, 1, 0, 21, 3, 105], [90, 2, 0, 3000, 90, 2500], 300
    q, k, v = rand(rng, R, 3, D), rand(rng, 8000, 1, D), rand(rng, 8000, 1, D)
    for opt in (dict(), dict(cap=20.0), dict(window=2000, prefix=3)):
        check(sv, q, k, v, rows, keys, **opt)
    check(sv, q, k, v, [0, 0, 0, 0, 0, 1], [9, 0, 5, 0, 0, 2000])
    none = sv.prompt_attend(q, k, v, i32([0, 0, 0]), B=2, cu_keys=i32([0, 3000, 8000]), prepared=True)
    res = none()
    for x in res.values():
        x.fill_(5)
    none()
    assert all(bool((x == 5).all()) for x in res.values())
