"""Trees of drafts on the GPU: attention over the 4-bit cache, adjusted logits and acceptance against the
64-bit definitions in tests/_step_ref.py, and a run of them together.

Tolerances of the attention are those of tests/test_gpu_cache.py (same kernel, same operations); a tree's positions are
integers.  Adjusted logits (u = 2^-24): a quotient or product, a product and a difference for the frequency, a difference for the
presence, one sum a bias, each rounded once in fp32 by u of a value that the magnitudes' sum M bounds, then one
rounding to the type: (4 + biases) u M + half a step |z|."""
import numpy as np
import pytest

from tests import _step_ref as ref
from tests._gpu import need_gpu
from tests.test_gpu_cache import dev, gpu_cache, quick_pool

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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def offsets(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)


def random_trees(rng, rows, loose=0.1):
    out = []
    for n in rows:
        p = [int(rng.integers(0, j)) if j else -1 for j in range(n)]
        out += [-1 if j and rng.random() < loose else x for j, x in enumerate(p)]
    return np.array(out, np.int64)


def check_tree(sv, c, q, rows, lens, parent, *, slot_pos=None, k_max=None, status_is=0, **kw):
    cu, R = offsets(rows), sum(rows)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    opt = dict(kw)
    if kw.get("slopes") is not None:
        opt["slopes"] = dev(np.asarray(kw["slopes"], np.float32))
    got = sv.cache_attend_tree(gpu_cache(sv, c), q, i32(cu), i32(lens), dev(c.table), i32(parent), B=len(rows),
                               k_max=max(rows) - 1 if k_max is None else k_max, status=status,
                               slot_pos=None if slot_pos is None else dev(slot_pos), **opt)
    torch.cuda.synchronize()
    assert int(status) == status_is
    out, lse, A, S = ref.tree(c, q[:R].double().cpu().numpy(), cu, lens, parent, slot_pos=slot_pos, **kw)
    u, D, cap = 2.0 ** -24, c.D, kw.get("cap", 0.0)
    bias = 0.0
    if kw.get("slopes") is not None:
        far = max(lens) if slot_pos is None else int(np.max(slot_pos)) + 32
        bias = float(np.max(np.abs(kw["slopes"]))) * far
    ds = (D * 2 * u + 4 * u) * S + cap * 2.0 ** -20 + 2 * u * bias
    rel = 2 * ds + 2.0 ** -20 + 2.0 ** -23 * (max(lens) / 16 + 16)
    seen = np.isfinite(lse)
    gl, go = got["lse"][:R].double().cpu().numpy(), got["out"][:R].double().cpu().numpy()
    assert np.array_equal(np.isfinite(gl), seen)
    err = np.abs(np.where(seen, gl, 0) - np.where(seen, lse, 0))
    tol = rel + 4 * u * np.abs(np.where(seen, lse, 0))
    assert (err <= tol).all(), float((err / tol).max())
    bf = q.dtype == torch.bfloat16
    w = rel + (2.0 ** -11 if bf else 2.0 ** -20)
    err, tol = np.abs(go - out), 1.01 * (A * w[..., None] + (2.0 ** -8 if bf else 2.0 ** -23) * np.abs(out)) + 1e-30
    assert (err <= tol).all(), float((err / tol).max())
    return got


TREES = [([1], [1], 1, 1, 64, 32), ([13], [900], 32, 8, 128, 64), ([32, 1, 7], [32, 200, 150], 5, 1, 128, 32),
         ([2, 31, 0, 30], [129, 160, 40, 300], 8, 2, 256, 64), ([26, 26], [4000, 517], 16, 4, 64, 128),
         ([32], [131], 7, 1, 128, 96), ([20, 9], [128, 140], 40, 8, 128, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lens,Hq,H,D,page", TREES)
def test_tree_attention(sv, rows, lens, Hq, H, D, page, dtype):
    rng = np.random.default_rng(sum(rows) + D)
    c = quick_pool(rng, B=len(rows), H=H, D=D, page=page, lens=lens, scaled=True)
    q = torch.from_numpy(rng.standard_normal((max(sum(rows), 1), Hq, D)).astype(np.float32)).to(DT[dtype]).cuda()
    check_tree(sv, c, q, rows, lens, random_trees(rng, rows))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("opt", [dict(cap=8.0), dict(slopes=True), dict(window=1), dict(window=3), dict(window=40, prefix=5),
                                 dict(window=2 ** 31 - 1), dict(cap=20.0, slopes=True, window=200, prefix=33)])
def test_tree_attention_options(sv, opt, gaps, dtype):
    rng = np.random.default_rng(5)
    rows, lens = [32, 4, 17], [700, 260, 20]
    c = quick_pool(rng, B=3, H=2, D=64, page=64, lens=lens)
    pos = None
    if gaps:
        pos = np.zeros((c.n_pages, c.page), np.int32)
        for b in range(3):
            pos[c.table[b]] = (np.cumsum(rng.integers(1, 4, c.table.shape[1] * c.page)) - 3).reshape(-1, c.page)
    q = torch.from_numpy(rng.standard_normal((sum(rows), 6, 64)).astype(np.float32)).to(DT[dtype]).cuda()
    kw = dict(opt)
    if kw.get("slopes"):
        kw["slopes"] = [0.3, 0.1, 0.03, 0.01, 0.0, 0.002]
    check_tree(sv, c, q, rows, lens, random_trees(rng, rows), slot_pos=pos, **kw)


def test_a_chain_is_the_attention_of_the_cache(sv):
    """parent = number - 1 gives cache_attend's results, bit for bit; a path of a tree those of the chain that it is."""
    rng = np.random.default_rng(6)
    rows, lens = [5, 32, 1], [300, 1000, 64]
    c = quick_pool(rng, B=3, H=2, D=128, page=64, lens=lens)
    for dtype in ("bf16", "f32"):
        for kw in (dict(), dict(window=90, cap=9.0, prefix=2)):
            q = torch.from_numpy(rng.standard_normal((sum(rows), 4, 128)).astype(np.float32)).to(DT[dtype]).cuda()
            parent = np.concatenate([np.arange(-1, n - 1) for n in rows])
            args = (gpu_cache(sv, c), q, i32(offsets(rows)), i32(lens), dev(c.table))
            a = sv.cache_attend(*args, B=3, k_max=31, **kw)
            b = sv.cache_attend_tree(*args, i32(parent), B=3, k_max=31, **kw)
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_bad_trees_and_lengths(sv):
    rng = np.random.default_rng(8)
    rows, lens = [4, 6, 3], [100, 80, 90]
    c = quick_pool(rng, B=3, H=1, D=64, page=32, lens=lens)
    q = torch.from_numpy(rng.standard_normal((13, 2, 64)).astype(np.float32)).cuda()
    parent = np.array([5, 0, 1, 2, -1, 0, 2, 7, -9, 1, -1, 0, 1])      # row 2 of the second names itself, 3 and 4 none
    check_tree(sv, c, q, rows, lens, parent, status_is=0x1000)
    parent[:4], parent[6:9] = [2 ** 31 - 1, 0, 1, 2], [1, 0, 0]
    check_tree(sv, c, q, rows, lens, parent)                            # a root's entry is not looked at
    check_tree(sv, c, q, rows, [100, 5, 90], parent, status_is=0x800)   # fewer slots than rows: they see nothing


def test_hidden_slots_of_a_tree_may_hold_anything(sv):
    """NaN scales in slots that the window hides from all nodes, and behind the length."""
    rng = np.random.default_rng(10)
    rows, lens = [9], [400]
    for dtype in ("bf16", "f32"):
        c = quick_pool(rng, B=1, H=1, D=128, page=64, lens=lens)
        q = torch.from_numpy(rng.standard_normal((9, 2, 128)).astype(np.float32)).to(DT[dtype]).cuda()
        parent = random_trees(rng, rows)
        a = check_tree(sv, c, q, rows, lens, parent, window=50, prefix=3)
        for slot in range(3, 391 - 49):                                 # root at 391, sees 342 ...
            blk = c.block(0, 0, slot)
            t = slot % 32
            blk[16 * 128 + t * 8:16 * 128 + t * 8 + 8] = 0x7F
            blk[34 * 128 + t:34 * 128 + 256:32] = 0x7F
        b = check_tree_only(sv, c, q, rows, lens, parent, window=50, prefix=3)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def check_tree_only(sv, c, q, rows, lens, parent, **kw):
    return sv.cache_attend_tree(gpu_cache(sv, c), q, i32(offsets(rows)), i32(lens), dev(c.table), i32(parent), B=len(rows),
                                k_max=max(rows) - 1, **kw)


# -------------------------------------------------------------- acceptance ---

@pytest.mark.parametrize("rows,k_max", [([1], 0), ([8], 7), ([32] * 3, 31), ([1, 2, 32, 5, 9, 17], 31), ([4] * 1000, 9)])
def test_acceptance(sv, rows, k_max):
    rng = np.random.default_rng(sum(rows))
    cu, R = offsets(rows), sum(rows)
    parent = random_trees(rng, rows)
    for V in (2, 4):                                                    # few tokens: siblings alike, long paths
        node, want = rng.integers(0, V, R), rng.integers(0, V, R)
        got = sv.tree_accept(i32(want), i32(node), i32(parent), i32(cu), B=len(rows), k_max=k_max)
        exp = ref.accept(want, node, parent, cu, k_max)
        for name, x in zip(("accepted_len", "out_tokens", "next_token", "path_rows"), exp):
            assert np.array_equal(got[name].cpu().numpy(), x), name


def test_acceptance_of_a_chain_is_the_verifications(sv):
    rng = np.random.default_rng(2)
    B, k, V = 30, 7, 512
    R = B * (k + 1)
    z = torch.from_numpy(rng.standard_normal((R, V)).astype(np.float32)).cuda()
    best = z.argmax(1).int()
    drafts = torch.where(torch.rand(R, device="cuda") < 0.7, best, 0).int()
    cu = i32(np.arange(0, R + 1, k + 1))
    want = sv.verify_greedy(z, cu, drafts, V=V, B=B, k_max=k)
    got = sv.tree_accept(want["row_token"], drafts.roll(1), i32(np.tile(np.arange(-1, k), B)), cu, B=B, k_max=k)
    for name in ("accepted_len", "out_tokens", "next_token"):
        assert torch.equal(got[name], want[name]), name


def test_acceptance_of_malformed_requests(sv):
    tok = i32(np.zeros(12))
    parent = i32([-1, 0, 1] * 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sv.tree_accept(tok, tok, parent, i32([0, 3, 3, 9, 12]), B=4, k_max=2, status=status)
    assert int(status) == 0x10                                          # no rows; six of at most three
    assert got["accepted_len"].tolist() == [2, 0, 0, 2] and got["next_token"].tolist() == [0, -1, -1, 0]
    assert got["out_tokens"][1].tolist() == [-1] * 3 == got["path_rows"][2].tolist()
    for bad in ([-1, 3, 6, 9, 12], [0, 3, 6, 9, 13], [2 ** 31 - 1, -2 ** 31, 6, 9, 12]):
        status.zero_()
        sv.tree_accept(tok, tok, parent, i32(bad), B=4, k_max=2, status=status)
        assert int(status) == 0x10
    status.zero_()
    got = sv.tree_accept(tok, tok, i32([7, 1, 2] * 4), i32([0, 3, 6, 9, 12]), B=4, k_max=2, status=status)
    assert int(status) == 0x1000 and got["accepted_len"].tolist() == [0] * 4


# ------------------------------------------------------------------ logits ---

def check_logits(sv, rng, rows, V, dtype, *, ld=None, history=0, penalties=True, path=True, tree=True, bias=0, mask=True,
                 in_place=False, shift=0, out_ld=None, few=None, bias_top=None):
    B, R, cu = len(rows), max(sum(rows), 1), offsets(rows)
    ld = ld or V
    z = torch.from_numpy((3 * rng.standard_normal(R * ld + shift)).astype(np.float32)).to(DT[dtype]).cuda()[shift:].view(R, ld)
    z[::3, ::5] = float("-inf")
    opt, kw = {}, {}
    top = few or V
    if penalties:
        n = rng.integers(0, history + 1, B)
        h = rng.integers(-2, top + 3, (B, max(history, 1)))
        kw.update(history=h, n_tokens=n, n_prompt=rng.integers(0, n + 1), repetition=rng.uniform(0.7, 1.5, B).astype(np.float32),
                  frequency=rng.uniform(-0.5, 1.0, B).astype(np.float32), presence=rng.uniform(-0.5, 1.0, B).astype(np.float32))
        for name, x in kw.items():
            opt[name] = dev(x) if x.dtype == np.float32 else i32(x)
    if path:
        kw["node_token"] = rng.integers(-1, top, R)
        opt["node_token"] = i32(kw["node_token"])
        if tree:
            kw["parent"] = np.concatenate([random_trees(rng, rows), [0] * (R - sum(rows))]).astype(np.int64)
            opt["parent"] = i32(kw["parent"])
    if bias:
        counts = rng.integers(0, bias + 1, B)
        ids, vals = rng.integers(-1, bias_top or min(V + 2, 40), counts.sum()), rng.standard_normal(counts.sum()).astype(np.float32)
        bc = offsets(counts)
        kw["bias"] = [(ids[bc[b]:bc[b + 1]], vals[bc[b]:bc[b + 1]]) for b in range(B)]
        if bias_top:                                                    # how many meet at a column at most
            bias = max([int(np.bincount(x + 1).max()) for x, _ in kw["bias"] if len(x)], default=0)
        opt.update(bias_cu=i32(bc), bias_ids=i32(ids), bias_values=dev(vals))
    if mask:
        kw["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (max(R // 2, 1), (V + 31) // 32 + 1)).astype(np.int32)
        kw["allowed"][0] = 0                                            # a mask that allows nothing
        kw["allowed_row"] = rng.integers(-1, len(kw["allowed"]), R)
        opt.update(allowed=dev(kw["allowed"]), allowed_row=i32(kw["allowed_row"]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, mag = ref.adjust(z.double().cpu().numpy(), cu, V, **kw)
    src = z.clone()
    out = src if in_place else None
    if out_ld:
        out = torch.zeros(R, out_ld, dtype=z.dtype, device="cuda")
    got = sv.adjust_logits(src, i32(cu), V=V, B=B, k_max=31, out=out, status=status, **opt)["logits"]
    torch.cuda.synchronize()
    assert int(status) == 0
    n = sum(rows)
    g, want, mag = got[:n, :V].double().cpu().numpy(), want[:n], mag[:n]
    gone = np.isneginf(want)
    assert np.array_equal(np.isneginf(g), gone)
    err = np.abs(np.where(gone, 0, g) - np.where(gone, 0, want))
    tol = (4 + bias) * 2.0 ** -24 * mag + HALF[dtype] * np.abs(np.where(gone, 0, want))
    assert (err <= 1.01 * tol).all(), float((err / np.maximum(tol, 1e-30)).max())
    if not in_place:
        assert torch.equal(src, z)
    elif ld > V:
        assert torch.equal(got[:, V:], z[:, V:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [([1], 1), ([1], 500), ([3, 1, 0, 5], 8192), ([32], 8193), ([2, 2], 31), ([4] * 9, 2049),
                                    ([1], 152064), ([5, 2], 50257), ([1, 6], 16391)])
def test_logits(sv, rows, V, dtype):
    rng = np.random.default_rng(V)
    check_logits(sv, rng, rows, V, dtype, history=200, bias=5)
    check_logits(sv, rng, rows, V, dtype, history=3000, few=50, bias=700, tree=False)


@pytest.mark.parametrize("in_place", [False, True])
def test_logits_of_many_requests(sv, in_place):
    """So many that no request's rows are dealt out to several CTAs."""
    rng = np.random.default_rng(37)
    check_logits(sv, rng, [2, 1] * 200, 8203, "bf16", history=60, bias=4, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kw", [dict(history=20000), dict(history=20000, bias=300, bias_top=8900), dict(bias=9000, bias_top=9011),
                                dict(bias=20000, bias_top=600, history=5000), dict(bias=3000, penalties=False, path=False)])
def test_logits_of_many_touched_columns(sv, kw, in_place):
    """More tokens, and more biases, than are kept or listed at a time; biases one a column and many."""
    rng = np.random.default_rng(39)
    check_logits(sv, rng, [3, 2], 9007, "f32", in_place=in_place, **kw)
    check_logits(sv, rng, [1], 9007, "bf16", in_place=in_place, **kw)


def test_a_bias_for_every_column(sv):
    """Sums of small integers: exact; repeated runs give the same bits."""
    rng = np.random.default_rng(41)
    V, B = 20011, 3
    z = torch.from_numpy(rng.integers(-50, 50, (B * 4, V)).astype(np.float32)).cuda()
    ids = np.concatenate([rng.permutation(V), rng.permutation(np.repeat(np.arange(V), 2)), rng.integers(0, 5, 700)])
    val = rng.integers(-9, 9, len(ids)).astype(np.float32)
    cu = np.array([0, V, 3 * V, 3 * V + 700])
    got = sv.adjust_logits(z, i32(np.arange(0, 13, 4)), V=V, B=B, k_max=3, bias_cu=i32(cu), bias_ids=i32(ids), bias_values=dev(val))["logits"]
    for b in range(B):
        add = np.zeros(V)
        np.add.at(add, ids[cu[b]:cu[b + 1]], val[cu[b]:cu[b + 1]])
        assert np.array_equal(got[4 * b:4 * b + 4].double().cpu().numpy(), z[4 * b:4 * b + 4].double().cpu().numpy() + add), b
    val = dev(rng.standard_normal(len(ids)).astype(np.float32))
    runs = [sv.adjust_logits(z, i32(np.arange(0, 13, 4)), V=V, B=B, k_max=3, bias_cu=i32(cu), bias_ids=i32(ids), bias_values=val)["logits"]
            for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_lengths_are_looked_at_without_penalties(sv):
    z = torch.zeros(2, 40, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n, is_bad in ((3, False), (4, True), (-1, True)):
        status.zero_()
        got = sv.adjust_logits(z, i32([0, 2]), V=40, B=1, k_max=1, history=i32([[1, 2, 3]]), n_tokens=i32([n]), status=status)["logits"]
        assert int(status) == (0x800 if is_bad else 0) and torch.equal(got, z)


def test_chains_and_trees_share_a_workspace_and_graphs(sv):
    """Both attentions and the acceptance captured, replayed in turn on one workspace, and on another stream."""
    rng = np.random.default_rng(43)
    rows, lens = [26, 9, 1], [1500, 400, 90]
    c = quick_pool(rng, B=3, H=2, D=128, page=64, lens=lens)
    q = torch.from_numpy(rng.standard_normal((36, 8, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
    parent = random_trees(rng, rows)
    args = (gpu_cache(sv, c), q, i32(offsets(rows)), i32(lens), dev(c.table))
    kw = dict(B=3, k_max=31)
    want = [sv.cache_attend(*args, **kw), sv.cache_attend_tree(*args, i32(parent), **kw), sv.cache_attend_tree(*args, i32(parent), window=70, **kw)]
    ws = sv.new_cache_workspace(args[0], args[4], Hq=8, **kw)
    token, node = i32(rng.integers(0, 2, 36)), i32(rng.integers(0, 2, 36))
    want.append(sv.tree_accept(token, node, i32(parent), args[2], **kw))
    calls = [sv.cache_attend(*args, workspace=ws, prepared=True, **kw), sv.cache_attend_tree(*args, i32(parent), workspace=ws, prepared=True, **kw),
             sv.cache_attend_tree(*args, i32(parent), workspace=ws, prepared=True, window=70, **kw),
             sv.tree_accept(token, node, i32(parent), args[2], prepared=True, **kw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for call in calls:
        call(stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    held = [call() for call in calls]                                   # where each writes
    for _ in range(3):
        for res in held:
            for x in res.values():
                x.fill_(0)
        for g in graphs:
            g.replay()
        for res, w in zip(held, want):
            assert all(torch.equal(res[x], w[x]) for x in w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(penalties=False), dict(path=False), dict(mask=False), dict(penalties=False, mask=False, bias=3),
                                dict(penalties=False, mask=False, path=False), dict(in_place=True), dict(in_place=True, ld=9011),
                                dict(ld=9008, out_ld=9003), dict(shift=3), dict(shift=1, out_ld=9000), dict(ld=9001, shift=5)])
def test_logits_of_every_kind(sv, kw, dtype):
    rng = np.random.default_rng(31)
    check_logits(sv, rng, [4, 1, 7], 9000, dtype, history=100, **{"bias": 9, **kw})


def test_logits_without_a_mask_index_and_bad_rules(sv):
    rng = np.random.default_rng(33)
    z = torch.from_numpy(rng.standard_normal((4, 64)).astype(np.float32)).cuda()
    cu, status = i32([0, 2, 4]), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda **kw: (status.zero_(), sv.adjust_logits(z, cu, V=64, B=2, k_max=1, status=status, **kw)["logits"])[1]
    bits = i32([[1, 0], [2, 0], [4, 0], [8, -2 ** 31]])
    got = call(allowed=bits)
    assert int(status) == 0 and got.isfinite().sum(1).tolist() == [1, 1, 1, 2]
    assert got[3, 63] == z[3, 63] and got[2, 2] == z[2, 2]
    got = call(allowed=bits, allowed_row=i32([0, 4, -1, -2]))
    assert int(status) == 0x4000 and got.isfinite().sum(1).tolist() == [1, 64, 64, 64]
    assert call(allowed=bits[:3])[3].isfinite().all() and int(status) == 0x4000
    one = torch.ones(2, device="cuda")
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        x = one.clone()
        x[1] = bad
        got = call(repetition=x, node_token=i32([0, 1, 2, 3]))
        assert int(status) == 0x2000 and torch.equal(got, z)
    got = call(frequency=one * float("nan"), presence=one * float("-inf"), node_token=i32([0, 1, 2, 3]))
    assert int(status) == 0x2000 and torch.equal(got, z)
    ids, val = i32([1, 2, 3]), torch.ones(3, device="cuda")
    for bad in ([0, 2, 4], [0, -1, 3], [2, 1, 3], [-1, 2, 3]):
        call(bias_cu=i32(bad), bias_ids=ids, bias_values=val)
        assert int(status) == 0x2000
    hist = i32([[5, 5, 5], [6, 6, 6]])
    got = call(history=hist, n_tokens=i32([3, 4]), frequency=one)
    assert int(status) == 0x800 and got[0, 5] == z[0, 5] - 3 and torch.equal(got[2:], z[2:])
    got = call(history=hist, n_tokens=i32([3, 2]), n_prompt=i32([-4, 9]), frequency=one)
    assert int(status) == 0 and got[0, 5] == z[0, 5] - 3 and torch.equal(got[2:], z[2:])
    got = call(parent=i32([-1, 3, 0, -2]), node_token=i32([0, 1, 2, 3]), presence=one)
    assert int(status) == 0x1000 and torch.equal(got, z)
    out = torch.full((4, 64), 9.0, device="cuda")
    sv.adjust_logits(z, i32([0, 2, 5]), V=64, B=2, k_max=3, status=status, out=out)
    assert torch.equal(out[:2], z[:2]) and bool((out[2:] == 9).all()) and int(status) & 0x10


def test_logits_handles_streams_and_graphs(sv):
    rng = np.random.default_rng(35)
    z = torch.from_numpy(rng.standard_normal((6, 9000)).astype(np.float32)).to(torch.bfloat16).cuda()
    kw = dict(V=9000, B=2, k_max=2, node_token=i32(rng.integers(0, 9000, 6)), presence=torch.ones(2, device="cuda"))
    cu = i32([0, 3, 6])
    want = sv.adjust_logits(z, cu, **kw)["logits"]
    call = sv.adjust_logits(z, cu, prepared=True, **kw)
    res = call()["logits"]
    assert torch.equal(res, want)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    with torch.cuda.graph(g):
        call()
    res.fill_(0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, want)
    got = sv.adjust_logits(z, cu, stream=side, **kw)["logits"]
    side.synchronize()
    assert torch.equal(got, want)
