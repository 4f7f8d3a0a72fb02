"""The 4-bit paged cache at the edges of its contract: limits of the arguments,
what hidden slots hold, streams, shared pages.  Bounds are those that
tests/test_gpu_cache.py derives."""
import numpy as np
import pytest

from tests import _cache_ref as ref
from tests._gpu import need_gpu
from tests.test_gpu_cache import check_attention, dev, gpu_cache, queries, quick_pool, run_attention

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def gapped_positions(rng, c, first=0):
    """Positions of every slot, rising by 1 to 3 from `first` in each request."""
    pos = np.zeros((c.n_pages, c.page), np.int32)
    for b in range(len(c.table)):
        pos[c.table[b]] = (first + np.cumsum(rng.integers(1, 4, c.table.shape[1] * c.page)) - 1).reshape(-1, c.page)
    return pos


# --------------------------------------------------------------- streams ---

def split_case(sv):
    """A call whose tasks are split between blocks, and its results."""
    rng = np.random.default_rng(40)
    lens = [9000, 17, 12000]
    c = quick_pool(rng, B=3, H=2, D=128, page=64, lens=lens)
    q = queries(rng, 9, 10, 128, "bf16")
    cache, tab = gpu_cache(sv, c), dev(c.table)
    cu, ln = dev(np.array([0, 3, 6, 9], np.int32)), dev(np.asarray(lens, np.int32))
    ws = sv.new_cache_workspace(cache, tab, B=3, k_max=2, Hq=10)
    want = sv.cache_attend(cache, q, cu, ln, tab, B=3, k_max=2, workspace=ws)
    torch.cuda.synchronize()
    return (cache, q, cu, ln, tab), {k: x.clone() for k, x in want.items()}, ws.numel()


def litter(n):
    """Free blocks of the current stream's memory, full of bytes that are no zeros."""
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    del junk


def test_a_call_on_another_stream_while_the_current_one_is_busy():
    sv = need_gpu()
    args, want, n = split_case(sv)
    side = torch.cuda.Stream()
    for _ in range(5):
        litter(n)
        torch.cuda._sleep(20_000_000)                     # what the current stream is given now comes late
        got = sv.cache_attend(*args, B=3, k_max=2, stream=side)
        late = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        side.synchronize()
        assert all(torch.equal(want[k].cpu(), got[k].cpu()) for k in want)
        torch.cuda.current_stream().synchronize()
        assert all(torch.equal(want[k], got[k]) for k in want) and all((x == 255).all() for x in late)


def test_a_handle_prepared_on_a_busy_stream_and_called_on_another():
    sv = need_gpu()
    args, want, n = split_case(sv)
    side = torch.cuda.Stream()
    litter(n)
    torch.cuda._sleep(20_000_000)
    call = sv.cache_attend(*args, B=3, k_max=2, prepared=True)
    for _ in range(3):
        got = call(stream=side)
        side.synchronize()
        assert all(torch.equal(want[k].cpu(), got[k].cpu()) for k in want)


def test_inputs_dropped_after_a_call_on_another_stream_stay():
    sv = need_gpu()
    args, want, n = split_case(sv)
    side = torch.cuda.Stream()
    for _ in range(5):
        q = args[1].clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = sv.cache_attend(args[0], q, *args[2:], B=3, k_max=2, stream=side)
        del q
        late = [torch.full_like(args[1], float("nan")) for _ in range(3)]
        side.synchronize()
        assert all(torch.equal(want[k], got[k]) for k in want)
        del late


# ------------------------------------------------------- limits of the arguments ---

@pytest.mark.parametrize("prefix", [2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 128, 1 << 30])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_prefix_beyond_every_slot_shows_all(dtype, prefix):
    """A window with such a prefix hides nothing."""
    sv = need_gpu()
    rng = np.random.default_rng(41)
    lens, cu = [700, 33, 1, 300], np.array([0, 3, 6, 7, 10])
    c = quick_pool(rng, B=4, H=2, D=64, page=64, lens=lens)
    q = queries(rng, 10, 4, 64, dtype)
    *_, status = check_attention(sv, c, q, cu, lens, 2, window=20, prefix=prefix)
    assert status == 0


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30])
def test_the_widest_window_over_negative_positions_shows_all(window):
    sv = need_gpu()
    rng = np.random.default_rng(42)
    lens, cu = [700, 33, 300], np.array([0, 2, 4, 6])
    c = quick_pool(rng, B=3, H=2, D=64, page=64, lens=lens)
    pos = gapped_positions(rng, c, first=-5000)
    q = queries(rng, 6, 4, 64, "bf16")
    *_, status = check_attention(sv, c, q, cu, lens, 1, window=window, slot_pos=pos)
    assert status == 0


@pytest.mark.parametrize("cap", [1e-39, 1e-45])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_cap_too_small_for_its_reciprocal(dtype, cap):
    """Scores of no size: every slot weighs the same, a row of zeros included."""
    sv = need_gpu()
    rng = np.random.default_rng(43)
    lens, cu = [300, 33], np.array([0, 2, 4])
    c = quick_pool(rng, B=2, H=2, D=128, page=64, lens=lens)
    q = queries(rng, 4, 4, 128, dtype)
    q[1] = 0
    check_attention(sv, c, q, cu, lens, 1, cap=cap)


# -------------------------------------------------- slots that the window hides ---

def poison(rng, c, hidden):
    """NaN scales, and any others, in the given slots of each request."""
    D = c.D
    for b, slots in enumerate(hidden):
        for s in slots:
            blk = c.pages[c.table[b, s // c.page], :, s % c.page // 32]
            t = s % 32
            blk[:, 16 * D + t * (D // 16):16 * D + (t + 1) * (D // 16)] = rng.choice(np.array([0x7F, 0xFF, 0x30], np.uint8), D // 16)
            blk[:, 34 * D + t:36 * D:32] = rng.choice(np.array([0x7F, 0xFF], np.uint8), D // 16)


HIDDEN = [  # rows, window, prefix, positions with gaps
    (1, 1, 0, False), (4, 33, 3, False), (3, 150, 40, False), (4, 100, 130, False),
    (1, 1, 0, True), (4, 33, 3, True), (3, 150, 40, True), (4, 100, 130, True)]


def hidden_case(rng, D, page, rows, window, prefix, gaps):
    lens = [1000, 641, 300, 129, 128, 5]
    n = [min(rows, x) for x in lens]
    cu = np.concatenate([[0], np.cumsum(n)])
    c = quick_pool(rng, B=len(lens), H=2, D=D, page=page, lens=lens)
    pos = gapped_positions(rng, c) if gaps else None
    hidden = []
    for b, (L, r) in enumerate(zip(lens, n)):
        i = np.arange(L)
        at = i if pos is None else pos[c.table[b, i // page], i % page].astype(np.int64)
        hidden.append(i[(at[L - r] - at >= window) & (i >= prefix) & (i < L - r)])
    return c, lens, cu, pos, hidden


def exact_bounds(c, q, cu, lens, **kw):
    """out, lse of the definition and how far results may be from them."""
    out, lse, A, S, w = ref.attention(c, q.float().cpu().numpy(), cu, lens, **kw)
    u = 2.0 ** -24
    ds = (c.D * 2 * u + 4 * u) * S
    bf = q.dtype == torch.bfloat16
    rel = 2 * ds + 2.0 ** -20 + 2.0 ** -23 * (max(lens) / 16 + 16) + (2.0 ** -11 if bf else 2.0 ** -20)
    tol = A * rel[..., None] + (2.0 ** -8 * np.abs(out) if bf else 0) + 1e-30
    return out, tol, lse, ds + 4 * u * np.abs(lse) + 2.0 ** -19, w


@pytest.mark.parametrize("rows,window,prefix,gaps", HIDDEN)
@pytest.mark.parametrize("D,page,dtype", [(64, 32, "bf16"), (128, 64, "f32"), (256, 96, "bf16"), (128, 32, "bf16")])
def test_what_hidden_slots_hold_does_not_matter(D, page, dtype, rows, window, prefix, gaps):
    """NaN scales and any codes in slots that no row sees, in the tiles that some row does."""
    sv = need_gpu()
    rng = np.random.default_rng(D + page + window)
    c, lens, cu, pos, hidden = hidden_case(rng, D, page, rows, window, prefix, gaps)
    assert any(len(h) for h in hidden)
    poison(rng, c, hidden)
    q = queries(rng, int(cu[-1]), 4, D, dtype)
    *_, status = check_attention(sv, c, q, cu, lens, rows - 1, window=window, prefix=prefix, slot_pos=pos)
    assert status == 0


@pytest.mark.parametrize("D,group,dtype", [(128, 12, "bf16"), (64, 16, "f32"), (256, 12, "bf16")])
@pytest.mark.parametrize("gaps", [False, True])
def test_what_hidden_slots_hold_over_many_columns(D, group, dtype, gaps):
    """32 rows in several column tiles, each with hidden slots of its own: what is NaN
    is hidden from all of them, what some row sees counts there."""
    sv = need_gpu()
    rng = np.random.default_rng(D + group)
    c, lens, cu, pos, hidden = hidden_case(rng, D, 32, 32, 20, 5, gaps)
    poison(rng, c, hidden)
    q = queries(rng, int(cu[-1]), 2 * group, D, dtype, 0.5)
    *_, status = check_attention(sv, c, q, cu, lens, 31, window=20, prefix=5, slot_pos=pos)
    assert status == 0


@pytest.mark.parametrize("rows,window,prefix,gaps", HIDDEN)
@pytest.mark.parametrize("page,dtype", [(32, "bf16"), (64, "f32"), (96, "bf16")])
def test_pages_that_the_window_hides_need_no_id(page, dtype, rows, window, prefix, gaps):
    """Pages of which no row sees a slot, given back: their entries name no page,
    nothing is reported, and the other slots count as before."""
    sv = need_gpu()
    rng = np.random.default_rng(page + window)
    c, lens, cu, pos, hidden = hidden_case(rng, 64, page, rows, window, prefix, gaps)
    q = queries(rng, int(cu[-1]), 4, 64, dtype)
    kw = dict(window=window, prefix=prefix, slot_pos=pos)
    out, tol, lse, lse_tol, w = exact_bounds(c, q, cu, lens, **kw)
    cut = ref.Cache(c.pages, c.table)
    gone = 0
    for b, slots in enumerate(hidden):
        for p in range(c.table.shape[1]):
            if len(slots) and np.isin(np.arange(p * page, (p + 1) * page), slots).all():
                cut.table[b, p] = (-1, c.n_pages, -2 ** 31)[p % 3]
                gone += 1
    assert gone
    res, score, status = run_attention(sv, cut, q, cu, lens, rows - 1, **kw)
    assert status == 0
    assert (np.abs(res["out"].float().cpu().numpy() - out) <= tol).all()
    assert (np.abs(res["lse"].cpu().numpy() - lse) <= lse_tol).all()
    got = score.cpu().numpy()
    for b, L in enumerate(lens):
        i = np.arange(L)
        ok = np.isin(i, hidden[b], invert=True)
        np.testing.assert_allclose(got[c.table[b, i // page], i % page][ok], w[b][ok], rtol=1e-4, atol=1e-30)


@pytest.mark.parametrize("gaps", [False, True])
def test_a_bad_page_among_the_visible_ones_is_reported(gaps):
    """... with a window too, and hides its own tokens alone."""
    sv = need_gpu()
    rng = np.random.default_rng(44)
    L, page, window = 2000, 32, 1200
    c = quick_pool(rng, B=1, H=1, D=64, page=page, lens=[L])
    pos = gapped_positions(rng, c) if gaps else None
    at = np.arange(L) if pos is None else pos[c.table[0, np.arange(L) // page], np.arange(L) % page].astype(np.int64)
    first = int(np.argmax(at > at[L - 1] - window))                 # the first visible slot
    q = queries(rng, 1, 2, 64, "f32")
    k, v = c.get(0, 0, np.arange(L))
    for p in (first // page + 1, (first + L) // 2 // page, L // page - 1):
        cut = ref.Cache(c.pages, c.table)
        cut.table[0, p] = -1
        cut.table[0, :first // page] = -1                            # given back, all of them
        res, _, status = run_attention(sv, cut, q, np.array([0, 1]), [L], 0, window=window, slot_pos=pos)
        assert status == 0x400
        see = (np.arange(L) >= first) & (np.arange(L) // page != p)
        for h in range(2):
            s = k[see] @ q[0, h].double().cpu().numpy() / 8
            e = np.exp(s - s.max())
            np.testing.assert_allclose(res["out"][0, h].cpu().numpy(), e @ v[see] / e.sum(), rtol=1e-4, atol=1e-4)


# ---------------------------------------------------------------------- read ---

def to_bf16(x):
    """x (64 bits, normal range) rounded once to bf16, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def test_read_rounds_once():
    """Head scales that put products of up to 30 bits within a rounding to fp32 of a
    tie of bf16: the values read are those of one rounding, all of them."""
    sv = need_gpu()
    rng = np.random.default_rng(45)
    codes = np.unique(np.outer(ref.E2M1[1:], ref.E4M3[0x30:0x40]))    # what code * scale can be
    g = []
    while len(g) < 64:
        a = rng.choice(codes)
        tie = (2 * int(rng.integers(128, 256)) + 1) / 512               # half way between two bf16 values
        x = np.float32(tie / a)
        near = np.float64(x) * a
        if near != tie and np.float64(np.float32(near)) == tie:
            g.append(x)
    g = np.array(g, np.float32)
    c = quick_pool(rng, B=1, H=64, D=64, page=32, lens=[256])
    live = rng.integers(0x30, 0x40, (c.n_pages, 64, 1, 2, 128), dtype=np.uint8)
    c.pages[..., 16 * 64:18 * 64], c.pages[..., 34 * 64:] = live[..., 0, :], live[..., 1, :]
    c.g = [g, g[::-1].copy()]
    cache, twice = gpu_cache(sv, c), 0
    args = (cache, dev(np.array([0, 256], np.int32)), dev(np.zeros(1, np.int32)), dev(c.table))
    got = sv.cache_read(*args, B=1, max_rows=256, dtype=torch.bfloat16)
    wide = sv.cache_read(*args, B=1, max_rows=256, dtype=torch.float32)
    for h in range(64):
        for name, x in zip("kv", c.get(0, h, np.arange(256))):
            np.testing.assert_array_equal(got[name][:, h].double().cpu().numpy(), to_bf16(x))
            np.testing.assert_array_equal(wide[name][:, h].cpu().numpy(), x.astype(np.float32))
            twice += (to_bf16(x.astype(np.float32).astype(np.float64)) != to_bf16(x)).sum()
    assert twice > 100                                               # (values that two roundings get wrong)


# ------------------------------------------------------------------ sharing ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_requests_that_share_pages_all_count(dtype):
    """48 requests behind one prompt: every one's weights arrive in its slots' scores."""
    sv = need_gpu()
    rng = np.random.default_rng(46)
    B, page, shared = 48, 64, 512
    lens = [shared + int(n) for n in rng.integers(2, 100, B)]
    c = quick_pool(rng, B=B, H=2, D=64, page=page, lens=lens)
    c.table[:, :shared // page] = c.table[0, :shared // page]
    cu = np.arange(0, 2 * B + 1, 2)
    q = queries(rng, 2 * B, 4, 64, dtype, 0.5)
    cache, tab = gpu_cache(sv, c), dev(c.table)
    cu_, ln = dev(cu.astype(np.int32)), dev(np.asarray(lens, np.int32))
    res = sv.cache_attend(cache, q, cu_, ln, tab, B=B, k_max=1)
    _, lse, _, S, w = ref.attention(c, q.float().cpu().numpy(), cu, lens)
    want = np.zeros((c.n_pages, page))
    for b, n in enumerate(lens):
        np.add.at(want, (c.table[b, np.arange(n) // page], np.arange(n) % page), w[b])
    u = 2.0 ** -24
    # of each weight as for pages of one's own, and a rounding for every request's addition
    rel = 2 * (64 * 2 * u + 4 * u) * S.max() + 4 * u * np.abs(lse).max() + 2.0 ** -18 + B * u
    for _ in range(10):
        score = torch.zeros(c.n_pages, page, device="cuda")
        sv.cache_weights(cache, q, res["lse"], cu_, ln, tab, score, B=B, k_max=1)
        assert (np.abs(score.cpu().numpy() - want) <= rel * want + 1e-30).all()


# ----------------------------------------------------------- rejected rows ---

@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0, window=50, prefix=2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_marked_by_an_infinite_lse_do_not_count(dtype, kw):
    """The weights of the other rows alone, whatever the marked ones would have added."""
    sv = need_gpu()
    rng = np.random.default_rng(47)
    lens, cu, took = [700, 33, 300], np.array([0, 4, 8, 12]), [1, 4, 2]
    c = quick_pool(rng, B=3, H=2, D=64, page=64, lens=lens)
    q = queries(rng, 12, 4, 64, dtype)
    cache, tab = gpu_cache(sv, c), dev(c.table)
    args = (dev(cu.astype(np.int32)), dev(np.asarray(lens, np.int32)), tab)
    lse = sv.cache_attend(cache, q, *args, B=3, k_max=3, **kw)["lse"]
    for b, n in enumerate(took):
        lse[cu[b] + n:cu[b + 1]] = float("-inf")
    score = torch.zeros(c.n_pages, 64, device="cuda")
    sv.cache_weights(cache, q, lse, *args, score, B=3, k_max=3, **kw)
    # the same rows by themselves: a cache that ends with the last one that stayed
    short = [L - (4 - n) for L, n in zip(lens, took)]
    rows = np.concatenate([np.arange(cu[b], cu[b] + n) for b, n in enumerate(took)])
    _, exact, _, S, w = ref.attention(c, q[rows].float().cpu().numpy(), np.concatenate([[0], np.cumsum(took)]), short, **kw)
    u = 2.0 ** -24
    rel = 2 * ((64 * 2 * u + 4 * u) * S.max() + kw.get("cap", 0) * 2.0 ** -20) + 4 * u * np.abs(exact).max() + 2.0 ** -18
    want = np.zeros((c.n_pages, 64))
    for b, n in enumerate(short):
        want[c.table[b, np.arange(n) // 64], np.arange(n) % 64] = w[b]
    assert (np.abs(score.cpu().numpy() - want) <= rel * want + 1e-30).all()


def test_the_example_leaves_rejected_rows_out(monkeypatch):
    """What examples/cached_step.py passes to the weights: -inf for the rows after the
    accepted prefix, a number for every other."""
    sv = need_gpu()
    from examples import cached_step
    seen = []
    verify, weights = sv.verify_greedy, sv.cache_weights

    def verified(*a, **kw):
        got = verify(*a, **kw)
        seen.append(got["accepted_len"].tolist())
        return got

    def weighed(cache, q, lse, *a, **kw):
        last = torch.isfinite(lse.view(8, 5, -1))
        for b, n in enumerate(seen[-1]):
            assert last[b, :n + 1].all() and not last[b, n + 1:].any()
        return weights(cache, q, lse, *a, **kw)

    monkeypatch.setattr(sv, "verify_greedy", verified)
    monkeypatch.setattr(sv, "cache_weights", weighed)
    cached_step.run(steps=6)
    assert len(seen) == 6


# ----------------------------------------------------------- long segments ---

@pytest.mark.parametrize("D,H,B,rows,group", [(128, 8, 64, 1, 1), (128, 4, 128, 5, 8), (64, 8, 64, 5, 8), (64, 8, 64, 1, 4),
                                              (256, 4, 128, 1, 1), (256, 4, 128, 3, 8)])
@pytest.mark.parametrize("louder,cap", [("none", 0.0), ("later", 0.0), ("earlier", 50.0)])
def test_long_sums_do_not_drift(D, H, B, rows, group, louder, cap):
    """More (request, kv head) pairs than blocks, each over half a million shared tokens
    with values of one sign: the outputs lie around the exact ones, not below them.
    `louder`: the half that scores far higher, the one visited last (a cap makes that
    the earlier one), so that references move behind the first sums.

    The mean error of N outputs, in half places of bf16, is that of N roundings
    (1 / sqrt(3 N), five of which are allowed) and of truncating a sum of 1024 steps:
    at each at most 2^-23 of the sum so far, half the whole on average, 2^-14 of the
    result and 2^-5 of a half place (2^-9 of it or more)."""
    sv = need_gpu()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(D + rows)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    n, page, step = 1 << 19, 256, 1 << 15
    cache = sv.new_cache(n // page, H, D, page, v_scale=1 + torch.rand(H, generator=gen, device="cuda"))
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").view(1, -1)
    mean = 0.5 + 1.5 * torch.rand(H, D, generator=gen, device="cuda")
    q = (0.5 * rand(B * rows, H * group, D)).bfloat16()
    last = q.view(B, rows, H, group, D)[:2, -1].double()              # of two requests the rows that see all
    num, den = torch.zeros(2, H, group, D, dtype=torch.double, device="cuda"), torch.zeros(2, H, group, dtype=torch.double, device="cuda")
    for at in range(0, n, step):
        loud = louder == ("later" if at >= n // 2 else "earlier")
        k, v = rand(step, H, D) * (4 if loud else 1), mean * (1 + 0.2 * rand(step, H, D))
        sv.cache_append(cache, k, v, i32([0, step]), i32([at]), table, B=1, max_rows=step)
        kv = sv.cache_read(cache, i32([0, step]), i32([at]), table, B=1, max_rows=step)
        p = torch.einsum("bhgd,nhd->bhgn", last, kv["k"].double()) / D ** 0.5
        p = torch.exp(cap * torch.tanh(p / cap) if cap else p)
        num += torch.einsum("bhgn,nhd->bhgd", p, kv["v"].double())
        den += p.sum(-1)
    want = num / den[..., None]
    cu = torch.arange(0, B * rows + 1, rows, dtype=torch.int32, device="cuda")
    got = sv.cache_attend(cache, q, cu, i32([n] * B), table.expand(B, -1).contiguous(), B=B, k_max=rows - 1,
                          cap=cap)
    out = got["out"].view(B, rows, H, group, D)[:2, -1].double()
    half = torch.exp2(torch.floor(torch.log2(want)) - 8)
    err = (out - want) / half
    assert abs(float(err.mean())) <= 2.0 ** -5 + 5 / (3 * err.numel()) ** 0.5, float(err.mean())
    lse = got["lse"].view(B, rows, H, group)[:2, -1].double()
    assert float((lse - torch.log(den)).abs().max()) <= 1e-4


# -------------------------------------------------- wide tables, large pages ---

@pytest.mark.parametrize("kw", [dict(), dict(window=100, prefix=5), dict(window=100, prefix=5, gaps=True)])
@pytest.mark.parametrize("page,dtype", [(32, "bf16"), (96, "f32"), (2048, "bf16"), (65536, "f32")])
def test_a_table_for_far_longer_contexts(page, dtype, kw):
    """Room for 131072 tokens and more, lengths up to 900: what the entries past a
    length hold does not matter, for attention, weights and eviction alike."""
    sv = need_gpu()
    kw = dict(kw)
    rng = np.random.default_rng(page)
    lens, cu = [900, 33, 1, 300, 129], np.array([0, 3, 6, 7, 10, 12])
    c = quick_pool(rng, B=5, H=2, D=64, page=page, lens=lens)
    if kw.pop("gaps", False):
        kw["slot_pos"] = gapped_positions(rng, c)
    exact = c.table
    wide = rng.integers(-2 ** 31, 2 ** 31, (5, 131072 // page + 3)).astype(np.int32)
    for b, n in enumerate(lens):
        used = -(-n // page)
        wide[b, :used] = exact[b, :used]
    c.table = wide
    q = queries(rng, 12, 4, 64, dtype, 0.5)
    *_, status = check_attention(sv, c, q, cu, lens, 2, **kw)
    assert status == 0
    budget, recent = 200, 16
    per = -(-budget // page)
    pool = np.concatenate([c.pages, np.zeros((5 * per, *c.pages.shape[1:]), np.uint8)])
    score = rng.exponential(1, (len(pool), page)).astype(np.float32)
    dst = np.arange(c.n_pages, len(pool)).reshape(5, per).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = sv.PagedCache(dev(pool))
    got = sv.cache_evict(cache, dev(score), dev(np.asarray(lens, np.int32)), dev(wide), dev(dst), B=5, budget=budget,
                         recent=recent, status=status)
    assert status.item() == 0
    after = ref.Cache(cache.pages.cpu().numpy(), dst)
    for b, n in enumerate(lens):
        i = np.arange(n)
        keep = ref.evict(score[wide[b, i // page], i % page], n, budget, recent)
        np.testing.assert_array_equal(got["kept"][b].cpu().numpy(), np.concatenate([keep, np.full(budget - len(keep), -1)]))
        for x, y in zip(after.get(b, 1, np.arange(len(keep))), c.get(b, 1, keep)):
            np.testing.assert_array_equal(x, y)


# --------------------------------------------------------- lengths in place ---

def test_eviction_can_update_the_lengths_in_place():
    """new_len in the place of len, with clusters of 8 blocks a request: kept, cut,
    and skipped requests alike, time and again."""
    import ctypes as C
    from speculative_decoding_verification_ragged_gb300.cache import _Eviction
    sv = need_gpu()
    rng = np.random.default_rng(48)
    page, budget, recent = 128, 6000, 64
    lens = [131072, 5000, 131072, 9000, -1, 100, 131072, 6000] * 4
    B, per, dper = len(lens), 1024, -(-budget // page)
    pages = torch.zeros(per + B * dper, 1, 4, 36 * 64, dtype=torch.uint8, device="cuda")
    score = dev(rng.exponential(1, (len(pages), page)).astype(np.float32))
    table = dev(np.tile(rng.permutation(per).astype(np.int32), (B, 1)))               # (read only: one prompt for all)
    dst = dev(np.arange(per, len(pages)).reshape(B, dper).astype(np.int32))
    cache = sv.PagedCache(pages)
    before = dev(np.asarray(lens, np.int32))
    want = sv.cache_evict(cache, score, before, table, dst, B=B, budget=budget, recent=recent)
    view = cache._view(table, B)
    for _ in range(10):
        ln, kept = before.clone(), torch.empty_like(want["kept"])
        ev = _Eviction(score.data_ptr(), None, ln.data_ptr(), budget, recent, dst.data_ptr(), dper, kept.data_ptr(),
                       ln.data_ptr(), None)
        assert sv.load_library().spec_cache_evict(C.byref(view), C.byref(ev), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(ln, want["new_len"]) and torch.equal(kept, want["kept"])
