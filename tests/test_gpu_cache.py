"""The 4-bit paged cache on the GPU against the 64-bit definitions in
tests/_cache_ref.py.

Tolerances, from the operations (u = 2^-24).  Codes, scales, moved bytes and
kept slots are exact.  A score is a sum of D exact products in fp32 (at most D
roundings or truncations, D * 2u * S with S = scale * sum |q k|), scaled (2
roundings), capped (tanh within 2^-21 absolute of 1, times cap) and biased (the
bias and the sum rounded once each):
    ds = D 2u S + 4u |s| + cap 2^-20 + 2u |bias|.
exp turns ds into a relative error ds (taken as 2 ds), its own within 2^-20 of
the weight.  A weight is rounded once to 11 bits for bf16 outputs (2^-11),
kept to 2^-20 for fp32; the weighted sum runs in fp32 over at most a few
thousand steps of one truncation each (2^-23 * steps of A, A = sum p |v|), and
a bf16 output is rounded once (2^-8 |o| covers half an ulp)."""
import numpy as np
import pytest

from tests import _cache_ref as ref
from tests._gpu import need_gpu

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dtype=None):
    x = torch.from_numpy(np.ascontiguousarray(a))
    return (x if dtype is None else x.to(dtype)).cuda()


def make_pool(rng, *, B, H, D, page, lens, scaled=False, spare=3):
    """A pool of random bytes (NaN scales among them) whose slots below each
    request's length hold quantised normal rows."""
    per = max(1, -(-max(max(lens), 1) // page))
    n = B * per + spare
    pages = rng.integers(0, 256, (n, H, page // 32, 36 * D), dtype=np.uint8)
    table = rng.permutation(n)[:B * per].reshape(B, per).astype(np.int32)
    g = [rng.uniform(0.05, 2.0, H).astype(np.float32) if scaled else None for _ in range(2)]
    c = ref.Cache(pages, table, *g)
    return c


def fill(sv, c, rng, lens, *, start=None, dtype="f32"):
    """Append rows through the library, and with the reference: both pools."""
    B = len(lens)
    start = [0] * B if start is None else start
    n = [a - s for a, s in zip(lens, start)]
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    R = max(int(cu[-1]), 1)
    k = torch.from_numpy(rng.standard_normal((R, c.H, c.D)).astype(np.float32)).to(DT[dtype])
    v = torch.from_numpy(rng.standard_normal((R, c.H, c.D)).astype(np.float32)).to(DT[dtype])
    cache = gpu_cache(sv, c)
    sv.cache_append(cache, k.cuda(), v.cuda(), dev(cu), dev(np.asarray(start, np.int32)), dev(c.table), B=B,
                    max_rows=max(max(n), 1))
    kn, vn = k.float().numpy(), v.float().numpy()
    for b in range(B):
        for i in range(n[b]):
            for h in range(c.H):
                c.put(b, h, start[b] + i, kn[cu[b] + i, h], vn[cu[b] + i, h])
    return cache, k, v, cu


def gpu_cache(sv, c):
    ks, vs = (None if (g == 1).all() else dev(g) for g in c.g)
    return sv.PagedCache(dev(c.pages), k_scale=ks, v_scale=vs)


def quick_pool(rng, *, B, H, D, page, lens, scaled=False):
    """A pool filled by the reference's quantiser in one go (no per-token loop):
    random codes and moderate scales below each length, garbage above."""
    c = make_pool(rng, B=B, H=H, D=D, page=page, lens=lens, scaled=scaled)
    live = np.zeros((c.n_pages, page), bool)
    for b, n in enumerate(lens):
        i = np.arange(n)
        live[c.table[b, i // page], i % page] = True
    live = live.reshape(c.n_pages, 1, page // 32, 32)
    sc = rng.integers(0x20, 0x34, c.pages.shape[:3] + (2, 32, D // 16), dtype=np.uint8)   # 2^-3 .. 1.5
    ks = c.pages[..., 16 * D:18 * D].reshape(*c.pages.shape[:3], 32, D // 16)
    ks[...] = np.where(live[..., None], sc[..., 0, :, :], ks)
    vs = c.pages[..., 34 * D:].reshape(*c.pages.shape[:3], D // 16, 32)
    vs[...] = np.where(live[..., None, :], sc[..., 1, :, :].swapaxes(-1, -2), vs)
    return c


def run_attention(sv, c, q, cu, lens, k_max, *, slopes=None, slot_pos=None, **kw):
    cache = gpu_cache(sv, c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    opt = dict(B=len(lens), k_max=k_max, status=status, slopes=None if slopes is None else dev(slopes),
               slot_pos=None if slot_pos is None else dev(slot_pos), **kw)
    cu_, len_, tab = dev(np.asarray(cu, np.int32)), dev(np.asarray(lens, np.int32)), dev(c.table)
    res = sv.cache_attend(cache, q, cu_, len_, tab, **opt)
    score = torch.zeros(c.n_pages, c.page, device="cuda")
    sv.cache_weights(cache, q, res["lse"], cu_, len_, tab, score, **opt)
    torch.cuda.synchronize()
    return res, score, int(status.item())


def check_attention(sv, c, q, cu, lens, k_max, **kw):
    """Outputs, lse and weights of every row against the definition."""
    res, score, status = run_attention(sv, c, q, cu, lens, k_max, **kw)
    R = int(cu[-1])
    out, lse, A, S, w = ref.attention(c, q[:R].float().cpu().numpy(), cu, lens, **kw)
    u, D, cap = 2.0 ** -24, c.D, kw.get("cap", 0.0)
    bias = 0.0
    if kw.get("slopes") is not None:
        far = c.page * c.table.shape[1] if kw.get("slot_pos") is None else int(np.max(kw["slot_pos"]))
        bias = float(np.max(np.abs(kw["slopes"]))) * far
    ds = (D * 2 * u + 4 * u) * S + cap * 2.0 ** -20 + 2 * u * bias                  # [R, Hq]
    rel = 2 * ds + 2.0 ** -20 + 2.0 ** -23 * (max(lens) / 16 + 16)
    bf = q.dtype == torch.bfloat16
    tol = A * (rel + (2.0 ** -11 if bf else 2.0 ** -20))[..., None] + (2.0 ** -8 * np.abs(out) if bf else 0)
    got = res["out"][:R].float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    bad = np.abs(got - out) > tol + 1e-30
    assert not bad.any(), (np.abs(got - out)[bad][:5], tol[bad][:5], np.argwhere(bad)[:5])
    gl = res["lse"][:R].cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isinf(gl), np.isinf(lse))
    fin = np.isfinite(lse)
    assert (np.abs(gl - lse)[fin] <= (ds + 4 * u * np.abs(lse) + 2.0 ** -19)[fin]).all()
    sc = score.cpu().numpy().astype(np.float64)
    seen = np.zeros_like(sc, bool)
    worst = float((2 * ds + 4 * u * np.where(fin, np.abs(lse), 0)).max(initial=0)) + 2.0 ** -18
    for b, n in enumerate(lens):
        i = np.arange(n)
        at = (c.table[b, i // c.page], i % c.page)
        seen[at] = True
        assert (np.abs(sc[at] - w[b]) <= worst * w[b] + 1e-30).all(), b
    assert (sc[~seen] == 0).all()
    return res, score, status


def queries(rng, R, Hq, D, dtype, gain=1.0):
    return torch.from_numpy((gain * rng.standard_normal((R, Hq, D))).astype(np.float32)).to(DT[dtype]).cuda()


# ------------------------------------------------------------ append, read ---

@pytest.mark.parametrize("D,page,dtype,scaled", [(64, 32, "f32", True), (128, 64, "bf16", False),
                                                 (256, 96, "bf16", True), (128, 128, "f32", False)])
def test_append_writes_the_defined_bytes(D, page, dtype, scaled):
    """Every byte of the pool, other slots' included, after two appends: whole
    blocks, then ragged rows starting inside a byte, a block and a page."""
    sv = need_gpu()
    rng = np.random.default_rng(D + page)
    lens0, lens1 = [33, 0, 31, 64, 1, 97], [38, 1, 33, 64, 70, 129]
    c = make_pool(rng, B=6, H=3, D=D, page=page, lens=lens1, scaled=scaled)
    cache, *_ = fill(sv, c, rng, lens0, dtype=dtype)
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), c.pages)
    cache, k, v, cu = fill(sv, c, rng, lens1, start=lens0, dtype=dtype)
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), c.pages)
    got = sv.cache_read(cache, dev(cu), dev(np.asarray(lens0, np.int32)), dev(c.table), B=6, max_rows=80,
                        R_cap=int(cu[-1]), dtype=DT[dtype])
    for b in range(6):
        slots = np.arange(lens0[b], lens1[b])
        for h in range(3):
            want = c.get(b, h, slots)
            for name, x in zip("kv", want):
                # code * scale is exact, the head scale and the type round it once each
                exp = torch.from_numpy(x).float().to(DT[dtype]).float().numpy() if not scaled else x
                g = got[name][cu[b]:cu[b + 1], h].float().cpu().numpy()
                np.testing.assert_allclose(g, exp, rtol=0 if not scaled else (2.0 ** -8 if dtype == "bf16" else 2.0 ** -23))


def test_append_extremes_and_ties():
    """Zeros, subnormals, values beyond the largest scale, and exact ties of both roundings."""
    sv = need_gpu()
    rng = np.random.default_rng(5)
    c = make_pool(rng, B=1, H=1, D=64, page=32, lens=[8])
    x = np.zeros((8, 1, 64), np.float32)
    x[1] = np.float32(1e-42)
    x[2] = 1e6
    x[3] = -1e30
    x[4, 0, ::2], x[4, 0, 1::2] = -0.0, 6 * 2.0 ** -9
    x[5] = np.tile([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0], 4)
    x[6] = np.tile([6 * (1 + 1 / 16), 1, 2, 3] * 4, 4)             # scale half way between two e4m3 values
    x[7] = np.tile([6 * 2.0 ** -10, 0, 0, 0] * 4, 4)               # half the smallest scale: ties to zero
    for i in range(8):
        c.put(0, 0, i, x[i, 0], x[i, 0])
    before = make_pool(np.random.default_rng(5), B=1, H=1, D=64, page=32, lens=[8])
    cache = gpu_cache(sv, before)
    sv.cache_append(cache, dev(x), dev(x), dev(np.array([0, 8], np.int32)), dev(np.zeros(1, np.int32)), dev(c.table), B=1, max_rows=8)
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), c.pages)


@pytest.mark.parametrize("exponent", [-42, -20, 0, 17, 40])
def test_append_rounds_every_quotient_as_ieee(exponent):
    """Two million values of one magnitude range, some a last place away from where
    the code changes, with head scales over the whole range of fp32."""
    sv = need_gpu()
    rng = np.random.default_rng(exponent + 100)
    n, H = 4096, 4
    c = ref.Cache(np.zeros((n // 32, H, 1, 36 * 64), np.uint8), np.arange(n // 32, dtype=np.int32)[None],
                  *[(rng.uniform(0.5, 2, H) * 10.0 ** np.array([0, -30, 25, -44])).astype(np.float32) for _ in range(2)])
    xs = []
    for g in c.g:
        x = rng.standard_normal((n, H, 64)) * 2.0 ** rng.integers(-3, 4, (n, H, 64)) * 2.0 ** exponent
        x = (x * g[:, None]).astype(np.float32)
        # near the places where a code changes, for the scale that the block will have
        s = quantised_scale(x, g)
        edge = rng.choice(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32), x.shape)
        near = np.nextafter((edge * s).astype(np.float32), np.float32(rng.choice([-np.inf, np.inf])))
        pick = (rng.random(x.shape) < 0.5) & (np.abs(near) < np.abs(x).reshape(n, H, 4, 16).max(-1).repeat(16, -1))
        xs.append(np.where(pick, near, x).astype(np.float32))
    cache = gpu_cache(sv, c)
    sv.cache_append(cache, dev(xs[0]), dev(xs[1]), dev(np.array([0, n], np.int32)), dev(np.zeros(1, np.int32)), dev(c.table),
                    B=1, max_rows=n)
    got = cache.pages.cpu().numpy()
    for h in range(H):
        kc, ks = ref.quantise(xs[0][:, h], c.g[0][h])
        vc, vs = ref.quantise(xs[1][:, h], c.g[1][h])
        blk = got[:, h, 0]                                              # [blocks, 36 * 64]
        k = blk[:, :1024].reshape(-1, 2, 32, 16).transpose(0, 2, 1, 3).reshape(n, 32)
        np.testing.assert_array_equal(k, kc[:, 0::2] | kc[:, 1::2] << 4)
        np.testing.assert_array_equal(blk[:, 1024:1152].reshape(n, 4), ks)
        v = blk[:, 1152:2176].reshape(-1, 64, 16).transpose(0, 2, 1)
        want = vc.reshape(-1, 32, 64)
        np.testing.assert_array_equal(v, want[:, 0::2] | want[:, 1::2] << 4)
        np.testing.assert_array_equal(blk[:, 2176:].reshape(-1, 4, 32).transpose(0, 2, 1).reshape(n, 4), vs)


def quantised_scale(x, g):
    """code scale * head scale of every value's block, as the definition takes it"""
    out = np.zeros_like(x)
    for h in range(x.shape[1]):
        _, s = ref.quantise(x[:, h], g[h])
        out[:, h] = (ref.E4M3[s].astype(np.float32) * g[h]).repeat(16, -1)
    return out


def test_append_strided_rows_scores_and_positions():
    """k and v as slices of one projection (unaligned heads), scores zeroed and positions written."""
    sv = need_gpu()
    rng = np.random.default_rng(6)
    c = make_pool(rng, B=2, H=2, D=64, page=32, lens=[40, 7])
    c.pages[...] = 0
    qkv = torch.from_numpy(rng.standard_normal((47, 4 * 64 + 3)).astype(np.float32)).cuda()
    k, v = (qkv[:, 3 + 128 * i:3 + 128 * (i + 1)].unflatten(1, (2, 64)) for i in range(2))
    cache, cu = gpu_cache(sv, c), dev(np.array([0, 40, 47], np.int32))
    score = torch.ones(c.n_pages, 32, device="cuda")
    pos = torch.full((c.n_pages, 32), -7, dtype=torch.int32, device="cuda")
    sv.cache_append(cache, k, v, cu, dev(np.zeros(2, np.int32)), dev(c.table), B=2, max_rows=40, score=score,
                    slot_pos=pos, pos0=dev(np.array([100, 5], np.int32)))
    for b, (lo, n) in enumerate([(0, 40), (40, 7)]):
        for i in range(n):
            for h in range(2):
                c.put(b, h, i, k[lo + i, h].cpu().numpy(), v[lo + i, h].cpu().numpy())
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), c.pages)
    want_s, want_p = np.ones((c.n_pages, 32), np.float32), np.full((c.n_pages, 32), -7)
    for b, n, p0 in [(0, 40, 100), (1, 7, 5)]:
        i = np.arange(n)
        want_s[c.table[b, i // 32], i % 32] = 0
        want_p[c.table[b, i // 32], i % 32] = p0 + i
    np.testing.assert_array_equal(score.cpu().numpy(), want_s)
    np.testing.assert_array_equal(pos.cpu().numpy(), want_p)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_read_into_strided_unaligned_rows(dtype):
    """The C call with strides and bases that allow no wide stores: the values
    of the aligned call, and nothing between the rows touched."""
    import ctypes as C
    from speculative_decoding_verification_ragged_gb300.cache import _Rows
    sv = need_gpu()
    rng = np.random.default_rng(8)
    c = quick_pool(rng, B=1, H=2, D=64, page=32, lens=[45])
    cache, tab = gpu_cache(sv, c), dev(c.table)
    cu, start = dev(np.array([0, 40], np.int32)), dev(np.array([5], np.int32))
    want = sv.cache_read(cache, cu, start, tab, B=1, max_rows=40, dtype=DT[dtype])
    wide = [torch.full((40, 2 * 67 + 1), 7.0, device="cuda", dtype=DT[dtype]) for _ in range(2)]
    view = cache._view(tab, 1)
    at = [w.data_ptr() + w.element_size() for w in wide]
    rows = _Rows(at[0], at[1], 1 if dtype == "bf16" else 0, 135, 67, 135, 67, 40, 40, cu.data_ptr(), start.data_ptr())
    assert sv.load_library().spec_cache_read(C.byref(view), C.byref(rows), None) == 0
    torch.cuda.synchronize()
    for w, x in zip(wide, (want["k"], want["v"])):
        for h in range(2):
            assert torch.equal(w[:, 1 + 67 * h:65 + 67 * h], x[:, h])
            w[:, 1 + 67 * h:65 + 67 * h] = 7.0
        assert (w == 7.0).all()


def test_append_and_read_skip_bad_requests():
    sv = need_gpu()
    rng = np.random.default_rng(7)
    c = make_pool(rng, B=4, H=1, D=64, page=32, lens=[64] * 4)
    c.table[1, 0] = c.n_pages                                        # bad page
    cache = gpu_cache(sv, c)
    x = dev(rng.standard_normal((20, 1, 64)).astype(np.float32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, start = np.array([0, 5, 10, 15, 20], np.int32), np.array([0, 30, 60, -1], np.int32)   # 60 + 5 > 64
    sv.cache_append(cache, x, x, dev(cu), dev(start), dev(c.table), B=4, max_rows=5, status=status)
    xn = x.cpu().numpy()
    for i in range(5):
        c.put(0, 0, i, xn[i, 0], xn[i, 0])
        if i >= 2:                                                   # slots 32.. lie on a good page
            c.put(1, 0, 30 + i, xn[5 + i, 0], xn[5 + i, 0])
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), c.pages)
    assert status.item() == 0x400 | 0x800
    status.zero_()
    got = sv.cache_read(cache, dev(cu), dev(start), dev(c.table), B=4, max_rows=5, R_cap=20, status=status)
    assert status.item() == 0x400 | 0x800
    assert (got["k"][5:7] == 0).all() and (got["v"][5:7] == 0).all()
    np.testing.assert_allclose(got["k"][7:10, 0].cpu().numpy(), c.get(1, 0, [32, 33, 34])[0], rtol=2.0 ** -23)
    status.zero_()
    pages = cache.pages.clone()
    sv.cache_append(cache, x, x, dev(np.array([0, 6, 3, 8, 30], np.int32)), dev(np.zeros(4, np.int32)), dev(c.table),
                    B=4, max_rows=4, status=status)                  # 6 > max_rows, < 0, 5 > max_rows, beyond R_cap
    assert status.item() == 0x10 and torch.equal(pages, cache.pages)


# ------------------------------------------------------------------ attend ---

LENS = [1, 5, 31, 32, 33, 96, 127, 128, 129, 300, 641, 7]


@pytest.mark.parametrize("D,H,group,rows,page,dtype", [
    (64, 2, 1, 1, 32, "bf16"), (64, 1, 8, 8, 96, "f32"), (64, 3, 5, 3, 64, "bf16"),
    (128, 2, 5, 5, 64, "bf16"), (128, 1, 3, 32, 32, "f32"), (128, 2, 1, 1, 128, "f32"),
    (128, 1, 16, 5, 256, "bf16"), (256, 1, 8, 3, 96, "bf16"), (256, 2, 4, 2, 32, "f32"), (256, 1, 1, 1, 64, "bf16")])
@pytest.mark.parametrize("scaled", [False, True])
def test_attention_over_ragged_lengths(D, H, group, rows, page, dtype, scaled):
    sv = need_gpu()
    rng = np.random.default_rng(D * 7 + rows + group)
    n = [min(max(1, rows - (5 * b) % 3), LENS[b]) for b in range(len(LENS))]
    cu = np.concatenate([[0], np.cumsum(n)])
    c = quick_pool(rng, B=len(LENS), H=H, D=D, page=page, lens=LENS, scaled=scaled)
    q = queries(rng, int(cu[-1]) + 2, H * group, D, dtype, 0.5)
    *_, status = check_attention(sv, c, q, cu, LENS, rows - 1)
    assert status == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(cap=20.0), dict(window=1), dict(window=40, prefix=3), dict(slopes=True),
                                dict(cap=30.0, slopes=True, window=150, prefix=2, gaps=True),
                                dict(window=33, prefix=700), dict(scale=-0.3), dict(scale=0.0), dict(window=2, gaps=True)])
def test_attention_score_options(kw, D, dtype):
    sv = need_gpu()
    kw = dict(kw)
    rng = np.random.default_rng(len(str(kw)) + D)
    n = [min(4, x) for x in LENS]
    cu = np.concatenate([[0], np.cumsum(n)])
    c = quick_pool(rng, B=len(LENS), H=2, D=D, page=64, lens=LENS)
    if kw.pop("slopes", False):
        kw["slopes"] = (2.0 ** -np.arange(1, 7)).astype(np.float32)
    if kw.pop("gaps", False):
        pos = np.zeros((c.n_pages, 64), np.int32)
        for b in range(len(LENS)):
            pos[c.table[b]] = (np.cumsum(rng.integers(1, 4, c.table.shape[1] * 64)) - 1).reshape(-1, 64)
        kw["slot_pos"] = pos
    q = queries(rng, int(cu[-1]), 6, D, dtype, 2.0)
    *_, status = check_attention(sv, c, q, cu, LENS, 3, **kw)
    assert status == 0


@pytest.mark.parametrize("D,dtype,rows,group", [(128, "bf16", 1, 4), (128, "bf16", 5, 5), (64, "f32", 2, 4), (256, "bf16", 3, 8)])
def test_attention_long_caches(D, dtype, rows, group):
    """Lengths over which the work is split and joined, with a peaked and a flat row among them."""
    sv = need_gpu()
    rng = np.random.default_rng(D + rows)
    lens = [20000, 4097, 3, 9000]
    c = quick_pool(rng, B=4, H=1, D=D, page=128, lens=lens)
    cu = np.arange(0, 4 * rows + 1, rows)
    lens[2] = max(lens[2], rows)
    q = queries(rng, 4 * rows, group, D, dtype)
    q[0] = 0
    q[rows] *= 16
    check_attention(sv, c, q, cu, lens, rows - 1)


@pytest.mark.parametrize("D,group,rows,dtype", [(64, 8, 8, "bf16"), (128, 8, 8, "bf16"), (128, 12, 32, "bf16"), (64, 16, 32, "f32")])
def test_attention_many_columns(D, group, rows, dtype):
    """64 columns of one kv head, and several column tiles of them."""
    sv = need_gpu()
    rng = np.random.default_rng(D + group)
    lens = [700, 40, 129, 33]
    cu = np.concatenate([[0], np.cumsum([rows, rows, 1, rows])])
    c = quick_pool(rng, B=4, H=1, D=D, page=64, lens=lens)
    check_attention(sv, c, queries(rng, int(cu[-1]), group, D, dtype, 0.5), cu, lens, rows - 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_over_many_requests(dtype):
    """More requests than a block has threads, empty ones, ones without rows and
    malformed ones among them."""
    sv = need_gpu()
    rng = np.random.default_rng(15)
    B = 1100
    lens = rng.integers(0, 90, B)
    lens[5], lens[901] = 3000, 1500
    n = rng.integers(0, 4, B)
    n[::7] = 0
    cu = np.concatenate([[0], np.cumsum(n)])
    c = quick_pool(rng, B=B, H=1, D=64, page=32, lens=list(lens))
    q = queries(rng, int(cu[-1]), 2, 64, dtype)
    check_attention(sv, c, q, cu, [int(x) for x in lens], 3)
    # with k_max = 0 the requests of several rows are malformed, and skipped
    res, _, status = run_attention(sv, c, q, cu, [int(x) for x in lens], int(n.max()) - 1)
    wide, _, status_w = run_attention(sv, c, q, cu, [int(x) for x in lens], 0)
    assert status == 0 and status_w == 0x10
    one = np.nonzero(n == 1)[0]
    for b in one[::9]:
        assert torch.equal(res["out"][cu[b]], wide["out"][cu[b]])


def test_a_workspace_serves_calls_of_different_shapes():
    sv = need_gpu()
    rng = np.random.default_rng(16)
    lens = [5000, 900, 3100, 70]
    c = quick_pool(rng, B=4, H=2, D=128, page=64, lens=lens)
    cache, tab, ln = gpu_cache(sv, c), dev(c.table), dev(np.asarray(lens, np.int32))
    shapes = [(4, 5, 10), (1, 1, 2), (3, 2, 8), (4, 1, 32), (2, 8, 16)]
    ws = torch.zeros(max(sv.cache_workspace_bytes(b, r - 1, hq, 2, 128, tab.shape[1] * 64) for b, r, hq in shapes),
                     dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for b, r, hq in shapes:
            q = queries(rng, b * r, hq, 128, "bf16")
            cu = dev(np.arange(0, b * r + 1, r).astype(np.int32))
            got = sv.cache_attend(cache, q, cu, ln, tab, B=b, k_max=r - 1, workspace=ws)
            want = sv.cache_attend(cache, q, cu, ln, tab, B=b, k_max=r - 1)
            assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("n,budget,recent", [(30000, 10000, 100), (70000, 69999, 0), (131072, 5, 2), (400001, 100000, 1000)])
def test_evict_from_long_caches(n, budget, recent):
    """Clusters of every size, and more scores than stay on chip."""
    sv = need_gpu()
    rng = np.random.default_rng(n)
    per = -(-n // 128)
    pages = torch.randint(0, 120, (per + -(-budget // 128), 1, 4, 36 * 64), dtype=torch.uint8, device="cuda")
    score = rng.exponential(1, (len(pages), 128)).astype(np.float32).round(3)
    table = rng.permutation(per).astype(np.int32)[None]
    dst = np.arange(per, len(pages), dtype=np.int32)[None]
    s = dev(score)
    got = sv.cache_evict(sv.PagedCache(pages), s, dev(np.array([n], np.int32)), dev(table), dev(dst), B=1, budget=budget,
                         recent=recent)
    i = np.arange(n)
    keep = ref.evict(score[table[0, i // 128], i % 128], n, budget, recent)
    np.testing.assert_array_equal(got["kept"].cpu().numpy()[0], keep)
    np.testing.assert_array_equal(s.cpu().numpy()[dst[0]].reshape(-1)[:budget], score[table[0, keep // 128], keep % 128])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rows_that_see_nothing(dtype):
    """len 0, len < rows, rows of zero length, a bad length, bad rows, a bad page."""
    sv = need_gpu()
    rng = np.random.default_rng(11)
    lens = [0, 2, 70, 40, 64, 50]
    cu = np.array([0, 3, 8, 8, 10, 12, 14])
    c = quick_pool(rng, B=6, H=1, D=64, page=32, lens=lens)
    q = queries(rng, 14, 3, 64, dtype)
    check_attention(sv, c, q, cu, lens, 4)
    # bad length: nothing seen; a bad page: its tokens hidden
    bad = list(lens)
    bad[3], bad[5] = 10 ** 6, -3
    hidden = ref.Cache(c.pages, c.table)
    hidden.table[4, 1] = -1
    res, score, status = run_attention(sv, hidden, q, cu, bad, 4)
    assert status == 0x400 | 0x800
    out, lse, *_ = ref.attention(c, q.float().cpu().numpy(), cu, lens)
    o = res["out"].float().cpu().numpy()
    assert (o[8:10] == 0).all() and (o[12:] == 0).all()
    assert torch.isinf(res["lse"][8:10]).all() and torch.isinf(res["lse"][12:]).all()
    short = ref.Cache(c.pages, c.table[4:5])
    k, v = short.get(0, 0, np.arange(32))
    for j in range(2):
        for h in range(3):
            s = k @ q[10 + j, h].double().cpu().numpy() / 8
            p = np.exp(s - s.max())
            np.testing.assert_allclose(o[10 + j, h], p @ v / p.sum(), atol=2.0 ** -7)
    # rows outside the batch leave every output of that request alone
    cu_bad = np.array([0, 3, 8, 8, 10, 12, 99])
    res, score, status = run_attention(sv, c, q, cu_bad, lens, 4)
    assert status == 0x10
    np.testing.assert_array_equal(res["lse"][:3].cpu().numpy(), -np.inf)
    np.testing.assert_allclose(res["lse"][3:12].cpu().numpy(), lse[3:12], rtol=1e-4)


def test_attention_is_deterministic_and_reuses_its_workspace():
    sv = need_gpu()
    rng = np.random.default_rng(12)
    lens = [6000, 17, 2500]
    c = quick_pool(rng, B=3, H=2, D=128, page=64, lens=lens)
    q = queries(rng, 9, 10, 128, "bf16")
    cache, tab = gpu_cache(sv, c), dev(c.table)
    cu, ln = dev(np.array([0, 3, 6, 9], np.int32)), dev(np.asarray(lens, np.int32))
    ws = sv.new_cache_workspace(cache, tab, B=3, k_max=2, Hq=10)
    call = sv.cache_attend(cache, q, cu, ln, tab, B=3, k_max=2, workspace=ws, prepared=True)
    first = {k: x.clone() for k, x in call().items()}
    side = torch.cuda.Stream()
    for i in range(20):
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            got = call()
        torch.cuda.default_stream().wait_stream(side)
        assert all(torch.equal(first[k], got[k]) for k in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    got["out"].zero_()
    graph.replay()
    assert all(torch.equal(first[k], got[k]) for k in first)


@pytest.mark.parametrize("gain", [0.01, 0.1, 1.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_small_scores_under_a_large_cap(dtype, gain):
    """The cap's error is relative to the score (2^-20 of it), not to the cap."""
    sv = need_gpu()
    rng = np.random.default_rng(23)
    lens, cu = [700, 33, 129, 1], np.array([0, 2, 4, 6, 7])
    c = quick_pool(rng, B=4, H=2, D=128, page=64, lens=lens)
    q = queries(rng, 7, 8, 128, dtype, gain)
    kw = dict(cap=500.0, scale=0.01)
    res, _, status = run_attention(sv, c, q, cu, lens, 1, **kw)
    assert status == 0
    _, lse, _, S, _ = ref.attention(c, q.float().cpu().numpy(), cu, lens, **kw)
    u = 2.0 ** -24
    tol = (c.D * 2 * u + 4 * u + 2.0 ** -20) * S + 4 * u * np.abs(lse) + 2.0 ** -19
    assert (np.abs(res["lse"].cpu().numpy().astype(np.float64) - lse) <= tol).all()


@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0, window=300, prefix=2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_with_nan_and_infinite_queries_ends(dtype, kw):
    """The call returns, without a timeout, and the other requests keep their results."""
    sv = need_gpu()
    rng = np.random.default_rng(17)
    lens, cu = [700, 300, 129, 2000], np.array([0, 2, 4, 6, 8])
    c = quick_pool(rng, B=4, H=2, D=128, page=64, lens=lens)
    q = queries(rng, 8, 8, 128, dtype)
    clean, _, status = run_attention(sv, c, q, cu, lens, 1, **kw)
    assert status == 0
    for poison in (float("nan"), float("inf"), -float("inf")):
        bad = q.clone()
        bad[2, 1, 5] = poison
        bad[7] = poison
        got, _, status = run_attention(sv, c, bad, cu, lens, 1, **kw)
        assert status == 0
        for r in (0, 1, 4, 5):
            assert torch.equal(got["out"][r], clean["out"][r]) and torch.equal(got["lse"][r], clean["lse"][r])


def test_attention_strided_queries():
    """q as a slice of a fused projection, at an odd element offset."""
    sv = need_gpu()
    rng = np.random.default_rng(13)
    lens, cu = [200, 33], np.array([0, 2, 5])
    c = quick_pool(rng, B=2, H=2, D=64, page=32, lens=lens)
    for dtype in ("bf16", "f32"):
        wide = queries(rng, 5, 7, 128, dtype)
        q = wide.view(5, -1)[:, 1:1 + 6 * 128].unflatten(1, (6, 128))[:, :, 3:67]
        got, *_ = run_attention(sv, c, q, cu, lens, 2)
        want, *_ = run_attention(sv, c, q.contiguous(), cu, lens, 2)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_offsets_beyond_4_gib():
    """Pages whose byte offsets pass 2^32: appended, read, attended, evicted."""
    sv = need_gpu()
    rng = np.random.default_rng(14)
    n_pages = 8100
    pages = torch.empty(n_pages, 8, 8, 36 * 256, dtype=torch.uint8, device="cuda")           # 4.78 GB
    cache = sv.PagedCache(pages)
    tab = dev(np.array([[8099, 3]], np.int32))
    x = dev(rng.standard_normal((300, 8, 256)).astype(np.float32))
    cu, zero = dev(np.array([0, 300], np.int32)), dev(np.zeros(1, np.int32))
    sv.cache_append(cache, x, x, cu, zero, tab, B=1, max_rows=300)
    got = sv.cache_read(cache, cu, zero, tab, B=1, max_rows=300)
    assert torch.equal(got["k"], got["v"])
    assert float((got["k"] - x).norm() / x.norm()) < 0.2            # 4 bits: a sixth of the block's largest
    small = ref.Cache(pages[tab[0].long()].cpu().numpy(), np.array([[0, 1]], np.int32))
    q = queries(rng, 2, 8, 256, "bf16")
    res = sv.cache_attend(cache, q, dev(np.array([0, 2], np.int32)), dev(np.array([300], np.int32)), tab, B=1, k_max=1)
    out, lse, A, *_ = ref.attention(small, q.float().cpu().numpy(), np.array([0, 2]), [300])
    assert (np.abs(res["out"].float().cpu().numpy() - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -10 * A).all()
    score = torch.zeros(n_pages, 256, device="cuda")
    score[8099, 7:47] = 1
    got = sv.cache_evict(cache, score, dev(np.array([300], np.int32)), tab, dev(np.array([[8098]], np.int32)), B=1, budget=60, recent=20)
    want = np.concatenate([np.arange(7, 47), np.arange(280, 300)])
    np.testing.assert_array_equal(got["kept"].cpu().numpy()[0], want)
    moved = sv.cache_read(cache, dev(np.array([0, 60], np.int32)), zero, dev(np.array([[8098]], np.int32)), B=1, max_rows=60)
    back = sv.cache_read(cache, cu, zero, tab, B=1, max_rows=300)
    assert torch.equal(moved["k"], back["k"][torch.from_numpy(want).cuda()])


# ------------------------------------------------------------------- evict ---

@pytest.mark.parametrize("D,page,lens,budget,recent", [
    (64, 32, [100, 64, 65, 1, 0, 33], 64, 10), (128, 64, [5000, 3000, 2049], 2048, 64), (256, 96, [400, 7], 1, 0),
    (64, 32, [90, 40], 37, 37), (128, 128, [20001], 777, 0), (64, 64, [300, 299], 299, 5)])
@pytest.mark.parametrize("kind", ["weights", "ties", "wild"])
def test_evict_keeps_the_defined_slots(D, page, lens, budget, recent, kind):
    sv = need_gpu()
    rng = np.random.default_rng(D + budget)
    B, H = len(lens), 2
    c = quick_pool(rng, B=B, H=H, D=D, page=page, lens=lens)
    dper = -(-min(budget, c.table.shape[1] * page) // page)
    dst = (c.n_pages + rng.permutation(B * dper)).reshape(B, dper).astype(np.int32)
    pool = np.concatenate([c.pages, rng.integers(0, 256, (B * dper, *c.pages.shape[1:]), dtype=np.uint8)])
    if kind == "weights":
        score = rng.exponential(1, (len(pool), page)).astype(np.float32) ** 3
    elif kind == "ties":
        score = rng.integers(0, 3, (len(pool), page)).astype(np.float32)
    else:
        score = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1.0, 3.4e38, 1.0, 2.0], np.float32), (len(pool), page))
    pos = rng.integers(0, 10 ** 6, (len(pool), page)).astype(np.int32)
    cache, s, p = sv.PagedCache(dev(pool)), dev(score), dev(pos)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sv.cache_evict(cache, s, dev(np.asarray(lens, np.int32)), dev(c.table), dev(dst), B=B, budget=budget,
                         recent=recent, slot_pos=p, status=status)
    kept, pages = got["kept"].cpu().numpy(), cache.pages.cpu().numpy()
    s, p = s.cpu().numpy(), p.cpu().numpy()
    assert status.item() == 0
    want_pages, want_s, want_p = pool.copy(), score.copy(), pos.copy()
    after = ref.Cache(pages, dst)
    for b, n in enumerate(lens):
        i = np.arange(n)
        keep = ref.evict(score[c.table[b, i // page], i % page], n, budget, recent)
        assert got["new_len"][b].item() == len(keep)
        np.testing.assert_array_equal(kept[b], np.concatenate([keep, np.full(budget - len(keep), -1)]))
        at = np.arange(len(keep))
        for x, old in [(s, score), (p, pos)]:
            np.testing.assert_array_equal(x[dst[b, at // page], at % page], old[c.table[b, keep // page], keep % page])
        for h in range(H):
            for x, y in zip(after.get(b, h, at), c.get(b, h, keep)):
                np.testing.assert_array_equal(x, y)
        # the tail of the last block is zero; what lies behind it, and every other page, is untouched
        tail = np.arange(len(keep), -(-len(keep) // 32) * 32)
        assert (s[dst[b, tail // page], tail % page] == 0).all() and (p[dst[b, tail // page], tail % page] == 0).all()
        if len(tail):
            for h in range(H):
                assert all((x == 0).all() for x in after.get(b, h, tail))
        blocks = np.zeros((dper, page // 32), bool)
        blocks.reshape(-1)[:-(-len(keep) // 32)] = True
        for k in range(dper):
            np.testing.assert_array_equal(pages[dst[b, k]][:, ~blocks[k]], pool[dst[b, k]][:, ~blocks[k]])
    np.testing.assert_array_equal(pages[:c.n_pages], pool[:c.n_pages])
    np.testing.assert_array_equal(s[:c.n_pages], score[:c.n_pages])


def test_evict_skips_bad_requests():
    sv = need_gpu()
    rng = np.random.default_rng(21)
    c = quick_pool(rng, B=4, H=1, D=64, page=32, lens=[90] * 4)
    cache = gpu_cache(sv, c)
    dst = np.array([[0, 1]] * 4, np.int32)                          # never written: every request is bad
    dst[2, 1] = c.n_pages
    table = c.table.copy()
    table[1, 2] = -1
    score = torch.rand(c.n_pages, 32, device="cuda")
    before, s0 = cache.pages.clone(), score.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sv.cache_evict(cache, score, dev(np.array([97, 90, 90, -1], np.int32)), dev(table), dev(dst), B=4, budget=50, status=status)
    assert (got["kept"] == -1).all() and (got["new_len"] == -1).all()
    assert torch.equal(before, cache.pages) and torch.equal(s0, score)
    assert status.item() == 0x400 | 0x800


# ---------------------------------------------------------------- together ---

def test_the_example_runs_and_repeats_itself():
    """examples/cached_step.py: the same tokens twice, and caches within budget."""
    need_gpu()
    from examples import cached_step
    out, lens = cached_step.run(steps=30)
    again, lens2 = cached_step.run(steps=30)
    assert out == again and lens == lens2
    assert all(n <= 320 + 5 for n in lens) and any(len(t) > 320 for t in out)


def test_a_serving_loop():
    """Prompt, verify steps with rejected rows, weights, eviction, more steps:
    the cache's values and the last step's attention against the definition."""
    sv = need_gpu()
    rng = np.random.default_rng(31)
    B, H, D, page, k = 3, 2, 64, 32, 3
    cache = sv.new_cache(24, H, D, page)
    tables = [dev(np.arange(12, dtype=np.int32).reshape(3, 4)), dev(np.arange(12, 24, dtype=np.int32).reshape(3, 4))]
    score = torch.zeros(24, page, device="cuda")
    pos = torch.zeros(24, page, dtype=torch.int32, device="cuda")
    lens, nxt = np.array([40, 3, 70]), np.array([40, 3, 70])
    rows = lambda n: torch.from_numpy(rng.standard_normal((n, H, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    i32 = lambda x: dev(np.asarray(x, np.int32))
    n = int(lens.sum())
    sv.cache_append(cache, rows(n), rows(n), i32(np.concatenate([[0], np.cumsum(lens)])), i32([0, 0, 0]), tables[0],
                    B=B, max_rows=70, score=score, slot_pos=pos)
    cu = i32(np.arange(0, B * (k + 1) + 1, k + 1))
    for step in range(6):
        tab = tables[step >= 3]
        sv.cache_append(cache, rows(B * (k + 1)), rows(B * (k + 1)), cu, i32(lens), tab, B=B, max_rows=k + 1,
                        score=score, slot_pos=pos, pos0=i32(nxt))
        q = queries(rng, B * (k + 1), 2 * H, D, "bf16")
        kw = dict(B=B, k_max=k, slot_pos=pos, window=60, prefix=2)
        res = sv.cache_attend(cache, q, cu, i32(lens + k + 1), tab, **kw)
        sv.cache_weights(cache, q, res["lse"], cu, i32(lens + k + 1), tab, score, **kw)
        c = ref.Cache(cache.pages.cpu().numpy(), tab.cpu().numpy())
        out, lse, A, *_ = ref.attention(c, q.float().cpu().numpy(), np.arange(0, 13, 4), lens + k + 1, window=60, prefix=2,
                                        slot_pos=pos.cpu().numpy())
        assert (np.abs(res["out"].float().cpu().numpy() - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -10 * A).all()
        took = rng.integers(1, k + 2, B)                            # accepted drafts and the bonus
        lens, nxt = lens + took, nxt + took
        if step == 2:
            got = sv.cache_evict(cache, score, i32(lens), tables[0], tables[1], B=B, budget=48, recent=8, slot_pos=pos)
            lens = got["new_len"].cpu().numpy().astype(np.int64)
            np.testing.assert_array_equal(lens, np.minimum(nxt, 48))
