"""Host-side checks of the 4-bit paged cache: argument errors are refused
before anything is launched (no device needed), and the plain reference that
the GPU tests use is itself pinned."""
import ctypes as C

import numpy as np
import pytest

from tests import _cache_ref as ref


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


FAKE = C.c_void_p(0x10000)


def _cache(**over):
    from speculative_decoding_verification_ragged_gb300.cache import _Cache
    return _Cache(**{**dict(pages=FAKE, n_pages=10, page_tokens=64, H=4, D=128, k_scale=None, v_scale=None, B=2,
                            max_pages=5, page_table=FAKE), **over})


def _rows(**over):
    from speculative_decoding_verification_ragged_gb300.cache import _Rows
    return _Rows(**{**dict(k=FAKE, v=FAKE, dtype=1, k_row=512, k_head=128, v_row=512, v_head=128, R_cap=8, max_rows=4,
                           cu_rows=FAKE, start=FAKE), **over})


def _attn(**over):
    from speculative_decoding_verification_ragged_gb300.cache import _Attention
    return _Attention(**{**dict(q=FAKE, dtype=1, q_row=1024, q_head=128, Hq=8, R_cap=8, k_max=3, cu_rows=FAKE, len=FAKE,
                                max_len=0, scale=0.1, cap=0.0, window=0, prefix=0), **over})


def _evict(**over):
    from speculative_decoding_verification_ragged_gb300.cache import _Eviction
    return _Eviction(**{**dict(score=FAKE, slot_pos=None, len=FAKE, budget=100, recent=10, dst_table=FAKE, dst_pages=2,
                               kept=FAKE, new_len=FAKE), **over})


BAD_CACHE = [(dict(pages=None), 1), (dict(page_table=None), 1), (dict(pages=C.c_void_p(0x10008)), 1), (dict(n_pages=0), 1),
             (dict(H=0), 1), (dict(B=0), 1), (dict(max_pages=0), 1), (dict(page_tokens=48), 1), (dict(page_tokens=0), 1),
             (dict(D=96), 2), (dict(H=70000), 2), (dict(B=70000), 2), (dict(page_tokens=65568), 2), (dict(max_pages=1 << 25), 2)]


@pytest.mark.parametrize("over,rc", BAD_CACHE)
def test_every_call_refuses_a_bad_cache(sv, over, rc):
    L, c = sv.load_library(), _cache(**over)
    n = 1 << 30
    assert L.spec_cache_append(C.byref(c), C.byref(_rows()), None) == rc
    assert L.spec_cache_read(C.byref(c), C.byref(_rows()), None) == rc
    assert L.spec_cache_attend(C.byref(c), C.byref(_attn()), FAKE, FAKE, FAKE, n, None) == rc
    assert L.spec_cache_weights(C.byref(c), C.byref(_attn()), FAKE, FAKE, None) == rc
    assert L.spec_cache_evict(C.byref(c), C.byref(_evict()), None) == rc


@pytest.mark.parametrize("over,rc", [(dict(k=None), 1), (dict(v=None), 1), (dict(cu_rows=None), 1), (dict(start=None), 1),
                                     (dict(dtype=5), 2), (dict(R_cap=0), 1), (dict(max_rows=0), 1),
                                     (dict(k=C.c_void_p(0x10001)), 1), (dict(v=C.c_void_p(0x10001)), 1)])
def test_rows_are_checked(sv, over, rc):
    L = sv.load_library()
    for f in (L.spec_cache_append, L.spec_cache_read):
        assert f(C.byref(_cache()), C.byref(_rows(**over)), None) == rc
        assert f(C.byref(_cache()), None, None) == 1


@pytest.mark.parametrize("over,rc", [(dict(q=None), 1), (dict(cu_rows=None), 1), (dict(len=None), 1), (dict(dtype=3), 2),
                                     (dict(Hq=6), 1), (dict(Hq=0), 1), (dict(R_cap=0), 1), (dict(k_max=-1), 1),
                                     (dict(k_max=32), 2), (dict(window=-1), 1), (dict(prefix=-1), 1),
                                     (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(cap=-1.0), 1),
                                     (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(max_len=321), 1),
                                     (dict(max_len=-1), 1), (dict(q=C.c_void_p(0x10001)), 1)])
def test_attention_is_checked(sv, over, rc):
    L = sv.load_library()
    a = _attn(**over)
    assert L.spec_cache_attend(C.byref(_cache()), C.byref(a), FAKE, FAKE, FAKE, 1 << 30, None) == rc
    assert L.spec_cache_weights(C.byref(_cache()), C.byref(a), FAKE, FAKE, None) == rc


def test_attention_outputs_and_workspace_are_checked(sv):
    L, c, a = sv.load_library(), _cache(), _attn()
    n = L.spec_cache_workspace_bytes(2, 3, 8, 4, 128, 320)
    assert n > 0
    assert L.spec_cache_attend(C.byref(c), C.byref(a), None, FAKE, FAKE, n, None) == 1
    assert L.spec_cache_attend(C.byref(c), C.byref(a), C.c_void_p(0x10001), FAKE, FAKE, n, None) == 1
    assert L.spec_cache_attend(C.byref(c), C.byref(a), FAKE, FAKE, None, n, None) == 4
    assert L.spec_cache_attend(C.byref(c), C.byref(a), FAKE, FAKE, FAKE, n - 1, None) == 4
    assert L.spec_cache_attend(C.byref(c), None, FAKE, FAKE, FAKE, n, None) == 1
    assert L.spec_cache_weights(C.byref(c), C.byref(a), None, FAKE, None) == 1
    assert L.spec_cache_weights(C.byref(c), C.byref(a), FAKE, None, None) == 1
    for bad in [(0, 3, 8, 4, 128, 320), (2, -1, 8, 4, 128, 320), (2, 32, 8, 4, 128, 320), (2, 3, 6, 4, 128, 320),
                (2, 3, 8, 4, 96, 320), (2, 3, 8, 4, 128, 0), (2, 3, 8, 0, 128, 320)]:
        assert L.spec_cache_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("over", [dict(score=None), dict(len=None), dict(dst_table=None), dict(kept=None), dict(new_len=None),
                                  dict(budget=0), dict(recent=-1), dict(recent=101), dict(dst_pages=0), dict(dst_pages=1),
                                  dict(budget=1000, dst_pages=4)])
def test_eviction_is_checked(sv, over):
    L = sv.load_library()
    assert L.spec_cache_evict(C.byref(_cache()), C.byref(_evict(**over)), None) == 1
    assert L.spec_cache_evict(C.byref(_cache()), None, None) == 1


def test_binding_refuses_host_tensors_and_bad_pools(sv):
    import torch
    with pytest.raises(sv.SpecError, match="36 D"):
        sv.PagedCache(torch.zeros(2, 1, 1, 36 * 96, dtype=torch.uint8))
    with pytest.raises(sv.SpecError, match="uint8"):
        sv.PagedCache(torch.zeros(2, 1, 1, 36 * 64))
    with pytest.raises(sv.SpecError, match="per kv head"):
        sv.PagedCache(torch.zeros(2, 1, 1, 36 * 64, dtype=torch.uint8), k_scale=torch.ones(2))
    for kw in (dict(D=96), dict(D=64, page_tokens=40), dict(D=64, page_tokens=0)):
        with pytest.raises(sv.SpecError):
            sv.new_cache(2, 1, **kw, device="cpu")
    c = sv.PagedCache(torch.zeros(2, 1, 1, 36 * 64, dtype=torch.uint8))
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(sv.SpecError, match="CUDA"):
        sv.cache_read(c, i32, i32, i32.view(1, 2), B=1, max_rows=1)
    with pytest.raises(sv.SpecError, match="CUDA"):
        sv.cache_attend(c, torch.zeros(1, 1, 64), i32, i32, i32.view(1, 2), B=1, k_max=0)
    with pytest.raises(sv.SpecError, match="CUDA"):
        sv.cache_evict(c, torch.zeros(2, 32), i32, i32.view(1, 2), i32.view(1, 2), B=1, budget=1)


# ----------------------------------------------------- the reference itself ---

def test_reference_grids():
    assert ref.E4M3[126] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6
    x = np.array([0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 100.0])
    np.testing.assert_array_equal(ref.E2M1[ref.nearest(x, ref.E2M1)], [0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6])


def test_reference_put_and_get_agree_and_touch_nothing_else():
    rng = np.random.default_rng(0)
    c = ref.Cache(rng.integers(0, 127, (3, 2, 2, 36 * 64), dtype=np.uint8), np.array([[2, 0]]))
    before = {(h, s): c.get(0, h, [s]) for h in range(2) for s in range(128)}
    k, v = rng.standard_normal((2, 64)).astype(np.float32)
    c.put(0, 1, 77, k, v)
    for (h, s), (ok, ov) in before.items():
        nk, nv = c.get(0, h, [s])
        if (h, s) == (1, 77):
            # a value is within half a grid step of its block's scale: at most a sixth of the largest
            big = np.abs(k.reshape(4, 16)).max(-1).repeat(16)
            assert (np.abs(nk[0] - k) <= big / 6 * 1.07).all()
        else:
            np.testing.assert_array_equal(nk, ok)
            np.testing.assert_array_equal(nv, ov)


def test_reference_attention_closed_forms():
    rng = np.random.default_rng(1)
    c = ref.Cache(rng.integers(0, 120, (2, 1, 1, 36 * 64), dtype=np.uint8), np.array([[0, 1]]))
    q = np.zeros((2, 1, 64))
    out, lse, A, S, w = ref.attention(c, q, np.array([0, 2]), [40])
    k, v = c.get(0, 0, np.arange(40))
    np.testing.assert_allclose(out[1, 0], v.mean(0))                  # equal scores: the mean
    np.testing.assert_allclose(out[0, 0], v[:39].mean(0))             # the first row does not see the second's slot
    np.testing.assert_allclose(lse[:, 0], np.log([39, 40]))
    np.testing.assert_allclose(w[0][:39], 1 / 39 + 1 / 40)
    out, lse, *_ = ref.attention(c, q, np.array([0, 2]), [40], window=1)
    np.testing.assert_allclose(out[:, 0], v[38:40])                   # itself alone
    out, lse, *_ = ref.attention(c, q, np.array([0, 2]), [1])
    assert lse[0, 0] == -np.inf and (out[0] == 0).all() and lse[1, 0] == 0


def test_reference_evict():
    s = np.array([3, 1, 2, 2, 9, 0, 0], np.float32)
    np.testing.assert_array_equal(ref.evict(s, 7, 4, 1), [0, 2, 4, 6])
    np.testing.assert_array_equal(ref.evict(s, 7, 7, 1), np.arange(7))
    np.testing.assert_array_equal(ref.evict(np.array([np.nan, -np.inf, 1, 0], np.float32), 4, 2, 0), [2, 3])
    np.testing.assert_array_equal(ref.evict(np.array([np.nan, -np.inf, 1, 0], np.float32), 4, 3, 0), [1, 2, 3])
