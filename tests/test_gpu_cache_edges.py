"""The 4-bit paged cache at the edges of its contract: limits of the arguments,
what hidden slots hold, streams, shared pages.  Bounds are those that
tests/test_gpu_cache.py derives."""
import numpy as np
import pytest

from tests._gpu import need_gpu
from tests.test_gpu_cache import check_attention, dev, gpu_cache, queries, quick_pool

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
