"""Host-side checks of the prompt and tree operators: argument errors are refused before
anything is launched (no device needed), and the plain references that the GPU tests use are
themselves pinned."""
import ctypes as C

import numpy as np
import pytest

from tests import _step_ref as ref


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


FAKE, ODD = C.c_void_p(0x10000), C.c_void_p(0x10002)


def _prompt(**over):
    from speculative_decoding_verification_ragged_gb300.prompt import _Prompt
    return _Prompt(**{**dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, D=128, Hq=8, H=2, q_row=1024, q_head=128, k_row=256, k_head=128,
                             v_row=256, v_head=128, B=2, R_cap=100, K_cap=100, cu_rows=FAKE, scale=0.1), **over})


def _tree(**over):
    from speculative_decoding_verification_ragged_gb300.tree import _Tree
    return _Tree(**{**dict(B=2, k_max=3, R_cap=8, cu_rows=FAKE, row_token=FAKE, node_token=FAKE, parent=FAKE, accepted_len=FAKE,
                           out_tokens=FAKE, next_token=FAKE), **over})


def _rules(**over):
    from speculative_decoding_verification_ragged_gb300.tree import _Rules
    return _Rules(**{**dict(logits=FAKE, dtype=1, V=1000, ld=1000, B=2, k_max=3, R_cap=8, cu_rows=FAKE), **over})


@pytest.mark.parametrize("over,rc", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cu_rows=None), 1), (dict(dtype=2), 2), (dict(D=96), 2),
    (dict(Hq=7), 1), (dict(Hq=0), 1), (dict(H=0), 1), (dict(B=0), 1), (dict(R_cap=0), 1), (dict(K_cap=0), 1), (dict(window=-1), 1),
    (dict(prefix=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(cap=-1.0), 1),
    (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(q=C.c_void_p(0x10001)), 1), (dict(dtype=0, k=ODD), 1),
    (dict(cu_rows=ODD), 1), (dict(cu_keys=ODD), 1), (dict(slopes=ODD), 1), (dict(status=ODD), 1), (dict(B=70000), 2),
    (dict(H=70000, Hq=70000), 2), (dict(R_cap=(1 << 30) + 1), 2), (dict(K_cap=(1 << 24) + 1), 2), (dict(R_cap=1 << 30), 2)])
def test_prompt_is_checked(sv, over, rc):
    L, a = sv.load_library(), _prompt(**over)
    assert L.spec_prompt_attend(C.byref(a), FAKE, FAKE, FAKE, 1 << 40, None) == rc


def test_prompt_outputs_and_workspace_are_checked(sv):
    L, a = sv.load_library(), _prompt()
    n = L.spec_prompt_workspace_bytes(8, 2, 128, 1)
    assert n > 0
    assert L.spec_prompt_attend(None, FAKE, FAKE, FAKE, n, None) == 1
    assert L.spec_prompt_attend(C.byref(a), None, FAKE, FAKE, n, None) == 1
    assert L.spec_prompt_attend(C.byref(a), C.c_void_p(0x10001), FAKE, FAKE, n, None) == 1
    assert L.spec_prompt_attend(C.byref(a), FAKE, ODD, FAKE, n, None) == 1
    assert L.spec_prompt_attend(C.byref(a), FAKE, FAKE, C.c_void_p(0x10008), n, None) == 1
    assert L.spec_prompt_attend(C.byref(a), FAKE, FAKE, None, n, None) == 4
    assert L.spec_prompt_attend(C.byref(a), FAKE, FAKE, FAKE, n - 1, None) == 4
    for bad in [(8, 0, 128, 1), (0, 1, 128, 1), (7, 2, 128, 1), (8, 2, 96, 1), (8, 2, 128, 2)]:
        assert L.spec_prompt_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("over,rc", [
    (dict(cu_rows=None), 1), (dict(row_token=None), 1), (dict(node_token=None), 1), (dict(parent=None), 1),
    (dict(accepted_len=None), 1), (dict(out_tokens=None), 1), (dict(next_token=None), 1), (dict(B=0), 1), (dict(k_max=-1), 1),
    (dict(k_max=32), 2), (dict(B=(1 << 30) + 1), 2), (dict(R_cap=0), 1), (dict(parent=ODD), 1), (dict(path_rows=ODD), 1), (dict(status=ODD), 1)])
def test_tree_is_checked(sv, over, rc):
    L, a = sv.load_library(), _tree(**over)
    assert L.spec_tree_accept(C.byref(a), None) == rc
    assert L.spec_tree_accept(None, None) == 1


def test_tree_attention_is_checked(sv):
    from tests.test_cache_host import BAD_CACHE, _attn, _cache
    L, c, a = sv.load_library(), _cache(), _attn()
    n = 1 << 30
    for over, rc in BAD_CACHE:
        assert L.spec_cache_attend_tree(C.byref(_cache(**over)), C.byref(a), FAKE, FAKE, FAKE, FAKE, n, None) == rc
    assert L.spec_cache_attend_tree(C.byref(c), C.byref(_attn(k_max=32)), FAKE, FAKE, FAKE, FAKE, n, None) == 2
    assert L.spec_cache_attend_tree(C.byref(c), C.byref(a), None, FAKE, FAKE, FAKE, n, None) == 1
    assert L.spec_cache_attend_tree(C.byref(c), C.byref(a), ODD, FAKE, FAKE, FAKE, n, None) == 1
    assert L.spec_cache_attend_tree(C.byref(c), C.byref(a), FAKE, None, FAKE, FAKE, n, None) == 1
    assert L.spec_cache_attend_tree(C.byref(c), C.byref(a), FAKE, FAKE, FAKE, None, n, None) == 4
    assert L.spec_cache_attend_tree(C.byref(c), C.byref(a), FAKE, FAKE, FAKE, FAKE, 16, None) == 4


@pytest.mark.parametrize("over,rc", [
    (dict(logits=None), 1), (dict(cu_rows=None), 1), (dict(dtype=2), 2), (dict(V=0), 1), (dict(ld=999), 1), (dict(B=0), 1),
    (dict(R_cap=0), 1), (dict(k_max=-1), 1), (dict(k_max=32), 2), (dict(B=70000), 2), (dict(logits=C.c_void_p(0x10001)), 1),
    (dict(history=FAKE, history_ld=10, history_cap=10), 1), (dict(history=FAKE, n_tokens=FAKE, history_ld=9, history_cap=10), 1),
    (dict(history=FAKE, n_tokens=FAKE, history_ld=10, history_cap=-1), 1), (dict(history=ODD, n_tokens=FAKE), 1),
    (dict(history=FAKE, n_tokens=FAKE, history_ld=1 << 31, history_cap=(1 << 31) - 1), 2),
    (dict(history=FAKE, n_tokens=FAKE, history_ld=1 << 28, history_cap=(1 << 28) - 63), 2),
    (dict(bias_cu=FAKE, n_bias=(1 << 30) + 1, bias_ids=FAKE, bias_values=FAKE), 2),
    (dict(bias_cu=FAKE, n_bias=-1), 1), (dict(bias_cu=FAKE, n_bias=3, bias_ids=FAKE), 1),
    (dict(bias_cu=FAKE, n_bias=3, bias_values=FAKE), 1), (dict(allowed=FAKE, n_allowed=0, allowed_ld=32), 1),
    (dict(allowed=FAKE, n_allowed=1, allowed_ld=31), 1), (dict(repetition=ODD), 1), (dict(parent=ODD), 1), (dict(status=ODD), 1)])
def test_logit_rules_are_checked(sv, over, rc):
    L, a = sv.load_library(), _rules(**over)
    assert L.spec_adjust_logits(C.byref(a), C.c_void_p(0x90000), 1000, None) == rc


def test_adjusted_logits_are_checked(sv):
    L, a = sv.load_library(), _rules(ld=1008)
    assert L.spec_adjust_logits(None, FAKE, 1000, None) == 1
    assert L.spec_adjust_logits(C.byref(a), None, 1000, None) == 1
    assert L.spec_adjust_logits(C.byref(a), C.c_void_p(0x90001), 1000, None) == 1
    assert L.spec_adjust_logits(C.byref(a), C.c_void_p(0x90000), 999, None) == 1
    assert L.spec_adjust_logits(C.byref(a), FAKE, 1000, None) == 1      # in place, but rows elsewhere


def test_binding_refuses_host_tensors(sv):
    import torch
    x, i = torch.zeros(4, 2, 64), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: sv.prompt_attend(x, x, x, i, B=2), lambda: sv.tree_accept(i, i, i, i, B=2, k_max=1),
                 lambda: sv.adjust_logits(x[0], i, V=64, B=2, k_max=0)):
        with pytest.raises(sv.SpecError, match="CUDA device"):
            call()


# ---------------------------------------------------------------- the references ---

def test_reference_of_the_acceptance_by_hand():
    # 0 -> 1 (7), 2 (8); 1 -> 3 (9); 2 -> 4 (9), 5 (9); row 6 hangs on none
    parent, token = [-1, 0, 0, 1, 2, 2, -1], [0, 7, 8, 9, 9, 9, 7]
    acc, out, nxt, path = ref.accept([8, 1, 9, 1, 5, 6, 7], token, parent, [0, 7], 7)
    assert acc[0] == 2 and nxt[0] == 5                       # the lower of the two 9s
    assert out[0].tolist() == [8, 9, 5, -1, -1, -1, -1, -1] and path[0].tolist() == [0, 2, 4, 4, 4, 4, 4, 4]
    acc, out, nxt, path = ref.accept([6, 1, 9, 1, 5, 6, 7], token, parent, [0, 7], 7)
    assert acc[0] == 0 and nxt[0] == 6 and path[0].tolist() == [0] * 8


def test_reference_of_the_acceptance_is_the_chains_own():
    from oracle import verify_greedy
    rng = np.random.default_rng(3)
    B, k, V = 40, 5, 6
    z = rng.standard_normal((B * (k + 1), V)).astype(np.float32)
    best = z.argmax(1)
    cu = np.arange(0, B * (k + 1) + 1, k + 1, dtype=np.int32)
    drafts = np.where(rng.random(len(best)) < 0.7, best, rng.integers(0, V, len(best))).astype(np.int32)
    want = verify_greedy(z, "f32", V, B, k, cu, drafts)
    node = np.roll(drafts, 1)
    parent = np.tile(np.arange(-1, k), B)
    acc, out, nxt, path = ref.accept(best, node, parent, cu, k)
    assert np.array_equal(acc, want.accepted_len) and np.array_equal(out, want.out_tokens)
    assert np.array_equal(nxt, want.next_token)


def test_reference_of_the_adjustment_by_hand():
    z = np.array([[2.0, -2.0, 1.0, 0.5, 3.0]] * 2)
    got, _ = ref.adjust(z, [0, 2], 5, history=[[0, 1, 1, 9, -1]], n_tokens=[5], n_prompt=[1], repetition=[2.0], frequency=[0.25],
                        presence=[1.0], node_token=[4, 4], bias=[([3, 3, 7], [1.0, 0.5, 9.0])],
                        allowed=np.array([[0b11011]], np.int32), allowed_row=[-1, 0])
    # token 0: prompt alone (2 / 2); token 1: twice generated (-2 * 2 - 0.5 - 1); the root's own token is in the history only
    assert got[0].tolist() == [1.0, -5.5, 1.0, 2.0, 3.0]
    # the second row comes after a draft of 4: 3 / 2 - 0.25 - 1; column 2 masked
    assert got[1].tolist() == [1.0, -5.5, -np.inf, 2.0, 0.25]


def test_reference_of_the_prompt_against_a_matrix():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((7, 2, 4)) for _ in range(3))
    out, lse, _, _ = ref.prompt(q, k, v, [0, 3, 7])
    for lo, hi in [(0, 3), (3, 7)]:
        for h in range(2):
            s = q[lo:hi, h] @ k[lo:hi, h].T / 2
            s = np.where(np.tril(np.ones_like(s)) > 0, s, -np.inf)
            p = np.exp(s)
            assert np.allclose(out[lo:hi, h], p / p.sum(1, keepdims=True) @ v[lo:hi, h])
            assert np.allclose(lse[lo:hi, h], np.log(p.sum(1)))
    # a piece: the last two rows over all keys
    piece, _, _, _ = ref.prompt(q[5:], k, v, [0, 0, 2], [0, 3, 7])
    assert np.allclose(piece, out[5:])
