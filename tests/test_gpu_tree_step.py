"""A step with a tree of drafts, the operators together: prompts, trees over the cache, penalties and masks,
acceptance, the path kept."""
import numpy as np
import pytest

from tests._gpu import need_gpu

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    need_gpu()
    import speculative_decoding_verification_ragged_gb300 as sv
    sv.build()
    return sv


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def test_the_example_runs(sv):
    from examples import tree_step
    for kw in (dict(), dict(penalties=False), dict(B=1, width=1, depth=6, D=64), dict(width=7, depth=4, Hq=4, H=4)):
        out, accepted = tree_step.run(steps=3, **kw)
        assert all(len(t) >= 4 for t in out) and accepted == sum(len(t) - 4 for t in out)
    out, _ = tree_step.run(steps=6)
    assert max(out[0][1:]) < 1024                                       # the grammar of request 0


def test_trees_give_the_tokens_of_plain_decoding(sv):
    """Greedy decoding with trees emits what decoding one token at a time does.  fp32 queries and logits.  An
    attention output is within 2^-19 of the weighted magnitudes (at most 1 here); a logit is a sum of 2048 of them times
    values of 4 * 2048^-1/2 N(0, 1), whose magnitudes are 0.07 on average: within 2048 * 2^-19 * 0.07 = 2.8e-4, so that two
    that are 1e-3 apart come out in one order on both ways; tokens are compared up to the first decision that is closer.  The drafts hold the right tokens up to some depth, in
    one of the chains."""
    from examples import tree_step
    from examples.cached_step import Target
    B, V, Hq, H, D, prompt, page, steps, depth = 6, 2048, 16, 4, 128, 200, 64, 8, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    model = Target(V, Hq, H, D, gen)
    room = prompt + steps * (depth + 1) + 13
    per = -(-room // page)
    cache = sv.new_cache(B * per, H, D, page)
    table = torch.randperm(B * per, generator=gen, device="cuda").int().view(B, per)
    lens = [prompt - 17 * (b % 5) for b in range(B)]
    history = torch.randint(0, V, (B, room), generator=gen, device="cuda").int()
    cu = i32([0] + torch.tensor(lens).cumsum(0).tolist())
    query, key, value = model.project(torch.cat([history[b, :lens[b]] for b in range(B)]).long())
    att = sv.prompt_attend(query, key, value, cu, B=B)
    sv.cache_append(cache, key, value, cu, i32([0] * B), table, B=B, max_rows=max(lens))
    length, root = i32(lens), (att["out"][cu[1:].long() - 1].flatten(1) @ model.head).argmax(1).int()
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    plain, clear = [[int(t)] for t in root], [1] * B                    # tokens before the first close decision
    for _ in range(steps * (depth + 1) + depth):
        query, key, value = model.project(root.long())
        sv.cache_append(cache, key, value, one, length, table, B=B, max_rows=1)
        length = length + 1
        att = sv.cache_attend(cache, query.float(), one, length, table, B=B, k_max=0)
        top = (att["out"].flatten(1) @ model.head.float()).topk(2)
        root = top.indices[:, 0].int()
        for b in range(B):
            if clear[b] == len(plain[b]) and float(top.values[b, 0] - top.values[b, 1]) > 1e-3:
                clear[b] += 1
            plain[b].append(int(root[b]))
    rng = np.random.default_rng(1)

    def drafts(model, root, length, width, depth):
        _, parent = tree_step.draft(model, root, length, width, depth)
        tokens = rng.integers(0, V, (B, len(parent)))
        tokens[:, 0] = root.cpu()
        for b in range(B):
            e, w = int(length[b]) - lens[b], int(rng.integers(0, width))
            right = int(rng.integers(0, depth + 1))                      # nodes 1 + w, 1 + w + width, ... are a chain
            tokens[b, 1 + w::width][:right] = plain[b][e + 1:e + 1 + right]
        return torch.from_numpy(tokens).cuda(), parent

    out, accepted = tree_step.run(steps=steps, penalties=False, dtype=torch.float32, drafts=drafts)
    assert accepted > B * steps
    assert sum(min(n, len(t)) for n, t in zip(clear, out)) > sum(len(t) for t in out) // 2
    for b, t in enumerate(out):
        assert t[:clear[b]] == plain[b][:len(t)][:clear[b]], b


def test_the_path_in_the_cache_is_a_chain(sv):
    """After a step the cache holds the accepted path slot by slot: the weights of the path's rows can be added as a
    chain's, and the next row sees root and path."""
    rng = np.random.default_rng(3)
    H, D, n, start = 2, 64, 7, 40
    cache, table = sv.new_cache(4, H, D, 32), i32([[3, 1, 0]])
    rand = lambda r: torch.from_numpy(rng.standard_normal((r, H, D)).astype(np.float32)).cuda()
    k0, v0 = rand(start), rand(start)
    sv.cache_append(cache, k0, v0, i32([0, start]), i32([0]), table, B=1, max_rows=start)
    key, value, q = rand(n), rand(n), rand(n)
    parent, node, want = i32([-1, 0, 0, 1, 2, 4, 4]), i32([0, 5, 6, 7, 8, 9, 9]), i32([6, 0, 8, 0, 9, 3, 4])
    rows = i32([0, n])
    sv.cache_append(cache, key, value, rows, i32([start]), table, B=1, max_rows=n)
    att = sv.cache_attend_tree(cache, q, rows, i32([start + n]), table, parent, B=1, k_max=n - 1)
    got = sv.tree_accept(want, node, parent, rows, B=1, k_max=n - 1)
    assert got["accepted_len"].tolist() == [3] and got["path_rows"][0].tolist() == [0, 2, 4, 5, 5, 5, 5]
    assert got["out_tokens"][0].tolist() == [6, 8, 9, 3, -1, -1, -1]
    at = got["path_rows"][0, :4].long()
    sv.cache_append(cache, key[at], value[at], i32([0, 4]), i32([start]), table, B=1, max_rows=4)
    chain = sv.cache_attend(cache, q[at], i32([0, 4]), i32([start + 4]), table, B=1, k_max=3)
    # the same slots with the same bytes, as a tree and as a chain: sums in another order
    assert torch.allclose(chain["out"], att["out"][at], atol=1e-5) and torch.allclose(chain["lse"], att["lse"][at], atol=1e-5)
    score = torch.zeros(4, 32, device="cuda")
    sv.cache_weights(cache, q[at], chain["lse"], i32([0, 4]), i32([start + 4]), table, score, B=1, k_max=3)
    assert abs(float(score.sum()) - 4 * H) < 1e-3
