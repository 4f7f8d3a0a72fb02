"""Speculative decoding steps over a 4-bit paged cache: the loop of a serving
engine around this library, with one attention layer of random weights in the
place of the target model and random tokens in the place of the draft's.

    python examples/cached_step.py [--steps 12]

Each step appends the k + 1 rows of every request, attends with them over the
cache, verifies the drafts greedily, keeps the accepted prefix, and adds up the
attention that the cached tokens got from the rows that stayed.  A request whose cache has outgrown its
budget loses the tokens that got the least.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_ragged_gb300 as sv  # noqa: E402


class Target:
    """One attention layer and a head over V tokens, bf16."""

    def __init__(self, V, Hq, H, D, gen):
        def rand(*shape, scale=1.0):
            return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(torch.bfloat16)
        E = Hq * D
        self.Hq, self.H, self.D, self.V = Hq, H, D, V
        self.embed = rand(V, E)
        self.wq, self.wk, self.wv = (rand(E, n * D, scale=E ** -0.5) for n in (Hq, H, H))
        self.head = rand(E, V, scale=4 * E ** -0.5)

    def project(self, tokens):
        x = self.embed[tokens]
        return tuple((x @ w).view(len(tokens), -1, self.D) for w in (self.wq, self.wk, self.wv))


def run(steps: int = 12, B: int = 8, k: int = 4, V: int = 2048, Hq: int = 16, H: int = 4, D: int = 128,
        prompt: int = 300, budget: int = 320, page: int = 64, seed: int = 0):
    """Runs the loop; returns the tokens of every request and the final lengths."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    model = Target(V, Hq, H, D, gen)
    per = -(-(budget + 64 + prompt) // page)                  # pages of a request, twice: eviction moves
    cache = sv.new_cache(2 * B * per, H, D, page)
    tables = torch.arange(2 * B * per, dtype=torch.int32, device="cuda").view(2, B, per)
    score = torch.zeros(cache.n_pages, page, device="cuda")   # attention each cached token got
    pos = torch.zeros(cache.n_pages, page, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = 0

    def i32(x):
        return torch.as_tensor(x, dtype=torch.int32, device="cuda")

    # the prompts: ragged, appended at once
    lens = [prompt - 17 * (b % 5) for b in range(B)]
    tokens = [torch.randint(0, V, (n,), generator=gen, device="cuda") for n in lens]
    cu = i32([0] + torch.tensor(lens).cumsum(0).tolist())
    _, key, value = model.project(torch.cat(tokens))
    sv.cache_append(cache, key, value, cu, i32([0] * B), tables[side], B=B, max_rows=max(lens), score=score,
                    slot_pos=pos, status=status)
    length, position = i32(lens), i32(lens)                   # tokens cached, tokens seen
    rows = B * (k + 1)
    cu = torch.arange(0, rows + 1, k + 1, dtype=torch.int32, device="cuda")
    current = torch.stack([t[-1] for t in tokens])            # the token each request goes on from
    out = [t.tolist() for t in tokens]
    for step in range(steps):
        # the drafts: k tokens a request, the last row is the bonus row
        drafts = torch.randint(0, V, (B, k), generator=gen, device="cuda")
        if step % 3 == 2:
            drafts[::2, 0] = current[::2]                     # (whatever the draft model proposes)
        fed = torch.cat([current[:, None], drafts], 1).flatten()
        query, key, value = model.project(fed)
        sv.cache_append(cache, key, value, cu, length, tables[side], B=B, max_rows=k + 1, score=score, slot_pos=pos,
                        pos0=position, status=status)
        options = dict(B=B, k_max=k, slot_pos=pos, cap=30.0, status=status)
        grown = length + (k + 1)
        att = sv.cache_attend(cache, query, cu, grown, tables[side], **options)
        logits = att["out"].flatten(1) @ model.head
        check = torch.cat([drafts, drafts.new_zeros(B, 1)], 1).flatten().int()
        got = sv.verify_greedy(logits, cu, check, V=V, B=B, k_max=k)
        # rows of rejected drafts have no say in what is evicted: lse = -inf counts as 0
        rejected = torch.arange(k + 1, device="cuda") > got["accepted_len"][:, None]
        lse = att["lse"].view(B, k + 1, Hq).masked_fill(rejected[..., None], float("-inf")).flatten(0, 1)
        sv.cache_weights(cache, query, lse, cu, grown, tables[side], score, **options)
        # the accepted drafts stay cached with the token before them; the next token
        # is not in the cache yet
        kept = got["accepted_len"] + 1
        length, position, current = length + kept, position + kept, got["next_token"].long()
        for b, row in enumerate(got["out_tokens"].tolist()):
            out[b] += [t for t in row if t >= 0]
        if int(length.max()) > budget:
            ev = sv.cache_evict(cache, score, length, tables[side], tables[1 - side], B=B, budget=budget, recent=32,
                                slot_pos=pos, status=status)
            length, side = ev["new_len"], 1 - side
    assert int(status) == 0
    return out, length.tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    sv.build()
    out, lens = run(a.steps)
    for b, (t, n) in enumerate(zip(out, lens)):
        print("request %d: %d tokens, %d cached, last %s" % (b, len(t), n, t[-5:]))
