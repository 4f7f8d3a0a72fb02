"""Speculative decoding with trees of drafts over a 4-bit paged cache: the loop of a
serving engine around this library, with one attention layer of random weights in
the place of the target model and its head without the attention as the draft (which
random weights rarely let hit).

    python examples/tree_step.py [--steps 12]

The prompts attend over themselves and enter the cache.  Each step drafts a tree of
tokens for every request, appends its nodes, attends over the cache and each node's
ancestors, adjusts the logits by the requests' penalties and what their grammar allows,
verifies all nodes greedily, and follows the target's tokens through the tree.  The accepted
path's keys and values are appended once more, one after another: the other nodes' slots are
overwritten.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_ragged_gb300 as sv  # noqa: E402
from examples.cached_step import Target  # noqa: E402


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def draft(model, root, length, width, depth):
    """A tree of drafts for every request, which goes on from token root[b] at length[b] cached ones: `width`
    children at the root, each the head of a chain.  Returns the nodes' tokens [B, n] (the root's first) and
    parents [n]."""
    def best(tokens, k):
        return (model.embed[tokens] @ model.head).float().topk(k).indices
    parent, level = [-1], best(root, width)                            # [B, width]
    nodes, at = [root[:, None]], [0] * width
    for _ in range(depth):
        nodes.append(level)
        first = len(parent)
        parent += at
        at = list(range(first, first + width))
        level = best(level.flatten(), 1).view(level.shape)
    return torch.cat(nodes, 1), i32(parent)


def run(steps: int = 12, B: int = 6, width: int = 3, depth: int = 4, V: int = 2048, Hq: int = 16, H: int = 4, D: int = 128,
        prompt: int = 200, page: int = 64, seed: int = 0, penalties: bool = True, dtype=torch.bfloat16, drafts=draft):
    """Runs the loop; returns the tokens of every request and how many drafts were accepted."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    model = Target(V, Hq, H, D, gen)
    n = 1 + width * depth                                              # nodes of a tree
    room = prompt + steps * (depth + 1) + n
    per = -(-room // page)
    cache = sv.new_cache(B * per, H, D, page)
    table = torch.randperm(B * per, generator=gen, device="cuda").int().view(B, per)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    # the prompts: ragged, over themselves and into the cache at once
    lens = [prompt - 17 * (b % 5) for b in range(B)]
    history = torch.randint(0, V, (B, room), generator=gen, device="cuda").int()
    tokens = torch.cat([history[b, :lens[b]] for b in range(B)]).long()
    cu = i32([0] + torch.tensor(lens).cumsum(0).tolist())
    query, key, value = model.project(tokens)
    att = sv.prompt_attend(query, key, value, cu, B=B, status=status)
    sv.cache_append(cache, key, value, cu, i32([0] * B), table, B=B, max_rows=max(lens), status=status)
    last = cu[1:].long() - 1
    root = (att["out"][last].flatten(1) @ model.head).argmax(1).int()  # the token that each request goes on from
    length, n_prompt = i32(lens), i32(lens)
    history[torch.arange(B, device="cuda"), length.long()] = root

    rows = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    path = torch.arange(0, B * (depth + 1) + 1, depth + 1, dtype=torch.int32, device="cuda")
    rule = dict(repetition=torch.full((B,), 1.1, device="cuda"), frequency=torch.full((B,), 0.2, device="cuda"),
                presence=torch.zeros(B, device="cuda"))
    # a grammar: request 0 has to answer in tokens below V / 2
    allowed = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    allowed[0, V // 64:] = 0
    allowed_row = torch.full((B * n,), -1, dtype=torch.int32, device="cuda")
    allowed_row[:n] = 0
    out, accepted = [[int(t)] for t in root], 0
    for _ in range(steps):
        fed, parent = drafts(model, root.long(), length, width, depth)
        fed, parent = fed.flatten(), parent.repeat(B)
        query, key, value = model.project(fed)
        sv.cache_append(cache, key, value, rows, length, table, B=B, max_rows=n, status=status)
        att = sv.cache_attend_tree(cache, query.to(dtype), rows, length + n, table, parent, B=B, k_max=n - 1, status=status)
        logits = att["out"].flatten(1) @ model.head.to(dtype)
        node = fed.int()
        if penalties:
            logits = sv.adjust_logits(logits, rows, V=V, B=B, k_max=n - 1, history=history, n_tokens=length + 1, n_prompt=n_prompt,
                                      node_token=node, parent=parent, allowed=allowed, allowed_row=allowed_row, status=status,
                                      **rule)["logits"]
        want = sv.verify_greedy(logits, rows, node, V=V, B=B, k_max=n - 1)["row_token"]
        got = sv.tree_accept(want, node, parent, rows, B=B, k_max=n - 1, status=status)
        # the path's keys and values once more, from the root's slot on (its rows behind the last accepted repeat that one,
        # in slots that the next step overwrites)
        at = got["path_rows"][:, :depth + 1].flatten().long()
        sv.cache_append(cache, key[at], value[at], path, length, table, B=B, max_rows=depth + 1, status=status)
        kept = got["accepted_len"] + 1
        new = got["out_tokens"][:, :depth + 1]
        slot = length[:, None].long() + 1 + torch.arange(depth + 1, device="cuda")
        history.scatter_(1, slot, torch.where(new >= 0, new, history.gather(1, slot)))
        length, root = length + kept, got["next_token"]
        accepted += int(got["accepted_len"].sum())
        for b, row in enumerate(new.tolist()):
            out[b] += [t for t in row if t >= 0]
    assert int(status) == 0
    return out, accepted


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    sv.build()
    out, accepted = run(a.steps)
    for b, t in enumerate(out):
        print("request %d: %d tokens, last %s" % (b, len(t), t[-5:]))
    print("%d drafts accepted in %d steps of %d requests" % (accepted, a.steps, len(out)))
