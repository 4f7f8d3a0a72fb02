"""The operators of a step with a tree of drafts: what is measured, and their
plain forms.

A prompt attends over itself (`prompt`); then, step by step, the nodes of a
tree of drafted tokens attend over the 4-bit paged cache and their ancestors
(`tree`), their logits get penalties, biases and grammar masks (`logits`), and
the path that the target's own tokens take through the tree is accepted
(`accept`).

`own` selects the side: False computes each operator in elementary torch
operations in 32 bits; True calls the library's entry points.

Cache layout (uint8): [page][kv head][block of 32 tokens][36 * D bytes], a
block holding
    K codes  [D/32][32 tokens][16]   byte j of a chunk: channels 2j (low nibble), 2j+1
    K scales [32 tokens][D/16]       e4m3, one per 16 channels of a token
    V codes  [D][16]                 byte j of a channel: tokens 2j (low nibble), 2j+1
    V scales [D/16][32 tokens]       e4m3
A code is e2m1 (sign, 2 exponent bits, 1 mantissa bit); a value is code * scale.
"""
import math

import numpy as np
import torch

own = False

TOK = 32                                    # tokens of a cache block
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------- cases ---

def _prompt(**kw):
    base = dict(op="prompt", B=1, rows=512, past=0, Hq=40, Hkv=8, D=128, dtype="bf16", ragged=True, cap=0.0,
                slopes=False, window=0, prefix=0)
    base.update(kw)
    return base


def _tree(**kw):
    base = dict(op="tree", B=1, rows=13, Hq=40, Hkv=8, D=128, len=1024, page=64, dtype="bf16", ragged=True, cap=0.0,
                slopes=False, window=0, prefix=0, gaps=False)
    base.update(kw)
    return base


def _logits(**kw):
    base = dict(op="logits", B=1, rows=1, V=152064, history=300, dtype="bf16", ragged=True, penalties=True, tree=True,
                mask=True, bias=8)
    base.update(kw)
    return base


def listed():
    return [
        # a short question: latency alone
        _prompt(name="prompt_one", rows=37, Hq=32, ragged=False),
        # prompts of odd lengths entering a server at once
        _prompt(name="prompt_batch", B=16, rows=4096),
        # one long document
        _prompt(name="prompt_long", rows=20011, Hq=32, ragged=False),
        # pieces of long prompts over what came before: capped scores, a window and an always-visible prefix, wide heads
        _prompt(name="prompt_pieces", B=6, rows=1000, past=9000, Hq=16, Hkv=4, D=256, cap=30.0, window=4096, prefix=4),
        # a small model in fp32 with distance biases, one kv head per query head
        _prompt(name="prompt_f32", B=5, rows=700, Hq=12, Hkv=12, D=64, dtype="f32", slopes=True),
        # a tree of 13 drafts for one short chat: latency alone
        _tree(name="tree_one", Hq=32, len=900, ragged=False),
        # a serving batch, trees of up to 26 nodes over ragged contexts
        _tree(name="tree_batch", B=64, rows=26, len=4096),
        # large trees over long documents in fp32: capped scores, a window and an always-visible prefix, over caches that
        # have lost tokens (positions with gaps)
        _tree(name="tree_long", B=3, rows=32, Hq=16, Hkv=4, D=64, len=60000, page=128, dtype="f32", cap=30.0,
              window=50000, prefix=4, gaps=True),
        # one token of one chat: latency alone
        _logits(name="logits_one", mask=False, ragged=False),
        # the benchmark batch's verify rows: 128 requests x 5 rows, histories of 4096 tokens, every second row under a grammar
        _logits(name="logits_batch", B=128, rows=5, history=4096, ragged=False),
        # one tree: latency alone
        dict(name="accept_one", op="accept", B=1, rows=8, V=152064, ragged=False),
        # as many requests as a large deployment verifies at once
        dict(name="accept_batch", op="accept", B=4096, rows=32, V=152064, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "logits", "logits", "accept"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    ragged = rng.random() < 0.7
    options = dict(cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.25,
                   window=rng.choice([0, 0, _log_int(rng, 1, 5000)]), prefix=rng.randint(0, 5))
    if op == "prompt":
        B = _log_int(rng, 1, 64)
        # at most 4e11 (f32: 4e10) flops of visible pairs, were every request of full length
        most = (4e10 if dtype == "f32" else 4e11) / (4.0 * D * Hq * B)
        past = rng.choice([0, 0, _log_int(rng, 1, 20000)])
        top = int((math.sqrt(past * past + 2 * most) - past))
        rows = _log_int(rng, 1, max(2, min(16000, 120000 // B, top)))
        return _prompt(B=B, rows=rows, past=past, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, ragged=ragged, **options)
    if op == "tree":
        B, rows = _log_int(rng, 1, 96), rng.randint(1, 32)
        n = _log_int(rng, 8, max(64, min(60000, 200000 * 8 // (B * Hkv * max(1, rows * Hq // Hkv // 20)))))
        return _tree(B=B, rows=rows, Hq=Hq, Hkv=Hkv, D=D, len=n, page=rng.choice([32, 64, 96, 128, 256]), dtype=dtype,
                     ragged=ragged, gaps=rng.random() < 0.3, **options)
    if op == "logits":
        V = _log_int(rng, 500, 260000)
        rows = rng.choice([1, 1, rng.randint(1, 32)])
        B = _log_int(rng, 1, max(1, min(256, 90000000 // (V * rows))))
        return _logits(B=B, rows=rows, V=V, history=_log_int(rng, 1, max(2, min(60000, 500000 // B))) - 1, dtype=dtype,
                       ragged=ragged, penalties=rng.random() < 0.8, tree=rng.random() < 0.5, mask=rng.random() < 0.6,
                       bias=rng.choice([0, 3, 300]))
    return dict(op="accept", B=_log_int(rng, 1, 4096), rows=rng.randint(1, 32), V=_log_int(rng, 500, 260000), ragged=ragged)


def _spread(n, most, least):
    """n sizes spread evenly over (least, most], in no order."""
    return [max(least, 1 + int((most - 1) * (((b + 1) * 0.6180339887) % 1.0))) if most else 0 for b in range(n)]


def _rows_of(c):
    """Rows of each request: prompts of odd lengths, or the nodes of its tree."""
    return _spread(c["B"], c["rows"], 1) if c["ragged"] else [c["rows"]] * c["B"]


def _keys_of(c):
    """Keys of each request: of a prompt's piece what came before too, of a tree's cache its own nodes too."""
    rows = _rows_of(c)
    if c["op"] == "prompt":
        past = _spread(c["B"], c["past"], 0) if c["ragged"] else [c["past"]] * c["B"]
        return [p + r for p, r in zip(past[::-1], rows)]
    lens = _spread(c["B"], c["len"], 1) if c["ragged"] else [c["len"]] * c["B"]
    return [max(n, r) for n, r in zip(lens, rows[::-1])] if c["op"] == "tree" else lens


def _history_of(c):
    return _spread(c["B"], c["history"], 0) if c["ragged"] else [c["history"]] * c["B"]


def _tree_rows(c):
    """Nodes of each request's tree (a large context goes with a small tree)."""
    return [min(r, n) for r, n in zip(_rows_of(c)[::-1], _keys_of(c))] if c["op"] == "tree" else _rows_of(c)


# -------------------------------------------------------------- inputs ---

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cu(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _trees(rows, seed):
    """Packed parents: node 0 of a request is its root, another hangs on some node before it, most on a recent one; now and
    then one hangs on none (a slot that the draft left unused)."""
    rng, out = np.random.default_rng(seed), []
    for n in rows:
        j = np.arange(n)
        up = np.minimum(rng.geometric(0.4, n), np.maximum(j, 1))
        p = np.where(rng.random(n) < 0.3, (rng.random(n) * np.maximum(j, 1)).astype(np.int64), j - up)
        p[rng.random(n) < 0.02] = -1
        p[:1] = -1
        out.append(p)
    return _i32(np.concatenate(out))


def _prepare_prompt(c, gen):
    rows, keys, dt = _rows_of(c), _keys_of(c), DTYPES[c["dtype"]]
    # queries and keys come out of one product, side by side; some channels of the keys are larger, as keys have
    chan = 1.0 + 3.0 * (torch.rand(c["Hkv"], c["D"], generator=gen, device="cuda") > 0.95)
    rand = lambda n, h: torch.randn(n, h, c["D"], generator=gen, device="cuda")
    st = dict(case=c, q=rand(sum(rows), c["Hq"]).to(dt), k=(rand(sum(keys), c["Hkv"]) * chan).to(dt),
              v=rand(sum(keys), c["Hkv"]).to(dt), cu=_cu(rows), cu_keys=_cu(keys) if c["past"] else None, slopes=None)
    if c["slopes"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["Hq"] + 1, device="cuda") / c["Hq"])
    return st


def _prepare_tree(c, gen, seed):
    """A pool of pages, each request's slots up to its length filled with codes and moderate scales (what lies behind them
    is whatever the memory held, NaN scales among it)."""
    B, H, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    rows, lens = _tree_rows(c), _keys_of(c)
    per = max(1, -(-max(lens) // page))
    total = B * per + 3
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table = order[:B * per].view(B, per).contiguous()
    pages = torch.randint(0, 256, (total, H, page // TOK, 36 * D), generator=gen, device="cuda", dtype=torch.uint8)
    live = torch.zeros(total, page, dtype=torch.bool, device="cuda")
    slot = torch.arange(per * page, device="cuda")
    live[table.long()] = (slot < torch.tensor(lens, device="cuda")[:, None]).view(B, per, page)
    live = live.view(total, 1, page // TOK, TOK)
    for at, shape in [(16 * D, (TOK, D // 16)), (34 * D, (D // 16, TOK))]:
        part = pages[..., at:at + 2 * D]
        scale = torch.randint(0x20, 0x32, (*pages.shape[:3], *shape), generator=gen, device="cuda", dtype=torch.uint8)
        ok = live[..., None] if shape[0] == TOK else live[..., None, :]
        part.copy_(torch.where(ok, scale, torch.full_like(scale, 0x7F)).flatten(-2))
    q = torch.randn(sum(rows), c["Hq"], D, generator=gen, device="cuda").to(DTYPES[c["dtype"]])
    st = dict(case=c, pages=pages, table=table, q=q, cu=_cu(rows), lens=_i32(lens), parent=_trees(rows, seed), slopes=None,
              pos=None)
    if c["slopes"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["Hq"] + 1, device="cuda") / c["Hq"])
    if c["gaps"]:
        step = torch.randint(1, 4, (B, per * page), generator=gen, device="cuda")
        st["pos"] = torch.zeros(total, page, dtype=torch.int32, device="cuda")
        st["pos"][table.long().flatten()] = (step.cumsum(1) - 1).int().view(-1, page)
    return st


def _tokens(gen, n, V):
    """Token ids as text has them: a few come again and again."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(V)) - 1).long().clamp(0, V - 1).mul(48271).remainder(V).int()


def _prepare_logits(c, gen, seed):
    B, V, rows, hist, dt = c["B"], c["V"], _rows_of(c), _history_of(c), DTYPES[c["dtype"]]
    R, width = sum(rows), max(1, max(hist))
    f = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=gen, device="cuda")
    st = dict(case=c, logits=(3.0 * torch.randn(R, V, generator=gen, device="cuda")).to(dt), cu=_cu(rows), parent=None)
    st["node_token"] = _tokens(gen, R, V)
    if c["tree"]:
        st["parent"] = _trees(rows, seed)
    if c["penalties"]:
        st.update(history=_tokens(gen, B * width, V).view(B, width), n_tokens=_i32(hist), n_prompt=_i32([n // 2 for n in hist]),
                  repetition=f(1.0, 1.4), frequency=f(-0.2, 0.8), presence=f(0.0, 0.6))
    if c["bias"]:
        st.update(bias_ids=torch.randint(0, V, (B * c["bias"],), generator=gen, device="cuda").int(),
                  bias_values=4.0 * torch.randn(B * c["bias"], generator=gen, device="cuda"),
                  bias_cu=torch.arange(0, B * c["bias"] + 1, c["bias"], dtype=torch.int32, device="cuda"))
    if c["mask"]:
        # a grammar for every second row: few tokens allowed, many, or none
        words = (V + 31) // 32
        some = torch.arange(0, R, 2, device="cuda")
        share = torch.rand(len(some), 1, generator=gen, device="cuda").pow(3)
        share[::7] = 0.0
        bits = torch.zeros(len(some), words, dtype=torch.int64, device="cuda")
        for i in range(32):
            bits |= (torch.rand(len(some), words, generator=gen, device="cuda") < share).long() << i
        bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits)
        st["allowed"] = bits.int()
        st["allowed_row"] = torch.full((R,), -1, dtype=torch.int32, device="cuda")
        st["allowed_row"][some] = torch.randperm(len(some), generator=gen, device="cuda").int()
    return st


def _prepare_accept(c, gen, seed):
    rows = _rows_of(c)
    R, rng = sum(rows), np.random.default_rng(seed)
    parent, token = _trees(rows, seed), rng.integers(0, c["V"], R)
    # the target's token at a row is one of the drafts on it three times in four
    up, want = parent.cpu().numpy(), rng.integers(0, c["V"], R)
    base = np.repeat(np.cumsum([0] + rows[:-1]), rows)
    child = np.flatnonzero((up >= 0) & (rng.random(R) < 0.75))
    want[base[child] + up[child]] = token[child]
    return dict(case=c, row_token=_i32(want), node_token=_i32(token), parent=parent, cu=_cu(rows))


def prepare(case, seed):
    c, gen = dict(case), _generator(seed)
    if c["op"] == "prompt":
        return _prepare_prompt(c, gen)
    if c["op"] == "tree":
        return _prepare_tree(c, gen, seed)
    if c["op"] == "logits":
        return _prepare_logits(c, gen, seed)
    return _prepare_accept(c, gen, seed)


# --------------------------------------------------------- plain forms ---

def _softmax_values(s, v):
    """out and log-sum-exp of scores [..., rows, keys] over values [..., keys, D]; rows of -inf alone: 0 and -inf."""
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.clamp(min=1e-37), (m + torch.log(total))[..., 0]


def _run_prompt(st):
    c = st["case"]
    H, D, group = c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    q, k, v = (st[n].float() for n in "qkv")
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    r0 = k0 = 0
    for n, m in zip(_rows_of(c), _keys_of(c)):
        step = max(1, (1 << 28) // (m * c["Hq"]))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            seen = m - n + i1                                            # keys that some row of the piece sees
            qq = q[r0 + i0:r0 + i1].view(i1 - i0, H, group, D).permute(1, 2, 0, 3).reshape(H, -1, D)
            kk, vv = (x[k0:k0 + seen].transpose(0, 1) for x in (k, v))
            s = (qq @ kk.transpose(1, 2)).view(H, group, i1 - i0, seen) / math.sqrt(D)
            if c["cap"] > 0:
                s = c["cap"] * torch.tanh(s / c["cap"])
            j = torch.arange(seen, device="cuda")
            dist = (m - n + torch.arange(i0, i1, device="cuda"))[:, None] - j
            if st["slopes"] is not None:
                s = s - st["slopes"].view(H, group, 1, 1) * dist.float()
            see = dist >= 0
            if c["window"] > 0:
                see = see & ((dist < c["window"]) | (j < c["prefix"]))
            s = torch.where(see, s, float("-inf")).flatten(1, 2)
            o, l = _softmax_values(s, vv)
            out[r0 + i0:r0 + i1] = o.view(H, group, i1 - i0, D).permute(2, 0, 1, 3).flatten(1, 2)
            lse[r0 + i0:r0 + i1] = l.view(H, group, i1 - i0).permute(2, 0, 1).flatten(1, 2)
        r0, k0 = r0 + n, k0 + m
    return {"out": out.to(DTYPES[c["dtype"]]), "lse": lse}


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _dense(st):
    """Keys and values of every request as fp32 [B, H, L, D]."""
    D = st["case"]["D"]
    blocks = st["pages"][st["table"].long()].transpose(1, 2).flatten(2, 3)          # [B, H, blocks, 36 D]
    kb, ks, vb, vs = blocks.split([16 * D, 2 * D, 16 * D, 2 * D], -1)
    lead = blocks.shape[:-1]
    kb = kb.reshape(*lead, D // 32, TOK, 16).transpose(-3, -2).reshape(*lead, TOK, D // 2)
    vb = vb.reshape(*lead, D, 16)
    lut = torch.tensor(_E2M1, device="cuda")
    scale = lambda x: x.contiguous().view(torch.float8_e4m3fn).float()
    k = lut[torch.stack([kb & 15, kb >> 4], -1).flatten(-2).int()]
    k = (k.unflatten(-1, (-1, 16)) * scale(ks).view(*lead, TOK, D // 16, 1)).flatten(-2)
    v = lut[torch.stack([vb & 15, vb >> 4], -1).flatten(-2).int()]
    v = (v.unflatten(-2, (-1, 16)) * scale(vs).view(*lead, D // 16, 1, TOK)).flatten(-3, -2)
    return k.flatten(2, 3), v.transpose(-1, -2).flatten(2, 3)


def _ancestors(st, rows):
    """[B, rows, rows]: whether node i is node j's ancestor or j itself, and the nodes' depths; rows past a tree's: none."""
    cu, parent = st["cu"].long(), st["parent"].long()
    B, j = cu.numel() - 1, torch.arange(rows, device="cuda")
    real = j < (cu[1:] - cu[:-1])[:, None]
    p = torch.where(real, parent[(cu[:-1, None] + j).clamp(max=parent.numel() - 1)], -1)
    anc = torch.eye(rows, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    for i in range(1, rows):
        up = anc.gather(1, p[:, i, None, None].clamp(min=0).expand(-1, 1, rows))[:, 0]
        anc[:, i] |= up & (p[:, i, None] >= 0)
    return anc, anc.sum(-1) - 1, real


def _run_tree(st):
    c = st["case"]
    B, H, D, rows, group = c["B"], c["Hkv"], c["D"], c["rows"], c["Hq"] // c["Hkv"]
    cu, lens = st["cu"].long(), st["lens"].long()
    anc, depth, real = _ancestors(st, rows)
    j = torch.arange(rows, device="cuda")
    q = st["q"].float()[(cu[:-1, None] + j).clamp(max=st["q"].shape[0] - 1)]
    q = q.view(B, rows, H, group, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    k, v = _dense(st)
    L = k.shape[2]
    s = (q @ k.transpose(-1, -2)).view(B, H, rows, group, L) / math.sqrt(D)
    if c["cap"] > 0:
        s = c["cap"] * torch.tanh(s / c["cap"])
    slot = torch.arange(L, device="cuda")
    root = lens - (cu[1:] - cu[:-1])                                     # slot of the tree's first node
    pos = slot.expand(B, L) if st["pos"] is None else st["pos"].long()[st["table"].long()].view(B, L)
    node = (slot - root[:, None]).clamp(0, rows - 1)
    in_tree = (slot >= root[:, None]) & (slot < lens[:, None])
    base = pos.gather(1, root[:, None])
    pos = torch.where(in_tree, base + depth.gather(1, node), pos)
    dist = (base + depth)[:, :, None] - pos[:, None]                     # [B, rows, L]
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, H, 1, group, 1) * dist[:, None, :, None].float()
    see = (slot < root[:, None])[:, None] | (in_tree[:, None] & anc.gather(2, node[:, None].expand(-1, rows, -1)))
    if c["window"] > 0:
        see = see & ((dist < c["window"]) | (slot < c["prefix"]))
    s = torch.where((see & real[:, :, None])[:, None, :, None], s, float("-inf"))
    v = torch.where((slot < lens[:, None])[:, None, :, None], v, 0.0)
    o, lse = _softmax_values(s.flatten(2, 3), v)
    o = o.view(B, H, rows, group, D).permute(0, 2, 1, 3, 4).flatten(2, 3)[real]
    lse = lse.view(B, H, rows, group).permute(0, 2, 1, 3).flatten(2, 3)[real]
    return {"out": o.to(DTYPES[c["dtype"]]), "lse": lse}


def _run_logits(st):
    c = st["case"]
    R, V, B, rows = st["logits"].shape[0], c["V"], c["B"], c["rows"]
    z = st["logits"].float()
    cu = st["cu"].long()
    r = torch.arange(R, device="cuda")
    owner = torch.searchsorted(cu, r, right=True) - 1
    if c["penalties"]:
        # how often each token came, in all and among the generated ones
        at = torch.arange(st["history"].shape[1], device="cuda")
        tok = st["history"].long()
        live, new = at < st["n_tokens"][:, None], at >= st["n_prompt"][:, None]
        seen = torch.zeros(B, V, device="cuda").scatter_add_(1, tok, live.float())
        made = torch.zeros(B, V, device="cuda").scatter_add_(1, tok, (live & new).float())
        seen, made = seen[owner], made[owner]
        # the drafts between the root and a row count as generated
        if st["parent"] is None:
            j = torch.arange(rows, device="cuda")
            anc = (j <= j[:, None]).expand(B, rows, rows)
            hung = anc & (j > 0)
        else:
            anc, _, _ = _ancestors(st, rows)
            p = st["parent"].long()[(cu[:-1, None] + torch.arange(rows, device="cuda")).clamp(max=R - 1)]
            hung = anc & (p >= 0)[:, None]
        token = st["node_token"].long()[(cu[:-1, None] + torch.arange(rows, device="cuda")).clamp(max=R - 1)]
        path = hung[owner, r - cu[owner]].float()
        seen.scatter_add_(1, token[owner], path)
        made.scatter_add_(1, token[owner], path)
        rep = st["repetition"][owner][:, None]
        z = torch.where(seen > 0, torch.where(z > 0, z / rep, z * rep), z)
        z = z - st["frequency"][owner][:, None] * made - st["presence"][owner][:, None] * (made > 0).float()
    if c["bias"]:
        bias = torch.zeros(B, V, device="cuda")
        bias.scatter_add_(1, st["bias_ids"].long().view(B, -1), st["bias_values"].view(B, -1))
        z = z + bias[owner]
    if c["mask"]:
        m = st["allowed_row"].long()
        w = st["allowed"][m.clamp(min=0)]
        bit = (w[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        ok = (bit.flatten(1)[:, :V] == 1) | (m < 0)[:, None]
        z = torch.where(ok, z, float("-inf"))
    return {"logits": z.to(DTYPES[c["dtype"]])}


def _run_accept(st):
    c = st["case"]
    B, rows = c["B"], c["rows"]
    cu = st["cu"].long()
    j = torch.arange(rows, device="cuda")
    real = j < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + j).clamp(max=st["parent"].numel() - 1)
    parent = torch.where(real, st["parent"].long()[at], -1)
    token, want = st["node_token"].long()[at], st["row_token"].long()[at]
    here = torch.zeros(B, 1, dtype=torch.long, device="cuda")
    going = torch.ones(B, 1, dtype=torch.bool, device="cuda")
    out = torch.full((B, rows), -1, dtype=torch.long, device="cuda")
    path = torch.zeros(B, rows, dtype=torch.long, device="cuda")
    length = torch.zeros(B, 1, dtype=torch.long, device="cuda")
    for i in range(rows):
        t = want.gather(1, here)
        out[:, i:i + 1] = torch.where(going, t, -1)
        path[:, i:i + 1] = here
        hit = (parent == here) & (token == t) & (j > 0)
        going = going & hit.any(1, keepdim=True)
        here = torch.where(going, hit.float().argmax(1, keepdim=True), here)
        length += going
    return {"accepted_len": length[:, 0].int(), "out_tokens": out.int(), "next_token": want.gather(1, here)[:, 0].int(),
            "path_rows": (cu[:-1, None] + path).int()}


def run(state):
    if not own:
        return {"prompt": _run_prompt, "tree": _run_tree, "logits": _run_logits, "accept": _run_accept}[state["case"]["op"]](state)
    call = state.get("call")
    if call is None:
        # the handle that a serving loop keeps: arguments marshalled once, workspace and outputs its own
        call = state["call"] = _call(state)
    res = call()
    return {n: res[n] for n in OUTPUTS[state["case"]["op"]]}


OUTPUTS = {"prompt": ("out", "lse"), "tree": ("out", "lse"), "logits": ("logits",),
           "accept": ("accepted_len", "out_tokens", "next_token", "path_rows")}


def _call(st):
    import speculative_decoding_verification_ragged_gb300 as sv
    c = st["case"]
    if c["op"] == "prompt":
        return sv.prompt_attend(st["q"], st["k"], st["v"], st["cu"], B=c["B"], cu_keys=st["cu_keys"], cap=c["cap"],
                                slopes=st["slopes"], window=c["window"], prefix=c["prefix"], prepared=True)
    if c["op"] == "tree":
        return sv.cache_attend_tree(sv.PagedCache(st["pages"]), st["q"], st["cu"], st["lens"], st["table"], st["parent"],
                                    B=c["B"], k_max=c["rows"] - 1, cap=c["cap"], slopes=st["slopes"], window=c["window"],
                                    prefix=c["prefix"], slot_pos=st["pos"], prepared=True)
    if c["op"] == "logits":
        names = ("history", "n_prompt", "n_tokens", "repetition", "frequency", "presence", "bias_cu", "bias_ids",
                 "bias_values", "allowed", "allowed_row")
        return sv.adjust_logits(st["logits"], st["cu"], V=c["V"], B=c["B"], k_max=c["rows"] - 1, node_token=st["node_token"],
                                parent=st["parent"], prepared=True, **{n: st.get(n) for n in names})
    return sv.tree_accept(st["row_token"], st["node_token"], st["parent"], st["cu"], B=c["B"], k_max=c["rows"] - 1,
                          prepared=True)


# ------------------------------------------------------ what it must do ---

def _visible(n, m, window, prefix):
    """Pairs of a request's rows and the keys that each sees."""
    i = np.arange(m - n, m, dtype=np.float64)
    if window <= 0:
        return float((i + 1).sum())
    near = np.minimum(i + 1, window)
    return float((near + np.minimum(np.maximum(i + 1 - window, 0), prefix)).sum())


def work(case):
    c = case
    elt = 2 if c.get("dtype", "bf16") == "bf16" else 4
    rows = _tree_rows(c)
    if c["op"] == "accept":
        return {"bytes": 12 * sum(rows) + c["B"] * (8 * c["rows"] + 12), "flops": 0}
    if c["op"] == "logits":
        n = sum(rows)
        words = 4 * ((c["V"] + 31) // 32)
        extra = (4 * sum(_history_of(c)) if c["penalties"] else 0) + (8 * c["B"] * c["bias"]) + (-(-n // 2) * words if c["mask"] else 0)
        return {"bytes": 2 * n * c["V"] * elt + extra + 8 * n, "flops": 4.0 * n * c["V"]}
    keys = _keys_of(c)
    qo = sum(rows) * c["Hq"] * (2 * c["D"] * elt + 4)
    if c["op"] == "prompt":
        seen = [min(m, c["window"] + n - 1 + c["prefix"]) if c["window"] > 0 else m for n, m in zip(rows, keys)]
        pairs = sum(_visible(n, m, c["window"], c["prefix"]) for n, m in zip(rows, keys)) * c["Hq"]
        return {"bytes": qo + sum(seen) * 2 * c["Hkv"] * c["D"] * elt, "flops": 4 * pairs * c["D"]}
    tok = 1.125 * c["D"] * c["Hkv"] + (4 if c["gaps"] else 0)
    seen = keys
    if c["window"] > 0:                     # with gaps positions advance by 2 a token on average
        near = c["window"] // (2 if c["gaps"] else 1)
        seen = [min(m, near + n - 1 + c["prefix"]) for n, m in zip(rows, keys)]
    pairs = float(sum(n * m for n, m in zip(rows, seen))) * c["Hq"]
    return {"bytes": sum(seen) * tok + qo, "flops": 4 * pairs * c["D"]}


# ------------------------------------------------- the definition in 64 bits ---

def _exact_attention(q, k, v, dist, see, c, slopes):
    """q [rows, group, D], k and v [keys, D], dist and see [rows, keys], all in 64 bits."""
    s = torch.einsum("rgd,nd->rgn", q, k) * c["D"] ** -0.5
    if c["cap"] > 0:
        s = c["cap"] * torch.tanh(s / c["cap"])
    if slopes is not None:
        s = s - slopes.double()[None, :, None] * dist.double()[:, None]
    s = s.masked_fill(~see[:, None], float("-inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.where(lse[..., None] > float("-inf"), torch.exp(s - lse[..., None]), 0.0)
    return torch.einsum("rgn,nd->rgd", p, v), lse


def _exact_prompt(st):
    c = st["case"]
    H, group = c["Hkv"], c["Hq"] // c["Hkv"]
    rows, keys = _rows_of(c), _keys_of(c)
    if sum(float(n) * (m - n / 2) for n, m in zip(rows, keys)) * 4 * c["D"] * c["Hq"] > 6e12:
        return None
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    r0 = k0 = 0
    for n, m in zip(rows, keys):
        step = max(1, (1 << 26) // (m * group))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            upto = m - n + i1
            dist = torch.arange(m - n + i0, upto, device="cuda")[:, None] - torch.arange(upto, device="cuda")[None]
            see = dist >= 0
            if c["window"] > 0:
                see &= (dist < c["window"]) | (torch.arange(upto, device="cuda") < c["prefix"])
            for h in range(H):
                g = slice(h * group, (h + 1) * group)
                o, l = _exact_attention(st["q"][r0 + i0:r0 + i1, g].double(), st["k"][k0:k0 + upto, h].double(),
                                        st["v"][k0:k0 + upto, h].double(), dist, see, c,
                                        None if st["slopes"] is None else st["slopes"][g])
                out[r0 + i0:r0 + i1, g], lse[r0 + i0:r0 + i1, g] = o, l
        r0, k0 = r0 + n, k0 + m
    return {"out": out, "lse": lse}


def _e4m3(b):
    e, m = ((b >> 3) & 15).double(), (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    return torch.where(b >= 128, -x, x)


def _e2m1(code):
    e, m = ((code >> 1) & 3).double(), (code & 1).double()
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
    return torch.where(code >= 8, -x, x)


def _cached(st, b, h, n):
    """Keys and values of the first n tokens of request b, kv head h, as [n, D] in 64 bits."""
    c = st["case"]
    D = c["D"]
    t = torch.arange(n, device="cuda")
    raw = st["pages"][st["table"][b, t // c["page"]].long(), h, t % c["page"] // TOK].int()      # [n, 36 D]
    i, d = (t % TOK)[:, None], torch.arange(D, device="cuda")[None]
    kb = raw.gather(1, (d // 32) * 512 + i * 16 + d % 32 // 2)
    ks = raw.gather(1, 16 * D + i * (D // 16) + d // 16)
    vb = raw.gather(1, 18 * D + d * 16 + i // 2)
    vs = raw.gather(1, 34 * D + d // 16 * 32 + i)
    return _e2m1((kb >> (4 * (d % 2))) & 15) * _e4m3(ks), _e2m1((vb >> (4 * (i % 2))) & 15) * _e4m3(vs)


def _paths(parent):
    """For each node of one tree the set of its ancestors and itself."""
    out = []
    for j, p in enumerate(parent):
        out.append((out[p] if p >= 0 else []) + [j])
    return out


def _exact_tree(st):
    c = st["case"]
    rows, lens, group = _tree_rows(c), _keys_of(c), c["Hq"] // c["Hkv"]
    if sum(n * r for n, r in zip(lens, rows)) * c["Hq"] * c["D"] > 1e12:
        return None
    parent, r0, outs, lses = st["parent"].tolist(), 0, [], []
    for b, (r, n) in enumerate(zip(rows, lens)):
        root, paths = n - r, _paths(parent[r0:r0 + r])
        i = torch.arange(n, device="cuda")
        pos = i if st["pos"] is None else st["pos"][st["table"][b].long()].flatten()[:n].long()
        depth = torch.tensor([len(p) - 1 for p in paths], device="cuda")
        pos = torch.cat([pos[:root], pos[root] + depth])
        see = torch.zeros(r, n, dtype=torch.bool, device="cuda")
        see[:, :root] = True
        for j, p in enumerate(paths):
            see[j, [root + x for x in p]] = True
        dist = pos[root:][:, None] - pos[None]
        if c["window"] > 0:
            see &= (dist < c["window"]) | (i[None] < c["prefix"])
        o_b, l_b = [], []
        for h in range(c["Hkv"]):
            g = slice(h * group, (h + 1) * group)
            k, v = _cached(st, b, h, n)
            o, l = _exact_attention(st["q"][r0:r0 + r, g].double(), k, v, dist, see, c,
                                    None if st["slopes"] is None else st["slopes"][g])
            o_b.append(o)
            l_b.append(l)
        outs.append(torch.cat(o_b, 1))
        lses.append(torch.cat(l_b, 1))
        r0 += r
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_logits(st):
    c = st["case"]
    rows, hist, V = _rows_of(c), _history_of(c), c["V"]
    if sum(rows) * V > 3e8:
        return None
    out = st["logits"].double()
    token = st["node_token"].tolist()
    parent = st["parent"].tolist() if st["parent"] is not None else None
    r0 = 0
    for b, n in enumerate(rows):
        paths = _paths(parent[r0:r0 + n] if parent else range(-1, n - 1))
        if c["penalties"]:
            h = st["history"][b, :hist[b]].long()
            seen = torch.bincount(h, minlength=V).double()
            made = torch.bincount(h[hist[b] // 2:], minlength=V).double()
        if c["bias"]:
            bias = torch.zeros(V, dtype=torch.float64, device="cuda")
            bias.index_add_(0, st["bias_ids"][b * c["bias"]:(b + 1) * c["bias"]].long(),
                            st["bias_values"][b * c["bias"]:(b + 1) * c["bias"]].double())
        for j, p in enumerate(paths):
            z = out[r0 + j]
            if c["penalties"]:
                hung = [x for x in p if (parent[r0 + x] >= 0 if parent else x > 0)]
                s, m = seen.clone(), made.clone()
                for x in hung:
                    s[token[r0 + x]] += 1
                    m[token[r0 + x]] += 1
                rep = st["repetition"][b].double()
                z = torch.where(s > 0, torch.where(z > 0, z / rep, z * rep), z)
                z = z - st["frequency"][b].double() * m - st["presence"][b].double() * (m > 0)
            if c["bias"]:
                z = z + bias
            if c["mask"] and int(st["allowed_row"][r0 + j]) >= 0:
                v = torch.arange(V, device="cuda")
                w = st["allowed"][int(st["allowed_row"][r0 + j])].long()[v // 32]
                z = torch.where((w >> (v % 32)) % 2 == 1, z, float("-inf"))
            out[r0 + j] = z
        r0 += n
    return {"logits": out}


def exact(case, seed):
    if case["op"] == "accept":
        return None
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "tree": _exact_tree, "logits": _exact_logits}[case["op"]](st)
