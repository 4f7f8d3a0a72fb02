"""The 4-bit paged cache operators: what is measured, and their plain forms.

A speculative-decoding step appends each request's k_b + 1 new keys and
values to its cache, attends with those rows over the whole cache, and then
verifies the drafts.  When a cache outgrows its budget, the tokens with the
least accumulated attention weight are dropped.

`own` selects the side: False computes each operator in elementary torch
operations in 32 bits; True calls the library's entry points.

Cache layout (uint8): [page][kv head][block of 32 tokens][36 * D bytes], a
block holding
    K codes  [D/32][32 tokens][16]   byte j of a chunk: channels 2j (low nibble), 2j+1
    K scales [32 tokens][D/16]       e4m3, one per 16 channels of a token
    V codes  [D][16]                 byte j of a channel: tokens 2j (low nibble), 2j+1
    V scales [D/16][32 tokens]       e4m3
A code is e2m1 (sign, 2 exponent bits, 1 mantissa bit); a value is
code * scale * head_scale.
"""
import math

import numpy as np
import torch

own = False

TOK = 32                                    # tokens of a cache block
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------- cases ---

def _attn(**kw):
    base = dict(op="attend", B=1, rows=1, Hq=32, Hkv=8, D=128, len=1024, page=64, dtype="bf16",
                ragged=True, cap=0.0, slopes=False, window=0, prefix=0, gaps=False, scaled=False)
    base.update(kw)
    return base


def listed():
    return [
        # the decode step's append: 128 requests x up to 5 verify rows, into partly filled blocks
        dict(name="append_step", op="append", B=128, rows=5, Hkv=8, D=128, len=2048, page=64,
             dtype="bf16", ragged=True, scaled=False),
        # prompts of odd lengths entering the cache at once, fp32 keys, per-head scales
        dict(name="append_prompts", op="append", B=9, rows=6007, Hkv=8, D=64, len=0, page=128,
             dtype="f32", ragged=True, scaled=True),
        # one request, one token, a short chat: latency alone
        _attn(name="attend_one", len=700),
        # the verify step of the benchmark batch: 128 requests, k = 4, ragged contexts
        _attn(name="attend_verify", B=128, rows=5, Hq=40, len=4096),
        # few requests with long documents, plain decoding
        _attn(name="attend_long", B=4, len=131071, ragged=False, page=128),
        # k = 7 drafts, fp32, capped scores with a distance bias, a window and an always-visible
        # prefix, over a cache that has lost tokens (positions with gaps)
        _attn(name="attend_capped", B=16, rows=8, Hq=16, Hkv=4, D=64, len=8191, page=32, dtype="f32",
              cap=30.0, slopes=True, window=3000, prefix=4, gaps=True, scaled=True),
        # one shared kv head with wide channels (every query head reads the same cache)
        _attn(name="attend_wide", B=48, rows=3, Hq=8, Hkv=1, D=256, len=16000, page=96),
        # accumulating the verify rows' weights for eviction
        _attn(name="weights_verify", op="weights", B=64, rows=5, Hq=40, len=4096),
        # long contexts, one kv head per query head, single tokens
        _attn(name="weights_long", op="weights", B=2, Hq=16, Hkv=16, D=64, len=65533, ragged=False,
              cap=50.0, dtype="f32"),
        # a serving batch over its budget: half of each cache goes
        dict(name="evict_batch", op="evict", B=32, Hkv=8, D=128, len=4096, page=64, ragged=True,
             budget=2048, recent=64),
        # two long documents cut down to a quarter
        dict(name="evict_long", op="evict", B=2, Hkv=8, D=128, len=131072, page=128, ragged=False,
             budget=32768, recent=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weights", "evict"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([32, 64, 96, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        B = _log_int(rng, 1, 160)
        rows = _log_int(rng, 1, max(2, 20000 // B))
        return dict(op=op, B=B, rows=rows, Hkv=Hkv, D=D, len=_log_int(rng, 1, 2000) - 1, page=page,
                    dtype=dtype, ragged=rng.random() < 0.7, scaled=rng.random() < 0.5)
    B = _log_int(rng, 1, 128)
    if op == "evict":
        n = _log_int(rng, 40, max(64, 200000 // B))
        budget = max(1, int(n * rng.uniform(0.2, 1.05)))
        return dict(op=op, B=B, Hkv=Hkv, D=D, len=n, page=page, ragged=rng.random() < 0.7,
                    budget=budget, recent=rng.randint(0, min(budget, 200)))
    rows = rng.randint(1, 8)
    group = rng.choice([1, 2, 4, 5, 7, 8])
    n = _log_int(rng, 8, max(64, min(100000, 400000 * 8 // (B * Hkv * max(1, rows * group // 10)))))
    return _attn(op=op, B=B, rows=rows, Hq=Hkv * group, Hkv=Hkv, D=D, len=n, page=page, dtype=dtype,
                 ragged=rng.random() < 0.7, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                 slopes=rng.random() < 0.3, window=rng.choice([0, 0, _log_int(rng, 1, 5000)]),
                 prefix=rng.randint(0, 5), gaps=rng.random() < 0.3, scaled=rng.random() < 0.3)


def _rows_of(c):
    """Rows of each request: the draft lengths of a ragged batch, or prompts of odd lengths."""
    if not c["ragged"]:
        return [c["rows"]] * c["B"]
    if c["rows"] <= 8:
        return [max(1, c["rows"] - (5 * b) % 3) for b in range(c["B"])]
    return [max(1, int(c["rows"] * (((b + 1) * 0.6180339887) % 1.0))) for b in range(c["B"])]


def _lens_of(c):
    """Cache length of each request, spread evenly over (0, len] in a ragged batch."""
    if not c["ragged"] or c["len"] == 0:
        return [c["len"]] * c["B"]
    return [1 + int((c["len"] - 1) * (((b + 1) * 0.6180339887) % 1.0)) for b in range(c["B"])]


def _attn_lens(c):
    return [max(n, r) for n, r in zip(_lens_of(c), _rows_of(c))]


# -------------------------------------------------------------- inputs ---

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _quantise(x, g):
    """x [..., H, D] fp32 -> e2m1 codes [..., H, D] and e4m3 scales [..., H, D/16], both uint8.
    The scale is the block's largest magnitude over 6 (in units of the head's scale), rounded to
    e4m3; a code is the nearest e2m1 value, ties to the even code."""
    xb = x.unflatten(-1, (-1, 16))
    g = g[:, None]
    s = (xb.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = s.float() * g
    y = torch.where(den[..., None] > 0, xb / den[..., None], torch.zeros_like(xb))
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (torch.signbit(y)).to(torch.uint8)
    return code.flatten(-2), s.view(torch.uint8)


def _pack(kc, ks, vc, vs):
    """Codes and scales [n, 32, H, ...] of whole blocks -> bytes [n, H, 36 D]."""
    n, _, H, D = kc.shape
    k = (kc[..., 0::2] | (kc[..., 1::2] << 4)).view(n, TOK, H, D // 32, 16).permute(0, 2, 3, 1, 4)
    v = (vc[:, 0::2] | (vc[:, 1::2] << 4)).permute(0, 2, 3, 1)
    parts = [k, ks.permute(0, 2, 1, 3), v, vs.permute(0, 2, 3, 1)]
    return torch.cat([p.reshape(n, H, -1) for p in parts], -1)


def _unpack(blocks, D):
    """Bytes [..., 36 D] -> K codes [..., 32, D], K scales [..., 32, D/16], V alike (uint8)."""
    lead = blocks.shape[:-1]
    kb, ks, vb, vs = blocks.split([16 * D, 2 * D, 16 * D, 2 * D], -1)
    kb = kb.reshape(*lead, D // 32, TOK, 16).transpose(-3, -2).reshape(*lead, TOK, D // 2)
    kc = torch.stack([kb & 15, kb >> 4], -1).flatten(-2)
    vb = vb.reshape(*lead, D, 16)
    vc = torch.stack([vb & 15, vb >> 4], -1).flatten(-2).transpose(-1, -2)
    return kc, ks.reshape(*lead, TOK, D // 16), vc, vs.reshape(*lead, D // 16, TOK).transpose(-1, -2)


def _value(code, scale):
    """Codes [..., D] and e4m3 bytes [..., D/16] -> fp32 values (head scale not applied)."""
    lut = torch.tensor(_E2M1, device=code.device)
    x = lut[code.int()].unflatten(-1, (-1, 16)) * scale.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    return x.flatten(-2)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _filled_cache(c, gen, lens, pool_pages):
    """A pool of pages of which each request owns enough for `lens`, filled with normal keys and
    values (some channels of the keys larger, as keys have); what lies past a request's length is
    whatever the memory held."""
    B, H, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    nblk = page // TOK
    per = max(1, -(-max(lens) // page))
    total = max(pool_pages, B * per)
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table = order[:B * per].view(B, per).contiguous()
    pages = torch.randint(0, 256, (total, H, nblk, 36 * D), generator=gen, device="cuda", dtype=torch.uint8)
    scaled = c.get("scaled", False)
    g = (0.05 + 0.1 * torch.rand(2, H, generator=gen, device="cuda")) if scaled else torch.ones(2, H, device="cuda")
    chan = 1.0 + 3.0 * (torch.rand(H, D, generator=gen, device="cuda") > 0.95)
    blocks = -(-max(lens) // TOK) if max(lens) else 0
    for b0 in range(0, B if blocks else 0, max(1, (1 << 28) // max(1, blocks * TOK * H * D))):
        b1 = min(B, b0 + max(1, (1 << 28) // (blocks * TOK * H * D)))
        n = (b1 - b0) * blocks
        k = torch.randn(n, TOK, H, D, generator=gen, device="cuda") * chan
        v = torch.randn(n, TOK, H, D, generator=gen, device="cuda")
        packed = _pack(*_quantise(k, g[0]), *_quantise(v, g[1])).view(b1 - b0, blocks, H, -1)
        at = torch.arange(blocks, device="cuda")
        lens_t = torch.tensor(lens[b0:b1], device="cuda")
        live = at[None] * TOK < lens_t[:, None]
        pg = table[b0:b1].long()[:, at // nblk][live]
        # the values of a block past the request's length stay as the pool had them
        old = _unpack(pages[pg, :, (at % nblk)[None].expand(b1 - b0, -1)[live]], D)
        new = _unpack(packed[live], D)
        slot = (at[None] * TOK).expand(b1 - b0, -1)[live][:, None] + torch.arange(TOK, device="cuda")
        ok = (slot < lens_t[:, None].expand(-1, blocks)[live][:, None])[:, None, :, None]
        mix = [torch.where(ok, x, y).transpose(1, 2) for x, y in zip(new, old)]
        pages[pg, :, (at % nblk)[None].expand(b1 - b0, -1)[live]] = _pack(*mix)
    return dict(pages=pages, table=table, g=g, k_scale=g[0].contiguous() if scaled else None,
                v_scale=g[1].contiguous() if scaled else None)


def _cu(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, gen = dict(case), _generator(seed)
    if c["op"] == "append":
        rows, start = _rows_of(c), _lens_of(c)
        st = _filled_cache(c, gen, [a + r for a, r in zip(start, rows)], 0)
        R, dt = sum(rows), DTYPES[c["dtype"]]
        st.update(k=torch.randn(R, c["Hkv"], c["D"], generator=gen, device="cuda").to(dt),
                  v=torch.randn(R, c["Hkv"], c["D"], generator=gen, device="cuda").to(dt),
                  cu=_cu(rows), start=torch.tensor(start, dtype=torch.int32, device="cuda"), case=c)
        return st
    if c["op"] == "evict":
        lens = _lens_of(c)
        dper = -(-min(c["budget"], max(lens)) // c["page"])
        st = _filled_cache(c, gen, lens, 0)
        per = st["table"].shape[1]
        n = st["pages"].shape[0]
        st["pages"] = torch.cat([st["pages"], torch.zeros_like(st["pages"][:1]).expand(c["B"] * dper, -1, -1, -1)])
        total = n + c["B"] * dper
        # weights accumulated over some steps: most tokens light, a few heavy, some never looked at
        score = torch.empty(total, c["page"], device="cuda").exponential_(generator=gen).pow_(3)
        score *= torch.rand(total, c["page"], generator=gen, device="cuda") > 0.1
        score[n:] = 0
        pos = torch.zeros(total, c["page"], dtype=torch.int32, device="cuda")
        pos[st["table"].long().flatten()] = torch.arange(per * c["page"], dtype=torch.int32, device="cuda").view(per, -1).repeat(c["B"], 1)
        st.update(score=score, pos=pos, first=n, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), case=c,
                  dst=(n + torch.randperm(c["B"] * dper, generator=gen, device="cuda").int()).view(c["B"], dper).contiguous())
        return st
    rows, lens = _rows_of(c), _attn_lens(c)
    st = _filled_cache(c, gen, lens, 0)
    per = st["table"].shape[1]
    q = torch.randn(sum(rows), c["Hq"], c["D"], generator=gen, device="cuda").to(DTYPES[c["dtype"]])
    st.update(case=c, q=q, cu=_cu(rows), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), slopes=None, pos=None)
    if c["slopes"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["Hq"] + 1, device="cuda") / c["Hq"])
    if c["gaps"]:
        step = torch.randint(1, 4, (c["B"], per * c["page"]), generator=gen, device="cuda")
        st["pos"] = torch.zeros(st["pages"].shape[0], c["page"], dtype=torch.int32, device="cuda")
        st["pos"][st["table"].long().flatten()] = (step.cumsum(1) - 1).int().view(-1, c["page"])
    if c["op"] == "weights":
        st["score"] = torch.zeros(st["pages"].shape[0], c["page"], device="cuda")
        st["lse"] = _attend(st)["lse"]
    return st


# --------------------------------------------------------- plain forms ---

def _slots(st, n):
    """(page, block in page, slot in block) index of token slots `n` [...] of every request."""
    c = st["case"]
    page = st["table"].long()[torch.arange(c["B"], device="cuda").view(-1, *[1] * (n.dim() - 1)), n // c["page"]]
    return page, n % c["page"]


def _append(st):
    c = st["case"]
    H, D, page = c["Hkv"], c["D"], c["page"]
    kc, ks = _quantise(st["k"].float(), st["g"][0])
    vc, vs = _quantise(st["v"].float(), st["g"][1])
    R = kc.shape[0]
    r = torch.arange(R, device="cuda")
    owner = torch.searchsorted(st["cu"].long(), r, right=True) - 1
    slot = st["start"].long()[owner] + r - st["cu"].long()[owner]
    pg = st["table"].long()[owner, slot // page]
    h = torch.arange(H, device="cuda")
    base = ((pg[:, None] * H + h) * (page // TOK) + (slot % page // TOK)[:, None]) * (36 * D)
    t = (slot % TOK)[:, None, None]
    flat = st["pages"].view(-1)
    j = torch.arange(D // 2, device="cuda")
    flat[base[..., None] + (j // 16) * 512 + t * 16 + j % 16] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    j = torch.arange(D // 16, device="cuda")
    flat[base[..., None] + 16 * D + t * (D // 16) + j] = ks
    flat[base[..., None] + 34 * D + j * 32 + t] = vs
    at = base[..., None] + 18 * D + torch.arange(D, device="cuda") * 16 + t // 2
    odd = slot % 2 == 1
    flat[at[~odd]] = (flat[at[~odd]] & 0xF0) | vc[~odd]
    flat[at[odd]] = (flat[at[odd]] & 0x0F) | (vc[odd] << 4)
    dt = DTYPES[c["dtype"]]
    return {"k": (_value(kc, ks) * st["g"][0][:, None]).to(dt), "v": (_value(vc, vs) * st["g"][1][:, None]).to(dt)}


def _dense(st, which):
    """The cache of every request as fp32 [B, H, L, D]: keys (0) or values (1)."""
    c = st["case"]
    blocks = st["pages"][st["table"].long()]                        # [B, pages, H, blocks, bytes]
    parts = _unpack(blocks.transpose(1, 2).flatten(2, 3), c["D"])   # [B, H, blocks, 32, ...]
    x = _value(parts[2 * which], parts[2 * which + 1]) * st["g"][which][None, :, None, None, None]
    return x.flatten(2, 3)


def _scores(st):
    """Scores [B, H, rows, group, L] with everything hidden at -inf, and which rows are real."""
    c = st["case"]
    B, H, D, group = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    cu, lens = st["cu"].long(), st["lens"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(c["rows"], device="cuda")
    real = j[None] < n[:, None]
    q = st["q"].float()[(cu[:-1, None] + j).clamp(max=st["q"].shape[0] - 1)]
    q = q.view(B, c["rows"], H, group, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    k = _dense(st, 0)
    L = k.shape[2]
    s = (q @ k.transpose(-1, -2)).view(B, H, c["rows"], group, L) / math.sqrt(D)
    if c["cap"] > 0:
        s = c["cap"] * torch.tanh(s / c["cap"])
    slot = torch.arange(L, device="cuda")
    pos = slot.expand(B, L) if st["pos"] is None else st["pos"].long()[st["table"].long()].view(B, L)
    last = lens[:, None] - n[:, None] + j                            # own slot of each row
    dist = pos.gather(1, last.clamp(0, L - 1))[:, :, None] - pos[:, None]
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, H, 1, group, 1) * dist[:, None, :, None].float()
    see = slot <= last[:, :, None]
    if c["window"] > 0:
        see = see & ((dist < c["window"]) | (slot < c["prefix"]))
    see = see & real[:, :, None]
    return torch.where(see[:, None, :, None], s, float("-inf")), real


def _attend(st):
    c = st["case"]
    s, real = _scores(st)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - m)
    total = p.sum(-1)
    v = _dense(st, 1)
    L = v.shape[2]
    v = torch.where((torch.arange(L, device="cuda") < st["lens"][:, None])[:, None, :, None], v, 0.0)
    o = (p.flatten(2, 3) @ v).view(*p.shape[:4], -1) / total.clamp(min=1e-37)[..., None]
    lse = m[..., 0] + torch.log(total)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[real]
    return {"out": o.to(DTYPES[c["dtype"]]), "lse": lse.permute(0, 2, 1, 3).flatten(2, 3)[real]}


def _weights(st):
    c = st["case"]
    s, real = _scores(st)
    lse = torch.full((*real.shape, c["Hq"]), float("inf"), device="cuda")
    lse[real] = st["lse"]
    lse = lse.view(c["B"], c["rows"], c["Hkv"], -1).permute(0, 2, 1, 3)
    w = torch.exp(s - lse[..., None]).sum((1, 2, 3))                 # [B, L]
    st["score"][st["table"].long().flatten()] += w.view(-1, c["page"])
    return {"score": st["score"]}


def _evict(st):
    c = st["case"]
    B, H, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    L, lens = st["table"].shape[1] * page, st["lens"].long()
    budget = min(c["budget"], L)
    slot = torch.arange(L, device="cuda")
    live = slot < lens[:, None]
    key = st["score"][st["table"].long()].view(B, L)
    key = torch.where(slot >= lens[:, None] - c["recent"], float("inf"), key)
    key = torch.where(live, key, float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :budget]
    new = lens.clamp(max=c["budget"])
    order = torch.where(torch.arange(budget, device="cuda") < new[:, None], order, L).sort(1)[0]
    kept = torch.full((B, c["budget"]), -1, dtype=torch.int32, device="cuda")
    kept[:, :budget] = torch.where(order < L, order, -1).int()
    # move: whole blocks of kept tokens, the last one's tail zero
    dpages = st["dst"].shape[1]
    pad = torch.full((B, dpages * page), L, device="cuda")
    pad[:, :budget] = order[:, :dpages * page]
    ok = pad < L
    src = pad.clamp(max=L - 1)
    pg, at = _slots(st, src)
    blocks = st["pages"][st["table"].long()].transpose(1, 2).flatten(2, 3)      # [B, H, blocks, bytes]
    parts = [p.flatten(2, 3) for p in _unpack(blocks, D)]                      # [B, H, L, .]
    moved = [torch.where(ok[:, None, :, None], p.gather(2, src[:, None, :, None].expand(-1, H, -1, p.shape[-1])), 0)
             for p in parts]
    moved = [p.unflatten(2, (-1, TOK)).permute(0, 2, 3, 1, 4).flatten(0, 1) for p in moved]
    packed = _pack(*moved).view(B * dpages, page // TOK, H, -1).transpose(1, 2)
    dst = st["dst"].long().flatten()
    touched = torch.arange(dpages * page // TOK, device="cuda")[None] * TOK < new[:, None]
    touched = touched.view(B * dpages, page // TOK)
    st["pages"][dst] = torch.where(touched[:, None, :, None], packed, st["pages"][dst])
    tok = touched.repeat_interleave(TOK, 1)
    for x in (st["score"], st["pos"]):
        x[dst] = torch.where(tok, torch.where(ok, x[pg, at], 0).view(-1, page), x[dst])
    n = st["first"]
    return {"kept": kept, "new_len": new.int(), "pages": st["pages"][n:], "score": st["score"][n:], "pos": st["pos"][n:]}


def run(state):
    if not own:
        return {"append": _append, "attend": _attend, "weights": _weights, "evict": _evict}[state["case"]["op"]](state)
    calls = state.get("calls")
    if calls is None:
        # the handles that a serving loop keeps: arguments marshalled once, workspace and outputs its own
        calls = state["calls"] = _calls(state)
    res = [f() for f in calls]
    if state["case"]["op"] == "evict":
        n = state["first"]
        return {"kept": res[0]["kept"], "new_len": res[0]["new_len"], "pages": state["pages"][n:],
                "score": state["score"][n:], "pos": state["pos"][n:]}
    if state["case"]["op"] == "weights":
        return {"score": state["score"]}
    if state["case"]["op"] == "append":
        return res[1]
    return {"out": res[0]["out"], "lse": res[0]["lse"]}


def _calls(st):
    import speculative_decoding_verification_ragged_gb300 as sv
    c = st["case"]
    cache = sv.PagedCache(st["pages"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    if c["op"] == "append":
        n = dict(B=c["B"], max_rows=max(_rows_of(c)), prepared=True)
        return [sv.cache_append(cache, st["k"], st["v"], st["cu"], st["start"], st["table"], **n),
                sv.cache_read(cache, st["cu"], st["start"], st["table"], R_cap=st["k"].shape[0],
                              dtype=st["k"].dtype, **n)]
    if c["op"] == "evict":
        return [sv.cache_evict(cache, st["score"], st["lens"], st["table"], st["dst"], B=c["B"], budget=c["budget"],
                               recent=c["recent"], slot_pos=st["pos"], prepared=True)]
    kw = dict(B=c["B"], k_max=c["rows"] - 1, cap=c["cap"], slopes=st["slopes"], window=c["window"],
              prefix=c["prefix"], slot_pos=st["pos"], prepared=True)
    if c["op"] == "weights":
        return [sv.cache_weights(cache, st["q"], st["lse"], st["cu"], st["lens"], st["table"], st["score"], **kw)]
    return [sv.cache_attend(cache, st["q"], st["cu"], st["lens"], st["table"], **kw)]


# ------------------------------------------------------ what it must do ---

def work(case):
    c = case
    H, D = c["Hkv"], c["D"]
    tok = 1.125 * D * H                     # bytes of a token's keys and values
    if c["op"] == "append":
        n = sum(_rows_of(c))
        elt = 2 if c["dtype"] == "bf16" else 4
        # values in, cache out; cache back in, values out
        return {"bytes": 2 * n * (2 * H * D * elt + tok), "flops": 8.0 * n * H * D}
    if c["op"] == "evict":
        lens = _lens_of(c)
        kept = sum(min(n, c["budget"]) for n in lens)
        return {"bytes": 4 * sum(lens) + kept * (2 * tok + 16 + 4), "flops": 0}
    rows, lens = _rows_of(c), _attn_lens(c)
    elt = 2 if c["dtype"] == "bf16" else 4
    seen = lens
    if c["window"] > 0 and not c["gaps"]:
        seen = [min(n, c["window"] + r - 1 + c["prefix"]) for n, r in zip(lens, rows)]
    elif c["window"] > 0:                   # positions advance by 2 a token on average
        seen = [min(n, c["window"] // 2 + r - 1 + c["prefix"]) for n, r in zip(lens, rows)]
    if c["gaps"]:
        tok += 4
    pairs = float(sum(n * r for n, r in zip(seen, rows))) * c["Hq"]
    qo = sum(rows) * c["Hq"]
    if c["op"] == "weights":
        return {"bytes": sum(seen) * (tok / 2 + 8) + qo * (D * elt + 4), "flops": 2 * pairs * D}
    return {"bytes": sum(seen) * tok + qo * (2 * D * elt + 4), "flops": 4 * pairs * D}


# ------------------------------------------------- the definition in 64 bits ---

def _e4m3(b):
    e, m = ((b >> 3) & 15).double(), (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    return torch.where(b >= 128, -x, x)


def _e2m1(code):
    e, m = ((code >> 1) & 3).double(), (code & 1).double()
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
    return torch.where(code >= 8, -x, x)


def _tokens(st, b, h, n):
    """Keys and values of the first n tokens of request b, kv head h, as [n, D] in 64 bits."""
    c = st["case"]
    D, nblk = c["D"], c["page"] // TOK
    t = torch.arange(n, device="cuda")
    raw = st["pages"][st["table"][b, t // c["page"]].long(), h, t % c["page"] // TOK].int()      # [n, 36 D]
    i, d = (t % TOK)[:, None], torch.arange(D, device="cuda")[None]
    kb = raw.gather(1, (d // 32) * 512 + i * 16 + d % 32 // 2)
    ks = raw.gather(1, 16 * D + i * (D // 16) + d // 16)
    vb = raw.gather(1, 18 * D + d * 16 + i // 2)
    vs = raw.gather(1, 34 * D + d // 16 * 32 + i)
    k = _e2m1((kb >> (4 * (d % 2))) & 15) * _e4m3(ks) * st["g"][0][h].double()
    v = _e2m1((vb >> (4 * (i % 2))) & 15) * _e4m3(vs) * st["g"][1][h].double()
    return k, v


def _nearest(x, grid):
    """The grid value nearest to x (the grid is ascending; ties go to the even index)."""
    i = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    up = (hi < lo) | ((hi == lo) & (i % 2 == 0))
    return grid[torch.where(up, i, i - 1)]


def _exact_quantised(x, g):
    e4 = _e4m3(torch.arange(127, device="cuda"))
    e2 = _e2m1(torch.arange(8, device="cuda"))
    x = x.double().unflatten(-1, (-1, 16))
    den = _nearest((x.abs().amax(-1) / (6 * g.double()[:, None])).clamp(max=448), e4) * g.double()[:, None]
    a = _nearest((x.abs() / den[..., None].clamp(min=1e-300)).clamp(max=6), e2)
    return (torch.sign(x) * a * den[..., None]).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "append":
        return {"k": _exact_quantised(st["k"], st["g"][0]), "v": _exact_quantised(st["v"], st["g"][1])}
    if c["op"] == "evict":
        out = torch.zeros(st["dst"].numel(), c["page"], dtype=torch.float64)
        score, table, dst = st["score"].cpu().numpy().astype(np.float64), st["table"].cpu().numpy(), st["dst"].cpu().numpy()
        for b, n in enumerate(_lens_of(c)):
            s = score[table[b]].reshape(-1)[:n]
            keep = np.arange(n)
            if n > c["budget"]:
                old = n - c["recent"]
                first = np.lexsort((np.arange(old), -s[:old]))[:c["budget"] - c["recent"]]
                keep = np.sort(np.concatenate([first, np.arange(old, n)])).astype(np.int64)
            for i in range(0, len(keep), c["page"]):
                part = s[keep[i:i + c["page"]]]
                out[dst[b, i // c["page"]] - st["first"], :len(part)] = torch.from_numpy(part)
        return {"kept": None, "new_len": None, "pages": None, "score": out, "pos": None}
    rows, lens, group = _rows_of(c), _attn_lens(c), c["Hq"] // c["Hkv"]
    if sum(lens) * c["Hkv"] * c["D"] > 3e9:
        return None
    outs, lses, r0 = [], [], 0
    score = torch.zeros(st["pages"].shape[0], c["page"], dtype=torch.float64, device="cuda") if c["op"] == "weights" else None
    for b, (r, n) in enumerate(zip(rows, lens)):
        i = torch.arange(n, device="cuda")
        pos = i if st["pos"] is None else st["pos"][st["table"][b].long()].flatten()[:n].long()
        mine = n - r + torch.arange(r, device="cuda")
        dist = (pos[mine][:, None] - pos[None]).double()
        see = i[None] <= mine[:, None]
        if c["window"] > 0:
            see &= (dist < c["window"]) | (i[None] < c["prefix"])
        o_b, l_b, w_b = [], [], torch.zeros(n, dtype=torch.float64, device="cuda")
        for h in range(c["Hkv"]):
            k, v = _tokens(st, b, h, n)
            q = st["q"][r0:r0 + r, h * group:(h + 1) * group].double()
            s = torch.einsum("rgd,nd->rgn", q, k) * c["D"] ** -0.5
            if c["cap"] > 0:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if st["slopes"] is not None:
                s = s - st["slopes"][h * group:(h + 1) * group].double()[None, :, None] * dist[:, None]
            s = s.masked_fill(~see[:, None], float("-inf"))
            if score is not None:
                w_b += torch.exp(s - st["lse"][r0:r0 + r, h * group:(h + 1) * group].double()[..., None]).sum((0, 1))
                continue
            o_b.append(torch.einsum("rgn,nd->rgd", torch.softmax(s, -1), v))
            l_b.append(torch.logsumexp(s, -1))
        if score is not None:
            at = st["table"][b, i // c["page"]].long()
            score[at, i % c["page"]] = w_b
        else:
            outs.append(torch.cat(o_b, 1))
            lses.append(torch.cat(l_b, 1))
        r0 += r
    if score is not None:
        return {"score": score}
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
