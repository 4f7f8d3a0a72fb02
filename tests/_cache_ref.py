"""The 4-bit paged cache in plain numpy, 64 bits: the definitions of
include/spec_cache.h written token by token, sharing nothing with the kernels."""
from __future__ import annotations

import numpy as np

TOK = 32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0, ties to the even index, saturating."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where((hi < lo) | ((hi == lo) & (i % 2 == 0)), i, i - 1)


def quantise(x, g):
    """x [..., D] float32, g a float32: codes [..., D] and scale bytes [..., D/16].
    The quotients are fp32 (IEEE), as the definition says; the roundings to the
    grids are made on exact values."""
    f = np.float32
    xb = np.asarray(x, f).reshape(*x.shape[:-1], -1, 16)
    t = np.minimum(np.abs(xb).max(-1) / (f(6) * f(g)), f(448))
    s = nearest(t.astype(np.float64), E4M3[:127])
    den = (E4M3[s].astype(f) * f(g)).astype(f)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(den[..., None] > 0, xb / den[..., None], f(0)).astype(f)
    code = nearest(np.abs(y).astype(np.float64), E2M1) + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


class Cache:
    """A pool as numpy bytes [n_pages, H, blocks, 36 D] with its page table."""

    def __init__(self, pages, table, k_scale=None, v_scale=None):
        self.pages, self.table = np.array(pages), np.array(table)
        self.n_pages, self.H, self.nblk, nbytes = self.pages.shape
        self.D, self.page = nbytes // 36, self.nblk * TOK
        one = np.ones(self.H, np.float32)
        self.g = [one if s is None else np.asarray(s, np.float32) for s in (k_scale, v_scale)]

    def block(self, b, h, slot):
        return self.pages[self.table[b, slot // self.page], h, slot % self.page // TOK]

    def put(self, b, h, slot, k, v):
        D, t = self.D, slot % TOK
        blk = self.block(b, h, slot)
        kc, ks = quantise(k, self.g[0][h])
        vc, vs = quantise(v, self.g[1][h])
        for d in range(0, D, 2):
            blk[d // 32 * 512 + t * 16 + d % 32 // 2] = kc[d] | kc[d + 1] << 4
        for d in range(D):
            at = 18 * D + d * 16 + t // 2
            old = int(blk[at])
            blk[at] = (old & 0xF0 | int(vc[d])) if t % 2 == 0 else (old & 0x0F | int(vc[d]) << 4)
        for g in range(D // 16):
            blk[16 * D + t * (D // 16) + g] = ks[g]
            blk[34 * D + g * TOK + t] = vs[g]

    def get(self, b, h, slots):
        """Keys and values [n, D] in 64 bits of the given slots."""
        D = self.D
        slots = np.asarray(slots, np.int64)
        raw = self.pages[self.table[b, slots // self.page], h, slots % self.page // TOK]
        t, d = (slots % TOK)[:, None], np.arange(D)[None]
        row = np.arange(len(slots))[:, None]
        kb, ks = raw[row, d // 32 * 512 + t * 16 + d % 32 // 2], raw[row, 16 * D + t * (D // 16) + d // 16]
        vb, vs = raw[row, 18 * D + d * 16 + t // 2], raw[row, 34 * D + d // 16 * TOK + t]
        kc, vc = kb >> (4 * (d % 2)).astype(np.uint8) & 15, vb >> (4 * (t % 2)).astype(np.uint8) & 15
        val = lambda c, s, g: np.where(c >= 8, -1, 1) * E2M1[c & 7] * np.where(s >= 128, -1, 1) * E4M3[s & 127] * np.float64(g)
        return val(kc, ks, self.g[0][h]), val(vc, vs, self.g[1][h])


def attention(cache, q, cu, lens, *, scale=None, cap=0.0, slopes=None, window=0, prefix=0, slot_pos=None):
    """out, lse, A = sum_j p_j |v_j| and S = the largest scale * sum |q k| of
    each (row, head), and the per-slot weights of each request."""
    R, Hq, D = q.shape
    group = Hq // cache.H
    scale = D ** -0.5 if scale is None else scale
    out, A = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    lse, S = np.full((R, Hq), -np.inf), np.zeros((R, Hq))
    weights = []
    for b in range(len(cu) - 1):
        n, L = cu[b + 1] - cu[b], int(lens[b])
        i = np.arange(L)
        pos = i if slot_pos is None else np.asarray(slot_pos)[cache.table[b, i // cache.page], i % cache.page].astype(np.int64)
        w = np.zeros(L)
        kv = [cache.get(b, h, i) for h in range(cache.H)]
        for j in range(n):
            own = L - n + j
            if own < 0:
                continue
            dist = pos[own] - pos
            see = i <= own
            if window > 0:
                see &= (dist < window) | (i < prefix)
            for h in range(Hq):
                k, v = (x[see] for x in kv[h // group])
                if not len(k):
                    continue
                qq = q[cu[b] + j, h].astype(np.float64)
                s = k @ qq * scale
                S[cu[b] + j, h] = (np.abs(k) @ np.abs(qq)).max() * abs(scale)
                if cap > 0:
                    s = cap * np.tanh(s / cap)
                if slopes is not None:
                    s = s - np.float64(slopes[h]) * dist[see]
                m = s.max()
                p = np.exp(s - m)
                lse[cu[b] + j, h] = m + np.log(p.sum())
                p /= p.sum()
                out[cu[b] + j, h] = p @ v
                A[cu[b] + j, h] = p @ np.abs(v)
                w[see] += p
        weights.append(w)
    return out, lse, A, S, weights


def evict(score, n, budget, recent):
    """Kept slots of one request of length n by the definition."""
    if n <= budget:
        return np.arange(n)
    old = n - recent
    s = np.where(np.isnan(score[:old]), -np.inf, score[:old].astype(np.float64)) + 0.0
    nan = np.isnan(score[:old])
    order = np.lexsort((np.arange(old), nan, -s))
    return np.sort(np.concatenate([order[:budget - recent], np.arange(old, n)])).astype(np.int64)
