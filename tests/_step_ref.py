"""Prompt and tree attention, logit adjustment and tree acceptance in plain numpy, 64 bits:
the definitions of include/spec_prompt.h and include/spec_tree.h written row by row, sharing
nothing with the kernels."""
from __future__ import annotations

import numpy as np


def softmax_row(q, k, v, dist, see, scale, cap, slope):
    """out, lse, A = sum p |v|, S = scale * max sum |q k| of one row over the keys it sees."""
    if not see.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    k, v, dist = k[see], v[see], dist[see]
    s = k @ q * scale
    S = (np.abs(k) @ np.abs(q)).max() * abs(scale)
    if cap > 0:
        s = cap * np.tanh(s / cap)
    s = s - np.float64(slope) * dist
    m = s.max()
    p = np.exp(s - m)
    t = p.sum()
    return p @ v / t, m + np.log(t), p @ np.abs(v) / t, S


def _empty(q):
    R, Hq, D = q.shape
    return np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf), np.zeros((R, Hq, D)), np.zeros((R, Hq))


def prompt(q, k, v, cu, cu_keys=None, *, scale=None, cap=0.0, slopes=None, window=0, prefix=0):
    """out, lse, A, S of every (row, head)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    cu_keys = cu if cu_keys is None else cu_keys
    Hq, group = q.shape[1], q.shape[1] // k.shape[1]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    res = _empty(q)
    for b in range(len(cu) - 1):
        n, m = cu[b + 1] - cu[b], cu_keys[b + 1] - cu_keys[b]
        j = np.arange(m)
        for i in range(n):
            dist = m - n + i - j
            see = dist >= 0
            if window > 0:
                see &= (dist < window) | (j < prefix)
            for h in range(Hq):
                kv = (x[cu_keys[b]:cu_keys[b + 1], h // group] for x in (k, v))
                row = softmax_row(q[cu[b] + i, h], *kv, dist, see, scale, cap, 0.0 if slopes is None else slopes[h])
                for to, x in zip(res, row):
                    to[cu[b] + i, h] = x
    return res


def paths(parent):
    """For each node of one tree its ancestors and itself; a parent that is not before its node is none."""
    out = []
    for j, p in enumerate(parent):
        out.append((out[p] if j > 0 and 0 <= p < j else []) + [j])
    return out


def tree(cache, q, cu, lens, parent, *, scale=None, cap=0.0, slopes=None, window=0, prefix=0, slot_pos=None):
    """out, lse, A, S of every (row, head) over a tests._cache_ref.Cache."""
    q = np.asarray(q, np.float64)
    Hq, D = q.shape[1:]
    group, scale = Hq // cache.H, D ** -0.5 if scale is None else scale
    res = _empty(q)
    for b in range(len(cu) - 1):
        n, L = cu[b + 1] - cu[b], int(lens[b])
        if L < n:
            continue
        root, i = L - n, np.arange(L)
        anc = paths(parent[cu[b]:cu[b + 1]])
        pos = i if slot_pos is None else np.asarray(slot_pos)[cache.table[b, i // cache.page], i % cache.page].astype(np.int64)
        pos = np.concatenate([pos[:root], [pos[root] + len(a) - 1 for a in anc]]).astype(np.int64) if n else pos
        kv = [cache.get(b, h, i) for h in range(cache.H)]
        for j in range(n):
            dist = pos[root + j] - pos
            see = i < root
            see[[root + a for a in anc[j]]] = True
            if window > 0:
                see &= (dist < window) | (i < prefix)
            for h in range(Hq):
                row = softmax_row(q[cu[b] + j, h], *kv[h // group], dist, see, scale, cap, 0.0 if slopes is None else slopes[h])
                for to, x in zip(res, row):
                    to[cu[b] + j, h] = x
    return res


def accept(row_token, node_token, parent, cu, k_max):
    """accepted_len, out_tokens, next_token, path_rows."""
    B = len(cu) - 1
    acc, nxt = np.zeros(B, np.int32), np.full(B, -1, np.int32)
    out, path = np.full((B, k_max + 1), -1, np.int32), np.full((B, k_max + 1), -1, np.int32)
    for b in range(B):
        lo, n = cu[b], cu[b + 1] - cu[b]
        at, taken = 0, [0]
        while True:
            t = row_token[lo + at]
            child = [c for c in range(1, n) if parent[lo + c] == at and c > at and node_token[lo + c] == t]
            out[b, len(taken) - 1] = nxt[b] = t
            if not child:
                break
            at = child[0]
            taken.append(at)
        acc[b] = len(taken) - 1
        path[b] = [lo + taken[min(i, len(taken) - 1)] for i in range(k_max + 1)]
    return acc, out, nxt, path


def adjust(z, cu, V, *, history=None, n_tokens=None, n_prompt=None, repetition=None, frequency=None, presence=None,
           node_token=None, parent=None, bias=None, allowed=None, allowed_row=None):
    """Adjusted logits [R, V] and the sum of the magnitudes that made each; bias: a list of (ids, values)."""
    out = np.array(z[:, :V], np.float64)
    mag = np.abs(np.where(np.isfinite(out), out, 0.0))
    for b in range(len(cu) - 1):
        lo, n = cu[b], cu[b + 1] - cu[b]
        seen0, made0 = np.zeros(V, np.int64), np.zeros(V, np.int64)
        if history is not None:
            h = np.asarray(history[b][:n_tokens[b]], np.int64)
            new = np.arange(len(h)) >= (0 if n_prompt is None else n_prompt[b])
            ok = (h >= 0) & (h < V)
            np.add.at(seen0, h[ok], 1)
            np.add.at(made0, h[ok & new], 1)
        rep = 1.0 if repetition is None else np.float64(repetition[b])
        fre = 0.0 if frequency is None else np.float64(frequency[b])
        pre = 0.0 if presence is None else np.float64(presence[b])
        up = list(range(-1, n - 1)) if parent is None else [p if 0 <= p < j else -1 for j, p in enumerate(parent[lo:lo + n])]
        anc = paths(up)
        for j in range(n):
            seen, made, x = seen0.copy(), made0.copy(), out[lo + j]
            if node_token is not None:
                for c in anc[j]:
                    t = node_token[lo + c]
                    if c > 0 and up[c] >= 0 and 0 <= t < V:
                        seen[t] += 1
                        made[t] += 1
            x = np.where(seen > 0, np.where(x > 0, x / rep, x * rep), x)
            mag[lo + j] = np.maximum(mag[lo + j], np.abs(np.where(np.isfinite(x), x, 0.0)))
            x = x - fre * made - pre * (made > 0)
            mag[lo + j] += np.abs(fre) * made + np.abs(pre) * (made > 0)
            if bias is not None:
                for i, w in zip(*bias[b]):
                    if 0 <= i < V:
                        x[i] += np.float64(w)
                        mag[lo + j, i] += abs(np.float64(w))
            if allowed is not None:
                m = lo + j if allowed_row is None else allowed_row[lo + j]
                if 0 <= m < len(allowed):
                    v = np.arange(V)
                    w = np.asarray(allowed[m]).view(np.uint32)[v // 32]
                    x = np.where(w >> (v % 32).astype(np.uint32) & 1, x, -np.inf)
            out[lo + j] = x
    return out, mag
