"""The target's pass over a paged KV cache, restated in 64-bit NumPy.

"Accelerating Speculative Decoding with Block Diffusion Draft Trees", section
3.4.5 (verification over the cached context and the new tokens) and "DFlash:
Block Diffusion for Flash Speculative Decoding", section 3.4.4 (sampled
verification): per-head norm and rotation, the append into pages, attention of
the new tokens over pages, and the target's token from a given random number.
Plain loops over requests, heads and rows; nothing here is shared with the
library."""
import math

import numpy as np


def angles(pos, head_dim, theta):
    i = np.arange(head_dim // 2)
    return np.asarray(pos, dtype=np.float64)[:, None] * float(theta) ** (-2.0 * i / head_dim)


def rotate(x, pos, theta):
    """x [rows, heads, head_dim] turned at pos [rows]; theta 0: as it is."""
    if theta == 0:
        return x.copy()
    half = x.shape[-1] // 2
    a = angles(pos, x.shape[-1], theta)[:, None]
    lo, hi = x[..., :half], x[..., half:]
    return np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)


def norm_rope(x, gain, eps, theta, pos):
    """x [rows, heads, head_dim]; gain None: no norm."""
    y = x
    if gain is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain
    return rotate(y, pos, theta)


def append(pool_k, pool_v, table, row_off, pos0, k, v, theta, pos=None):
    """New pools.  k, v [rows, n_kv, head_dim]; pools [pages, n_kv, page, head_dim]."""
    pool_k, pool_v = pool_k.copy(), pool_v.copy()
    n_pages, _, page, _ = pool_k.shape
    for r in range(table.shape[0]):
        for i, row in enumerate(range(row_off[r], min(row_off[r + 1], k.shape[0]))):
            slot = pos0[r] + i
            at = slot if pos is None else pos[row]
            if at < 0 or slot < 0 or slot // page >= table.shape[1]:
                continue
            pg = table[r, slot // page]
            if not 0 <= pg < n_pages:
                continue
            pool_k[pg, :, slot % page] = rotate(k[row:row + 1], [at], theta)[0]
            pool_v[pg, :, slot % page] = v[row]
    return pool_k, pool_v


def slots(pool, table_row, n):
    """The first n slots of a request: [n_kv, n, head_dim]; no page: zeros."""
    n_pages, n_kv, page, hd = pool.shape
    out = np.zeros((n_kv, n, hd))
    for t in range(0, n, page):
        pg = table_row[t // page]
        if 0 <= pg < n_pages:
            m = min(page, n - t)
            out[:, t:t + m] = pool[pg, :, :m]
    return out


def visible(n, p0, kv, mask=None):
    """[n, kv]: which slots each of a request's n new rows sees."""
    t = np.arange(kv)
    if mask is None:
        return t[None] <= p0 + np.arange(n)[:, None]
    see = np.zeros((n, kv), dtype=bool)
    see[:, :p0] = True
    for i in range(n):
        for j in range(min(n, 32 * mask.shape[1], kv - p0)):
            see[i, p0 + j] = (int(mask[i, j // 32]) >> (j % 32)) & 1
    return see


def attention(q, pool_k, pool_v, table, row_off, pos0, n_q, mask=None):
    """q [rows, n_q, head_dim] -> (out, spread): the softmax average over the
    slots each row sees (those past the table left out), and the same average of
    |v| (the scale that rounding errors of the weights act on)."""
    n_kv, hd = pool_k.shape[1], pool_k.shape[3]
    page = pool_k.shape[2]
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    for r in range(table.shape[0]):
        a, b = row_off[r], min(row_off[r + 1], q.shape[0])
        if b <= a:
            continue
        kv = min(pos0[r] + b - a, table.shape[1] * page)
        see = visible(b - a, pos0[r], kv, None if mask is None else mask[a:b])
        ks, vs = slots(pool_k, table[r], kv), slots(pool_v, table[r], kv)
        for h in range(n_q):
            g = h // (n_q // n_kv)
            for i in range(b - a):
                on = see[i]
                if not on.any():
                    continue
                s = ks[g][on] @ q[a + i, h] / math.sqrt(hd)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[a + i, h] = p @ vs[g][on]
                spread[a + i, h] = p @ np.abs(vs[g][on])
    return out, spread


def kept(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Token ids (ascending) and their masses after the filters."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    best = x.max()
    if best == -np.inf:
        return np.zeros(0, dtype=np.int64), np.zeros(0)
    order = np.lexsort((np.arange(len(x)), -x))
    if not temperature > 0:
        return order[:1], np.ones(1)
    w = np.zeros(len(x))
    on = x > -np.inf
    w[on] = 1.0 if best == np.inf else np.exp((x[on] - best) / temperature)
    if best == np.inf:
        w[x < np.inf] = 0.0
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        before = np.cumsum(w[order]) - w[order]
        take = before < top_p * w[order].sum()
        take[0] = True
        order = order[take]
    if min_p > 0:
        lim = temperature * math.log(min(min_p, 1.0))
        order = order[[x[v] == best or x[v] - best >= lim for v in order]]
    ids = np.sort(order[w[order] > 0])
    return ids, w[ids]


def sample(logits, u, **how):
    """(token, its log-share of the kept mass); -1 where nothing is left."""
    ids, w = kept(logits, **how)
    if len(ids) == 0:
        return -1, -np.inf
    cum = np.cumsum(w)
    j = min(int(np.searchsorted(cum, min(max(u, 0.0), 1.0) * cum[-1], side="right")), len(ids) - 1)
    return int(ids[j]), math.log(w[j] / cum[-1])
