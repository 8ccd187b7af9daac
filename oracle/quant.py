"""A paged KV cache held in 8 bits, and logits before sampling, restated in 64-bit
NumPy: e4m3 codes with a power-of-two scale for each block of 16 slots of a KV head,
the append into them, and bias, penalties and allowed tokens over a row's past.

The verification pass of "Accelerating Speculative Decoding with Block Diffusion
Draft Trees", section 3.4.5, reads such a cache and makes the target's choices.
Plain loops; nothing here is shared with the library."""
import numpy as np

from . import paged

BLOCK = 16


def e4m3_values():
    """The value of each of the 256 codes."""
    out = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        if e == 15 and f == 7:
            v = np.nan
        out[c] = -v if c >> 7 else v
    return out


VALUES = e4m3_values()


def encode(x):
    """The nearest codes, ties to the even one; not finite: NaN.  |x| <= 448."""
    x = np.asarray(x, dtype=np.float64)
    pos = VALUES[:127]                                  # 0 .. 448, ascending
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    take = (up < down) | ((up == down) & (hi % 2 == 0))
    code = np.where(take, hi, lo) + 128 * np.signbit(x)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def exponent(top):
    """The smallest e >= -127 with top <= 448 * 2^e."""
    e = -127
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def held(codes, scale):
    """Values of a pool [pages, n_kv, page, hd] with scales [pages, n_kv, page / 16]."""
    e = np.repeat(scale.astype(np.float64) - 127.0, BLOCK, axis=2)[..., None]
    return VALUES[codes] * 2.0 ** e


def append(codes_k, codes_v, scale_k, scale_v, table, row_off, pos0, k, v, theta, pos=None):
    """New pools and scales, and what the new rows were before rounding: (codes_k,
    codes_v, scale_k, scale_v, exact_k, exact_v), exact NaN where nothing new lies.
    k, v [rows, n_kv, head_dim]."""
    out = [a.copy() for a in (codes_k, codes_v, scale_k, scale_v)]
    exact = [np.full(codes_k.shape, np.nan) for _ in range(2)]
    n_pages, n_kv, page, _ = codes_k.shape
    for r in range(table.shape[0]):
        blocks = {}
        for i, row in enumerate(range(row_off[r], min(row_off[r + 1], k.shape[0]))):
            slot = pos0[r] + i
            at = slot if pos is None else pos[row]
            if at < 0 or slot < 0 or slot // page >= table.shape[1]:
                continue
            if 0 <= table[r, slot // page] < n_pages:
                blocks.setdefault(slot // BLOCK, []).append((slot, row, at))
        for b, rows in blocks.items():
            pg, s0 = table[r, b * BLOCK // page], b * BLOCK % page
            old = max(pos0[r] - b * BLOCK, 0)
            for which, x in ((0, k), (1, v)):
                codes, scale = out[which], out[2 + which]
                new = {slot: paged.rotate(x[row:row + 1], [at], theta if which == 0 else 0)[0]
                       for slot, row, at in rows}
                for g in range(n_kv):
                    y = np.concatenate([new[s][g] for s in new])
                    y = y[np.isfinite(y)]
                    e = exponent(np.abs(y).max() if len(y) else 0.0)
                    if old:
                        was = int(scale[pg, g, s0 // BLOCK]) - 127
                        if e > was:
                            c = codes[pg, g, s0:s0 + old]
                            codes[pg, g, s0:s0 + old] = encode(VALUES[c] * 2.0 ** (was - e))
                        e = max(e, was)
                    scale[pg, g, s0 // BLOCK] = e + 127
                    for s in new:
                        codes[pg, g, s % page] = encode(new[s][g] * 2.0 ** -e)
                        exact[which][pg, g, s % page] = new[s][g]
    return (*out, *exact)


def adjust(logits, row_off, history=None, prompt_len=None, repetition=None, presence=None,
           frequency=None, tok=None, mask=None, bias=None, allowed=None):
    """Adjusted logits [rows, vocab] and the size of what was added up for each.
    history: a list of tokens for each request; bias: a list of (token, value) for each;
    mask, allowed: rows of 32-bit words."""
    out = np.array(logits, dtype=np.float64)
    size = np.abs(np.where(np.isfinite(out), out, 0.0))
    rows, vocab = out.shape
    for r in range(len(row_off) - 1):
        a, b = row_off[r], min(row_off[r + 1], rows)
        past = list(history[r]) if history is not None else []
        cut = int(prompt_len[r]) if prompt_len is not None else 0
        for i in range(a, b):
            path = []
            if tok is not None:
                for j in range(b - a):
                    if mask is None:
                        see = j <= i - a
                    else:
                        see = j // 32 < mask.shape[1] and (int(mask[i, j // 32]) >> (j % 32)) & 1
                    if see:
                        path.append(int(tok[a + j]))
            held_, made = {}, {}
            for n, t in enumerate(past + path):
                if 0 <= t < vocab:
                    held_[t] = True
                    if n >= cut or n >= len(past):
                        made[t] = made.get(t, 0) + 1
            for t, x in dict(bias[r] if bias is not None else []).items():
                if 0 <= t < vocab:
                    out[i, t] += x
                    size[i, t] += abs(x)
            rho = 1.0 if repetition is None else float(repetition[r])
            phi = 0.0 if frequency is None else float(frequency[r])
            pi = 0.0 if presence is None else float(presence[r])
            for t in held_:
                out[i, t] = out[i, t] / rho if out[i, t] > 0 else out[i, t] * rho
                size[i, t] *= max(rho, 1 / rho)
            for t, c in made.items():
                out[i, t] -= phi * c + pi
                size[i, t] += 2 * abs(phi * c) + abs(pi)
            if allowed is not None:
                ok = np.unpackbits(np.ascontiguousarray(allowed[i]).astype("<u4").view(np.uint8), bitorder="little")
                out[i, ok[:vocab] == 0] = -np.inf
    return out, size
