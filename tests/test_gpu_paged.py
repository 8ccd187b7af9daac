"""GPU parity of the paged-cache operators (norm and rotation, append,
attention) against the 64-bit oracle, through the C ABI.

Tolerances, element by element, with h = 2^-8 (bf16) or 2^-24 (fp32), half a
step of the output type relative to the value:
- norm_rope, append: the output's rounding, h |ref|, plus fp32 arithmetic
  before it: the sum of squares and the products (head_dim + 32 roundings at
  most), and an angle known to 2^-21 rad, all relative to |a| + |b|, the pair
  that is turned.  Values are copied, so they are equal bit for bit.
- attention: each probability is rounded to bf16 before the second product
  (2^-8 of sum p |v|, the oracle's spread), the output once more (2^-8 |ref|);
  the fp32 sums over kv keys add kv 2^-24 of the spread, twice;
  a score's fp32 sum of head_dim products and its exponential's 2^-22 move the
  probabilities by (head_dim + 8) 2^-24 S + 2^-20, S = max over keys of
  sum |q k| / sqrt(head_dim), twice (numerator and denominator)."""
import math

import numpy as np
import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding as bd
from oracle import ddtree as odt
from oracle import paged as op

pytestmark = pytest.mark.gpu

DEV = "cuda"
THETA = 1.0e6
BF, F32 = torch.bfloat16, torch.float32


def _t(a, dtype=BF):
    return torch.as_tensor(np.asarray(a, dtype=np.float32)).to(dtype).to(DEV)


def _i(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _ws(n_q, n_kv, hd):
    return torch.zeros(bd.paged_attention_workspace_bytes(n_q, n_kv, hd), dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------

def _rope_tol(ref, src, hd, dtype):
    """src: the turned vector's values before the rotation, [rows, heads, hd]."""
    half = hd // 2
    pair = np.abs(src[..., :half]) + np.abs(src[..., half:])
    pair = np.concatenate([pair, pair], -1)
    return _half(dtype) * np.abs(ref) + ((hd + 32) * 2.0 ** -24 + 2.0 ** -21) * pair + 1e-30


@pytest.mark.parametrize("rows,n_q,n_kv,hd,dtype,pad", [
    (1, 32, 8, 128, BF, 0), (33, 14, 2, 64, BF, 0), (5, 5, 1, 128, F32, 0), (70, 64, 8, 64, F32, 0),
    (9, 3, 2, 128, BF, 5),        # rows off 16-byte boundaries
    (257, 32, 8, 128, BF, 0), (4, 100, 30, 128, BF, 8),      # more heads than one round of a CTA
    (1501, 6, 2, 128, BF, 0), (1203, 3, 1, 64, F32, 0), (1000, 40, 7, 64, BF, 3),   # several rows to a CTA
])
def test_norm_rope(rows, n_q, n_kv, hd, dtype, pad):
    rng = np.random.default_rng(rows + hd)
    x = _t(rng.normal(size=(rows, (n_q + 2 * n_kv) * hd + pad)) * 3, dtype)
    q, k = x[:, :n_q * hd], x[:, n_q * hd:(n_q + n_kv) * hd]
    gq, gk = (_t(1 + 0.3 * rng.normal(size=hd), dtype) for _ in range(2))
    pos = rng.integers(0, 1 << 20, size=rows).astype(np.int32)
    pos[0] = 0
    if rows > 4:
        pos[3] = -1
    qo = torch.full((rows, n_q * hd + pad), 7.0, dtype=dtype, device=DEV)[:, :n_q * hd]
    ko = torch.full((rows, n_kv * hd), 7.0, dtype=dtype, device=DEV)
    before = x.clone()
    bd.qk_norm_rope(q, k, gq, gk, 1e-6, THETA, _i(pos), hd, qo, ko)
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    live = pos >= 0
    for src, gain, got, heads in ((q, gq, qo, n_q), (k, gk, ko, n_kv)):
        s = _f64(src).reshape(rows, heads, hd)
        flat = op.norm_rope(s, _f64(gain), 1e-6, 0.0, None)
        ref = op.rotate(flat, pos, THETA)
        g = _f64(got).reshape(rows, heads, hd)
        assert np.all(np.abs(g - ref)[live] <= _rope_tol(ref, flat, hd, dtype)[live])
        assert np.all(g[~live] == 7.0)
    # in place, the same values
    bd.qk_norm_rope(q, k, gq, gk, 1e-6, THETA, _i(pos), hd)
    torch.cuda.synchronize()
    on = torch.as_tensor(live, device=DEV)
    assert torch.equal(q[on], qo[on]) and torch.equal(k[on], ko[on])
    assert torch.equal(q[~on], before[~on][:, :n_q * hd])
    assert torch.equal(x[:, (n_q + n_kv) * hd:], before[:, (n_q + n_kv) * hd:])


def test_norm_rope_parts():
    """No gain: rotation alone; theta 0: norm alone, no positions; keys alone; no rows."""
    rng = np.random.default_rng(3)
    x = _t(rng.normal(size=(6, 4 * 64)))
    g = _t(rng.normal(size=64))
    pos = _i([0, 1, 2, 3, 4, 100000])
    out = torch.empty_like(x)
    s = _f64(x).reshape(6, 4, 64)
    bd.qk_norm_rope(None, x, None, None, 0.0, THETA, pos, 64, None, out)
    ref = op.rotate(s, pos.cpu().numpy(), THETA)
    assert np.all(np.abs(_f64(out).reshape(s.shape) - ref) <= _rope_tol(ref, s, 64, BF))
    bd.qk_norm_rope(x, None, g, None, 1e-6, 0.0, None, 64, out)
    ref = op.norm_rope(s, _f64(g), 1e-6, 0.0, None)
    assert np.all(np.abs(_f64(out).reshape(s.shape) - ref) <= _rope_tol(ref, ref, 64, BF))
    bd.qk_norm_rope(x[:0], x[:0], g, g, 1e-6, THETA, pos[:0], 64)
    # a row of zeros has no direction: zeros, not NaN
    z = torch.zeros(1, 64, dtype=BF, device=DEV)
    bd.qk_norm_rope(z, None, g, None, 1e-6, THETA, pos[:1], 64)
    assert not z.any()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _paged(rng, rows, ctx, n_kv, hd, page, dtype=BF, spare=3, wide=0):
    need = [-(-(n + c) // page) for n, c in zip(rows, ctx)]
    total = sum(need) + spare
    order = rng.permutation(total)
    table = np.full((len(rows), max(max(need), 1) + wide), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    pk, pv = (_t(rng.normal(size=(total, n_kv, page, hd)), dtype) for _ in range(2))
    row_off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return pk, pv, table, row_off


@pytest.mark.parametrize("rows,ctx,n_kv,hd,page,dtype,theta,pad", [
    ([1], [0], 8, 128, 16, BF, THETA, 0),
    ([1, 0, 5, 17], [15, 9, 0, 30], 2, 64, 16, BF, THETA, 0),
    ([40, 1, 3], [100, 63, 64], 1, 128, 64, F32, THETA, 0),
    ([0, 0, 33], [5, 5, 5], 5, 64, 32, F32, 0.0, 3),
    ([130, 2], [7, 1000], 3, 128, 1024, BF, THETA, 1),      # rows off 16-byte boundaries
    ([2] * 70, list(range(70)), 1, 64, 16, BF, THETA, 0),   # more requests than a warp
    ([7], [2], 40, 128, 16, BF, THETA, 0),                  # more heads than one round of a CTA
    ([900, 0, 303], [40, 7, 100], 2, 128, 32, BF, THETA, 0),    # several rows to a CTA
    ([1, 1099], [0, 3], 3, 64, 16, F32, THETA, 1),
])
def test_append(rows, ctx, n_kv, hd, page, dtype, theta, pad):
    rng = np.random.default_rng(len(rows) * 7 + hd)
    pk, pv, table, off = _paged(rng, rows, ctx, n_kv, hd, page, dtype)
    n = sum(rows)
    kv = _t(rng.normal(size=(n + 2, 2 * n_kv * hd + pad)), dtype)    # two rows behind the last one
    k, v = kv[:, :n_kv * hd], kv[:, n_kv * hd:2 * n_kv * hd]
    k64, v64 = (_f64(x).reshape(n + 2, n_kv, hd) for x in (k, v))
    for pos in (None, rng.integers(-1, 5000, size=n + 2).astype(np.int32)):
        a, b = pk.clone(), pv.clone()
        bd.paged_append(bd.Pages(a, b, _i(table)), k, v, _i(off), _i(ctx), theta=theta,
                        pos=None if pos is None else _i(pos))
        torch.cuda.synchronize()
        rk, rv = op.append(_f64(pk), _f64(pv), table, off, ctx, k64, v64, theta, pos)
        # the size of the pair that was turned, laid out as the pool is
        sk, _ = op.append(np.abs(_f64(pk)), _f64(pv), table, off, ctx, k64, v64, 0.0, pos)
        assert np.array_equal(_f64(b), rv)
        written = np.any(rk != _f64(pk), axis=-1)
        tol = _rope_tol(rk, sk, hd, dtype) if theta else 0.0
        assert np.all(np.abs(_f64(a) - rk) <= tol)
        assert np.array_equal(_f64(a)[~written], _f64(pk)[~written])


def test_append_without_a_page_stores_nothing():
    rng = np.random.default_rng(5)
    pk, pv, table, off = _paged(rng, [40], [10], 2, 64, 16)
    table[0, 1] = -1                                # slots 16..31
    table[0, 2] = pk.shape[0]                       # slots 32..47: one past the pool
    k, v = (_t(rng.normal(size=(40, 128))) for _ in range(2))
    a, b = pk.clone(), pv.clone()
    # the table ends at slot 64; positions 10 .. 49 and then 60 .. 99
    for p0 in (10, 60):
        bd.paged_append(bd.Pages(a, b, _i(table)), k, v, _i(off), _i([p0]))
    torch.cuda.synchronize()
    rk, rv = _f64(pk), _f64(pv)
    for p0 in (10, 60):
        rk, rv = op.append(rk, rv, table, off, [p0], _f64(k).reshape(40, 2, 64),
                           _f64(v).reshape(40, 2, 64), 0.0)
    assert np.array_equal(_f64(a), rk) and np.array_equal(_f64(b), rv)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _attn_tol(ref, spread, q, pk, kv, hd):
    # S: a bound over all keys of the pool (Cauchy-Schwarz)
    s = np.linalg.norm(q, axis=-1, keepdims=True) * np.linalg.norm(pk, axis=-1).max() / math.sqrt(hd)
    delta = (hd + 8) * 2.0 ** -24 * s + 2.0 ** -20 + kv * 2.0 ** -24
    return (2.0 ** -8 * (1 + 2.0 ** -7) + 2 * delta) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30


def _tree_mask(rng, rows, words):
    out = np.zeros((sum(rows), words), dtype=np.uint32)
    at = 0
    for n in rows:
        bits = []
        for i in range(n):
            bits.append((bits[rng.integers(max(0, i - 9), i)] if i else 0) | (1 << i))
            for w in range(words):
                out[at + i, w] = (bits[i] >> (32 * w)) & 0xFFFFFFFF
        at += n
    return out


CASES = [
    # rows, ctx, n_q, n_kv, hd, page, tree
    ([1], [0], 4, 1, 128, 16, False),                       # one token, nothing before it
    ([1], [1], 1, 1, 64, 16, False),
    ([1], [2047], 32, 8, 128, 16, False),
    ([1, 1, 1, 1, 1], [0, 15, 16, 63, 500], 8, 2, 128, 16, False),
    ([1] * 40, list(range(0, 400, 10)), 2, 2, 64, 32, False),   # more requests than a warp
    ([1, 0, 1, 1, 0] * 61, list(range(305)), 2, 1, 64, 16, False),   # many to a lane, some without rows
    ([0] * 40 + [20, 0, 70] + [0] * 30, list(range(73)), 4, 1, 64, 32, False),
    ([3] * 1100, [5] * 1100, 2, 1, 64, 16, False),          # more than a warp of runs of 32
    ([1], [300], 16, 1, 128, 32, False),                    # 16 heads to a KV head
    ([1, 1], [77, 0], 40, 1, 64, 16, False),                # 40: several tiles for one token
    ([3, 0, 5], [10, 20, 0], 14, 2, 64, 16, False),         # 7 heads, and a request without rows
    ([16, 16], [100, 333], 32, 8, 128, 32, False),
    ([1, 33, 2], [900, 31, 64], 6, 2, 128, 64, False),
    ([70], [0], 4, 4, 128, 16, False),                      # a prompt from nothing
    ([200, 1], [57, 1000], 8, 2, 128, 128, False),
    ([129, 64], [0, 130], 5, 1, 64, 256, False),
    ([300], [100], 4, 1, 128, 1024, False),                 # one page holds everything
    ([17], [200], 8, 2, 128, 16, True),
    ([65, 40], [300, 0], 8, 2, 128, 16, True),
    ([130, 1], [129, 5], 4, 1, 64, 64, True),
    ([257], [64], 8, 2, 128, 32, True),
]


def _build(rows, ctx, n_q, n_kv, hd, page, tree, seed=0, spare=3):
    rng = np.random.default_rng(seed + sum(rows) + sum(ctx))
    pk, pv, table, off = _paged(rng, rows, ctx, n_kv, hd, page, spare=spare)
    n = sum(rows)
    q = _t(rng.normal(size=(n, n_q * hd)))
    mask = _tree_mask(rng, rows, (max(rows) + 31) // 32) if tree else None
    return dict(pk=pk, pv=pv, table=table, off=off, ctx=ctx, q=q, mask=mask, n_q=n_q, hd=hd,
                n_kv=n_kv, rows=rows)


def _attend(d, ws=None, out=None, max_rows=None, stream=None):
    out = torch.full_like(d["q"], 7.0) if out is None else out
    ws = _ws(d["n_q"], d["n_kv"], d["hd"]) if ws is None else ws
    mask = None if d["mask"] is None else torch.as_tensor(d["mask"].view(np.int32), device=DEV)
    bd.paged_attention(bd.Pages(d["pk"], d["pv"], _i(d["table"])), d["q"], _i(d["off"]), _i(d["ctx"]),
                       max(d["rows"]) if max_rows is None else max_rows, out, ws, mask=mask,
                       stream=stream)
    return out, ws


def _check(d, out):
    n = d["q"].shape[0]
    q = _f64(d["q"]).reshape(n, d["n_q"], d["hd"])
    pk = _f64(d["pk"])
    ref, spread = op.attention(q, pk, _f64(d["pv"]), d["table"], d["off"], d["ctx"], d["n_q"], d["mask"])
    used = np.where(np.isfinite(pk), pk, 0.0)
    kv = max(a + b for a, b in zip(d["rows"], d["ctx"]))
    tol = _attn_tol(ref, spread, q, used, kv, d["hd"])
    live = int(d["off"][-1])
    got = _f64(out).reshape(q.shape)
    err = np.abs(got - ref)[:live]
    assert np.all(np.isfinite(got[:live]))
    assert np.all(err <= tol[:live]), float((err / tol[:live]).max())


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}+{max(c[1])}q{c[2]}kv{c[3]}d{c[4]}p{c[5]}{'t' if c[6] else ''}")
def test_attention(case):
    d = _build(*case)
    out, ws = _attend(d)
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 0
    _check(d, out)
    # the counters are left at zero, and a second call agrees bit for bit
    again, _ = _attend(d, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


@pytest.mark.parametrize("rows,tree", [([1, 1], False), ([20, 3], False), ([20, 3], True),
                                       ([300, 40], False), ([140, 40], True)])
def test_attention_ignores_what_no_row_may_see(rows, tree):
    """NaN and infinities in slots past the requests' ends, in pages of nobody,
    and (chunks) in a value that only later rows see."""
    d = _build(rows, [70, 9], 8, 2, 128, 16, tree)
    clean, _ = _attend(d)
    dirty = dict(d, pk=torch.full_like(d["pk"], float("nan")), pv=torch.full_like(d["pv"], float("inf")))
    for r in range(2):
        for t in range(rows[r] + d["ctx"][r]):
            pg = d["table"][r, t // 16]
            dirty["pk"][pg, :, t % 16] = d["pk"][pg, :, t % 16]
            dirty["pv"][pg, :, t % 16] = d["pv"][pg, :, t % 16]
    got, _ = _attend(dirty)
    torch.cuda.synchronize()
    assert torch.equal(got, clean)


@pytest.mark.parametrize("n,ctx,tree", [(3, 40, False), (20, 40, False), (20, 0, True), (200, 130, False),
                                        (140, 100, True)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_bad_value_reaches_only_the_rows_that_see_it(n, ctx, tree, bad):
    d = _build([n], [ctx], 4, 2, 128, 16, tree, seed=3)
    clean, _ = _attend(d)
    j = n // 2                                       # the new token whose value is bad
    pg = int(d["table"][0, (ctx + j) // 16])
    pv = d["pv"].clone()
    pv[pg, 1, (ctx + j) % 16, 5] = bad
    out, _ = _attend(dict(d, pv=pv))
    torch.cuda.synchronize()
    o = out.view(n, 4, 128)
    see = op.visible(n, ctx, n + ctx, d["mask"])[:, ctx + j]
    hit = torch.zeros(n, 4, 128, dtype=torch.bool, device=DEV)
    hit[torch.as_tensor(see, device=DEV), 2:, 5] = True
    assert see.any() and not see.all()
    assert not torch.isfinite(o[hit]).any()
    assert torch.equal(torch.isfinite(o), ~hit)
    err = (o.float() - clean.view(n, 4, 128).float())[~hit].abs().max().item()
    assert err <= 2.0 ** -6 * clean.float().abs().max().item()


def test_attention_masks_at_the_edges():
    """Rows with no bit set (the context alone; zeros where there is none), bits
    that are not causal, and bits past the request's rows."""
    d = _build([5, 4], [20, 0], 4, 1, 128, 16, True, seed=9)
    m = np.zeros((9, 1), dtype=np.uint32)
    m[1], m[2], m[3], m[4] = 0b11111, 1 << 4, 0xFFFFFFFF, 0b10000
    m[6], m[7] = 0xFFFFFFF0, 0b1
    d["mask"] = m
    out, _ = _attend(d)
    torch.cuda.synchronize()
    _check(d, out)
    assert not out[5].any() and not out[6].any() and not out[8].any()
    assert out[0].any() and out[7].any()


def test_attention_rows_behind_the_last_sequence_are_left():
    d = _build([3, 2], [30, 8], 4, 2, 64, 16, False)
    d["off"] = np.array([0, 3, 4], dtype=np.int32)
    out, _ = _attend(d)
    torch.cuda.synchronize()
    assert torch.all(out[4:] == 7.0)
    _check(dict(d, rows=[3, 1]), out)


def test_attention_strided_rows():
    """Queries inside a projection's rows, outputs inside wider rows."""
    d = _build([6, 1], [40, 100], 4, 2, 128, 16, False)
    n = 7
    wide = _t(np.random.default_rng(0).normal(size=(n, 4 * 128 + 512)))
    wide[:, 256:768] = d["q"]
    dst = torch.full((n, 4 * 128 + 8), 7.0, dtype=BF, device=DEV)
    want, _ = _attend(d)
    got, _ = _attend(dict(d, q=wide[:, 256:768]), out=dst[:, 8:])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.all(dst[:, :8] == 7.0)


def test_attention_missing_page_is_reported():
    d = _build([1, 2], [100, 40], 4, 2, 128, 16, False)
    for bad in (-1, d["pk"].shape[0], 1 << 30):
        t = d["table"].copy()
        t[0, 3] = bad
        out, ws = _attend(dict(d, table=t))
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 1
        _check(dict(d, table=t), out)                # the slots read as zeros


def test_attention_max_rows_is_only_a_hint():
    d = _build([40, 1, 7], [30, 200, 0], 8, 2, 128, 16, False)
    for hint in (1, 7, 40, 1000):
        out, _ = _attend(d, max_rows=hint)
        torch.cuda.synchronize()
        _check(d, out)


def test_attention_in_a_graph_serves_growing_contexts():
    """Append and attention captured once: the contexts grow on the device."""
    rng = np.random.default_rng(8)
    rows, cap, n_q, n_kv, hd = [1, 2, 1], 300, 8, 2, 128
    pk, pv, table, off = _paged(rng, [0, 0, 0], [cap, cap, cap], n_kv, hd, 32)
    pages = bd.Pages(pk, pv, _i(table))
    pos0, d_off = _i([17, 150, 0]), _i(off * 0 + np.array([0, 1, 3, 4]))
    q, k, v = (_t(rng.normal(size=(4, w * hd))) for w in (n_q, n_kv, n_kv))
    out, ws = torch.empty_like(q), _ws(n_q, n_kv, hd)
    grow = _i(rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        bd.paged_append(pages, k, v, d_off, pos0, theta=THETA)
        bd.paged_attention(pages, q, d_off, pos0, 2, out, ws)
        pos0.add_(grow)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(3):
        g.replay()
        for x in (q, k, v):
            x.copy_(_t(rng.normal(size=tuple(x.shape))))
        p0 = pos0.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        d = dict(pk=pk, pv=pv, table=table, off=np.array([0, 1, 3, 4]), ctx=p0.tolist(), q=q, mask=None,
                 n_q=n_q, hd=hd, n_kv=n_kv, rows=rows)
        _check(d, out)
    assert bd.read_status(ws) == 0


def test_two_streams_with_a_workspace_each():
    a = _build([1] * 6, [900, 3, 250, 77, 1024, 600], 8, 2, 128, 16, False)
    b = _build([40], [500], 8, 2, 128, 32, False)
    want = [_attend(x)[0] for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [_ws(8, 2, 128) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for x, s, w in zip((a, b), streams, ws):
            with torch.cuda.stream(s):
                got.append(_attend(x, w)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))


# ---------------------------------------------------------------------------
# the pass as a whole
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_verification_layer_over_pages(kind):
    """norm_rope -> append -> attention of draft trees (or chains) over pages: the
    new keys and values land in the pages, and the attention is the one that
    dflash_tree_attention computes over a contiguous cache."""
    rng = np.random.default_rng(21)
    n_req, B, D, K, n_q, n_kv, hd, page = 2, 40, 6, 4, 8, 2, 128, 16
    ctx = [150, 33]
    lp = np.sort(rng.normal(size=(n_req, D, K)).astype(np.float32) - 3, axis=2)[:, :, ::-1].copy()
    ids = rng.integers(0, 1000, size=(n_req, D, K)).astype(np.int32)
    bufs = bd.tree_buffers(n_req, B)
    root = _i([3, 4])
    if kind == "tree":
        bd.ddtree_build(torch.as_tensor(lp, device=DEV), _i(ids), root, B, *bufs)
    else:
        bd.chain_tree(_i(ids), root, B, *bufs)
    n_nodes, tok, parent, depth, rank, mask = bufs
    n = n_req * (B + 1)
    pk, pv, table, off = _paged(rng, [B + 1] * n_req, ctx, n_kv, hd, page)
    pages = bd.Pages(pk, pv, _i(table))
    qkv = _t(rng.normal(size=(n, (n_q + 2 * n_kv) * hd)))
    gq, gk = (_t(1 + 0.2 * rng.normal(size=hd)) for _ in range(2))
    d_off, d_ctx = _i(off), _i(ctx)
    pos = torch.where(depth >= 0, depth + d_ctx[:, None], -1).reshape(-1).contiguous()
    q = torch.zeros(n, n_q * hd, dtype=BF, device=DEV)
    k = torch.zeros(n, n_kv * hd, dtype=BF, device=DEV)
    v = qkv[:, (n_q + n_kv) * hd:].contiguous()
    bd.qk_norm_rope(qkv[:, :n_q * hd], qkv[:, n_q * hd:(n_q + n_kv) * hd], gq, gk, 1e-6, THETA, pos, hd,
                    q, k)
    # rows past the last node are stored nowhere: their slots keep NaN
    for r in range(n_req):
        for t in range(ctx[r], ctx[r] + B + 1):
            pk[table[r, t // page], :, t % page] = float("nan")
            pv[table[r, t // page], :, t % page] = float("nan")
    bd.paged_append(pages, k, v, d_off, d_ctx, pos=pos)
    out = torch.empty_like(q)
    ws = _ws(n_q, n_kv, hd)
    bd.paged_attention(pages, q, d_off, d_ctx, B + 1, out, ws, mask=mask.view(n, -1))
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 0
    # the contiguous form
    cap = 192
    ck = torch.zeros(n_req, n_kv, cap, hd, dtype=BF, device=DEV)
    cv = torch.zeros_like(ck)
    for r in range(n_req):
        for t in range(ctx[r]):
            ck[r, :, t] = pk[table[r, t // page], :, t % page]
            cv[r, :, t] = pv[table[r, t // page], :, t % page]
    ref = torch.empty(n_req, B + 1, n_q * hd, dtype=BF, device=DEV)
    tws = torch.zeros(bd.tree_attention_workspace_bytes(n_req, n_q, n_kv, hd, B, max(ctx)),
                      dtype=torch.uint8, device=DEV)
    bd.tree_attention(q.view(n_req, B + 1, -1), k.view(n_req, B + 1, -1), v.view(n_req, B + 1, -1), ck, cv,
                      d_ctx, max(ctx), mask, n_nodes, ref, tws)
    torch.cuda.synchronize()
    nn = n_nodes.cpu().numpy()
    assert (nn == (min(B, D) if kind == "chain" else B)).all()
    for r in range(n_req):
        for i in range(nn[r] + 1):
            a, b = _f64(out[r * (B + 1) + i]), _f64(ref[r, i])
            # both round each probability and the output to bf16: 2^-8 of the
            # values' size (N(0, 1), at most 5) for each, on both sides
            assert np.max(np.abs(a - b)) <= 4 * 2.0 ** -8 * 5
            assert np.linalg.norm(a - b) <= 2.0 ** -6 * np.linalg.norm(b)


@pytest.mark.parametrize("rows,tree", [([1, 2], False), ([16], False), ([70, 3], False), ([90], True)])
def test_attention_maxima_that_climb(rows, tree):
    """Scores up to a few hundred apart, the largest ones late: the running maximum
    moves by little, by much and by more than a step may lag, in every kernel."""
    d = _build(rows, [900, 400][:len(rows)], 8, 2, 128, 16, tree, seed=4)
    d["q"] = d["q"] * 16
    for r in range(len(rows)):
        kv = d["ctx"][r] + rows[r]
        for t in range(kv):
            d["pk"][d["table"][r, t // 16], :, t % 16] *= 0.05 + (t / kv) ** 3
    out, _ = _attend(d)
    torch.cuda.synchronize()
    _check(d, out)


def test_pools_past_32_bit_offsets():
    """Pages whose elements lie beyond 2^32 (9.8 GB pools)."""
    rng = np.random.default_rng(31)
    n_pages, n_kv, page, hd, n_q = 300_000, 8, 16, 128, 32
    assert n_pages * n_kv * page * hd > 2 ** 32
    pk = torch.empty(n_pages, n_kv, page, hd, dtype=BF, device=DEV)
    pv = torch.empty_like(pk)
    for rows, ctx in (([1, 2], [70, 31]), ([20], [60]), ([100], [40])):
        need = [-(-(n + c) // page) for n, c in zip(rows, ctx)]
        ids = rng.choice(np.arange(n_pages - 5000, n_pages), size=sum(need), replace=False).astype(np.int32)
        table = np.full((len(rows), max(need)), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = ids[at:at + n]
            at += n
        n = sum(rows)
        small = (sum(need), n_kv, page, hd)
        pk[ids.tolist()], pv[ids.tolist()] = _t(rng.normal(size=small)), _t(rng.normal(size=small))
        off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        k, v = (_t(rng.normal(size=(n, n_kv * hd))) for _ in range(2))
        pages = bd.Pages(pk, pv, _i(table))
        bd.paged_append(pages, k, v, _i(off), _i(ctx))
        q, ws = _t(rng.normal(size=(n, n_q * hd))), _ws(n_q, n_kv, hd)
        out = torch.empty_like(q)
        bd.paged_attention(pages, q, _i(off), _i(ctx), max(rows), out, ws)
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 0
        # the same on pools of these pages alone
        again = {int(p): i for i, p in enumerate(ids)}
        own = np.vectorize(lambda p: again.get(int(p), -1))(table).astype(np.int32)
        d = dict(pk=pk[ids.tolist()], pv=pv[ids.tolist()], table=own, off=off, ctx=ctx, q=q, mask=None, n_q=n_q, hd=hd,
                 n_kv=n_kv, rows=rows)
        for r in range(len(rows)):
            for i in range(rows[r]):
                t = ctx[r] + i
                assert torch.equal(d["pv"][own[r, t // page], :, t % page].reshape(-1), v[off[r] + i])
        _check(d, out)


@pytest.mark.parametrize("rows,ctx,n_q,n_kv,hd,page,tree", [
    ([16] * 10 + [7], [50 + 61 * i for i in range(11)], 32, 8, 128, 16, False),
    ([16] * 10 + [7], [50 + 61 * i for i in range(11)], 32, 8, 64, 64, True),
    ([150, 90, 33], [300, 700, 0], 32, 8, 128, 64, False),
    ([150, 90, 33], [300, 700, 0], 32, 8, 128, 16, True),
    ([600], [500], 16, 8, 64, 128, False),
    ([260, 300], [90, 31], 16, 8, 64, 32, True),
])
def test_attention_more_tiles_than_parts(rows, ctx, n_q, n_kv, hd, page, tree):
    """Tiles enough that each falls into few parts, which the CTAs join themselves."""
    test_attention((rows, ctx, n_q, n_kv, hd, page, tree))


@pytest.mark.parametrize("rows,ctx,n_q,n_kv,hd,tree", [
    ([16], [30000], 4, 1, 128, False), ([12], [27000], 4, 1, 64, True), ([64], [10000], 4, 1, 128, False),
    ([33], [7000], 8, 1, 64, True), ([100, 0, 1], [4000, 3, 800], 4, 1, 128, False)])
def test_attention_few_tiles_in_many_parts(rows, ctx, n_q, n_kv, hd, tree):
    """One long context on all SMs: tens of parts to a tile, more than are weighed at once."""
    test_attention((rows, ctx, n_q, n_kv, hd, 16, tree))


@pytest.mark.parametrize("n,n_q", [(10, 2), (30, 4), (90, 8)])
def test_attention_pages_that_no_row_sees_may_be_missing(n, n_q):
    """A draft tree in a request of more rows (those past its last node see nothing new):
    pages behind the last node need not be there.  With a bit for one of them they do."""
    d = _build([n, 2], [24, 40], n_q, 2, 128, 16, True, seed=2)
    nodes = n // 2
    d["mask"][nodes:n] = 0
    d["table"][0, -(-(24 + nodes) // 16):] = -1
    out, ws = _attend(d)
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 0
    _check(d, out)
    j = n - 1
    d["mask"][1, j // 32] |= np.uint32(1 << (j % 32))
    out, ws = _attend(d)
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 1
    _check(d, out)                                   # the slot reads as zeros


@pytest.mark.parametrize("n,n_q", [(3, 2), (30, 4), (90, 8)])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_slots_past_the_table_are_reported(n, n_q, tree):
    """Slots that a row sees past its page table: an error in the status word, and the
    softmax runs over the slots that the table has."""
    def status(d):
        out, ws = _attend(d)
        torch.cuda.synchronize()
        got = bd.read_status(ws)
        _check(dict(d, ctx=[min(c, cap) for c in d["ctx"]]), out)   # (past the table: all of it is seen)
        return got

    cap = 160
    base = _build([n, 2], [cap - n, 40], n_q, 2, 128, 16, tree, seed=6)
    assert base["table"].shape[1] * 16 == cap
    assert status(base) == 0                         # up to the table's last slot
    for p0 in (cap - n + 1, cap - 1, cap, cap + 1, 1 << 30, 2 ** 31 - 1):
        assert status(dict(base, ctx=[p0, 40])) == 1, p0
        # a request without rows sees nothing
        none = dict(base, off=np.array([0, 0, 2], dtype=np.int32), ctx=[p0, 40], rows=[0, 2])
        assert status(none) == 0, p0
    out, ws = _attend(dict(base, ctx=[-1, 40]))
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 1                   # there is no slot before the first
    if tree:
        # the rows past a tree's last node may lie past the table: no row sees them
        m = base["mask"].copy()
        m[n // 2:n] = 0
        assert status(dict(base, mask=m, ctx=[cap - n // 2, 40])) == 0
        m[0, (n - 1) // 32] |= np.uint32(1 << ((n - 1) % 32))
        assert status(dict(base, mask=m, ctx=[cap - n // 2, 40])) == 1


def test_one_row_out_of_a_wider_tensor():
    """The row stride of a single row says nothing: keys out of a projection's row beside
    values of their own, and rows whose stride is no multiple of eight."""
    rng = np.random.default_rng(17)
    pk, pv, table, off = _paged(rng, [1], [20], 2, 64, 16)
    kv = _t(rng.normal(size=(3, 300)))
    k, v = kv[1:2, 8:136], kv[1:2, 136:264].clone()
    a, b = pk.clone(), pv.clone()
    bd.paged_append(bd.Pages(a, b, _i(table)), k, v, _i(off), _i([20]), theta=THETA)
    c, e = pk.clone(), pv.clone()
    bd.paged_append(bd.Pages(c, e, _i(table)), k.clone(), v, _i(off), _i([20]), theta=THETA)
    wide = _t(rng.normal(size=(2, 261)))
    q, out = wide[:1, :256], torch.full((1, 259), 7.0, dtype=BF, device=DEV)[:, :256]
    want, ws = torch.empty(1, 256, dtype=BF, device=DEV), _ws(4, 2, 64)
    pages = bd.Pages(a, b, _i(table))
    bd.paged_attention(pages, q.clone(), _i(off), _i([20]), 1, want, ws)
    bd.paged_attention(pages, q, _i(off), _i([20]), 1, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(b, e) and torch.equal(out, want)
    # in place and out of place, of two strides
    g = _t(rng.normal(size=64))
    pos = _i([5])
    y = torch.empty(1, 256, dtype=BF, device=DEV)
    bd.qk_norm_rope(q, None, g, None, 1e-6, THETA, pos, 64, y)
    bd.qk_norm_rope(q, None, g, None, 1e-6, THETA, pos, 64)
    torch.cuda.synchronize()
    assert torch.equal(q, y)


def test_attention_refuses_a_mask_of_no_words():
    """(Its pointer is null, which the library takes as causal.)"""
    d = _build([1, 2], [100, 40], 4, 2, 128, 16, False)
    d["mask"] = np.zeros((3, 0), dtype=np.uint32)
    with pytest.raises(ValueError, match="mask"):
        _attend(d)


def test_trace_hook_sees_every_launch():
    """One pair of callbacks to a kernel, the join of tiles in many parts among them."""
    seen = []
    bd.set_trace_hook(lambda kernel, phase, stream: seen.append((kernel, phase)))
    try:
        for rows, names in (([1], ["paged_attn_small"]), ([40], ["paged_attn_tc", "paged_join"]),
                            ([4000], ["paged_attn_tc"])):
            d = _build(rows, [600], 8, 8, 64, 64, False)
            seen.clear()
            _attend(d)
            torch.cuda.synchronize()
            assert seen == [(n, p) for n in names for p in (0, 1)]
    finally:
        bd.set_trace_hook(None)


@pytest.mark.parametrize("rows,n_q", [([1] * 60, 14), ([2, 3, 0, 4] * 10, 8), ([7, 20] * 4, 6), ([40, 100], 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_what_no_row_sees_changes_no_bit(rows, n_q, bad):
    """Slots between others that no row's mask has a bit for, of NaN keys and of values
    that are not finite; some rows see nothing new, some nothing at all."""
    for seed in range(4):
        rng = np.random.default_rng(seed)
        ctx = [int(c) * (i % 5 > 0) for i, c in enumerate(rng.integers(1, 60, size=len(rows)))]
        d = _build(rows, ctx, n_q, 2, 128, 64, True, seed=seed)
        m = (rng.integers(0, 1 << 32, size=d["mask"].shape) & rng.integers(0, 1 << 32, size=d["mask"].shape)).astype(np.uint32)
        m[rng.random(len(m)) < 0.4] = 0
        d["mask"] = m
        clean, ws = _attend(d)
        dirty = dict(d, pk=torch.full_like(d["pk"], float("nan")), pv=torch.full_like(d["pv"], bad))
        for r, (n, c) in enumerate(zip(rows, ctx)):
            a = d["off"][r]
            for t in np.flatnonzero(op.visible(n, c, n + c, m[a:a + n]).any(0)):
                pg = d["table"][r, t // 64]
                dirty["pk"][pg, :, t % 64] = d["pk"][pg, :, t % 64]
                dirty["pv"][pg, :, t % 64] = d["pv"][pg, :, t % 64]
        got, _ = _attend(dirty, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, clean)
        _check(d, got)
