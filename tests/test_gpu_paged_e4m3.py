"""GPU parity of the 8-bit paged cache (append, attention) against the 64-bit oracle,
through the C ABI.

Tolerances, element by element:
- append: a code stands for the value before rounding to half a step: 2^-4 of it, or half
  of the codes' smallest step, 2^-10, times the scale; a rotated key adds what fp32 does
  before that (test_gpu_paged.py), which may move it over the border between two codes.
  Scales are equal unless that error crosses a border between two of them.  Values and
  unrotated keys, and earlier tokens' codes at an unchanged scale, are equal.
- attention: weights are rounded to fp16, half a step 2^-11 of sum p |v| (the oracle's
  spread), and below fp16's normal range by 2^-25 of the largest weight: with
  W = max over keys of p 2^b (b the value block's exponent), W 2^-25 sum |d| over the
  keys' value codes d; the output to bf16, 2^-8 |ref|; fp32 sums over kv keys add
  kv 2^-24 of the spread, twice; a score's fp32 sum of head_dim products, the rounding of q's
  elements (fp16: 2^-39 of the row's largest; two codes: 2^-17 of it, so that at most
  2^-17 max|q| sum |k| / sqrt(hd) <= 2^-17 max|q| |k|) and an exponential's 2^-22 move the
  exponents by delta = (head_dim + 8) 2^-24 S + 2^-17 max|q| |k| + 2^-20, S a bound of
  sum |q k| / sqrt(hd).  A probability p = e^s / sum e^s then lies between p e^(-2 delta) and
  p e^(2 delta), so that sum |p' - p| |v| <= (e^(2 delta) - 1) sum p |v| (2 delta of the
  spread where delta is small; nothing is claimed where scores pass fp32's resolution)."""
import math

import numpy as np
import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding as bd
from oracle import paged as op
from oracle import quant as oq
from test_gpu_paged import BF, CASES, DEV, F32, THETA, _f64, _i, _paged, _t, _tree_mask

pytestmark = pytest.mark.gpu
WIDE = 1 << 17         # slots of a page table that may hold long requests


def _u8(a):
    return torch.as_tensor(np.asarray(a, dtype=np.uint8), device=DEV)


def _ws(n_q, n_kv, hd):
    return torch.zeros(bd.paged_attention_e4m3_workspace_bytes(n_q, n_kv, hd), dtype=torch.uint8, device=DEV)


def _np(t):
    return t.view(torch.uint8).cpu().numpy()


def _pool(rng, total, n_kv, page, hd, spread=1.0, center=119):
    """Codes of all sizes (none NaN) and scales some octaves apart."""
    x = np.abs(rng.normal(size=(total, n_kv, page, hd))) * 100
    codes = oq.encode(np.minimum(x, 448.0)) + 128 * rng.integers(0, 2, size=x.shape).astype(np.uint8)
    scale = np.clip(np.round(rng.normal(size=(total, n_kv, page // 16)) * spread) + center, 0, 254).astype(np.uint8)
    return codes.astype(np.uint8), scale


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,ctx,n_kv,hd,page,dtype,theta,pad", [
    ([1], [0], 8, 128, 16, BF, THETA, 0),
    ([1, 0, 5, 17], [15, 9, 0, 30], 2, 64, 16, BF, THETA, 0),
    ([40, 1, 3], [100, 63, 64], 1, 128, 64, F32, THETA, 0),
    ([0, 0, 33], [5, 5, 5], 5, 64, 32, F32, 0.0, 3),
    ([130, 2], [7, 1000], 3, 128, 1024, BF, THETA, 1),      # rows off 16-byte boundaries
    ([2] * 70, list(range(70)), 1, 64, 16, BF, THETA, 0),   # more requests than a warp
    ([0] * 40 + [1, 31] + [0] * 50, list(range(92)), 2, 64, 16, BF, 0.0, 0),
    ([7], [2], 40, 128, 16, BF, THETA, 0),                  # more heads than one round of a CTA
    ([900, 0, 303], [40, 7, 100], 2, 128, 32, BF, THETA, 0),
    ([16] * 600, [16 * (i % 3) + 1 for i in range(600)], 1, 64, 16, BF, 0.0, 0),    # all of a block to a CTA
    ([1, 1099], [0, 3], 3, 64, 16, F32, THETA, 1),
])
def test_append(rows, ctx, n_kv, hd, page, dtype, theta, pad):
    rng = np.random.default_rng(len(rows) * 7 + hd)
    _, _, table, off = _paged(rng, rows, ctx, 1, 1, page)
    total = int(table.max()) + 4
    (ck, sk), (cv, sv) = (_pool(rng, total, n_kv, page, hd) for _ in range(2))
    n = sum(rows)
    kv = rng.normal(size=(n + 2, 2 * n_kv * hd + pad)) * np.exp(2 * rng.normal(size=(n + 2, 1)))
    kv = _t(kv, dtype)                                               # two rows behind the last one
    k, v = kv[:, :n_kv * hd], kv[:, n_kv * hd:2 * n_kv * hd]
    k64, v64 = (_f64(x).reshape(n + 2, n_kv, hd) for x in (k, v))
    for pos in (None, rng.integers(-1, 5000, size=n + 2).astype(np.int32)):
        got = [_u8(a) for a in (ck, cv, sk, sv)]
        bd.paged_append_e4m3(bd.PagesE4M3(*got, _i(table)), k, v, _i(off), _i(ctx), theta=theta,
                             pos=None if pos is None else _i(pos))
        torch.cuda.synchronize()
        gk, gv, gsk, gsv = (t.cpu().numpy() for t in got)
        rk, rv, rsk, rsv, ek, ev = oq.append(ck, cv, sk, sv, table, off, ctx, k64, v64, theta, pos)
        assert np.array_equal(gv, rv) and np.array_equal(gsv, rsv)
        new = np.isfinite(ek)
        assert np.array_equal(new, np.isfinite(ev))
        if theta == 0:
            assert np.array_equal(gk, rk) and np.array_equal(gsk, rsk)
            continue
        # the size of the pair that was turned, laid out as the pool is
        flat = oq.append(ck, cv, sk, sv, table, off, ctx, np.abs(k64), v64, 0.0, pos)[4]
        pair = np.nan_to_num(flat[..., :hd // 2] + flat[..., hd // 2:])
        err = ((hd + 32) * 2.0 ** -24 + 2.0 ** -21) * np.concatenate([pair, pair], -1)
        for at in np.argwhere(gsk != rsk):                           # only where fp32 decides
            pg, g, b = at
            blk = np.s_[pg, g, 16 * b:16 * b + 16]
            lo, hi = ((np.abs(np.nan_to_num(ek[blk])) + s * err[blk]).max() for s in (-1, 1))
            assert oq.exponent(lo) <= int(gsk[pg, g, b]) - 127 <= oq.exponent(hi)
        e = np.repeat(gsk.astype(np.float64) - 127, 16, axis=2)[..., None]
        step = np.maximum(2.0 ** -4 * (np.abs(ek) + err), 2.0 ** (e - 10))
        off_by = np.abs(oq.held(gk, gsk) - ek)
        assert np.all((off_by <= step + err)[new])
        same = np.repeat(gsk == rsk, 16, axis=2)[..., None] & ~new
        assert np.array_equal(gk[same], rk[same])


def test_append_special_values():
    """Infinities and NaN are stored as NaN and count for no scale; zeros, the smallest and
    the largest numbers; a block of nothing else."""
    n_kv, hd = 2, 64
    x = np.zeros((16, n_kv * hd))
    x[0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    x[1, :3] = [448.0, -0.0, 2.0 ** -9]
    x[2, 64:70] = [3.3e38, -1.0, 1e-38, np.inf, 1e30, -3.3e38]
    table = np.array([[1, 0, 2]], dtype=np.int32)
    for dtype in (BF, F32):
        for rows, p0 in ((16, 0), (3, 5), (2, 31), (1, 0)):
            k, v = _t(x[:rows], dtype), _t(x[:rows][:, ::-1].copy() * 1e-40, dtype)
            ck, sk = _pool(np.random.default_rng(1), 3, n_kv, 16, hd)
            got = [_u8(a) for a in (ck, ck, sk, sk)]
            bd.paged_append_e4m3(bd.PagesE4M3(*got, _i(table)), k, v, _i([0, rows]), _i([p0]))
            torch.cuda.synchronize()
            ref = oq.append(ck, ck, sk, sk, table, [0, rows], [p0], *(
                _f64(t).reshape(rows, n_kv, hd) for t in (k, v)), 0.0)
            for g, r in zip(got, ref):
                g = g.cpu().numpy()
                if g.ndim == 4:                                      # (either code of NaN)
                    g, r = (np.where(a & 127 == 127, 127, a) for a in (g, r))
                assert np.array_equal(g, r)


def test_append_token_by_token():
    """Tokens one by one, the scale growing under earlier ones, drafted ones taken back:
    as the oracle has it, step by step; and close to what one call would store."""
    rng = np.random.default_rng(3)
    n_kv, hd, page = 2, 128, 32
    table = np.array([[2, 0]], dtype=np.int32)
    x = rng.normal(size=(40, n_kv * hd)) * np.exp(3 * rng.normal(size=(40, 1)))
    k, v = _t(x, F32), _t(x[::-1].copy(), F32)
    ck, sk = _pool(rng, 3, n_kv, page, hd)
    state = [ck, ck.copy(), sk, sk.copy()]
    got = [_u8(a) for a in state]
    pages = bd.PagesE4M3(*got, _i(table))
    p0 = 0
    for take, keep in ((1, 1), (3, 2), (1, 1), (5, 1), (9, 9), (4, 3), (1, 1), (7, 5), (2, 2), (6, 6)):
        bd.paged_append_e4m3(pages, k[p0:p0 + take], v[p0:p0 + take], _i([0, take]), _i([p0]))
        torch.cuda.synchronize()
        state = list(oq.append(*state, table, [0, take], [p0], *(
            _f64(t[p0:p0 + take]).reshape(take, n_kv, hd) for t in (k, v)), 0.0)[:4])
        for g, r in zip(got, state):
            assert np.array_equal(g.cpu().numpy(), r)
        p0 += keep
    one = [_u8(a) for a in (ck, ck, sk, sk)]
    bd.paged_append_e4m3(bd.PagesE4M3(*one, _i(table)), k[:p0], v[:p0], _i([0, p0]), _i([0]))
    a, b = (oq.held(g[0].cpu().numpy(), g[2].cpu().numpy())[2, :, :p0 % 32 or 32] for g in (got, one))
    # both within half a step of the same values, of the larger scale's steps at least
    assert np.linalg.norm(a - b) <= 2.0 ** -3 * np.linalg.norm(b)


def test_append_without_a_page_stores_nothing():
    rng = np.random.default_rng(5)
    ck, sk = _pool(rng, 7, 2, 16, 64)
    table = np.array([[4, -1, 7, 0]], dtype=np.int32)        # 16..31: none; 32..47: one past the pool
    x = _t(rng.normal(size=(40, 128)))
    got = [_u8(a) for a in (ck, ck, sk, sk)]
    ref = [ck, ck, sk, sk]
    x64 = _f64(x).reshape(40, 2, 64)
    for p0 in (10, 60, 64, 1 << 30, 2 ** 31 - 1, -7, -100):
        bd.paged_append_e4m3(bd.PagesE4M3(*got, _i(table)), x, x, _i([0, 40]), _i([p0]))
        ref = list(oq.append(*ref, table, [0, 40], [p0], x64, x64, 0.0)[:4])
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        assert np.array_equal(g.cpu().numpy(), r)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _build(rows, ctx, n_q, n_kv, hd, page, tree, seed=0, spare=3, spread=1.0):
    rng = np.random.default_rng(seed + sum(rows) + sum(ctx))
    _, _, table, off = _paged(rng, rows, ctx, 1, 1, page, spare=spare)
    total = int(table.max()) + 1 + spare
    ck, sk = _pool(rng, total, n_kv, page, hd, spread)
    cv, sv = _pool(rng, total, n_kv, page, hd, spread)
    mask = _tree_mask(rng, rows, (max(rows) + 31) // 32) if tree else None
    return dict(ck=ck, cv=cv, sk=sk, sv=sv, table=table, off=off, ctx=ctx, q=_t(rng.normal(size=(sum(rows), n_q * hd))),
                mask=mask, n_q=n_q, hd=hd, n_kv=n_kv, rows=rows)


def _attend(d, ws=None, out=None, max_rows=None, stream=None):
    out = torch.full_like(d["q"], 7.0) if out is None else out
    ws = _ws(d["n_q"], d["n_kv"], d["hd"]) if ws is None else ws
    mask = None if d["mask"] is None else torch.as_tensor(d["mask"].view(np.int32), device=DEV)
    table = _i(d["table"])
    if d.get("wide"):                                # as a serving loop keeps it: for lengths to come
        table = torch.nn.functional.pad(table, (0, WIDE // d["ck"].shape[2]), value=-1)
    pages = bd.PagesE4M3(*(_u8(d[x]) for x in ("ck", "cv", "sk", "sv")), table)
    bd.paged_attention_e4m3(pages, d["q"], _i(d["off"]), _i(d["ctx"]), max(d["rows"]) if max_rows is None else max_rows,
                            out, ws, mask=mask, stream=stream)
    return out, ws


def _small_weights(d, q):
    """W sum |d| of every (row, head, column), as in the tolerances above."""
    n_kv, hd, page = d["n_kv"], d["hd"], d["ck"].shape[2]
    out = np.zeros(q.shape)
    pk = oq.held(d["ck"], d["sk"])
    codes = np.abs(np.nan_to_num(oq.VALUES[d["cv"]]))
    for r in range(len(d["rows"])):
        a, b = d["off"][r], min(d["off"][r + 1], q.shape[0])
        if b <= a:
            continue
        kv = min(d["ctx"][r] + b - a, d["table"].shape[1] * page)
        see = op.visible(b - a, d["ctx"][r], kv, None if d["mask"] is None else d["mask"][a:b])
        ks, ds = op.slots(pk, d["table"][r], kv), op.slots(codes, d["table"][r], kv)
        e = op.slots(np.repeat(d["sv"].astype(float) - 127, 16, axis=2)[..., None], d["table"][r], kv)[..., 0]
        for h in range(d["n_q"]):
            g = h // (d["n_q"] // n_kv)
            s = q[a:b, h] @ np.nan_to_num(ks[g]).T / math.sqrt(hd)
            s = np.where(see, s, -np.inf)
            top = s.max(1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
            w = (p * 2.0 ** e[g]).max(1)
            out[a:b, h] = w[:, None] * (see.astype(float) @ ds[g])
    return out


def _check(d, out):
    n, hd = d["q"].shape[0], d["hd"]
    q = _f64(d["q"]).reshape(n, d["n_q"], hd)
    pk, pv = oq.held(d["ck"], d["sk"]), oq.held(d["cv"], d["sv"])
    ref, spread = op.attention(q, pk, pv, d["table"], d["off"], d["ctx"], d["n_q"], d["mask"])
    used = np.unique(d["table"][(d["table"] >= 0) & (d["table"] < len(pk))])
    key = np.linalg.norm(np.nan_to_num(pk[used]), axis=-1).max() if len(used) else 0.0
    kv = max(a + b for a, b in zip(d["rows"], d["ctx"]))
    s = np.linalg.norm(q, axis=-1, keepdims=True) * key / math.sqrt(hd)
    top = np.abs(q).max(-1, keepdims=True)
    delta = (hd + 8) * 2.0 ** -24 * s + 2.0 ** -17 * top * key + 2.0 ** -20 + kv * 2.0 ** -24
    tol = (2.0 ** -11 + np.expm1(np.minimum(2 * delta, 300.0))) * spread * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(ref) + \
        2.0 ** -25 * _small_weights(d, q) * (1 + 2.0 ** -7) + 1e-30
    live = int(d["off"][-1])
    got = _f64(out).reshape(q.shape)
    err = np.abs(got - ref)[:live]
    assert np.isfinite(got[:live]).all()
    assert (err <= tol[:live]).all(), float((err / tol[:live]).max())


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


@pytest.mark.parametrize("rows,ctx,n_q,n_kv,hd,page,tree", [
    ([16] * 10 + [7], [50 + 61 * i for i in range(11)], 32, 8, 128, 16, False),
    ([16] * 10 + [7], [50 + 61 * i for i in range(11)], 32, 8, 64, 64, True),
    ([150, 90, 33], [300, 700, 0], 32, 8, 128, 64, False),
    ([150, 90, 33], [300, 700, 0], 32, 8, 128, 16, True),
    ([600], [500], 16, 8, 64, 128, False),
    ([260, 300], [90, 31], 16, 8, 64, 32, True),
    ([1], [60000], 4, 1, 128, 64, False), ([2], [40000], 4, 1, 64, 16, True),
    ([16], [30000], 4, 1, 128, 16, False), ([12], [27000], 4, 1, 64, 16, True), ([64], [10000], 4, 1, 128, 16, False),
    ([33], [7000], 8, 1, 64, 16, True), ([100, 0, 1], [4000, 3, 800], 4, 1, 128, 16, False)])
def test_attention_tiles_in_few_and_many_parts(rows, ctx, n_q, n_kv, hd, page, tree):
    test_attention((rows, ctx, n_q, n_kv, hd, page, tree))


@pytest.mark.parametrize("case", [c for c in CASES if 8 < max(c[0]) * c[2] // c[3] <= 64] + [
    ([4], [700], 32, 8, 128, 16, False), ([7, 0, 5], [300, 9, 0], 4, 2, 64, 64, True), ([3], [20000], 5, 1, 128, 32, False),
    ([8, 2], [100, 3000], 8, 2, 128, 16, True)], ids=str)
def test_attention_wide_table(case):
    """Tables for many slots take other tiles than those that hold few."""
    d = dict(_build(*case), wide=True)
    out, ws = _attend(d)
    again, _ = _attend(d, ws)
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 0
    _check(d, out)
    assert torch.equal(out, again)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,tree", [([1, 2], False), ([4], False), ([16], False), ([70, 3], False), ([90], True),
                                       ([300], False)])
@pytest.mark.parametrize("spread,q_size", [(8.0, 2.0 ** -14), (3.0, 1.0), (0.0, 3e4), (1.0, 1e-30), (20.0, 1e-6)])
def test_attention_scales_far_apart(rows, tree, spread, q_size, wide):
    """Blocks whose scales differ by many octaves, queries of any size: maxima that climb
    by little, by much and by more than a step may lag."""
    d = dict(_build(rows, [900, 400][:len(rows)], 8, 2, 128, 16, tree, seed=4, spread=spread), wide=wide)
    d["q"] = (d["q"].float() * q_size).to(BF)
    if q_size > 1:
        d["sk"] = (d["sk"] - 14).astype(np.uint8)
    out, ws = _attend(d)
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 0
    _check(d, out)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,tree", [([1, 1], False), ([3, 1], False), ([6, 1], True), ([20, 3], False), ([20, 3], True),
                                       ([300, 40], False), ([140, 40], True)])
def test_attention_ignores_what_no_row_may_see(rows, tree, wide):
    """NaN codes in slots past the requests' ends and in pages of nobody, any scales in
    blocks that hold no token."""
    d = dict(_build(rows, [70, 9], 8, 2, 128, 16, tree), wide=wide)
    clean, _ = _attend(d)
    for byte in (0, 255):
        dirty = dict(d, ck=np.full_like(d["ck"], 127), cv=np.full_like(d["cv"], 255), sk=np.full_like(d["sk"], byte),
                     sv=np.full_like(d["sv"], byte))
        for r in range(2):
            for t in range(rows[r] + d["ctx"][r]):
                pg = d["table"][r, t // 16]
                for x in ("ck", "cv"):
                    dirty[x][pg, :, t % 16] = d[x][pg, :, t % 16]
                for x in ("sk", "sv"):
                    dirty[x][pg] = d[x][pg]
        got, ws = _attend(dirty)
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 0
        assert torch.equal(got, clean)


@pytest.mark.parametrize("rows,n_q", [([1] * 60, 14), ([2, 3, 0, 4] * 10, 8), ([7, 20] * 4, 6), ([40, 100], 8)])
@pytest.mark.parametrize("bad", [127, 255])
@pytest.mark.parametrize("wide", [False, True])
def test_attention_what_no_row_sees_changes_no_bit(rows, n_q, bad, wide):
    """NaN keys and values between others that no row's mask has a bit for; some rows see
    nothing new, some nothing at all."""
    for seed in range(3):
        rng = np.random.default_rng(seed)
        ctx = [int(c) * (i % 5 > 0) for i, c in enumerate(rng.integers(1, 60, size=len(rows)))]
        d = dict(_build(rows, ctx, n_q, 2, 128, 64, True, seed=seed), wide=wide)
        m = (rng.integers(0, 1 << 32, size=d["mask"].shape) & rng.integers(0, 1 << 32, size=d["mask"].shape)).astype(np.uint32)
        m[rng.random(len(m)) < 0.4] = 0
        d["mask"] = m
        clean, ws = _attend(d)
        dirty = dict(d, ck=np.full_like(d["ck"], bad), cv=np.full_like(d["cv"], bad))
        for r, (n, c) in enumerate(zip(rows, ctx)):
            a = d["off"][r]
            for t in np.flatnonzero(op.visible(n, c, n + c, m[a:a + n]).any(0)):
                pg = d["table"][r, t // 64]
                for x in ("ck", "cv"):
                    dirty[x][pg, :, t % 64] = d[x][pg, :, t % 64]
        got, _ = _attend(dirty, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, clean)
        _check(d, got)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n,ctx,tree", [(3, 40, False), (7, 40, False), (14, 3, True), (20, 40, False), (20, 0, True),
                                        (200, 130, False), (140, 100, True)])
def test_attention_bad_value_reaches_only_the_rows_that_see_it(n, ctx, tree, wide):
    for hd in (64, 128):
        d = dict(_build([n], [ctx], 4, 2, hd, 16, tree, seed=3), wide=wide)
        clean, _ = _attend(d)
        j = n // 2                                   # the new token whose value is bad
        pg = int(d["table"][0, (ctx + j) // 16])
        cv = d["cv"].copy()
        for col in (5, 48):
            cv[pg, 1, (ctx + j) % 16, col] = 127 if col == 5 else 255
        out, _ = _attend(dict(d, cv=cv))
        torch.cuda.synchronize()
        o = out.view(n, 4, hd)
        see = op.visible(n, ctx, n + ctx, d["mask"])[:, ctx + j]
        hit = torch.zeros(n, 4, hd, dtype=torch.bool, device=DEV)
        for col in (5, 48):
            hit[torch.as_tensor(see, device=DEV), 2:, col] = True
        assert see.any() and not see.all()
        assert torch.isnan(o[hit]).all()
        assert torch.equal(torch.isfinite(o), ~hit)
        assert torch.equal(o[~hit], clean.view(n, 4, hd)[~hit])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n,ctx", [(3, 40), (7, 40), (20, 40), (90, 40)])
def test_attention_bad_key_reaches_the_rows_that_see_it(n, ctx, wide):
    d = dict(_build([n], [ctx], 4, 2, 128, 16, False, seed=3), wide=wide)
    clean, _ = _attend(d)
    j = n // 2
    ck = d["ck"].copy()
    ck[int(d["table"][0, (ctx + j) // 16]), 1, (ctx + j) % 16, 77] = 127
    out, _ = _attend(dict(d, ck=ck))
    torch.cuda.synchronize()
    o, c = (x.view(n, 4, 128).double() for x in (out, clean))
    assert torch.isnan(o[j:, 2:]).all()
    # elsewhere the same up to when sums are rescaled: twice the roundings of weights
    # (2^-11 of sum p |v|) and of outputs
    tol = 2.0 ** -7 * c.abs() + 2.0 ** -9 * np.nanmax(np.abs(oq.held(d["cv"], d["sv"])))
    near = (o - c).abs() <= tol
    assert near[:j].all() and near[:, :2].all()


def test_attention_masks_at_the_edges():
    """Rows with no bit set (the context alone; zeros where there is none), bits
    that are not causal, and bits past the request's rows."""
    for n_q in (2, 4, 16, 64):
        d = _build([5, 4], [20, 0], n_q, 1, 128, 16, True, seed=9)
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
    for n_q in (2, 4, 32):
        d = _build([3, 2], [30, 8], n_q, 2, 64, 16, False)
        d["off"] = np.array([0, 3, 4], dtype=np.int32)
        out, _ = _attend(d)
        torch.cuda.synchronize()
        assert torch.all(out[4:] == 7.0)
        _check(dict(d, rows=[3, 1]), out)


@pytest.mark.parametrize("n", [2, 6, 60])
def test_attention_strided_rows(n):
    """Queries inside a projection's rows, outputs inside wider rows."""
    d = _build([n, 1], [40, 100], 4, 2, 128, 16, False)
    wide = _t(np.random.default_rng(0).normal(size=(n + 1, 4 * 128 + 512)))
    wide[:, 256:768] = d["q"]
    dst = torch.full((n + 1, 4 * 128 + 8), 7.0, dtype=BF, device=DEV)
    want, _ = _attend(d)
    got, _ = _attend(dict(d, q=wide[:, 256:768]), out=dst[:, 8:])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.all(dst[:, :8] == 7.0)


def test_attention_missing_page_is_reported():
    for rows in ([1, 2], [40, 3], [200, 1]):
        d = _build(rows, [100, 40], 4, 2, 128, 16, False)
        for bad in (-1, d["ck"].shape[0], 1 << 30):
            t = d["table"].copy()
            t[0, 3] = bad
            out, ws = _attend(dict(d, table=t))
            torch.cuda.synchronize()
            assert bd.read_status(ws) == 1
            _check(dict(d, table=t), out)            # the slots read as zeros


@pytest.mark.parametrize("n,n_q", [(3, 2), (30, 4), (90, 8)])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_slots_past_the_table_are_reported(n, n_q, tree):
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
    for p0 in (cap - n + 1, cap, cap + 1, 2 ** 31 - 1):
        assert status(dict(base, ctx=[p0, 40])) == 1, p0
        none = dict(base, off=np.array([0, 0, 2], dtype=np.int32), ctx=[p0, 40], rows=[0, 2])
        assert status(none) == 0, p0                 # a request without rows sees nothing
    out, ws = _attend(dict(base, ctx=[-1, 40]))
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 1                   # there is no slot before the first


@pytest.mark.parametrize("n,n_q", [(10, 2), (30, 4), (90, 8)])
def test_attention_pages_that_no_row_sees_may_be_missing(n, n_q):
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


def test_attention_max_rows_is_only_a_hint():
    d = _build([40, 1, 7], [30, 200, 0], 8, 2, 128, 16, False)
    for hint in (0, 1, 2, 7, 40, 1000):
        out, _ = _attend(d, max_rows=hint)
        torch.cuda.synchronize()
        _check(d, out)


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


def test_pools_past_32_bit_offsets():
    """Pages whose codes lie beyond 2^32 (4.9 GB pools)."""
    rng = np.random.default_rng(31)
    n_pages, n_kv, page, hd, n_q = 300_000, 8, 16, 128, 32
    assert n_pages * n_kv * page * hd > 2 ** 32
    pools = [torch.empty(n_pages, n_kv, page, hd, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.empty(n_pages, n_kv, 1, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for rows, ctx in (([1, 2], [70, 31]), ([20], [60]), ([100], [40])):
        need = [-(-(n + c) // page) for n, c in zip(rows, ctx)]
        ids = rng.choice(np.arange(n_pages - 5000, n_pages), size=sum(need), replace=False)
        table, own = (np.full((len(rows), max(need)), -1, dtype=np.int32) for _ in range(2))
        at = 0
        for r, n in enumerate(need):
            table[r, :n], own[r, :n] = ids[at:at + n], np.arange(at, at + n)
            at += n
        small = [_pool(rng, sum(need), n_kv, page, hd) for _ in range(2)]
        for pool, scale, (c, s) in zip(pools, scales, small):
            pool[ids.tolist()], scale[ids.tolist()] = _u8(c), _u8(s)
        n = sum(rows)
        off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        k, v = (_t(rng.normal(size=(n, n_kv * hd))) for _ in range(2))
        pages = bd.PagesE4M3(*pools, *scales, _i(table))
        bd.paged_append_e4m3(pages, k, v, _i(off), _i(ctx))
        q, ws = _t(rng.normal(size=(n, n_q * hd))), _ws(n_q, n_kv, hd)
        out = torch.empty_like(q)
        bd.paged_attention_e4m3(pages, q, _i(off), _i(ctx), max(rows), out, ws)
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 0
        now = [t[ids.tolist()].cpu().numpy() for t in (*pools, *scales)]
        ref = oq.append(small[0][0], small[1][0], small[0][1], small[1][1], own, off, ctx,
                        *(_f64(t).reshape(n, n_kv, hd) for t in (k, v)), 0.0)
        for a, b in zip(now, ref):
            assert np.array_equal(a, b)
        _check(dict(ck=now[0], cv=now[1], sk=now[2], sv=now[3], table=own, off=off, ctx=ctx, q=q, mask=None, n_q=n_q,
                    hd=hd, n_kv=n_kv, rows=rows), out)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_in_a_graph_serves_growing_contexts():
    """Append and attention captured once: the contexts grow on the device."""
    rng = np.random.default_rng(8)
    rows, cap, n_q, n_kv, hd = [1, 2, 1], 300, 8, 2, 128
    _, _, table, _ = _paged(rng, [0, 0, 0], [cap, cap, cap], 1, 1, 32)
    held = [_u8(a) for a in (*_pool(rng, int(table.max()) + 1, n_kv, 32, hd), *_pool(rng, int(table.max()) + 1, n_kv, 32, hd))]
    ck, sk, cv, sv = held
    pages = bd.PagesE4M3(ck, cv, sk, sv, _i(table))
    off = np.array([0, 1, 3, 4])
    pos0, d_off = _i([17, 150, 0]), _i(off)
    q, k, v = (_t(rng.normal(size=(4, w * hd))) for w in (n_q, n_kv, n_kv))
    out, ws = torch.empty_like(q), _ws(n_q, n_kv, hd)
    grow = _i(rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        bd.paged_append_e4m3(pages, k, v, d_off, pos0, theta=THETA)
        bd.paged_attention_e4m3(pages, q, d_off, pos0, 2, out, ws)
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
        _check(dict(ck=_np(ck), cv=_np(cv), sk=_np(sk), sv=_np(sv), table=table, off=off, ctx=p0.tolist(), q=q,
                    mask=None, n_q=n_q, hd=hd, n_kv=n_kv, rows=rows), out)
    assert bd.read_status(ws) == 0


@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_verification_layer(kind):
    """norm_rope -> append -> attention of draft trees (or chains): close to the same pass
    over a cache of 16 bits.  Torch's 8-bit types are taken as they are."""
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
    fp8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    ck, cv = (torch.full(pk.shape, 127, dtype=torch.uint8, device=DEV).view(fp8) for _ in range(2))
    sk, sv = (torch.full((*pk.shape[:2], 1), 255, dtype=torch.uint8, device=DEV).view(e8) for _ in range(2))
    p8, p16 = bd.PagesE4M3(ck, cv, sk, sv, _i(table)), bd.Pages(pk, pv, _i(table))
    # the context
    first = _i(np.concatenate([[0], np.cumsum(ctx)]))
    k0, v0 = (_t(rng.normal(size=(sum(ctx), n_kv * hd))) for _ in range(2))
    bd.paged_append(p16, k0, v0, first, _i([0, 0]), theta=THETA)
    bd.paged_append_e4m3(p8, k0, v0, first, _i([0, 0]), theta=THETA)
    # the drafted rows
    qkv = _t(rng.normal(size=(n, (n_q + 2 * n_kv) * hd)))
    gq, gk = (_t(1 + 0.2 * rng.normal(size=hd)) for _ in range(2))
    d_off, d_ctx = _i(off), _i(ctx)
    pos = torch.where(depth >= 0, depth + d_ctx[:, None], -1).reshape(-1).contiguous()
    q = torch.zeros(n, n_q * hd, dtype=BF, device=DEV)
    k = torch.zeros(n, n_kv * hd, dtype=BF, device=DEV)
    v = qkv[:, (n_q + n_kv) * hd:].contiguous()
    bd.qk_norm_rope(qkv[:, :n_q * hd], qkv[:, n_q * hd:(n_q + n_kv) * hd], gq, gk, 1e-6, THETA, pos, hd, q, k)
    bd.paged_append(p16, k, v, d_off, d_ctx, pos=pos)
    bd.paged_append_e4m3(p8, k, v, d_off, d_ctx, pos=pos)
    a, b = torch.empty_like(q), torch.empty_like(q)
    ws = torch.zeros(bd.paged_attention_workspace_bytes(n_q, n_kv, hd), dtype=torch.uint8, device=DEV)
    bd.paged_attention(p16, q, d_off, d_ctx, B + 1, a, ws, mask=mask.view(n, -1))
    w8 = _ws(n_q, n_kv, hd)
    bd.paged_attention_e4m3(p8, q, d_off, d_ctx, B + 1, b, w8, mask=mask.view(n, -1))
    torch.cuda.synchronize()
    assert bd.read_status(w8) == 0
    nn = n_nodes.cpu().numpy()
    live = np.concatenate([np.arange(n).reshape(n_req, -1)[r, :nn[r] + 1] for r in range(n_req)])
    got = dict(ck=_np(ck), cv=_np(cv), sk=_np(sk), sv=_np(sv), table=table, off=off, ctx=ctx, q=q,
               mask=mask.view(n, -1).cpu().numpy().view(np.uint32), n_q=n_q, hd=hd, n_kv=n_kv, rows=[B + 1] * n_req)
    _check(got, b)
    # a code is off by 2^-4 at most, 2^-5.5 in the mean; keys' errors move a score by their
    # share of its spread (1 for N(0, 1)): a quarter of a row's norm bounds both amply
    x, y = _f64(a)[live], _f64(b)[live]
    assert np.all(np.linalg.norm(x - y, axis=1) <= 0.25 * np.linalg.norm(x, axis=1))


def test_captured_graphs_share_a_workspace():
    """Decoding, a chain and a tree captured apart with one workspace, replayed in turn: each
    call leaves the counters as it found them."""
    cases = [_build([1, 1], [4000, 77], 32, 8, 128, 16, False), _build([16], [900], 32, 8, 128, 32, False),
             _build([100], [2500], 32, 8, 128, 64, True), _build([5, 2], [600, 30], 8, 8, 128, 16, False)]
    want = [_attend(d)[0] for d in cases]
    ws = _ws(32, 8, 128)
    args = []
    for d in cases:
        mask = None if d["mask"] is None else torch.as_tensor(d["mask"].view(np.int32), device=DEV)
        pages = bd.PagesE4M3(*(_u8(d[x]) for x in ("ck", "cv", "sk", "sv")), _i(d["table"]))
        args.append((pages, d["q"], _i(d["off"]), _i(d["ctx"]), max(d["rows"]), torch.empty_like(d["q"]), ws, mask))
    torch.cuda.synchronize()
    graphs = []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bd.paged_attention_e4m3(*a)
        graphs.append(g)
    for _ in range(3):
        for a in args:
            a[5].fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[5], w) for a, w in zip(args, want))
    assert bd.read_status(ws) == 0


def test_trace_hook_sees_every_launch():
    d = _build([1, 2], [100, 40], 4, 2, 128, 16, False)
    few, many = _build([40], [100], 4, 2, 128, 16, False), _build([70] * 40, [5] * 40, 8, 2, 64, 16, False)
    seen = []
    bd.set_trace_hook(lambda kernel, phase, stream: seen.append((kernel, phase)))
    try:
        for x in (d, few, many):
            _attend(x)
        pages = bd.PagesE4M3(*(_u8(d[x]) for x in ("ck", "cv", "sk", "sv")), _i(d["table"]))
        k = _t(np.ones((3, 256)))
        bd.paged_append_e4m3(pages, k, k, _i(d["off"]), _i(d["ctx"]))
        x = torch.zeros(3, 100, device=DEV)
        bd.logits_adjust(x, x, _i([0, 3]))
        torch.cuda.synchronize()
    finally:
        bd.set_trace_hook(None)
    names = [n for n, phase in seen if phase == 0]
    assert names == ["paged_attn_small_e4m3", "paged_attn_tc_e4m3", "paged_join", "paged_attn_tc_e4m3",
                     "paged_append_e4m3", "logits_adjust"]
    assert [p for _, p in seen] == [0, 1] * len(names)


@pytest.mark.parametrize("rows,ctx,n_q,page", [
    ([64] * 20, 2000, 4, 64),        # 64-row tiles, joined by the last of their CTAs
    ([64] * 12, 8000, 4, 16),        # 64-row tiles, joined by a kernel
    ([1500], 2900, 16, 128),         # 256-row tiles, joined by the last of their CTAs
    ([64] * 8, 8000, 16, 64),        # 256-row tiles, joined by a kernel
])
def test_wait_runs_out_then_recovers(rows, ctx, n_q, page):
    """The waits between the tensor-core kernel's warps, made to run out by a limit of 1 us.
    The new tokens' values are NaN, which the softmax looks up for its rows one by one, while
    the CTA's other warps wait for it."""
    d = _build(rows, [ctx + 50 * i for i in range(len(rows))], n_q, 4, 128, page, False, seed=5)
    bad = d["cv"].copy()
    for r, (n, c) in enumerate(zip(rows, d["ctx"])):
        for t in range(c, c + n):
            bad[d["table"][r, t // page], :, t % page] = 127
    held = [_u8(d[x]) for x in ("ck", "cv", "sk", "sv")]
    table = _i(d["table"])
    finite, pages = bd.PagesE4M3(*held, table), bd.PagesE4M3(held[0], _u8(bad), *held[2:], table)
    off, pos0, ws = _i(d["off"]), _i(d["ctx"]), _ws(n_q, 4, 128)

    def run(pages):
        out = torch.full_like(d["q"], float("inf"))
        bd.paged_attention_e4m3(pages, d["q"], off, pos0, max(rows), out, ws)
        torch.cuda.synchronize()
        return out

    usual, want = run(finite), run(pages)
    assert bd.read_status(ws) == 0 and torch.isfinite(usual).all() and torch.isnan(want).all()   # (every row sees its own)
    bd.workspace_set_wait_limit(ws, 1000)
    run(pages)
    assert bd.read_status(ws) == 5
    # the context is intact, and after workspace_init the call is what it was
    assert float((torch.ones(8, device=DEV) * 2).sum()) == 16.0
    bd.workspace_init(ws)
    for _ in range(2):
        assert torch.equal(run(finite), usual) and torch.isnan(run(pages)).all()
        assert bd.read_status(ws) == 0
