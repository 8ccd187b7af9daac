"""GPU parity of the 8-bit paged cache at the ends of its ranges: requests so long that a
tile falls into a part for every CTA, values of the smallest scale, NaN whose weights
vanish, the largest scales, scores far past fp32's steps; and a workspace that calls of both
caches share.  Tolerances as in test_gpu_paged_e4m3.py."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding as bd
from oracle import quant as oq
from test_gpu_paged import BF, DEV, F32, _f64, _i, _t
from test_gpu_paged_e4m3 import _attend, _build, _check, _pool, _u8

pytestmark = pytest.mark.gpu


def _parts(slots, tiles, sms):
    """The most CTAs that a tile of few rows is shared out to: every tile is 4 units and a
    unit for each 64 slots, shares are equal and weigh 2 at least, three CTAs to an SM."""
    length = 4 + -(-slots // 64)
    ctas = min(3 * sms, length * tiles // 2)
    q, m = divmod(length * tiles, ctas)

    def owner(s):
        return s // (q + 1) if s < m * (q + 1) else m + (s - m * (q + 1)) // q
    return max(owner((t + 1) * length - 1) - owner(t * length + 4) + 1 for t in range(tiles))


@pytest.mark.parametrize("rows,ctx,n_q,n_kv,hd,page,tree,wide", [
    ([1], [60000], 4, 1, 64, 64, False, False),
    ([2], [59000], 4, 1, 64, 16, True, False),
    ([8], [70001], 1, 1, 64, 1024, False, False),
    ([16], [30000], 2, 2, 64, 16, False, True),
    ([3], [60000], 4, 1, 128, 32, False, True),
    ([16], [60000], 1, 1, 128, 64, True, True),
    ([16], [100000], 1, 1, 64, 256, False, True),
])
def test_attention_of_long_requests(rows, ctx, n_q, n_kv, hd, page, tree, wide):
    """More parts to a tile than the loading ring of the CTA that joins them has room for
    (max, sum) pairs of: 24 KB with heads of 64, 48 KB with 128."""
    tile = 16 if wide else 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert _parts(sum(rows) + ctx[0], n_kv, sms) * tile * 8 > 384 * hd
    d = dict(_build(rows, ctx, n_q, n_kv, hd, page, tree), wide=wide)
    out, ws = _attend(d)
    again, _ = _attend(d, ws)
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 0
    _check(d, out)
    assert torch.equal(out, again)


KERNELS = [([1], False, False), ([3, 1], False, True), ([16], False, True), ([20], True, False), ([64, 3], False, False),
           ([100], True, False), ([128], False, False), ([300, 40], False, False)]


@pytest.mark.parametrize("rows,tree,wide", KERNELS)
@pytest.mark.parametrize("ctx", [70, 3000])
def test_attention_where_every_value_is_nan(rows, tree, wide, ctx):
    """As an append leaves values that are NaN or infinite throughout: their blocks have the
    smallest scale.  Another KV head's outputs keep their bits."""
    for hd in (64, 128):
        d = dict(_build(rows, [ctx, 9][:len(rows)], 2, 2, hd, 16, tree), wide=wide)
        clean, _ = _attend(d)
        cv, sv = d["cv"].copy(), d["sv"].copy()
        cv[:, 0], sv[:, 0] = 127, 0
        got, ws = _attend(dict(d, cv=cv, sv=sv))
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 0
        assert torch.isnan(got[:, :hd]).all() and torch.equal(got[:, hd:], clean[:, hd:])


@pytest.mark.parametrize("rows,tree,wide", KERNELS)
@pytest.mark.parametrize("ctx", [300, 3000])
def test_attention_nan_under_the_smallest_weight(rows, tree, wide, ctx):
    """A NaN value whose weight vanishes beside another key's (2^-456 of it) reaches the rows
    that see it, whichever part of the work it falls into."""
    hd = 128
    d = dict(_build(rows, [ctx] * len(rows), 2, 1, hd, 16, tree, spread=0.0), wide=wide)
    d["ck"] = np.zeros_like(d["ck"])
    d["sk"] = np.full_like(d["sk"], 127)
    q = torch.zeros_like(d["q"])
    q.view(-1, 2, hd)[:, :, 0] = 8.0
    for top in (ctx - 1, ctx - 130, 3):
        e = dict(d, q=q, ck=d["ck"].copy(), cv=d["cv"].copy())
        at = [(r, e["table"][r, top // 16], top % 16) for r in range(len(rows))]
        for r, pg, slot in at:
            e["ck"][pg, 0, slot, 0] = 126                    # 448
        for col, t in ((7, 5), (40, ctx - 140), (99, ctx - 20)):
            for r in range(len(rows)):
                e["cv"][e["table"][r, t // 16], 0, t % 16, col] = 127
        out, ws = _attend(e)
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 0
        o = out.view(-1, 2, hd).double().cpu().numpy()
        bad = np.zeros(hd, dtype=bool)
        bad[[7, 40, 99]] = True
        assert np.isnan(o[:, :, bad]).all()
        for r, pg, slot in at:                               # elsewhere that key's value, exact in bf16
            want = oq.held(e["cv"], e["sv"])[pg, 0, slot][~bad]
            assert (o[e["off"][r]:e["off"][r + 1]][:, :, ~bad] == want).all()


@pytest.mark.parametrize("rows,tree,wide", KERNELS)
@pytest.mark.parametrize("ctx", [70, 3000])
def test_attention_of_the_smallest_values(rows, tree, wide, ctx):
    """All blocks at the smallest scale, 2^-127: outputs are normal numbers of bf16."""
    for hd in (64, 128):
        d = dict(_build(rows, [ctx, 9][:len(rows)], 4, 2, hd, 16, tree), wide=wide)
        d["cv"] = np.maximum(d["cv"] & 127, 64)              # 2 .. 448: no sum below 2 (2^-126)
        d["sv"] = np.zeros_like(d["sv"])
        out, ws = _attend(d)
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 0
        _check(dict(d, sv=np.full_like(d["sv"], 127)), out.double() * 2.0 ** 127)


def test_one_workspace_serves_both_caches():
    """Calls over the 16-bit and the 8-bit cache, of every kernel, in turn on one workspace:
    each leaves it as the others need it."""
    n_q, n_kv, hd, page = 8, 2, 128, 16
    shapes = [([100], [2500], True), ([1] * 40, [4000 + 61 * i for i in range(40)], False), ([16], [6000], False),
              ([3], [20000], False), ([300, 40], [900, 5000], False), ([8, 4], [9000, 30], False)]
    eight = [_build(rows, ctx, n_q, n_kv, hd, page, tree) for rows, ctx, tree in shapes]
    size = max(bd.paged_attention_workspace_bytes(n_q, n_kv, hd), bd.paged_attention_e4m3_workspace_bytes(n_q, n_kv, hd))
    assert size > 0

    def sixteen(d, ws):
        n_pages = d["ck"].shape[0]
        gen = torch.Generator(device=DEV).manual_seed(n_pages)
        k, v = (torch.randn(n_pages, n_kv, page, hd, generator=gen, device=DEV).to(BF) for _ in range(2))
        mask = None if d["mask"] is None else torch.as_tensor(d["mask"].view(np.int32), device=DEV)
        out = torch.full_like(d["q"], 7.0)
        bd.paged_attention(bd.Pages(k, v, _i(d["table"])), d["q"], _i(d["off"]), _i(d["ctx"]), max(d["rows"]), out, ws,
                           mask=mask)
        return out

    def fresh():
        return torch.zeros(size, dtype=torch.uint8, device=DEV)

    want = [(sixteen(d, fresh()), _attend(d, fresh())[0]) for d in eight]
    ws = fresh()
    for i, a in enumerate(eight):
        for j, b in enumerate(eight):
            x, y = sixteen(a, ws), _attend(b, ws)[0]
            torch.cuda.synchronize()
            assert torch.equal(x, want[i][0]) and torch.equal(y, want[j][1]), (i, j)
    assert bd.read_status(ws) == 0


@pytest.mark.parametrize("byte", [253, 254, 255])
def test_append_beside_the_largest_scales(byte):
    """Earlier tokens at the largest scales keep their codes and their scale; 255 is read as
    254."""
    rng = np.random.default_rng(6)
    n_kv, hd = 2, 64
    table = np.array([[1, 0]], dtype=np.int32)
    x = _t(rng.normal(size=(20, n_kv * hd)) * 5e37, F32)
    for rows, p0 in ((2, 5), (20, 3), (1, 15)):
        ck, _ = _pool(rng, 2, n_kv, 16, hd)
        sk = np.full((2, n_kv, 1), byte, dtype=np.uint8)
        got = [_u8(a) for a in (ck, ck, sk, sk)]
        bd.paged_append_e4m3(bd.PagesE4M3(*got, _i(table)), x[:rows], x[:rows], _i([0, rows]), _i([p0]))
        torch.cuda.synchronize()
        x64 = _f64(x[:rows]).reshape(rows, n_kv, hd)
        ref = oq.append(ck, ck, np.minimum(sk, 254), np.minimum(sk, 254), table, [0, rows], [p0], x64, x64, 0.0)
        for g, r in zip(got, ref):
            g = g.cpu().numpy()
            assert np.array_equal(g if g.ndim == 4 else np.minimum(g, 254), r)


@pytest.mark.parametrize("rows,tree,wide", KERNELS)
def test_attention_reads_scale_255_as_254(rows, tree, wide):
    for hd in (64, 128):
        d = dict(_build(rows, [300, 9][:len(rows)], 4, 2, hd, 16, tree), wide=wide)
        d["cv"] = d["cv"] & 129                              # 2^-9 at most: values of 2^118
        for x in ("sv", "sk"):
            out = []
            for byte in (254, 255):
                o, ws = _attend(dict(d, **{x: np.full_like(d[x], byte)}))
                torch.cuda.synchronize()
                assert bd.read_status(ws) == 0
                out.append(o)
            # sums of weights up to 2^14 times 309 such values may pass 2^128, in both alike
            assert torch.isfinite(out[0]).any() and torch.equal(*(o.nan_to_num(0.0) for o in out))
            assert torch.equal(*(torch.isnan(o) for o in out))


@pytest.mark.parametrize("rows,tree,wide", KERNELS)
@pytest.mark.parametrize("ctx", [300, 3000])
@pytest.mark.parametrize("size", [4.0, 2.0 ** 10, 2.0 ** 30])
def test_attention_of_scores_far_past_fp32_steps(rows, tree, wide, ctx, size):
    """Scores of 2^17 to 2^46, the best key ahead of every other by a seventh: its value alone
    comes out, exact in bf16.  Two that are equal: the mean of their values, whose blocks'
    scales differ."""
    hd = 128
    d = dict(_build(rows, [ctx] * len(rows), 2, 1, hd, 16, tree, spread=0.0), wide=wide)
    rng = np.random.default_rng(len(rows) + ctx)
    keys = np.minimum(d["ck"] & 127, 124)                    # 384 at most
    keys[..., 1:] = 0
    d["ck"], d["sk"] = keys, np.full_like(d["sk"], 137)      # 2^10
    d["sv"] = rng.integers(117, 123, size=d["sv"].shape).astype(np.uint8)
    d["q"] = torch.zeros_like(d["q"])
    d["q"].view(-1, 2, hd)[:, :, 0] = size
    held = oq.held(d["cv"], d["sv"])
    for tops in ((ctx - 1,), (2,), (ctx - 150,), (1, ctx - 3), (ctx - 40, ctx - 160), (7, 40)):
        e = dict(d, ck=d["ck"].copy())
        for r in range(len(rows)):
            for t in tops:
                e["ck"][e["table"][r, t // 16], 0, t % 16, 0] = 126     # 448
        out, ws = _attend(e)
        torch.cuda.synchronize()
        assert bd.read_status(ws) == 0
        o = _f64(out).reshape(-1, 2, hd)
        for r in range(len(rows)):
            v = np.stack([held[e["table"][r, t // 16], 0, t % 16] for t in tops])
            want = v.mean(0)
            # equal scores have equal weights, powers of two: bf16 rounds the mean
            tol = 0.0 if len(tops) == 1 else 2.0 ** -8 * np.abs(want)
            assert (np.abs(o[e["off"][r]:e["off"][r + 1]] - want) <= tol).all(), (r, tops)
