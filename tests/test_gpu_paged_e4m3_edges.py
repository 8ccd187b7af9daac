"""GPU parity of the 8-bit paged cache at the ends of its ranges: requests so long that a
tile falls into a part for every CTA, and values of the smallest scale.  Tolerances as in
test_gpu_paged_e4m3.py."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding as bd
from test_gpu_paged_e4m3 import _attend, _build, _check

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
    """More parts to a tile than the shared memory of the CTA that joins them holds
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
