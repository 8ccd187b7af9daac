"""Pins of the paged oracle: pages against a contiguous cache, the rotation
against complex numbers, causal and tree visibility against one another, and
the filtered sampler against distributions computed by hand."""
import math

import numpy as np
import pytest

from oracle import paged as op
from oracle import verify as ov


def _pool(rng, ctx, n_kv, hd, page, spare=2):
    n = -(-ctx // page)
    table = rng.permutation(n + spare)[:n][None].astype(np.int32)
    return rng.normal(size=(n + spare, n_kv, page, hd)), rng.normal(size=(n + spare, n_kv, page, hd)), table


def test_rotation_is_a_complex_turn():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 8))
    pos = np.array([0, 5, 1000])
    z = (x[..., :4] + 1j * x[..., 4:]) * np.exp(1j * op.angles(pos, 8, 1e4))[:, None]
    got = op.rotate(x, pos, 1e4)
    assert np.allclose(got, np.concatenate([z.real, z.imag], -1), atol=1e-12)
    assert np.array_equal(op.rotate(x, pos, 0.0), x)


def test_norm_has_unit_rms_and_gain():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 3, 16)) * 7
    y = op.norm_rope(x, np.ones(16), 0.0, 1e4, np.arange(4))
    assert np.allclose((y * y).mean(-1), 1.0)
    g = rng.normal(size=16)
    assert np.allclose(op.norm_rope(x, g, 0.0, 0.0, None), op.norm_rope(x, np.ones(16), 0.0, 0.0, None) * g)


def test_append_then_slots_returns_the_rows():
    rng = np.random.default_rng(2)
    pk, pv, table = _pool(rng, 50, 2, 8, 16)
    k, v = rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    pos = np.arange(9) + 100
    pos[4] = -1
    nk, nv = op.append(pk, pv, table, [0, 9], [13], k, v, 1e4, pos)
    got = op.slots(nv, table[0], 50)
    was = op.slots(pv, table[0], 50)
    for i in range(9):
        assert np.array_equal(got[:, 13 + i], was[:, 17] if i == 4 else v[i])
    assert np.array_equal(got[:, :13], was[:, :13]) and np.array_equal(got[:, 22:], was[:, 22:])
    assert np.allclose(op.slots(nk, table[0], 50)[:, 14], op.rotate(k[1:2], [101], 1e4)[0])
    # a slot past the table or without a page is stored nowhere
    gone = table.copy()
    gone[0, 1] = -1
    n2, _ = op.append(pk, pv, gone, [0, 9], [13], k, v, 0.0)
    assert np.array_equal(op.slots(n2, gone[0], 16)[:, 13:], k[:3].transpose(1, 0, 2))
    assert np.array_equal(n2[table[0, 1]], pk[table[0, 1]])


def test_attention_over_pages_is_the_tree_attention_over_a_cache():
    rng = np.random.default_rng(3)
    n, ctx, n_q, n_kv, hd = 7, 37, 4, 2, 8
    pk, pv, table = _pool(rng, ctx + n, n_kv, hd, 16)
    q = rng.normal(size=(n, n_q, hd))
    parents = [-1, 0, 0, 1, 1, 2, 5]
    mask = np.zeros((n, 1), dtype=np.uint32)
    for i, p in enumerate(parents):
        mask[i, 0] = (mask[p, 0] if p >= 0 else 0) | np.uint32(1 << i)
    out, _ = op.attention(q, pk, pv, table, [0, n], [ctx], n_q, mask)
    ks, vs = op.slots(pk, table[0], ctx + n), op.slots(pv, table[0], ctx + n)
    ref = ov.tree_attention(q, ks[:, ctx:].transpose(1, 0, 2), vs[:, ctx:].transpose(1, 0, 2),
                            ks[:, :ctx], vs[:, :ctx], ctx, mask, n - 1, n_q, n_kv)
    assert np.allclose(out, ref, atol=1e-12)


def test_causal_is_the_mask_of_a_chain():
    rng = np.random.default_rng(4)
    n, ctx = 40, 5
    chain = np.array([[(1 << min(i + 1, 32)) - 1, (1 << max(i + 1 - 32, 0)) - 1] for i in range(n)],
                     dtype=np.uint32)
    assert np.array_equal(op.visible(n, ctx, n + ctx), op.visible(n, ctx, n + ctx, chain))


def test_a_row_that_sees_nothing_is_zero():
    rng = np.random.default_rng(5)
    pk, pv, table = _pool(rng, 3, 1, 8, 16)
    out, _ = op.attention(rng.normal(size=(3, 1, 8)), pk, pv, table, [0, 3], [0], 1,
                          np.array([[0], [3], [4]], dtype=np.uint32))
    assert not out[0].any() and out[1].any() and np.allclose(out[2, 0], pv[table[0, 0], 0, 2])


LOGITS = np.log(np.array([0.1, 0.4, 0.1, 0.25, 0.15]))


@pytest.mark.parametrize("how, ids", [
    (dict(), [0, 1, 2, 3, 4]),
    (dict(top_k=2), [1, 3]),
    (dict(top_k=4), [0, 1, 3, 4]),                  # the tie at 0.1: the lower id
    (dict(top_p=0.0), [1]),
    (dict(top_p=0.39), [1]),
    (dict(top_p=0.41), [1, 3]),
    (dict(top_p=0.85), [0, 1, 3, 4]),
    (dict(min_p=0.3), [1, 3, 4]),
    (dict(min_p=2.0), [1]),
    (dict(top_k=3, top_p=0.5), [1]),                # half of 0.8 is what the best holds
    (dict(temperature=0.0), [1]),
])
def test_kept_sets_by_hand(how, ids):
    got, w = op.kept(LOGITS, **how)
    assert got.tolist() == ids
    if not how:
        assert np.allclose(w / w.sum(), np.exp(LOGITS))


def test_sample_walks_the_cumulated_masses():
    for u, tok in [(0.0, 0), (0.0999, 0), (0.1001, 1), (0.4999, 1), (0.5001, 2), (0.6001, 3), (0.9999, 4),
                   (1.0, 4)]:
        assert op.sample(LOGITS, u)[0] == tok, u
    tok, lp = op.sample(LOGITS, 0.99, top_k=2)
    assert tok == 3 and math.isclose(lp, math.log(0.25 / 0.65))
    # temperature: the masses are powers
    w = np.exp(LOGITS) ** 2
    got = np.bincount([op.sample(LOGITS, (i + 0.5) / 4000, temperature=0.5)[0] for i in range(4000)])
    assert np.allclose(got / 4000, w / w.sum(), atol=1e-3)


def test_sample_of_masked_rows():
    assert op.sample(np.full(5, -np.inf), 0.5) == (-1, -np.inf)
    x = np.array([-np.inf, 1.0, np.nan, 1.0])
    assert op.sample(x, 0.0)[0] == 1 and op.sample(x, 0.9)[0] == 3
    x = np.array([0.0, np.inf, 1.0, np.inf])
    assert op.sample(x, 0.6) == (3, math.log(0.5))
