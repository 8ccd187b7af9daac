"""GPU parity of the filtered sampler against the 64-bit oracle, through the C
ABI.  A draw is decided where the cumulated mass passes u times the kept mass.
The library's masses are 40-bit sums of fp32 exponentials: a token at distance
d = (max - l) / T carries a relative error of 2^-22 (the exponential) plus
2^-23 d (the argument), sums of eight add 8 * 2^-24, and tokens beyond d = 24
weigh less than 2^-34 of the best.  So a mass is off by less than eps = 2^-17
of the whole, and a token is right if u lies within 2 eps of its share's
interval.  The same holds for top-p's border: there the kept set may gain or
lose tokens whose cumulated mass lies within eps of it."""
import math

import numpy as np
import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding as bd
from oracle import ddtree as odt
from oracle import paged as op

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -17


def _run(x, u, how, vocab=None):
    n = x.shape[0]
    tok = torch.full((n,), -7, dtype=torch.int32, device=DEV)
    lp = torch.full((n,), 7.0, device=DEV)
    dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else F32, device=DEV) for k, v in how.items()}
    bd.logits_sample_filtered(x, torch.tensor(u, dtype=F32, device=DEV), tok, lp, vocab=vocab, **dev)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy().astype(np.float64)


def _check(x, u, how, vocab=None):
    tok, lp = _run(x, u, how, vocab)
    rows = x.float().cpu().numpy().astype(np.float64)[:, :vocab]
    u32 = np.asarray(u, dtype=np.float32).astype(np.float64)
    for i in range(len(rows)):
        h = {k: (int(v[i]) if k == "top_k" else float(np.float32(v[i]))) for k, v in how.items()}
        want, wlp = op.sample(rows[i], u32[i], **h)
        if want < 0:
            assert tok[i] == -1 and lp[i] == -np.inf
            continue
        # the kept sets on either side of top-p's border
        fits = False
        for p in ({h["top_p"] * (1 - EPS), h["top_p"], h["top_p"] * (1 + EPS)} if h.get("top_p", 1) < 1 else {1.0}):
            ids, w = op.kept(rows[i], **dict(h, top_p=p))
            j = np.searchsorted(ids, tok[i])
            if j == len(ids) or ids[j] != tok[i]:
                continue
            cum, uu = np.cumsum(w) / w.sum(), min(max(u32[i], 0.0), 1.0)
            lo = cum[j - 1] if j else 0.0
            if lo - 2 * EPS <= uu <= cum[j] + 2 * EPS:
                ref = math.log(w[j] / w.sum())
                # the mass's error, the log's, and the fp32 result's half step
                if abs(lp[i] - ref) <= 2 * EPS + 2.0 ** -23 * abs(ref):
                    fits = True
        assert fits, (i, tok[i], want, lp[i], wlp, h, u32[i])


def _logits(rng, n, vocab, dtype, scale=1.5, fav=8.0):
    x = rng.normal(size=(n, vocab)) * scale
    if fav:
        x[np.arange(n), rng.integers(0, vocab, size=n)] += fav
    return torch.as_tensor(x.astype(np.float32)).to(dtype).to(DEV)


GRID = [dict(), dict(temperature=0.7), dict(top_k=20), dict(top_p=0.9), dict(min_p=0.05),
        dict(temperature=1.7, top_k=300, top_p=0.8), dict(temperature=0.9, top_p=0.95, min_p=0.02),
        dict(temperature=2.5, top_k=50, top_p=0.5, min_p=0.3), dict(top_p=0.999), dict(temperature=8.0, top_p=0.6)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 1000, 4099, 40000])
def test_sample(vocab, dtype):
    rng = np.random.default_rng(vocab)
    for g, how in enumerate(GRID):
        n = 4
        x = _logits(rng, n, vocab, dtype, fav=8.0 if g % 2 else 0.0)
        _check(x, rng.random(n), {k: [v] * n for k, v in how.items()})


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sample_full_vocabulary_rows_of_their_own(dtype):
    rng = np.random.default_rng(3)
    n, vocab = 24, 151936
    x = _logits(rng, n, vocab, dtype, scale=math.sqrt(2.0))
    how = dict(temperature=rng.choice([0.0, 0.6, 0.8, 1.0, 1.3, 2.0], size=n),
               top_k=rng.choice([0, 0, 1, 20, 50, 1000, 200000], size=n),
               top_p=rng.choice([1.0, 0.3, 0.8, 0.95], size=n), min_p=rng.choice([0.0, 0.05, 0.2], size=n))
    _check(x, rng.random(n), how)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sample_longer_than_shared_memory(dtype):
    rng = np.random.default_rng(4)
    vocab = 900001                                    # also rows off 16-byte boundaries
    x = _logits(rng, 3, vocab, dtype)
    _check(x, rng.random(3), dict(temperature=[1.0, 0.8, 1.5], top_k=[0, 40, 100000], top_p=[0.9, 1.0, 0.7]))


def test_sample_strided_rows_and_shorter_vocabulary():
    rng = np.random.default_rng(5)
    x = _logits(rng, 6, 1007, BF)
    wide = torch.full((6, 1300), 50.0, dtype=BF, device=DEV)      # what lies past a row would win
    wide[:, 3:1010] = x
    u = rng.random(6)
    how = dict(top_p=[0.9] * 6)
    a, la = _run(x, u, how)
    b, lb = _run(wide[:, 3:1010], u, how)
    c, lc = _run(wide[:, 3:], u, how, vocab=1007)
    assert np.array_equal(a, b) and np.array_equal(a, c) and np.array_equal(la, lb) and np.array_equal(la, lc)
    _check(x, u, how)


def test_sample_ties_go_to_the_lowest_ids():
    """Whole rows of equal logits: the k lowest ids share the mass equally."""
    n, vocab = 8, 5000
    x = torch.zeros(n, vocab, dtype=BF, device=DEV)
    u = [(i + 0.5) / n for i in range(n)]
    tok, lp = _run(x, u, dict(top_k=[8] * n))
    assert tok.tolist() == list(range(n)) and np.allclose(lp, -math.log(8), atol=1e-6)
    # half of the mass: the lower half of the ids
    tok, lp = _run(x, [0.99999] * n, dict(top_p=[0.5] * n))
    assert (tok == 2499).all() and np.allclose(lp, -math.log(2500), atol=1e-6)
    # ties on both sides of a part's end, and a better token among them
    y = x.clone()
    y[:, 4000] = 1.0
    _check(y, u, dict(top_k=[3000] * n, top_p=[0.7] * n))
    tok, _ = _run(y, [0.999999] * n, dict(top_k=[2] * n))
    assert (tok == 4000).all()
    tok, _ = _run(y, [0.0] * n, dict(top_k=[2] * n))
    assert (tok == 0).all()


def test_sample_masked_infinite_and_nan_logits():
    inf, nan = float("inf"), float("nan")
    x = torch.full((9, 300), -inf, device=DEV)
    x[1, 200] = 0.5                                    # one token left
    x[2, 5], x[2, 6], x[2, 7] = 1.0, nan, 1.0          # NaN counts as -inf
    x[3] = nan
    x[4] = 0.0
    x[4, 100], x[4, 250] = inf, inf                    # +inf takes everything
    x[5] = torch.finfo(F32).min                        # the type's lowest value everywhere
    x[6] = torch.finfo(F32).min
    x[6, 9] = 3.0
    x[7, :10] = -1e30
    x[8, 299] = torch.finfo(F32).max
    u = [0.5, 0.9, 0.9, 0.5, 0.75, 0.5, 0.999, 0.55, 0.1]
    for how in (dict(), dict(top_k=[5] * 9), dict(top_p=[0.9] * 9), dict(min_p=[0.1] * 9),
                dict(top_k=[250] * 9, top_p=[0.999] * 9, min_p=[0.01] * 9, temperature=[0.5] * 9)):
        for dtype in (F32, BF):
            tok, lp = _run(x.to(dtype), u, how)
            assert tok[0] == -1 and tok[3] == -1 and lp[0] == -inf
            assert tok[1] == 200 and lp[1] == 0 and tok[2] in (5, 7) and tok[6] == 9 and tok[8] == 299
            assert tok[4] in (100, 250)
            xx = x.to(dtype)
            _check(xx, u, how)


def test_sample_parameters_at_the_edges():
    rng = np.random.default_rng(6)
    x = _logits(rng, 1, 3000, F32).repeat(14, 1)
    best = int(x[0].argmax())
    inf, nan = float("inf"), float("nan")
    u = [0.3, 0.0, 1.0, -1.0, nan, 0.9, 0.9, 0.9, 0.9, 0.9, 0.9, 0.9, 0.9, 0.9]
    t = [1.0] * 5 + [0.0, -3.0, nan, 1e-30, inf, 1.0, 1.0, 1.0, 1.0]
    k = [0] * 10 + [1, -4, 5000, 3000]
    tok, lp = _run(x, u, dict(temperature=t, top_k=k))
    assert (tok[[5, 6, 7, 8, 10]] == best).all() and (lp[[5, 6, 7, 8, 10]] == 0).all()
    assert tok[1] == tok[3] == tok[4] == 0             # u clamped to 0: the first token
    assert tok[2] == 2999                              # u clamped below 1: the last one
    # infinite T: uniform; 0.9 in fp32 is 0.89999998, and 3000 times that is 2699.9999
    assert tok[9] == math.floor(3000 * float(np.float32(0.9))) == 2699
    assert abs(lp[9] + math.log(3000)) < 1e-5
    assert tok[11] == tok[12] == tok[13]               # no top-k
    tok, lp = _run(x[:4], [0.9] * 4, dict(top_p=[0.0, -1.0, 1.0, nan]))
    assert tok[0] == tok[1] == best and tok[2] == tok[3] != best
    tok, _ = _run(x[:3], [0.9] * 3, dict(min_p=[1.0, 7.0, nan]))
    assert tok[0] == tok[1] == best and tok[2] != best


def test_sample_frequencies():
    """Over an even grid of u the tokens come out in proportion to the kept mass."""
    rng = np.random.default_rng(7)
    n = 4096
    row = _logits(rng, 1, 200, F32, fav=0.0)
    tok, _ = _run(row.repeat(n, 1), [(i + 0.5) / n for i in range(n)],
                  dict(temperature=[0.8] * n, top_k=[30] * n, top_p=[0.9] * n))
    ids, w = op.kept(row[0].cpu().numpy(), temperature=float(np.float32(0.8)), top_k=30, top_p=float(np.float32(0.9)))
    got = np.bincount(tok, minlength=200)
    assert set(np.flatnonzero(got)) <= set(ids)
    assert np.all(np.abs(got[ids] / n - w / w.sum()) <= 1.0 / n + EPS)   # a grid of n points


def test_sampled_targets_walk_the_tree():
    """The LM head's logits, a draw at every node, and the verifier walk."""
    rng = np.random.default_rng(9)
    n_req, B, D, K, vocab, d = 2, 16, 4, 3, 1024, 128
    lp = -np.sort(rng.random((n_req, D, K)).astype(np.float32), axis=2)
    ids = np.stack([[rng.choice(vocab, K, replace=False) for _ in range(D)] for _ in range(n_req)]).astype(np.int32)
    bufs = bd.tree_buffers(n_req, B)
    bd.ddtree_build(torch.as_tensor(lp, device=DEV), torch.as_tensor(ids, device=DEV),
                    torch.tensor([1, 2], dtype=torch.int32, device=DEV), B, *bufs)
    n_nodes, tok, parent, depth, rank, mask = bufs
    M = n_req * (B + 1)
    X = torch.as_tensor(rng.normal(size=(M, d)).astype(np.float32)).to(BF).to(DEV)
    W = torch.as_tensor(rng.normal(size=(vocab, d)).astype(np.float32) * 0.2).to(BF).to(DEV)
    Y = torch.empty(M, vocab, device=DEV)
    ws = torch.zeros(bd.linear_workspace_bytes(M, vocab, d), dtype=torch.uint8, device=DEV)
    bd.linear_bf16(X, W, Y, ws)
    # at some nodes the target all but agrees with a child
    t, p = tok.cpu().numpy(), parent.cpu().numpy()
    for r in range(n_req):
        for c in range(1, B + 1, 2):
            Y[r * (B + 1) + p[r, c], t[r, c]] += 40.0
    u = rng.random(M)
    how = dict(temperature=[0.8] * M, top_k=[50] * M, top_p=[0.9] * M)
    _check(Y, u, how)
    picked, _ = _run(Y, u, how)
    target = torch.tensor(picked.reshape(n_req, B + 1), dtype=torch.int32, device=DEV)
    al, bonus = (torch.empty(n_req, dtype=torch.int32, device=DEV) for _ in range(2))
    acc = torch.empty(n_req, D, dtype=torch.int32, device=DEV)
    bd.ddtree_accept(D, B, n_nodes, tok, parent, target, al, acc, bonus)
    torch.cuda.synchronize()
    for r in range(n_req):
        a, nodes, bon = odt.accept_walk(t[r], p[r], int(n_nodes[r]), picked.reshape(n_req, B + 1)[r], D)
        assert int(al[r]) == a and int(bonus[r]) == bon and np.array_equal(acc[r].cpu().numpy(), nodes)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab", [(200, 1), (150, 3), (160, 33), (90, 1000), (45, 4099), (80, 24000), (40, 45001), (42, 100001)])
def test_sample_many_rows(n, vocab, dtype):
    """Rows enough that two or four CTAs share one, every row with its own filters; the
    last in fp32 long enough to be read again instead of kept."""
    rng = np.random.default_rng(n)
    x = _logits(rng, n, vocab, dtype, scale=math.sqrt(2.0))
    how = dict(temperature=rng.choice([0.0, 0.6, 1.0, 2.0], size=n), top_k=rng.choice([0, 0, 0, 1, 30, 300, 700], size=n),
               top_p=rng.choice([1.0, 0.3, 0.8, 0.95], size=n), min_p=rng.choice([0.0, 0.0, 0.05], size=n))
    _check(x, rng.random(n), how)


@pytest.mark.parametrize("n", [6, 60])
@pytest.mark.parametrize("steps", [1, 4, 64])
def test_sample_logits_of_few_values(steps, n):
    """Many tokens at each value (`steps` to a unit): more of them lie near a border
    than are kept aside there, and the bins' middles misjudge their weights."""
    rng = np.random.default_rng(steps)
    vocab = 20011
    x = torch.as_tensor((np.round(rng.normal(size=(n, vocab)) * steps) / steps).astype(np.float32)).to(DEV)
    for how in (dict(top_p=0.9), dict(temperature=0.5, top_p=0.6), dict(top_k=5000, top_p=0.7), dict(temperature=3.0, top_p=0.3)):
        _check(x, rng.random(n), {k: [v] * n for k, v in how.items()})


@pytest.mark.parametrize("far", [3.0, 12.0, 40.0])
def test_sample_mass_in_few_tokens(far):
    """A handful of tokens holds the mass that top-p asks for, the rest lies far below."""
    rng = np.random.default_rng(9)
    n, vocab = 8, 30000
    for dtype in (BF, F32):
        x = _logits(rng, n, vocab, dtype, scale=0.5, fav=0.0)
        for j in range(5):
            x[torch.arange(n), torch.as_tensor(rng.integers(0, vocab, size=n))] = far + 0.25 * j
        for p in (0.2, 0.5, 0.9, 0.999):
            _check(x, rng.random(n), dict(top_p=[p] * n))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sample_border_just_below_zero(dtype):
    """Borders among the smallest negative numbers, next to logits of both zeros: the
    codes of a search's bracket skip -0, which no token has.  The best token's value
    moves, so that brackets end at every place."""
    n = 192
    vocab = 3000
    x = torch.zeros(n, vocab, device=DEV)
    x[:, ::3] = -0.0
    x[:, 600:] = -1e-39                                # (subnormal in both types)
    x[:, 2000:] = -3.0
    x[:, 7] = torch.arange(n, device=DEV) / 16 + 4
    x = x.to(dtype)
    u = (np.arange(n) + 0.5) / n
    for how in (dict(top_k=1000), dict(top_k=600), dict(top_k=601), dict(top_p=0.6), dict(top_p=0.6, top_k=1500),
                dict(temperature=0.01, top_k=900, top_p=0.999)):
        _check(x, u, {k: [v] * n for k, v in how.items()})
    # the first 1000 ids, of 600 tokens at 0 or above and ties below them
    tok, lp = _run(x, [1.0] * n, dict(top_k=[1000] * n, temperature=[1e30] * n))
    assert (tok == 999).all() and np.allclose(lp, -math.log(1000), atol=1e-6)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top_k", [0, 50, 300, 1000])
def test_sample_infinite_temperature_with_min_p(top_k, dtype):
    """At T = inf all tokens weigh the same; a min-p of 1 or more still leaves the best
    alone, a smaller one everything.  (inf * ln 1 has no value of its own.)"""
    rng = np.random.default_rng(top_k)
    x = _logits(rng, 1, 3000, dtype).repeat(6, 1)
    p = [0.5, 1.0, 7.0] * 2
    how = dict(temperature=[float("inf")] * 6, min_p=p, top_k=[top_k] * 6)
    _check(x, [0.7] * 6, how)
    tok, lp = _run(x, [0.7] * 6, how)
    best = int(x[0].argmax())
    for i in (1, 2, 4, 5):
        assert tok[i] == best and lp[i] == 0
    assert abs(lp[0] + math.log(top_k or 3000)) < 1e-5
    # with top-p between them
    _check(x, [0.3] * 6, dict(how, top_p=[0.4] * 6))


def test_sample_small_masses_next_to_large_ones():
    """A token keeps its own mass whatever its neighbours weigh: seven tokens of 2^-24.1
    beside the best one, at u = 1 (the last mass) and in the best one's log share."""
    w = math.exp(-16.7)
    for dtype in (F32, BF):
        x = torch.full((2, 8), -16.7, device=DEV)
        x[:, 0] = 0.0
        x = x.to(dtype)
        w = math.exp(float(x[0, 1]))
        tok, lp = _run(x, [1.0, 0.0], dict())
        assert tok.tolist() == [7, 0]
        # a mass is a multiple of 2^-40: half a step for each of seven; their sum with the
        # best one's, 1 + 7 w, reaches the logarithm as an fp32 number: half a step of 2^-23
        assert abs(lp[1] + math.log1p(7 * w)) <= 7 * 2.0 ** -41 + 7 * w * 2.0 ** -20 + 2.0 ** -24


def test_sample_does_not_depend_on_the_batch():
    """A row gives the same token and the same log share alone (a cluster of eight CTAs)
    and among many (of two or four), whichever way its border is found."""
    # the k best in places where clusters of two gather them and clusters of eight search
    vocab, k = 16000, 500
    row = torch.full((1, vocab), -30.0, device=DEV)
    row[0, 3000:3300] = row[0, 12000:12300] = -16.7
    row[0, 3000] = 0.0
    how = dict(top_k=[k])
    many = 60
    u = [0.2, 0.99999]
    for ui in u:
        t1, l1 = _run(row, [ui], how)
        t2, l2 = _run(row.repeat(many, 1), [ui] * many, {n: v * many for n, v in how.items()})
        assert (t2 == t1[0]).all() and (l2 == l1[0]).all()
    _check(row, u[:1], how)
    rng = np.random.default_rng(12)
    for dtype in (F32, BF):
        for vocab in (5000, 24001, 70001):
            x = _logits(rng, 4, vocab, dtype, scale=3.0)
            x[2] = torch.round(x[2].float() * 4).to(dtype) / 4     # long ties
            for how in GRID + [dict(top_k=500), dict(top_k=500, top_p=0.9), dict(top_k=3000, top_p=0.99, min_p=1e-4)]:
                u = rng.random(4)
                t2, l2 = _run(x.repeat(24, 1), np.tile(u, 24), {n: [v] * 96 for n, v in how.items()})
                for i in range(4):
                    t1, l1 = _run(x[i:i + 1], u[i:i + 1], {n: [v] for n, v in how.items()})
                    assert (t2[i::4] == t1[0]).all() and (l2[i::4] == l1[0]).all(), (dtype, vocab, how, i)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sample_largest_vocabulary(dtype):
    """2^22 equal logits: the most tokens to a thread, each of the largest mass, whose sum
    is 2^62; then random ones."""
    vocab = 1 << 22
    x = torch.zeros(3, vocab, dtype=dtype, device=DEV)
    for how, kept in ((dict(), vocab), (dict(top_p=0.5), vocab // 2), (dict(top_k=1000000), 1000000),
                      (dict(top_k=3000000, top_p=0.25), 750000), (dict(top_k=500), 500)):
        tok, lp = _run(x, [0.5, 0.0, 1.0], {k: [v] * 3 for k, v in how.items()})
        assert tok.tolist() == [kept // 2, 0, kept - 1]
        assert np.all(np.abs(lp + math.log(kept)) <= 2.0 ** -23 * math.log(kept) + 2.0 ** -23)
    rng = np.random.default_rng(13)
    x = _logits(rng, 2, vocab, dtype)
    _check(x, rng.random(2), dict(top_p=[1.0, 0.9], top_k=[0, 2000000]))
