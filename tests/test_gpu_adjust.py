"""GPU parity of dflash_logits_adjust against the 64-bit oracle, through the C ABI.

Tolerance, element by element: four fp32 roundings at most (bias, repetition, frequency,
presence), each 2^-24 of the sizes added up until then (the oracle's second result), and
half a step of the output's type, 2^-24 or 2^-8 of the value.  Logits that nothing
changes are equal bit for bit."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding as bd
from oracle import quant as oq
from test_gpu_paged import BF, DEV, F32, _i, _tree_mask

pytestmark = pytest.mark.gpu


def _case(rows, vocab, dtype, hist, tree=False, bias=0, grammar=False, seed=0, pad=0, low=1.0):
    """low: the share of the vocabulary that histories and paths come from."""
    rng = np.random.default_rng(seed + sum(rows) + vocab)
    n, n_req = sum(rows), len(rows)
    wide = torch.as_tensor(rng.normal(size=(n + 1, vocab + pad)) * 3, device=DEV).to(dtype)
    most = max(max(hist), 1)
    history = rng.integers(-1, max(1, int(low * vocab)), size=(n_req, most)).astype(np.int32)
    history[rng.random(history.shape) < 0.02] = vocab        # no token
    d = dict(logits=wide[:, :vocab], rows=rows, off=np.concatenate([[0], np.cumsum(rows)]), history=history,
             hist=np.array(hist), prompt=np.array([rng.integers(0, h + 1) for h in hist]),
             rep=rng.choice([1.0, 1.3, 0.7], size=n_req), pres=rng.choice([0.0, 0.5, -0.25], size=n_req),
             freq=rng.choice([0.0, 0.1, -0.3], size=n_req),
             tok=rng.integers(-1, max(1, int(low * vocab)), size=n + 1).astype(np.int32),
             mask=None, bias_tok=None, bias_val=None, allowed=None)
    if tree:
        d["mask"] = np.concatenate([_tree_mask(rng, rows, (max(rows) + 31) // 32), np.zeros((1, (max(rows) + 31) // 32), np.uint32)])
    if bias:
        d["bias_tok"] = rng.integers(-1, vocab + 1, size=(n_req, bias)).astype(np.int32)   # some twice
        d["bias_val"] = (rng.normal(size=(n_req, bias)) * 5).astype(np.float32)
    if grammar:
        words = (vocab + 31) // 32 + 2
        a = rng.integers(0, 1 << 32, size=(n + 1, words), dtype=np.uint64).astype(np.uint32)
        a[::3] = 0xFFFFFFFF
        a[1] = 0                                             # nothing is allowed
        d["allowed"] = a
    return d


def _dev(a, dtype=None):
    return None if a is None else torch.as_tensor(a.view(np.int32) if a.dtype == np.uint32 else a, dtype=dtype, device=DEV)


def _run(d, out=None, **over):
    x = d["logits"]
    out = torch.full_like(x, 7.0) if out is None else out
    kw = dict(history=_dev(d["history"]), history_len=_i(d["hist"]), prompt_len=_i(d["prompt"]),
              repetition=_dev(d["rep"], F32), presence=_dev(d["pres"], F32), frequency=_dev(d["freq"], F32),
              tok=_dev(d["tok"]), mask=_dev(d["mask"]), bias_tok=_dev(d["bias_tok"]), bias_val=_dev(d["bias_val"]),
              allowed=_dev(d["allowed"]))
    kw.update(over)
    bd.logits_adjust(x, out, _i(d["off"]), **kw)
    return out


def _oracle(d, **over):
    kw = dict(history=[h[:n] for h, n in zip(d["history"], d["hist"])], prompt_len=d["prompt"], repetition=np.float32(d["rep"]),
              presence=np.float32(d["pres"]), frequency=np.float32(d["freq"]), tok=d["tok"], mask=d["mask"],
              bias=None if d["bias_tok"] is None else [list(zip(t, v.astype(np.float64))) for t, v in zip(d["bias_tok"], d["bias_val"])],
              allowed=d["allowed"])
    kw.update(over)
    n = int(d["off"][-1])
    return oq.adjust(d["logits"][:n].double().cpu().numpy(), d["off"], **kw)


def _check(d, out, ref=None, size=None):
    if ref is None:
        ref, size = _oracle(d)
    n = int(d["off"][-1])
    got, was = out[:n].double().cpu().numpy(), d["logits"][:n].double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(ref))
    on = np.isfinite(ref)
    half = torch.finfo(d["logits"].dtype).eps / 2
    tol = 4 * 2.0 ** -24 * size + half * np.abs(np.where(on, ref, 0.0)) * (1 + 2.0 ** -7)
    assert np.all(np.abs(got[on] - ref[on]) <= tol[on])
    same = on & (ref == was)
    assert np.array_equal(got[same], was[same])
    assert torch.all(out[n:] == 7.0) or out.data_ptr() == d["logits"].data_ptr()


@pytest.mark.parametrize("rows,vocab,dtype,hist,tree,bias,grammar,pad", [
    ([1], 1, F32, [0], False, 0, False, 0),
    ([1], 5, BF, [9], False, 2, True, 0),
    ([1], 5000, F32, [700], False, 33, True, 0),
    ([1], 5003, BF, [3000], False, 1, True, 0),             # rows off 16-byte boundaries
    ([3, 0, 5], 4099, BF, [100, 50, 0], False, 7, True, 3),
    ([3, 0, 5], 4096, F32, [100, 50, 0], True, 0, False, 5),
    ([16] * 5, 8191, BF, [10, 900, 4, 0, 33], False, 40, True, 1),
    ([16, 17, 15, 1, 33], 9001, F32, [10, 900, 4, 0, 33], True, 40, True, 0),
    ([70], 12345, BF, [500], True, 3, True, 0),
    ([1] * 100, 300, F32, list(range(100)), False, 2, True, 0),     # more requests than a warp
    ([0] * 50 + [40] + [0] * 50, 600, BF, [5] * 101, True, 2, False, 0),
    ([2] * 600, 300, BF, [7] * 600, False, 3, True, 4),     # long stretches, groups of many rows
    ([40, 3, 0, 50] * 4, 20001, F32, [50] * 16, True, 5, True, 0),
])
def test_adjust(rows, vocab, dtype, hist, tree, bias, grammar, pad):
    for low in (1.0, 0.01):
        d = _case(rows, vocab, dtype, hist, tree, bias, grammar, pad=pad, low=low)
        out = _run(d)
        torch.cuda.synchronize()
        ref, size = _oracle(d)
        _check(d, out, ref, size)
        # a second call and one in place agree bit for bit
        again = _run(d)
        copy = torch.empty(d["logits"].shape[0], vocab + pad, dtype=dtype, device=DEV)[:, :vocab]
        copy.copy_(d["logits"])
        live = int(d["off"][-1])
        keep = copy[live:].clone()
        _run(dict(d, logits=copy), out=copy)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(out[:live], copy[:live]) and torch.equal(copy[live:], keep)


def test_adjust_parts():
    """Each setting alone, and none: a copy."""
    d = _case([5, 9, 1], 7000, F32, [300, 0, 40], True, 12, True, seed=5, low=0.02)
    off = {"history": None, "prompt_len": None, "repetition": None, "presence": None, "frequency": None, "tok": None,
           "mask": None, "bias": None, "allowed": None}
    full = dict(history=dict(history=[h[:n] for h, n in zip(d["history"], d["hist"])]), prompt_len=dict(prompt_len=d["prompt"]),
                repetition=dict(repetition=np.float32(d["rep"])), presence=dict(presence=np.float32(d["pres"])),
                frequency=dict(frequency=np.float32(d["freq"])), tok=dict(tok=d["tok"]), mask=dict(mask=d["mask"]),
                bias=dict(bias=[list(zip(t, v.astype(np.float64))) for t, v in zip(d["bias_tok"], d["bias_val"])]),
                allowed=dict(allowed=d["allowed"]))
    for on in ([], ["allowed"], ["bias"], ["history", "repetition"], ["history", "prompt_len", "frequency"],
               ["tok", "presence"], ["tok", "mask", "frequency", "repetition"], ["repetition"], ["tok", "mask"]):
        want = dict(off)
        for x in on:
            want.update(full[x])
        drop = {x: None for x in off if x not in on and x != "bias"}
        if "bias" not in on:
            drop.update(bias_tok=None, bias_val=None)
        if "history" not in on:
            drop["history_len"] = None
        out = _run(d, **drop)
        torch.cuda.synchronize()
        ref, size = _oracle(d, **want)
        _check(d, out, ref, size)
        if not on:
            assert torch.equal(out[:15], d["logits"][:15])


def test_adjust_special_values():
    """Infinities and NaN pass through; signs decide the repetition; lengths out of range."""
    x = torch.tensor([[float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1.0, -1.0, 2.0]], device=DEV)
    for dtype in (F32, BF):
        y = x.to(dtype)
        out = torch.empty_like(y)
        hist = _i([[0, 1, 2, 3, 4, 5, 6, 9]])
        bd.logits_adjust(y, out, _i([0, 1]), history=hist, history_len=_i([100]), prompt_len=_i([100]),
                         repetition=torch.tensor([2.0], device=DEV))
        torch.cuda.synchronize()
        assert out[0, :2].tolist() == [float("inf"), -float("inf")] and torch.isnan(out[0, 2])
        assert out[0, 3:].tolist() == [0.0, 0.0, 0.5, -2.0, 2.0]
        for n, p in ((-5, 0), (0, -7)):
            bd.logits_adjust(y, out, _i([0, 1]), history=hist, history_len=_i([n]), prompt_len=_i([p]),
                             repetition=torch.tensor([2.0], device=DEV))
            torch.cuda.synchronize()
            assert torch.equal(out.nan_to_num(99.0), y.nan_to_num(99.0))
    # more counts than any float step: a token 70000 times
    h = torch.full((1, 70000), 3, dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    bd.logits_adjust(x, out, _i([0, 1]), history=h, history_len=_i([70000]), frequency=torch.tensor([0.5], device=DEV))
    torch.cuda.synchronize()
    assert out[0, 3].item() == -35000.0


def test_adjust_leaves_columns_past_the_vocabulary():
    d = _case([4, 5], 3000, BF, [50, 60], False, 5, True)
    x = d["logits"]
    out = torch.full_like(x, 7.0)
    _run(d, out=out, vocab=2777, allowed=_dev(d["allowed"][:, :87].copy()))
    torch.cuda.synchronize()
    assert torch.all(out[:, 2777:] == 7.0)
    cut = dict(d, logits=x[:, :2777])
    _check(cut, out[:, :2777])


def test_adjust_reads_a_slice_of_a_wider_grammar():
    d = _case([7], 2000, F32, [20], False, 0, True)
    wide = torch.zeros(8, 100, dtype=torch.int32, device=DEV)
    wide[:, 9:9 + 65] = _dev(d["allowed"])
    out = _run(d, allowed=wide[:, 9:9 + 65])
    torch.cuda.synchronize()
    _check(d, out)


def test_adjust_in_a_graph_serves_growing_histories():
    d = _case([3, 1], 6000, F32, [40, 40], False, 5, False, low=0.01)
    length, off = _i([10, 20]), _i(d["off"])
    x, out = d["logits"].clone(), torch.full_like(d["logits"], 7.0)
    kw = dict(history=_dev(d["history"]), history_len=length, repetition=_dev(d["rep"], F32),
              frequency=_dev(d["freq"], F32), tok=_dev(d["tok"]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bd.logits_adjust(x, out, off, **kw)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        bd.logits_adjust(x, out, off, **kw)
    for n in ([10, 20], [0, 40], [33, 1]):
        length.copy_(_i(n))
        g.replay()
        torch.cuda.synchronize()
        ref, size = oq.adjust(x[:4].double().cpu().numpy(), d["off"], history=[h[:m] for h, m in zip(d["history"], n)],
                              repetition=np.float32(d["rep"]), frequency=np.float32(d["freq"]), tok=d["tok"])
        _check(dict(d, logits=x), out, ref, size)


def test_a_tree_node_is_penalised_as_its_path_would_be():
    """ddtree_build -> adjust -> filtered sampling -> the walk: at every node the target
    chooses as it would after generating the node's path one token at a time."""
    rng = np.random.default_rng(2)
    n_req, B, D, K, vocab = 3, 20, 5, 4, 4000
    lp = np.sort(rng.normal(size=(n_req, D, K)).astype(np.float32) - 3, axis=2)[:, :, ::-1].copy()
    ids = rng.integers(0, 50, size=(n_req, D, K)).astype(np.int32)       # tokens recur along a path
    bufs = bd.tree_buffers(n_req, B)
    bd.ddtree_build(torch.as_tensor(lp, device=DEV), _i(ids), _i([3, 4, 5]), B, *bufs)
    n_nodes, tok, parent, depth, rank, mask = bufs
    n = n_req * (B + 1)
    logits = torch.as_tensor(rng.normal(size=(n, vocab)) * 2, device=DEV).float()
    logits[:, :50] += 4
    hist = rng.integers(0, 50, size=(n_req, 30)).astype(np.int32)
    lens = [30, 7, 0]
    rep, freq = torch.tensor([1.4, 1.0, 1.2], device=DEV), torch.tensor([0.3, 1.5, 0.0], device=DEV)
    off = _i(np.arange(n_req + 1) * (B + 1))
    out = torch.empty_like(logits)
    bd.logits_adjust(logits, out, off, history=_i(hist), history_len=_i(lens), repetition=rep, frequency=freq,
                     tok=tok.view(-1), mask=mask.view(n, -1))
    u = torch.rand(n, device=DEV)
    temp, top_k = torch.full((n,), 0.8, device=DEV), torch.full((n,), 20, dtype=torch.int32, device=DEV)
    choice, logp = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, device=DEV)
    bd.logits_sample_filtered(out, u, choice, logp, temperature=temp, top_k=top_k)
    al, acc, bon = _i(np.zeros(n_req)), _i(np.zeros((n_req, D))), _i(np.zeros(n_req))
    bd.ddtree_accept(D, B, n_nodes, tok, parent, choice.view(n_req, B + 1), al, acc, bon)
    torch.cuda.synchronize()
    tok_h, par_h = tok.cpu().numpy(), parent.cpu().numpy()
    one_out, one_tok, one_lp = torch.empty(1, vocab, device=DEV), _i([0]), torch.empty(1, device=DEV)
    for r in range(n_req):
        for i in range(int(n_nodes[r]) + 1):
            path, j = [], i
            while j >= 0:
                path.append(int(tok_h[r, j]))
                j = int(par_h[r, j]) if j else -1
            past = list(hist[r, :lens[r]]) + path[::-1]
            row = r * (B + 1) + i
            bd.logits_adjust(logits[row:row + 1], one_out, _i([0, 1]), history=_i([past]), history_len=_i([len(past)]),
                             repetition=rep[r:r + 1], frequency=freq[r:r + 1])
            assert torch.equal(one_out[0], out[row])
            bd.logits_sample_filtered(one_out, u[row:row + 1], one_tok, one_lp, temperature=temp[:1], top_k=top_k[:1])
            assert int(one_tok) == int(choice[row])


def test_adjust_more_row_tokens_than_are_listed():
    """A mask over a thousand rows whose tokens all lie close together, paths of hundreds."""
    rng = np.random.default_rng(4)
    n, vocab = 1000, 700
    d = _case([n], vocab, F32, [300], False, 5, False, low=0.1)
    mask = rng.integers(0, 1 << 32, size=(n + 1, 32), dtype=np.uint64).astype(np.uint32)
    mask[::2] &= rng.integers(0, 1 << 32, size=mask[::2].shape, dtype=np.uint64).astype(np.uint32) & 0x11111111
    mask[5:60] = 0
    mask[20] = 1 << 31
    for tokens in (rng.integers(0, 60, size=n + 1), rng.integers(-1, vocab, size=n + 1)):
        e = dict(d, mask=mask, tok=tokens.astype(np.int32))
        out = _run(e)
        torch.cuda.synchronize()
        _check(e, out)


@pytest.mark.parametrize("rows,vocab,dtype,hist,tree,bias,grammar,pad", [
    ([1] * 40, 20001, F32, [25 * i for i in range(40)], False, 3, True, 0),
    ([1] * 40, 12296, BF, [5000 - 7 * i for i in range(40)], False, 30, True, 3),
    ([2, 0, 3, 1] * 60, 9001, F32, [9] * 240, True, 2, False, 1),
    ([0, 2, 1, 2] * 90, 8193, BF, [30] * 360, True, 0, True, 5),
    ([900] + [0] * 1000, 3000, F32, [40] * 1001, True, 1, False, 0),        # more row tokens than are listed
    ([0] * 1000 + [700], 4500, BF, [40] * 1001, False, 0, False, 1),
])
def test_adjust_requests_of_few_rows(rows, vocab, dtype, hist, tree, bias, grammar, pad):
    test_adjust(rows, vocab, dtype, hist, tree, bias, grammar, pad)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_adjust_alone_and_in_a_batch_agree(dtype):
    """However rows are shared out, bit for bit: a batch, a request, a row at a time."""
    rows = [16] * 20 + [1] * 4
    d = _case(rows, 20000, dtype, [300 + i for i in range(24)], False, 6, True, low=0.05)
    out = _run(d)
    torch.cuda.synchronize()
    for r in (0, 7, 19, 23):
        a, b = int(d["off"][r]), int(d["off"][r + 1])
        one = dict(d, logits=d["logits"][a:b], off=np.array([0, b - a]), tok=d["tok"][a:b], allowed=d["allowed"][a:b],
                   **{k: d[k][r:r + 1] for k in ("history", "hist", "prompt", "rep", "pres", "freq", "bias_tok", "bias_val")})
        got = _run(one)
        torch.cuda.synchronize()
        assert torch.equal(got, out[a:b])
        last = dict(one, logits=one["logits"][-1:], off=np.array([0, 1]), allowed=one["allowed"][-1:], tok=one["tok"][-1:],
                    history=np.concatenate([one["history"][:, :one["hist"][0]], one["tok"][None, :-1]], 1),
                    hist=one["hist"] + b - a - 1)
        got = _run(last)
        torch.cuda.synchronize()
        assert torch.equal(got[0], out[b - 1])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,span,few", [(257, 900, 1), (257, 40, 1), (600, 3000, 1), (200, 1000, 40), (65, 64, 1)])
def test_adjust_long_paths_through_common_tokens(dtype, n, span, few):
    """Masks that are chains, so that rows have up to n tokens of their own close together,
    some many times; one request, and many of few rows beside it."""
    rng = np.random.default_rng(n + span)
    rows = [n] + [1] * (few - 1) * 9
    d = _case(rows, 5003, dtype, [700] * len(rows), True, 20, True, seed=1, low=0.1, pad=1)
    d["mask"] = np.zeros((n + len(rows), (n + 31) // 32), dtype=np.uint32)
    for i in range(n):
        bits = np.arange(32 * d["mask"].shape[1]) <= i
        d["mask"][i] = np.packbits(bits, bitorder="little").view(np.uint32)
    d["mask"][n:, 0] = 1
    d["tok"] = rng.integers(-1, span, size=len(d["tok"])).astype(np.int32)
    out = _run(d)
    again = _run(d)
    torch.cuda.synchronize()
    _check(d, out)
    assert torch.equal(out, again)
