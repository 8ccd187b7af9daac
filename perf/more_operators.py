"""Operators of the target's pass next to those of perf/operators.py: a paged KV
cache held in 8 bits, and what a sampler's settings do to logits, in plain PyTorch
and through the library, on real sizes.

  append      keys (rotated on the way) and values into a paged cache of e4m3 codes
              with a power-of-two scale for each block of 16 slots and KV head
  attention   the new tokens over that cache, causal or by a tree's mask
  adjust      bias, penalties for repeated tokens and a grammar's mask on the
              logits of every row, before the target's token is drawn

Where `own` is false, run() computes the plain forms; where it is true, it calls
the library (block_diffusion_speculative_kv_gb300.binding)."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 16            # slots that share a scale
TOP = 448.0           # the largest e4m3 value


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    """Head counts, contexts, block length, tree budget and vocabulary are those
    of the repository's Qwen3-shaped workloads; the odd ones are generic."""
    q8 = dict(n_q=32, n_kv=8, hd=128)
    return [
        # one interactive request, one token at a time: latency
        dict(name="attn8 decode 1x2048", op="attention", n_req=1, rows_lo=1, rows_hi=1, ctx_lo=2048,
             ctx_hi=2048, page=16, tree=False, lens=0, **q8),
        # a serving batch of plain decoding, contexts as ragged as the batched workload's
        dict(name="attn8 decode 32xragged", op="attention", n_req=32, rows_lo=1, rows_hi=1,
             ctx_lo=512, ctx_hi=8192, page=16, tree=False, lens=3, **q8),
        # the batch verifies drafted chains: anchor + 15 drafted tokens for each request
        dict(name="attn8 chain 32x16", op="attention", n_req=32, rows_lo=16, rows_hi=16, ctx_lo=512,
             ctx_hi=8192, page=32, tree=False, lens=4, **q8),
        # one request verifies a 256-node draft tree over a long context
        dict(name="attn8 tree 1x257", op="attention", n_req=1, rows_lo=257, rows_hi=257, ctx_lo=8192,
             ctx_hi=8192, page=64, tree=True, lens=5, **q8),
        # a chunk of a prompt over what is already cached
        dict(name="attn8 chunk 2048+8192", op="attention", n_req=1, rows_lo=2048, rows_hi=2048,
             ctx_lo=8192, ctx_hi=8192, page=128, tree=False, lens=6, **q8),
        # a mixed batch: requests that decode, wait (no row) or read prompts; 7 queries per KV head
        dict(name="attn8 mixed 9 hd64", op="attention", n_req=9, rows_lo=0, rows_hi=701, ctx_lo=0,
             ctx_hi=2999, page=16, tree=False, lens=7, n_q=14, n_kv=2, hd=64),
        # the keys and values of one decoded token of each of 32 requests
        dict(name="append8 32x1", op="append", n_req=32, rows_lo=1, rows_hi=1, ctx_lo=100, ctx_hi=500,
             page=16, dtype="bf16", rope=True, lens=8, n_kv=8, hd=128),
        # prompts of several requests at once
        dict(name="append8 6xragged", op="append", n_req=6, rows_lo=1000, rows_hi=4001, ctx_lo=0,
             ctx_hi=700, page=64, dtype="bf16", rope=True, lens=9, n_kv=8, hd=128),
        # the same from a projection that keeps 32 bits, keys rotated before
        dict(name="append8 5xragged fp32 hd64", op="append", n_req=5, rows_lo=1, rows_hi=3001, ctx_lo=0,
             ctx_hi=700, page=32, dtype="fp32", rope=False, lens=10, n_kv=5, hd=64),
        # the next token of one request with every setting on
        dict(name="adjust 1 fp32", op="adjust", n_req=1, rows_lo=1, rows_hi=1, hist_lo=2048, hist_hi=2048,
             vocab=151936, dtype="fp32", tree=False, bias=300, grammar=True, lens=11),
        # the drafted positions of 32 requests, each with its own history and settings
        dict(name="adjust 32x15 bf16", op="adjust", n_req=32, rows_lo=15, rows_hi=15, hist_lo=512,
             hist_hi=8192, vocab=151936, dtype="bf16", tree=False, bias=40, grammar=True, lens=12),
        # every node of one draft tree: a node's history is the context and its ancestors
        dict(name="adjust tree 257 fp32", op="adjust", n_req=1, rows_lo=257, rows_hi=257, hist_lo=8192,
             hist_hi=8192, vocab=151936, dtype="fp32", tree=True, bias=0, grammar=False, lens=13),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "adjust"])
    lens = rng.randrange(1 << 30)
    if op == "attention":
        n_q, n_kv = rng.choice([(32, 8), (16, 4), (8, 8), (14, 2), (64, 8), (32, 2), (5, 1), (24, 8)])
        hd = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128, 256])
        kind = rng.choice(["decode", "chain", "tree", "chunk"])
        hi = {"decode": 1, "chain": _log_int(rng, 2, 32), "tree": _log_int(rng, 17, 513),
              "chunk": _log_int(rng, 33, 2048)}[kind]
        ctx_hi = _log_int(rng, 16, 16384)
        n_req = _log_int(rng, 1, 32)
        # what a plain form holds stays below the largest listed case's
        while (n_req * n_q * hi * (ctx_hi + hi) > 3 * 10 ** 8 or
               n_req * n_kv * (ctx_hi + hi) * hd > 2 * 10 ** 8):
            if n_req > 1:
                n_req //= 2
            else:
                ctx_hi, hi = (ctx_hi * 2 // 3, hi) if ctx_hi > hi else (ctx_hi, hi * 2 // 3)
        return dict(op=op, n_req=n_req, rows_lo=min(rng.choice([0, 1, hi]), hi), rows_hi=hi,
                    ctx_lo=rng.choice([0, ctx_hi // 3]), ctx_hi=ctx_hi, page=page, tree=kind == "tree",
                    lens=lens, n_q=n_q, n_kv=n_kv, hd=hd)
    if op == "append":
        n_req = _log_int(rng, 1, 48)
        hi = max(1, _log_int(rng, 1, 12000) // n_req)
        return dict(op=op, n_req=n_req, rows_lo=rng.choice([0, 1, hi]), rows_hi=hi, ctx_lo=0,
                    ctx_hi=_log_int(rng, 1, 600), page=rng.choice([16, 32, 64, 128, 256]),
                    dtype=rng.choice(["bf16", "fp32"]), rope=rng.random() < 0.8, lens=lens,
                    n_kv=rng.choice([1, 2, 5, 8]), hd=rng.choice([64, 128]))
    vocab = _log_int(rng, 1000, 160000)
    n_req = _log_int(rng, 1, 40)
    tree = rng.random() < 0.4
    hi = min(_log_int(rng, 1, 257 if tree else 32), max(1, 70 * 10 ** 6 // vocab // n_req))
    hist_hi = _log_int(rng, 1, 12000)
    return dict(op=op, n_req=n_req, rows_lo=min(rng.choice([0, 1, hi]), hi), rows_hi=hi,
                hist_lo=rng.choice([0, hist_hi // 3]), hist_hi=hist_hi, vocab=vocab,
                dtype=rng.choice(["bf16", "fp32"]), tree=tree, bias=rng.choice([0, 1, 33, 300]),
                grammar=rng.random() < 0.5, lens=lens)


def _lengths(case):
    """Rows and earlier context (or history) of each request: the case's alone."""
    rng = random.Random(case["lens"])
    lo, hi = ("hist_lo", "hist_hi") if case["op"] == "adjust" else ("ctx_lo", "ctx_hi")
    rows = [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["n_req"])]
    ctx = [rng.randint(case[lo], case[hi]) for _ in range(case["n_req"])]
    rows[-1] = max(rows[-1], 1)
    return rows, ctx


def _dtype(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


THETA = 1.0e6


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------

def _prefix(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)


def _page_table(case, rows, ctx, gen):
    """A shuffled page table and the pool's size: some pages belong to nobody."""
    need = [-(-(r + c) // case["page"]) for r, c in zip(rows, ctx)]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((case["n_req"], max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _tree_masks(rows, seed):
    """Ancestor masks of random trees, one row of bits for each new row."""
    rng = random.Random(seed)
    words = (max(rows) + 31) // 32
    out = np.zeros((sum(rows), words), dtype=np.uint32)
    at = 0
    for n in rows:
        bits = []
        for i in range(n):
            parent = bits[rng.randrange(max(0, i - 40), i)] if i else 0
            bits.append(parent | (1 << i))
            out[at + i] = np.frombuffer(bits[i].to_bytes(4 * words, "little"), dtype=np.uint32)
        at += n
    return torch.from_numpy(out.view(np.int32)).to(DEV)


def _held(n_pages, n_kv, page, hd, outliers, gen):
    """A pool in 8 bits as earlier steps left it: codes, and the blocks' scales as
    biased exponents.  Magnitudes differ from block to block; keys have a few channels
    that stand out."""
    x = torch.randn(n_pages, n_kv, page // BLOCK, BLOCK, hd, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(n_pages, n_kv, page // BLOCK, 1, 1, generator=gen, device=DEV))
    if outliers:
        x[..., torch.randint(0, hd, (3,), generator=gen, device=DEV)] *= 5.0
    e = torch.ceil(torch.log2(x.abs().amax((-1, -2), keepdim=True) / TOP)).clamp(min=-127)
    codes = (x * torch.exp2(-e)).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    scale = (e + 127).to(torch.uint8).view(n_pages, n_kv, page // BLOCK)
    return codes.view(n_pages, n_kv, page, hd), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    rows, ctx = _lengths(case)
    n = sum(rows)
    s = {"case": case, "op": op, "n": n, "row_off": _prefix(rows), "max_rows": max(rows)}

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=DEV).to(dtype)

    if op in ("attention", "append"):
        n_kv, hd, dt = case["n_kv"], case["hd"], _dtype(case)
        table, n_pages = _page_table(case, rows, ctx, gen)
        s.update(max_kv=max(r + c for r, c in zip(rows, ctx)), table=table,
                 pos0=torch.tensor(ctx, dtype=torch.int32, device=DEV))
        s["pool_k"], s["scale_k"] = _held(n_pages, n_kv, case["page"], hd, True, gen)
        s["pool_v"], s["scale_v"] = _held(n_pages, n_kv, case["page"], hd, False, gen)
        if op == "attention":
            s["q"] = normal(n, case["n_q"] * hd)
            s["out"] = torch.empty_like(s["q"])
            s["mask"] = _tree_masks(rows, seed) if case["tree"] else None
        else:
            # the K and V columns of a projection's rows, some tokens larger than others
            kv = normal(n, 2 * n_kv * hd, dtype=dt)
            kv *= torch.exp(0.5 * torch.randn(n, 1, generator=gen, device=DEV)).to(dt)
            s["k"], s["v"] = kv[:, :n_kv * hd], kv[:, n_kv * hd:]
            # slots of a request's last block that hold earlier tokens
            s["earlier"] = sum(c % BLOCK for r, c in zip(rows, ctx) if r)
    else:
        vocab, n_req, dt = case["vocab"], case["n_req"], _dtype(case)
        rng = random.Random(seed)
        # N(0, 2) and a planted favourite, as the repository's logits workload has them
        x = torch.randn(n, vocab, generator=gen, device=DEV) * math.sqrt(2.0)
        fav = torch.randint(0, vocab, (n, 1), generator=gen, device=DEV)
        s["logits"] = x.scatter_add_(1, fav, torch.full((n, 1), 8.0, device=DEV)).to(dt)
        s["out"] = torch.empty_like(s["logits"])

        def tokens(*shape):      # few tokens make up most of a text
            u = torch.rand(*shape, generator=gen, device=DEV, dtype=torch.float64)
            return torch.exp(u * math.log(vocab)).to(torch.int32) - 1

        s["history"] = tokens(n_req, max(max(ctx), 1))
        s["history_len"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["prompt_len"] = torch.tensor([rng.randint(0, c) for c in ctx], dtype=torch.int32, device=DEV)

        def per_request(values):
            return torch.tensor([rng.choice(values) for _ in range(n_req)], dtype=torch.float32, device=DEV)

        s["repetition"] = per_request([1.0, 1.1, 1.2, 1.5] if n_req > 1 else [1.1])
        s["presence"] = per_request([0.0, 0.4, 1.5, -0.3] if n_req > 1 else [0.4])
        s["frequency"] = per_request([0.0, 0.1, 0.7, -0.2] if n_req > 1 else [0.1])
        s["tok"] = tokens(n)
        s["mask"] = _tree_masks(rows, seed) if case["tree"] else None
        s["bias_tok"] = s["bias_val"] = s["allowed"] = None
        if case["bias"]:
            # each request its own tokens; lists shorter than the longest end in -1
            m = case["bias"]
            start = torch.randint(0, vocab, (n_req, 1), generator=gen, device=DEV)
            step = max(1, vocab // (m + 1))
            at = (start + step * torch.arange(m, device=DEV)) % vocab
            at = torch.where(torch.arange(m, device=DEV) < vocab // step, at, -1)
            ends = torch.tensor([[rng.randint(0, m) if n_req > 1 else m] for _ in range(n_req)], device=DEV)
            s["bias_tok"] = torch.where(torch.arange(m, device=DEV) < ends, at, -1).to(torch.int32)
            s["bias_val"] = 4.0 * torch.randn(n_req, m, generator=gen, device=DEV)
        if case["grammar"]:
            # rows that may take anything, most tokens, or a few of them
            words = (vocab + 31) // 32
            bits = torch.randint(-2 ** 31, 2 ** 31, (n, words), generator=gen, device=DEV)
            few = torch.randint(0, words, (n, 4), generator=gen, device=DEV)
            some = torch.zeros_like(bits).scatter_(1, few, torch.gather(bits, 1, few) | 1)
            kind = torch.tensor([rng.randrange(3) for _ in range(n)], device=DEV)[:, None]
            bits = torch.where(kind == 0, -1, torch.where(kind == 1, bits | (bits >> 1), some))
            s["allowed"] = bits.to(torch.int32)
    if own:
        from block_diffusion_speculative_kv_gb300 import binding as bd
        if op in ("attention", "append"):
            s["pages"] = bd.PagesE4M3(s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"], s["table"])
        if op == "attention":
            nbytes = bd.paged_attention_e4m3_workspace_bytes(case["n_q"], case["n_kv"], case["hd"])
            s["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _places(s):
    """The request and the place in it of every new row."""
    n = (s["row_off"][1:] - s["row_off"][:-1]).long()
    req = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=s["n"])
    return req, torch.arange(s["n"], device=DEV) - s["row_off"].long()[req]


def _bits(mask, width):
    """Rows of words as rows of truth values."""
    b = (mask[:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    return b.reshape(mask.shape[0], -1)[:, :width].bool()


def _attention(s):
    c = s["case"]
    n_kv, hd, G = c["n_kv"], c["hd"], c["n_q"] // c["n_kv"]
    req, at = _places(s)
    R, T = s["max_rows"], s["max_kv"]
    table = s["table"].long().clamp(min=0)

    def slots(pool, scale):     # [n_req, n_kv, T, hd] in 32 bits
        p = pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).permute(0, 2, 1, 3, 4).float()
        e = torch.exp2(scale[table].permute(0, 2, 1, 3).float() - 127)
        p = p.reshape(p.shape[0], n_kv, -1, BLOCK, hd) * e.reshape(p.shape[0], n_kv, -1, 1, 1)
        return p.reshape(p.shape[0], n_kv, -1, hd)[:, :, :T]

    q = torch.zeros(c["n_req"], R, n_kv, G, hd, device=DEV)
    q[req, at] = s["q"].view(-1, n_kv, G, hd).float()
    q = q.permute(0, 2, 3, 1, 4).reshape(c["n_req"], n_kv, G * R, hd)
    score = (q @ slots(s["pool_k"], s["scale_k"]).transpose(2, 3)) * hd ** -0.5
    score = score.view(c["n_req"], n_kv, G, R, T)
    # which slots each row sees: [n_req, R, T]
    t = torch.arange(T, device=DEV)
    pos0 = s["pos0"].long()
    if s["mask"] is None:
        last = pos0[:, None] + torch.arange(R, device=DEV)
        sees = t <= last[:, :, None]
    else:
        bits = torch.nn.functional.pad(_bits(s["mask"], 32 * s["mask"].shape[1]), (0, 1))
        new = t - pos0[:, None]                                     # [n_req, T]
        new = torch.where((new < 0) | (new >= bits.shape[1]), bits.shape[1] - 1, new)
        row_sees = torch.gather(bits, 1, new[req]) | (t < pos0[req][:, None])
        sees = torch.zeros(c["n_req"], R, T, dtype=torch.bool, device=DEV)
        sees[req, at] = row_sees
    score = torch.where(sees[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = p.view(c["n_req"], n_kv, G * R, T) @ slots(s["pool_v"], s["scale_v"])
    o = o.view(c["n_req"], n_kv, G, R, hd)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4)[req, at].reshape(s["n"], -1).to(s["q"].dtype)


def _angles(pos, hd):
    """cos and sin of pos * theta^(-2i/hd), formed in 64 bits."""
    i = torch.arange(hd // 2, device=pos.device, dtype=torch.float64)
    a = pos.double()[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64, device=pos.device),
                                          -2.0 * i / hd)
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, cos, sin):
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append(s):
    """A block's scale is the smallest power of two at which its largest new value fits;
    a block that holds earlier tokens of the request keeps its scale or takes a larger
    one, at which those are then rounded again."""
    c = s["case"]
    n_kv, page, per = c["n_kv"], c["page"], c["page"] // BLOCK
    req, at = _places(s)
    pos0 = s["pos0"].long()
    slot = pos0[req] + at
    k = s["k"].reshape(-1, n_kv, c["hd"]).float()
    if c["rope"]:
        k = _rotate(k, *_angles(slot, c["hd"]))
    table = s["table"].long()
    where = table[req, slot // page]
    heads = torch.arange(n_kv, device=DEV)
    block = (where[:, None] * n_kv + heads) * per + (slot % page // BLOCK)[:, None]    # [n, n_kv]
    # the earlier tokens of the blocks that requests with new rows begin in
    some = s["row_off"][1:] > s["row_off"][:-1]
    n_old = torch.where(some, pos0 % BLOCK, 0)
    req_o = torch.repeat_interleave(torch.arange(c["n_req"], device=DEV), n_old, output_size=s["earlier"])
    at_o = torch.arange(s["earlier"], device=DEV) - (torch.cumsum(n_old, 0) - n_old)[req_o]
    slot_o = pos0[req_o] // BLOCK * BLOCK + at_o
    where_o = table[req_o, slot_o // page]
    block_o = (where_o[:, None] * n_kv + heads) * per + (slot_o % page // BLOCK)[:, None]
    for x, pool, scale in ((k, s["pool_k"], s["scale_k"]),
                           (s["v"].reshape(-1, n_kv, c["hd"]).float(), s["pool_v"], s["scale_v"])):
        flat, codes = scale.view(-1), pool.view(torch.uint8)
        top = torch.zeros(flat.numel(), device=DEV)
        top.scatter_reduce_(0, block.reshape(-1), x.abs().amax(-1).reshape(-1), "amax")
        m, e = torch.frexp(top)
        e = torch.where(top > 0, e - 9 + (m > 0.875).int() + 127, 0).clamp(min=0)
        old = torch.gather(flat, 0, block_o.reshape(-1)).int()
        e.scatter_reduce_(0, block_o.reshape(-1), old, "amax")
        shift = (old - e[block_o.reshape(-1)]).view(block_o.shape).float()
        was = codes[where_o, :, slot_o % page].view(torch.float8_e4m3fn).float()
        codes[where_o, :, slot_o % page] = (was * torch.exp2(shift)[:, :, None]).to(
            torch.float8_e4m3fn).view(torch.uint8)
        new = x * torch.exp2(127.0 - e[block].float())[:, :, None]
        codes[where, :, slot % page] = new.to(torch.float8_e4m3fn).view(torch.uint8)
        flat.scatter_(0, block.reshape(-1), e[block.reshape(-1)].to(torch.uint8))
    return s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"]


def _adjust(s):
    c = s["case"]
    vocab, n_req = c["vocab"], c["n_req"]
    req, at = _places(s)
    # how often a token occurred, in all and in what was generated: [n_req, vocab]
    h = s["history"].long()
    i = torch.arange(h.shape[1], device=DEV)
    there = (i < s["history_len"][:, None]).float()
    after = there * (i >= s["prompt_len"][:, None])
    seen = torch.zeros(n_req, vocab, device=DEV).scatter_add_(1, h, there)[req]
    made = torch.zeros(n_req, vocab, device=DEV).scatter_add_(1, h, after)[req]
    # the row's own path: the tokens of the rows of its request that it sees
    R = s["max_rows"]
    if s["mask"] is None:
        path = torch.arange(R, device=DEV) <= at[:, None]
    else:
        path = _bits(s["mask"], R)
    other = s["row_off"].long()[req][:, None] + torch.arange(R, device=DEV)
    path &= other < s["row_off"].long()[req + 1][:, None]
    tok = s["tok"].long()[other.clamp(max=s["n"] - 1)]
    seen.scatter_add_(1, tok, path.float())
    made.scatter_add_(1, tok, path.float())
    y = s["logits"].float()
    if s["bias_tok"] is not None:
        b = torch.zeros(n_req, vocab + 1, device=DEV)
        b.scatter_(1, torch.where(s["bias_tok"] < 0, vocab, s["bias_tok"]).long(), s["bias_val"])
        y = y + b[req, :vocab]
    rho, phi, pi = (s[k][req][:, None] for k in ("repetition", "frequency", "presence"))
    y = torch.where(seen > 0, torch.where(y > 0, y / rho, y * rho), y)
    y = y - phi * made - pi * (made > 0)
    if s["allowed"] is not None:
        y = torch.where(_bits(s["allowed"], vocab), y, -math.inf)
    return y.to(s["logits"].dtype)


def _library(s):
    from block_diffusion_speculative_kv_gb300 import binding as bd
    c = s["case"]
    if s["op"] == "attention":
        bd.paged_attention_e4m3(s["pages"], s["q"], s["row_off"], s["pos0"], s["max_rows"], s["out"],
                                s["ws"], mask=s["mask"])
        return s["out"]
    if s["op"] == "append":
        bd.paged_append_e4m3(s["pages"], s["k"], s["v"], s["row_off"], s["pos0"],
                             theta=THETA if c["rope"] else 0.0)
        return s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"]
    bd.logits_adjust(s["logits"], s["out"], s["row_off"], history=s["history"],
                     history_len=s["history_len"], prompt_len=s["prompt_len"],
                     repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                     tok=s["tok"], mask=s["mask"], bias_tok=s["bias_tok"], bias_val=s["bias_val"],
                     allowed=s["allowed"])
    return s["out"]


def run(state):
    if own:
        return _library(state)
    return {"attention": _attention, "append": _append, "adjust": _adjust}[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = 4 if case.get("dtype") == "fp32" else 2
    rows, ctx = _lengths(case)
    n = sum(rows)
    masks = 4 * n * ((max(rows) + 31) // 32) if case.get("tree") else 0
    if op == "adjust":
        vocab = case["vocab"]
        return {"bytes": 2 * n * vocab * size + 4 * sum(c for r, c in zip(rows, ctx) if r) + 4 * n + masks +
                (n * 4 * ((vocab + 31) // 32) if case["grammar"] else 0) + 8 * case["n_req"] * case["bias"],
                "flops": 2.0 * n * vocab}
    n_kv, hd = case["n_kv"], case["hd"]
    tables = sum(4 * -(-(r + c) // case["page"]) for r, c in zip(rows, ctx)) + 8 * len(rows) + 4
    if op == "append":
        blocks = sum(-(-(c % BLOCK + r) // BLOCK) for r, c in zip(rows, ctx))
        # rows of K and V in, their codes out, a scale for each block
        return {"bytes": 2 * n * n_kv * hd * (size + 1) + 2 * blocks * n_kv + tables,
                "flops": 4.0 * n * n_kv * hd}
    held = sum(r + c for r, c in zip(rows, ctx) if r)      # slots some row reads
    # a tree's rows see the whole context and, on average, few of each other
    seen = sum(r * c + (r * (r + 1) // 2 if not case["tree"] else r) for r, c in zip(rows, ctx))
    return {"bytes": 2 * held * n_kv * hd + 2 * n_kv * (held // BLOCK) + 4 * n * case["n_q"] * hd +
            tables + masks, "flops": 4.0 * seen * case["n_q"] * hd}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_64(x):
    """The e4m3 values nearest to x (ties to even), |x| <= 448, in 64 bits: steps of
    an eighth of the power of two below, of 2^-9 at least."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)) + 1e-12) - 3)
    return torch.round(x / step) * step


def _scale_64(top):
    """The smallest e >= -127 with top <= 448 * 2^e."""
    e = -127
    while top > TOP * 2.0 ** e:
        e += 1
    return e


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    hd = case.get("hd")
    f64 = torch.float64
    rows, ctx = _lengths(case)
    off = np.concatenate([[0], np.cumsum(rows)])
    if op == "attention":
        G = case["n_q"] // case["n_kv"]
        out = torch.zeros(s["n"], case["n_q"], hd, dtype=f64, device=DEV)

        def held(pool, scale, i, g):      # a page of a KV head
            e = scale[i, g].to(f64).repeat_interleave(BLOCK)[:, None] - 127
            return torch.ldexp(pool[i, g].to(torch.float32).to(f64), e)

        for r in range(case["n_req"]):
            n, kv = rows[r], rows[r] + ctx[r]
            if n == 0:
                continue
            ids = s["table"][r, :-(-kv // case["page"])].tolist()
            hidden = torch.arange(kv, device=DEV)[None] > ctx[r] + torch.arange(n, device=DEV)[:, None]
            if case["tree"]:
                m = s["mask"][off[r]:off[r + 1]].cpu().numpy().view(np.uint32)
                bits = np.unpackbits(m.view(np.uint8), axis=1, bitorder="little")[:, :n]
                hidden[:, ctx[r]:] = torch.from_numpy(bits == 0).to(DEV)
                hidden[:, :ctx[r]] = False
            for g in range(case["n_kv"]):
                keys = torch.cat([held(s["pool_k"], s["scale_k"], i, g) for i in ids])[:kv]
                values = torch.cat([held(s["pool_v"], s["scale_v"], i, g) for i in ids])[:kv]
                for h in range(g * G, (g + 1) * G):
                    q = s["q"][off[r]:off[r + 1], h * hd:(h + 1) * hd].to(f64)
                    a = (q @ keys.T / math.sqrt(hd)).masked_fill_(hidden, -math.inf)
                    lse = torch.logsumexp(a, 1, keepdim=True)
                    out[off[r]:off[r + 1], h] = a.sub_(lse).exp_() @ values
        return out.view(s["n"], -1)
    if op == "append":
        n_kv, page = case["n_kv"], case["page"]
        codes = [s[k].to(torch.float32).to(f64) for k in ("pool_k", "pool_v")]
        for r in range(case["n_req"]):
            t, a, end = ctx[r], off[r], ctx[r] + rows[r]
            while t < end:                                    # a block at a time
                m = min(BLOCK - t % BLOCK, end - t)
                p, b = int(s["table"][r, t // page]), t % page // BLOCK
                for x, held in ((s["k"], codes[0]), (s["v"], codes[1])):
                    y = x[a:a + m].to(f64).view(m, n_kv, hd)
                    if x is s["k"] and case["rope"]:
                        y = _turn(y, torch.arange(t, t + m, device=DEV))
                    scale = s["scale_k" if x is s["k"] else "scale_v"][p, :, b]
                    was = (scale.to(torch.int32) - 127).tolist()
                    tops = y.abs().amax((0, 2)).tolist()
                    now = [max(_scale_64(v), w if t % BLOCK else -127) for v, w in zip(tops, was)]
                    e = torch.tensor(now, device=DEV, dtype=f64)
                    fresh = _e4m3_64(torch.ldexp(y, -e[:, None])).transpose(0, 1)
                    held[p, :, t % page:t % page + m] = fresh
                    if t % BLOCK:
                        old = held[p, :, b * BLOCK:t % page]
                        by = torch.tensor(was, device=DEV, dtype=f64) - e
                        held[p, :, b * BLOCK:t % page] = _e4m3_64(torch.ldexp(old, by[:, None, None]))
                    scale.copy_((e + 127).to(torch.uint8))
                t, a = t + m, a + m
        return codes[0], codes[1], s["scale_k"], s["scale_v"]
    # adjusted logits, row by row
    vocab = case["vocab"]
    host = {k: v.cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor) and v.dtype is not torch.bfloat16}
    out = s["logits"].double().cpu().numpy()
    for r in range(case["n_req"]):
        past = host["history"][r, :ctx[r]]
        new = past[host["prompt_len"][r]:]
        rho, phi, pi = (float(host[k][r]) for k in ("repetition", "frequency", "presence"))
        for i in range(off[r], off[r + 1]):
            if case["tree"]:
                bits = np.unpackbits(host["mask"][i].view(np.uint8), bitorder="little")
                path = host["tok"][off[r]:off[r + 1]][bits[:rows[r]] == 1]
            else:
                path = host["tok"][off[r]:i + 1]
            y = out[i]
            if case["bias"]:
                for v, b in zip(host["bias_tok"][r], host["bias_val"][r]):
                    if v >= 0:
                        y[v] += float(b)
            known = np.unique(np.concatenate([past, path]))
            y[known] = np.where(y[known] > 0, y[known] / rho, y[known] * rho)
            made, count = np.unique(np.concatenate([new, path]), return_counts=True)
            y[made] -= phi * count + pi
            if case["grammar"]:
                y[np.unpackbits(host["allowed"][i].view(np.uint8), bitorder="little")[:vocab] == 0] = -np.inf
    return torch.from_numpy(out)


def _turn(y, pos):
    """Pairs (i, i + hd/2) of each head turned by pos * theta^(-2i/hd), as complex numbers."""
    half = y.shape[-1] // 2
    angle = pos.to(torch.float64)[:, None, None] * torch.exp(
        -math.log(THETA) * torch.arange(half, device=y.device, dtype=torch.float64) / half)
    z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1)
