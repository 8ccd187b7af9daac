"""The target model's side of a speculative cycle over a paged KV cache: its
operators in plain PyTorch and through the library, on real sizes.

A verification pass takes the new tokens of every request (one token, a drafted
chain, a draft tree, or a chunk of a prompt) through these steps per layer:

  norm_rope   per-head RMSNorm of queries and keys, then the position rotation
  append      keys (rotated on the way) and values into the paged cache
  attention   the new tokens over the paged cache, causal or by a tree's mask

and, after the LM head,

  sample      the target's token of every row from given random numbers under
              temperature, top-k, top-p and min-p

Where `own` is false, run() computes the plain forms; where it is true, it calls
the library (block_diffusion_speculative_kv_gb300.binding)."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    """Head counts, contexts, block length, tree budget and vocabulary are those
    of the repository's Qwen3-shaped workloads; the odd ones are generic."""
    q8 = dict(n_q=32, n_kv=8, hd=128)
    return [
        # one interactive request, one token at a time: latency
        dict(name="attn decode 1x2048", op="attention", n_req=1, rows_lo=1, rows_hi=1, ctx_lo=2048,
             ctx_hi=2048, page=16, tree=False, lens=0, **q8),
        # a serving batch of plain decoding, contexts as ragged as the batched workload's
        dict(name="attn decode 32xragged", op="attention", n_req=32, rows_lo=1, rows_hi=1,
             ctx_lo=512, ctx_hi=8192, page=16, tree=False, lens=3, **q8),
        # the batch verifies drafted chains: anchor + 15 drafted tokens for each request
        dict(name="attn chain 32x16", op="attention", n_req=32, rows_lo=16, rows_hi=16, ctx_lo=512,
             ctx_hi=8192, page=32, tree=False, lens=4, **q8),
        # one request verifies a 256-node draft tree over a long context
        dict(name="attn tree 1x257", op="attention", n_req=1, rows_lo=257, rows_hi=257, ctx_lo=8192,
             ctx_hi=8192, page=64, tree=True, lens=5, **q8),
        # a chunk of a prompt over what is already cached
        dict(name="attn chunk 2048+8192", op="attention", n_req=1, rows_lo=2048, rows_hi=2048,
             ctx_lo=8192, ctx_hi=8192, page=128, tree=False, lens=6, **q8),
        # a mixed batch: requests that decode, wait (no row) or read prompts; 7 queries per KV head
        dict(name="attn mixed 9 hd64", op="attention", n_req=9, rows_lo=0, rows_hi=701, ctx_lo=0,
             ctx_hi=2999, page=16, tree=False, lens=7, n_q=14, n_kv=2, hd=64),
        # the keys and values of one decoded token of each of 32 requests
        dict(name="append 32x1", op="append", n_req=32, rows_lo=1, rows_hi=1, ctx_lo=100,
             ctx_hi=500, page=16, dtype="bf16", rope=True, lens=8, n_kv=8, hd=128),
        # prompts of several requests at once
        dict(name="append 6xragged", op="append", n_req=6, rows_lo=1000, rows_hi=4001, ctx_lo=0,
             ctx_hi=700, page=64, dtype="bf16", rope=True, lens=9, n_kv=8, hd=128),
        # queries and keys of 32 decoded tokens
        dict(name="norm_rope 32", op="norm_rope", rows=32, dtype="bf16", far=8192, **q8),
        # queries and keys of a prompt chunk, out of one QKV projection's rows
        dict(name="norm_rope 8197", op="norm_rope", rows=8197, dtype="bf16", far=16384, **q8),
        # the next token of one request
        dict(name="sample 1 fp32", op="sample", rows=1, vocab=151936, dtype="fp32", params=10),
        # the target's token at every drafted position of 32 requests, each with its own settings
        dict(name="sample 480 bf16", op="sample", rows=480, vocab=151936, dtype="bf16", params=11),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "norm_rope", "sample"])
    lens = rng.randrange(1 << 30)
    if op == "attention":
        n_q, n_kv = rng.choice([(32, 8), (16, 4), (8, 8), (14, 2), (64, 8), (32, 2), (5, 1), (24, 8)])
        hd = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128, 256])
        kind = rng.choice(["decode", "chain", "tree", "chunk"])
        hi = {"decode": 1, "chain": _log_int(rng, 2, 32), "tree": _log_int(rng, 17, 513),
              "chunk": _log_int(rng, 33, 2048)}[kind]
        lo = rng.choice([0, 1, hi])
        ctx_hi = _log_int(rng, 16, 16384)
        n_req = _log_int(rng, 1, 32)
        # what a plain form holds stays below the largest listed case's
        while (n_req * n_q * hi * (ctx_hi + hi) > 3 * 10 ** 8 or
               n_req * n_kv * (ctx_hi + hi) * hd > 2 * 10 ** 8):
            if n_req > 1:
                n_req //= 2
            else:
                ctx_hi, hi = (ctx_hi * 2 // 3, hi) if ctx_hi > hi else (ctx_hi, hi * 2 // 3)
        lo = min(lo, hi)
        return dict(op=op, n_req=n_req, rows_lo=lo, rows_hi=hi, ctx_lo=rng.choice([0, ctx_hi // 3]),
                    ctx_hi=ctx_hi, page=page, tree=kind == "tree", lens=lens, n_q=n_q, n_kv=n_kv,
                    hd=hd)
    if op == "append":
        n_req = _log_int(rng, 1, 48)
        hi = max(1, _log_int(rng, 1, 12000) // n_req)
        return dict(op=op, n_req=n_req, rows_lo=rng.choice([0, 1, hi]), rows_hi=hi, ctx_lo=0,
                    ctx_hi=_log_int(rng, 1, 600), page=rng.choice([16, 32, 64, 128, 256]),
                    dtype=rng.choice(["bf16", "fp32"]), rope=rng.random() < 0.8, lens=lens,
                    n_kv=rng.choice([1, 2, 5, 8]), hd=rng.choice([64, 128]))
    if op == "norm_rope":
        n_q, n_kv = rng.choice([(32, 8), (16, 4), (8, 8), (14, 2), (5, 1)])
        return dict(op=op, rows=_log_int(rng, 1, 8000), dtype=rng.choice(["bf16", "fp32"]),
                    far=_log_int(rng, 64, 1 << 20), n_q=n_q, n_kv=n_kv, hd=rng.choice([64, 128]))
    return dict(op=op, rows=_log_int(rng, 1, 400), vocab=_log_int(rng, 1000, 160000),
                dtype=rng.choice(["bf16", "fp32"]), params=lens)


def _lengths(case):
    """Rows and earlier context of each request: the case's alone."""
    rng = random.Random(case["lens"])
    rows = [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["n_req"])]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n_req"])]
    rows[-1] = max(rows[-1], 1)
    return rows, ctx


def _dtype(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


THETA = 1.0e6
EPS = 1.0e-6


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


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=DEV).to(dtype)

    s = {"case": case, "op": op}
    if op in ("attention", "append"):
        rows, ctx = _lengths(case)
        n, n_kv, hd, dt = sum(rows), case["n_kv"], case["hd"], _dtype(case)
        table, n_pages = _page_table(case, rows, ctx, gen)
        s.update(max_rows=max(rows), max_kv=max(r + c for r, c in zip(rows, ctx)), n=n,
                 row_off=_prefix(rows), pos0=torch.tensor(ctx, dtype=torch.int32, device=DEV),
                 table=table)
        s["pool_k"] = normal(n_pages, n_kv, case["page"], hd, dtype=dt)
        s["pool_v"] = normal(n_pages, n_kv, case["page"], hd, dtype=dt)
        if op == "attention":
            s["q"] = normal(n, case["n_q"] * hd)
            s["out"] = torch.empty_like(s["q"])
            s["mask"] = _tree_masks(rows, seed) if case["tree"] else None
        else:
            # the K and V columns of a projection's rows
            kv = normal(n, 2 * n_kv * hd, dtype=dt)
            s["k"], s["v"] = kv[:, :n_kv * hd], kv[:, n_kv * hd:]
    elif op == "norm_rope":
        n, n_q, n_kv, hd, dt = case["rows"], case["n_q"], case["n_kv"], case["hd"], _dtype(case)
        qkv = normal(n, (n_q + 2 * n_kv) * hd, dtype=dt)
        s["q"], s["k"] = qkv[:, :n_q * hd], qkv[:, n_q * hd:(n_q + n_kv) * hd]
        s["q_gain"] = (1 + 0.2 * torch.randn(hd, generator=gen, device=DEV)).to(dt)
        s["k_gain"] = (1 + 0.2 * torch.randn(hd, generator=gen, device=DEV)).to(dt)
        s["pos"] = torch.randint(0, case["far"], (n,), generator=gen, device=DEV).to(torch.int32)
        s["q_out"] = torch.empty(n, n_q * hd, dtype=dt, device=DEV)
        s["k_out"] = torch.empty(n, n_kv * hd, dtype=dt, device=DEV)
    else:
        n, vocab = case["rows"], case["vocab"]
        # N(0, 2) and a planted favourite, as the repository's logits workload has them
        x = torch.randn(n, vocab, generator=gen, device=DEV) * math.sqrt(2.0)
        fav = torch.randint(0, vocab, (n, 1), generator=gen, device=DEV)
        s["logits"] = x.scatter_add_(1, fav, torch.full((n, 1), 8.0, device=DEV)).to(_dtype(case))
        rng = random.Random(case["params"])

        def per_row(values, dtype):
            return torch.tensor([rng.choice(values) for _ in range(n)], dtype=dtype, device=DEV)

        s["temperature"] = per_row([0.0, 0.6, 0.7, 0.85, 1.0, 1.3, 2.0] if n > 1 else [0.8],
                                   torch.float32)
        s["top_k"] = per_row([0, 0, 1, 20, 50, 400] if n > 1 else [50], torch.int32)
        s["top_p"] = per_row([1.0, 0.5, 0.8, 0.9, 0.95] if n > 1 else [0.95], torch.float32)
        s["min_p"] = per_row([0.0, 0.0, 0.02, 0.1] if n > 1 else [0.01], torch.float32)
        s["u"] = torch.rand(n, generator=gen, device=DEV)
        s["tok"] = torch.empty(n, dtype=torch.int32, device=DEV)
        s["logp"] = torch.empty(n, dtype=torch.float32, device=DEV)
    if own:
        from block_diffusion_speculative_kv_gb300 import binding as bd
        if op in ("attention", "append"):
            s["pages"] = bd.Pages(s["pool_k"], s["pool_v"], s["table"])
        if op == "attention":
            nbytes = bd.paged_attention_workspace_bytes(case["n_q"], case["n_kv"], case["hd"])
            s["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _angles(pos, hd):
    """cos and sin of pos * theta^(-2i/hd), formed in 64 bits."""
    i = torch.arange(hd // 2, device=pos.device, dtype=torch.float64)
    a = pos.double()[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64, device=pos.device),
                                          -2.0 * i / hd)
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, cos, sin):
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _places(s):
    """The request and the place in it of every new row."""
    n = (s["row_off"][1:] - s["row_off"][:-1]).long()
    req = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=s["n"])
    return req, torch.arange(s["n"], device=DEV) - s["row_off"].long()[req]


def _attention(s):
    c = s["case"]
    n_kv, hd, G = c["n_kv"], c["hd"], c["n_q"] // c["n_kv"]
    req, at = _places(s)
    R, T = s["max_rows"], s["max_kv"]
    table = s["table"].long().clamp(min=0)

    def slots(pool):     # [n_req, n_kv, T, hd] in 32 bits
        p = pool[table].permute(0, 2, 1, 3, 4)
        return p.reshape(p.shape[0], n_kv, -1, hd)[:, :, :T].float()

    q = torch.zeros(c["n_req"], R, n_kv, G, hd, device=DEV)
    q[req, at] = s["q"].view(-1, n_kv, G, hd).float()
    q = q.permute(0, 2, 3, 1, 4).reshape(c["n_req"], n_kv, G * R, hd)
    score = (q @ slots(s["pool_k"]).transpose(2, 3)) * hd ** -0.5
    score = score.view(c["n_req"], n_kv, G, R, T)
    # which slots each row sees: [n_req, R, T]
    t = torch.arange(T, device=DEV)
    pos0 = s["pos0"].long()
    if s["mask"] is None:
        last = pos0[:, None] + torch.arange(R, device=DEV)
        sees = t <= last[:, :, None]
    else:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        bits = torch.nn.functional.pad(bits.reshape(s["n"], -1), (0, 1)).bool()
        new = t - pos0[:, None]                                     # [n_req, T]
        new = torch.where((new < 0) | (new >= bits.shape[1]), bits.shape[1] - 1, new)
        row_sees = torch.gather(bits, 1, new[req]) | (t < pos0[req][:, None])
        sees = torch.zeros(c["n_req"], R, T, dtype=torch.bool, device=DEV)
        sees[req, at] = row_sees
    score = torch.where(sees[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(c["n_req"], n_kv, G * R, T) @ slots(s["pool_v"])).view(c["n_req"], n_kv, G, R, hd)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4)[req, at].reshape(s["n"], -1).to(s["q"].dtype)


def _append(s):
    c = s["case"]
    req, at = _places(s)
    slot = s["pos0"].long()[req] + at
    k = s["k"].view(-1, c["n_kv"], c["hd"])
    if c["rope"]:
        k = _rotate(k.float(), *_angles(slot, c["hd"])).to(k.dtype)
    page = s["table"].long()[req, slot // c["page"]]
    s["pool_k"][page, :, slot % c["page"]] = k
    s["pool_v"][page, :, slot % c["page"]] = s["v"].view(-1, c["n_kv"], c["hd"])
    return s["pool_k"], s["pool_v"]


def _norm_rope(s):
    cos, sin = _angles(s["pos"], s["case"]["hd"])

    def one(x, gain):
        h = x.view(x.shape[0], -1, s["case"]["hd"]).float()
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * gain.float()
        return _rotate(h, cos, sin).reshape(x.shape).to(x.dtype)

    return one(s["q"], s["q_gain"]), one(s["k"], s["k_gain"])


def _sample(s):
    """Temperature, top-k, top-p of what is left, min-p against the best; then the
    first token, by id, whose cumulated mass passes u times the whole."""
    x = s["logits"].double()
    n, vocab = x.shape
    T = s["temperature"].double()[:, None]
    greedy = T <= 0
    T = torch.where(greedy, 1.0, T)
    v, order = torch.sort(x, dim=1, descending=True, stable=True)
    best = v[:, :1]
    w = torch.exp((v - best) / T)
    rank = torch.arange(vocab, device=DEV)
    k = s["top_k"].long()[:, None]
    w = torch.where((k > 0) & (rank >= k), 0.0, w)
    before = torch.cumsum(w, 1) - w
    p = s["top_p"].double()[:, None]
    whole = w.sum(1, keepdim=True)
    w = torch.where((p < 1) & (before >= p * whole) & (rank > 0), 0.0, w)
    m = s["min_p"].double()[:, None]
    w = torch.where((m > 0) & (v - best < T * torch.log(torch.where(m > 0, m, 1.0))), 0.0, w)
    w = torch.where(greedy & (rank > 0), 0.0, w)
    by_id = torch.zeros_like(w).scatter_(1, order, w)
    cum = torch.cumsum(by_id, 1)
    whole = cum[:, -1:].contiguous()
    tok = torch.searchsorted(cum, s["u"].double()[:, None] * whole, right=True).clamp(max=vocab - 1)
    logp = torch.log(torch.gather(by_id, 1, tok) / whole)
    return tok[:, 0].to(torch.int32), logp[:, 0].float()


def _library(s):
    from block_diffusion_speculative_kv_gb300 import binding as bd
    c = s["case"]
    if s["op"] == "attention":
        bd.paged_attention(s["pages"], s["q"], s["row_off"], s["pos0"], s["max_rows"], s["out"],
                           s["ws"], mask=s["mask"])
        return s["out"]
    if s["op"] == "append":
        bd.paged_append(s["pages"], s["k"], s["v"], s["row_off"], s["pos0"],
                        theta=THETA if c["rope"] else 0.0)
        return s["pool_k"], s["pool_v"]
    if s["op"] == "norm_rope":
        bd.qk_norm_rope(s["q"], s["k"], s["q_gain"], s["k_gain"], EPS, THETA, s["pos"], c["hd"],
                        s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    bd.logits_sample_filtered(s["logits"], s["u"], s["tok"], s["logp"],
                              temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                              min_p=s["min_p"])
    return s["tok"], s["logp"]


def run(state):
    if own:
        return _library(state)
    return {"attention": _attention, "append": _append, "norm_rope": _norm_rope,
            "sample": _sample}[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = 4 if case.get("dtype") == "fp32" else 2
    if op == "sample":
        n, vocab = case["rows"], case["vocab"]
        return {"bytes": n * (vocab * size + 28), "flops": 2.0 * n * vocab}
    if op == "norm_rope":
        n, heads, hd = case["rows"], case["n_q"] + case["n_kv"], case["hd"]
        return {"bytes": n * (2 * heads * hd * size + 4) + 2 * hd * size,
                "flops": 8.0 * n * heads * hd}
    rows, ctx = _lengths(case)
    n, n_kv, hd = sum(rows), case["n_kv"], case["hd"]
    tables = sum(4 * -(-(r + c) // case["page"]) for r, c in zip(rows, ctx)) + 8 * len(rows) + 4
    if op == "append":
        return {"bytes": n * 4 * n_kv * hd * size + tables, "flops": 3.0 * n * n_kv * hd}
    held = sum(r + c for r, c in zip(rows, ctx) if r)      # slots some row reads
    # a tree's rows see the whole context and, on average, few of each other
    seen = sum(r * c + (r * (r + 1) // 2 if not case["tree"] else r) for r, c in zip(rows, ctx))
    mask = 4 * n * ((max(rows) + 31) // 32) if case["tree"] else 0
    return {"bytes": 4 * held * n_kv * hd + 4 * n * case["n_q"] * hd + tables + mask,
            "flops": 4.0 * seen * case["n_q"] * hd}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    hd = case.get("hd")
    f64 = torch.float64
    if op == "attention":
        rows, ctx = _lengths(case)
        off = np.concatenate([[0], np.cumsum(rows)])
        G = case["n_q"] // case["n_kv"]
        out = torch.zeros(s["n"], case["n_q"], hd, dtype=f64, device=DEV)
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
                keys = torch.cat([s["pool_k"][i, g] for i in ids])[:kv].to(f64)
                values = torch.cat([s["pool_v"][i, g] for i in ids])[:kv].to(f64)
                for h in range(g * G, (g + 1) * G):
                    q = s["q"][off[r]:off[r + 1], h * hd:(h + 1) * hd].to(f64)
                    a = (q @ keys.T / math.sqrt(hd)).masked_fill_(hidden, -math.inf)
                    lse = torch.logsumexp(a, 1, keepdim=True)
                    out[off[r]:off[r + 1], h] = a.sub_(lse).exp_() @ values
        return out.view(s["n"], -1)
    if op == "append":
        rows, ctx = _lengths(case)
        off = np.concatenate([[0], np.cumsum(rows)])
        pools = [s["pool_k"].to(f64), s["pool_v"].to(f64)]
        for r in range(case["n_req"]):
            for i0 in range(0, rows[r]):
                t = ctx[r] + i0
                if i0 and t % case["page"]:
                    continue                                  # a page's rows go together
                m = min(case["page"] - t % case["page"], rows[r] - i0)
                page = int(s["table"][r, t // case["page"]])
                a = off[r] + i0
                for x, pool in ((s["k"], pools[0]), (s["v"], pools[1])):
                    y = x[a:a + m].to(f64).view(m, case["n_kv"], hd)
                    if x is s["k"] and case["rope"]:
                        y = _turn(y, torch.arange(t, t + m, device=DEV))
                    pool[page, :, t % case["page"]:t % case["page"] + m] = y.transpose(0, 1)
        return tuple(pools)
    if op == "norm_rope":
        got = []
        for x, g in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            y = x.to(f64).reshape(x.shape[0], -1, hd)
            y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / hd + EPS).sqrt()
            got.append(_turn(y * g.to(f64), s["pos"]).reshape(x.shape))
        return tuple(got)
    # sampling: row by row, over the tokens sorted by (logit, -id)
    logits = s["logits"].double().cpu().numpy()
    par = {k: s[k].double().cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    logp = np.zeros(case["rows"])
    for i in range(case["rows"]):
        x, T = logits[i], par["temperature"][i]
        if T <= 0:
            continue                                          # the best token, for certain
        k = int(par["top_k"][i]) or len(x)
        if k < len(x):                                        # the k best, lower ids first
            cut = np.partition(x, len(x) - k)[len(x) - k]
            keep = np.flatnonzero(x > cut)
            keep = np.concatenate([keep, np.flatnonzero(x == cut)[:k - len(keep)]])
        else:
            keep = np.arange(len(x))
        keep = keep[np.lexsort((keep, -x[keep]))]
        w = np.exp((x[keep] - x.max()) / T)
        if par["top_p"][i] < 1:
            cum = np.cumsum(w)
            keep = keep[:max(1, np.searchsorted(cum, par["top_p"][i] * cum[-1], side="left") + 1)]
        if par["min_p"][i] > 0:
            keep = keep[x[keep] - x.max() >= T * math.log(par["min_p"][i])]
        keep = np.sort(keep)
        w = np.exp((x[keep] - x.max()) / T)
        cum = np.cumsum(w)
        j = min(np.searchsorted(cum, par["u"][i] * cum[-1], side="right"), len(keep) - 1)
        logp[i] = math.log(w[j] / cum[-1])
    return None, torch.from_numpy(logp)


def _turn(y, pos):
    """Pairs (i, i + hd/2) of each head turned by pos * theta^(-2i/hd), as complex numbers."""
    half = y.shape[-1] // 2
    angle = pos.to(torch.float64)[:, None, None] * torch.exp(
        -math.log(THETA) * torch.arange(half, device=y.device, dtype=torch.float64) / half)
    z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1)
