"""Workloads of the paged KV-cache operators, for timing and for comparing results.

One verification step of speculative decoding over a block-quantized, paged
KV cache is made of four operators, each reached through this package:

  kv_plan         pages given to and taken back from requests of changed
                  length; block tables and slot maps built on the device
  kv_append,      K / V rows quantized into the pages by the slot map, and the
  kv_compact      rows of the accepted path moved together
  attn_tree       attention of a tree of drafted tokens over the cache
  logits_process  penalties, biases and grammar masks on the logits

A case is a dict of plain values; request lengths that differ within a case
follow from its "mix".  `own` chooses between the plain torch form and the
package's calls.  Head layouts (32 query / 8 kv heads of 128, and the 32-, 64-
and 256-wide ones), the 32,768-position cache, the 32,000 and 128,256
vocabularies and the cache types are those of the package's own benchmark
and tests.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = {"Q8_0": 34, "Q5_0": 22, "Q4_0": 18}      # bytes of a 32-weight block
LEVELS = {"Q8_0": 127.0, "Q5_0": 15.0, "Q4_0": 7.0}
TREE_MAX = 64                                     # drafted tokens of one request, at most


def _qk():
    import gguf_quant_dequant_gb300 as qk
    return qk


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # Page bookkeeping between two steps of a server with a handful of
        # requests: only the latency of the call counts.
        dict(op="plan", name="plan_few", n_req=5, page=16, pages=64, tokens=9, scarce=False, mix=1),
        # A full batch of long requests, some finished, some new prompts of
        # thousands of tokens, more pages asked for than are free.
        dict(op="plan", name="plan_many", n_req=997, page=32, pages=1024, tokens=120, scarce=True, mix=2),
        # One drafted tree of a single user, accepted path kept.
        dict(op="append", name="append_tree", type="Q8_0", n_req=1, n=13, n_kv=8, d=128, page=16, act="f32", gap=0,
             compact=True, mix=3),
        # The drafted trees of a batch; k and v are slices of one fused
        # projection's output.
        dict(op="append", name="append_batch", type="Q5_0", n_req=61, n=29, n_kv=8, d=64, page=64, act="bf16", gap=2048,
             compact=True, mix=4),
        # A long prompt written to the cache.
        dict(op="append", name="append_prompt", type="Q4_0", n_req=4, n=8191, n_kv=8, d=128, page=32, act="bf16", gap=0,
             compact=False, mix=5),
        # A short chat, one token: the smallest attention call.
        dict(op="tree", name="tree_one_short", type="Q8_0", n_req=1, ctx_lo=211, ctx_hi=211, n_lo=1, n_hi=1, heads=32,
             n_kv=8, d=128, page=16, mix=6),
        # One user at a 32k context verifying a 16-token tree.
        dict(op="tree", name="tree_one_32k", type="Q8_0", n_req=1, ctx_lo=32749, ctx_hi=32749, n_lo=16, n_hi=16, heads=32,
             n_kv=8, d=128, page=32, mix=7),
        # A batch of ragged lengths, small trees, the 4-bit cache.
        dict(op="tree", name="tree_ragged_q4", type="Q4_0", n_req=27, ctx_lo=1, ctx_hi=8190, n_lo=1, n_hi=9, heads=32,
             n_kv=8, d=128, page=16, mix=8),
        # The largest trees: 64 nodes, eight query heads to a kv head.
        dict(op="tree", name="tree_wide_q5", type="Q5_0", n_req=7, ctx_lo=900, ctx_hi=6001, n_lo=57, n_hi=64, heads=32,
             n_kv=4, d=64, page=64, mix=9),
        # A server's whole batch: 1 GB of cache read by one call.
        dict(op="tree", name="tree_batch_q8", type="Q8_0", n_req=64, ctx_lo=500, ctx_hi=15000, n_lo=4, n_hi=8, heads=32,
             n_kv=8, d=128, page=128, mix=10),
        # One row of a small vocabulary: single-token decode.
        dict(op="logits", name="logits_one", n_req=1, n=1, vocab=32000, act="f32", hist=700, n_bias=6, grammar=False, mix=11),
        # A batch of drafted trees at the large vocabulary, grammar masks on.
        dict(op="logits", name="logits_trees", n_req=48, n=8, vocab=128256, act="f32", hist=4096, n_bias=40, grammar=True,
             mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "tree", "tree", "tree", "logits"])
    mix = rng.randrange(1 << 20)
    if op == "plan":
        return dict(op=op, n_req=_log(rng, 1, 997), page=rng.choice([16, 32, 64, 128, 256]), pages=_log(rng, 40, 1024),
                    tokens=_log(rng, 1, 120), scarce=rng.random() < 0.5, mix=mix)
    if op == "append":
        compact = rng.random() < 0.5
        n_req = _log(rng, 1, 61) if compact else _log(rng, 1, 4)
        n = _log(rng, 1, TREE_MAX) if compact else _log(rng, 1, 8191)
        return dict(op=op, type=rng.choice(list(BLOCK)), n_req=n_req, n=n, n_kv=rng.choice([1, 2, 4, 5, 8]),
                    d=rng.choice([32, 64, 128]), page=rng.choice([16, 32, 64, 128, 256]), act=rng.choice(["f32", "bf16"]),
                    gap=rng.choice([0, 0, 96, 2048]), compact=compact, mix=mix)
    if op == "tree":
        heads, n_kv, d = rng.choice([(32, 8, 128), (32, 4, 128), (8, 8, 128), (32, 4, 64), (8, 1, 64), (6, 2, 32), (12, 4, 256),
                                     (8, 2, 256)])
        n_req = _log(rng, 1, 64)
        # at most the largest listed case's cache bytes (about 2^29 positions x elements)
        hi = max(2, min(32752, (1 << 29) // (n_req * n_kv * d)))
        a, b = sorted((_log(rng, 1, hi), _log(rng, 1, hi)))
        n_top = TREE_MAX if n_req <= 8 else 8
        n_lo, n_hi = sorted((_log(rng, 1, n_top), _log(rng, 1, n_top)))
        return dict(op=op, type=rng.choice(list(BLOCK)), n_req=n_req, ctx_lo=a, ctx_hi=b, n_lo=n_lo, n_hi=n_hi, heads=heads,
                    n_kv=n_kv, d=d, page=rng.choice([16, 32, 64, 128, 256]), mix=mix)
    vocab = rng.choice([_log(rng, 1000, 128256), 32000, 32003, 50257, 128256])
    n_req = _log(rng, 1, 48)
    n = _log(rng, 1, max(1, min(TREE_MAX, 384 // n_req)))
    return dict(op=op, n_req=n_req, n=n, vocab=vocab, act=rng.choice(["f32", "f32", "bf16"]), hist=_log(rng, 1, 4096),
                n_bias=rng.choice([0, 1, 40]), grammar=rng.random() < 0.5, mix=mix)


def _lengths(case):
    """(context lengths, drafted tokens) of a tree case's requests."""
    r = random.Random(case["mix"])
    lo, hi = case["ctx_lo"], case["ctx_hi"]
    ctx = [r.randint(lo, hi) for _ in range(case["n_req"])]
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["n_req"])]
    ctx[0] = hi
    return ctx, n


def _resizes(case):
    """(have, start, want) of a plan case's requests: most grow by a few
    tokens, some were cut back to their accepted length, some are finished,
    some are new prompts."""
    r = random.Random(case["mix"])
    cap = case["pages"] * case["page"]
    have, start, want = [], [], []
    for _ in range(case["n_req"]):
        kind, h = r.random(), r.randint(1, cap // 2)
        if kind < 0.1:
            h, s, w = h, 0, 0                                   # finished
        elif kind < 0.25:
            s, w = 0, r.randint(1, min(cap, 16 * case["tokens"]))   # a new prompt
            h = 0
        elif kind < 0.5:
            s = max(0, h - r.randint(1, TREE_MAX))              # rejected drafts given back
            w = min(cap, s + r.randint(0, case["tokens"]))
        else:
            s, w = h, min(cap, h + r.randint(1, case["tokens"]))
        have.append(h)
        start.append(s)
        want.append(w)
    return have, start, want


def _tree(r, n):
    """Ancestor bits (own bit included) of a random tree of n nodes, each
    node's parent before it."""
    bits = []
    for i in range(n):
        p = r.randint(max(0, i - 6), i - 1) if i else -1
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return bits


def _signed(bits):
    return [b - (1 << 64) if b >> 63 else b for b in bits]


# ----------------------------------------------------- the block formats ----

def _pack(name, x):
    """fp32 [..., 32 m] -> packed bytes [..., m * block bytes]: d = fp16(max|x|
    / levels), code = round half away (x / d), clamped."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    top = g.abs().amax(-1, keepdim=True)
    d = (top / torch.full_like(top, LEVELS[name])).to(torch.float16)     # a true division: no reciprocal of a scalar
    df = d.float()
    q = torch.where(df != 0, g / torch.where(df != 0, df, torch.ones_like(df)), torch.zeros_like(g))
    a = torch.floor(q.abs())
    q = torch.sign(q) * (a + (q.abs() - a >= 0.5))
    head = d.contiguous().view(torch.uint8).reshape(*g.shape[:-1], 2)
    if name == "Q8_0":
        body = q.clamp(-128, 127).to(torch.int8).view(torch.uint8)
    else:
        off = 16 if name == "Q5_0" else 8
        u = (q + off).clamp(0, 2 * off - 1).to(torch.int32)
        body = ((u[..., :16] & 15) | ((u[..., 16:] & 15) << 4)).to(torch.uint8)
        if name == "Q5_0":
            b5 = (u >> 4).reshape(*u.shape[:-1], 4, 8)
            w = torch.tensor([1 << k for k in range(8)], device=x.device, dtype=torch.int32)
            body = torch.cat([(b5 * w).sum(-1).to(torch.uint8), body], -1)
    return torch.cat([head, body], -1).reshape(*x.shape[:-1], -1)


def _unpack(name, b, dtype=torch.float32):
    """Packed bytes [..., m * block bytes] -> the values they stand for [..., 32 m]."""
    blk = b.reshape(*b.shape[:-1], -1, BLOCK[name])
    d = blk[..., :2].contiguous().view(torch.float16).to(dtype)
    if name == "Q8_0":
        q = blk[..., 2:].contiguous().view(torch.int8).to(dtype)
    else:
        off, at = (16, 6) if name == "Q5_0" else (8, 2)
        u = torch.cat([blk[..., at:] & 15, blk[..., at:] >> 4], -1)
        if name == "Q5_0":
            sh = torch.arange(8, device=b.device, dtype=torch.uint8)
            b5 = (blk[..., 2:6, None] >> sh) & 1
            u = u | (b5.reshape(*b5.shape[:-2], 32) << 4)
        q = u.to(dtype) - off
    return (q * d).reshape(*b.shape[:-1], -1)


# ---------------------------------------------------------------- prepare --

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(case)
    if case["op"] == "plan":
        have, start, want = _resizes(case)
        page = case["page"]
        held = [-(-h // page) for h in have]
        grown = sum(max(0, -(-w // page) - p) for w, p in zip(want, held))
        given = sum(max(0, p - -(-w // page)) for w, p in zip(want, held))
        spare = max(0, int(grown * 0.8) - given) if case["scarce"] else grown + 10
        order = rng.permutation(sum(held) + spare + 7).astype(np.int32)
        table = np.full((case["n_req"], case["pages"]), -1, np.int32)
        at = 0
        for i, p in enumerate(held):
            table[i, :p] = order[at:at + p]
            at += p
        free = np.full(order.size, -1, np.int32)
        free[:spare] = order[at:at + spare]
        total = sum(max(0, w - b) for w, b in zip(want, start))
        s.update(have=i32(have), start=i32(start), want=i32(want), table=torch.from_numpy(table).to(dev),
                 free=torch.from_numpy(free).to(dev), n_free=i32([spare]), cap=(total + 64) // 64 * 64)
        return s
    if case["op"] == "append":
        n_req, n, n_kv, d, page = (case[k] for k in ("n_req", "n", "n_kv", "d", "page"))
        width = 2 * n_kv * d + case["gap"]
        rows = torch.randn((n_req * n, width), device=dev, generator=g)
        rows *= torch.exp(0.8 * torch.randn((n_req * n, 1), device=dev, generator=g))
        rows = rows.to(torch.bfloat16 if case["act"] == "bf16" else torch.float32)
        k = rows[:, :n_kv * d].unflatten(1, (n_kv, d))
        v = rows[:, width - n_kv * d:].unflatten(1, (n_kv, d))
        base = [random.Random(case["mix"] + i).randint(0, 3 * page) for i in range(n_req)]
        P = max(-(-(b + n) // page) for b in base)
        n_pages = n_req * P + 2
        table = torch.from_numpy(rng.permutation(n_pages)[:n_req * P].astype(np.int32).reshape(n_req, P)).to(dev)
        pos = torch.tensor(base, device=dev)[:, None] + torch.arange(n, device=dev)
        slots = (torch.gather(table.long(), 1, pos // page) * page + pos % page).reshape(-1)
        pb = n_kv * page * d // 32 * BLOCK[case["type"]]
        s.update(k=k, v=v, slots=slots, table=table, K=torch.zeros((n_pages, pb), dtype=torch.uint8, device=dev),
                 V=torch.zeros((n_pages, pb), dtype=torch.uint8, device=dev), n_pages=n_pages)
        if case["compact"]:
            r = random.Random(int(seed))
            path, used = [], []
            for _ in range(n_req):
                m = r.randint(0, n)
                path.append(sorted(r.sample(range(n), m)) + [0] * (n - m))
                used.append(m)
            s.update(base=i32(base), path=i32(path), n_path=i32(used))
        return s
    if case["op"] == "tree":
        ctx, n = _lengths(case)
        heads, n_kv, d, page = (case[k] for k in ("heads", "n_kv", "d", "page"))
        held = [-(-(c + m) // page) for c, m in zip(ctx, n)]
        P, n_pages = max(held), sum(held) + 3
        order = rng.permutation(n_pages).astype(np.int32)
        table = np.full((case["n_req"], P), -1, np.int32)
        at = 0
        for i, p in enumerate(held):
            table[i, :p] = order[at:at + p]
            at += p
        chan = torch.exp(0.5 * torch.randn((n_kv, 1, d), device=dev, generator=g))
        pools = []
        for c in (chan, None):
            pool = torch.empty((n_pages, n_kv * page * d // 32 * BLOCK[case["type"]]), dtype=torch.uint8, device=dev)
            step = max(1, (1 << 26) // (n_kv * page * d))
            for a in range(0, n_pages, step):
                x = torch.randn((min(step, n_pages - a), n_kv, page, d), device=dev, generator=g)
                pool[a:a + step] = _pack(case["type"], x if c is None else x * c).reshape(x.shape[0], -1)
            pools.append(pool)
        r = random.Random(int(seed))
        bits = [b for m in n for b in _tree(r, m)]
        cu = np.concatenate([[0], np.cumsum(n)])
        q = torch.randn((int(cu[-1]), heads, d), device=dev, generator=g).to(torch.bfloat16)
        s.update(K=pools[0], V=pools[1], table=torch.from_numpy(table).to(dev), ctx=i32(ctx), cu=i32(cu.tolist()), q=q,
                 mask=torch.tensor(_signed(bits), dtype=torch.int64, device=dev), max_q=max(n), scale=1.0 / math.sqrt(d))
        return s
    n_req, n, V = case["n_req"], case["n"], case["vocab"]
    rows = n_req * n
    logits = (3.0 * torch.randn((rows, V), device=dev, generator=g)).to(torch.bfloat16 if case["act"] == "bf16" else torch.float32)
    # Texts repeat themselves: token ids by a power law.
    zipf = lambda shape: torch.from_numpy(np.minimum((V * rng.random(shape) ** 4).astype(np.int64), V - 1).astype(np.int32)).to(dev)  # noqa: E731
    r = random.Random(int(seed))
    used = [r.randint(max(1, case["hist"] // 2), case["hist"]) for _ in range(n_req)]
    nb = case["n_bias"]
    s.update(logits=logits, cu=torch.arange(n_req + 1, dtype=torch.int32, device=dev) * n, hist=zipf((n_req, case["hist"])),
             hist_len=i32(used), draft=zipf((rows,)),
             mask=torch.tensor(_signed([b for _ in range(n_req) for b in _tree(r, n)]), dtype=torch.int64, device=dev),
             rep=1.0 + 0.3 * torch.rand(n_req, device=dev, generator=g), pres=0.5 * torch.rand(n_req, device=dev, generator=g),
             freq=0.2 * torch.rand(n_req, device=dev, generator=g),
             bias_tok=torch.stack([torch.randperm(V, device=dev, generator=g)[:nb] for _ in range(n_req)]).to(torch.int32) if nb else None,
             bias_val=4.0 * torch.randn((n_req, nb), device=dev, generator=g) if nb else None,
             bias_len=i32([r.randint(0, nb) for _ in range(n_req)]) if nb else None,
             grammar=torch.randint(-2**31, 2**31, (rows, -(-V // 32)), device=dev, generator=g, dtype=torch.int64).to(torch.int32)
             if case["grammar"] else None)
    return s


# -------------------------------------------------------------------- run --

def run(s):
    if s["op"] == "plan":
        return _plan_own(s) if own else _plan_plain(s)
    if s["op"] == "append":
        return _append_own(s) if own else _append_plain(s)
    if s["op"] == "tree":
        if own:
            qk = _qk()
            return qk.attn_tree(qk.TYPES[s["type"]], s["q"], s["K"], s["V"], s["page"], s["n_kv"], s["table"], s["ctx"], s["cu"],
                                s["mask"], s["max_q"], s["scale"])
        return _tree_plain(s)
    if own:
        return _qk().logits_process(s["logits"], s["cu"], s["hist"], s["hist_len"], s["rep"], s["pres"], s["freq"],
                                    draft=s["draft"], mask=s["mask"], bias_tok=s["bias_tok"], bias_val=s["bias_val"],
                                    bias_len=s["bias_len"], grammar=s["grammar"])
    return _logits_plain(s)


def _plan_own(s):
    p = _qk().kv_plan(s["have"], s["start"], s["want"], s["table"], s["free"], s["n_free"], s["page"], s["cap"])
    return {"table": s["table"], "free": s["free"], **p}


def _plan_plain(s):
    have, start, want, page = s["have"].long(), s["start"].long(), s["want"].long(), s["page"]
    table, free, n_free = s["table"].clone(), s["free"].clone(), s["n_free"].long()
    old, new = (have + page - 1) // page, (want + page - 1) // page
    grow, shrink = (new - old).clamp(min=0), (old - new).clamp(min=0)
    col = torch.arange(table.shape[1], device=table.device)
    freed = table[(col >= new[:, None]) & (col < old[:, None])]
    stack = torch.cat([free, freed])
    avail = n_free + shrink.sum()
    upto = grow.cumsum(0)
    granted = (grow == 0) | (upto <= avail)
    more = (col >= old[:, None]) & (col < new[:, None]) & granted[:, None]
    at = avail - 1 - ((upto - grow)[:, None] + col - old[:, None])      # place in the stack: free pages, then freed ones
    at = torch.where(at < n_free, at, at - n_free + free.numel())
    table[more] = stack[at[more]]
    taken = torch.where(granted & (grow > 0), upto, torch.zeros_like(upto)).max()
    left = torch.arange(freed.numel(), device=table.device) < shrink.sum() - taken
    free[(n_free + torch.arange(freed.numel(), device=table.device))[left]] = freed[left]
    n = (want - start).clamp(min=0)
    cu = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
    i = torch.arange(s["cap"], device=table.device)
    live = i < cu[-1]
    req = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=n.numel() - 1)
    pos = start[req] + i - cu[req]
    slot = table[req, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    none = torch.full_like(i, -1)
    return {"table": table, "free": free, "n_free": (avail - taken).int(), "cu": cu.int(), "granted": granted.int(),
            "slots": torch.where(live & granted[req], slot, none), "pos": torch.where(live, pos, none).int(),
            "req": torch.where(live, req, none).int()}


def _append_own(s):
    qk = _qk()
    t, n_kv, d, page = qk.TYPES[s["type"]], s["n_kv"], s["d"], s["page"]
    qk.kv_append(t, s["k"], s["v"], s["slots"], s["K"], s["V"], page)
    if s["compact"]:
        qk.kv_compact(t, s["K"], s["V"], page, n_kv, d, s["table"], s["base"], s["path"], s["n_path"])
    rows = s["n_pages"] * n_kv * page
    return {"K": qk.dequant(t, s["K"], rows, d), "V": qk.dequant(t, s["V"], rows, d)}


def _append_plain(s):
    n_kv, d, page = s["n_kv"], s["d"], s["page"]
    out = {}
    for name, x in (("K", s["k"]), ("V", s["v"])):
        values = _unpack(s["type"], _pack(s["type"], x.float()))
        pool = torch.zeros((s["n_pages"], page, n_kv, d), device=x.device)
        pool[s["slots"] // page, s["slots"] % page] = values
        if s["compact"]:
            j = torch.arange(s["path"].shape[1], device=x.device)
            live = j < s["n_path"][:, None]
            to, fro = s["base"][:, None].long() + j, s["base"][:, None].long() + s["path"]
            P = s["table"].shape[1]
            page_of = lambda p: torch.gather(s["table"].long(), 1, (p // page).clamp(max=P - 1))  # noqa: E731
            moved = pool[page_of(fro), fro % page]
            pool[page_of(to)[live], (to % page)[live]] = moved[live]
        out[name] = pool.transpose(1, 2).reshape(-1, d)
    return out


def _tree_plain(s):
    heads, n_kv, d, page, m = s["heads"], s["n_kv"], s["d"], s["page"], s["max_q"]
    dev, G = s["q"].device, s["heads"] // s["n_kv"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    n = cu[1:] - cu[:-1]
    pages = s["table"].long().clamp(min=0)

    def cached(pool):   # [requests, kv heads, positions, d]
        x = pool.reshape(pool.shape[0], n_kv, page, -1)[pages]
        return _unpack(s["type"], x.transpose(1, 2).flatten(2, 3))

    tok = (cu[:-1, None] + torch.arange(m, device=dev)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[tok].reshape(-1, m, n_kv, G, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (q @ cached(s["K"]).transpose(-1, -2) * s["scale"]).unflatten(2, (G, m))
    at = torch.arange(score.shape[-1], device=dev)[None] - ctx[:, None]
    drafted = (at >= 0) & (at < n[:, None])
    bit = (s["mask"][tok][:, :, None] >> at.clamp(0, 63)[:, None]) & 1
    seen = ((at < 0)[:, None] | (drafted[:, None] & (bit == 1)))[:, None, None]
    top = score.masked_fill(~seen, -math.inf).amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top).masked_fill(~seen, 0.0)
    total = p.sum(-1, keepdim=True)
    o = (p / torch.where(total > 0, total, torch.ones_like(total))).flatten(2, 3) @ cached(s["V"])
    o = o.unflatten(2, (G, m)).permute(0, 3, 1, 2, 4).reshape(-1, m, heads, d)
    return o[torch.arange(m, device=dev) < n[:, None]].to(torch.bfloat16)


def _logits_plain(s):
    x = s["logits"].float()
    rows, V = x.shape
    dev, n_req = x.device, s["cu"].numel() - 1
    cu = s["cu"].long()
    req = torch.repeat_interleave(torch.arange(n_req, device=dev), cu[1:] - cu[:-1])
    h = torch.arange(s["hist"].shape[1], device=dev) < s["hist_len"][:, None]
    count = torch.zeros((n_req, V), device=dev)
    count.scatter_add_(1, s["hist"].long(), h.float())
    count = count[req]
    j = torch.arange(rows, device=dev)[None] - cu[req][:, None]          # another row's index within this row's request
    inside = (req[None] == req[:, None]) & (((s["mask"][:, None] >> j.clamp(0, 63)) & 1) == 1)
    count.scatter_add_(1, s["draft"].long()[None].expand(rows, rows), inside.float())
    rep, pres, freq = (s[k][req][:, None] for k in ("rep", "pres", "freq"))
    y = torch.where(count > 0, torch.where(x > 0, x / rep, x * rep) - freq * count - pres, x)
    if s["bias_tok"] is not None:
        b = torch.arange(s["bias_tok"].shape[1], device=dev) < s["bias_len"][:, None]
        add = torch.zeros((n_req, V), device=dev)
        add.scatter_add_(1, s["bias_tok"].long(), s["bias_val"] * b)
        y = y + add[req]
    if s["grammar"] is not None:
        v = torch.arange(V, device=dev)
        y = y.masked_fill(((s["grammar"][:, v // 32] >> (v % 32).int()) & 1) == 0, -math.inf)
    return y.to(s["logits"].dtype)


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "plan":
        have, start, want = _resizes(case)
        page = case["page"]
        moved = sum(abs(-(-w // page) - -(-h // page)) for w, h in zip(want, have))
        total = sum(max(0, w - b) for w, b in zip(want, start))
        # three lengths in, two numbers out per request; a page id in and out per page that changes hands; a page id
        # in per page of new positions; slot, position and request out per token
        return {"bytes": 20 * case["n_req"] + 8 * moved + 4 * (total // page + case["n_req"]) + 16 * total, "flops": 0}
    if case["op"] == "append":
        n = case["n_req"] * case["n"]
        vals = 2 * n * case["n_kv"] * case["d"]
        packed = vals // 32 * BLOCK[case["type"]]
        pages = case["n_req"] * -(-(case["n"] + 3 * case["page"]) // case["page"])
        pool = 2 * pages * case["page"] * case["n_kv"] * case["d"]
        # rows in, blocks out; then (the values handed back) every block in and every value out
        return {"bytes": vals * (2 if case["act"] == "bf16" else 4) + packed + (packed if case["compact"] else 0)
                + pool // 32 * BLOCK[case["type"]] + 4 * pool, "flops": 4 * vals}
    if case["op"] == "tree":
        ctx, n = _lengths(case)
        row = case["n_kv"] * case["d"] // 32 * BLOCK[case["type"]]
        cache = sum(c + m for c, m in zip(ctx, n)) * row * 2
        q = sum(n) * case["heads"] * case["d"]
        return {"bytes": cache + 4 * q, "flops": sum(4 * m * (c + m / 2) for c, m in zip(ctx, n)) * case["heads"] * case["d"]}
    rows = case["n_req"] * case["n"]
    el = 2 if case["act"] == "bf16" else 4
    return {"bytes": rows * case["vocab"] * 2 * el + (rows * case["vocab"] // 8 if case["grammar"] else 0)
            + 4 * case["n_req"] * case["hist"], "flops": 0}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The definitions in 64 bits, request by request."""
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None          # whole numbers only
    if case["op"] == "append":
        return _append_exact(s)
    if case["op"] == "tree":
        return _tree_exact(s)
    return _logits_exact(s)


def _append_exact(s):
    # The quantized values by the definition: d the half-precision max |x| /
    # levels, the code the nearest whole number to x / d (halves away from 0).
    lo, hi = {"Q8_0": (-128, 127), "Q5_0": (-16, 15), "Q4_0": (-8, 7)}[s["type"]]
    out = {}
    for name, x in (("K", s["k"]), ("V", s["v"])):
        x = x.cpu().double().numpy()
        g = x.reshape(-1, 32)
        top = np.abs(g).max(1).astype(np.float32) / np.float32(LEVELS[s["type"]])
        d = top.astype(np.float16).astype(np.float64)[:, None]
        ratio = np.divide(g, d, out=np.zeros_like(g), where=d != 0).astype(np.float32).astype(np.float64)
        code = np.clip(np.copysign(np.floor(np.abs(ratio) + 0.5), ratio), lo, hi)
        values = (code * d).reshape(x.shape)
        pool = np.zeros((s["n_pages"], s["n_kv"], s["page"], s["d"]))
        slots = s["slots"].cpu().numpy()
        for i, at in enumerate(slots):
            pool[at // s["page"], :, at % s["page"]] = values[i]
        if s["compact"]:
            table, base, path, used = (s[k].cpu().numpy() for k in ("table", "base", "path", "n_path"))
            for r in range(len(base)):
                where = lambda p: (table[r, p // s["page"]], slice(None), p % s["page"])  # noqa: E731
                rows = [pool[where(base[r] + path[r, j])].copy() for j in range(used[r])]
                for j, row in enumerate(rows):
                    pool[where(base[r] + j)] = row
        out[name] = pool.reshape(-1, s["d"])
    return out


def _tree_exact(s):
    G = s["heads"] // s["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    rb = s["d"] // 32 * BLOCK[s["type"]]
    for r in range(len(ctx)):
        n, T = cu[r + 1] - cu[r], ctx[r] + cu[r + 1] - cu[r]
        ids = s["table"][r, :-(-T // s["page"])].long()
        see = torch.ones((n, T), dtype=torch.bool, device=out.device)
        for i, b in enumerate(s["mask"][cu[r]:cu[r + 1]].tolist()):
            see[i, ctx[r]:] = torch.tensor([(b >> j) & 1 == 1 for j in range(n)])
        for h in range(s["n_kv"]):
            K, V = (_unpack(s["type"], s[k].view(-1, s["n_kv"], s["page"], rb)[ids, h].reshape(-1, rb)[:T], torch.float64) for k in "KV")
            q = s["q"][cu[r]:cu[r + 1], h * G:(h + 1) * G].double()
            a = torch.einsum("ngd,td->gnt", q, K) * s["scale"]
            a = torch.softmax(a.masked_fill(~see, -math.inf), -1).nan_to_num(0.0)
            out[cu[r]:cu[r + 1], h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", a, V)
    return out


def _logits_exact(s):
    x = s["logits"].double()
    cu = s["cu"].tolist()
    V = x.shape[1]
    for r in range(len(cu) - 1):
        seen = torch.bincount(s["hist"][r, :int(s["hist_len"][r])].long(), minlength=V)
        rep, pres, freq = (float(s[k][r]) for k in ("rep", "pres", "freq"))
        for i in range(cu[r], cu[r + 1]):
            c = seen.clone()
            b = int(s["mask"][i])
            for j in range(cu[r + 1] - cu[r]):
                if (b >> j) & 1:
                    c[int(s["draft"][cu[r] + j])] += 1
            y = x[i]
            z = torch.where(y > 0, y / rep, y * rep) - (pres + freq * c.double())
            y = torch.where(c > 0, z, y)
            if s["bias_tok"] is not None:
                m = int(s["bias_len"][r])
                y[s["bias_tok"][r, :m].long()] += s["bias_val"][r, :m].double()
            if s["grammar"] is not None:
                words = s["grammar"][i].cpu().numpy().view(np.uint8)
                ok = np.unpackbits(words, bitorder="little")[:V]
                y = torch.where(torch.from_numpy(ok.astype(bool)).to(y.device), y, torch.full_like(y, -math.inf))
            x[i] = y
    return x
