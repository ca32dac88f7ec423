"""Workloads of the operators around the paged cache and the packed weights, for timing and for comparing results.

A decode or verification step of a model takes, besides the products over
packed weights and the attention over the cache:

  norm_rope        RMS norms of every query and key head with the position
                   rotation in the same pass, rows in and rows out
  kv_append_rope   the same on the way into the paged cache: keys normed,
                   rotated and quantized into their pages, values quantized,
                   queries handed on in bf16
  moe_ffn          a mixture-of-experts layer over packed expert weights for a
                   few tokens: router, the chosen experts' gated products, and
                   their weighted sum
  verify_tree      the drafted trees judged against the target's
                   probabilities, from given random numbers: the accepted
                   path, its tokens and the token after them

A case is a dict of plain values.  `own` chooses between the plain torch form
and the package's calls.  Head layouts, cache types, page sizes, vocabularies
and the 4096 x 14336 products are those of the package's own benchmark and
tests; expert counts and the narrower experts are generic.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

TREE_MAX = 64                                     # drafted tokens of one request, at most
CACHE = {"Q8_0": 127.0, "Q5_0": 15.0, "Q4_0": 7.0}    # the cache's block types: largest code
# (bytes of a block, weights of a block, where its half-precision scales are, standard deviation of a random block's weights
# over its scale; the types with a second scale, the minimum's, take it as that many times the first)
FORMAT = {"Q4_K": (144, 256, 0, 2, 257.0, 7.5), "Q6_K": (210, 256, 208, None, 1366.0, 0), "Q8_0": (34, 32, 0, None, 74.0, 0),
          "Q5_0": (22, 32, 0, None, 9.2, 0), "Q4_0": (18, 32, 0, None, 4.6, 0), "Q5_K": (176, 256, 0, 2, 530.0, 15.5),
          "Q2_K": (84, 256, 80, 82, 13.9, 1.5), "Q3_K": (110, 256, 108, None, 43.0, 0)}


def _qk():
    import gguf_quant_dequant_gb300 as qk
    return qk


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # One decoded token of a single user whose cache is not paged: queries
        # and keys come back as rows.  Only the latency of the call counts.
        dict(op="rope", name="rope_one", n=1, heads=32, n_kv=8, d=128, rot=128, act="f32", out="f32", norm=True, pairs=False,
             far=1000, gap=0, mix=1),
        # A prefill chunk at far positions, 256-wide heads of which a part turns.
        dict(op="rope", name="rope_far_chunk", n=4099, heads=12, n_kv=4, d=256, rot=64, act="bf16", out="bf16", norm=True,
             pairs=True, far=1000000, gap=320, mix=2),
        # One drafted tree of a single user, straight into the pages.
        dict(op="append", name="append_rope_tree", type="Q8_0", n_req=1, n=13, heads=32, n_kv=8, d=128, rot=128, act="f32",
             norm=True, pairs=False, far=32000, gap=0, page=16, mix=3),
        # The drafted trees of a batch, slices of a fused projection's output.
        dict(op="append", name="append_rope_batch", type="Q5_0", n_req=61, n=29, heads=32, n_kv=8, d=64, rot=64, act="bf16",
             norm=False, pairs=True, far=15000, gap=128, page=64, mix=4),
        # Long prompts of several requests.
        dict(op="append", name="append_rope_prompt", type="Q4_0", n_req=4, n=8191, heads=32, n_kv=8, d=128, rot=128, act="bf16",
             norm=True, pairs=False, far=0, gap=0, page=32, mix=5),
        # A chain of drafts of one user, picked without probabilities.
        dict(op="verify", name="verify_one", n_req=1, n=6, chain=True, vocab=32000, act="f32", drafter=False, mix=6),
        # A server's batch of chains with the drafter's probabilities.
        dict(op="verify", name="verify_batch", n_req=48, n=8, chain=True, vocab=128256, act="f32", drafter=True, mix=7),
        # Wide trees of a few requests.
        dict(op="verify", name="verify_trees", n_req=7, n=64, chain=False, vocab=128256, act="bf16", drafter=False, mix=8),
        # One token through many narrow experts: the shortest layer.
        dict(op="moe", name="moe_one", n=1, experts=128, k=8, cols=2048, rows=768, up="Q4_K", down="Q6_K", norm=True, mix=9),
        # A drafted tree's tokens through the same experts: nearly all are met.
        dict(op="moe", name="moe_tree", n=61, experts=128, k=8, cols=2048, rows=768, up="Q4_K", down="Q6_K", norm=True, mix=10),
        # One token through two of eight wide experts.
        dict(op="moe", name="moe_wide_one", n=1, experts=8, k=2, cols=4096, rows=14336, up="Q4_K", down="Q4_K", norm=True,
             mix=11),
        # A small batch through the wide experts.
        dict(op="moe", name="moe_wide_batch", n=13, experts=8, k=2, cols=4096, rows=14336, up="Q4_K", down="Q6_K", norm=False,
             mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8, 128), (32, 4, 128), (8, 8, 128), (32, 8, 64), (8, 1, 64), (6, 2, 32), (12, 4, 256), (8, 2, 256)]


def draw(rng):
    op = rng.choice(["rope", "append", "append", "verify", "verify", "moe", "moe", "moe"])
    mix = rng.randrange(1 << 20)
    if op in ("rope", "append"):
        heads, n_kv, d = rng.choice(HEADS)
        case = dict(op=op, heads=heads, n_kv=n_kv, d=d, rot=rng.choice([d, d, d // 2]), act=rng.choice(["f32", "bf16"]),
                    norm=rng.random() < 0.5, pairs=rng.random() < 0.5, far=rng.choice([0, 5000, 1000000]),
                    gap=rng.choice([0, 0, 96, 320]), mix=mix)
        if op == "rope":
            return dict(case, n=_log(rng, 1, 4099), out=rng.choice(["f32", "bf16"]))
        few = rng.random() < 0.6
        n_req = _log(rng, 1, 61) if few else _log(rng, 1, 4)
        return dict(case, type=rng.choice(list(CACHE)), n_req=n_req, n=_log(rng, 1, TREE_MAX if few else 8191 * 4096 // max(4096, heads * d)),
                    page=rng.choice([16, 32, 64, 128, 256]))
    if op == "verify":
        vocab = rng.choice([_log(rng, 1000, 128256), 32000, 32003, 50257, 128256])
        n_req = _log(rng, 1, 48)
        return dict(op=op, n_req=n_req, n=_log(rng, 1, max(1, min(TREE_MAX, 384 // n_req))), chain=rng.random() < 0.5, vocab=vocab,
                    act=rng.choice(["f32", "f32", "bf16"]), drafter=rng.random() < 0.5, mix=mix)
    up, down = rng.choice(list(FORMAT)), rng.choice(list(FORMAT))
    step = lambda t: FORMAT[t][1]  # noqa: E731
    experts = rng.choice([2, 8, 16, 60, 64, 128, 256])
    k = min(experts, rng.choice([1, 2, 4, 6, 8]))
    cols = _log(rng, 512 // step(up), 4096 // step(up)) * step(up)
    most = min(14336, 6 * 4096 * 14336 // (experts * cols))
    rows = _log(rng, 1, max(1, most // step(down))) * step(down)
    return dict(op=op, n=_log(rng, 1, min(61, 13 * 2 * 8 * 14336 // (k * experts) // 64 + 1)), experts=experts, k=k, cols=cols, rows=rows,
                up=up, down=down, norm=rng.random() < 0.7, mix=mix)


def _tree(r, n, chain):
    """Ancestor bits (own bit included) and parents of n nodes, each node's parent before it."""
    bits, parents = [], []
    for i in range(n):
        p = (i - 1 if chain else r.randint(max(0, i - 6), i - 1)) if i else -1
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
        parents.append(p)
    return bits, parents


def _signed(bits):
    return [b - (1 << 64) if b >> 63 else b for b in bits]


# ---------------------------------------------------------------- prepare --

def _positions(case, rng):
    """Positions of the tokens: prompts count up from 0, drafted tokens sit behind texts of up to `far` positions."""
    base = rng.integers(0, case["far"] + 1, case.get("n_req", 1))
    if case["n"] <= TREE_MAX and case["op"] == "append":
        depth = [0]
        for i in range(1, case["n"]):
            depth.append(depth[int(rng.integers(max(0, i - 6), i))] + 1)
    else:
        depth = list(range(case["n"]))
    return (base[:, None] + np.array(depth)).reshape(-1).astype(np.int32)


def _blocks(name, rows, cols, dev, g):
    """Random blocks of weights of about 1 / sqrt(cols), [rows, bytes of a row]."""
    size, elems, at, at_min, spread, ratio = FORMAT[name]
    n = rows * cols // elems
    w = torch.randint(0, 256, (n, size), dtype=torch.uint8, device=dev, generator=g)
    d = torch.exp(0.3 * torch.randn((n, 1), device=dev, generator=g)) / (spread * math.sqrt(cols))
    if name in ("Q6_K", "Q8_0", "Q3_K"):
        d = torch.where(torch.rand((n, 1), device=dev, generator=g) < 0.5, -d, d)
    w[:, at:at + 2] = d.to(torch.float16).view(torch.uint8)
    if at_min is not None:
        w[:, at_min:at_min + 2] = (ratio * d).to(torch.float16).view(torch.uint8)
    return w.view(rows, -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rng = np.random.default_rng([int(seed), case["mix"]])
    i32 = lambda v: torch.as_tensor(np.asarray(v, np.int32)).to(dev)  # noqa: E731
    s = dict(case)
    if case["op"] in ("rope", "append"):
        heads, n_kv, d, rot = (case[k] for k in ("heads", "n_kv", "d", "rot"))
        n = case["n"] * case.get("n_req", 1)
        width = (heads + 2 * n_kv) * d + case["gap"]
        x = torch.randn((n, width), device=dev, generator=g)
        x *= torch.exp(0.5 * torch.randn((1, width), device=dev, generator=g))
        x = x.to(torch.bfloat16 if case["act"] == "bf16" else torch.float32)
        part = lambda a, h: x[:, a * d:(a + h) * d].unflatten(1, (h, d))  # noqa: E731
        weight = lambda: 1.0 + 0.2 * torch.randn(d, device=dev, generator=g) if case["norm"] else None  # noqa: E731
        # Inverse frequencies of the usual base, the far half stretched as long-context models do.
        freq = 500000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        freq[rot // 4:] /= 8.0
        s.update(q=part(0, heads), k=part(heads, n_kv), v=part(heads + n_kv, n_kv), pos=i32(_positions(case, rng)), q_norm=weight(),
                 k_norm=weight(), freq=freq.float(), eps=1e-6)
        if case["op"] == "append":
            n_req, page = case["n_req"], case["page"]
            base = np.random.default_rng(case["mix"]).integers(0, 3 * page + 1, n_req)     # what the requests hold already
            P = int(max(-(-(b + case["n"]) // page) for b in base))
            n_pages = n_req * P + 2
            table = rng.permutation(n_pages)[:n_req * P].reshape(n_req, P)
            at = base[:, None] + np.arange(case["n"])
            slots = np.take_along_axis(table, at // page, 1) * page + at % page
            size = n_kv * page * d // 32 * FORMAT[case["type"]][0]
            s.update(slots=torch.from_numpy(slots.reshape(-1).astype(np.int64)).to(dev), n_pages=n_pages,
                     K=torch.zeros((n_pages, size), dtype=torch.uint8, device=dev),
                     V=torch.zeros((n_pages, size), dtype=torch.uint8, device=dev))
        return s
    if case["op"] == "verify":
        n_req, n, V = case["n_req"], case["n"], case["vocab"]
        rows = n_req * n
        r = random.Random(int(seed) * 1000003 + case["mix"])
        trees = [_tree(r, n, case["chain"]) for _ in range(n_req)]
        parent = torch.tensor([p for _, t in trees for p in t], device=dev)
        above = torch.arange(rows, device=dev) // n * n + parent.clamp(min=0)       # the parent's row
        logits = 3.0 * torch.randn((rows, V), device=dev, generator=g)
        probs = None
        if case["drafter"]:     # the drafter is near the target, and its tokens come from its own probabilities
            probs = torch.softmax(logits + 0.4 * torch.randn((rows, V), device=dev, generator=g), -1)
            draft = torch.multinomial(probs[above], 1, generator=g)[:, 0]
        else:                   # the target gives most drafted tokens a good part of its mass
            draft = torch.from_numpy(np.minimum((V * rng.random(rows) ** 4).astype(np.int64), V - 1)).to(dev)
            kids = torch.zeros(rows, device=dev).index_add_(0, above, (parent >= 0).float())
            lift = torch.logsumexp(logits, -1) + 1.0 - torch.log(kids.clamp(min=1.0))
            put = torch.where(parent >= 0, lift[above], logits[above, draft])
            logits[above, draft] = put
        temp = 0.5 + 0.75 * torch.rand(n_req, device=dev, generator=g)
        temp[torch.arange(n_req, device=dev) % 5 == 3] = 0.0          # some requests decode greedily
        u = lambda k: torch.rand(k, device=dev, generator=g)  # noqa: E731
        s.update(logits=logits.to(torch.bfloat16 if case["act"] == "bf16" else torch.float32), probs=probs,
                 draft=draft.to(torch.int32), cu=i32(np.arange(n_req + 1) * n),
                 mask=torch.tensor(_signed([b for t, _ in trees for b in t]), dtype=torch.int64, device=dev), temp=temp,
                 u_accept=u(rows), u_sample=u(n_req), max_path=n)
        return s
    n, E, k, cols, rows = (case[key] for key in ("n", "experts", "k", "cols", "rows"))
    x = torch.randn((n, cols), device=dev, generator=g) * torch.exp(0.4 * torch.randn(cols, device=dev, generator=g))
    s.update(x=x, router=torch.randn((E, cols), device=dev, generator=g) / math.sqrt(cols),
             gate_w=_blocks(case["up"], E * rows, cols, dev, g), up_w=_blocks(case["up"], E * rows, cols, dev, g),
             down_w=_blocks(case["down"], E * cols, rows, dev, g), scale=1.0 if case["norm"] else 2.5)
    return s


# -------------------------------------------------------------------- run --

def run(s):
    return {"rope": _rope_own if own else _rope_plain, "append": _append_own if own else _append_plain,
            "verify": _verify_own if own else _verify_plain, "moe": _moe_own if own else _moe_plain}[s["op"]](s)


def _rope_own(s):
    q, k = _qk().norm_rope(s["q"], s["k"], s["pos"], s["freq"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"],
                           pairs=s["pairs"], out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)
    return {"q": q, "k": k}


def _append_own(s):
    qk = _qk()
    t = qk.TYPES[s["type"]]
    q = qk.kv_append_rope(t, s["q"], s["k"], s["v"], s["pos"], s["freq"], s["slots"], s["K"], s["V"], s["page"], q_norm=s["q_norm"],
                          k_norm=s["k_norm"], eps=s["eps"], pairs=s["pairs"])
    rows = s["n_pages"] * s["n_kv"] * s["page"]
    return {"q": q, "K": qk.dequant(t, s["K"], rows, s["d"]), "V": qk.dequant(t, s["V"], rows, s["d"])}


def _verify_own(s):
    return _qk().verify_tree(s["logits"], s["cu"], s["draft"], s["mask"], s["temp"], s["u_accept"], s["u_sample"], probs=s["probs"],
                        max_path=s["max_path"])


def _moe_own(s):
    qk = _qk()
    out, ids, gate = qk.moe_ffn(qk.TYPES[s["up"]], s["gate_w"], s["up_w"], qk.TYPES[s["down"]], s["down_w"], s["experts"], s["rows"],
                            s["cols"], s["x"], s["k"], router=s["router"], norm=s["norm"], scale=s["scale"])
    return {"out": out, "ids": ids, "gate": gate}


# --------------------------------------------------- norm and rotation -----

def _turned(x, w, s):
    """fp32 [n, heads, d]: normed by pairwise sums (so that the value is the same wherever it is computed), then turned by
    angles taken in 64 bits."""
    x = x.float()
    if w is not None:
        square = functools.reduce(lambda t, _: t[..., 0::2] + t[..., 1::2], range(int(math.log2(s["d"]))), x * x)
        x = x * (1.0 / torch.sqrt(square / s["d"] + s["eps"])) * w
    angle = s["pos"].double()[:, None] * s["freq"].double()
    c, z, rot = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None], s["rot"]
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if s["pairs"] else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * z
    y[..., b] = x[..., b] * c + x[..., a] * z
    return y


def _rope_plain(s):
    dtype = torch.bfloat16 if s["out"] == "bf16" else torch.float32
    return {"q": _turned(s["q"], s["q_norm"], s).to(dtype), "k": _turned(s["k"], s["k_norm"], s).to(dtype)}


def _stored(name, x):
    """The values that fp32 [..., 32 m] has after quantization: d = fp16(max|x| / levels), code = round half away (x / d)."""
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    d = (top / torch.full_like(top, CACHE[name])).to(torch.float16).float()     # a true division: no reciprocal of a scalar
    q = torch.where(d != 0, g / torch.where(d != 0, d, torch.ones_like(d)), torch.zeros_like(g))
    a = torch.floor(q.abs())
    q = torch.sign(q) * (a + (q.abs() - a >= 0.5))
    top = 128 if name == "Q8_0" else int(CACHE[name]) + 1
    return (q.clamp(-top, top - 1) * d).flatten(-2)


def _append_plain(s):
    out = {"q": _turned(s["q"], s["q_norm"], s).to(torch.bfloat16)}
    for name, x in (("K", _turned(s["k"], s["k_norm"], s)), ("V", s["v"].float())):
        pool = torch.zeros((s["n_pages"], s["page"], s["n_kv"], s["d"]), device=x.device)
        pool[s["slots"] // s["page"], s["slots"] % s["page"]] = _stored(s["type"], x)
        out[name] = pool.transpose(1, 2).reshape(-1, s["d"])
    return out


# ------------------------------------------------------- verification ------

def _verify_plain(s):
    """A token's weight at a row is exp((x - max) / T) in 32 bits; sums of weights, and what is compared with a random
    number, are in 64.  All requests walk at once, node by node."""
    x, V, dev = s["logits"].float(), s["vocab"], s["logits"].device
    n_req, n = s["cu"].numel() - 1, s["n"]
    first = s["cu"][:-1].long()
    top = x.amax(-1, keepdim=True)
    greedy = s["temp"] < 2.0**-20
    rate = 1.0 / torch.where(greedy, torch.ones_like(s["temp"]), s["temp"])
    at, every = torch.arange(V, device=dev), torch.arange(n_req, device=dev)
    node = torch.arange(n, device=dev)
    below = (1 << node.long()) - 1
    parent = torch.where(node > 0, ((s["mask"].view(n_req, n, 1) & below[:, None]) >> node & 1).mul(node + 1).amax(-1) - 1, -1)
    length = torch.ones(n_req, dtype=torch.long, device=dev)
    path = torch.full((n_req, s["max_path"]), -1, dtype=torch.long, device=dev)
    path[:, 0] = 0

    def weights(cur):       # a row's weights, or for greedy requests all of it on the first largest
        row = first + cur
        e = torch.exp((x[row] - top[row]) * rate[:, None])
        best = torch.where(x[row] == top[row], at, V).amin(-1)
        return torch.where(greedy[:, None], (at == best[:, None]).float(), e)

    cur = torch.zeros(n_req, dtype=torch.long, device=dev)
    base = weights(cur)
    w, total = base, base.double().sum(-1)
    used = torch.zeros(n_req, dtype=torch.float64, device=dev)     # the drafter's mass taken off by rejections, in units of w
    for i in range(1, n):
        tried = parent[:, i] == cur
        token = s["draft"][first + i].long()
        mine = w[every, token].double()
        price = s["u_accept"][first + i].double()
        if s["probs"] is not None:
            q = s["probs"][first + cur]
            price = torch.where(greedy, price, price * q[every, token].double())
        ok = tried & (price * total < mine)
        no = tried & ~ok
        if s["probs"] is not None:
            used = torch.where(no, used + total, used)
            less = (base - used.float()[:, None] * q).clamp(min=0.0)
            less = torch.where(greedy[:, None], torch.where(at == token[:, None], torch.zeros_like(w), w), less)
        else:
            less = torch.where(at == token[:, None], torch.zeros_like(w), w)
        w = torch.where(no[:, None], less, w)
        cur = torch.where(ok, i, cur)
        path[every, torch.where(ok, length, length - 1)] = cur
        length = length + ok
        base = torch.where(ok[:, None], weights(cur), base)
        w = torch.where(ok[:, None], base, w)
        used = torch.where(ok, 0.0, used)
        total = w.double().sum(-1)
    w = torch.where((total > 0)[:, None], w, base)
    upto = w.double().cumsum(-1)
    last = (s["u_sample"].double()[:, None] * upto[:, -1:] >= upto).sum(-1).clamp(max=V - 1)
    path = torch.where(torch.arange(s["max_path"], device=dev) < length[:, None], path, -1)
    tokens = torch.where(path > 0, s["draft"][(first[:, None] + path).clamp(min=0)].long(), -1).roll(-1, 1)
    tokens[every, length - 1] = last
    return {"path": path.int(), "n_path": length.int(), "tokens": tokens.int()}


# ------------------------------------------------------ packed weights -----

def _half(b):
    return b.contiguous().view(torch.float16).float()


def _unpack(name, b):
    """Packed bytes [..., row bytes] -> fp32 weights [..., cols]."""
    blk = b.unflatten(-1, (-1, FORMAT[name][0]))
    cut = lambda a, z: blk[..., a:z].int()  # noqa: E731
    if name in ("Q8_0", "Q5_0", "Q4_0"):
        d = _half(blk[..., :2])
        if name == "Q8_0":
            return (d * blk[..., 2:].contiguous().view(torch.int8).float()).flatten(-2)
        c = cut(6 if name == "Q5_0" else 2, None)
        u = torch.cat([c & 15, c >> 4], -1)
        if name == "Q5_0":
            u = u | (((cut(2, 6)[..., None] >> torch.arange(8, device=b.device)) & 1).flatten(-2) << 4)
        return (d * (u - (16 if name == "Q5_0" else 8)).float()).flatten(-2)
    even = torch.arange(0, 8, 2, device=b.device)
    if name in ("Q4_K", "Q5_K"):
        f = cut(4, 16).unflatten(-1, (3, 4))
        sc = torch.cat([f[..., 0, :] & 63, (f[..., 2, :] & 15) | (f[..., 0, :] >> 6 << 4)], -1)
        mn = torch.cat([f[..., 1, :] & 63, (f[..., 2, :] >> 4) | (f[..., 1, :] >> 6 << 4)], -1)
        c = cut(16 if name == "Q4_K" else 48, None).unflatten(-1, (4, 32))
        u = torch.stack([c & 15, c >> 4], -2)
        if name == "Q5_K":
            high = (cut(16, 48)[..., None, :] >> torch.arange(8, device=b.device)[:, None]) & 1
            u = u | (high.unflatten(-2, (4, 2)) << 4)
        u = u.flatten(-3, -2).float()
        d, m = _half(blk[..., :2]), _half(blk[..., 2:4])
        return ((d * sc)[..., None] * u - (m * mn)[..., None]).flatten(-3)
    if name == "Q6_K":
        low = cut(0, 128).unflatten(-1, (2, 2, 32))
        low = torch.cat([low & 15, low >> 4], -2)
        high = (cut(128, 192).unflatten(-1, (2, 1, 32)) >> even[:, None]) & 3
        u = (low | (high << 4)).flatten(-3).unflatten(-1, (16, 16)) - 32
        sc = _half(blk[..., 208:210]) * blk[..., 192:208].contiguous().view(torch.int8).float()
        return (sc[..., None] * u.float()).flatten(-3)
    at = 16 if name == "Q2_K" else 32
    u = ((cut(at, at + 64).unflatten(-1, (2, 1, 32)) >> even[:, None]) & 3).flatten(-3, -2)
    if name == "Q2_K":
        sm = cut(0, 16)
        sc, mn = _half(blk[..., 80:82]) * (sm & 15), _half(blk[..., 82:84]) * (sm >> 4)
        return (sc[..., None] * u.flatten(-2).unflatten(-1, (16, 16)).float() - mn[..., None]).flatten(-3)
    bit = (cut(0, 32)[..., None, :] >> torch.arange(8, device=b.device)[:, None]) & 1
    f, h = cut(96, 104), cut(104, 108)
    sc = (torch.cat([f & 15, f >> 4], -1) | (((h[..., None, :] >> even[:, None]) & 3).flatten(-2) << 4)) - 32
    sc = _half(blk[..., 108:110]) * sc
    return (sc[..., None] * (u + 4 * bit - 4).flatten(-2).unflatten(-1, (16, 16)).float()).flatten(-3)


# ------------------------------------------------------------- experts -----

def _moe_plain(s):
    x, E, k, rows, cols, n = (s[key] for key in ("x", "experts", "k", "rows", "cols", "n"))
    logits = x.double() @ s["router"].double().T          # in 64 bits: the choice is made between near values
    order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids, p = order.indices[:, :k], torch.softmax(order.values, -1)[:, :k]
    gate = (p / p.sum(-1, keepdim=True) if s["norm"] else p) * s["scale"]
    met, which = torch.unique(ids, return_inverse=True)
    take = lambda name, w, r: _unpack(name, w.view(E, r, -1)[met])  # noqa: E731
    h = torch.nn.functional.silu(take(s["up"], s["gate_w"], rows) @ x.T) * (take(s["up"], s["up_w"], rows) @ x.T)
    share = torch.zeros((met.numel(), n), device=x.device).index_put_((which, torch.arange(n, device=x.device)[:, None]), gate.float())
    y = take(s["down"], s["down_w"], cols) @ torch.where(share[:, None] > 0, h, torch.zeros_like(h))
    return {"out": (y * share[:, None]).sum(0).T.contiguous(), "ids": ids.int(), "gate": gate.float()}


# ------------------------------------------------------------------- work --

def _wide(act):
    return 2 if act == "bf16" else 4


def work(case):
    if case["op"] in ("rope", "append"):
        n = case["n"] * case.get("n_req", 1)
        q, k = n * case["heads"] * case["d"], n * case["n_kv"] * case["d"]
        if case["op"] == "rope":
            return {"bytes": (q + k) * (_wide(case["act"]) + _wide(case["out"])) + 4 * n, "flops": 10 * (q + k)}
        size = FORMAT[case["type"]][0]
        pages = case["n_req"] * -(-(case["n"] + 3 * case["page"]) // case["page"])
        pool = 2 * pages * case["page"] * case["n_kv"] * case["d"]
        # rows in, queries and blocks out; then (the values handed back) every block in and every value out
        return {"bytes": (q + 2 * k) * _wide(case["act"]) + 2 * q + 2 * k // 32 * size + 12 * n + pool // 32 * size + 4 * pool,
                "flops": 10 * (q + 2 * k)}
    if case["op"] == "verify":
        # the rows of a path on which three of four tries succeed, and the drafter's row where it ends
        reach = min(case["n"], (1 - 0.75 ** case["n"]) / 0.25)
        return {"bytes": case["n_req"] * case["vocab"] * (reach * _wide(case["act"]) + (4 if case["drafter"] else 0)),
                "flops": 4 * case["n_req"] * case["vocab"] * reach}
    n, E, k, cols, rows = (case[key] for key in ("n", "experts", "k", "cols", "rows"))
    met = E * (1 - (1 - k / E) ** n)
    size = lambda t: FORMAT[t][0] / FORMAT[t][1]  # noqa: E731
    return {"bytes": met * rows * cols * (2 * size(case["up"]) + size(case["down"])) + 4 * E * cols + 8 * n * cols + 8 * n * k,
            "flops": 6 * n * k * rows * cols + 2 * n * E * cols}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "verify":
        return None          # whole numbers only
    return {"rope": _rope_exact, "append": _append_exact, "moe": _moe_exact}[case["op"]](s)


def _turned_exact(x, w, s):
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + np.float32(s["eps"]).astype(np.float64)).sqrt() * w.double()
    head, tail = y[..., :s["rot"]], y[..., s["rot"]:]
    z = head.unflatten(-1, (-1, 2)) if s["pairs"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turn = torch.polar(torch.ones(1, 1, dtype=torch.float64, device=y.device), s["pos"].double()[:, None] * s["freq"].double()[None])
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None])
    return torch.cat([z.flatten(-2) if s["pairs"] else z.transpose(-1, -2).flatten(-2), tail], -1)


def _turned_stepwise(x, w, s):
    """The values that are quantized: by the operator's definition each square, sum (by neighbours, then by neighbouring
    sums), quotient, root, product, cosine and sine is rounded to 32 bits, and the bytes follow from them."""
    step = lambda t: t.float().double()  # noqa: E731
    y = x.double()
    if w is not None:
        total = step(y * y)
        while total.shape[-1] > 1:
            total = step(total.unflatten(-1, (-1, 2)).sum(-1))
        root = step(step(step(total / s["d"]) + float(np.float32(s["eps"]))).sqrt())
        y = step(step(y * step(1.0 / root)) * w.double())
    head, tail = y[..., :s["rot"]], y[..., s["rot"]:]
    z = head.unflatten(-1, (-1, 2)) if s["pairs"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turn = torch.polar(torch.ones(1, 1, dtype=torch.float64, device=y.device), s["pos"].double()[:, None] * s["freq"].double()[None])
    c, d = step(turn.real)[:, None], step(turn.imag)[:, None]
    z = torch.stack([step(step(z[..., 0] * c) - step(z[..., 1] * d)), step(step(z[..., 1] * c) + step(z[..., 0] * d))], -1)
    return torch.cat([z.flatten(-2) if s["pairs"] else z.transpose(-1, -2).flatten(-2), tail], -1)


def _rope_exact(s):
    return {"q": _turned_exact(s["q"], s["q_norm"], s), "k": _turned_exact(s["k"], s["k_norm"], s)}


def _append_exact(s):
    lo, hi = {"Q8_0": (-128, 127), "Q5_0": (-16, 15), "Q4_0": (-8, 7)}[s["type"]]
    out = {"q": _turned_exact(s["q"], s["q_norm"], s)}
    page, off = s["slots"] // s["page"], s["slots"] % s["page"]
    for name, x in (("K", _turned_stepwise(s["k"], s["k_norm"], s)), ("V", s["v"].double())):
        g = x.reshape(-1, 32)
        d = (g.abs().max(1, keepdim=True).values / hi).float().half().double()
        ratio = torch.nan_to_num((g / d).float().double(), 0.0, 0.0, 0.0)
        code = torch.copysign((ratio.abs() + 0.5).floor(), ratio).clip(lo, hi)
        pool = torch.zeros((s["n_pages"], s["n_kv"], s["page"], s["d"]), dtype=torch.float64, device=x.device)
        head = torch.arange(s["n_kv"], device=x.device)
        pool[page[:, None], head[None], off[:, None]] = (code * d).view(x.shape)
        out[name] = pool.view(-1, s["d"])
    return out


@functools.lru_cache(maxsize=None)
def _places(name):
    """Where weight i of a block keeps its bits: (byte, shift, mask) of the low ones, (byte, shift, mask, by how much they go
    up) of the high ones, the code of weight zero, and the group of its scale."""
    i = np.arange(FORMAT[name][1])
    z = np.zeros_like(i)
    if name in ("Q8_0", "Q5_0", "Q4_0"):
        if name == "Q8_0":
            return 2 + i, z, 255, z, z, 0, 0, 0, z
        at = 6 if name == "Q5_0" else 2
        return (at + i % 16, i // 16 * 4, 15, 2 + i // 8 if name == "Q5_0" else z, i % 8, 1 if name == "Q5_0" else 0, 4,
                16 if name == "Q5_0" else 8, z)
    l, t, g = i % 32, i // 128, i // 32 % 4
    if name in ("Q4_K", "Q5_K"):
        c, h = i // 64, i // 32 % 2
        return (16 if name == "Q4_K" else 48) + 32 * c + l, 4 * h, 15, 16 + l, 2 * c + h, 0 if name == "Q4_K" else 1, 4, 0, i // 32
    if name == "Q6_K":
        return 64 * t + 32 * (g & 1) + l, g // 2 * 4, 15, 128 + 32 * t + l, 2 * g, 3, 4, 32, i // 16
    if name == "Q2_K":
        return 16 + 32 * t + l, 2 * g, 3, z, z, 0, 0, 0, i // 16
    return 32 + 32 * t + l, 2 * g, 3, l, 4 * t + g, 1, 2, 4, i // 16


def _weights64(name, w):
    """[rows, row bytes] -> fp64 [rows, cols], by the table of places."""
    size, elems, at, at_min = FORMAT[name][:4]
    byte, shift, mask, hbyte, hshift, hmask, up, zero, group = _places(name)
    b = w.reshape(-1, size).to(torch.int16)
    t = lambda v: torch.as_tensor(np.asarray(v)).to(w.device)  # noqa: E731
    code = (b[:, t(byte)] >> t(shift).to(torch.int16)) & mask
    if hmask:
        code = code | (((b[:, t(hbyte)] >> t(hshift).to(torch.int16)) & hmask) << up)
    code = code.double() - zero
    if name == "Q8_0":
        code = torch.where(code > 127, code - 256, code)
    real = lambda a: w.reshape(-1, size)[:, a:a + 2].contiguous().view(torch.float16).double()  # noqa: E731
    j = np.arange(8 if name in ("Q4_K", "Q5_K") else 16)
    low = 0.0
    if name in ("Q4_K", "Q5_K"):
        s0, s4, s8 = (b[:, t(a + j % 4)] for a in (4, 8, 12))
        late = t(j >= 4)
        sc = torch.where(late, (s8 & 15) + (s0 >> 6) * 16, s0 & 63).double()
        low = real(at_min) * torch.where(late, (s8 >> 4) + (s4 >> 6) * 16, s4 & 63).double()
    elif name == "Q2_K":
        sc, low = (b[:, t(j)] & 15).double(), real(at_min) * (b[:, t(j)] >> 4).double()
    elif name == "Q3_K":
        sc = (((b[:, t(96 + j % 8)] >> t(j // 8 * 4).to(torch.int16)) & 15) +
              ((b[:, t(104 + j % 4)] >> t(j // 4 * 2).to(torch.int16)) & 3) * 16 - 32).double()
    elif name == "Q6_K":
        sc = b[:, t(192 + j)].double()
        sc = torch.where(sc > 127, sc - 256, sc)
    else:
        sc = torch.ones((b.shape[0], 1), dtype=torch.float64, device=w.device)
    g = t(group)
    value = (real(at) * sc)[:, g] * code
    if at_min is not None:
        value = value - low[:, g]
    return value.view(w.shape[0], -1)


def _moe_exact(s):
    x, E, rows, cols = s["x"].double(), s["experts"], s["rows"], s["cols"]
    score = x @ s["router"].double().T
    top = torch.topk(score, s["k"], -1)
    share = torch.exp(top.values - (torch.logsumexp(top.values, -1) if s["norm"] else torch.logsumexp(score, -1))[:, None]) * s["scale"]
    out = torch.zeros_like(x)
    for e in torch.unique(top.indices).tolist():
        tok, j = torch.where(top.indices == e)
        g = x[tok] @ _weights64(s["up"], s["gate_w"][e * rows:(e + 1) * rows]).T
        u = x[tok] @ _weights64(s["up"], s["up_w"][e * rows:(e + 1) * rows]).T
        y = (g / (1 + torch.exp(-g)) * u) @ _weights64(s["down"], s["down_w"][e * cols:(e + 1) * cols]).T
        out.index_add_(0, tok, y * share[tok, j][:, None])
    return {"out": out, "ids": None, "gate": share}
