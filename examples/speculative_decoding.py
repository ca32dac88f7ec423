"""Speculative decoding of several requests over the paged, block-quantized KV
cache: the calls of a server's step, run together.

    python examples/speculative_decoding.py [--steps 12] [--requests 3]

A small decoder with random Q8_0 weights stands in for the model.  Each step
verifies one tree of drafted tokens per request in one pass:
  kv_plan         pages and slots for the drafted tokens (and pages back),
  gemm            the projections over the packed weights,
  kv_append       the tokens' K and V rows, quantized into their pages,
  attn_tree       every token attends to the committed positions and to its
                  ancestors in the tree,
  logits_process  repetition penalties over the request's text and the
                  token's own ancestors, and a mask of forbidden tokens,
  kv_compact      the rows of the accepted path moved together.
The greedy choice at each accepted node is the text; the drafts only decide how
many tokens a step yields.  main() checks that against decoding the same
requests one token at a time.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gguf_quant_dequant_gb300 as qk  # noqa: E402

T = qk.Q8_0
HIDDEN, HEADS, N_KV, D, VOCAB, LAYERS, PAGE = 256, 8, 2, 64, 1000, 2, 16


class Model:
    def __init__(self, seed: int, dev):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        w = lambda rows, cols, s: qk.quantize(T, s * torch.randn((rows, cols), device=dev, generator=g))  # noqa: E731
        self.qkv = [w((HEADS + 2 * N_KV) * D, HIDDEN, 0.12) for _ in range(LAYERS)]
        self.o = [w(HIDDEN, HEADS * D, 0.08) for _ in range(LAYERS)]
        self.head = w(VOCAB, HIDDEN, 0.3)
        self.embed = torch.randn((VOCAB, HIDDEN), device=dev, generator=g)
        self.place = 0.3 * torch.randn((512, HIDDEN), device=dev, generator=g)


class Server:
    """Requests, their pages and texts.  text[r] ends with a token that is not
    in the cache yet: the root of the request's next tree."""

    def __init__(self, model: Model, prompts, pages: int, dev):
        self.m, self.dev, n = model, dev, len(prompts)
        self.text = [list(p) for p in prompts]
        self.K, self.V = ([torch.zeros((pages, qk.kv_page_bytes(T, N_KV, D, PAGE)), dtype=torch.uint8, device=dev)
                           for _ in range(LAYERS)] for _ in range(2))
        self.table = torch.full((n, 16), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(pages, dtype=torch.int32, device=dev)
        self.n_free = self.i32([pages])
        self.have, self.len = [0] * n, [0] * n      # positions with pages, committed positions
        f = lambda v: torch.full((n,), v, device=dev)  # noqa: E731
        self.rep, self.pres, self.freq = f(1.1), f(0.1), f(0.05)
        allowed = torch.ones(-(-VOCAB // 32) * 32, dtype=torch.int64)
        allowed[7::50] = 0                            # tokens that a grammar forbids
        words = (allowed.view(-1, 32) << torch.arange(32)).sum(1)
        self.grammar = (words - ((words >> 31) << 32)).to(torch.int32).to(dev)
        for r in range(n):                            # prompts: a chain of tokens, 64 at a time
            while self.len[r] < len(self.text[r]) - 1:
                a = self.len[r]
                chain = self.text[r][a:min(a + qk.TREE_MAX, len(self.text[r]) - 1)]
                drafts = [(chain, list(range(-1, len(chain) - 1))) if i == r else ([], []) for i in range(n)]
                self.verify(drafts, keep=[len(chain) if i == r else 0 for i in range(n)])

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.dev)

    def verify(self, drafts, keep=None):
        """drafts[r]: (tokens, parents) of request r's tree, parents before
        children.  Keeps the path of the greedy choices (or the first keep[r]
        tokens of a prompt) and returns, per request, the accepted nodes and
        the token chosen after each node."""
        n, m = len(drafts), self.m
        tokens, bits, place, sizes = [], [], [], [len(t) for t, _ in drafts]
        for r, (toks, parents) in enumerate(drafts):
            own, depth = [], []
            for i, p in enumerate(parents):
                own.append((own[p] if p >= 0 else 0) | (1 << i))
                depth.append(depth[p] + 1 if p >= 0 else 0)
            tokens += toks
            bits += [b - (1 << 64) if b >> 63 else b for b in own]
            place += [self.len[r] + k for k in depth]
        total, start = len(tokens), self.i32(self.len)
        want = [a + s for a, s in zip(self.len, sizes)]
        plan = qk.kv_plan(self.i32(self.have), start, self.i32(want), self.table, self.free, self.n_free, PAGE, total)
        self.n_free, self.have = plan["n_free"], want
        mask = torch.tensor(bits, dtype=torch.int64, device=self.dev)
        toks = torch.tensor(tokens, device=self.dev)
        x = m.embed[toks] + m.place[torch.tensor(place, device=self.dev)]
        norm = lambda v: (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)  # noqa: E731
        for i in range(LAYERS):
            h = qk.gemm(T, m.qkv[i], (HEADS + 2 * N_KV) * D, HIDDEN, norm(x)).view(total, HEADS + 2 * N_KV, D)
            q = h[:, :HEADS].to(torch.bfloat16)
            qk.kv_append(T, h[:, HEADS:HEADS + N_KV], h[:, HEADS + N_KV:], plan["slots"], self.K[i], self.V[i], PAGE)
            a = qk.attn_tree(T, q, self.K[i], self.V[i], PAGE, N_KV, self.table, start, plan["cu"], mask, max(sizes), D ** -0.5)
            x = x + qk.gemm(T, m.o[i], HIDDEN, HEADS * D, a.view(total, HEADS * D))
        logits = qk.gemm(T, m.head, VOCAB, HIDDEN, norm(x))
        past = [t[:k] for t, k in zip(self.text, self.len)]      # the trees hold the rest
        hist = torch.zeros((n, max(1, max(map(len, past)))), dtype=torch.int32)
        for r, t in enumerate(past):
            hist[r, :len(t)] = torch.tensor(t, dtype=torch.int32)
        qk.logits_process(logits, plan["cu"], hist.to(self.dev), self.i32([len(t) for t in past]), self.rep, self.pres, self.freq,
                          draft=toks.to(torch.int32), mask=mask, grammar=self.grammar.expand(total, -1).contiguous(), out=logits)
        best, at = logits.argmax(-1).tolist(), 0
        paths, choices = [], []
        for r, (t, parents) in enumerate(drafts):
            mine = best[at:at + sizes[r]]
            at += sizes[r]
            path = list(range(keep[r])) if keep else []
            node = 0 if t and not keep else None
            while node is not None:                  # the child that carries the token chosen at the node
                path.append(node)
                node = next((i for i, p in enumerate(parents) if p == node and t[i] == mine[node]), None)
            paths.append(path)
            choices.append(mine)
        most = max(1, max(map(len, paths)))
        p = self.i32([q + [0] * (most - len(q)) for q in paths])
        for i in range(LAYERS):
            qk.kv_compact(T, self.K[i], self.V[i], PAGE, N_KV, D, self.table, start, p, self.i32([len(q) for q in paths]))
        for r, q in enumerate(paths):
            self.len[r] += len(q)
            if not keep:
                self.text[r] += [choices[r][i] for i in q]
        return paths, choices


def drafted_tree(text, guess, rng):
    """A tree under the text's last token: the guessed continuation with a
    wrong sibling at every level, and a wrong branch of two."""
    tokens, parents, node = [text[-1]], [-1], 0
    for g in guess:
        tokens += [int(torch.randint(VOCAB, (1,), generator=rng)), g]
        parents += [node, node]
        node = len(tokens) - 1
    tokens += [int(torch.randint(VOCAB, (1,), generator=rng)) for _ in range(2)]
    parents += [0, len(tokens) - 2]
    return tokens, parents


def main(steps: int = 12, requests: int = 3, seed: int = 1) -> dict:
    dev = torch.device("cuda")
    model, rng = Model(seed, dev), torch.Generator()
    rng.manual_seed(seed)
    prompts = [torch.randint(VOCAB, (20 + 41 * r,), generator=rng).tolist() for r in range(requests)]
    plain = Server(model, prompts, 16 * requests, dev)
    for _ in range(steps):                            # a tree of one node is ordinary decoding
        plain.verify([([t[-1]], [-1]) for t in plain.text])
    fast, passes = Server(model, prompts, 16 * requests, dev), 0
    while min(len(t) - len(p) for t, p in zip(fast.text, prompts)) < steps:
        trees = []
        for r, t in enumerate(fast.text):
            right = plain.text[r][len(t):len(t) + 3]  # a drafter that is right three times, then wrong
            trees.append(drafted_tree(t, right + [int(torch.randint(VOCAB, (1,), generator=rng))], rng))
        fast.verify(trees)
        passes += 1
    qk.device_status()
    same = [sum(a == b for a, b in zip(f[len(p):], s[len(p):])) for f, s, p in zip(fast.text, plain.text, prompts)]
    return {"steps": steps, "passes": passes, "equal": same, "texts": [t[len(p):len(p) + steps] for t, p in zip(fast.text, prompts)]}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--requests", type=int, default=3)
    a = ap.parse_args()
    got = main(a.steps, a.requests)
    print(f"{got['steps']} tokens for each of {a.requests} requests in {got['passes']} passes; equal to one-by-one decoding: "
          f"{got['equal']} of {got['steps']}")
