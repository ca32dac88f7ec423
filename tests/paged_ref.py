"""Plain 64-bit (and whole-number) implementations of the paged KV-cache,
tree-attention and logits calls, one request at a time, for their tests."""
from __future__ import annotations

import numpy as np

import gguf_quant_dequant_gb300 as qk
import oracle
import synth


def pool(name: str, n_pages: int, n_kv: int, page: int, d: int, seed: int, **kw) -> np.ndarray:
    """Random blocks [n_pages, n_kv, page, row bytes]."""
    b = synth.random_blocks(name, n_pages * n_kv * page, d, seed, **kw)
    return np.ascontiguousarray(b, dtype=np.uint8).reshape(n_pages, n_kv, page, -1)


def values(name: str, rows: np.ndarray, d: int) -> np.ndarray:
    """[..., row bytes] -> fp64 [..., d]."""
    flat = np.ascontiguousarray(rows).reshape(-1, rows.shape[-1])
    w = oracle.dequant(synth.TYPE_IDS[name], flat.reshape(-1), flat.shape[0], d)
    return np.asarray(w, np.float64).reshape(*rows.shape[:-1], d)


def plan(have, start, want, table, free_pages, n_free, page, cap):
    """qk_kv_plan, sequentially; table and free_pages are changed in place."""
    n, stride = len(have), table.shape[1]
    up = lambda x: -(-x // page)  # noqa: E731
    valid = [h >= 0 and w >= 0 and s >= 0 and up(h) <= stride and up(w) <= stride for h, s, w in zip(have, start, want)]
    stack = list(free_pages[:n_free])
    for r in range(n):
        if valid[r]:
            stack += list(table[r, up(want[r]):up(have[r])])
    before = list(stack)
    avail, asked = len(stack), 0
    granted = []
    for r in range(n):
        grow = max(0, up(want[r]) - up(have[r])) if valid[r] else 0
        asked += grow
        ok = valid[r] and (grow == 0 or asked <= avail)
        granted.append(int(ok))
        if ok:
            for c in range(up(have[r]), up(want[r])):
                table[r, c] = stack.pop()
    for i in range(n_free, len(stack)):
        if i < len(free_pages):
            free_pages[i] = before[i]
    cu, slots, pos, req = [0], [], [], []
    for r in range(n):
        for p in range(start[r], want[r] if valid[r] else start[r]):
            slots.append(int(table[r, p // page]) * page + p % page if granted[r] else -1)
            pos.append(p)
            req.append(r)
        cu.append(len(slots))
    fill = lambda v: (v + [-1] * cap)[:cap]  # noqa: E731
    return {"n_free": [len(stack)], "granted": granted, "cu": cu, "slots": fill(slots), "pos": fill(pos), "req": fill(req)}


def visible(mask, n: int, i: int):
    bits = [j <= i for j in range(n)] if mask is None else [(int(mask[i]) >> j) & 1 == 1 for j in range(n)]
    return np.array(bits, bool)


def attn_tree(name, q, K, V, page, n_kv, table, ctx, cu, mask, max_q, scale):
    """q fp64 [n_tok, heads, d]; K, V byte pools [n_pages, n_kv, page, row
    bytes]; mask uint64 or None.  Returns (out, sum p|V|, max_t |scale| sum
    |q k|, sum |V| of the visible); out is NaN in rows that no request has."""
    n_tok, heads, d = q.shape
    G = heads // n_kv
    out, Sv, V1 = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros(q.shape)
    A = np.zeros((n_tok, heads))
    for r in range(len(ctx)):
        n = min(int(cu[r + 1] - cu[r]), max_q)
        T = int(ctx[r]) + n
        p = np.arange(T)
        ids = table[r][p // page] if T else np.zeros(0, int)
        for g in range(n_kv):
            k, v = (values(name, x[ids, g, p % page], d) if T else np.zeros((0, d)) for x in (K, V))
            for i in range(n):
                tok = cu[r] + i
                see = np.ones(T, bool)
                see[int(ctx[r]):] = visible(None if mask is None else mask[cu[r]:cu[r + 1]], n, i)
                for h in range(g * G, (g + 1) * G):
                    if not see.any():
                        out[tok, h] = 0.0
                        continue
                    s = k[see] @ q[tok, h] * scale
                    A[tok, h] = np.max(np.abs(k[see]) @ np.abs(q[tok, h])) * abs(scale)
                    e = np.exp(s - s.max())
                    w = e / e.sum()
                    out[tok, h] = w @ v[see]
                    Sv[tok, h] = w @ np.abs(v[see])
                    V1[tok, h] = np.abs(v[see]).sum(0)
    return out, Sv, A, V1


def logits(x, cu, hist, hist_len, rep, pres, freq, draft=None, mask=None, bias_tok=None, bias_val=None, bias_len=None,
           grammar=None):
    """fp64 [n_rows, vocab] and the magnitude of the terms each value is a sum of."""
    y = np.array(x, np.float64)
    size = np.abs(y)
    n_rows, V = y.shape
    for r in range(len(cu) - 1):
        for row in range(cu[r], cu[r + 1]):
            c = np.zeros(V)
            toks = list(hist[r][:max(int(hist_len[r]), 0)])
            if draft is not None:
                see = visible(None if mask is None else mask[cu[r]:cu[r + 1]], cu[r + 1] - cu[r], row - cu[r]) \
                    if mask is None or cu[r + 1] - cu[r] <= 64 else [(int(mask[row]) >> j) & 1 for j in range(64)]
                toks += [draft[cu[r] + j] for j, s in enumerate(see) if s]
            for t in toks:
                if 0 <= t < V:
                    c[t] += 1
            hit = c > 0
            with np.errstate(invalid="ignore", over="ignore"):
                z = np.where(y[row] > 0, y[row] / float(rep[r]), y[row] * float(rep[r]))
                z = np.where(np.abs(z) > np.finfo(np.float32).max, np.copysign(np.inf, z), z)   # fp32 arithmetic overflows
                size[row] = np.where(hit, np.abs(z) + abs(float(freq[r])) * c + abs(float(pres[r])), size[row])
                y[row] = np.where(hit, z - float(freq[r]) * c - float(pres[r]), y[row])
            if bias_tok is not None:
                m = max(int(bias_len[r]), 0)
                last = {int(t): float(b) for t, b in zip(bias_tok[r][:m], bias_val[r][:m])}
                for t, b in last.items():
                    if 0 <= t < V:
                        y[row, t] += b
                        size[row, t] += abs(b)
    if grammar is not None:
        v = np.arange(V)
        ok = (grammar[:, v // 32].astype(np.int64) >> (v % 32)) & 1
        y = np.where(ok == 1, y, -np.inf)
    return y, size
