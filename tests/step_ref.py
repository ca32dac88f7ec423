"""Plain 64-bit (and stepwise fp32) implementations of the head norms and
rotation, and a replay of tree verification, for their tests."""
from __future__ import annotations

import numpy as np


def angles(pos, freq):
    """(cos, sin) fp64 [n, rot / 2], good to 2^-50 for every int32 position: the position in two parts whose products with
    a 24-bit frequency are exact in 53 bits, and the addition formula."""
    p, f = np.asarray(pos, np.int64), np.asarray(freq, np.float64)[None]
    a, b = ((p >> 16) << 16).astype(np.float64)[:, None] * f, (p & 0xFFFF).astype(np.float64)[:, None] * f
    return np.cos(a) * np.cos(b) - np.sin(a) * np.sin(b), np.sin(a) * np.cos(b) + np.cos(a) * np.sin(b)


def _split(y, rot, pairs):
    return (y[..., 0:rot:2], y[..., 1:rot:2]) if pairs else (y[..., :rot // 2], y[..., rot // 2:rot])


def turned(x, pos, freq, w, eps, pairs):
    """fp64 result for x [n, heads, d], and the magnitude |y_p cos| + |y_q sin| of each value's terms."""
    y = np.asarray(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps))) * np.asarray(w, np.float64)
    out, size = y.copy(), np.abs(y)
    if len(freq):
        rot = 2 * len(freq)
        c, s = (t[:, None] for t in angles(pos, freq))
        a, b = _split(y, rot, pairs)
        oa, ob = _split(out, rot, pairs)
        sa, sb = _split(size, rot, pairs)
        oa[...], ob[...] = a * c - b * s, b * c + a * s
        sa[...], sb[...] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return out, size


def turned_stepwise(x, pos, freq, w, eps, pairs):
    """The same with every operation rounded to fp32, as include/qk.h states it."""
    f = np.float32
    y = np.asarray(x, f)
    if w is not None:
        t = y * y
        while t.shape[-1] > 1:
            t = t[..., 0::2] + t[..., 1::2]
        y = y * (f(1) / np.sqrt(t / f(y.shape[-1]) + f(eps))) * np.asarray(w, f)
    out = y.copy()
    if len(freq):
        c, s = (t[:, None].astype(f) for t in angles(pos, freq))
        a, b = _split(y, 2 * len(freq), pairs)
        oa, ob = _split(out, 2 * len(freq), pairs)
        oa[...], ob[...] = a * c - b * s, b * c + a * s
    return out


# ---------------------------------------------------------- verification --

# A weight exp((x - top) / T) in fp32: the difference is exact to 2^-24 on both sides alike, the reciprocal of T and the
# product round alike, and the two exp differ by at most 4 units of 2^-24; sums are in 64 bits.  So weights, their sums
# and products with given numbers are 2^-21 off at most, and a decision that is nearer than that may fall either way.
SLACK = 2.0**-20


def weights(x, temp):
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float32)).astype(np.float32)
    top = x.max()
    if top == -np.inf:
        return np.zeros(len(x))
    if top == np.inf:
        return (x == np.inf).astype(np.float64)
    rate = np.float32(1) / np.float32(temp)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp(((x - top) * rate).astype(np.float32)).astype(np.float64)
    return np.where(x == -np.inf, 0.0, e)


def parents(n, mask):
    if mask is None:
        return list(range(-1, n - 1))
    up = [int(m) & ((1 << i) - 1) for i, m in enumerate(mask[:n])]
    return [u.bit_length() - 1 for u in up]


def replay(logits, draft, mask, temp, u_accept, u_sample, probs, stride, path, n_path, tokens):
    """Checks one request's answer against the rule, decision by decision (rows of that request only; mask as unsigned)."""
    n = min(len(draft), 64)
    if n == 0:
        assert n_path == 0 and (path == -1).all() and (tokens == -1).all()
        return
    assert 1 <= n_path <= min(n, stride)
    assert path[0] == 0 and (path[n_path:] == -1).all() and (tokens[n_path:] == -1).all()
    par, V = parents(n, mask), logits.shape[1]
    greedy = not temp >= 2.0**-20
    for at in range(n_path):
        cur = int(path[at])
        nxt = int(path[at + 1]) if at + 1 < n_path else None
        kids = [i for i in range(cur + 1, n) if par[i] == cur] if at + 1 < stride else []
        if nxt is not None:
            assert nxt in kids and tokens[at] == draft[nxt]
        x = np.where(np.isnan(logits[cur]), -np.inf, logits[cur])
        if greedy:
            best = int(np.argmax(x)) if x.max() > -np.inf else -1
            want = next((i for i in kids if draft[i] == best), None)
            assert nxt == want
            if nxt is None:
                assert tokens[at] == best
            continue
        e = weights(x, temp)
        q = None if probs is None else probs[cur].astype(np.float64)
        w, tau, slack = e.copy(), 0.0, SLACK * e
        for c in kids:
            y = int(draft[c])
            inside = 0 <= y < V
            price = float(u_accept[c]) * (q[y] if q is not None and inside else 1.0) * w.sum()
            mine, near = (w[y], slack[y]) if inside else (0.0, 0.0)
            if c == nxt:
                assert price < mine + near + SLACK * price, (c, price, mine)
                break
            assert price >= mine - near - SLACK * price - SLACK * slack.sum() * float(u_accept[c]) or mine == 0.0, (c, price, mine)
            if q is None:
                if inside:
                    w[y] = slack[y] = 0.0
            else:
                tau += w.sum()
                w = np.maximum(e - tau * q, 0.0)
                slack = SLACK * (e + tau * q)
        if nxt is None:
            if not w.sum() > 0.0:
                w, slack = e, SLACK * e
            t = int(tokens[at])
            if not e.sum() > 0.0:
                assert t == -1
                return
            total = w.sum()
            if total <= slack.sum():       # what is left is rounding: any token of the row, or of what is left
                assert 0 <= t < V and e[t] > 0
                return
            target = float(u_sample) * total
            upto = w.cumsum()
            off = slack.cumsum()[t] + float(u_sample) * slack.sum() + SLACK * total
            assert 0 <= t < V and w[t] + slack[t] > 0
            assert upto[t] - w[t] - off <= target <= upto[t] + off, (t, target, upto[t] - w[t], upto[t])
