"""The expert layer against the oracle: the router's choice, and the products
of the chosen experts within a bound that follows from each product's.

A product of a row w = ds q - dm (Q6_K: q in 0 .. 63, dm = 32 ds) with x is within
e = 2^-17 sum (|ds q| + |dm|) |x| + 1e-6: x as two fp16 terms is 2^-22 off, the fp32 sums have one rounding
(or, inside an MMA, truncation) per 16 weights, block and slice of at most 2^6
blocks, up to 2^7 of 2^-24 together.  |SiLU'| <= 1.1, so h = SiLU(g) u is within
eh = 1.1 eg (|u| + eu) + |SiLU(g)| eu + 2^-20 |h|, the down product of h within
its own e and sum |w| eh; the gates' error and the fp32 sum over k experts add
(k + 24) 2^-24 of the terms' magnitude."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import oracle
import synth
from gpu_helpers import dev_f32, dev_u8, gpu, type_id  # noqa: F401

pytestmark = pytest.mark.gpu


def layer(seed, E, rows, cols, up, down):
    kw = dict(d_scale=2e-4, dmin_scale=1e-3) if up in ("Q4_K", "Q5_K") else {}
    kd = dict(d_scale=2e-4, dmin_scale=1e-3) if down in ("Q4_K", "Q5_K") else {}
    return (synth.random_blocks(up, E * rows, cols, seed, **kw), synth.random_blocks(up, E * rows, cols, seed + 1, **kw),
            synth.random_blocks(down, E * cols, rows, seed + 2, **kd))


def reference(W, E, rows, cols, up, down, x, ids, gate):
    """fp64 output and its bound, by the oracle's dequantized weights."""
    n, k = ids.shape
    out, tol = np.zeros((n, cols)), np.zeros((n, cols))
    cache = {}
    silu = lambda z: z / (1 + np.exp(-np.clip(z, -700, 700)))  # noqa: E731

    def mat(w, name, e, r, c):
        """Expert e's weights, and |ds q| + |dm| of each."""
        t, b = type_id(name), w.reshape(E, -1)[e]
        v = np.asarray(oracle.dequant(t, b, r, c), np.float64)
        if name == "Q6_K":
            _, sc, _, d, _ = oracle.unpack(t, b, r * c // 256)
            dm = 32 * np.repeat(np.asarray(sc, np.float64).reshape(-1, 16) * np.asarray(d, np.float64).reshape(-1, 1), 16, 1).reshape(r, c)
            return v, np.abs(v + dm) + np.abs(dm)
        if name not in ("Q4_K", "Q5_K", "Q2_K"):
            return v, np.abs(v)
        _, _, mins, _, dmin = oracle.unpack(t, b, r * c // 256)
        each = 16 if name == "Q2_K" else 32
        dm = np.abs((np.asarray(mins, np.float64).reshape(-1, 16)[:, :256 // each] * np.asarray(dmin, np.float64).reshape(-1, 1)))
        dm = np.repeat(dm, each, 1).reshape(r, c)
        sign = np.repeat(np.repeat(np.sign(np.asarray(dmin, np.float64)).reshape(-1, 1), 256, 1), 1, 1).reshape(r, c)
        return v, np.abs(v + sign * dm) + dm

    def mats(e):
        if e not in cache:
            cache[e] = mat(W[0], up, e, rows, cols), mat(W[1], up, e, rows, cols), mat(W[2], down, e, cols, rows)
        return cache[e]

    for i in range(n):
        for j in range(k):
            e = int(ids[i, j])
            if not 0 <= e < E:
                continue
            (wg, mg), (wu, mu), (wd, md) = mats(e)
            xi = x[i].astype(np.float64)
            g, u = wg @ xi, wu @ xi
            eg, eu = (2.0**-17 * (m @ np.abs(xi)) + 1e-6 for m in (mg, mu))
            h = silu(g) * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 2.0**-20 * np.abs(h)
            a = abs(float(gate[i, j]))
            big = md @ (np.abs(h) + eh)
            out[i] += float(gate[i, j]) * (wd @ h)
            tol[i] += a * (np.abs(wd) @ eh + 2.0**-17 * big + 1e-6) + a * big * (k + 24) * 2.0**-24
    return out, tol


def route(x, router, k, norm, scale):
    """(ids, gate, how near the next expert is to the last chosen, in logits) in 64 bits."""
    l = x.astype(np.float64) @ router.astype(np.float64).T
    order = np.argsort(-l, axis=1, kind="stable")
    top = np.take_along_axis(l, order, 1)
    e = np.exp(top - top[:, :1])
    gate = e[:, :k] / (e[:, :k] if norm else e).sum(1, keepdims=True) * scale
    gap = np.min((top[:, :-1] - top[:, 1:])[:, :k], axis=1, initial=np.inf)      # among the chosen and to the next
    return order[:, :k], gate, gap, np.abs(x).astype(np.float64) @ np.abs(router).astype(np.float64).T


CASES = [  # n, E, k, cols, rows, up, down, norm
    (1, 128, 8, 2048, 768, "Q4_K", "Q6_K", True),
    (1, 8, 2, 512, 256, "Q6_K", "Q4_K", False),
    (1, 1, 1, 256, 256, "Q2_K", "Q3_K", True),
    (2, 8, 2, 768, 512, "Q5_K", "Q5_K", True),
    (3, 4, 4, 32, 32, "Q8_0", "Q4_0", True),
    (5, 16, 4, 96, 160, "Q5_0", "Q8_0", False),
    (7, 8, 2, 4096, 256, "Q8_0", "Q8_0", True),
    (9, 3, 3, 1280, 2560, "Q3_K", "Q2_K", True),
    (13, 8, 2, 2304, 512, "Q4_K", "Q4_K", False),
    (16, 60, 6, 544, 1120, "Q4_0", "Q5_0", True),
    (31, 512, 16, 256, 64, "Q4_K", "Q4_0", True),
    (61, 128, 8, 512, 256, "Q4_K", "Q6_K", True),
    (64, 2, 1, 1024, 288, "Q6_K", "Q8_0", True),
    (64, 2, 2, 256, 256, "Q3_K", "Q3_K", False),
    (64, 512, 16, 2048, 32, "Q8_0", "Q8_0", True),
    (4, 4, 2, 4352, 2304, "Q8_0", "Q6_K", True),
    (17, 300, 5, 288, 96, "Q5_0", "Q5_0", False),
]


@pytest.mark.parametrize("n,E,k,cols,rows,up,down,norm", CASES)
def test_layer(gpu, n, E, k, cols, rows, up, down, norm):
    W = layer(500 + n + E, E, rows, cols, up, down)
    x = synth.activations(n, cols, 77 + n)
    router = (synth.activations(E, cols, 78 + E) / np.sqrt(cols)).astype(np.float32)
    scale = 1.0 if norm else 2.5
    Wd = [dev_u8(w, gpu) for w in W]
    out, ids, gate = qk.moe_ffn(type_id(up), Wd[0], Wd[1], type_id(down), Wd[2], E, rows, cols, dev_f32(x, gpu), k,
                                router=dev_f32(router, gpu), norm=norm, scale=scale)
    want_ids, want_gate, gap, size = route(x, router, k, norm, scale)
    got_ids, got_gate = ids.cpu().numpy(), gate.cpu().numpy()
    # a lane's share of the products in four running sums, then shuffles: cols / 128 + 8 roundings
    off = (cols / 128 + 8) * 2.0**-24 * size.max(1)
    sure = gap > 2 * off
    assert sure.mean() > 0.9 or n < 8
    assert np.array_equal(got_ids[sure], want_ids[sure])
    # the gate's error: twice the logits' (its own and the sum's) and a few roundings of exp, sum and quotient
    err = np.abs(got_gate - want_gate)[sure]
    assert (err <= (2.2 * off[sure, None] + (k + E / 32 + 20) * 2.0**-24) * np.abs(want_gate[sure])).all()
    ref, tol = reference(W, E, rows, cols, up, down, x, got_ids, got_gate)
    bad = np.abs(out.cpu().numpy() - ref) > tol
    assert not bad.any(), (bad.sum(), np.max(np.abs(out.cpu().numpy() - ref) / tol))
    # given ids and gates: the same bytes
    again, _, _ = qk.moe_ffn(type_id(up), Wd[0], Wd[1], type_id(down), Wd[2], E, rows, cols, dev_f32(x, gpu), k, ids=ids, gate=gate)
    assert torch.equal(again, out)
    qk.device_status()


def test_given_ids_outside_and_twice(gpu):
    n, E, k, cols, rows = 6, 5, 4, 512, 256
    W = layer(1, E, rows, cols, "Q4_K", "Q6_K")
    x = synth.activations(n, cols, 3)
    ids = np.array([[0, 0, 1, 0], [-1, 5, 7, -9], [2, -1, 2, 3], [4, 3, 2, 1], [1, 1, 1, 1], [2147483647, 0, -2147483648, 4]], np.int32)
    gate = synth.activations(n, k, 4)
    Wd = [dev_u8(w, gpu) for w in W]
    args = (qk.Q4_K, Wd[0], Wd[1], qk.Q6_K, Wd[2], E, rows, cols)
    out, _, _ = qk.moe_ffn(*args, dev_f32(x, gpu), k, ids=torch.from_numpy(ids).to(gpu), gate=dev_f32(gate, gpu))
    ref, tol = reference(W, E, rows, cols, "Q4_K", "Q6_K", x, ids, gate)
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all() and (out[1] == 0).all()
    for i in (0, 1, 5):          # one token alone
        one, _, _ = qk.moe_ffn(*args, dev_f32(x[i:i + 1], gpu), k, ids=torch.from_numpy(ids[i:i + 1]).to(gpu),
                               gate=dev_f32(gate[i:i + 1], gpu))
        assert (np.abs(one.cpu().numpy() - ref[i:i + 1]) <= tol[i:i + 1]).all()
    none, _, _ = qk.moe_ffn(*args, dev_f32(x, gpu), k, ids=torch.full((n, k), -1, dtype=torch.int32, device=gpu), gate=dev_f32(gate, gpu))
    assert (none == 0).all()


def test_all_tokens_on_one_expert(gpu):
    n, E, cols, rows = 64, 7, 768, 512
    W = layer(9, E, rows, cols, "Q5_K", "Q4_K")
    x = synth.activations(n, cols, 5)
    ids, gate = np.full((n, 1), 6, np.int32), synth.activations(n, 1, 6)
    Wd = [dev_u8(w, gpu) for w in W]
    out, _, _ = qk.moe_ffn(qk.Q5_K, Wd[0], Wd[1], qk.Q4_K, Wd[2], E, rows, cols, dev_f32(x, gpu), 1, ids=torch.from_numpy(ids).to(gpu),
                           gate=dev_f32(gate, gpu))
    ref, tol = reference(W, E, rows, cols, "Q5_K", "Q4_K", x, ids, gate)
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()


def test_ties_and_special_logits(gpu):
    n, E, k, cols, rows = 5, 40, 6, 64, 32
    W = layer(2, E, rows, cols, "Q8_0", "Q8_0")
    x = np.zeros((n, cols), np.float32)
    router = np.zeros((E, cols), np.float32)
    x[1, 0], router[:, 0] = 1.0, -np.arange(E) // 4
    x[2, 1], router[7, 1] = 1.0, np.inf
    x[3] = np.nan
    x[4, 2], router[:, 2] = -0.0, 1.0
    Wd = [dev_u8(w, gpu) for w in W]
    out, ids, gate = qk.moe_ffn(qk.Q8_0, Wd[0], Wd[1], qk.Q8_0, Wd[2], E, rows, cols, dev_f32(x, gpu), k, router=dev_f32(router, gpu))
    ids, gate = ids.cpu().numpy(), gate.cpu().numpy()
    # expert 7's logit is NaN (0 * inf) or inf for every token, token 3's all are: it ranks first, and the gates are NaN
    for i in (0, 1, 2, 4):
        assert ids[i].tolist() == [7, 0, 1, 2, 3, 4], i
    assert ids[3].tolist() == [0, 1, 2, 3, 4, 5] and np.isnan(gate).all() and out.isnan().all()
    router[7, 1] = 0.0
    x[3] = 0.0
    out, ids, gate = qk.moe_ffn(qk.Q8_0, Wd[0], Wd[1], qk.Q8_0, Wd[2], E, rows, cols, dev_f32(x, gpu), k, router=dev_f32(router, gpu))
    ids = ids.cpu().numpy()
    for i in (0, 2, 3, 4):
        assert ids[i].tolist() == [0, 1, 2, 3, 4, 5], i
    assert ids[1].tolist() == [0, 1, 2, 3, 4, 5] and torch.allclose(gate[0].cpu(), torch.full((6,), 1 / 6))
    assert out.isfinite().all()


def test_one_token_s_nan_stays_its_own(gpu):
    n, E, k, cols, rows = 12, 4, 2, 512, 512
    W = layer(3, E, rows, cols, "Q4_K", "Q6_K")
    x = synth.activations(n, cols, 8)
    ids = np.stack([np.arange(n) % E, (np.arange(n) + 1) % E], 1).astype(np.int32)
    gate = np.full((n, k), 0.5, np.float32)
    Wd = [dev_u8(w, gpu) for w in W]
    f = lambda x: qk.moe_ffn(qk.Q4_K, Wd[0], Wd[1], qk.Q6_K, Wd[2], E, rows, cols, dev_f32(x, gpu), k,  # noqa: E731
                             ids=torch.from_numpy(ids).to(gpu), gate=dev_f32(gate, gpu))[0]
    want = f(x)
    x[4, 100], x[7, 3] = np.nan, np.inf
    got = f(x)
    ok = torch.ones(n, dtype=torch.bool, device=gpu)
    ok[4] = ok[7] = False
    assert torch.equal(got[ok], want[ok]) and got[4].isnan().all() and not got[7].isfinite().all()


def test_outlier_activations(gpu):
    n, E, k, cols, rows = 6, 4, 2, 1024, 256
    W = layer(4, E, rows, cols, "Q4_K", "Q4_K")
    x = synth.activations(n, cols, 9)
    x[:, ::32] *= 1e4
    ids = np.stack([np.arange(n) % E, (np.arange(n) + 2) % E], 1).astype(np.int32)
    gate = np.full((n, k), 0.5, np.float32)
    Wd = [dev_u8(w, gpu) for w in W]
    out = qk.moe_ffn(qk.Q4_K, Wd[0], Wd[1], qk.Q4_K, Wd[2], E, rows, cols, dev_f32(x, gpu), k, ids=torch.from_numpy(ids).to(gpu),
                     gate=dev_f32(gate, gpu))[0]
    ref, tol = reference(W, E, rows, cols, "Q4_K", "Q4_K", x, ids, gate)
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()


def test_streams_and_graph(gpu):
    n, E, k, cols, rows = 9, 16, 4, 1024, 512
    W = [dev_u8(w, gpu) for w in layer(5, E, rows, cols, "Q4_K", "Q6_K")]
    xs = [dev_f32(synth.activations(n, cols, 20 + i), gpu) for i in range(2)]
    router = dev_f32(synth.activations(E, cols, 30) / 32, gpu)
    f = lambda x, **kw: qk.moe_ffn(qk.Q4_K, W[0], W[1], qk.Q6_K, W[2], E, rows, cols, x, k, router=router, **kw)  # noqa: E731
    want = [f(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [f(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    ws = torch.empty(qk.moe_workspace(qk.Q4_K, qk.Q6_K, E, rows, cols, k, n), dtype=torch.uint8, device=gpu)
    outs = [[torch.zeros_like(v) for v in want[0]] for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):           # two calls that share a workspace
        for x, o in zip(xs, outs):
            f(x, out=o[0], ids=o[1], gate=o[2], ws=ws)
    for _ in range(3):
        ws.random_(0, 256)
        for o in outs:
            o[0].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    qk.device_status()
