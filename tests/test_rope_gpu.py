"""Norms and rotation of heads, as rows and on the way into the paged cache,
against 64-bit and stepwise fp32 implementations.

Tolerance of a value against 64 bits, in units of 2^-24 of the magnitude of its
terms: the sum of squares has a rounding per square and one per level of its
tree (log2 d <= 8), of which the root halves the relative error (4.5); the
division, the sum with eps (before the root: half each), the root and the
reciprocal 3; the products with inv and w 2; cos or sin 2 (the nearest or the
next value); its product and the last sum 2.  That is 13.5, taken as 15; then
the rounding to the output's type, eps / 2 of it."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import step_ref
from gpu_helpers import gpu, type_id  # noqa: F401

pytestmark = pytest.mark.gpu


def inputs(gpu, n, heads, n_kv, d, rot, seed, dtype=torch.float32, gap=0, far=5000):
    g = torch.Generator().manual_seed(seed)
    width = (heads + 2 * n_kv) * d + gap
    x = (torch.randn((n, width), generator=g) * torch.exp(0.5 * torch.randn((1, width), generator=g))).to(dtype).to(gpu)
    part = lambda a, h: x[:, a * d:(a + h) * d].unflatten(1, (h, d))  # noqa: E731
    pos = torch.randint(0, far + 1, (n,), generator=g, dtype=torch.int64).to(torch.int32).to(gpu)
    freq = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(gpu)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(gpu) for _ in range(2)]
    return part(0, heads), part(heads, n_kv), part(heads + n_kv, n_kv), pos, freq, w


def np_(t):
    return None if t is None else t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def check(out, x, pos, freq, w, eps, pairs, what):
    want, size = step_ref.turned(np_(x), np_(pos), np_(freq), np_(w), eps, pairs)
    got = out.double().cpu().numpy()
    half = 0.0 if out.dtype is torch.float32 else torch.finfo(out.dtype).eps / 2
    bound = 15 * 2.0**-24 * size * (1 + half) + half * np.abs(want) + 1e-37
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{what}: {np.max(err / bound):.3g} of the bound"


CASES = [  # n, heads, n_kv, d, rot, dtype, out, norm, pairs, gap, far
    (1, 32, 8, 128, 128, "f32", "f32", True, False, 0, 700),
    (1, 1, 1, 32, 32, "bf16", "f32", False, True, 0, 0),
    (7, 6, 2, 32, 16, "bf16", "bf16", True, False, 3, 40000),
    (13, 8, 1, 64, 64, "f32", "bf16", True, True, 5, 1 << 20),
    (33, 12, 4, 256, 64, "bf16", "bf16", True, False, 8, 1 << 30),
    (700, 32, 8, 64, 48, "f32", "f32", False, False, 96, 2147483647),
    (331, 5, 3, 128, 96, "f32", "f32", True, False, 0, 1000000),
    (3, 4, 2, 128, 0, "bf16", "f32", True, False, 0, 10),
    (2, 3, 3, 256, 256, "f32", "bf16", False, False, 1, 10),
    (6001, 12, 4, 64, 32, "bf16", "f32", True, True, 0, 1 << 24),
    (9973, 5, 2, 32, 32, "f32", "f32", True, False, 7, 1 << 20),
]


@pytest.mark.parametrize("n,heads,n_kv,d,rot,act,out,norm,pairs,gap,far", CASES)
def test_rows(gpu, n, heads, n_kv, d, rot, act, out, norm, pairs, gap, far):
    ty = {"f32": torch.float32, "bf16": torch.bfloat16}
    q, k, _, pos, freq, w = inputs(gpu, n, heads, n_kv, d, rot, 100 + n + d, ty[act], gap, far)
    w = w if norm else [None, None]
    a, b = qk.norm_rope(q, k, pos, freq, q_norm=w[0], k_norm=w[1], eps=1e-5, pairs=pairs, out_dtype=ty[out])
    assert a.shape == q.shape and b.shape == k.shape and a.dtype is ty[out]
    check(a, q, pos, freq, w[0], 1e-5, pairs, "q")
    check(b, k, pos, freq, w[1], 1e-5, pairs, "k")
    # every step is rounded as stated: equal but where a cosine or sine is the next value (one in some ten thousand)
    if out == "f32":
        for got, x, ww in ((a, q, w[0]), (b, k, w[1])):
            want = step_ref.turned_stepwise(np_(x), np_(pos), np_(freq), np_(ww), 1e-5, pairs)
            assert (got.cpu().numpy() == want).mean() >= 0.999


def test_negative_positions_and_odd_frequencies(gpu):
    q, k, _, _, _, _ = inputs(gpu, 9, 2, 1, 64, 64, 5)
    pos = torch.tensor([-1, -7, -2147483648, 2147483647, 0, 1, 1 << 24, (1 << 24) + 1, -(1 << 30)], dtype=torch.int32, device=gpu)
    f = torch.logspace(-12, 6, 32, dtype=torch.float64).float()
    f[3], f[5], f[7] = 0.0, -0.25, 1e-40
    a, _ = qk.norm_rope(q, None, pos, f.to(gpu))
    check(a, q, pos, f, None, 0.0, False, "q")


def test_frequencies_that_are_none(gpu):
    q, _, _, pos, freq, _ = inputs(gpu, 3, 2, 1, 32, 32, 6)
    freq = freq.clone()
    freq[1], freq[2], freq[4] = float("nan"), float("inf"), 2.0**64
    a, _ = qk.norm_rope(q, None, pos, freq)
    bad = torch.zeros(32, dtype=torch.bool, device=gpu)
    for j in (1, 2, 4):
        bad[j] = bad[j + 16] = True
    assert a[..., bad].isnan().all() and a[..., ~bad].isfinite().all()


def test_in_place_and_strided_out(gpu):
    q, k, _, pos, freq, w = inputs(gpu, 21, 6, 2, 64, 64, 7, torch.bfloat16, 16)
    want = qk.norm_rope(q, k, pos, freq, q_norm=w[0], k_norm=w[1])
    wide = torch.full((21, 9 * 64 + 3), 7.0, dtype=torch.bfloat16, device=gpu)
    o = wide[:, :6 * 64].unflatten(1, (6, 64))
    qk.norm_rope(q, None, pos, freq, q_norm=w[0], q_out=o)
    assert torch.equal(o, want[0]) and (wide[:, 6 * 64:] == 7).all()
    qk.norm_rope(q, k, pos, freq, q_norm=w[0], k_norm=w[1], q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_special_values(gpu):
    q, _, _, pos, freq, w = inputs(gpu, 4, 2, 1, 32, 32, 8)
    q = q.clone()
    q[0, 0, 3], q[1, 1, 4], q[2, 0] = float("nan"), float("inf"), 0.0
    a, _ = qk.norm_rope(q, None, pos, freq, q_norm=w[0], eps=0.0)
    assert a[0, 0].isnan().all() and a[2, 0].isnan().all()       # 0 / 0 without eps
    assert a[1, 1, 4].isnan() and a[0, 1].isfinite().all() and a[1, 0].isfinite().all() and a[3].isfinite().all()
    b, _ = qk.norm_rope(q, None, pos, freq, q_norm=w[0], eps=1e-6)
    assert (b[2, 0] == 0).all()


APPEND = [  # type, n, heads, n_kv, d, rot, dtype, norm, pairs, gap, page
    ("Q8_0", 1, 32, 8, 128, 128, "f32", True, False, 0, 16),
    ("Q4_0", 13, 8, 2, 64, 32, "bf16", True, True, 1, 32),
    ("Q5_0", 40, 12, 4, 256, 256, "f32", True, False, 2, 64),
    ("Q4_0", 400, 32, 8, 128, 128, "bf16", False, False, 128, 16),
    ("Q8_0", 65, 0, 1, 32, 32, "bf16", False, True, 0, 256),
    ("Q5_0", 90, 6, 2, 32, 0, "f32", True, False, 3, 128),
    ("Q8_0", 5003, 8, 4, 128, 64, "f32", True, False, 4, 32),
    ("Q4_0", 8009, 3, 3, 64, 64, "bf16", True, True, 0, 16),
]


@pytest.mark.parametrize("name,n,heads,n_kv,d,rot,act,norm,pairs,gap,page", APPEND)
def test_append(gpu, name, n, heads, n_kv, d, rot, act, norm, pairs, gap, page):
    t = type_id(name)
    q, k, v, pos, freq, w = inputs(gpu, n, heads, n_kv, d, rot, 300 + n, torch.bfloat16 if act == "bf16" else torch.float32, gap, 1 << 21)
    w = w if norm else [None, None]
    g = torch.Generator().manual_seed(n)
    n_pages = -(-n // page) + 3
    slots = torch.randperm(n_pages * page, generator=g)[:n]
    slots[n // 2] = -1
    slots = slots.to(gpu)
    pools = [torch.randint(0, 256, (n_pages, qk.kv_page_bytes(t, n_kv, d, page)), dtype=torch.uint8, generator=g).to(gpu)
             for _ in range(2)]
    mine, want = [p.clone() for p in pools], [p.clone() for p in pools]
    out = qk.kv_append_rope(t, q if heads else None, k, v, pos, freq if rot else None, slots, *mine, page, q_norm=w[0], k_norm=w[1],
                            eps=1e-6, pairs=pairs)
    qr, kr = qk.norm_rope(q if heads else None, k, pos, freq if rot else None, q_norm=w[0], k_norm=w[1], eps=1e-6, pairs=pairs,
                          out_dtype=torch.float32)
    qk.kv_append(t, kr, v.float(), slots, *want, page)
    assert torch.equal(mine[0], want[0]) and torch.equal(mine[1], want[1])      # and what no slot names stays
    if heads:
        assert torch.equal(out, qr.to(torch.bfloat16))
    else:
        assert out is None
    qk.device_status()


def test_append_reports_bad_slots(gpu):
    q, k, v, pos, freq, _ = inputs(gpu, 4, 2, 1, 32, 32, 9)
    pools = [torch.zeros((2, qk.kv_page_bytes(qk.Q8_0, 1, 32, 16)), dtype=torch.uint8, device=gpu) for _ in range(2)]
    slots = torch.tensor([3, 32, -2, 5], device=gpu)
    qk.kv_append_rope(qk.Q8_0, q, k, v, pos, freq, slots, *pools, 16)
    with pytest.raises(qk.QKError) as e:
        qk.device_status()
    assert e.value.status == 8
    rows = pools[0].view(2, 16, 34).any(-1)
    assert rows[0, 3] and rows[0, 5] and rows.sum() == 2


def test_two_streams_and_a_graph(gpu):
    a, b = (inputs(gpu, n, 8, 2, 128, 128, n) for n in (60, 350))
    want = [qk.norm_rope(x[0], x[1], x[3], x[4], q_norm=x[5][0]) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [qk.norm_rope(x[0], x[1], x[3], x[4], q_norm=x[5][0], stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u[0], v[0]) and torch.equal(u[1], v[1])
    graph, out = torch.cuda.CUDAGraph(), [torch.zeros_like(a[0]), torch.zeros_like(a[1])]
    with torch.cuda.graph(graph):
        qk.norm_rope(a[0], a[1], a[3], a[4], q_norm=a[5][0], q_out=out[0], k_out=out[1])
    for _ in range(2):
        out[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0][0]) and torch.equal(out[1], want[0][1])
