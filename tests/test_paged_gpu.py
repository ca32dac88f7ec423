"""The paged KV cache (qk_kv_plan, qk_kv_append, qk_kv_compact) and
qk_logits_process on the GPU, against the plain implementations of
paged_ref.py: integers and packed bytes exactly; logits within the roundings
of their fp32 operations (and of the bf16 output)."""
import random

import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import oracle
import paged_ref
import synth
from gpu_helpers import gpu, type_id  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


# ------------------------------------------------------------------- plan --

def plan_both(gpu, have, start, want, P, page, spare, cap, seed, capacity=None):
    rng = np.random.default_rng(seed)
    held = [-(-max(h, 0) // page) for h in have]
    held = [p if p <= P else 0 for p in held]
    order = rng.permutation(sum(held) + spare + 3).astype(np.int32)
    table = np.full((len(have), P), -7, np.int32)
    at = 0
    for r, p in enumerate(held):
        table[r, :p] = order[at:at + p]
        at += p
    free = np.full(capacity or order.size, -9, np.int32)
    free[:spare] = order[at:at + spare]
    td, fd = torch.from_numpy(table.copy()).to(gpu), torch.from_numpy(free.copy()).to(gpu)
    nd = i32([spare], gpu)
    a = [i32(v, gpu).reshape(-1) for v in (have, start, want)]
    got = [qk.kv_plan(*a, td, fd, nd, page, cap) for _ in range(2)]      # repeatable on the same buffers
    want_ = paged_ref.plan(have, start, want, table, free, spare, page, cap)
    for g in got:
        for k, v in want_.items():
            assert g[k].cpu().tolist() == v, k
    assert np.array_equal(td.cpu().numpy(), table) and np.array_equal(fd.cpu().numpy(), free)
    assert nd.item() == spare
    qk.device_status()
    return want_


def test_plan_grow_shrink_finish_new(gpu):
    got = plan_both(gpu, [20, 16, 30, 0, 64, 5], [18, 16, 0, 0, 31, 5], [40, 33, 0, 100, 31, 6], 9, 16, 12, 170, 1)
    assert all(got["granted"])


def test_plan_scarce_pages_are_refused_in_order(gpu):
    got = plan_both(gpu, [16] * 6, [16] * 6, [17, 100, 33, 16, 20, 17], 9, 16, 4, 200, 2)
    assert got["granted"] == [1, 0, 0, 1, 0, 0]


def test_plan_invalid_requests(gpu):
    big = 2**31 - 1
    got = plan_both(gpu, [16, -1, 0, 300, 5, 0, 0], [0, 0, 0, 0, -2, 9, big], [20, 30, big, 8, 9, 5, 7], 4, 16, 9, 64, 3)
    assert got["granted"] == [1, 0, 0, 0, 0, 1, 1]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n", [1, 31, 1023, 1024, 1025, 3001])
def test_plan_many_requests(gpu, page, n):
    r = random.Random(n * page)
    P = 6
    have = [r.choice([0, r.randint(0, P * page)]) for _ in range(n)]
    want = [r.choice([0, h, min(P * page, h + r.randint(0, 40)), r.randint(0, P * page)]) for h in have]
    start = [r.randint(0, h) for h in have]
    total = sum(max(0, w - s) for w, s in zip(want, start))
    for spare, cap in ((3 * n, total + 5), (n // 3, max(1, total // 2))):
        plan_both(gpu, have, start, want, P, page, spare, cap, n + page)


def test_plan_largest_batch_and_none(gpu):
    n = 8192
    plan_both(gpu, [1] * n, [1] * n, [17 if r % 2 else 2 for r in range(n)], 2, 16, n, 10 * n, 5)
    e = i32([], gpu)
    got = qk.kv_plan(e, e, e, i32([], gpu).reshape(0, 4), i32([4, 5, 6], gpu), i32([2], gpu), 16, 3)
    assert got["cu"].tolist() == [0] and got["n_free"].item() == 2 and got["slots"].tolist() == [-1, -1, -1]


def test_plan_full_stack_drops_what_does_not_fit(gpu):
    plan_both(gpu, [64, 64], [0, 0], [0, 0], 4, 16, 3, 4, 6, capacity=6)


# ----------------------------------------------------------------- append --

def scattered_slots(rng, n, n_pages, page, holes=0):
    s = rng.permutation(n_pages * page)[:n].astype(np.int64)
    s[:holes] = -1
    return s


def append_both(gpu, name, k, v, slots, n_pages, page, kd=None, vd=None):
    t = type_id(name)
    n, n_kv, d = k.shape
    pb = qk.kv_page_bytes(t, n_kv, d, page)
    pools = [torch.full((n_pages, pb), 0xA5, dtype=torch.uint8, device=gpu) for _ in range(2)]
    kd = torch.from_numpy(k).to(gpu) if kd is None else kd
    vd = torch.from_numpy(v).to(gpu) if vd is None else vd
    qk.kv_append(t, kd, vd, torch.from_numpy(slots).to(gpu), *pools, page)
    for x, p in ((k, pools[0]), (v, pools[1])):
        ref = np.full((n_pages, n_kv, page, pb // (n_kv * page)), 0xA5, np.uint8)
        rows = oracle.quantize(t, x.reshape(n * n_kv, d)).reshape(n, n_kv, qk.row_bytes(t, d))
        for i, s in enumerate(slots):
            if 0 <= s < n_pages * page:
                ref[s // page, :, s % page] = rows[i]
        assert np.array_equal(p.cpu().numpy().reshape(ref.shape), ref)


@pytest.mark.parametrize("name", ["Q8_0", "Q5_0", "Q4_0"])
@pytest.mark.parametrize("n,n_kv,d,page", [(1, 1, 32, 16), (1, 8, 128, 16), (37, 3, 64, 32), (130, 2, 256, 256), (300, 8, 128, 64),
                                           (65, 5, 32, 128)])
def test_append_bytes_equal_the_quantizer(gpu, name, n, n_kv, d, page):
    rng = np.random.default_rng(n * d)
    k, v = ((rng.standard_normal((n, n_kv, d)) * np.exp(rng.standard_normal((n, n_kv, 1)))).astype(np.float32) for _ in range(2))
    k[0, 0, :32] = 0.0
    n_pages = n // page + 3
    append_both(gpu, name, k, v, scattered_slots(rng, n, n_pages, page, holes=n // 9), n_pages, page)
    qk.device_status()


@pytest.mark.parametrize("name", ["Q8_0", "Q5_0", "Q4_0"])
def test_append_ties_extremes_and_non_finite(gpu, name):
    # Values on half codes, subnormal and overflowing scales, NaN and infinities.
    top = {"Q8_0": 127, "Q5_0": 15, "Q4_0": 7}[name]
    x = np.zeros((8, 1, 64), np.float32)
    x[0, 0, :32] = (np.arange(32) - 15.5) * top / 15.5
    x[0, 0, 32:] = np.where(np.arange(32) % 2, top, 0.5)
    x[1] = 1e-7 * np.arange(64) / 64
    x[2] = 1e30
    x[3, 0, 5], x[3, 0, 40] = np.inf, -np.inf
    x[4] = np.linspace(-2, 2, 64)
    x[4, 0, 3], x[4, 0, 50] = np.nan, np.nan
    x[5] = np.nan
    x[6] = -0.0
    x[7] = np.float32(65504.0) * np.linspace(-1, 1, 64)
    append_both(gpu, name, x, x[::-1].copy(), np.arange(8, dtype=np.int64)[::-1].copy(), 1, 16)
    qk.device_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gap,shift", [(0, 0), (32, 0), (8, 8), (3, 1), (1, 3)])
def test_append_fused_slices(gpu, dtype, gap, shift):
    # k and v inside one projection's rows, aligned and not.
    n, n_kv, d = 21, 3, 64
    g = torch.Generator(device=gpu)
    g.manual_seed(gap)
    rows = torch.randn((n, shift + 2 * n_kv * d + gap), device=gpu, generator=g).to(dtype)
    k = rows[:, shift:shift + n_kv * d].unflatten(1, (n_kv, d))
    v = rows[:, shift + n_kv * d:shift + 2 * n_kv * d].unflatten(1, (n_kv, d))
    host = lambda x: x.float().cpu().numpy()  # noqa: E731
    append_both(gpu, "Q5_0", host(k), host(v), scattered_slots(np.random.default_rng(1), n, 3, 16), 3, 16, k, v)


def test_append_skips_and_reports_bad_slots(gpu):
    k = np.random.default_rng(3).standard_normal((6, 2, 64)).astype(np.float32)
    append_both(gpu, "Q8_0", k, k, np.array([31, -1, 32, 4, -5, 2**40], np.int64), 2, 16)
    with pytest.raises(qk.QKError) as e:
        qk.device_status()
    assert e.value.status == 8
    qk.device_status()   # cleared
    append_both(gpu, "Q8_0", k[:0], k[:0], np.zeros(0, np.int64), 2, 16)


# ---------------------------------------------------------------- compact --

def compact_ref(p, page, table, base, path, n_path):
    out = p.copy()
    for r in range(len(base)):
        m = min(max(n_path[r], 0), path.shape[1], 64)
        for j in range(m):
            a, b = base[r] + path[r, j], base[r] + j
            if not (0 <= path[r, j] < 64) or base[r] < 0 or max(a, b) // page >= table.shape[1]:
                continue
            pa, pb = table[r, a // page], table[r, b // page]
            if 0 <= pa < len(p) and 0 <= pb < len(p):
                out[pb, :, b % page] = p[pa, :, a % page]
    return out


@pytest.mark.parametrize("name,n_kv,d,page", [("Q8_0", 2, 128, 16), ("Q4_0", 1, 32, 32), ("Q5_0", 3, 256, 64), ("Q8_0", 1, 256, 16)])
def test_compact_moves_paths(gpu, name, n_kv, d, page):
    rng = np.random.default_rng(d + page)
    n_req, P = 9, -(-140 // page)
    pools = [paged_ref.pool(name, n_req * P, n_kv, page, d, 60 + i) for i in range(2)]
    table = rng.permutation(n_req * P).astype(np.int32).reshape(n_req, P)
    base = rng.integers(0, 70, n_req).astype(np.int32)
    path = np.stack([np.sort(rng.permutation(64)) for _ in range(n_req)]).astype(np.int32)
    for r in range(n_req):
        keep = np.sort(rng.permutation(64)[:rng.integers(1, 64)])
        path[r, :len(keep)] = keep
    path[3] = rng.permutation(64)          # any order, overlaps both ways
    n_path = rng.integers(0, 64, n_req).astype(np.int32)
    n_path[3], n_path[4], n_path[5] = 64, 99, -4
    dev = [torch.from_numpy(p).to(gpu) for p in pools]
    qk.kv_compact(type_id(name), *dev, page, n_kv, d, *(torch.from_numpy(a).to(gpu) for a in (table, base, path, n_path)))
    qk.device_status()
    for p, got in zip(pools, dev):
        assert np.array_equal(got.cpu().numpy(), compact_ref(p, page, table, base, path, n_path))


def test_compact_leaves_rows_without_a_page(gpu):
    p = paged_ref.pool("Q8_0", 3, 1, 16, 64, 70)
    table = np.array([[0, 77], [2, 1]], np.int32)
    base, path, n_path = np.array([10, 28], np.int32), np.array([[1, 9, 3], [2, 70, 5]], np.int32), np.array([3, 3], np.int32)
    dev = [torch.from_numpy(p).to(gpu) for _ in range(2)]
    qk.kv_compact(qk.Q8_0, *dev, 16, 1, 64, *(torch.from_numpy(a).to(gpu) for a in (table, base, path, n_path)))
    ref = compact_ref(p, 16, table, base, path, n_path)
    assert np.array_equal(dev[0].cpu().numpy(), ref) and np.array_equal(dev[1].cpu().numpy(), ref)
    with pytest.raises(qk.QKError):
        qk.device_status()


def test_append_and_compact_past_32_bit_offsets(gpu):
    # The last pages of a pool of 4.6 GB (more bytes than 32 bits count).
    t, n_kv, d, page = qk.Q8_0, 8, 128, 64
    pb = qk.kv_page_bytes(t, n_kv, d, page)
    n_pages = (1 << 32) // pb + 4000
    K = torch.zeros((n_pages, pb), dtype=torch.uint8, device=gpu)
    V = torch.zeros_like(K)
    x = np.random.default_rng(9).standard_normal((3, n_kv, d)).astype(np.float32)
    last = n_pages * page
    xd = torch.from_numpy(x).to(gpu)
    qk.kv_append(t, xd, xd, torch.tensor([last - 1, last - 2, last - 3], device=gpu), K, V, page)
    rows = oracle.quantize(t, x.reshape(-1, d)).reshape(3, n_kv, -1)
    for P in (K, V):
        got = P[-1].cpu().numpy().reshape(n_kv, page, -1)
        assert np.array_equal(got[:, -3:], rows[::-1].transpose(1, 0, 2)) and not got[:, :-3].any()
        assert not P[:-1].any()
    table = i32([[n_pages - 1]], gpu)
    qk.kv_compact(t, K, V, page, n_kv, d, table, i32([0], gpu), i32([[61, 63]], gpu), i32([2], gpu))
    for P in (K, V):
        got = P[-1].cpu().numpy().reshape(n_kv, page, -1)
        assert np.array_equal(got[:, 0], rows[2]) and np.array_equal(got[:, 1], rows[0])
    qk.device_status()


# ----------------------------------------------------------------- logits --

def logits_both(gpu, x, out=None, in_place=False, **kw):
    """kw: the lists as numpy arrays; x a CUDA tensor."""
    dev = {k: None if v is None else torch.from_numpy(np.ascontiguousarray(v).view(np.int32 if v.dtype == np.uint32 else
                                                      np.int64 if v.dtype == np.uint64 else v.dtype)).to(gpu)
           for k, v in kw.items()}
    src = x.float().cpu().numpy()
    got = qk.logits_process(x, out=x if in_place else out, **dev)
    y = got.float().cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        ref, size = paged_ref.logits(src, **kw)
        # quotient or product, freq * c, two differences, the bias: five fp32 roundings of terms no larger than their
        # sum of magnitudes, then the output's
        tol = 5 * 2.0**-24 * size + (2.0**-8 if x.dtype is torch.bfloat16 else 0.0) * np.abs(ref) * (1 + 2.0**-8)
        fine = np.isfinite(ref)
        assert np.array_equal(np.isnan(y), np.isnan(ref)) and np.array_equal(y[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
        bad = np.abs(y - ref)[fine] > tol[fine]
    assert not bad.any(), f"{bad.sum()} logits off, worst {np.max((np.abs(y - ref)[fine] / np.maximum(tol[fine], 1e-300))):.3g} of the tolerance"
    return got


def lists(rng, cu, V, H=50, B=7, n_mask=True):
    n_req, rows = len(cu) - 1, int(cu[-1])
    zipf = lambda *s: np.minimum((V * rng.random(s) ** 3).astype(np.int32), V - 1)  # noqa: E731
    mask = rng.integers(0, 2**63, rows).astype(np.uint64) | (np.uint64(1) << np.uint64(63)) * rng.integers(0, 2, rows).astype(np.uint64)
    return dict(cu=np.array(cu, np.int32), hist=zipf(n_req, H), hist_len=rng.integers(0, H + 1, n_req).astype(np.int32),
                rep=(1 + 0.5 * rng.random(n_req)).astype(np.float32), pres=rng.random(n_req).astype(np.float32),
                freq=rng.random(n_req).astype(np.float32), draft=zipf(rows), mask=mask if n_mask else None,
                bias_tok=zipf(n_req, B), bias_val=rng.standard_normal((n_req, B)).astype(np.float32),
                bias_len=rng.integers(0, B + 1, n_req).astype(np.int32),
                grammar=rng.integers(0, 2**32, (rows, -(-V // 32))).astype(np.uint32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 31, 33, 1000, 4095, 4096, 4097, 8200, 32003])
def test_logits_ragged_requests(gpu, dtype, V):
    rng = np.random.default_rng(V)
    cu = [0, 3, 3, 4, 13, 30]
    x = torch.from_numpy((3 * rng.standard_normal((30, V))).astype(np.float32)).to(gpu).to(dtype)
    logits_both(gpu, x, **lists(rng, cu, V))


@pytest.mark.parametrize("off", [("draft", "mask"), ("mask",), ("bias_tok", "bias_val", "bias_len"), ("grammar",),
                                 ("draft", "mask", "bias_tok", "bias_val", "bias_len", "grammar")])
def test_logits_parts_left_out(gpu, off):
    rng = np.random.default_rng(11)
    kw = lists(rng, [0, 9, 20], 700)
    kw.update({k: None for k in off})
    logits_both(gpu, torch.from_numpy(rng.standard_normal((20, 700)).astype(np.float32)).to(gpu), **kw)


def test_logits_chain_longer_than_a_mask(gpu):
    rng = np.random.default_rng(12)
    kw = lists(rng, [0, 90, 91], 300, n_mask=False)
    logits_both(gpu, torch.from_numpy(rng.standard_normal((91, 300)).astype(np.float32)).to(gpu), **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stride,shift", [(1024, 0), (1003, 0), (1008, 4), (1001, 1)])
def test_logits_strides_alignment_in_place(gpu, dtype, stride, shift):
    rng = np.random.default_rng(stride)
    V = 1000
    base = torch.from_numpy(rng.standard_normal(12 * stride + 8).astype(np.float32)).to(gpu).to(dtype)
    x = base[shift:shift + 12 * stride].view(12, stride)[:, :V]
    kw = lists(rng, [0, 5, 12], V)
    before = base.clone()
    a = logits_both(gpu, x, **kw)
    assert torch.equal(base, before)
    b = logits_both(gpu, x, in_place=True, **kw)
    assert torch.equal(a, b)
    rest = torch.ones_like(base, dtype=torch.bool)
    rest[shift:shift + 12 * stride].view(12, stride)[:, :V] = False
    assert torch.equal(base[rest], before[rest])      # nothing outside the rows is touched


def test_logits_special_values_and_ids(gpu):
    rng = np.random.default_rng(14)
    V = 96
    x = rng.standard_normal((4, V)).astype(np.float32)
    x[0, :6] = [np.inf, -np.inf, np.nan, 0.0, -0.0, np.finfo(np.float32).min]
    kw = lists(rng, [0, 2, 4], V, H=20, B=6)
    kw["hist"][0, :8] = [0, 1, 2, 3, 4, 5, -1, V]
    kw["hist_len"][:] = [20, 500]          # longer than the row: cut to it
    kw["hist"][1, 3], kw["draft"][1] = 2**31 - 1, -3
    kw["bias_tok"][0] = [7, 7, 9, V, -1, 7]   # the last entry of a token counts
    kw["bias_len"][:] = [6, -2]
    kw["grammar"][3] = 0                   # nothing allowed
    y = logits_both(gpu, torch.from_numpy(x).to(gpu), **kw)
    assert torch.isinf(y[3]).all()


def test_logits_rows_of_no_request(gpu):
    rng = np.random.default_rng(15)
    x = rng.standard_normal((10, 50)).astype(np.float32)
    kw = lists(rng, [2, 4, 7], 50)
    kw["draft"], kw["mask"], kw["grammar"] = (np.resize(kw[k], (10,) + kw[k].shape[1:]) for k in ("draft", "mask", "grammar"))
    logits_both(gpu, torch.from_numpy(x).to(gpu), **kw)
    e = {k: kw[k][:0] for k in ("hist", "hist_len", "rep", "pres", "freq")}
    logits_both(gpu, torch.from_numpy(x).to(gpu), cu=np.zeros(1, np.int32), grammar=kw["grammar"], **e)
