"""qk_attn_tree (attention of drafted-token trees over the paged, block-
quantized cache) against the 64-bit implementation of paged_ref.py on the same
blocks.

Tolerance, per output, from the roundings of the call's documented arithmetic:
the output to bf16 (2^-8 of it); each probability and each V element to fp16
(2^-11 each, together 2^-10 of sum p|V|); each K element to fp16, which moves a
score by at most 2^-11 A (A the largest scale * sum |q k| of a visible
position) and a probability by twice that, 2^-10 A of sum p|V|; 2^-13 for the
fp32 sums and exponentials; and where a probability is too small for fp16 (it
is held times 2^7 at least, against the row's largest), half a step, 2^-32 of
its |V|."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import oracle
import paged_ref
import synth
from gpu_helpers import gpu, type_id  # noqa: F401

pytestmark = pytest.mark.gpu


def make(name, ctx, n, heads, n_kv, d, page, seed, q_scale=1.0, spare=2, table_cols=None, **kw):
    """A case as numpy arrays; pages in random order, unused table entries -1."""
    rng = np.random.default_rng(seed)
    held = [-(-(c + m) // page) for c, m in zip(ctx, n)]
    n_pages = sum(held) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(ctx), table_cols or max(max(held), 1)), -1, np.int32)
    at = 0
    for r, p in enumerate(held):
        table[r, :p] = order[at:at + p]
        at += p
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    bits = []
    for m in n:
        own = []
        for i in range(m):
            p = int(rng.integers(-1, i))
            own.append((own[p] if p >= 0 else 0) | (1 << i))
        bits += own
    q = torch.from_numpy((q_scale * rng.standard_normal((int(cu[-1]), heads, d))).astype(np.float32)).to(torch.bfloat16)
    return dict(name=name, q=q, K=paged_ref.pool(name, n_pages, n_kv, page, d, seed + 1, **kw),
                V=paged_ref.pool(name, n_pages, n_kv, page, d, seed + 2, **kw), page=page, n_kv=n_kv, table=table,
                ctx=np.array(ctx, np.int32), cu=cu, mask=np.array(bits, np.uint64), max_q=max(max(n), 1), scale=1 / np.sqrt(d))


def to_dev(c, gpu):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(gpu)  # noqa: E731
    mask = None if c["mask"] is None else t(c["mask"].view(np.int64))
    return (c["q"].to(gpu), t(c["K"]), t(c["V"]), c["page"], c["n_kv"], t(c["table"]), t(c["ctx"]), t(c["cu"]), mask, c["max_q"],
            float(c["scale"]))


def check(c, out, ref=None):
    ref, Sv, A, V1 = ref or paged_ref.attn_tree(c["name"], c["q"].double().numpy(), c["K"], c["V"], c["page"], c["n_kv"], c["table"],
                                            c["ctx"], c["cu"], c["mask"], c["max_q"], c["scale"])
    got = out.float().cpu().numpy().astype(np.float64)
    rows = ~np.isnan(ref).all(axis=(1, 2))
    tol = 2.0**-8 * np.abs(ref) + (2.0**-10 * (1 + A[..., None]) + 2.0**-13) * Sv + 2.0**-32 * V1 + 1e-30
    bad = ~(np.abs(got - ref) <= tol)[rows]
    assert not bad.any(), f"{bad.sum()} outputs off, worst {np.nanmax((np.abs(got - ref) / tol)[rows]):.3g} of the tolerance"
    return ref, Sv, A, V1


def run(c, gpu):
    out = qk.attn_tree(type_id(c["name"]), *to_dev(c, gpu))
    qk.device_status()
    check(c, out)
    return out


@pytest.mark.parametrize("name", ["Q8_0", "Q5_0", "Q4_0"])
@pytest.mark.parametrize("heads,n_kv,d", [(8, 2, 128), (4, 4, 64), (6, 2, 32), (8, 1, 256), (3, 1, 128), (12, 4, 64)])
def test_layouts(gpu, name, heads, n_kv, d):
    run(make(name, [77, 0, 300], [5, 3, 1], heads, n_kv, d, 32, 100 + d), gpu)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500])
def test_lengths(gpu, T):
    run(make("Q8_0", [T - 1, max(0, T - 7)], [1, min(7, T)], 8, 2, 128, 16, 200 + T), gpu)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_page_sizes(gpu, page, d):
    run(make("Q5_0", [page - 3, page, 2 * page + 1, 333], [5, 1, 9, 2], 4, 2, d, page, 300 + page + d), gpu)


@pytest.mark.parametrize("n,heads,n_kv,d", [(64, 8, 1, 64), (64, 32, 8, 128), (63, 4, 1, 128), (33, 16, 4, 32), (17, 16, 1, 256),
                                            (64, 64, 1, 32), (2, 64, 1, 128)])
def test_wide_trees(gpu, n, heads, n_kv, d):
    run(make("Q4_0", [190], [n], heads, n_kv, d, 64, 400 + n), gpu)


def test_many_ragged_requests(gpu):
    rng = np.random.default_rng(7)
    ctx, n = rng.integers(0, 900, 40), rng.integers(0, 9, 40)
    run(make("Q8_0", ctx.tolist(), n.tolist(), 8, 2, 64, 16, 500), gpu)


def test_long_context_is_split(gpu):
    run(make("Q4_0", [9001], [3], 4, 1, 64, 128, 510), gpu)
    run(make("Q8_0", [7000, 12], [2, 30], 4, 1, 128, 16, 511), gpu)


def test_chain_without_mask_and_decode(gpu):
    c = make("Q8_0", [40, 41, 0], [6, 1, 64], 4, 2, 64, 16, 520)
    c["mask"] = None
    run(c, gpu)
    c = make("Q8_0", [1, 40, 399], [1, 1, 1], 8, 2, 128, 16, 521)     # batched single-token decoding
    c["mask"] = None
    run(c, gpu)


def test_rows_that_see_nothing(gpu):
    c = make("Q8_0", [0, 0, 50], [4, 1, 3], 4, 2, 64, 16, 530)
    c["mask"][:] = [0, 0b0010, 0, 0b1001, 0, 0, 0b1000, 0b111]    # bits past a request's tokens count for nothing
    out = run(c, gpu)
    assert not out[0].any() and not out[2].any() and not out[4].any()


def test_full_mask_bits(gpu):
    c = make("Q5_0", [10, 3], [64, 64], 2, 1, 64, 16, 531)
    c["mask"][:] = np.uint64(2**64 - 1)
    run(c, gpu)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 6e4])
def test_what_is_not_seen_does_not_matter(gpu, bad, d):
    # A drafted row with a non-finite (or huge) scale that some tokens see,
    # and stale NaN bytes past the last position and in unused pages.
    c = make("Q8_0", [21, 5], [6, 4], 4, 2, d, 16, 540)
    c["mask"][:6] = [1, 3, 7, 0b1001, 0b11001, 0b111111]
    rb = c["K"].shape[-1]
    for r, T in ((0, 27), (1, 9)):
        for p in range(T, c["table"].shape[1] * 16):
            if c["table"][r, p // 16] >= 0:
                for x in (c["K"], c["V"]):
                    x[c["table"][r, p // 16], :, p % 16] = 0xFF
    ids = {int(i) for i in c["table"].ravel() if i >= 0}
    for i in set(range(len(c["K"]))) - ids:
        c["K"][i] = c["V"][i] = 0xFF
    at = 21 + 2                                            # token 2: seen by tokens 2 and 5
    clean = {k: v.copy() for k, v in c.items() if k in "KV"}
    for x in (c["K"], c["V"]):
        blocks = x[c["table"][0, at // 16], :, at % 16].reshape(2, rb // 34, 34)
        blocks[..., :2] = np.array([bad], np.float16).view(np.uint8)
        x[c["table"][0, at // 16], :, at % 16] = blocks.reshape(2, rb)
    out = qk.attn_tree(qk.Q8_0, *to_dev(c, gpu))
    qk.device_status()
    ref = paged_ref.attn_tree("Q8_0", c["q"].double().numpy(), clean["K"], clean["V"], 16, 2, c["table"], c["ctx"], c["cu"], c["mask"],
                              c["max_q"], c["scale"])
    others = [0, 1, 3, 4, 6, 7, 8, 9]
    check({**c, "q": c["q"][others]}, out[others], tuple(x[others] for x in ref))
    if not np.isfinite(bad):
        assert torch.isnan(out[[2, 5]].float()).all()


@pytest.mark.parametrize("name", ["Q8_0", "Q4_0"])
@pytest.mark.parametrize("k_scale,v_scale", [(1e-7, 1e-7), (1e-2, 1e-5), (0.3, 200.0), (1e-4, 1.0)])
def test_scale_range(gpu, name, k_scale, v_scale):
    c = make(name, [300, 90], [4, 7], 8, 2, 128, 32, 550)
    c["K"] = paged_ref.pool(name, len(c["K"]), 2, 32, 128, 551, d_scale=k_scale)
    c["V"] = paged_ref.pool(name, len(c["V"]), 2, 32, 128, 552, d_scale=v_scale)
    run(c, gpu)


def test_masked_large_values_cost_no_accuracy(gpu):
    # One drafted row 2^20 times the others' size, hidden from token 0.
    c = make("Q8_0", [100], [2], 4, 1, 128, 32, 555)
    c["mask"][:] = [1, 3]
    at = 101
    row = c["V"][c["table"][0, at // 32], 0, at % 32].reshape(4, 34)
    row[:, :2] = np.array([400.0], np.float16).view(np.uint8)
    c["V"][c["table"][0, at // 32], 0, at % 32] = row.reshape(-1)
    run(c, gpu)


@pytest.mark.parametrize("q_scale", [1e-6, 30.0, 1e5])
def test_query_range(gpu, q_scale):
    # tiny queries, peaked scores, and queries past fp16's range against a
    # cache small enough for finite scores
    c = make("Q8_0", [200], [5], 8, 2, 128, 16, 560, q_scale=q_scale, **({"d_scale": 1e-6} if q_scale > 1e4 else {}))
    run(c, gpu)


def test_strided_query_and_output(gpu):
    c = make("Q5_0", [50, 20], [7, 3], 6, 2, 64, 16, 570)
    dev = list(to_dev(c, gpu))
    wide = torch.zeros((10, 6 * 64 + 72), dtype=torch.bfloat16, device=gpu)
    wide[:, 8:8 + 384] = dev[0].reshape(10, 384)
    dev[0] = wide[:, 8:8 + 384].unflatten(1, (6, 64))
    buf = torch.full((10, 500), 7.0, dtype=torch.bfloat16, device=gpu)
    out = qk.attn_tree(qk.Q5_0, *dev, out=buf[:, 3:387].unflatten(1, (6, 64)))
    check(c, out)
    assert (buf[:, :3] == 7).all() and (buf[:, 387:] == 7).all()


def test_rows_of_no_request_and_max_q(gpu):
    c = make("Q8_0", [30, 20], [7, 3], 4, 1, 64, 16, 580)
    dev = list(to_dev(c, gpu))
    dev[0] = torch.cat([dev[0], dev[0][:2]])
    dev[8] = torch.cat([dev[8], dev[8][:2]])
    out = torch.full((12, 4, 64), 7.0, dtype=torch.bfloat16, device=gpu)
    qk.attn_tree(qk.Q8_0, *dev, out=out)
    check(c, out[:10])
    assert (out[10:] == 7).all()
    dev[9] = c["max_q"] = 4
    out.fill_(7.0)
    qk.attn_tree(qk.Q8_0, *dev, out=out)
    assert (out[4:7] == 7).all()
    ref = paged_ref.attn_tree("Q8_0", c["q"].double().numpy(), c["K"], c["V"], 16, 1, c["table"], c["ctx"], c["cu"], c["mask"], 4,
                              c["scale"])
    keep = [0, 1, 2, 3, 7, 8, 9]
    check(c, out[keep], tuple(x[keep] for x in ref))


def test_bad_pages_are_not_followed_and_reported(gpu):
    c = make("Q8_0", [40, 35], [2, 2], 4, 1, 64, 16, 590)
    good = c["table"].copy()
    c["table"][0, 1] = 10**6
    c["table"][1, 0] = -3
    out = qk.attn_tree(qk.Q8_0, *to_dev(c, gpu))
    with pytest.raises(qk.QKError) as e:
        qk.device_status()
    assert e.value.status == 8
    qk.device_status()
    # as if the positions of those pages did not exist
    for r, lost in ((0, range(16, 32)), (1, range(0, 16))):
        n = 2
        T = int(c["ctx"][r]) + n
        left = [p for p in range(T) if p not in lost]
        k, v = (np.stack([x[good[r, p // 16], 0, p % 16] for p in left]) for x in (c["K"], c["V"]))
        pad = lambda x: np.concatenate([x, np.zeros((48 - len(x), x.shape[1]), np.uint8)]).reshape(3, 1, 16, -1)  # noqa: E731
        tok = slice(int(c["cu"][r]), int(c["cu"][r + 1]))
        sub = dict(c, q=c["q"][tok], mask=c["mask"][tok])
        ref = paged_ref.attn_tree("Q8_0", sub["q"].double().numpy(), pad(k), pad(v), 16, 1, np.array([[0, 1, 2]]), [len(left) - n], [0, n],
                                  sub["mask"], 2, c["scale"])
        check(sub, out[tok], ref)


def test_table_shorter_than_the_length(gpu):
    c = make("Q8_0", [40], [2], 4, 1, 64, 16, 595)
    dev = list(to_dev(c, gpu))
    dev[5] = dev[5][:, :2].contiguous()
    qk.attn_tree(qk.Q8_0, *dev)
    with pytest.raises(qk.QKError):
        qk.device_status()


def test_pool_past_32_bit_offsets(gpu):
    c = make("Q8_0", [200], [4], 8, 8, 128, 64, 600)
    pb = qk.kv_page_bytes(qk.Q8_0, 8, 128, 64)
    far = (1 << 32) // pb + 1000
    dev = list(to_dev(c, gpu))
    for i in (1, 2):
        big = torch.zeros((far + len(c["K"]), pb), dtype=torch.uint8, device=gpu)
        big[far:] = dev[i].reshape(len(c["K"]), pb)
        dev[i] = big
    dev[5] = torch.where(dev[5] >= 0, dev[5] + far, dev[5])
    out = qk.attn_tree(qk.Q8_0, *dev)
    qk.device_status()
    check(c, out)


def test_deterministic_and_on_another_stream(gpu):
    c = make("Q8_0", [3000, 700, 5], [8, 3, 20], 8, 2, 128, 16, 610)
    dev = to_dev(c, gpu)
    a = qk.attn_tree(qk.Q8_0, *dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = qk.attn_tree(qk.Q8_0, *dev)
    s.synchronize()
    assert torch.equal(a, b)
    check(c, a)


def test_a_step_in_a_graph(gpu):
    # plan, append, attention, compaction and logits captured once; replayed
    # with other lengths, queries and tokens in the same buffers.
    t, n_kv, heads, d, page, P, R, n = qk.Q8_0, 2, 8, 64, 16, 8, 3, 5
    pb = qk.kv_page_bytes(t, n_kv, d, page)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=gpu)  # noqa: E731
    K, V = (torch.zeros((R * P, pb), dtype=torch.uint8, device=gpu) for _ in range(2))
    table = torch.full((R, P), -1, dtype=torch.int32, device=gpu)
    free = torch.arange(R * P, dtype=torch.int32, device=gpu)
    n_free = i32(R * P)
    have, start, want = i32(0, 0, 0), i32(0, 0, 0), i32(n, n, n)
    mask = torch.tensor([1, 3, 5, 11, 21] * R, dtype=torch.int64, device=gpu)
    g = torch.Generator(device=gpu)
    g.manual_seed(1)
    kv = torch.randn((2, R * n, n_kv, d), device=gpu, generator=g).to(torch.bfloat16)
    q = torch.randn((R * n, heads, d), device=gpu, generator=g).to(torch.bfloat16)
    path, n_path = i32(0, 1, 3).repeat(R, 1).contiguous(), i32(3, 3, 3)

    def step():
        p = qk.kv_plan(have, start, want, table, free, n_free, page, R * n)
        qk.kv_append(t, kv[0], kv[1], p["slots"], K, V, page)
        out = qk.attn_tree(t, q, K, V, page, n_kv, table, start, p["cu"], mask, n, 0.125)
        qk.kv_compact(t, K, V, page, n_kv, d, table, start, path, n_path)
        return p, out

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    table.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, out = step()
    Kr, Vr = np.zeros((R, P * page, n_kv, qk.row_bytes(t, d)), np.uint8), np.zeros((R, P * page, n_kv, qk.row_bytes(t, d)), np.uint8)
    for it in range(6):
        kv.normal_(generator=g)
        q.normal_(generator=g)
        base = start.cpu().tolist()
        graph.replay()
        torch.cuda.synchronize()
        for x, ref in ((kv[0], Kr), (kv[1], Vr)):
            rows = oracle.quantize(t, x.float().cpu().numpy().reshape(-1, d)).reshape(R, n, n_kv, -1)
            for r in range(R):
                ref[r, base[r]:base[r] + n] = rows[r]
        c = dict(name="Q8_0", q=q.cpu(), K=Kr.reshape(R * P, page, n_kv, -1).transpose(0, 2, 1, 3),
                 V=Vr.reshape(R * P, page, n_kv, -1).transpose(0, 2, 1, 3), page=page, n_kv=n_kv,
                 table=np.arange(R * P).reshape(R, P), ctx=np.array(base), cu=p["cu"].cpu().numpy(),
                 mask=mask.cpu().numpy().view(np.uint64), max_q=n, scale=0.125)
        check(c, out)
        for ref in (Kr, Vr):
            for r in range(R):
                ref[r, base[r]:base[r] + 3] = ref[r, [base[r] + j for j in (0, 1, 3)]]
        have.copy_(want)
        n_free.copy_(p["n_free"])
        start.add_(3)
        want.copy_(start + n)
    qk.device_status()


def test_references_that_grow_along_the_positions(gpu):
    # Keys that point more and more along the query: every tile outgrows the
    # references of the one before, in one CTA and across several.
    for ctx, n_req in ((1500, 1), (700, 40)):
        c = make("Q8_0", [ctx] * n_req, [3] * n_req, 4, 1, 64, 64, 620)
        u = np.random.default_rng(1).standard_normal(64).astype(np.float32)
        c["q"] = torch.from_numpy(np.broadcast_to(u, c["q"].shape).copy()).to(torch.bfloat16)
        for r in range(n_req):
            for p in range(ctx + 3):
                k = (u * (p / 40.0) / 8.0).astype(np.float32)
                c["K"][c["table"][r, p // 64], 0, p % 64] = oracle.quantize(qk.Q8_0, k[None])
        run(c, gpu)


def test_large_v_tiles_among_ordinary_ones(gpu):
    # V past fp16's range in the first tile, in a middle one and in the last,
    # with references that are renewed in between.
    c = make("Q8_0", [600], [4], 4, 1, 128, 32, 630, q_scale=3.0)
    for p in (5, 300, 601):
        row = c["V"][c["table"][0, p // 32], 0, p % 32].reshape(4, 34)
        row[:, :2] = np.array([3000.0], np.float16).view(np.uint8)
        c["V"][c["table"][0, p // 32], 0, p % 32] = row.reshape(-1)
    run(c, gpu)
    c = make("Q4_0", [20, 300], [4, 4], 4, 2, 256, 32, 631, q_scale=3.0)
    c["V"] = paged_ref.pool("Q4_0", len(c["V"]), 2, 32, 256, 632, d_scale=9000.0)     # every tile
    run(c, gpu)


def test_non_finite_v_in_the_context(gpu):
    # A committed row with a NaN scale in one 32-block: that block of every token of its request and kv head, nothing else.
    c = make("Q8_0", [150, 40], [3, 2], 4, 2, 128, 16, 640)
    clean = c["V"].copy()
    at = 70
    c["V"][c["table"][0, at // 16], 1, at % 16, 34:36] = 0xFF
    out = qk.attn_tree(qk.Q8_0, *to_dev(c, gpu))
    qk.device_status()
    ref = paged_ref.attn_tree("Q8_0", c["q"].double().numpy(), c["K"], clean, 16, 2, c["table"], c["ctx"], c["cu"], c["mask"], 3,
                              c["scale"])
    got = out.float().cpu()
    assert torch.isnan(got[:3, 2:, 32:64]).all()
    got[:3, 2:, 32:64] = torch.from_numpy(ref[0][:3, 2:, 32:64]).float()
    check(c, got, ref)


@pytest.mark.parametrize("n_req,n_kv", [(897, 1), (2000, 4)])
def test_many_short_units(gpu, n_req, n_kv):
    # More requests than the scan takes at once, and dozens of one-tile units
    # per CTA.
    rng = np.random.default_rng(n_req)
    ctx, n = rng.integers(0, 40, n_req), rng.integers(0, 3, n_req)
    ctx[rng.integers(0, n_req, 20)] = 300
    run(make("Q4_0", ctx.tolist(), n.tolist(), 2 * n_kv, n_kv, 32, 16, 650), gpu)


def test_negative_scale_and_zero_queries(gpu):
    c = make("Q5_0", [130, 7], [5, 2], 8, 2, 64, 16, 660)
    c["scale"] = -0.2
    c["q"][1] = 0
    run(c, gpu)


def test_nan_query_stays_in_its_row(gpu):
    c = make("Q8_0", [100], [3], 8, 2, 64, 16, 670)
    dev = list(to_dev(c, gpu))
    dev[0] = dev[0].clone()
    dev[0][1, 5, 3] = float("nan")
    out = qk.attn_tree(qk.Q8_0, *dev)
    ref = paged_ref.attn_tree("Q8_0", c["q"].double().numpy(), c["K"], c["V"], 16, 2, c["table"], c["ctx"], c["cu"], c["mask"], 3,
                              c["scale"])
    assert torch.isnan(out[1, 5].float()).all()
    got = out.float().cpu()
    got[1, 5] = torch.from_numpy(ref[0][1, 5]).float()
    check(c, got, ref)
