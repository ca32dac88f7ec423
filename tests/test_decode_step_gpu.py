"""A decode step of a mixture-of-experts model over drafted trees, all calls as
they follow one another: pages planned, keys and values normed, rotated and
written, tree attention, the expert layer, logits processed and judged, the
cache compacted.  Each call's own test says how exact it is; here every call
reads what the one before wrote, eagerly and from a captured graph."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import step_ref
import synth
import test_moe_gpu
from gpu_helpers import dev_u8, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

H, KV, D, PAGE, HID, E, ROWS, K, V = 4, 2, 64, 16, 256, 8, 256, 2, 777
T, UP, DOWN = qk.Q8_0, qk.Q4_K, qk.Q6_K


def model(gpu):
    g = torch.Generator().manual_seed(3)
    W = test_moe_gpu.layer(900, E, ROWS, HID, "Q4_K", "Q6_K")
    r = lambda *s, by=1.0: (by * torch.randn(s, generator=g)).to(gpu)  # noqa: E731
    return dict(host=W, W=[dev_u8(w, gpu) for w in W], router=r(E, HID, by=0.2), head=r(HID, V, by=0.3), embed=r(V, (H + 2 * KV) * D),
                freq=(10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(gpu),
                norms=[(1 + 0.2 * torch.randn(D, generator=g)).to(gpu) for _ in range(2)])


def batch(gpu, seed, ctx, sizes):
    """The trees of a step, on caches of ctx tokens."""
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    par = [[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)] for n in sizes]
    masks, depth = [], []
    for p in par:
        for i, a in enumerate(p):
            base = len(masks) - i
            masks.append((masks[base + a] if a >= 0 else 0) | 1 << i)
            depth.append(depth[base + a] + 1 if a >= 0 else 0)
    n, r = sum(sizes), len(sizes)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    pos = [c + depth[sum(sizes[:j]) + i] for j, c in enumerate(ctx) for i in range(sizes[j])]
    return dict(ctx=i32(ctx), want=i32([c + s for c, s in zip(ctx, sizes)]), pos=i32(pos), cu=i32(np.concatenate([[0], np.cumsum(sizes)])),
                mask=torch.tensor(masks, dtype=torch.int64, device=gpu), draft=torch.randint(0, V, (n,), generator=g).to(torch.int32).to(gpu),
                temp=(0.5 + torch.rand(r, generator=g)).to(gpu), u=(torch.rand(n, generator=g) > 0.7).float().to(gpu), u2=torch.rand(r, generator=g).to(gpu),
                hist=torch.randint(0, V, (r, 9), generator=g).to(torch.int32).to(gpu), hist_len=i32([9] * r),
                pen=[torch.full((r,), v, device=gpu) for v in (1.2, 0.1, 0.05)], max_q=max(sizes))


def cache(gpu, ctx, n_pages, P):
    """Pools with bytes in them, a table that gives the requests their pages, and the free ones."""
    g = torch.Generator().manual_seed(5)
    pools = [dev_u8(synth.random_blocks("Q8_0", n_pages * KV * PAGE, D, 70 + i), gpu).view(n_pages, -1) for i in range(2)]
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table, at = torch.full((len(ctx), P), -1, dtype=torch.int32), 0
    for r, c in enumerate(ctx):
        for p in range(-(-c // PAGE)):
            table[r, p], at = order[at], at + 1
    free = torch.zeros(n_pages, dtype=torch.int32)
    free[:n_pages - at] = order[at:]
    return dict(pools=pools, table=table.to(gpu), free=free.to(gpu), n_free=torch.tensor([n_pages - at], dtype=torch.int32, device=gpu))


def step(m, b, c):
    n = b["pos"].numel()
    plan = qk.kv_plan(b["ctx"], b["ctx"], b["want"], c["table"], c["free"], c["n_free"], PAGE, n)
    x = m["embed"][b["draft"].long()].to(torch.bfloat16)
    q, k, v = (x[:, a * D:(a + h) * D].unflatten(1, (h, D)) for a, h in ((0, H), (H, KV), (H + KV, KV)))
    q = qk.kv_append_rope(T, q, k, v, b["pos"], m["freq"], plan["slots"], *c["pools"], PAGE, q_norm=m["norms"][0], k_norm=m["norms"][1])
    o = qk.attn_tree(T, q, *c["pools"], PAGE, KV, c["table"], b["ctx"], b["cu"], b["mask"], b["max_q"], D ** -0.5)
    h = o.view(n, HID).float()
    y, ids, gate = qk.moe_ffn(UP, m["W"][0], m["W"][1], DOWN, m["W"][2], E, ROWS, HID, h, K, router=m["router"])
    logits = (h + y / y.abs().amax()) @ m["head"]
    z = qk.logits_process(logits, b["cu"], b["hist"], b["hist_len"], *b["pen"], draft=b["draft"], mask=b["mask"])
    got = qk.verify_tree(z, b["cu"], b["draft"], b["mask"], b["temp"], b["u"], b["u2"])
    before = [p.clone() for p in c["pools"]]
    qk.kv_compact(T, *c["pools"], PAGE, KV, D, c["table"], b["ctx"], got["path"], got["n_path"])
    return dict(got, slots=plan["slots"], q=q, h=h, y=y, ids=ids, gate=gate, z=z, before=before, n_free=plan["n_free"])


CTX, SIZES, PAGES = [37, 0, 16, 90], [7, 1, 12, 5], 24


def test_the_calls_follow_one_another(gpu):
    m, b, c = model(gpu), batch(gpu, 1, CTX, SIZES), cache(gpu, CTX, PAGES, 8)
    s = step(m, b, c)
    qk.device_status()
    host = {k: v.cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor) and v.dtype is not torch.bfloat16}
    # the rows that the plan named hold the keys, and nothing else was written
    _, kr = qk.norm_rope(None, m["embed"][b["draft"].long()].to(torch.bfloat16)[:, H * D:(H + KV) * D].unflatten(1, (KV, D)), b["pos"],
                         m["freq"], k_norm=m["norms"][1], out_dtype=torch.float32)
    fresh = cache(gpu, CTX, PAGES, 8)["pools"][0]
    vs = torch.zeros_like(fresh)
    qk.kv_append(T, kr, kr, s["slots"], fresh, vs, PAGE)
    assert torch.equal(fresh, s["before"][0]) and (host["slots"] >= 0).all()
    # the expert layer on what attention gave
    ref, tol = test_moe_gpu.reference(m["host"], E, ROWS, HID, "Q4_K", "Q6_K", host["h"], host["ids"], host["gate"])
    assert (np.abs(host["y"] - ref) <= tol).all()
    # the walk over the processed logits
    at = np.concatenate([[0], np.cumsum(SIZES)])
    for r in range(len(SIZES)):
        rows = slice(at[r], at[r + 1])
        step_ref.replay(host["z"][rows], b["draft"].cpu().numpy()[rows], [int(v) & (2**64 - 1) for v in b["mask"][rows].cpu()],
                        float(b["temp"][r]), b["u"].cpu().numpy()[rows], float(b["u2"][r]), None, 64, host["path"][r], host["n_path"][r],
                        host["tokens"][r])
    # the cache behind the walk: the path's rows, in order
    table, page = c["table"].cpu().numpy(), lambda p: p.view(PAGES, KV, PAGE, -1)
    for now, then in zip(c["pools"], s["before"]):
        for r, base in enumerate(CTX):
            for j in range(host["n_path"][r]):
                a, z = base + j, base + int(host["path"][r, j])
                assert torch.equal(page(now)[table[r, a // PAGE], :, a % PAGE], page(then)[table[r, z // PAGE], :, z % PAGE])
    assert host["n_path"].max() > 1 and host["n_path"].min() >= 1


def test_a_captured_step_is_the_eager_one(gpu):
    m = model(gpu)
    steps = [batch(gpu, s, CTX, SIZES) for s in (1, 2, 3)]
    want = [step(m, b, cache(gpu, CTX, PAGES, 8)) for b in steps]
    torch.cuda.synchronize()
    b, c = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in steps[0].items()}, cache(gpu, CTX, PAGES, 8)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(m, b, c)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = step(m, b, c)
    for i in (1, 2, 0, 1):
        fresh = cache(gpu, CTX, PAGES, 8)
        for k in ("table", "free", "n_free"):
            c[k].copy_(fresh[k])
        for p, f in zip(c["pools"], fresh["pools"]):
            p.copy_(f)
        for k, v in steps[i].items():
            if isinstance(v, torch.Tensor):
                b[k].copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want[i].items():
            if isinstance(v, torch.Tensor):
                assert torch.equal(got[k], v), k
            else:
                assert all(torch.equal(x, y) for x, y in zip(got[k], v)), k
    qk.device_status()
