"""Tree verification: every decision of the walk replayed against the rule in
64 bits, the distribution of the tokens, and the corners of its inputs."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import step_ref
from gpu_helpers import gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def tree_bits(rng, n, chain):
    bits = []
    for i in range(n):
        p = (i - 1 if chain else int(rng.integers(max(0, i - 6), i))) if i else -1
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return bits


def signed(bits):
    bits = [b & ((1 << 64) - 1) for b in bits]
    return torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64)


def make(seed, sizes, V, drafter, chain=False, dtype=torch.float32, likely=True):
    """Host inputs: logits near the drafter's, drafted tokens that are often taken."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    rows, r = sum(sizes), len(sizes)
    cu = np.concatenate([[0], np.cumsum(sizes)])
    masks = [b for n in sizes for b in tree_bits(rng, n, chain)]
    logits = (2.0 * torch.randn((rows, V), generator=g)).to(dtype)
    probs = torch.softmax(logits.float() + 0.5 * torch.randn((rows, V), generator=g), -1) if drafter else None
    draft = torch.randint(0, V, (rows,), generator=g)
    for a, n in zip(cu, sizes):
        par = step_ref.parents(n, masks[a:a + n])
        for i in range(1, n):
            if drafter:
                draft[a + i] = torch.multinomial(probs[a + par[i]], 1, generator=g)[0]
            elif likely:
                draft[a + i] = torch.multinomial(torch.softmax(2 * logits[a + par[i]].float(), -1), 1, generator=g)[0]
    return dict(logits=logits, cu=torch.tensor(cu, dtype=torch.int32), draft=draft.to(torch.int32), mask=signed(masks),
                temp=0.4 + torch.rand(r, generator=g), u_accept=torch.rand(rows, generator=g), u_sample=torch.rand(r, generator=g),
                probs=probs)


def run(gpu, s, stride=64, **kw):
    d = {k: None if v is None else v.to(gpu) for k, v in s.items()}
    return qk.verify_tree(d["logits"], d["cu"], d["draft"], d["mask"], d["temp"], d["u_accept"], d["u_sample"], probs=d["probs"],
                          max_path=stride, **kw)


def check(s, out, stride=64):
    h = {k: None if v is None else v.float().numpy() if v.is_floating_point() else v.numpy() for k, v in s.items()}
    path, tokens, n_path = (out[k].cpu().numpy() for k in ("path", "tokens", "n_path"))
    for r in range(len(n_path)):
        a, b = int(h["cu"][r]), int(h["cu"][r + 1])
        m = None if h["mask"] is None else [int(x) & (2**64 - 1) for x in h["mask"][a:b]]
        step_ref.replay(h["logits"][a:b], h["draft"][a:b], m, float(h["temp"][r]), h["u_accept"][a:b], h["u_sample"][r],
                        None if h["probs"] is None else h["probs"][a:b], stride, path[r], int(n_path[r]), tokens[r])
    return n_path


CASES = [  # sizes, vocab, drafter, chain, dtype
    ([6], 32000, False, True, torch.float32),
    ([1], 1, False, True, torch.float32),
    ([3, 1, 5], 7, True, False, torch.float32),
    ([8] * 9, 1003, True, True, torch.float32),
    ([64, 1, 17, 40], 5000, False, False, torch.bfloat16),
    ([20, 64], 32003, True, False, torch.bfloat16),
    ([4] * 50, 4096, False, False, torch.float32),
    ([2] * 400, 130, True, False, torch.float32),
    ([12, 9], 128256, True, False, torch.float32),
]


@pytest.mark.parametrize("sizes,V,drafter,chain,dtype", CASES)
def test_walk(gpu, sizes, V, drafter, chain, dtype):
    s = make(40 + V, sizes, V, drafter, chain, dtype)
    n_path = check(s, run(gpu, s))
    if len(sizes) >= 9:
        assert n_path.max() > 1
    if chain:
        out = run(gpu, s)
        s["mask"] = None
        plain = run(gpu, s)
        assert all(torch.equal(out[k], plain[k]) for k in out)


@pytest.mark.parametrize("drafter", [False, True])
def test_same_tokens_again_and_refusals(gpu, drafter):
    # siblings that carry the same token, tokens outside the vocabulary, and a drafter far from the target
    s = make(3, [64] * 6, 50, drafter, likely=False)
    star = [1] + [(1 << i) | 1 for i in range(1, 64)]
    s["mask"] = signed(star * 6)
    s["draft"] = torch.arange(64).remainder(9).to(torch.int32).repeat(6)
    s["draft"][5], s["draft"][6], s["draft"][70], s["draft"][71] = -1, -2, 50, 2147483647
    s["u_accept"] = 0.5 + 0.5 * s["u_accept"]
    check(s, run(gpu, s))


@pytest.mark.parametrize("drafter", [False, True])
def test_tokens_are_distributed_as_the_target(gpu, drafter):
    # the first token after the root over many requests with the same two rows: counts within 5 standard deviations
    N, V = 60000, 11
    g = torch.Generator().manual_seed(8)
    base = 1.5 * torch.randn(V, generator=g)
    p = torch.softmax(base / 0.8, -1)
    qrow = torch.softmax(1.5 * torch.randn(V, generator=g), -1)
    kids = 3
    logits = base.repeat(N * (kids + 1), 1)
    draft = torch.multinomial(qrow.repeat(N, 1), kids + 1, replacement=True, generator=g)
    if not drafter:
        draft[:, 1:] = torch.tensor([4, 1, 4])
    s = dict(logits=logits, cu=torch.arange(N + 1, dtype=torch.int32) * (kids + 1), draft=draft.reshape(-1).to(torch.int32),
             mask=torch.tensor([1, 3, 5, 9]).repeat(N), temp=torch.full((N,), 0.8), u_accept=torch.rand(N * (kids + 1), generator=g),
             u_sample=torch.rand(N, generator=g), probs=qrow.repeat(N * (kids + 1), 1) if drafter else None)
    out = run(gpu, s, stride=2)
    first = out["tokens"][:, 0].cpu().long()
    count = torch.bincount(first, minlength=V).double()
    sigma = (N * p * (1 - p)).double().sqrt()
    assert ((count - N * p).abs() <= 5 * sigma + 1).all(), (count, N * p)
    taken = (out["n_path"] == 2).double().mean().item()
    # without probabilities a child is taken as often as the target has the children's tokens (4 and 1); with them the
    # first child alone is taken with sum min(p, q)
    often = (p[4] + p[1] if not drafter else torch.minimum(p, qrow).sum()).item()
    off = 5 * (often * (1 - often) / N) ** 0.5 + 1 / N
    assert often - off <= taken <= (1.0 if drafter else often + off)


def test_greedy(gpu):
    s = make(11, [9, 30, 1, 12], 777, False)
    s["temp"] = torch.tensor([0.0, -1.0, float("nan"), 2.0**-21])
    s["logits"][:9, 5] = s["logits"][:9, 300] = 40.0             # equals: the lowest token
    s["draft"][:9] = 5
    s["mask"][:9] = signed([(2 << i) - 1 for i in range(9)])     # a chain that is right throughout
    out = run(gpu, s)
    check(s, out)
    assert out["n_path"][0] == 9 and (out["tokens"][0, :9] == 5).all()


def test_rows_without_weight_and_specials(gpu):
    s = make(12, [3, 3, 3, 3, 3], 2000, False, chain=True)
    x = s["logits"]
    x[0] = float("-inf")
    x[3, ::2] = float("nan")
    x[6, 100] = x[6, 1500] = float("inf")
    x[9] = float("-inf")
    x[9, 1999] = -3e38
    s["draft"][7], s["draft"][10] = 1500, 1999
    s["u_accept"][7] = 0.4
    s["temp"][4] = float("inf")
    s["draft"][1] = 2147483647
    out = run(gpu, s)
    greedy = dict(s, temp=torch.zeros(5))
    check(greedy, run(gpu, greedy))
    check(s, out)
    assert out["n_path"][0] == 1 and out["tokens"][0, 0] == -1
    assert out["tokens"][2, 0] == 1500 and out["tokens"][3, 0] == 1999 and out["n_path"][3] > 1


def test_random_numbers_at_the_ends(gpu):
    for u in (0.0, 1.0 - 2.0**-24, 1.0, 7.0, float("nan")):
        s = make(13, [5, 5], 300, True)
        s["u_accept"][:], s["u_sample"][:] = u, u
        out = run(gpu, s)
        t = out["tokens"].cpu()
        n = out["n_path"].cpu()
        assert all(0 <= t[r, n[r] - 1] < 300 for r in range(2))
        if u < 1.0:
            check(s, out)


def test_requests_without_rows_and_long_ones(gpu):
    s = make(14, [0, 3, 70, 0], 900, False, chain=True)
    s["mask"] = None
    s["u_accept"][:] = 0.0          # everything that has weight is taken
    out = run(gpu, s)
    check(s, out)
    assert out["n_path"].tolist() == [0, 3, 64, 0]
    none = qk.verify_tree(torch.zeros((0, 5), device=gpu), torch.zeros(1, dtype=torch.int32, device=gpu),
                          *(torch.zeros(0, dtype=t, device=gpu) for t in (torch.int32, torch.int64, torch.float32, torch.float32, torch.float32)))
    assert none["n_path"].shape == (0,)


def test_a_path_ends_at_the_stride(gpu):
    s = make(15, [10, 10], 500, False, chain=True)
    s["u_accept"][:] = 0.0
    for stride in (1, 4):
        out = run(gpu, s, stride=stride)
        check(s, out, stride)
        assert (out["n_path"] == stride).all()


def test_strided_rows_and_given_outputs(gpu):
    s = make(16, [7, 5], 515, True)
    want = run(gpu, s)
    wide = torch.zeros((12, 600)), torch.zeros((12, 521))
    wide[0][:, :515], wide[1][:, :515] = s["logits"], s["probs"]
    d = {k: None if v is None else v.to(gpu) for k, v in s.items()}
    out = {"path": torch.full((2, 64), 9, dtype=torch.int32, device=gpu), "tokens": torch.full((2, 64), 9, dtype=torch.int32, device=gpu),
           "n_path": torch.full((2,), 9, dtype=torch.int32, device=gpu)}
    qk.verify_tree(wide[0].to(gpu)[:, :515], d["cu"], d["draft"], d["mask"], d["temp"], d["u_accept"], d["u_sample"],
                   probs=wide[1].to(gpu)[:, :515], out=out)
    assert all(torch.equal(out[k], want[k]) for k in want)


def test_a_graph_and_two_streams(gpu):
    s, z = make(17, [8] * 5, 9000, True), make(18, [30], 32000, False)
    want = run(gpu, s), run(gpu, z)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(gpu, s, stream=one), run(gpu, z, stream=two)
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert all(torch.equal(u[k], v[k]) for k in u)
    d = {k: None if v is None else v.to(gpu) for k, v in s.items()}
    graph = torch.cuda.CUDAGraph()
    out = {k: torch.zeros_like(v) for k, v in want[0].items()}
    with torch.cuda.graph(graph):
        qk.verify_tree(d["logits"], d["cu"], d["draft"], d["mask"], d["temp"], d["u_accept"], d["u_sample"], probs=d["probs"], out=out)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[0][k]) for k in out)


@pytest.mark.parametrize("drafter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_children_near_their_threshold(gpu, drafter, dtype):
    """u beside W / (q S) by a part of 2^-15, more than the walk's sums are off and less than the pieces' may be."""
    n, r, V = 9, 8, 5000
    s = make(19, [n] * r, V, drafter, chain=True, dtype=dtype)
    x = s["logits"].float().numpy()
    for i in range(r):
        for j in range(1, n):
            up = i * n + j - 1
            e, y = step_ref.weights(x[up], float(s["temp"][i])), int(s["draft"][up + 1])
            q = float(s["probs"][up, y]) if drafter else 1.0
            s["u_accept"][up + 1] = e[y] / (q * e.sum()) * (1 + (2.0**-15 if j > i else -2.0**-15))
    out = run(gpu, s)
    check(s, out)
    assert out["n_path"].tolist() == [i + 1 for i in range(r)]


def test_nodes_behind_refusals(gpu):
    """Walks that leave the line of first children: every first child is refused."""
    s = make(20, [40, 3, 64, 1], 3000, False)
    at, first = 0, []
    for n in (40, 3, 64, 1):
        par = step_ref.parents(n, [int(v) & (2**64 - 1) for v in s["mask"][at:at + n]])
        first += [i > 0 and par.index(par[i]) == i for i in range(n)]
        at += n
    s["u_accept"] = torch.where(torch.tensor(first), torch.full_like(s["u_accept"], 1e9), 0.3 * s["u_accept"])
    check(s, run(gpu, s))
    # two children everywhere: the first is refused, the second has some weight and costs nothing
    n = 41
    s = make(23, [n, n], 3000, False, likely=False)
    bits = [1]
    for i in range(1, n):
        bits.append(bits[(i - 1) // 2 * 2] | 1 << i)
    s["mask"] = signed(bits * 2)
    s["u_accept"] = torch.tensor([1e9 if i % 2 else 0.0 for i in range(n)] * 2)
    out = run(gpu, s)
    check(s, out)
    assert out["n_path"].tolist() == [n // 2 + 1] * 2 and out["path"][0, :n // 2 + 1].tolist() == list(range(0, n, 2))


def test_given_workspaces(gpu):
    s, z = make(21, [8] * 5, 9000, True, chain=True), make(22, [8] * 5, 9000, True, chain=True)
    want = run(gpu, s), run(gpu, z)
    ws = torch.full((qk.verify_workspace(40, 5, 9000),), 255, dtype=torch.uint8, device=gpu)
    assert ws.numel() == 40 * 9 * 16
    graph, got = torch.cuda.CUDAGraph(), []
    d = [{k: None if v is None else v.to(gpu) for k, v in c.items()} for c in (s, z)]
    with torch.cuda.graph(graph):           # two calls that share it
        for c in d:
            got.append(qk.verify_tree(c["logits"], c["cu"], c["draft"], c["mask"], c["temp"], c["u_accept"], c["u_sample"],
                                      probs=c["probs"], ws=ws))
    for _ in range(3):
        ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(a[k], b[k]) for k in a)
    with pytest.raises(qk.QKError) as e:
        run(gpu, s, ws=ws[:-16])
    assert e.value.status == 5
    with pytest.raises(qk.QKError) as e:
        run(gpu, s, ws=ws[::2])
    assert e.value.status == 8


def test_rows_of_no_request(gpu):
    s = make(24, [1, 4, 1], 2500, False, chain=True)
    s["cu"] = torch.tensor([2, 3, 3, 5], dtype=torch.int32)       # one row, none, two; the others are nobody's
    s["temp"][2], s["mask"] = 0.7, None
    out = run(gpu, s)
    check(s, out)
    assert out["n_path"][1] == 0
    s["cu"] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    out = run(gpu, s)
    check(s, out)
    assert out["n_path"].tolist() == [1, 1, 1]
