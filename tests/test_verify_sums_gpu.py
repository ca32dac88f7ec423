"""Sums of a verified row: whole numbers of 2^-46 of its largest weight (2^-45
for more than 65,536 tokens), weight by weight, so that no answer depends on how
a row is shared out, and a row with weight never answers with no token."""
import pytest
import torch

from gpu_helpers import gpu  # noqa: F401
from test_verify_gpu import run, signed

pytestmark = pytest.mark.gpu


def same(rows, n_req, masks, draft, u_accept, u_sample, probs=None, temp=1.0):
    """n_req requests with the same tree: rows [n, vocab] of logits (and of the drafter's probabilities)."""
    n = len(masks)
    assert rows.shape[0] == len(draft) == len(u_accept) == n
    return dict(logits=rows.repeat(n_req, 1), cu=torch.arange(n_req + 1, dtype=torch.int32) * n,
                draft=torch.tensor(draft, dtype=torch.int32).repeat(n_req), mask=signed(masks).repeat(n_req),
                temp=torch.full((n_req,), temp), u_accept=torch.tensor(u_accept, dtype=torch.float32).repeat(n_req),
                u_sample=torch.full((n_req,), u_sample), probs=None if probs is None else probs.repeat(n_req, 1))


def tokens_at(out, i):
    return out["tokens"][:, i].cpu().tolist()


@pytest.mark.parametrize("u", [0.0, 2.0**-40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_req", [1, 60])
def test_many_weights_below_the_unit(gpu, u, dtype, n_req):
    """896 weights of exp(-33.3) = 2^-48 round to nothing in units of 2^-45: token 2000 has all there is."""
    V = 128256
    row = torch.full((1, V), float("-inf"), dtype=dtype)
    row[0, 128:1024], row[0, 2000] = -33.3, 0.0
    assert tokens_at(run(gpu, same(row.to(gpu), n_req, [1], [0], [0.0], u)), 0) == [2000] * n_req
    two = row.repeat(2, 1).to(gpu)
    tree = [1, 3], [0, 5000], [0.0, 0.5]                # a child without weight
    assert tokens_at(run(gpu, same(two, n_req, *tree, u)), 0) == [2000] * n_req
    q = torch.zeros((2, V), device=gpu)
    q[:, 5000] = 1.0
    assert tokens_at(run(gpu, same(two, n_req, *tree, u, q)), 0) == [2000] * n_req


def halves(V, dtype, seed):
    """A row whose second half holds the logits of the first in another order: its halves have the same weight.  The largest
    logit is 0, token 1's and its partner's are -17.  -> row, the partners of the first half's tokens."""
    g = torch.Generator().manual_seed(seed)
    h = (2.0 * torch.randn(V // 2, generator=g)).to(dtype)
    h = torch.where(h == h.max(), torch.zeros_like(h), h - h.max().abs())
    h[1] = -17.0
    to = torch.randperm(V // 2, generator=g)
    row = torch.empty(V, dtype=dtype)
    row[:V // 2], row[V // 2 + to] = h, h
    return row, V // 2 + to


SHAPES = [(32000, 1), (32000, 40), (32000, 400), (65536, 3), (128256, 2), (128256, 60), (131074, 1), (1002, 7)]


@pytest.mark.parametrize("V,n_req", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_halves(gpu, V, n_req, dtype):
    """u = 1/2 of a row of two equal halves: the first token of the second half, for its sum must be above the first half's."""
    for seed in range(4):
        row, to = halves(V, dtype, seed)
        plain = same(row[None].to(gpu), n_req, [1], [0], [0.0], 0.5)
        assert tokens_at(run(gpu, plain), 0) == [V // 2] * n_req
        for less in (False, True):          # a weight of 2^-24 in the last half by one step of its logit smaller (larger)
            other = row.clone()
            z = other[to[1]:to[1] + 1]
            z[:] = torch.nextafter(z, torch.full_like(z, float("-inf") if less else 0.0))
            assert other[to[1]] != row[to[1]] and row[V // 2 - 1] > -16.9
            s = same(other[None].to(gpu), n_req, [1], [0], [0.0], 0.5)
            assert tokens_at(run(gpu, s), 0) == [V // 2 - less] * n_req
        # two children that carry a token and its partner, both refused
        i = next(k for k in range(5, V // 2) if int(to[k]) != V // 2)
        tree = [1, 3, 5], [0, i, int(to[i])], [0.0, 1e9, 1e9]
        three = row.repeat(3, 1).to(gpu)
        assert tokens_at(run(gpu, same(three, n_req, *tree, 0.5)), 0) == [V // 2] * n_req
        # and the drafter's probabilities, in the same order: the halves' residuals have the same weight
        g = torch.Generator().manual_seed(100 + seed)
        q = torch.softmax(row[:V // 2].double() + 0.5 * torch.randn(V // 2, generator=g).double(), -1)
        at = int((to == V // 2).nonzero())
        q[at] = 0.0                          # what the second half begins with keeps its weight
        both = torch.empty(V, dtype=torch.float32)
        both[:V // 2], both[to] = (q / 2).float(), (q / 2).float()
        s = same(three, n_req, *tree, 0.5, both.repeat(3, 1).to(gpu))
        assert tokens_at(run(gpu, s), 0) == [V // 2] * n_req


@pytest.mark.parametrize("V,first", [(65535, True), (65536, True), (65537, False), (131072, False)])
def test_the_unit(gpu, V, first):
    """A weight of 0.6 2^-46 counts as one unit of 2^-46 and as none of 2^-45."""
    row = torch.full((1, V), float("-inf"))
    row[0, 0], row[0, 500] = -32.3955, 0.0
    assert tokens_at(run(gpu, same(row, 1, [1], [0], [0.0], 0.0)), 0) == [0 if first else 500]
