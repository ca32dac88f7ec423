"""A node whose children were all refused although they have all its weight (an
acceptance number of 1 or more): the token after it is drawn from the row's own
weights."""
import pytest
import torch

from gpu_helpers import gpu  # noqa: F401
from test_verify_gpu import run
from test_verify_sums_gpu import same, tokens_at

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1, 300, 32000, 140000])
@pytest.mark.parametrize("u", [1.0, 3.0, float("nan")])
@pytest.mark.parametrize("drafter", [False, True])
def test_nothing_left(gpu, V, u, drafter):
    for top in sorted({0, V // 5, V - 1}):
        rows = torch.full((2, V), float("-inf"))
        rows[:, top] = 3.0
        q = torch.zeros((2, V))
        q[:, top] = 1.0
        out = run(gpu, same(rows, 3, [1, 3], [0, top], [0.0, u], 0.25, q if drafter else None))
        assert tokens_at(out, 0) == [top] * 3 and out["n_path"].tolist() == [1] * 3


@pytest.mark.parametrize("u", [0.0, 2.0**-40])
@pytest.mark.parametrize("drafter", [False, True])
def test_only_weights_below_the_unit_left(gpu, u, drafter):
    V = 128256
    rows = torch.full((2, V), float("-inf"))
    rows[:, 128:1024], rows[:, 2000] = -33.3, 0.0
    q = torch.zeros((2, V))
    q[:, 2000] = 1.0
    for n_req in (1, 60):
        out = run(gpu, same(rows.to(gpu), n_req, [1, 3], [0, 2000], [0.0, 7.0], u, q.to(gpu) if drafter else None))
        assert tokens_at(out, 0) == [2000] * n_req


def test_all_tokens_refused(gpu):
    # every token of a small vocabulary on a child, all refused: any of them, by the row's weights
    V = 5
    rows = torch.tensor([0.0, -1.0, 0.5, float("-inf"), 1.0]).repeat(V + 1, 1)
    masks = [1] + [1 | 1 << i for i in range(1, V + 1)]
    w = (rows[0] - 1.0).exp().double()
    for u, want in ((0.0, 0), (0.2, 1), (0.3, 2), (0.99, 4)):
        assert int((w.cumsum(0) / w.sum() > u).nonzero()[0]) == want
        out = run(gpu, same(rows, 2, masks, [0, *range(V)], [0.0] + [2.0] * V, u))
        assert tokens_at(out, 0) == [want] * 2
