"""qk_attn_tree over caches in which V blocks past fp16's range lie among
ordinary and tiny ones: the large block may cost the others no accuracy,
whether it is visible or hidden, in their own 32-block of channels or in another.  Against
paged_ref.py with the tolerance of test_tree_gpu.py, whose terms are per
channel."""
import numpy as np
import pytest

import paged_ref
from gpu_helpers import gpu  # noqa: F401
from test_tree_gpu import make, run

pytestmark = pytest.mark.gpu

BB = {"Q8_0": 34, "Q5_0": 22, "Q4_0": 18}
BIG = {"Q8_0": 3000.0, "Q5_0": 9000.0, "Q4_0": 30000.0}     # times the largest code past 65504


def enlarge(c, r, pos, g, blk):
    name, page = c["name"], c["page"]
    row = c["V"][c["table"][r, pos // page], g, pos % page].reshape(-1, BB[name])
    row[blk, :2] = np.array([BIG[name]], np.float16).view(np.uint8)
    c["V"][c["table"][r, pos // page], g, pos % page] = row.reshape(-1)


def case(name, ctx, n, heads, n_kv, d, page, seed, v_scale):
    c = make(name, ctx, n, heads, n_kv, d, page, seed)
    c["V"] = paged_ref.pool(name, len(c["V"]), n_kv, page, d, seed + 2, d_scale=v_scale)
    return c


@pytest.mark.parametrize("name", ["Q8_0", "Q5_0", "Q4_0"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("v_scale", [1e-6, 1e-4])
def test_a_large_block_hidden_and_visible(gpu, name, d, v_scale):
    c = case(name, [100, 60], [4, 2], 4, 2, d, 32, 800 + d, v_scale)
    c["mask"][:4] = [0b0001, 0b0011, 0b0101, 0b1101]
    enlarge(c, 0, 101, 0, d // 32 - 1)        # drafted: token 1 alone sees it; its own channels and head 0 alone hold it
    enlarge(c, 1, 33, 1, 0)                   # committed: every token of request 1
    run(c, gpu)


def test_many_large_tiles_in_many_units(gpu):
    # Several units and tiles a CTA, large ones first, last, alone and in a row.
    rng = np.random.default_rng(5)
    ctx = rng.integers(300, 900, 40).tolist()
    c = case("Q8_0", ctx, [2] * 40, 4, 4, 64, 16, 820, 1e-4)
    for r in range(40):
        for t in range(-(-(ctx[r] + 2) // 128)):
            if rng.random() < 0.4 or r % 7 == 0:
                for _ in range(int(rng.integers(1, 4))):
                    enlarge(c, r, min(ctx[r] + 1, 128 * t + int(rng.integers(0, 128))), int(rng.integers(0, 4)), int(rng.integers(0, 2)))
    run(c, gpu)


def test_large_blocks_in_a_cut_unit_with_growing_references(gpu):
    c = case("Q4_0", [9000], [3], 4, 1, 128, 64, 830, 1e-5)
    c["q"] = c["q"] * 4
    for p in (3, 130, 2000, 2001, 8999, 9001):
        enlarge(c, 0, p, 0, p % 4)
    run(c, gpu)
