"""qk_attn_tree with scales that leave no multiplier of the scores: zero, and
so small that scale times the query's power of two underflows.  Every visible
position then has the same weight, whatever is hidden beside it.  Against
paged_ref.py with the tolerance of test_tree_gpu.py."""
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
from gpu_helpers import gpu, type_id  # noqa: F401
from test_tree_gpu import make, run, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45])
@pytest.mark.parametrize("name,heads,n_kv,d", [("Q8_0", 8, 2, 128), ("Q5_0", 4, 4, 64), ("Q4_0", 8, 1, 256), ("Q8_0", 6, 2, 32)])
def test_scale_of_zero_is_the_plain_mean(gpu, name, heads, n_kv, d, scale):
    # partial tiles, hidden drafts, a request of drafts only, and (128 + 128 + 1 positions) a whole tile between others
    c = make(name, [77, 0, 256, 300], [5, 3, 1, 2], heads, n_kv, d, 32, 700 + d)
    c["scale"] = scale
    c["mask"][6] = 0                     # sees nothing: zeros
    out = run(c, gpu)
    assert not out[6].any()


@pytest.mark.parametrize("sign", [1, -1])
def test_tiny_queries_and_scale(gpu, sign):
    # scale 2^ex is below the smallest fp32 number, the scores are 0
    c = make("Q8_0", [130, 7], [5, 2], 8, 2, 64, 16, 710, q_scale=1e-38)
    c["scale"] = sign * 1e-9
    run(c, gpu)


def test_zero_scale_over_many_tiles(gpu):
    c = make("Q4_0", [5000], [4], 4, 1, 128, 64, 720)
    c["scale"] = 0.0
    run(c, gpu)


def test_zero_scale_of_a_non_finite_query(gpu):
    # 0 times infinity is NaN: its row, and no other
    c = make("Q8_0", [40], [3], 4, 2, 64, 16, 730)
    c["scale"] = 0.0
    dev = list(to_dev(c, gpu))
    clean = qk.attn_tree(qk.Q8_0, *dev)
    dev[0] = dev[0].clone()
    dev[0][1, 2, 7] = float("inf")
    out = qk.attn_tree(qk.Q8_0, *dev)
    assert torch.isnan(out[1, 2].float()).all()
    out[1, 2] = clean[1, 2]
    assert torch.equal(out, clean)
