"""qk_attn_tree where a score has no finite value: cached K past fp16's range,
non-finite queries and scales.  The tokens that see such a score give NaN,
never a softmax without it; the others, and tokens that see nothing, are not
touched.  Against paged_ref.py with the tolerance of test_tree_gpu.py."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import paged_ref
from gpu_helpers import gpu, type_id  # noqa: F401
from test_tree_gpu import check, make, run, to_dev

pytestmark = pytest.mark.gpu

BB = {"Q8_0": 34, "Q5_0": 22, "Q4_0": 18}


def k_block(c, r, pos, g, blk):
    row = c["K"][c["table"][r, pos // c["page"]], g, pos % c["page"]]
    return row.reshape(-1, BB[c["name"]])[blk]


@pytest.mark.parametrize("q_value", [1e-6, -1e-6])
@pytest.mark.parametrize("name,scale,d", [("Q8_0", 1000.0, 64), ("Q8_0", 60000.0, 128), ("Q5_0", 6000.0, 64), ("Q4_0", 20000.0, 256)])
def test_k_past_half_precision(gpu, name, scale, d, q_value):
    # All codes of the block negative and the query of one sign, so that the overflowed score is one infinity.
    c = make(name, [21, 40], [6, 2], 4, 2, d, 16, 900)
    c["mask"][:6] = [1, 3, 7, 0b1001, 0b11001, 0b111111]
    c["q"] = torch.full_like(c["q"], q_value)
    ref = paged_ref.attn_tree(name, c["q"].double().numpy(), c["K"], c["V"], 16, 2, c["table"], c["ctx"], c["cu"], c["mask"], 6,
                              c["scale"])
    for g in range(2):
        b = k_block(c, 0, 23, g, 1)                     # drafted token 2: tokens 2 and 5 see it
        b[:] = 0x80 if name == "Q8_0" else 0            # the lowest code everywhere
        b[:2] = np.array([scale], np.float16).view(np.uint8)
    out = qk.attn_tree(type_id(name), *to_dev(c, gpu))
    qk.device_status()
    assert torch.isnan(out[[2, 5]].float()).all()
    others = [0, 1, 3, 4, 6, 7]
    check({**c, "q": c["q"][others]}, out[others], tuple(x[others] for x in ref))


def test_k_within_half_precision_under_a_large_scale(gpu):
    # Scales whose largest code would overflow, codes that do not: exact to the tolerance.
    c = make("Q8_0", [150], [3], 4, 1, 64, 16, 910, q_scale=1e-5)
    rng = np.random.default_rng(1)
    for p in range(0, 153, 5):
        b = k_block(c, 0, p, 0, p % 2)
        b[:2] = np.array([600.0], np.float16).view(np.uint8)
        b[2:] = rng.integers(-109, 110, 32).astype(np.int8).view(np.uint8)      # |w| <= 65400
    run(c, gpu)


@pytest.mark.parametrize("value", [np.inf, -np.inf])
def test_infinite_query_against_codes_of_one_sign(gpu, value):
    # Every score of the row is the same infinity: NaN, as for mixed ones.
    c = make("Q8_0", [140], [3], 4, 2, 64, 16, 920)
    codes = c["K"].reshape(-1, 34)[:, 2:].view(np.int8)
    codes[:] = np.maximum(np.abs(codes.astype(np.int16)), 1).clip(1, 127).astype(np.int8)
    d = c["K"].reshape(-1, 34)[:, :2].copy().view(np.float16)
    c["K"].reshape(-1, 34)[:, :2] = np.maximum(d, np.float16(1e-3)).view(np.uint8)
    c["mask"][:] = [1, 3, 0]
    dev = list(to_dev(c, gpu))
    ref = qk.attn_tree(qk.Q8_0, *dev)
    check(c, ref)
    dev[0] = dev[0].clone()
    dev[0][1, 3, 9] = float(value)
    out = qk.attn_tree(qk.Q8_0, *dev)
    assert torch.isnan(out[1, 3].float()).all()
    out[1, 3] = ref[1, 3]
    assert torch.equal(out, ref)
    # a row that sees nothing gives zeros, whatever its query holds
    c = make("Q8_0", [0], [3], 4, 2, 64, 16, 921)
    c["mask"][:] = [1, 0, 5]
    dev = list(to_dev(c, gpu))
    ref = qk.attn_tree(qk.Q8_0, *dev)
    dev[0] = dev[0].clone()
    dev[0][1, 3, 9] = float(value)
    out = qk.attn_tree(qk.Q8_0, *dev)
    assert torch.equal(out, ref) and not out[1].any()


@pytest.mark.parametrize("scale", [np.inf, -np.inf, np.nan])
def test_non_finite_scale(gpu, scale):
    c = make("Q8_0", [0, 90], [3, 2], 4, 2, 64, 16, 930)
    c["mask"][:3] = [1, 0, 7]
    c["scale"] = scale
    out = qk.attn_tree(qk.Q8_0, *to_dev(c, gpu)).float()
    qk.device_status()
    assert torch.isnan(out[[0, 2, 3, 4]]).all() and not out[1].any()
