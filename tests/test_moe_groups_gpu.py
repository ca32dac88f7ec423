"""The expert products of every type, with groups of four and of eight pairs:
within the elementwise bound of their other tests, and in the norm.

In the norm: a product's roundings (fp16 pairs for x, blocks, slices: up to 2^7 of
them, 2^-25 of a partial sum each) are independent of one another and add as
squares, 2^-21.5; partial sums of raw codes are up to twice as large as those of
the weights; two such stages in a row (gate and up, down) give sqrt(2) 2^-20.5 =
2^-20 of the layer's norm.  x without its second fp16 term is 2^-12 off."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import synth
from gpu_helpers import dev_f32, dev_u8, gpu, type_id  # noqa: F401
from test_moe_gpu import layer, reference

NORM = 2.0**-20
SMS = 152

BIG = [  # n, experts, k, cols, rows, up, down: groups of eight in both products
    (21, 2, 1, 2048, 2304, "Q4_K", "Q4_K"),
    (14, 3, 2, 2304, 2048, "Q6_K", "Q6_K"),
    (29, 2, 1, 1056, 2080, "Q8_0", "Q8_0"),
    (15, 2, 2, 2080, 1120, "Q5_0", "Q5_0"),
    (13, 2, 2, 2208, 1184, "Q4_0", "Q4_0"),
    (61, 3, 1, 1536, 2560, "Q5_K", "Q5_K"),
    (23, 2, 2, 2560, 1024, "Q2_K", "Q2_K"),
    (64, 2, 1, 1024, 3328, "Q3_K", "Q3_K"),
]
SMALL = [  # groups of four in both products
    (4, 3, 2, 1056, 544, "Q8_0", "Q5_0"),
    (3, 2, 2, 544, 1056, "Q5_0", "Q4_0"),
    (4, 2, 1, 288, 800, "Q4_0", "Q8_0"),
    (4, 3, 2, 1024, 512, "Q2_K", "Q4_K"),
    (2, 4, 3, 512, 1280, "Q3_K", "Q6_K"),
    (4, 2, 2, 768, 768, "Q4_K", "Q5_K"),
    (3, 5, 2, 1280, 256, "Q5_K", "Q2_K"),
    (4, 2, 2, 256, 1024, "Q6_K", "Q3_K"),
]


def group(case, down, sms):
    n, E, k, cols, rows, up, dn = case
    return qk.load().qk_test_moe_group(type_id(up), type_id(dn), E, rows, cols, k, n, down, sms)


def test_every_kernel_is_reached():
    from gguf_quant_dequant_gb300 import build
    build.build()
    assert all(group(c, down, SMS) == 8 for c in BIG for down in (0, 1))
    assert all(group(c, down, SMS) == 4 for c in SMALL for down in (0, 1))
    for cases in (BIG, SMALL):
        assert {c[5] for c in cases} == {c[6] for c in cases} == set(synth.TYPE_IDS)
    assert group((65, 2, 2, 256, 256, "Q4_K", "Q4_K"), 0, SMS) == group((0, 2, 2, 256, 256, "Q4_K", "Q4_K"), 0, SMS) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("case", BIG + SMALL)
def test_products(gpu, case, near):
    n, E, k, cols, rows, up, down = case
    assert [group(case, d, 0) for d in (0, 1)] == [8 if case in BIG else 4] * 2
    W = layer(900 + n + rows, E, rows, cols, up, down)
    x = synth.activations(n, cols, 55 + n)
    if near:          # a step of 2^-12 from fp16 numbers, all to the same side
        x = (x.astype(np.float16).astype(np.float32) * np.float32(1 + 2.0**-12)).astype(np.float32)
    rng = np.random.default_rng(n + E)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    gate = synth.activations(n, k, 56 + n)
    out, _, _ = qk.moe_ffn(type_id(up), dev_u8(W[0], gpu), dev_u8(W[1], gpu), type_id(down), dev_u8(W[2], gpu), E, rows, cols,
                           dev_f32(x, gpu), k, ids=torch.from_numpy(ids).to(gpu), gate=dev_f32(gate, gpu))
    out = out.cpu().numpy()
    ref, tol = reference(W, E, rows, cols, up, down, x, ids, gate)
    assert (np.abs(out - ref) <= tol).all()
    off = np.linalg.norm(out - ref) / np.linalg.norm(ref)
    assert off <= NORM, off
    if case is SMALL[0]:          # the bound sees a product of fp16 x
        coarse, _ = reference(W, E, rows, cols, up, down, x.astype(np.float16).astype(np.float32), ids, gate)
        assert np.linalg.norm(coarse - ref) > 2**6 * NORM * np.linalg.norm(ref)
    qk.device_status()
