"""qk_attn_tree when a wait runs out, without a GPU fault: the copies of V stop
at a given tile of each CTA and the wait for them is cut to a millisecond.  The
call returns, the status word says QK_ERR_TIMEOUT, nothing outside out and the
workspace is written, and the next call is right."""
import time

import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
from gpu_helpers import gpu, type_id  # noqa: F401
from test_tree_gpu import check, make, to_dev

pytestmark = pytest.mark.gpu

CASES = {                            # one cut unit; several whole units a CTA; a wide one; many small ones; d = 256
    "long": lambda: make("Q8_0", [9001], [3], 4, 1, 128, 64, 1000),
    "ragged": lambda: make("Q4_0", [900, 20, 333, 70] * 20, [3, 1, 2, 5] * 20, 8, 4, 64, 16, 1010),
    "wide": lambda: make("Q5_0", [700, 300], [64, 40], 32, 4, 64, 64, 1020),
    "short": lambda: make("Q8_0", [30] * 700, [1, 2] * 350, 4, 2, 32, 16, 1030),
    "d256": lambda: make("Q8_0", [500, 90] * 10, [4, 2] * 10, 8, 2, 256, 32, 1040),
}


def large_v(c):
    """Every third V row with blocks past fp16's range."""
    rows = c["V"].reshape(-1, c["V"].shape[-1])
    rows[::3, 1] = 0x70              # scales of 2^13 and more
    return c


def run_stalled(gpu, c, tile):
    dev = to_dev(c, gpu)
    n, heads, d = dev[0].shape
    need = qk.attn_tree_workspace(type_id(c["name"]), len(c["ctx"]), c["max_q"], c["table"].shape[1] * c["page"], heads, c["n_kv"], d)
    ws = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device=gpu)
    out = torch.full((n + 8, heads, d), 7.0, dtype=torch.bfloat16, device=gpu)
    t0 = time.perf_counter()
    qk.test_attn_tree_stalled(1000, tile, type_id(c["name"]), *dev, out=out[4:-4], ws=ws[4096:4096 + need])
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert (ws[:4096] == 0x5A).all() and (ws[4096 + need:] == 0x5A).all()
    assert (out[:4] == 7).all() and (out[-4:] == 7).all()
    return out[4:-4], took


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("name,tiles", [("long", [0]), ("ragged", [0, 1, 2, 3, 5]), ("wide", [0]), ("short", [0, 1, 2, 3, 4, 7]),
                                        ("d256", [0, 1])])
def test_a_wait_that_runs_out_is_reported(gpu, name, tiles, large):
    c = large_v(CASES[name]()) if large else CASES[name]()
    qk.device_status()
    for tile in tiles:
        out, took = run_stalled(gpu, c, tile)
        with pytest.raises(qk.QKError) as e:
            qk.device_status()
        assert e.value.status == 7
        assert took < 1.0                                   # a wait's limit and the way out, not the ordinary 2 s
        qk.device_status()                                  # cleared
    if not large:
        check(c, qk.attn_tree(type_id(c["name"]), *to_dev(c, gpu)))
        qk.device_status()


def test_a_tile_that_no_cta_reaches(gpu):
    c = CASES["ragged"]()
    out, _ = run_stalled(gpu, c, 10**6)
    qk.device_status()
    check(c, out)


@pytest.mark.parametrize("limit", [0, 2000001])
def test_limits(gpu, limit):
    with pytest.raises(qk.QKError) as e:
        qk.test_attn_tree_stalled(limit, 0, qk.Q8_0, *to_dev(make("Q8_0", [5], [1], 4, 1, 64, 16, 1050), gpu))
    assert e.value.status == 8
