"""qk_attn_tree at the end of the positions that 32 bits count: what lies past
the last position it walks is reported like any other position without a
place, not dropped in silence.  Every table entry names the same page, so the
cache itself is small."""
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
from gpu_helpers import gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx", [2**31 - 100, 2**31 - 1])
def test_positions_past_the_last_are_reported(gpu, ctx):
    t, d, page = qk.Q4_0, 32, 256
    K, V = (torch.zeros((1, qk.kv_page_bytes(t, 1, d, page)), dtype=torch.uint8, device=gpu) for _ in range(2))
    V.view(page, d // 32 * 18)[:, 1] = 0x3C             # scale 1, codes 0: every value is -8
    table = torch.zeros((1, 2**31 // page), dtype=torch.int32, device=gpu)
    q = torch.zeros((1, 1, d), dtype=torch.bfloat16, device=gpu)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    out = qk.attn_tree(t, q, K, V, page, 1, table, i32(ctx), i32(0, 1), None, 1, 1.0)
    with pytest.raises(qk.QKError) as e:
        qk.device_status()
    assert e.value.status == 8
    qk.device_status()
    # the positions before it are walked: the mean of equal values, give or take fp32 sums of 2^31 of them (a CTA's
    # 110,377 tiles of at most 128 positions add to both sums in 16-position steps, each off by 2^-23 at worst)
    assert (out.float() + 8).abs().max() <= 8 * (2.0**-8 + 2 * 8 * 110377 * 2.0**-23)
