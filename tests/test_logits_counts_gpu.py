"""qk_logits_process at the end of what it counts: a token that stands 2^20 - 1
times is exact; a request whose history and drafted chain could go past that is
reported, and its drafts are left out instead of spilling into the biases."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
from gpu_helpers import gpu  # noqa: F401

pytestmark = pytest.mark.gpu

H = (1 << 20) - 65          # the longest history row


def call(gpu, rows, bias, vocab=8, mask=None):
    x = torch.arange(rows * vocab, dtype=torch.float32, device=gpu).view(rows, vocab) / 8 + 1
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    f = lambda v: torch.tensor([v], device=gpu)  # noqa: E731
    kw = dict(bias_tok=i32(5).view(1, 1), bias_val=f(100.0).view(1, 1), bias_len=i32(0)) if bias else {}
    hist = torch.full((1, H), 3, dtype=torch.int32, device=gpu)
    y = qk.logits_process(x, i32(0, rows), hist, i32(H), f(1.0), f(0.0), f(2.0**-20), mask=mask,
                          draft=torch.full((rows,), 3, dtype=torch.int32, device=gpu), **kw)
    return x.cpu().numpy().astype(np.float64), y.cpu().numpy().astype(np.float64)


def expected(x, counts):
    y = x.copy()
    y[:, 3] -= 2.0**-20 * counts
    return y


@pytest.mark.parametrize("bias", [False, True])
def test_the_largest_count(gpu, bias):
    x, y = call(gpu, 64, bias)
    qk.device_status()
    ref = expected(x, H + 1 + np.arange(64))              # up to 2^20 - 1
    # freq * c is exact, the difference is rounded to fp32 once
    assert (np.abs(y - ref) <= 2.0**-24 * np.abs(ref)).all()


@pytest.mark.parametrize("bias", [True, False])
def test_more_than_can_be_counted_is_reported(gpu, bias):
    x, y = call(gpu, 100, bias)
    with pytest.raises(qk.QKError) as e:
        qk.device_status()
    assert e.value.status == 8 and "2^20" in str(e.value)
    qk.device_status()
    ref = expected(x, np.full(100, H))                    # the drafts are left out
    assert (np.abs(y - ref) <= 2.0**-24 * np.abs(ref)).all()


def test_masked_drafts_fit_whatever_the_rows(gpu):
    mask = torch.full((100,), -1, dtype=torch.int64, device=gpu)
    x, y = call(gpu, 100, True, mask=mask)                # 64 ancestors each: 2^20 - 1
    qk.device_status()
    ref = expected(x, np.full(100, H + 64))
    assert (np.abs(y - ref) <= 2.0**-24 * np.abs(ref)).all()
