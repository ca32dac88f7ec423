"""Frequencies so low that 2^-96 of a turn, the unit of an angle, is a part of them."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
from gpu_helpers import gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [False, True])
def test_small_frequencies(gpu, pairs):
    freq = np.array([2.0**-40, 3e-13, 2.0**-56, 1e-20, 1e-25, -1e-30, 2.0**-126, 2.0**-149], np.float32)
    pos = np.array([0, 1, -5, 77, 2**31 - 1, -2**31], np.int64)
    x = torch.zeros((len(pos), 1, 32))
    x[:, :, 0:16:2 if pairs else 1] = 1.0
    if not pairs:
        x[:, :, 8:] = 0.0
    y = qk.norm_rope(x.to(gpu), None, torch.tensor(pos, dtype=torch.int32, device=gpu), torch.tensor(freq, device=gpu), pairs=pairs)[0]
    y = y[:, 0].cpu().double().numpy()
    cos, sin = (y[:, 0:16:2], y[:, 1:16:2]) if pairs else (y[:, :8], y[:, 8:16])
    a = pos[:, None].astype(np.float64) * freq.astype(np.float64)      # exact: 31 by 24 bits, or a power of two
    assert (np.abs(cos - np.cos(a)) <= 2.0**-24).all()
    # the unit, 2 pi 2^-96 below 2^-93, a position; up to four roundings of what lies below 2^-64 turns, 2 pi 2^-89 below 2^-86
    # each; half a step of fp32
    bound = 2.0**-24 * np.abs(np.sin(a)) + 2.0**-84 + np.abs(pos[:, None]) * 2.0**-93
    # from 2^-46 on half a step, and 2^-12 of it more
    low = np.abs(freq) < 2.0**-46
    bound[:, ~low] = 2.0**-24 * (1 + 2.0**-12) * np.abs(np.sin(a))[:, ~low]
    assert (np.abs(sin - np.sin(a)) <= bound).all()
    assert low.sum() == 6
