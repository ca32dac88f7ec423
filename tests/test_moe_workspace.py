"""The workspace that moe_ffn takes for itself is the one its call's device asks
for: sizes of another device, or of a call that failed, are not used again (a
stand-in for the library, no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch

import gguf_quant_dequant_gb300 as qk


class Library:
    """Devices whose layers need 1000 bytes times their factor; unknown ones are taken for a device of factor 1."""

    def __init__(self):
        self.factor, self.known, self.asked = 1, True, 0

    def qk_row_bytes(self, t, cols):
        return cols

    def qk_last_error(self):
        return b"stand-in"

    def qk_moe_workspace(self, *sizes):
        self.asked += 1
        return 1000 * (self.factor if self.known else 1)

    def qk_moe_ffn(self, *a):
        if not self.known:
            return 6
        return 0 if a[-2] >= 1000 * self.factor else 5


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(qk, "load", lambda: lib)
    monkeypatch.setattr(qk, "_of", lambda x, *a: 0)
    monkeypatch.setattr(qk, "_stream_on", lambda x, stream: 0)
    monkeypatch.setattr(qk, "_empty", lambda size, dtype, like, stream, kept=True: torch.empty(size, dtype=dtype))
    qk._moe_bytes.cache_clear()
    yield lib
    qk._moe_bytes.cache_clear()
    getattr(qk, "_moe_need", {}).clear()


def call(device):
    x = SimpleNamespace(shape=(3, 256), device=SimpleNamespace(index=device))
    return qk.moe_ffn(qk.Q4_K, None, None, qk.Q6_K, None, 8, 512, 256, x, 2, router=x)


def test_two_devices(lib):
    call(0)
    lib.factor = 3
    call(1)
    lib.factor = 1
    call(0)
    assert lib.asked == 2          # a size that served is kept


def test_a_device_that_was_not_known_yet(lib):
    lib.factor, lib.known = 2, False
    with pytest.raises(qk.QKError) as e:
        call(0)
    assert e.value.status == 6
    lib.known = True
    call(0)


def test_many_sizes(lib):
    for n in range(1, 65):
        for k in range(1, 9):
            x = SimpleNamespace(shape=(n, 256), device=SimpleNamespace(index=0))
            qk.moe_ffn(qk.Q4_K, None, None, qk.Q6_K, None, 8, 512, 256, x, k, router=x)
    assert len(qk._moe_need) <= 256
