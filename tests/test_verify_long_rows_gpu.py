"""Tree verification where a thread's part of a row does not fit its registers
(more than 32 logits: large vocabularies, or batches whose requests get few CTAs),
so that rows are read again for each sum: the walk replayed, and sums of more
weights than one running word holds."""
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import test_verify_sums_gpu
from gpu_helpers import gpu  # noqa: F401
from test_verify_gpu import check, make, run

pytestmark = pytest.mark.gpu
SMS = 152


def logits_of_a_thread(n_req, V, dtype, vec):
    """The launch's geometry: CTAs of a request (16 warps each), then whole steps of 16 bytes a lane for each warp."""
    cluster = max(1, min(8, 2 * SMS // n_req, V // 1024))
    step = 32 * ((8 if dtype is torch.bfloat16 else 4) if vec else 1)
    return -(-V // (16 * cluster) // step) * step // 32


CASES = [  # sizes, vocab, drafter, dtype
    ([3] * 40, 128256, True, torch.float32),
    ([3] * 40, 128256, False, torch.float32),
    ([4, 2] * 20, 128256, True, torch.bfloat16),
    ([12], 151936, True, torch.float32),
    ([9], 151936, False, torch.bfloat16),
    ([9], 151936, True, torch.bfloat16),
    ([7, 5], 256000, True, torch.float32),
    ([12], 140001, True, torch.float32),
    ([12], 140001, True, torch.bfloat16),
    ([8], 151935, False, torch.bfloat16),
    ([8], 140003, False, torch.float32),
    ([3] * 320, 17000, True, torch.float32),
    ([3] * 320, 17003, True, torch.float32),
    ([2] * 320, 17008, False, torch.bfloat16),
    ([2] * 320, 17001, True, torch.bfloat16),
]


@pytest.mark.parametrize("sizes,V,drafter,dtype", CASES)
@pytest.mark.parametrize("refused", [False, True])
def test_walk(gpu, sizes, V, drafter, dtype, refused):
    assert logits_of_a_thread(len(sizes), V, dtype, V % (8 if dtype is torch.bfloat16 else 4) == 0) > 32
    s = make(60 + V + len(sizes), sizes, V, drafter, False, dtype)
    if refused:          # the first node behind every root never, the others as they come
        at = s["cu"][:-1].long() + 1
        s["u_accept"][at[torch.tensor(sizes) > 1]] = 1e9
    out = run(gpu, s)
    check(s, out)
    again = run(gpu, s)
    assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n_req", [(151936, 2), (5000, 2)])
@pytest.mark.parametrize("shift", [0, 1])
def test_drafter_rows_off_boundaries(gpu, V, n_req, dtype, shift):
    """Logits on 16-byte boundaries, the drafter's rows not: by their stride, or by their start too."""
    s = make(90 + V, [6] * n_req, V, True, False, dtype)
    s["u_accept"][1::6] = 1e9
    want = run(gpu, s)
    check(s, want)
    wide = torch.full((6 * n_req, V + 5), float("nan"), device=gpu)
    probs = wide[:, shift:shift + V]
    probs.copy_(s["probs"])
    assert probs.stride(0) % 4 and (probs.data_ptr() % 16 != 0) == bool(shift)
    d = {k: v.to(gpu) for k, v in s.items()}
    out = qk.verify_tree(d["logits"], d["cu"], d["draft"], d["mask"], d["temp"], d["u_accept"], d["u_sample"], probs=probs)
    assert all(torch.equal(out[k], want[k]) for k in out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [240000, 240002])
def test_more_weights_than_a_word_holds(gpu, V, dtype):
    """One CTA a request: 469 weights and more a thread."""
    assert logits_of_a_thread(160, V, dtype, V == 240000) > 447
    test_verify_sums_gpu.test_equal_halves(gpu, V, 160, dtype)


def test_greedy(gpu):
    for V, dtype in ((151936, torch.float32), (151936, torch.bfloat16), (140001, torch.float32), (140001, torch.bfloat16)):
        s = make(95, [5, 7], V, False, False, dtype)
        s["temp"][:] = 0.0
        top = s["logits"].float().argmax(1)
        s["draft"][1:4] = top[0]
        s["logits"][6, V - 1] = s["logits"][6, V - 9] = s["logits"].max() + 1     # equals: the lowest token
        out = run(gpu, s)
        check(s, out)
        assert out["n_path"][0] > 1
