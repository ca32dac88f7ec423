"""Calls given a stream that is not the current one: the tensors that a call
allocates for itself may neither be bytes that queued work of the current stream
still writes, nor be handed on while the call's kernels run."""
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import synth
from gpu_helpers import gpu  # noqa: F401
from test_tree_gpu import check, make, to_dev

pytestmark = pytest.mark.gpu

BUSY = 400_000_000               # clocks: a fifth of a second


def calls(gpu):
    """Calls by name, each on inputs of its own."""
    n, d, vocab, rows, cols = 700, 64, 4096, 512, 1024
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    W = torch.from_numpy(synth.random_blocks("Q8_0", rows, cols, 1)).to(gpu)
    x = torch.randn((3, cols), device=gpu)
    xb = x.to(torch.bfloat16)
    logits, hist = torch.randn((64, vocab), device=gpu), torch.randint(0, vocab, (1, 50), device=gpu).to(torch.int32)
    lists = (i32(0, 64), hist, i32(50), *(torch.full((1,), v, device=gpu) for v in (1.2, 0.3, 0.1)))
    table, free = torch.full((n, 4), -1, dtype=torch.int32, device=gpu), torch.arange(4 * n, dtype=torch.int32, device=gpu)
    zeros, wants, n_free = torch.zeros(n, dtype=torch.int32, device=gpu), torch.full((n,), 40, dtype=torch.int32, device=gpu), i32(4 * n)
    tree = to_dev(make("Q8_0", [300] * 40, [8] * 40, 8, 2, d, 16, 1100), gpu)
    return {
        "dequant": lambda **k: qk.dequant(qk.Q8_0, W, rows, cols, **k),
        "quantize": lambda **k: qk.quantize(qk.Q8_0, x, **k),
        "gemv": lambda **k: qk.gemv(qk.Q8_0, W, rows, cols, x, **k),
        "gemm": lambda **k: qk.gemm(qk.Q8_0, W, rows, cols, xb, **k),
        "logits_process": lambda **k: qk.logits_process(logits, *lists, **k),
        "kv_plan": lambda **k: qk.kv_plan(zeros, zeros, wants, table, free, n_free, 16, 40 * n, **k),   # repeatable
        "attn_tree": lambda **k: qk.attn_tree(qk.Q8_0, *tree, **k),
    }


def parts(r):
    return list(r.values()) if isinstance(r, dict) else [r]


@pytest.mark.parametrize("name", ["dequant", "quantize", "gemv", "gemm", "logits_process", "kv_plan", "attn_tree"])
def test_results_are_not_bytes_that_queued_work_still_writes(gpu, name):
    call = calls(gpu)[name]
    want = [t.clone() for t in parts(call())]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t).fill_(9) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in old:
        t.fill_(9)                   # runs after the sleep; by then the bytes are nobody's
    del old, t
    got = parts(call(stream=s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    qk.device_status()


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_the_workspace_stays_the_calls_until_it_has_run(gpu, how):
    # one long request: cut into a piece per SM, joined through the workspace
    c = make("Q8_0", [9001], [3], 4, 1, 64, 64, 1110)
    dev = to_dev(c, gpu)
    need = qk.attn_tree_workspace(qk.Q8_0, 1, 3, dev[5].shape[1] * 64, 4, 1, 64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    out = qk.attn_tree(qk.Q8_0, *dev, stream=s if how == "stream" else s.cuda_stream)
    for _ in range(4):               # the current stream goes on allocating and writing
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=gpu) for n in (need, need, max(need // 2, 1))]
        torch.cuda.current_stream().synchronize()
    torch.cuda.synchronize()
    del junk
    check(c, out)
    qk.device_status()


def test_default_stream_from_another_one(gpu):
    c = make("Q5_0", [500, 30], [4, 2], 8, 2, 64, 16, 1120)
    dev = to_dev(c, gpu)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out = qk.attn_tree(qk.Q5_0, *dev, stream=0)
        torch.cuda.default_stream().synchronize()
    check(c, out)


def test_a_dropped_result_waits_for_the_current_stream(gpu):
    # Used on the current stream and dropped: the next call's result may not overwrite it there.
    call = calls(gpu)["logits_process"]
    want = call()
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    a = call(stream=s)
    s.synchronize()
    torch.cuda._sleep(BUSY)
    kept = a + 0                     # reads a after the sleep
    del a
    with torch.cuda.stream(s):
        for _ in range(3):
            torch.empty_like(want).fill_(9)
    cur.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
