"""qk_kv_plan from two host threads at once, with batches that need different
amounts of shared memory: a call may not depend on what another asks for."""
import threading

import pytest
import torch

import gguf_quant_dequant_gb300 as qk
from gpu_helpers import gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def test_planning_from_two_threads(gpu):
    errors, rounds, start = [], 3000, threading.Barrier(2, timeout=120)

    def work(n):
        try:
            zeros, ones = torch.zeros(n, dtype=torch.int32, device=gpu), torch.ones(n, dtype=torch.int32, device=gpu)
            table, free = torch.full((n, 1), -1, dtype=torch.int32, device=gpu), torch.arange(n, dtype=torch.int32, device=gpu)
            n_free = torch.tensor([n], dtype=torch.int32, device=gpu)
            with torch.cuda.stream(torch.cuda.Stream()):
                torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
                out = qk.kv_plan(zeros, zeros, ones, table, free, n_free, 16, n)
                start.wait()
                for _ in range(rounds):
                    qk.kv_plan(zeros, zeros, ones, table, free, n_free, 16, n, out=out)
                torch.cuda.current_stream().synchronize()
                assert out["cu"][-1].item() == n and out["granted"].all()
        except Exception as e:   # noqa: BLE001  (reported by the main thread)
            errors.append((n, e))

    threads = [threading.Thread(target=work, args=(n,)) for n in (1, 8192)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
