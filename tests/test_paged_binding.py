"""What the binding of the paged calls refuses before anything reaches the C
side: memory that is not the GPU's, and, on CUDA tensors, wrong types, counts
and strides.  Each refusal names its reason."""
import pytest
import torch

import gguf_quant_dequant_gb300 as qk


@pytest.fixture(scope="module")
def lib():
    from gguf_quant_dequant_gb300 import build
    build.build()
    return qk.load()


def calls(dev):
    """name: (call, its arguments, all valid but for where they lie)."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    pool = lambda: torch.zeros(4 * qk.kv_page_bytes(qk.Q8_0, 2, 64, 16), dtype=torch.uint8, device=dev)  # noqa: E731
    f = lambda: torch.ones(2, device=dev)  # noqa: E731
    n = 3
    ws = qk.attn_tree_workspace(qk.Q8_0, 2, 2, 64, 4, 2, 64)
    bf = lambda: torch.zeros(n, 4, 64, dtype=torch.bfloat16, device=dev)  # noqa: E731
    i64 = lambda: torch.zeros(n, dtype=torch.int64, device=dev)  # noqa: E731
    return {
        "kv_append": (qk.kv_append, dict(t=qk.Q8_0, k=torch.zeros(n, 2, 64, device=dev), v=torch.zeros(n, 2, 64, device=dev),
                                         slots=i64() - 1, K=pool(), V=pool(), page=16)),
        "kv_compact": (qk.kv_compact, dict(t=qk.Q8_0, K=pool(), V=pool(), page=16, n_kv=2, d=64, table=i32(2, 4), base=i32(2),
                                           path=i32(2, 3), n_path=i32(2))),
        "kv_plan": (qk.kv_plan, dict(have=i32(2), start=i32(2), want=i32(2), table=i32(2, 4), free_pages=i32(9), n_free=i32(1), page=16,
                                     cap=8)),
        "attn_tree": (qk.attn_tree, dict(t=qk.Q8_0, q=bf(), K=pool(), V=pool(), page=16, n_kv=2, table=i32(2, 4), ctx=i32(2), cu=i32(3),
                                         mask=i64(), max_q=2, scale=0.1, out=bf(),
                                         ws=torch.zeros(max(ws, 16), dtype=torch.uint8, device=dev))),
        "logits_process": (qk.logits_process, dict(logits=torch.zeros(n, 50, device=dev), cu=i32(3), hist=i32(2, 5), hist_len=i32(2),
                                                   rep=f(), pres=f(), freq=f(), draft=i32(n), mask=i64(), bias_tok=i32(2, 1),
                                                   bias_val=torch.zeros(2, 1, device=dev), bias_len=i32(2), grammar=i32(n, 2),
                                                   out=torch.zeros(n, 50, device=dev))),
    }


def refused(name, status, words, dev="cpu", **change):
    fn, args = calls(dev)[name]
    with pytest.raises(qk.QKError, match=words) as e:
        fn(**{**args, **change}, stream=0 if dev == "cpu" else None)
    assert e.value.status == status and name in str(e.value)


@pytest.mark.parametrize("name", ["kv_append", "kv_compact", "kv_plan", "attn_tree", "logits_process"])
def test_host_memory_is_refused(lib, name):
    refused(name, 8, "CUDA tensor expected")


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["kv_append", "kv_compact", "kv_plan", "attn_tree", "logits_process"])
def test_each_tensor_on_the_host_is_refused(name):
    fn, args = calls("cuda")[name]
    fn(**args)                                   # valid as it stands
    qk.device_status()
    tensors = [k for k, v in args.items() if torch.is_tensor(v)]
    assert len(tensors) >= 5
    for k in tensors:
        refused(name, 8, "CUDA tensor expected", "cuda", **{k: args[k].cpu()})
    qk.device_status()


@pytest.mark.gpu
def test_wrong_cuda_tensors_are_refused():
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    f32, i64, bf = torch.float32, torch.int64, torch.bfloat16
    for name, status, words, change in [
            ("kv_append", 8, "float16", dict(k=z(3, 2, 64, t=torch.float16), v=z(3, 2, 64, t=torch.float16))),
            ("kv_append", 2, "k and v differ", dict(v=z(2, 2, 64, t=f32))),
            ("kv_append", 8, "contiguous rows", dict(k=z(3, 64, 2, t=f32).transpose(1, 2))),
            ("kv_append", 8, "int64 expected", dict(slots=z(3))),
            ("kv_append", 2, "whole number", dict(K=z(100, t=torch.uint8))),
            ("kv_compact", 2, "8 elements", dict(table=z(2, 5)[:, :4].contiguous()[:1])),
            ("kv_plan", 8, "int32 expected", dict(want=z(2, t=i64))),
            ("kv_plan", 2, "2 elements", dict(start=z(3))),
            ("attn_tree", 8, "q must be bfloat16", dict(q=z(3, 4, 64, t=f32))),
            ("attn_tree", 8, "int64 expected", dict(mask=z(3))),
            ("attn_tree", 2, "3 elements", dict(cu=z(2))),
            ("attn_tree", 2, "out must", dict(out=z(3, 4, 32, t=bf))),
            ("attn_tree", 8, "contiguous ws", dict(ws=z(1, t=torch.uint8).expand(1 << 20))),
            ("attn_tree", 8, "contiguous ws", dict(ws=z(1 << 20, t=torch.uint8)[::2])),
            ("attn_tree", 5, "workspace", dict(ws=z(16, t=torch.uint8))),
            ("attn_tree", 2, "bad attention shape", dict(max_q=65)),
            ("logits_process", 8, "float64", dict(rep=torch.ones(2, dtype=torch.float64, device="cuda"))),
            ("logits_process", 2, "10 elements", dict(hist=z(3, 5))),
            ("logits_process", 8, "contiguous rows", dict(logits=z(50, 3, t=f32).t(), out=None))]:
        refused(name, status, words, "cuda", **change)
    qk.device_status()
