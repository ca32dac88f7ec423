"""Refusals of the head norms, rotation, append and verification calls: on the
host, before anything is queued (no GPU needed)."""
import ctypes

import pytest
import torch

import gguf_quant_dequant_gb300 as qk

F = 0x10000                       # 16-byte aligned, never dereferenced
SHAPE, ALIGN, NULL, ARG, TYPE = 2, 3, 4, 8, 1


@pytest.fixture(scope="module")
def lib():
    from gguf_quant_dequant_gb300 import build
    build.build()
    return qk.load()


def call(fn, base, **kw):
    args = dict(base)
    unknown = set(kw) - set(args)
    assert not unknown, unknown
    args.update(kw)
    return fn(*args.values())


ROPE = dict(q=F, k=F, dtype=0, n_tok=4, q_stride=512, k_stride=128, n_heads=4, n_kv=1, d=128, pos=F, q_norm=F, k_norm=F,
            eps=1e-6, freq=F, rot=64, pairs=0, q_out=F + 4096, k_out=F + 8192, out_dtype=1, qo_stride=512, ko_stride=128, stream=None)
APPEND = dict(type=qk.Q8_0, q=F, k=F, v=F, dtype=0, n_tok=4, q_stride=512, k_stride=128, v_stride=128, n_heads=4, n_kv=1, d=128,
              pos=F, q_norm=F, k_norm=F, eps=1e-6, freq=F, rot=64, pairs=0, slots=F, K=F, V=F, n_pages=3, page=16, q_out=F + 4096,
              q_out_stride=512, stream=None)
BOTH = [(dict(d=96), SHAPE), (dict(rot=8), SHAPE), (dict(rot=144), SHAPE), (dict(rot=-16), SHAPE), (dict(n_tok=-1), SHAPE),
        (dict(n_tok=1 << 31), SHAPE), (dict(n_heads=-1), SHAPE), (dict(n_heads=70000), SHAPE), (dict(q_stride=511), SHAPE),
        (dict(k_stride=127), SHAPE), (dict(q_stride=1 << 31), SHAPE), (dict(dtype=2), ARG), (dict(eps=-1.0), ARG),
        (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(q=None), NULL), (dict(k=None), NULL), (dict(pos=None), NULL),
        (dict(freq=None), NULL), (dict(q_out=None), NULL), (dict(q=F + 2), ALIGN), (dict(k=F + 2), ALIGN), (dict(pos=F + 2), ALIGN),
        (dict(freq=F + 1), ALIGN), (dict(q_norm=F + 2), ALIGN), (dict(k_norm=F + 2), ALIGN), (dict(q_out=F + 1), ALIGN),
        (dict(q_out=F), ARG)]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(out_dtype=7), ARG), (dict(qo_stride=511), SHAPE), (dict(ko_stride=127), SHAPE), (dict(k_out=None), NULL),
    (dict(k_out=F + 1), ALIGN), (dict(k_out=F), ARG), (dict(q_out=F, out_dtype=0, qo_stride=640), ARG)])
def test_norm_rope_refusals(lib, kw, status):
    assert call(lib.qk_norm_rope, ROPE, **kw) == status
    assert lib.qk_last_error()


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(type=qk.Q4_K), TYPE), (dict(n_kv=0), SHAPE), (dict(page=24), SHAPE), (dict(n_pages=-1), SHAPE), (dict(K=None), NULL),
    (dict(V=F + 8), ALIGN), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(slots=F + 4), ALIGN), (dict(v=F + 2), ALIGN),
    (dict(v_stride=127), SHAPE), (dict(q_out_stride=511), SHAPE)])
def test_kv_append_rope_refusals(lib, kw, status):
    assert call(lib.qk_kv_append_rope, APPEND, **kw) == status
    assert lib.qk_last_error()


def test_nothing_to_do(lib):
    assert call(lib.qk_norm_rope, ROPE, n_tok=0, q=None, pos=None) == 0
    assert call(lib.qk_norm_rope, ROPE, n_heads=0, n_kv=0, q=None, k=None) == 0
    assert call(lib.qk_kv_append_rope, APPEND, n_tok=0, q=None, v=None) == 0
    assert call(lib.qk_verify_tree, VERIFY, n_req=0, logits=None, ws=None) == 0
    assert [qk.verify_workspace(*a) for a in ((6, 2, 100), (6, 2, 1025), (2, 2, 100), (0, 1, 9), (-1, 1, 9), (6, 0, 9))] == \
        [6 * 16, 6 * 2 * 16, 0, 0, 0, 0]


VERIFY = dict(logits=F, dtype=0, n_rows=6, vocab=100, row_stride=100, cu=F, n_req=2, draft=F, mask=F, temp=F, u_accept=F, u_sample=F,
              probs=F, probs_stride=100, path=F, path_stride=8, n_path=F, tokens=F, ws=F, ws_bytes=96, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), ARG), (dict(n_rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=1 << 31), SHAPE), (dict(n_req=-1), SHAPE),
    (dict(n_req=(1 << 27) + 1), SHAPE), (dict(path_stride=0), SHAPE), (dict(row_stride=99), SHAPE), (dict(probs_stride=99), SHAPE),
    (dict(logits=None), NULL), (dict(cu=None), NULL), (dict(draft=None), NULL), (dict(temp=None), NULL), (dict(u_accept=None), NULL),
    (dict(u_sample=None), NULL), (dict(path=None), NULL), (dict(n_path=None), NULL), (dict(tokens=None), NULL),
    (dict(logits=F + 2), ALIGN), (dict(mask=F + 4), ALIGN), (dict(probs=F + 2), ALIGN), (dict(path=F + 2), ALIGN), (dict(ws=None), NULL),
    (dict(ws=F + 8), ALIGN), (dict(ws_bytes=95), 5)])
def test_verify_tree_refusals(lib, kw, status):
    assert call(lib.qk_verify_tree, VERIFY, **kw) == status
    assert lib.qk_last_error()


def test_binding_refusals(lib):
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)  # noqa: E731
    i32 = torch.int32
    q, k, pos, freq = z(3, 4, 64), z(3, 2, 64), z(3, dtype=i32), z(32)

    def refused(status, fn, *a, **kw):
        with pytest.raises(qk.QKError) as e:
            fn(*a, **kw)
        assert e.value.status == status, e.value

    refused(4, qk.norm_rope, None, None, pos, freq)
    refused(2, qk.norm_rope, q, z(3, 2, 32), pos, freq)
    refused(2, qk.norm_rope, q, k.to(torch.bfloat16), pos, freq)
    refused(2, qk.norm_rope, q, k, pos, freq, q_out=z(3, 4, 32))
    refused(2, qk.norm_rope, q, k, pos, freq, out_dtype=torch.bfloat16, q_out=z(3, 4, 64))
    refused(8, qk.norm_rope, q.transpose(1, 2), None, pos, freq)          # rows that are not contiguous
    refused(8, qk.norm_rope, q.half(), None, pos, freq)
    refused(8, qk.norm_rope, q, k, pos, freq)                             # host tensors
    pool = z(1, qk.kv_page_bytes(qk.Q8_0, 2, 64, 16), dtype=torch.uint8)
    slots = z(3, dtype=torch.int64)
    refused(2, qk.kv_append_rope, qk.Q8_0, q, k, z(3, 2, 32), pos, freq, slots, pool, pool, 16)
    refused(2, qk.kv_append_rope, qk.Q8_0, z(2, 4, 64), k, k, pos, freq, slots, pool, pool, 16)
    refused(2, qk.kv_append_rope, qk.Q8_0, q, k, k, pos, freq, slots, pool, pool, 24)
    refused(8, qk.kv_append_rope, qk.Q8_0, q, k, k, pos, freq, slots, pool, pool, 16)
    x, cu = z(4, 10), z(3, dtype=i32)
    args = (z(4, dtype=i32), z(4, dtype=torch.int64), z(2), z(4), z(2))
    refused(2, qk.verify_tree, x, cu, *args, probs=z(4, 9))
    refused(2, qk.verify_tree, x, cu, *args, probs=z(4, 10, dtype=torch.float64))
    refused(8, qk.verify_tree, x, cu, *args)


def test_signatures_are_the_header_s(lib):
    assert ctypes.sizeof(ctypes.c_void_p) == 8
    for name, n in (("qk_norm_rope", len(ROPE)), ("qk_kv_append_rope", len(APPEND)), ("qk_verify_tree", len(VERIFY))):
        assert len(qk.SIGNATURES[name][1]) == n


MOE = dict(type=qk.Q4_K, Wg=F, Wu=F, type_down=qk.Q6_K, Wd=F, n_exp=8, rows=512, cols=256, router=F, k=2, norm=1, scale=1.0, x=F,
           n_tok=3, ids=F, gate=F, out=F, ws=F, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=0), TYPE), (dict(type_down=9), TYPE), (dict(n_exp=0), SHAPE), (dict(n_exp=513), SHAPE), (dict(k=0), SHAPE),
    (dict(k=9), SHAPE), (dict(n_exp=64, k=17), SHAPE), (dict(rows=0), SHAPE), (dict(rows=500), SHAPE), (dict(cols=300), SHAPE),
    (dict(cols=0), SHAPE), (dict(rows=(1 << 16) + 256), SHAPE), (dict(cols=(1 << 16) + 256), SHAPE), (dict(n_tok=65), SHAPE),
    (dict(n_tok=-1), SHAPE), (dict(scale=float("nan")), ARG), (dict(Wg=None), NULL), (dict(Wu=None), NULL), (dict(Wd=None), NULL),
    (dict(x=None), NULL), (dict(ids=None), NULL), (dict(gate=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(Wg=F + 8), ALIGN), (dict(router=F + 4), ALIGN), (dict(x=F + 8), ALIGN), (dict(ws=F + 8), ALIGN), (dict(ids=F + 2), ALIGN),
    (dict(out=F + 1), ALIGN), (dict(ws_bytes=100), 5)])
def test_moe_ffn_refusals(lib, kw, status):
    assert call(lib.qk_moe_ffn, MOE, **kw) == status
    assert lib.qk_last_error()


def test_moe_sizes_and_binding_refusals(lib):
    assert len(qk.SIGNATURES["qk_moe_ffn"][1]) == len(MOE)
    assert qk.moe_workspace(qk.Q4_K, qk.Q6_K, 8, 512, 256, 2, 3) >= 3 * 2 * (2 * 512 + 256) * 4
    for bad in ((qk.Q4_K, qk.Q6_K, 8, 512, 256, 2, 65), (qk.Q4_K, qk.Q6_K, 8, 512, 256, 9, 3), (0, qk.Q6_K, 8, 512, 256, 2, 3),
                (qk.Q4_K, qk.Q6_K, 8, 512, 300, 2, 3)):
        assert qk.moe_workspace(*bad) == 0
    assert call(lib.qk_moe_ffn, MOE, n_tok=0, x=None, ws=None, ws_bytes=0) == 0
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    up, down, x = 2 * 512 * 144, 2 * 256 * 420, torch.zeros((3, 256))
    args = (qk.Q4_K, u8(up), u8(up), qk.Q6_K, u8(down), 2, 512, 256)

    def refused(status, *a, **kw):
        with pytest.raises(qk.QKError) as e:
            qk.moe_ffn(*a, **kw)
        assert e.value.status == status, e.value

    refused(4, *args, x, 2)
    refused(2, *args[:6], 500, 256, x, 2, router=torch.zeros((2, 256)))
    refused(2, qk.Q4_K, u8(up - 1), *args[2:], x, 2, router=torch.zeros((2, 256)))
    refused(8, *args, x, 2, router=torch.zeros((2, 256)))          # host tensors
