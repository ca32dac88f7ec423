"""The paged KV-cache, tree-attention and logits calls without a GPU: sizes,
refusals on the host (no compute call is made), the binding's own checks, and
the tests' plain implementations against the oracle and each other."""
import ctypes

import numpy as np
import pytest
import torch

import gguf_quant_dequant_gb300 as qk
import oracle
import paged_ref
import synth

OK, TYPE, SHAPE, ALIGN, NULL, WORKSPACE, ARG = 0, 1, 2, 3, 4, 5, 8
A16, A8, A4, A2, A1 = (ctypes.c_void_p(v) for v in (0x10000, 0x10008, 0x10004, 0x10002, 0x10001))   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gguf_quant_dequant_gb300 import build
    build.build()
    return qk.load()


class refused:
    """The block raises QKError, and for the arguments, not for want of a GPU."""

    def __enter__(self):
        self.raises = pytest.raises(qk.QKError)
        self.info = self.raises.__enter__()

    def __exit__(self, *exc):
        caught = self.raises.__exit__(*exc)
        assert self.info.value.status in (TYPE, SHAPE, ALIGN, NULL, WORKSPACE, ARG), self.info.value
        return caught


def call(fn, good, **change):
    args = dict(good, **change)
    return fn(*args.values())


def test_page_bytes(lib):
    assert qk.kv_page_bytes(qk.Q8_0, 8, 128, 16) == 8 * 16 * 136
    assert qk.kv_page_bytes(qk.Q5_0, 1, 32, 256) == 256 * 22
    for name in ("Q8_0", "Q5_0", "Q4_0"):
        for d in (32, 64, 128, 256):
            for page in (16, 32, 64, 128, 256):
                assert qk.kv_page_bytes(qk.TYPES[name], 1, d, page) % 16 == 0   # every (page, head) slab is
    for bad in ((qk.Q4_K, 8, 128, 16), (qk.Q8_0, 0, 128, 16), (qk.Q8_0, 8, 96, 16), (qk.Q8_0, 8, 128, 8),
                (qk.Q8_0, 8, 128, 48), (qk.Q8_0, 8, 128, 512), (qk.Q8_0, 4097, 128, 16)):
        assert qk.kv_page_bytes(*bad) == 0


def test_plan_refusals(lib):
    good = dict(have=A4, start=A4, want=A4, n_req=4, page=16, table=A4, stride=8, free=A4, cap_f=9, n_free=A4, n_out=A16,
                granted=A4, cu=A4, slots=A8, pos=None, req=None, cap=0, stream=None)
    f = lib.qk_kv_plan
    assert call(f, good, n_req=-1) == SHAPE
    assert call(f, good, n_req=8193) == SHAPE
    assert call(f, good, page=24) == SHAPE
    for k in ("stride", "cap_f", "cap"):
        assert call(f, good, **{k: -1}) == SHAPE
        assert call(f, good, **{k: 1 << 31}) == SHAPE
    for k in ("have", "start", "want", "table", "free", "n_free", "n_out", "granted", "cu"):
        assert call(f, good, **{k: None}) == NULL, k
        assert call(f, good, **{k: A2}) == ALIGN, k
    assert call(f, good, cap=5, slots=None) == NULL
    assert call(f, good, slots=A4) == ALIGN
    assert call(f, good, pos=A2) == ALIGN and call(f, good, req=A1) == ALIGN
    assert call(f, good, n_out=A4) == ARG
    assert b"n_free_out" in lib.qk_last_error()


def test_append_refusals(lib):
    good = dict(t=qk.Q8_0, k=A16, v=A16, dtype=0, n=5, ks=1024, vs=1024, n_kv=8, d=128, slots=A8, K=A16, V=A16, pages=4,
                page=16, stream=None)
    f = lib.qk_kv_append
    for t in (0, qk.Q4_K, qk.Q6_K, 9):
        assert call(f, good, t=t) == TYPE
    for k, v in (("d", 96), ("d", 512), ("n_kv", 0), ("n_kv", 4097), ("page", 17), ("pages", -1), ("n", -1), ("ks", 1023), ("vs", 0),
                 ("n", 1 << 40)):
        assert call(f, good, **{k: v}) == SHAPE, (k, v)
    for k in ("k", "v", "slots", "K", "V"):
        assert call(f, good, **{k: None}) == NULL, k
    for k, v in (("k", A2), ("v", A1), ("slots", A4), ("K", A8), ("V", A8)):
        assert call(f, good, **{k: v}) == ALIGN, k
    assert call(f, good, dtype=1, k=A1) == ALIGN
    assert call(f, good, dtype=2) == ARG
    assert call(f, good, n=0, k=None, v=None, slots=None) == OK


def test_compact_refusals(lib):
    good = dict(t=qk.Q4_0, K=A16, V=A16, pages=4, page=32, n_kv=2, d=64, table=A4, stride=3, base=A4, path=A4, ps=8, n=A4,
                n_req=2, stream=None)
    f = lib.qk_kv_compact
    assert call(f, good, t=qk.Q5_K) == TYPE
    for k, v in (("d", 48), ("page", 0), ("pages", 1 << 31), ("n_req", -1), ("stride", -1), ("ps", -1)):
        assert call(f, good, **{k: v}) == SHAPE, k
    for k in ("K", "V", "table", "base", "path", "n"):
        assert call(f, good, **{k: None}) == NULL, k
    for k in ("table", "base", "path", "n"):
        assert call(f, good, **{k: A2}) == ALIGN, k
    assert call(f, good, K=A8) == ALIGN
    assert call(f, good, n_req=0) == OK and call(f, good, ps=0) == OK


def test_tree_refusals(lib):
    ws = qk.attn_tree_workspace(qk.Q8_0, 2, 7, 16 * 16, 32, 8, 128)
    assert ws > 0
    good = dict(t=qk.Q8_0, q=A16, n_tok=9, qs=4096, K=A16, V=A16, pages=40, page=16, table=A4, stride=16, ctx=A4, cu=A4,
                mask=A8, n_req=2, max_q=7, heads=32, n_kv=8, d=128, scale=ctypes.c_float(0.1), out=A2, os=4096, ws=A16,
                wsb=ws, stream=None)
    f = lib.qk_attn_tree
    assert call(f, good, t=qk.Q6_K) == TYPE
    for k, v in (("d", 96), ("page", 12), ("n_kv", 0), ("heads", 30), ("heads", 8 * 65), ("max_q", 0), ("max_q", 65), ("n_req", -1),
                 ("n_req", 65536), ("n_tok", -1), ("stride", -1), ("qs", 4095), ("os", 100), ("pages", -3)):
        assert call(f, good, **{k: v}) == SHAPE, (k, v)
    for k in ("q", "K", "V", "table", "ctx", "cu", "out", "ws"):
        assert call(f, good, **{k: None}) == NULL, k
    for k, v in (("q", A8), ("qs", 4100), ("K", A8), ("V", A4), ("out", A1), ("ws", A8), ("table", A2), ("ctx", A2), ("cu", A1),
                 ("mask", A4)):
        assert call(f, good, **{k: v}) == ALIGN, k
    assert call(f, good, wsb=ws - 1) == WORKSPACE
    assert call(f, good, n_tok=0) == OK and call(f, good, n_req=0) == OK
    for bad in ((qk.Q4_K, 2, 7, 256, 32, 8, 128), (qk.Q8_0, 2, 65, 256, 32, 8, 128), (qk.Q8_0, 2, 7, 256, 30, 8, 128),
                (qk.Q8_0, 2, 7, -1, 32, 8, 128), (qk.Q8_0, 2, 7, 256, 32, 8, 80)):
        assert qk.attn_tree_workspace(*bad) == 0


def test_logits_refusals(lib):
    good = dict(x=A4, dtype=0, n=3, V=100, rs=100, cu=A4, n_req=2, hist=A4, hs=9, hl=A4, rep=A4, pres=A4, freq=A4, draft=A4,
                mask=A8, bt=A4, bv=A4, bs=3, bl=A4, gr=A4, gs=4, out=A8, os=104, stream=None)
    f = lib.qk_logits_process
    assert call(f, good, dtype=3) == ARG
    for k, v in (("n", -1), ("V", -1), ("n_req", -1), ("rs", 99), ("os", 64), ("hs", -1), ("hs", (1 << 20) - 64), ("bs", 4096),
                 ("bs", -1), ("gs", 3), ("n", 1 << 31)):
        assert call(f, good, **{k: v}) == SHAPE, (k, v)
    for k in ("x", "out", "cu", "hist", "hl", "rep", "pres", "freq", "bv", "bl"):
        assert call(f, good, **{k: None}) == NULL, k
    for k, v in (("x", A2), ("out", A2), ("cu", A2), ("hist", A1), ("draft", A2), ("mask", A4), ("bt", A2), ("gr", A2)):
        assert call(f, good, **{k: v}) == ALIGN, k
    assert call(f, good, out=A4, os=104) == ARG     # in place with another stride
    assert call(f, good, n=0, x=None) == OK and call(f, good, V=0) == OK


def test_binding_refuses_wrong_tensors(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros(4 * qk.kv_page_bytes(qk.Q8_0, 2, 64, 16), dtype=torch.uint8)
    k = torch.zeros(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    for bad in (dict(k=k.half(), v=k.half()), dict(v=k[:2]), dict(k=k.transpose(1, 2).reshape(3, 2, 64).transpose(0, 1).contiguous()),
                dict(slots=slots.int()), dict(K=pool[:-16]), dict(page=24), dict(K=pool.float()),
                dict(k=torch.zeros(3, 64, 2).transpose(1, 2))):
        a = dict(dict(k=k, v=k, slots=slots, K=pool, V=pool, page=16), **bad)
        with refused():
            qk.kv_append(qk.Q8_0, a["k"], a["v"], a["slots"], a["K"], a["V"], a["page"], stream=0)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    args = dict(table=i32(2, 4), ctx=i32(2), cu=i32(3), mask=torch.zeros(3, dtype=torch.int64))
    for bad in (dict(q=q.float()), dict(cu=i32(2)), dict(table=i32(3, 4)), dict(mask=i32(3)), dict(max_q=65),
                dict(out=torch.zeros(3, 4, 32, dtype=torch.bfloat16)), dict(ws=torch.zeros(16, dtype=torch.uint8))):
        a = dict(dict(args, q=q, max_q=2, out=None, ws=None), **bad)
        with refused():
            qk.attn_tree(qk.Q8_0, a["q"], pool, pool, 16, 2, a["table"], a["ctx"], a["cu"], a["mask"], a["max_q"], 0.1,
                         out=a["out"], ws=a["ws"], stream=0)
    x, f = torch.zeros(3, 50), torch.ones(2)
    base = dict(logits=x, cu=i32(3), hist=i32(2, 5), hist_len=i32(2), rep=f, pres=f, freq=f)
    for bad in (dict(logits=x.half()), dict(hist=i32(3, 5)), dict(rep=f.double()), dict(draft=i32(2)), dict(grammar=i32(3, 1)),
                dict(grammar=i32(2, 2)), dict(out=torch.zeros(3, 51)), dict(logits=x.t())):
        with refused():
            qk.logits_process(**dict(base, **bad), stream=0)
    n = i32(3)
    with refused():
        qk.kv_plan(n, n, n, i32(2, 4), i32(9), i32(1), 16, 8, stream=0)
    with refused():
        qk.kv_plan(n, n, n.long(), i32(3, 4), i32(9), i32(1), 16, 8, stream=0)


# ------------------------------------------- the plain implementations ----

def test_plain_tree_equals_the_oracles_decode_attention(oracle_mod):
    # One request, one token, pages in order: the contiguous cache.
    n_kv, heads, d, page, T = 2, 6, 64, 16, 37
    K, V = (paged_ref.pool("Q5_0", 3, n_kv, page, d, s) for s in (1, 2))
    q = synth.activations(heads, d, 3).reshape(1, heads, d)
    out, Sv, _, _ = paged_ref.attn_tree("Q5_0", q.astype(np.float64), K, V, page, n_kv, np.array([[0, 1, 2]]), [T - 1], [0, 1], None, 1,
                                     0.125)
    flat = lambda p: np.ascontiguousarray(p.transpose(0, 2, 1, 3)).reshape(-1, n_kv, p.shape[-1])[:T].reshape(-1)  # noqa: E731
    ref, Sr = oracle.attn_decode(qk.Q5_0, q[0], flat(K), flat(V), T, heads, n_kv, d, 0.125)
    assert np.allclose(out[0], ref, rtol=1e-12, atol=1e-12) and np.allclose(Sv[0], Sr, rtol=1e-12, atol=1e-12)


def test_plain_tree_masks():
    K, V = (paged_ref.pool("Q8_0", 2, 1, 16, 32, s) for s in (4, 5))
    q = synth.activations(3, 32, 6).reshape(3, 1, 32).astype(np.float64)
    table = np.array([[1]])
    args = (q, K, V, 16, 1, table, [0], [0, 3])
    full, *_ = paged_ref.attn_tree("Q8_0", *args, np.array([1, 3, 7], np.uint64), 3, 0.3)
    chain, *_ = paged_ref.attn_tree("Q8_0", *args, None, 3, 0.3)
    assert np.array_equal(full, chain)
    alone, *_ = paged_ref.attn_tree("Q8_0", *args, np.array([0, 2, 0], np.uint64), 3, 0.3)
    assert not alone[0].any() and not alone[2].any()
    assert np.allclose(alone[1, 0], paged_ref.values("Q8_0", V[1, 0, 1], 32))


def test_plain_plan_and_logits_by_hand():
    table = np.array([[5, 6, -1], [7, -1, -1], [8, 9, -1]], np.int32)
    free = np.array([0, 1, -1, -1, -1], np.int32)
    got = paged_ref.plan([20, 16, 30], [18, 16, 0], [40, 33, 0], table, free, 2, 16, 40)
    # request 2 gives 8 and 9 back; request 0 takes 9; request 1 takes 8 and 1
    assert got["granted"] == [1, 1, 1] and got["n_free"] == [1] and got["cu"] == [0, 22, 39, 39]
    assert table[0].tolist() == [5, 6, 9] and table[1].tolist() == [7, 8, 1]
    assert got["slots"][0] == 6 * 16 + 2 and got["slots"][21] == 9 * 16 + 7 and got["slots"][38] == 1 * 16 and got["slots"][39] == -1
    y, _ = paged_ref.logits([[2.0, -2.0, 1.0, 4.0]], [0, 1], [[0, 1, 1]], [3], [2.0], [0.5], [0.25], bias_tok=[[3, 3]],
                            bias_val=[[9.0, 1.0]], bias_len=[2], grammar=np.array([[0b1011]]))
    assert y.tolist() == [[1.0 - 0.25 - 0.5, -4.0 - 0.5 - 0.5, -np.inf, 5.0]]
