"""Refusals of the long-context operators: through the C ABI before any CUDA call, and in the Python binding
before the library is reached.  Nothing here launches a kernel.  Also the float64 forms of their tests on
cases that can be counted by hand."""
import ctypes

import numpy as np
import pytest
import torch

import long_ref as lr
from test_step_host import bf, caller, f32, i32, lib, u8  # noqa: F401

RULES = dict(cap=0.0, slopes=None, pos=None, window=0, prefix=None, doc=None)
SHAPE = [(dict(B=-1), -2), (dict(B=65536), -2), (dict(q_len=0), -2), (dict(q_len=65), -2), (dict(H=0), -2), (dict(H=129), -2),
         (dict(stride=8), -2), (dict(stride=(1 << 30) + 1), -2), (dict(pool=0), -2), (dict(pool=1 << 31), -2),
         (dict(scale=float("nan")), -8), (dict(mask=16, bits=16), -8), (dict(bits=12), -3), (dict(table=18), -3),
         (dict(seq=18), -3), (dict(lse=18), -3), (dict(out=18), -3), (dict(q=24), -3), (dict(cap=-1.0), -8), (dict(cap=float("inf")), -8),
         (dict(cap=float("nan")), -8), (dict(window=-1), -8), (dict(slopes=18), -3), (dict(pos=18), -3), (dict(prefix=18), -3),
         (dict(doc=18), -3), (dict(table=None), -1), (dict(seq=None), -1), (dict(q=None), -1), (dict(lse=None), -1),
         (dict(out=None), -1)]


def test_attn_rules_refusals(lib):
    f = caller(lib, "mla_verify_attn_fp8_rules", q=16, lat=16, sc=16, rope=16, pool=10, table=16, stride=16, seq=16, mask=None,
               bits=None, B=1, q_len=9, H=8, scale=0.1, **RULES, out=16, lse=16, ns=1, ws=None, wsb=0, st=None)
    for kw, code in SHAPE + [(dict(ns=-1), -5), (dict(ns=1025), -5), (dict(lat=24), -3), (dict(rope=24), -3), (dict(out=24), -3),
                             (dict(sc=18), -3), (dict(lat=None), -1), (dict(sc=None), -1), (dict(rope=None), -1)]:
        assert f(**kw) == code, kw
    assert f(B=0, q=None) == 0


def test_key_weights_refusals(lib):
    tail = dict(lse=16, counted=None, w=None, decay=1.0, out=16, ws=None, wsb=0, st=None)
    common = dict(pool=10, table=16, stride=16, seq=16, mask=None, bits=None, B=1, q_len=9, H=8, scale=0.1, **RULES, **tail)
    f = caller(lib, "mla_key_weights_fp8", q=16, lat=16, sc=16, rope=16, **common)
    g = caller(lib, "mla_key_weights", q=16, kv=16, **common)
    for kw, code in SHAPE + [(dict(decay=float("nan")), -8), (dict(decay=float("inf")), -8), (dict(w=18), -3)]:
        assert f(**kw) == code and g(**kw) == code, kw
    for name in ("lat", "sc", "rope"):
        assert f(**{name: None}) == -1 and f(**{name: 18}) == -3
    assert g(kv=None) == -1 and g(kv=24) == -3
    assert f(B=0, q=None) == 0 and g(B=0, q=None) == 0
    for kw in (dict(), dict(ws=256, wsb=2 * 3 * 16 * 4 - 1)):          # 130 rows: two tiles
        assert f(B=3, q_len=13, H=10, **kw) == -4 and g(B=3, q_len=13, H=10, **kw) == -4
    assert f(B=3, q_len=13, H=10, ws=258, wsb=1 << 20) == -3


def test_key_weights_workspace(lib):
    ws = lib.mla_key_weights_workspace_bytes
    assert ws(4, 16, 8, 1000) == 0 and ws(4, 1, 128, 1000) == 0
    assert ws(4, 17, 8, 1000) == 2 * 4 * 1000 * 4 and ws(1, 64, 128, 1 << 20) == 64 << 22
    assert ws(0, 64, 128, 10) == ws(1, 0, 128, 10) == ws(1, 65, 128, 10) == ws(1, 64, 129, 10) == ws(1, 64, 128, 0) == 0


def test_evict_refusals(lib):
    f = caller(lib, "mla_kv_evict", table=16, seq=16, w=16, pos=None, doc=None, B=2, stride=100, budgets=None, budget=10, sink=1,
               recent=1, to=16, lo=16, wo=16, po=None, do=None, freed=None, nf=None, ws=None, wsb=0, st=None)
    for kw, code in [(dict(B=-1), -2), (dict(B=65536), -2), (dict(stride=0), -2), (dict(stride=(1 << 30) + 1), -2),
                     (dict(sink=-1), -8), (dict(recent=-1), -8), (dict(do=16), -8), (dict(freed=16), -1), (dict(nf=16), -1)]:
        assert f(**kw) == code, kw
    for name in ("table", "seq", "w", "to", "lo", "wo"):
        assert f(**{name: None}) == -1 and f(**{name: 18}) == -3, name
    for name in ("pos", "doc", "budgets", "po"):
        assert f(**{name: 18}) == -3, name
    assert f(ws=24) == -3
    assert f(B=0, table=None) == 0


def test_evict_workspace(lib):
    """Only streams that are longer than their cluster takes at once need one."""
    ws = lib.mla_kv_evict_workspace_bytes
    assert ws(1, 8192, 1, 152) == 0 and ws(1, 16 * 8192, 0, 152) == 0 and ws(64, 16384, 1, 152) == 0
    up = lambda x: (x + 255) // 256 * 256
    want = lambda B, n, k: up(B * 8258 * 4) + up(B * 4) + up(B * 24) + up(B * -(-n // 8192) * 4) + up(B * -(-n // 8192) * 128) + k * up(B * n * 4)
    assert ws(64, 16385, 0, 152) == want(64, 16385, 2) and ws(2, 1 << 20, 1, 152) == want(2, 1 << 20, 6)
    assert ws(0, 1 << 20, 0, 152) == ws(65536, 1 << 20, 0, 152) == ws(2, 0, 0, 152) == ws(2, (1 << 30) + 1, 0, 152) == 0
    assert ws(2, 1 << 20, 0, 0) == 0


def test_binding_refusals():
    import mla_speculative_verify_attention_gb300 as mv
    q, cache, kv = bf(2, 3, 4, 576), (u8(8, 512), f32(8), bf(8, 64)), bf(8, 576)
    table, seq, lse = i32(2, 20), i32(2), f32(2, 3, 4)
    attn = lambda *a, **k: mv.verify_attn_fp8_rules(q, *cache, table, seq, None, 0.1, **k)
    fp8 = lambda *a, **k: mv.key_weights_fp8(q, *cache, table, seq, None, 0.1, lse, **k)
    b16 = lambda *a, **k: mv.key_weights(q, kv, table, seq, None, 0.1, lse, **k)
    for call in (attn, fp8, b16):
        with pytest.raises(ValueError, match="CUDA"):
            call()
        for bad in (dict(slopes=f32(3)), dict(key_pos=i32(2, 19)), dict(prefix_lens=i32(3)), dict(key_doc=i32(20)),
                    dict(window=-1), dict(window=1 << 31)):
            with pytest.raises(ValueError):
                call(**bad)
        for bad in (dict(slopes=bf(4)), dict(key_pos=f32(2, 20)), dict(prefix_lens=f32(2)), dict(key_doc=u8(2, 20))):
            with pytest.raises(TypeError):
                call(**bad)
    for call in (fp8, b16):
        for bad in (dict(weights=f32(2, 21)), dict(counted=u8(2, 4)), dict(out=f32(2))):
            with pytest.raises(ValueError):
                call(**bad)
        with pytest.raises(TypeError):
            call(counted=torch.zeros((2, 3), dtype=torch.bool))
    with pytest.raises(ValueError):
        mv.key_weights(q, bf(8, 575), table, seq, None, 0.1, lse)
    with pytest.raises(ValueError):
        mv.key_weights(q, kv, table, seq, u8(2, 3, 4), 0.1, lse)
    ev = lambda **k: mv.kv_evict(table, seq, f32(2, 20), k.pop("budget", 5), **k)
    with pytest.raises(ValueError, match="CUDA"):
        ev()
    for bad in (dict(budget=-1), dict(budget=1 << 31), dict(sink=-1), dict(recent=1 << 31), dict(budget=i32(3)), dict(doc_out=table),
                dict(key_pos=i32(2, 21)), dict(table_out=i32(2, 21)), dict(n_freed=i32(3)), dict(freed=i32(2))):
        with pytest.raises(ValueError):
            ev(**bad)
    for bad in (dict(budget=f32(2)), dict(key_doc=f32(2, 20)), dict(weights_out=table)):
        with pytest.raises(TypeError):
            ev(**bad)
    with pytest.raises(ValueError, match="contiguous"):
        mv.kv_evict(i32(20, 2).t(), seq, f32(2, 20), 5)


def test_rules_by_hand():
    """Ten keys, two drafts (keys 8 and 9) in a chain."""
    pos = np.array([[0, 2, 4, 6, 8, 10, 12, 14, 16, 18]], np.int32)
    doc = np.array([[-1, 0, 0, 1, 1, 0, 0, 0, 0, 1]], np.int32)
    see = lambda t, **k: lr.Rules(**k).seen(None, 0, t, 10, 2)[0].nonzero()[0].tolist()
    assert see(0) == list(range(9)) and see(1) == list(range(10))
    assert see(0, window=3) == [6, 7, 8] and see(1, window=3) == [7, 8, 9]
    assert see(0, window=3, key_pos=pos) == [7, 8] and see(1, window=3, key_pos=pos) == [8, 9]
    assert see(0, window=3, prefix_lens=np.array([2])) == [0, 1, 6, 7, 8]
    assert see(0, window=3, prefix_lens=np.array([5]), key_pos=pos) == [0, 1, 2, 7, 8]
    assert see(0, prefix_lens=np.array([10])) == list(range(10))          # a prefix is seen both ways
    assert see(0, key_doc=doc) == [0, 1, 2, 5, 6, 7, 8] and see(1, key_doc=doc) == [0, 3, 4, 9]
    assert lr.Rules(key_pos=pos).seen(None, 0, 1, 10, 2)[1].tolist() == [-18, -16, -14, -12, -10, -8, -6, -4, -2, 0]


def test_evict_by_hand():
    x = dict(table=np.arange(10, 18, dtype=np.int32)[None], weights=np.array([[9, 1, 5, 1, np.nan, 0, 1, 8]], np.float32))
    outs = dict(table_out=np.zeros((1, 8), np.int32), lens_out=np.zeros(1, np.int32), weights_out=np.zeros((1, 8), np.float32),
                pos_out=np.zeros((1, 8), np.int32), doc_out=None, freed=np.zeros((1, 8), np.int32), n_freed=np.zeros(1, np.int32))
    go = lambda budget, sink, recent: lr.evict(x["table"], np.array([8]), x["weights"], budget, sink, recent, None, None, outs)
    o = go(4, 0, 0)
    assert o["pos_out"][0, :4].tolist() == [0, 2, 4, 7] and o["freed"][0, :4].tolist() == [11, 13, 15, 16]
    o = go(5, 0, 2)
    assert o["table_out"][0, :5].tolist() == [10, 12, 14, 16, 17] and o["lens_out"][0] == 5 and o["n_freed"][0] == 3
    assert go(5, 3, 0)["pos_out"][0, :5].tolist() == [0, 1, 2, 4, 7]
    assert go(1, 2, 2)["pos_out"][0, :4].tolist() == [0, 1, 6, 7]
    assert go(6, 0, 0)["pos_out"][0, :6].tolist() == [0, 1, 2, 3, 4, 7]   # of the ones that tie, the first
