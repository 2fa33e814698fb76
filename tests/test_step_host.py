"""Refusals of the operators around the fp8 cache: through the C ABI before any CUDA call, and in
the Python binding before the library is reached.  Nothing here launches a kernel."""
import ctypes

import numpy as np
import pytest
import torch

import step_ref as ref
import workloads as w

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from mla_speculative_verify_attention_gb300 import build
    build.build()
    import mla_speculative_verify_attention_gb300 as mv
    return mv.load()


def caller(lib, fn, **base):
    def call(**kw):
        a = dict(base)
        assert set(kw) <= set(a)
        a.update(kw)
        return getattr(lib, fn)(*a.values())
    return call


def test_norm_rope_refusals(lib):
    f = caller(lib, "mla_qk_norm_rope", q=16, kv=16, wq=16, wk=16, pos=16, freq=16, eps=1e-6, inter=1, n=4, H=8, qo=16,
               ko=16, st=None)
    assert f(H=0) == -2 and f(H=129) == -2 and f(n=-1) == -2 and f(n=1 << 31) == -2
    assert f(q=None, kv=None) == -1 and f(qo=None) == -1 and f(ko=None) == -1 and f(pos=None) == -1 and f(freq=None) == -1
    assert f(eps=-1.0) == -8 and f(eps=float("nan")) == -8 and f(eps=float("inf")) == -8
    for name in ("q", "kv", "wq", "wk", "qo", "ko"):
        assert f(**{name: 24}) == -3, name
    assert f(pos=18) == -3 and f(freq=18) == -3
    assert f(n=0, q=None, kv=None) == 0


@pytest.mark.parametrize("fn", ["mla_kv_append_quant", "mla_kv_read_fp8"])
def test_cache_rows_refusals(lib, fn):
    f = caller(lib, fn, lat=16, sc=16, rope=16, pool=8, slots=16, rows=16, n=2, st=None)
    assert f(n=-1) == -2 and f(pool=0) == -2 and f(pool=1 << 31) == -2
    for name in ("lat", "sc", "rope", "slots", "rows"):
        assert f(**{name: None}) == -1, name
        assert f(**{name: 18}) == -3, name
    assert f(n=0, lat=None) == 0


def test_verify_fp8_refusals(lib):
    f = caller(lib, "mla_verify_attn_fp8", q=16, lat=16, sc=16, rope=16, pool=10, table=16, stride=16, seq=16, mask=None,
               bits=None, B=1, q_len=9, H=8, scale=0.1, out=16, lse=16, ns=1, ws=None, wsb=0, st=None)
    for kw, code in [(dict(B=-1), -2), (dict(B=65536), -2), (dict(q_len=0), -2), (dict(q_len=65), -2), (dict(H=0), -2),
                     (dict(H=129), -2), (dict(stride=8), -2), (dict(pool=0), -2), (dict(pool=1 << 31), -2),
                     (dict(ns=-1), -5), (dict(ns=1025), -5), (dict(scale=float("nan")), -8),
                     (dict(mask=16, bits=16), -8), (dict(bits=12), -3), (dict(q=24), -3), (dict(lat=24), -3),
                     (dict(rope=24), -3), (dict(out=24), -3), (dict(sc=18), -3), (dict(lse=18), -3), (dict(table=18), -3),
                     (dict(seq=18), -3)]:
        assert f(**kw) == code, kw
    for name in ("q", "lat", "sc", "rope", "table", "seq", "out", "lse"):
        assert f(**{name: None}) == -1, name
    assert f(B=0, q=None) == 0


def test_verify_fp8_workspace(lib):
    """What the automatic call wants: zero for bad arguments or one split, no more than a wave of splits
    otherwise, and never more than the largest split count's."""
    f = lib.mla_verify_fp8_workspace_bytes
    f.argtypes, f.restype = [ctypes.c_int] * 5, ctypes.c_size_t
    ws = lib.mla_verify_workspace_bytes
    assert f(0, 9, 8, 100, 152) == f(1, 0, 8, 100, 152) == f(1, 65, 8, 100, 152) == f(1, 9, 129, 100, 152) == 0
    assert f(1, 9, 8, 0, 152) == f(1, 9, 8, 100, 0) == 0
    assert f(1, 9, 8, 48, 152) == 0                                                # one tile, one split
    assert f(1, 9, 8, 265, 152) == ws(1, 9, 8, 6)                                  # a tile of 48 keys a split
    assert f(1, 9, 8, 1 << 20, 152) == ws(1, 9, 8, 152) and f(1, 9, 64, 1 << 20, 152) == ws(1, 9, 64, 19)
    assert f(8, 9, 8, 46089, 152) == ws(1, 9, 8, 152)                              # one wave of slots, all streams
    assert f(128, 1, 16, 1000, 152) == 0                                           # nearly a wave of whole streams
    for args in [(200, 1, 8, 4000, 152), (65535, 64, 128, 1 << 30, 152), (1, 64, 128, 5000, 152), (1, 1, 1, (1 << 31) - 1, 1)]:
        assert f(*args) <= ws(*args[:3], 1024)


def test_draft_verify_refusals(lib):
    f = caller(lib, "mla_draft_verify", p=16, q=16, tok=16, par=16, u=16, un=16, B=2, q_len=9, V=100, n=16, out=16, path=16,
               st=None)
    assert f(B=-1) == -2 and f(B=65536) == -2 and f(q_len=0) == -2 and f(q_len=65) == -2
    assert f(V=0) == -2 and f(V=(1 << 24) + 1) == -2
    for name in ("p", "tok", "u", "un", "n", "out", "path"):
        assert f(**{name: None}) == -1, name
    for name in ("p", "q"):
        assert f(**{name: 24}) == -3, name
    for name in ("tok", "par", "u", "un", "n", "out", "path"):
        assert f(**{name: 18}) == -3, name
    assert f(B=0, p=None) == 0


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_binding_refusals():
    import mla_speculative_verify_attention_gb300 as mv
    cpu = pytest.raises(ValueError, match="CUDA")
    cache = (u8(8, 512), f32(8), bf(8, 64))
    with cpu:
        mv.qk_norm_rope(bf(2, 4, 576), bf(2, 576), i32(2), f32(32))
    with cpu:
        mv.kv_append_quant(*cache, i32(3), bf(3, 576))
    with cpu:
        mv.kv_read_fp8(*cache, i32(3))
    with cpu:
        mv.verify_attn_fp8(bf(2, 4, 8, 576), *cache, i32(2, 8), i32(2), None, 0.1)
    with cpu:
        mv.draft_verify(f32(2, 3, 10), f32(2, 3, 10), i32(2, 3), None, f32(2, 3), f32(2))
    for call in (
            lambda: mv.qk_norm_rope(None, None, i32(2), f32(32)),
            lambda: mv.qk_norm_rope(bf(2, 4, 575), None, i32(2), f32(32)),
            lambda: mv.qk_norm_rope(bf(3, 4, 576), None, i32(2), f32(32)),
            lambda: mv.qk_norm_rope(bf(2, 4, 576), None, i32(2), f32(64)),
            lambda: mv.qk_norm_rope(bf(2, 4, 576), None, i32(2), f32(32), kv_out=bf(2, 576)),
            lambda: mv.kv_append_quant(u8(8, 511), f32(8), bf(8, 64), i32(3), bf(3, 576)),
            lambda: mv.kv_append_quant(u8(8, 512), f32(7), bf(8, 64), i32(3), bf(3, 576)),
            lambda: mv.kv_append_quant(*cache, i32(4), bf(3, 576)),
            lambda: mv.kv_read_fp8(*cache, i32(3), out=bf(2, 576)),
            lambda: mv.verify_attn_fp8(bf(2, 4, 8, 576), *cache, i32(3, 8), i32(2), None, 0.1),
            lambda: mv.verify_attn_fp8(bf(2, 4, 8, 576), *cache, i32(2, 8), i32(2), u8(2, 4, 3), 0.1),
            lambda: mv.verify_attn_fp8(bf(2, 4, 8, 576), *cache, i32(2, 8), i32(2), torch.zeros((2, 3), dtype=torch.int64), 0.1),
            lambda: mv.draft_verify(f32(2, 3, 10), f32(2, 3, 11), i32(2, 3), None, f32(2, 3), f32(2)),
            lambda: mv.draft_verify(f32(2, 3, 10), None, i32(2, 2), None, f32(2, 3), f32(2)),
            lambda: mv.draft_verify(f32(2, 3, 10), None, i32(2, 3), i32(3, 3), f32(2, 3), f32(2))):
        with pytest.raises(ValueError):
            call()
    for call in (
            lambda: mv.qk_norm_rope(f32(2, 4, 576), None, i32(2), f32(32)),
            lambda: mv.qk_norm_rope(bf(2, 4, 576), None, i32(2).long(), f32(32)),
            lambda: mv.kv_append_quant(*cache, i32(3).long(), bf(3, 576)),
            lambda: mv.kv_append_quant(*cache, i32(3), f32(3, 576)),
            lambda: mv.verify_attn_fp8(bf(2, 4, 8, 576), *cache, i32(2, 8), i32(2), f32(2, 4, 4), 0.1),
            lambda: mv.verify_attn_fp8(bf(2, 4, 8, 576), *cache, i32(2, 8), i32(2), None, 0.1, out=f32(2, 4, 8, 512)),
            lambda: mv.draft_verify(bf(2, 3, 10), None, i32(2, 3), None, f32(2, 3), f32(2))):
        with pytest.raises(TypeError):
            call()


# ---- the float64 forms that the GPU tests compare with, pinned on their own
def test_quantise_reference():
    x = torch.tensor(np.random.default_rng(0).normal(size=(40, 512))).to(torch.bfloat16).float()
    code, scale = ref.quantise(x.numpy())
    want = (x / torch.from_numpy(scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(code, want.view(torch.uint8).numpy())
    assert np.all(np.abs(ref.e4m3_values()[code]).max(1) == 448)


def test_accept_reference_keeps_the_target():
    """The walk's first token, averaged exactly over a fine grid of u and u_next, has the target's
    distribution: the property that makes rejection sampling right."""
    p = np.array([[0.5, 0.25, 0.25]] * 2, np.float32)
    q = np.array([[0.25, 0.5, 0.25]] * 2, np.float32)
    n, got = 64, np.zeros(3)
    for x in range(3):
        for i in range(n):
            for j in range(n):
                _, t, _ = ref.accept(p, q, [0, x], None, [0, (i + 0.5) / n], (j + 0.5) / n)
                got[t[0]] += q[0, x] / n ** 2
    assert np.allclose(got, p[0], atol=1e-12)


def test_norm_rope_reference_turns():
    x = np.zeros((1, 1, 576))
    x[0, 0, 512], x[0, 0, 513] = 1.0, 0.0
    y, _ = ref.norm_rope(x, None, np.array([1.0]), np.full(32, np.pi / 2), 0.0, True)
    assert np.allclose(y[0, 0, 512:514], [0, 1], atol=1e-12)
    x = np.zeros((1, 1, 576))
    x[0, 0, 512 + 5] = 1.0
    y, _ = ref.norm_rope(x, None, np.array([1.0]), np.full(32, np.pi / 2), 0.0, False)
    assert np.allclose(y[0, 0, 512 + 5], 0, atol=1e-12) and np.allclose(y[0, 0, 512 + 37], 1)
