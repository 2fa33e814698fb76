"""mla_qk_norm_rope against a float64 form, at the roundings' own bounds (step_ref.norm_rope)."""
import numpy as np
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

FREQ = 10000.0 ** (-np.arange(0, 64, 2) / 64)


def make(T, H, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(spread * torch.randn((T, 1, 1), generator=g))
    q = (torch.randn((T, H, 576), generator=g) * size).to(torch.bfloat16)
    kv = (torch.randn((T, 576), generator=g) * size[:, 0]).to(torch.bfloat16)
    wt = (1 + 0.2 * torch.randn((2, 512), generator=g)).to(torch.bfloat16)
    return q, kv, wt[0].contiguous(), wt[1].contiguous()


def check(got, want, tol):
    g = ref.f64(got).reshape(want.shape)
    assert np.all(np.isfinite(g))
    worst = np.max(np.abs(g - want) - tol)
    assert worst <= 0, f"off by {worst:.3e} more than the roundings allow"


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H", [(1, 1), (9, 8), (3, 128), (17, 5), (130, 64), (1, 7)])
@pytest.mark.parametrize("norms", ["both", "kv", "none"])
def test_against_float64(cuda_lib, T, H, interleaved, norms):
    mv = cuda_lib
    q, kv, wq, wk = make(T, H, seed=T * 131 + H, spread=2.0)
    wq = wq if norms == "both" else None
    wk = wk if norms != "none" else None
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    freq = torch.tensor(FREQ, dtype=torch.float32)
    c = lambda t: None if t is None else t.cuda()
    yq, yk = mv.qk_norm_rope(c(q), c(kv), c(pos), c(freq), q_weight=c(wq), kv_weight=c(wk), eps=1e-5,
                             interleaved=interleaved)
    torch.cuda.synchronize()
    args = (pos.numpy().astype(np.float64), ref.f64(freq), float(np.float32(1e-5)), interleaved)
    check(yq, *ref.norm_rope(ref.f64(q), None if wq is None else ref.f64(wq), *args))
    check(yk, *ref.norm_rope(ref.f64(kv)[:, None], None if wk is None else ref.f64(wk), *args))
    if wq is None:                                     # untouched latent dims, bit for bit
        assert torch.equal(yq[..., :512].cpu(), q[..., :512])


@pytest.mark.parametrize("pos", [0, 1, -1, -70000, 65545, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)])
def test_far_positions(cuda_lib, pos):
    """Frequencies with many turns a position and positions up to 2^31: the angle's whole turns
    drop out exactly."""
    mv = cuda_lib
    q, _, _, _ = make(2, 3, seed=9)
    freq = torch.tensor(np.concatenate([FREQ[:16], np.linspace(0.1, 700.0, 16)]), dtype=torch.float32)
    p = torch.full((2,), pos, dtype=torch.int32)
    yq, none = mv.qk_norm_rope(q.cuda(), None, p.cuda(), freq.cuda())
    assert none is None
    # up to 700 rad a position = 112 turns: the fp64 product rounds at 2^-53 of the whole, 112 2^-53
    # turns a position, so the far bound is 224 times step_ref's
    x, f = ref.f64(q), ref.f64(freq)
    want, tol = ref.norm_rope(x, None, p.numpy().astype(np.float64), f, 0.0, True)
    far = 2 * np.pi * abs(pos) * 2.0 ** -53 * 224
    tol[..., 512:] += far * np.repeat(np.abs(x[..., 512::2]) + np.abs(x[..., 513::2]), 2, -1)
    check(yq, want, tol)


def test_in_place_and_keys_alone(cuda_lib):
    mv = cuda_lib
    q, kv, wq, wk = (t.cuda() for t in make(33, 16, seed=3))
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    freq = torch.tensor(FREQ, dtype=torch.float32, device="cuda")
    for inter in (True, False):
        a, b = mv.qk_norm_rope(q, kv, pos, freq, q_weight=wq, kv_weight=wk, interleaved=inter)
        q2, kv2 = q.clone(), kv.clone()
        mv.qk_norm_rope(q2, kv2, pos, freq, q_weight=wq, kv_weight=wk, interleaved=inter, q_out=q2, kv_out=kv2)
        _, alone = mv.qk_norm_rope(None, kv, pos, freq, kv_weight=wk, interleaved=inter)
        torch.cuda.synchronize()
        assert torch.equal(a, q2) and torch.equal(b, kv2) and torch.equal(alone, b)


def test_leading_shapes_zero_tokens_and_zero_rows(cuda_lib):
    mv = cuda_lib
    q, kv, wq, wk = (t.cuda() for t in make(12, 4, seed=4))
    pos = torch.arange(12, dtype=torch.int32, device="cuda") * 37
    freq = torch.tensor(FREQ, dtype=torch.float32, device="cuda")
    a, b = mv.qk_norm_rope(q, kv, pos, freq, q_weight=wq, kv_weight=wk)
    a2, b2 = mv.qk_norm_rope(q.view(3, 4, 4, 576), kv.view(3, 4, 576), pos.view(3, 4), freq, q_weight=wq, kv_weight=wk)
    assert torch.equal(a2.view_as(a), a) and torch.equal(b2.view_as(b), b)
    e, _ = mv.qk_norm_rope(q[:0], kv[:0], pos[:0], freq)
    assert e.shape == (0, 4, 576)
    z, _ = mv.qk_norm_rope(torch.zeros_like(q), None, pos, freq, q_weight=wq, eps=1e-6)
    torch.cuda.synchronize()
    assert int(z.count_nonzero()) == 0


def test_nan_and_infinity_stay_in_their_row(cuda_lib):
    mv = cuda_lib
    q, kv, wq, wk = (t.cuda() for t in make(4, 3, seed=6))
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    freq = torch.tensor(FREQ, dtype=torch.float32, device="cuda")
    good, _ = mv.qk_norm_rope(q, None, pos, freq, q_weight=wq)
    bad = q.clone()
    bad[1, 1, 7] = float("nan")
    bad[2, 0, 520] = float("inf")
    got, _ = mv.qk_norm_rope(bad, None, pos, freq, q_weight=wq)
    torch.cuda.synchronize()
    assert bool(torch.isnan(got[1, 1, :512]).all())
    same = torch.ones((4, 3), dtype=torch.bool, device="cuda")
    same[1, 1] = same[2, 0] = False
    assert torch.equal(got[same], good[same])
    assert torch.equal(got[2, 0, :512], good[2, 0, :512])
