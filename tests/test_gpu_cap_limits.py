"""Caps at the ends of their range, and the cap's symmetry: rows that see a single key, whose log-sum-exp is the
capped score itself."""
import numpy as np
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24                                          # half a step of fp32, relative


def one_key(scores, beside=0.0):
    """A stream a score: one draft, which is its own only key, one head; q.k = the score (exact in bf16).
    `beside`: a further element of the query that the key does not have."""
    B = len(scores)
    q = torch.zeros((B, 1, 1, 576), dtype=torch.bfloat16)
    q[:, 0, 0, 512] = torch.from_numpy(np.asarray(scores, np.float64))
    q[:, 0, 0, 513] = beside
    assert np.array_equal(ref.f64(q)[:, 0, 0, 512], scores)
    lat, scale = torch.zeros((B, 512), dtype=torch.uint8), torch.ones(B)
    rope = torch.zeros((B, 64), dtype=torch.bfloat16)
    rope[:, 0] = 1
    table, seq = torch.arange(B, dtype=torch.int32)[:, None], torch.ones(B, dtype=torch.int32)
    return [t.cuda().contiguous() for t in (q, lat, scale, rope, table, seq)]


def capped(mv, scores, cap, scale=1.0, beside=0.0):
    _, lse = mv.verify_attn_fp8_rules(*one_key(scores, beside), None, scale, softcap=cap, nsplit=1)
    assert mv.device_status() == 0
    return ref.f64(lse)[:, 0, 0]


def bound(z):
    """tanh 2^-21; scale log2 e, the cap in log2 units, their quotient, the products and the way back take ten
    roundings; the log-sum-exp carries the score with 7 taken off and added back, and log2 of 2^7."""
    z = np.abs(z)
    return z * (2.0 ** -21 + 10 * STEP) + 4 * STEP * (1.4427 * z + 14)


@pytest.mark.parametrize("beside", [0.0, 64.0])
@pytest.mark.parametrize("cap", [1e4, 1e25, 2.0 ** 100, 1e35, 2.3e38, 2.4e38, 3.4e38])
def test_large_caps(cuda_lib, cap, beside):
    """A cap that no score comes near leaves the scores as they are, caps of the largest numbers of fp32 too."""
    scores = np.array([0.0, 2.0 ** -100, 2.0 ** -30, 0.015625, 1.0, -3.0, 100.0, -29952.0, 2.0 ** 40, -2.0 ** 60])
    want = cap * np.tanh(scores / cap)
    got = capped(cuda_lib, scores, cap, beside=beside)
    assert np.all(np.abs(got - want) <= bound(want)), (got, want)


@pytest.mark.parametrize("beside", [0.0, 1024.0])
@pytest.mark.parametrize("cap", [1e-30, 1e-38, 1e-42, 1.5e-45])
def test_small_caps(cuda_lib, cap, beside):
    """A score of zero stays zero, all others shrink to the cap, next to nothing."""
    scores = np.array([0.0, 1024.0, -1024.0, 1.0, 2.0 ** -20])
    for scale in (1.0, -1.0):
        got = capped(cuda_lib, scores, cap, scale, beside)
        assert np.all(np.abs(got) <= bound(cap)), got


@pytest.mark.parametrize("beside", [0.0, 64.0])
@pytest.mark.parametrize("cap", [1e-44, 50.0, 1e36, 3.4e38])
def test_key_weights(cuda_lib, cap, beside):
    """The same caps in the key weights: with the capped score as the log-sum-exp every weight is one."""
    mv = cuda_lib
    scores = np.array([0.0, 1.0, -8.0, 40.0, 1024.0, 2.0 ** -60])
    z = cap * np.tanh(scores / cap)
    lse = torch.from_numpy(z).float().view(-1, 1, 1).cuda()
    q, lat, scale, rope, table, seq = one_key(scores, beside)
    kv = torch.zeros((len(scores), 576), dtype=torch.bfloat16, device="cuda")
    kv[:, 512] = 1
    # (the error of the score and of the log-sum-exp's rounding, each times log2 e in two roundings, and ex2's)
    tol = bound(z) + 6 * STEP * np.abs(z) + 2.0 ** -21
    for got in (mv.key_weights_fp8(q, lat, scale, rope, table, seq, None, 1.0, lse, softcap=cap),
                mv.key_weights(q, kv, table, seq, None, 1.0, lse, softcap=cap)):
        assert np.all(np.abs(ref.f64(got)[:, 0] - 1) <= tol * 1.01), ref.f64(got)


def test_capped_scores_are_odd(cuda_lib):
    """cap tanh(-z / cap) is the negative of cap tanh(z / cap), bit for bit, beyond the cap as within it.  (In log2
    units these are between 39 and 57 in size: the 7 that the log-sum-exp takes off and adds back are exact.)"""
    a = np.array([i / 4 for i in range(148, 256)] + [i / 2 for i in range(128, 256)] + list(range(128, 256, 3)))
    for scale in (1.0, 1.01, 1.7):
        cap = 37.0
        up, down = capped(cuda_lib, a, cap, scale), capped(cuda_lib, -a, cap, scale)
        assert np.array_equal(up, -down), int((up != -down).sum())
        want = cap * np.tanh(float(np.float32(scale)) * a / cap)
        assert np.all(np.abs(up - want) <= bound(want))
