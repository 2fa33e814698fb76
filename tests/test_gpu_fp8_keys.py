"""mla_verify_attn_fp8 takes every visible key once, at its own scale: inputs that count the keys
(counted_keys.py).  A key left out, taken twice or read from another slot shows at once, which the
tolerances of random data do not promise."""
import numpy as np
import pytest
import torch

import step_ref as ref
from counted_keys import ONE, Counted

pytestmark = pytest.mark.gpu


def check(mv, c, **kw):
    q = torch.zeros((c.B, c.q_len, c.H, 576), dtype=torch.bfloat16, device="cuda")
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()
    out, lse = mv.verify_attn_fp8(q, dev(c.lat), dev(c.scale), dev(c.rope).to(torch.bfloat16), dev(c.table), dev(c.seq),
                                  dev(c.mask), 1.0, **kw)
    out, lse = ref.f64(out), ref.f64(lse)
    assert mv.device_status(clear=True) == 0
    for b in range(c.B):
        for t in range(c.q_len):
            s = c.keys(b, t)
            if not len(s):
                assert np.all(out[b, t] == 0) and np.all(np.isneginf(lse[b, t])), (b, t)
            else:
                assert c.agree(out[b, t], lse[b, t], *c.expected(s)), (b, t, kw)


BORDERS = [1, 2, 3, 31, 47, 48, 49, 95, 96, 97, 143, 144, 145, 191, 193, 241, 479, 480, 481, 577]


@pytest.mark.parametrize("nsplit", [0, 1, 2, 3, 5, 8])
@pytest.mark.parametrize("H", [1, 8, 64, 72, 73, 80, 96, 97, 128])
def test_tile_and_split_borders(cuda_lib, H, nsplit):
    """Lengths around multiples of a tile of 48 keys; one row tile of every size and two of them."""
    check(cuda_lib, Counted(1, H, BORDERS, seed=H), nsplit=nsplit)


@pytest.mark.parametrize("nsplit", [0, 1, 4])
@pytest.mark.parametrize("q_len,H", [(9, 8), (5, 16), (17, 8), (9, 64), (64, 2)])
def test_masked_drafts(cuda_lib, q_len, H, nsplit):
    """Random masks over drafts that lie across tile borders; some rows see no key at all."""
    lengths = [q_len, q_len + 1, 48 if q_len <= 48 else q_len + 2, 96, 97, 100 + q_len // 2, 385]
    check(cuda_lib, Counted(q_len, H, lengths, seed=q_len + H, mask=True), nsplit=nsplit)


@pytest.mark.parametrize("B,H", [(2, 8), (5, 16), (17, 8), (40, 72), (64, 4), (64, 80), (70, 8)])
def test_balanced_chunks(cuda_lib, B, H):
    """Streams of very different length in one call: equal chunks over all of them (up to 64 streams)."""
    rng = np.random.default_rng(B + H)
    lengths = np.exp(rng.uniform(0, np.log(3001), B)).astype(int)
    lengths[0], lengths[-1] = 3000, 1
    check(cuda_lib, Counted(1, H, lengths, seed=B))


@pytest.mark.parametrize("lengths", [[20003, 6], [29009]])
@pytest.mark.parametrize("H", [8, 24])
def test_long_streams(cuda_lib, lengths, H):
    for nsplit in (0, 1, 7):
        check(cuda_lib, Counted(3, H, lengths, seed=3, mask=True), nsplit=nsplit)


def test_table_wider_than_the_streams(cuda_lib):
    """Splits planned from the table's width: most of them have no key."""
    for lengths in ([300], [50, 1, 200]):
        check(cuda_lib, Counted(1, 8, lengths, seed=4, extra_stride=20000))


def test_probabilities_carry_eleven_bits(cuda_lib):
    """One key a dim, scores k / 64 without a rounding: an output is off by its own rounding (half a bf16
    step) and its probability's, half an fp16 step, 2^-11; probabilities of bf16 would go past that at
    many dims.  (Scores up to 4: probabilities well inside fp16's normal range.)"""
    rng = np.random.default_rng(0)
    n, H = 512, 8
    c = Counted(1, H, [n], seed=9)
    s = c.table[0]
    c.scale[s] = 1.0
    c.lat[s] = 0
    c.lat[s, np.arange(n)] = ONE
    g = rng.integers(0, 256, n) / 64
    c.rope[s] = 0
    c.rope[s, 0] = g
    q = torch.zeros((1, 1, H, 576), dtype=torch.bfloat16)
    size = np.array([1.0, 0.5, 0.75, 0.25, 0.875, 0.625, 0.125, 0.375])
    q[0, 0, :, 512] = torch.from_numpy(size)
    cuda = lambda x: torch.from_numpy(x).cuda()
    for nsplit in (1, 3):
        out, lse = cuda_lib.verify_attn_fp8(q.cuda(), cuda(c.lat), cuda(c.scale), cuda(c.rope).to(torch.bfloat16),
                                            cuda(c.table), cuda(c.seq), None, 1.0, nsplit=nsplit)
        e = np.exp(size[:, None] * g)
        want = e / e.sum(1, keepdims=True)
        # fp32: score times scale log2 e (2^-23 of at most 6), ex2, the row's sum, 1 / l, the merge
        rel = (1 + 2.0 ** -8) * (1 + 2.0 ** -11 + 2.0 ** -17) - 1
        assert np.all(np.abs(ref.f64(out)[0, 0] - want) <= want * rel)
        assert np.all(np.abs(ref.f64(lse)[0, 0] - np.log(e.sum(1))) <= 2.0 ** -17)
