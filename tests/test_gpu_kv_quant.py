"""The fp8 cache's quantising append and read-back, bit for bit against numpy."""
import numpy as np
import pytest
import torch

import oracle
import step_ref as ref
import workloads as w

pytestmark = pytest.mark.gpu


def cache(n_pool, seed):
    rng = np.random.default_rng(seed)
    lat = torch.from_numpy(rng.integers(0, 0x7F, (n_pool, 512), dtype=np.uint8))
    sc = torch.from_numpy(rng.uniform(0.5, 2, n_pool).astype(np.float32))
    rope = torch.from_numpy(rng.normal(size=(n_pool, 64)).astype(np.float32)).to(torch.bfloat16)
    return lat, sc, rope


def rows_of(n, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, 576), generator=g) * torch.exp(spread * torch.randn((n, 1), generator=g))).to(torch.bfloat16)


def expect(lat, sc, rope, slots, rows):
    lat, sc, rope = lat.clone(), sc.clone(), rope.clone()
    code, scale = ref.quantise(rows.float().numpy())
    lat[slots.long()] = torch.from_numpy(code)
    sc[slots.long()] = torch.from_numpy(scale)
    rope[slots.long()] = rows[:, 512:]
    return lat, sc, rope


def bits_equal(a, b):
    it = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.cpu().contiguous().view(it), b.cpu().contiguous().view(it))


@pytest.mark.parametrize("n,n_pool", [(1, 1), (2, 9), (72, 300), (1001, 1500), (4105, 4105)])
def test_append_bit_exact(cuda_lib, n, n_pool):
    mv = cuda_lib
    c = cache(n_pool, seed=n)
    rows = rows_of(n, seed=n + 1)
    slots = torch.randperm(n_pool, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    dev = [t.cuda() for t in c]
    mv.kv_append_quant(*dev, slots.cuda(), rows.cuda())
    torch.cuda.synchronize()
    for name, got, want in zip(("codes", "scales", "ropes"), dev, expect(*c, slots, rows)):
        assert bits_equal(got, want), name             # the other pool rows untouched, too
    assert mv.device_status() == 0


def test_append_special_values(cuda_lib):
    """Zeros, one-value rows, subnormals, the largest values, ties, infinities and NaN."""
    mv = cuda_lib
    bf = torch.finfo(torch.bfloat16)
    x = rows_of(9, seed=8, spread=0.0)
    x[0] = 0.0
    x[1] = 0.0; x[1, 3] = -2.5
    x[2] = 9.1835e-41                                  # smallest bf16 subnormal
    x[3, :512] = bf.max
    x[4, 5] = float("inf"); x[4, 6] = float("-inf")
    x[5, 100] = float("nan")
    x[6, :512] = float("inf")
    # ties of the code grid: scale 1 (maximum 448), halfway between neighbouring codes
    x[7, :512] = torch.tensor([448.0, 17.0, 19.0, -17.0, 0.0009765625, -0.0029296875, 25.0, 27.0] * 64)
    x[8, :512] = float("nan")
    c = cache(9, seed=1)
    dev = [t.cuda() for t in c]
    slots = torch.arange(9, dtype=torch.int32)
    mv.kv_append_quant(*dev, slots.cuda(), x.cuda())
    torch.cuda.synchronize()
    lat, sc, rope = expect(*c, slots, x)
    nan = ((lat & 0x7F) == 0x7F)
    got = dev[0].cpu()
    assert torch.equal((got & 0x7F) == 0x7F, nan)      # a NaN's sign is not kept track of
    assert torch.equal(got[~nan], lat[~nan])
    assert bits_equal(dev[1], sc) and bits_equal(dev[2], rope)


def test_quantisation_error_bound(cuda_lib):
    """Read back, every value is within half an e4m3 step (relative 2^-4, or 2^-10 of the scale
    below the normal range) and one bf16 rounding of what was written."""
    mv = cuda_lib
    n = 500
    dev = [t.cuda() for t in cache(n, seed=2)]
    rows = rows_of(n, seed=3)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    mv.kv_append_quant(*dev, slots, rows.cuda())
    got = ref.f64(mv.kv_read_fp8(*dev, slots))
    x, scale = ref.f64(rows), ref.f64(dev[1])[:, None]
    quant = np.maximum(np.abs(x[:, :512]) * 2.0 ** -4, scale * 2.0 ** -10)
    # the scale's rounding may put the maximum a step over 448 (saturated), the quotient rounds once
    tol = quant * (1 + 2.0 ** -8) + np.abs(x[:, :512]) * (2.0 ** -8 + 4 * 2.0 ** -24)
    assert np.all(np.abs(got[:, :512] - x[:, :512]) <= tol)
    assert np.array_equal(got[:, 512:], x[:, 512:])


@pytest.mark.parametrize("n,n_pool", [(1, 1), (3, 2), (72, 300), (4105, 5000)])
def test_read_bit_exact(cuda_lib, n, n_pool):
    mv = cuda_lib
    lat, sc, rope = cache(n_pool, seed=n + 7)
    lat[0, :256] = torch.arange(256, dtype=torch.uint8)     # every code, NaN among them
    slots = torch.randint(0, n_pool, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)   # duplicates too
    slots[0] = 0
    got = mv.kv_read_fp8(lat.cuda(), sc.cuda(), rope.cuda(), slots.cuda()).cpu()
    s = slots.long()
    val = torch.from_numpy(ref.e4m3_values().astype(np.float32))[lat[s].long()]
    want = torch.cat([(val * sc[s][:, None]).to(torch.bfloat16), rope[s]], 1)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert bits_equal(torch.where(nan, torch.zeros_like(got), got), torch.where(nan, torch.zeros_like(want), want))
    assert mv.device_status() == 0


def test_bad_slots(cuda_lib):
    mv = cuda_lib
    c = cache(50, seed=4)
    rows = rows_of(6, seed=5)
    slots = torch.tensor([3, -1, 50, 7, 2 ** 31 - 1, 9], dtype=torch.int32)
    good = torch.tensor([0, 3, 5])
    dev = [t.cuda() for t in c]
    mv.device_status(clear=True)
    mv.kv_append_quant(*dev, slots.cuda(), rows.cuda())
    assert mv.device_status(clear=True) == mv.DEV_BAD_SLOT
    for got, want in zip(dev, expect(*c, slots[good], rows[good])):
        assert bits_equal(got, want)
    back = mv.kv_read_fp8(*dev, slots.cuda()).cpu()
    assert mv.device_status(clear=True) == mv.DEV_BAD_SLOT
    assert int(back[[1, 2, 4]].count_nonzero()) == 0
    assert bits_equal(back[good], mv.kv_read_fp8(*dev, slots[good].cuda()))


def test_no_rows(cuda_lib):
    mv = cuda_lib
    c = cache(5, seed=6)
    dev = [t.cuda() for t in c]
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    mv.kv_append_quant(*dev, none, torch.zeros((0, 576), dtype=torch.bfloat16, device="cuda"))
    assert mv.kv_read_fp8(*dev, none).shape == (0, 576)
    torch.cuda.synchronize()
    assert all(bits_equal(a, b) for a, b in zip(dev, c))


def test_appended_rows_serve_the_sparse_decode(cuda_lib):
    """The cache that the quantising append writes is the one mla_sparse_fp8_decode reads."""
    mv = cuda_lib
    n, B, H = 400, 2, 16
    rows = rows_of(n, seed=11, spread=0.3)
    dev = [torch.zeros_like(t).cuda() for t in cache(n, seed=12)]
    mv.kv_append_quant(*dev, torch.arange(n, dtype=torch.int32, device="cuda"), rows.cuda())
    q = torch.randn((B, H, 576), generator=torch.Generator().manual_seed(13)).to(torch.bfloat16)
    topk = torch.stack([torch.randperm(n, generator=torch.Generator().manual_seed(b))[:300] for b in range(B)]).to(torch.int32)
    out, lse = mv.sparse_fp8_decode(q.cuda(), *dev, topk.cuda(), w.default_scale())
    torch.cuda.synchronize()
    code, scale = ref.quantise(rows.float().numpy())
    u16 = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)
    ro, rl = oracle.sparse_fp8(u16(q), code, scale, u16(rows[:, 512:]), topk.numpy(), w.default_scale())
    # that kernel rounds each key value to bf16: a score moves by at most 2^-8 scale sum |q k|, the
    # lse by no more, and an output by the scores' two-sided error and two more bf16 roundings
    kk = ref.dequantise_rows(code, scale, ref.f64(rows[:, 512:]))
    qs = ref.f64(q)
    for b in range(B):
        k = kk[topk[b].numpy()]
        ds = 2.0 ** -8 * w.default_scale() * (np.abs(qs[b]) @ np.abs(k).T).max(1) + 1e-5
        assert np.all(np.abs(lse[b].double().cpu().numpy() - rl[b]) <= ds)
        p = np.exp(w.default_scale() * qs[b] @ k.T - rl[b][:, None])
        size = p @ np.abs(k[:, :512])
        tol = size * (2 * ds[:, None] * 1.1 + 2.05 * 2.0 ** -8) + 1e-5
        assert np.all(np.abs(out[b].double().cpu().numpy() - ro[b]) <= tol)
