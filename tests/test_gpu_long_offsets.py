"""The long-context operators where byte and element offsets pass 32 bits: rows far out in a large cache, the last
stream of tables with more than 2^31 entries.  Against the same call on small tensors."""
import numpy as np
import pytest
import torch

import long_ref as lr
import workloads as w
from test_gpu_attn_rules import packed

pytestmark = pytest.mark.gpu
SCALE = w.default_scale()
ROWS = 9_000_000                                          # 4.6 GB of codes, 10.4 GB of bf16 rows
B, STRIDE = 520, 1 << 22                                  # 2.2e9 entries a table


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("not enough free memory on this GPU")


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
def test_rows_far_out(cuda_lib, cache):
    mv = cuda_lib
    room(24)
    s = lr.Step(61, [500, 77], 3, 8, cache=cache)
    q, *small, table, seq, mask = s.on("cuda")
    rules = lr.Rules(softcap=20.0, key_doc=packed([500, 77], s.stride, (0.5, 0.8))).on("cuda")
    n = small[0].shape[0]
    large = [torch.empty((ROWS, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in small]
    for t, u in zip(large, small):
        t[ROWS - n:] = u
    far = table + (ROWS - n)
    lse = torch.rand((2, 3, 8), device="cuda")
    f = mv.key_weights_fp8 if cache == "fp8" else mv.key_weights
    got = [f(q, *c, tb, seq, mask, SCALE, lse, **rules) for c, tb in ((small, table), (large, far))]
    assert torch.equal(*got)
    if cache == "fp8":
        a, b = [mv.verify_attn_fp8_rules(q, *c, tb, seq, mask, SCALE, **rules) for c, tb in ((small, table), (large, far))]
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert mv.device_status() == 0


def test_last_stream_of_large_tables(cuda_lib):
    """Every other stream holds one key."""
    mv = cuda_lib
    room(64)
    s = lr.Step(67, [6000], 1, 4)
    q, lat, scale, rope, table, seq, _ = s.on("cuda")
    doc = torch.from_numpy(packed([6000], 6000, (0.4, 0.7))).cuda()
    lse, weights = torch.rand((1, 1, 4), device="cuda"), torch.rand((1, 6000), device="cuda")
    tables = []
    for t in (table, doc, weights):
        u = torch.empty((B, STRIDE), dtype=t.dtype, device="cuda")
        u[:, 0] = 0
        u[-1, :6000] = t[0]
        tables.append(u)
    qs, lses = q.expand(B, 1, 4, 576).contiguous(), lse.expand(B, 1, 4).contiguous()
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    lens[-1] = 6000
    want = mv.verify_attn_fp8_rules(q, lat, scale, rope, table, seq, None, SCALE, softcap=20.0, key_doc=doc, nsplit=4)
    got = mv.verify_attn_fp8_rules(qs, lat, scale, rope, tables[0], lens, None, SCALE, softcap=20.0, key_doc=tables[1], nsplit=4)
    assert torch.equal(got[0][-1], want[0][0]) and torch.equal(got[1][-1], want[1][0])
    new = mv.key_weights_fp8(q, lat, scale, rope, table, seq, None, SCALE, lse, key_doc=doc, weights=weights, decay=0.5)
    out = mv.key_weights_fp8(qs, lat, scale, rope, tables[0], lens, None, SCALE, lses, key_doc=tables[1], weights=tables[2], decay=0.5)
    assert torch.equal(out[-1, :6000], new[0])
    assert mv.device_status() == 0


@pytest.mark.parametrize("inplace", [False, True])
def test_eviction_of_the_last_stream_of_large_tables(cuda_lib, inplace):
    mv = cuda_lib
    room(100)
    n = 100000
    r = np.random.default_rng(71)
    table, weights = r.permutation(n).astype(np.int32)[None], r.random((1, n), dtype=np.float32)
    outs = dict(table_out=table, lens_out=np.array([n], np.int32), weights_out=weights, pos_out=None, doc_out=None,
                freed=np.zeros((1, n), np.int32), n_freed=np.zeros(1, np.int32))
    want = lr.evict(table, np.array([n], np.int32), weights, 3000, 4, 50, None, None, outs)
    big = lambda dtype: torch.empty((B, STRIDE), dtype=dtype, device="cuda")
    t, x, lens = big(torch.int32), big(torch.float32), torch.zeros(B, dtype=torch.int32, device="cuda")
    t[-1, :n], x[-1, :n], lens[-1] = torch.from_numpy(table[0]), torch.from_numpy(weights[0]), n
    more = {} if inplace else dict(table_out=big(torch.int32), weights_out=big(torch.float32))
    e = mv.kv_evict(t, lens, x, 3000, sink=4, recent=50, **more)
    assert int(e.seq_lens[-1]) == 3000 and int(e.n_freed[-1]) == n - 3000 and int(e.seq_lens[:-1].sum()) == 0
    assert np.array_equal(e.slot_table[-1, :3000].cpu().numpy(), want["table_out"][0, :3000])
    assert np.array_equal(e.weights[-1, :3000].cpu().numpy(), want["weights_out"][0, :3000])
    assert np.array_equal(e.freed[-1, :n - 3000].cpu().numpy(), want["freed"][0, :n - 3000])
    assert mv.device_status() == 0
