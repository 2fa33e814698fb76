"""key_weights_fp8 and key_weights against their float64 form: both caches, rules, counted drafts, decay,
borders of tiles, one row to thousands, rows that see nothing, bad lengths and slots."""
import numpy as np
import pytest
import torch

import long_ref as lr
import step_ref as ref
import workloads as w
from test_gpu_attn_rules import KINDS, packed, rules_of

pytestmark = pytest.mark.gpu
SCALE = w.default_scale()


def call(mv, s, args, lse, **kw):
    return (mv.key_weights_fp8 if s.cache == "fp8" else mv.key_weights)(*args, SCALE, lse, **kw)


def true_lse(s, rules):
    _, l, _, _ = lr.attention(ref.f64(s.q), s.keys_of, s.seq, s.mask, SCALE, rules)
    return l.astype(np.float32)


def check(mv, s, rules, *, counted=None, decay=0.9, weights=True, lse=None, inplace=False, status=0, **kw):
    lse = true_lse(s, rules) if lse is None else lse
    g = torch.Generator().manual_seed(5)
    old = torch.rand((s.B, s.stride), generator=g) * 3 if weights else None
    before = torch.full((s.B, s.stride), 7.5)
    out = before.cuda()
    dev_old = old.cuda() if weights else None
    if inplace:
        out, before = dev_old, old
    args = s.on("cuda")
    got = call(mv, s, args, torch.from_numpy(lse).cuda(), weights=dev_old, decay=decay, out=out,
               counted=None if counted is None else torch.from_numpy(counted).cuda(), **rules.on("cuda"), **kw)
    torch.cuda.synchronize()
    assert mv.device_status() == status
    want, tol = lr.key_weights(ref.f64(s.q), s.keys_of, s.seq, s.mask, SCALE, rules, lse.astype(np.float64), counted,
                               None if old is None else old.numpy().astype(np.float64), float(np.float32(decay)),
                               before.numpy().astype(np.float64))
    assert got is out
    d = np.abs(ref.f64(got) - want)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(ref.f64(got)), nan)
    assert np.all(d[~nan] <= tol[~nan]), (float((d - tol)[~nan].max()), np.argwhere((d > tol) & ~nan)[:5])
    return got


SHAPES = [([1], 1, 1, "chain"), ([48, 49, 7], 5, 3, "tree"), ([265], 9, 8, "packed"), ([97, 300, 193], 9, 8, "tree"),
          ([150, 600], 1, 64, "chain"), ([130], 17, 24, "packed"), ([144, 145], 64, 2, "tree"), ([200], 6, 16, "chain"),
          ([96, 33], 1, 128, "chain"), ([75], 16, 128, "tree"), ([70], 64, 128, "chain")]


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("lens,q_len,H,mask", SHAPES)
def test_plain(cuda_lib, cache, lens, q_len, H, mask):
    check(cuda_lib, lr.Step(31, lens, q_len, H, mask=mask, cache=cache), lr.Rules())


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,q_len,H,mask", [([97, 300, 193], 9, 8, "tree"), ([150, 600], 1, 64, "chain"),
                                               ([130], 17, 24, "packed")])
def test_rules(cuda_lib, cache, kind, lens, q_len, H, mask):
    s = lr.Step(33, lens, q_len, H, mask=mask, cache=cache)
    check(cuda_lib, s, rules_of(kind, s))


@pytest.mark.parametrize("window,prefix", [(1, None), (48, 1), (49, 0), (40, 700), (150, 64), (2 ** 31 - 1, 3)])
def test_windows(cuda_lib, window, prefix):
    """Keys between the prefix and the window are not looked at, but their former weights decay."""
    s = lr.Step(35, [400, 150, 9], 3, 4)
    check(cuda_lib, s, lr.Rules(window=window, prefix_lens=None if prefix is None else np.full(3, prefix, np.int32)))


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
def test_counted_drafts(cuda_lib, cache):
    s = lr.Step(37, [90, 200], 6, 8, mask="tree", cache=cache)
    for counted in ([[1, 0, 0, 255, 0, 0], [0] * 6], [[0] * 6, [0, 0, 1, 0, 0, 1]]):
        check(cuda_lib, s, lr.Rules(), counted=np.array(counted, np.uint8))


def test_former_weights(cuda_lib):
    """None, in place, decays of 0, 1 and below 0; a NaN or infinity before stays in its key."""
    s = lr.Step(39, [120, 61], 5, 4)
    check(cuda_lib, s, lr.Rules(), weights=False)
    for decay in (0.0, 1.0, -0.5):
        check(cuda_lib, s, lr.Rules(), decay=decay, inplace=True)
    lse = torch.from_numpy(true_lse(s, lr.Rules())).cuda()
    old = torch.ones((2, s.stride), device="cuda")
    old[0, 3], old[1, 7], old[1, 58] = float("nan"), float("inf"), float("nan")   # (1, 58) is a draft's own key
    got = cuda_lib.key_weights_fp8(*s.on("cuda"), SCALE, lse, weights=old)
    assert got is old and torch.isnan(got[0, 3]) and torch.isinf(got[1, 7])
    assert int(torch.isfinite(got).logical_not().sum()) == 2
    fresh = cuda_lib.key_weights_fp8(*s.on("cuda"), SCALE, lse)
    assert (fresh[1, 61:] == 0).all() and (fresh[0] > 0).all()


def test_log_sums_that_are_not_numbers(cuda_lib):
    """-inf: the row adds nothing; +inf: nothing; NaN: NaN in the keys that the row sees and in no other."""
    s = lr.Step(41, [70, 80], 4, 3)
    lse = true_lse(s, lr.Rules())
    lse[0, 1, 2], lse[0, 2, 0], lse[1, 0, 1] = -np.inf, np.inf, np.nan
    got = check(cuda_lib, s, lr.Rules(), lse=lse)
    assert torch.isnan(got[1, :77]).all() and torch.isfinite(got[1, 77:]).all()


def test_bad_keys_stay_by_themselves(cuda_lib):
    """A NaN in one key's row gives NaN there and nowhere else; where no draft sees it, nothing."""
    s = lr.Step(43, [150], 5, 8)
    lse = true_lse(s, lr.Rules())
    want = call(cuda_lib, s, s.on("cuda"), torch.from_numpy(lse).cuda())
    s.lat[s.table[0, 17], 3] = 0x7F
    s.rope[s.table[0, 60], 5] = float("nan")
    got = call(cuda_lib, s, s.on("cuda"), torch.from_numpy(lse).cuda())
    bad = torch.isnan(got[0])
    assert bad.nonzero().flatten().tolist() == [17, 60]
    assert torch.equal(got[0][~bad], want[0][~bad])
    doc = np.zeros((1, s.stride), np.int32)
    doc[0, [17, 60]] = 4
    assert torch.isfinite(call(cuda_lib, s, s.on("cuda"), torch.from_numpy(lse).cuda(), **lr.Rules(key_doc=doc).on("cuda"))).all()


def test_weights_of_a_row_sum_to_one(cuda_lib):
    """With the attention's own lse every row hands out a weight of 1."""
    mv = cuda_lib
    s = lr.Step(45, [1000, 300, 45], 9, 8, mask="tree")
    rules = lr.Rules(softcap=30.0, slopes=lr.slopes(8), window=200, prefix_lens=np.array([8, 4, 0], np.int32))
    args, dev = s.on("cuda"), rules.on("cuda")
    _, lse = mv.verify_attn_fp8_rules(*args, SCALE, **dev)
    total = mv.key_weights_fp8(*args, SCALE, lse, **dev).double().sum(1)
    assert torch.allclose(total, torch.full_like(total, 72.0), rtol=1e-4)


def test_same_bits_every_time(cuda_lib):
    s = lr.Step(47, [700, 333], 33, 16, cache="bf16")
    args, lse = s.on("cuda"), torch.from_numpy(true_lse(s, lr.Rules())).cuda()
    first = call(cuda_lib, s, args, lse)
    for _ in range(5):
        assert torch.equal(call(cuda_lib, s, args, lse), first)


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
def test_bad_lengths_and_slots(cuda_lib, cache):
    """A stream of a bad length is left alone; a bad slot reads pool row 0 and is reported."""
    mv = cuda_lib
    s = lr.Step(49, [100, 60, 80], 4, 4, cache=cache)
    lse = torch.from_numpy(true_lse(s, lr.Rules())).cuda()
    args = s.on("cuda")
    table, seq = args[-3], args[-2]
    seq[0], seq[1] = 3, s.stride + 1
    out = torch.full((3, s.stride), 5.0, device="cuda")
    call(mv, s, args, lse, out=out)
    assert mv.device_status() == 2
    assert (out[:2] == 5).all() and (out[2, 80:] == 5).all() and (out[2, :80] != 5).all()
    seq.copy_(torch.from_numpy(s.seq))
    table[1, 50], table[2, 79] = (s.lat if cache == "fp8" else s.kv).shape[0], -1
    got = call(mv, s, args, lse)
    assert mv.device_status() == 1
    table[1, 50], table[2, 79] = 0, 0
    assert torch.equal(call(mv, s, args, lse), got) and mv.device_status() == 0


def test_many_streams_wide_table_side_stream(cuda_lib):
    lens = [4 + 7 * (i % 30) for i in range(70)]
    s = lr.Step(51, lens, 4, 4, stride=400)
    check(cuda_lib, s, lr.Rules(window=64, slopes=lr.slopes(4)))
    lse = torch.from_numpy(true_lse(s, lr.Rules())).cuda()
    args = s.on("cuda")
    want = call(cuda_lib, s, args, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(cuda_lib, s, args, lse, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
def test_captured(cuda_lib, cache):
    """Captured once, replayed on other lengths; two graphs that know nothing of each other."""
    mv = cuda_lib
    s = lr.Step(53, [300, 200], 5, 32, cache=cache)
    args = s.on("cuda")
    lse = torch.zeros((2, 5, 32), device="cuda")
    outs = [torch.zeros((2, s.stride), device="cuda") for _ in range(2)]
    call(mv, s, args, lse, out=outs[0])
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(mv, s, args, lse, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for lens in ([300, 200], [120, 7]):
        s.seq[:] = lens
        args[-2].copy_(torch.from_numpy(s.seq))
        l = true_lse(s, lr.Rules())
        lse.copy_(torch.from_numpy(l))
        for o in outs:
            o.fill_(-1)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        want, tol = lr.key_weights(ref.f64(s.q), s.keys_of, s.seq, None, SCALE, lr.Rules(), l.astype(np.float64), None,
                                   None, 1.0, np.full((2, s.stride), -1.0))
        for o in outs:
            assert np.all(np.abs(ref.f64(o) - want) <= tol)


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("lens,q_len,H", [([1500], 9, 8), ([700, 60, 1300], 2, 4), ([400], 40, 16), ([60] * 70, 1, 8)])
def test_expired_waits_end_the_call(cuda_lib, cache, lens, q_len, H):
    """The first tile withheld by the test hook: the status says so, keys without a sum are NaN, and the next call
    on the same buffers is right."""
    mv = cuda_lib
    s = lr.Step(55, lens, q_len, H, cache=cache)
    lse = torch.from_numpy(true_lse(s, lr.Rules())).cuda()
    args = s.on("cuda")
    out = torch.zeros((s.B, s.stride), device="cuda")
    mv.device_status(clear=True)
    assert mv.load().mla_debug_stall_next_launch() == 0
    call(mv, s, args, lse, out=out)
    torch.cuda.synchronize()
    assert mv.device_status(clear=True) == mv.DEV_TIMEOUT
    for b, n in enumerate(lens):
        assert torch.isnan(out[b, :n]).any() and (out[b, n:] == 0).all()
    check(mv, s, lr.Rules())


def test_no_streams(cuda_lib):
    e = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda")
    q, kv = e(0, 3, 4, 576, dtype=torch.bfloat16), e(5, 576, dtype=torch.bfloat16)
    assert cuda_lib.key_weights(q, kv, e(0, 9), e(0), None, 0.1, e(0, 3, 4, dtype=torch.float32)).shape == (0, 9)
    assert cuda_lib.kv_evict(e(0, 9), e(0), e(0, 9, dtype=torch.float32), 4).n_freed.shape == (0,)


def test_rows_of_every_size(cuda_lib):
    """Queries whose elements differ by many orders of magnitude, tiny and huge rows: the two pieces of a query hold
    it to 2^-20 of the row's largest element."""
    s = lr.Step(57, [200], 4, 8)
    g = torch.Generator().manual_seed(1)
    spread = torch.exp2(torch.randint(-24, 1, s.q.shape, generator=g).float())
    row = torch.exp2(torch.tensor([-120., -60., -8., -1., 0., 1., 3., 4.]))[None, None, :, None]
    s.q = (s.q.float() * spread * row * 0.3).to(torch.bfloat16)
    top = np.abs(ref.f64(s.q)).max(-1)
    rules = lr.Rules()
    lse = true_lse(s, rules)
    k = np.abs(s.keys_of(0)[:200, :512]).sum(1).max()
    extra = 2.0 ** -20 * top.max() * k * SCALE            # what the pieces leave out, as an error of the score
    old = torch.zeros((1, s.stride), device="cuda")
    got = call(cuda_lib, s, s.on("cuda"), torch.from_numpy(lse).cuda(), out=old)
    want, tol = lr.key_weights(ref.f64(s.q), s.keys_of, s.seq, None, SCALE, rules, lse.astype(np.float64), None, None, 1.0,
                               np.zeros((1, s.stride)))
    assert np.all(np.abs(ref.f64(got) - want) <= tol + want * extra * 1.01)
    s.q[0, 1, 3, 100] = float("inf")
    got = call(cuda_lib, s, s.on("cuda"), torch.from_numpy(lse).cuda())
    assert torch.isnan(got[0, :198]).all() and torch.isfinite(got[0, 198:200]).all()   # the keys that draft 1 sees


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("kind", ["docs", "window", "hidden", "seen"])
@pytest.mark.parametrize("lens,q_len,H", [([700 - i for i in range(100)], 1, 1), ([3300, 2900], 16, 128), ([9000, 40], 32, 64)])
def test_keys_that_no_draft_sees(cuda_lib, cache, kind, lens, q_len, H):
    """Long runs of hidden keys are left out: their former weights decay, with one row tile and with several."""
    s = lr.Step(41, lens, q_len, H, cache=cache)
    doc = packed(lens, s.stride, (0.3, 0.7))
    if kind == "hidden":
        doc[:] = 3
        for b, n in enumerate(lens):
            doc[b, n - q_len:n] = 4
    elif kind == "seen":
        doc[:] = 1
    rules = lr.Rules(key_doc=doc)
    if kind == "window":
        rules = lr.Rules(key_pos=lr.gaps(3, s.B, s.stride), window=200, prefix_lens=np.full(s.B, 64, np.int32))
    need = cuda_lib.load().mla_key_weights_workspace_bytes(s.B, q_len, H, s.stride)
    room = torch.empty(need + 256 + 8 * s.B, dtype=torch.uint8, device="cuda")
    for inplace in (False, True):
        check(cuda_lib, s, rules, inplace=inplace, workspace=room)
    check(cuda_lib, s, rules, weights=False, workspace=room)
