"""verify_attn_fp8_rules against its float64 form: caps, distance biases, windows, prefixes, documents, and
what they do together, at tile and split borders and where rows see nothing."""
import numpy as np
import pytest
import torch

import long_ref as lr
import step_ref as ref
import workloads as w

pytestmark = pytest.mark.gpu
SCALE = w.default_scale()


def check(mv, s, rules, **kw):
    out, lse = mv.verify_attn_fp8_rules(*s.on("cuda"), SCALE, **rules.on("cuda"), **kw)
    torch.cuda.synchronize()
    assert mv.device_status() == 0
    o, l, t_out, t_lse = lr.attention(ref.f64(s.q), s.keys_of, s.seq, s.mask, SCALE, rules)
    got_o, got_l = ref.f64(out), ref.f64(lse)
    none = np.isneginf(l)
    assert np.array_equal(np.isneginf(got_l), none) and np.all(got_o[none] == 0)
    assert np.all(np.abs(got_o - o) <= t_out), float(np.max(np.abs(got_o - o) - t_out))
    assert np.all(np.abs(got_l[~none] - l[~none]) <= t_lse[~none])
    return out, lse


def rules_of(kind, s):
    B, st, H = s.B, s.stride, s.H
    r = np.random.default_rng(7)
    docs = np.sort(r.integers(-1, 3, (B, st)), 1).astype(np.int32)
    return {
        "cap": lambda: lr.Rules(softcap=5.0),
        "bias": lambda: lr.Rules(slopes=lr.slopes(H)),
        "window": lambda: lr.Rules(window=50),
        "window-prefix": lambda: lr.Rules(window=33, prefix_lens=r.integers(0, 40, B).astype(np.int32)),
        "window-pos": lambda: lr.Rules(window=50, key_pos=lr.gaps(1, B, st)),
        "prefix": lambda: lr.Rules(prefix_lens=(s.seq - 1).astype(np.int32)),
        "docs": lambda: lr.Rules(key_doc=docs),
        "all": lambda: lr.Rules(softcap=30.0, slopes=lr.slopes(H), key_pos=lr.gaps(2, B, st), window=90,
                                prefix_lens=r.integers(0, 20, B).astype(np.int32), key_doc=docs),
    }[kind]()


KINDS = ("cap", "bias", "window", "window-prefix", "window-pos", "prefix", "docs", "all")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,q_len,H,mask,nsplit", [
    ([1], 1, 1, "chain", 0), ([48, 49, 7], 5, 3, "tree", 1), ([265], 9, 8, "packed", 0), ([97, 300, 193], 9, 8, "tree", 3),
    ([150, 600], 1, 64, "chain", 0), ([130], 17, 24, "packed", 2), ([144, 145], 64, 2, "tree", 0), ([200], 6, 16, "chain", 0)])
def test_rules(cuda_lib, kind, lens, q_len, H, mask, nsplit):
    s = lr.Step(3 + len(lens), lens, q_len, H, mask=mask)
    check(cuda_lib, s, rules_of(kind, s), nsplit=nsplit)


def test_no_rules_is_the_plain_attention(cuda_lib):
    """Every rule off: bit for bit verify_attn_fp8."""
    s = lr.Step(1, [500, 77, 260], 9, 8, mask="tree")
    args = s.on("cuda")
    a = cuda_lib.verify_attn_fp8(*args, SCALE)
    b = cuda_lib.verify_attn_fp8_rules(*args, SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("cap", [0.05, 1.0, 4.0, 30.0, 1e4, 1e30])
def test_caps(cuda_lib, cap):
    """Small caps flatten every score, huge ones leave them: tanh is right near zero, far out and between."""
    check(cuda_lib, lr.Step(9, [130, 60], 4, 8, q_size=4.0), lr.Rules(softcap=cap))


@pytest.mark.parametrize("window", [1, 2, 47, 48, 49, 96, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("prefix", [None, 0, 1, 48, 5000])
def test_windows(cuda_lib, window, prefix):
    """Windows and prefixes at tile borders; keys between them are skipped, whatever their rows hold."""
    s = lr.Step(11, [400, 150, 9], 3, 4)
    rules = lr.Rules(window=window, prefix_lens=None if prefix is None else np.full(3, prefix, np.int32))
    check(cuda_lib, s, rules)
    check(cuda_lib, s, lr.Rules(window=window, prefix_lens=rules.prefix_lens,
                                key_pos=np.broadcast_to(np.arange(s.stride, dtype=np.int32), (3, s.stride))))


def test_rows_that_see_nothing(cuda_lib):
    """A draft whose mask shows no draft and whose document has no key: out 0, lse -inf, its neighbours right."""
    s = lr.Step(13, [100, 60], 4, 2, mask="tree")
    s.mask[0, 2] = 0
    doc = np.zeros((2, s.stride), np.int32)
    doc[0, 100 - 4 + 2] = 9
    _, lse = check(cuda_lib, s, lr.Rules(key_doc=doc))
    assert torch.isneginf(lse[0, 2]).all() and torch.isfinite(lse[1]).all()


def test_masked_rows_may_hold_anything(cuda_lib):
    """NaN codes, infinite scales and NaN rotated parts in keys that no draft sees change nothing."""
    s = lr.Step(17, [300], 5, 8)
    doc = np.zeros((1, s.stride), np.int32)
    doc[0, 20:200] = 1
    rules = lr.Rules(key_doc=doc, softcap=20.0, slopes=lr.slopes(8))
    want = check(cuda_lib, s, rules)
    bad = s.table[0, 20:200].long()
    s.lat[bad[::2]] = 0x7F
    s.scale[bad[1::3]] = float("inf")
    s.rope[bad[::5]] = float("nan")
    out, lse = cuda_lib.verify_attn_fp8_rules(*s.on("cuda"), SCALE, **rules.on("cuda"))
    assert torch.equal(lse, want[1]) and torch.equal(out, want[0])


def test_far_positions(cuda_lib):
    """Positions near 2^31 and negative ones: differences and the window's edge stay exact."""
    s = lr.Step(19, [200, 90], 4, 4)
    for start in (2 ** 31 - 1 - 2 * 200, -2 ** 31):
        pos = lr.gaps(3, 2, s.stride, start=start)
        check(cuda_lib, s, lr.Rules(slopes=lr.slopes(4), key_pos=pos, window=60))
        check(cuda_lib, s, lr.Rules(slopes=-lr.slopes(4), key_pos=pos, window=2 ** 31 - 1))


@pytest.mark.parametrize("spread", [2 ** 20, 2 ** 24, 2 ** 26, 2 ** 30])
def test_drafts_far_apart(cuda_lib, spread):
    """Positions of keys and drafts alike all over a wide range: distances of a few next to far ones."""
    s = lr.Step(20, [190, 70], 6, 4, mask="tree")
    r = np.random.default_rng(3)
    pos = (r.integers(0, 4, (2, s.stride)) * (spread // 4) + r.integers(0, 50, (2, s.stride))).astype(np.int32)
    for slopes in (lr.slopes(4) * np.float32(8.0 / spread), lr.slopes(4)):
        check(cuda_lib, s, lr.Rules(slopes=slopes, key_pos=pos))
    check(cuda_lib, s, lr.Rules(slopes=slopes, key_pos=pos, window=spread // 4, prefix_lens=np.array([9, 30], np.int32)))


def test_positions_in_any_order(cuda_lib):
    s = lr.Step(21, [170], 9, 8, mask="packed")
    pos = np.random.default_rng(1).permutation(170).astype(np.int32)[None]
    check(cuda_lib, s, lr.Rules(slopes=lr.slopes(8), key_pos=pos, window=40, prefix_lens=np.array([12], np.int32)))


def packed(lens, stride, cuts):
    """Documents one behind the other: stream b's start at the given shares of its keys."""
    doc = np.zeros((len(lens), stride), np.int32)
    for b, n in enumerate(lens):
        for i, c in enumerate(cuts):
            doc[b, int(c * n):] = i + 1
    return doc


@pytest.mark.parametrize("kind", ["last", "two", "first", "shared", "blocks", "hidden", "seen", "window", "all"])
@pytest.mark.parametrize("lens,q_len,H,nsplit", [
    ([900, 37, 640], 3, 2, 1), ([700, 31, 32, 33], 1, 24, 3), ([24000, 20000, 90], 2, 1, 0), ([20000], 1, 2, 20)])
def test_keys_that_no_draft_sees(cuda_lib, kind, lens, q_len, H, nsplit):
    """Long runs of keys of other documents or behind the window are left out: at the beginning, between, up to the
    drafts, in pieces, none and all of them."""
    s = lr.Step(29 + len(lens), lens, q_len, H)
    B, st = s.B, s.stride
    doc, more = packed(lens, st, (0.3, 0.62)), {}
    if kind == "two":                                     # drafts of the last two documents
        for b, n in enumerate(lens):
            doc[b, n - q_len:n - q_len // 2] = 1
    elif kind == "first":                                 # drafts of the first one, behind another's keys
        for b, n in enumerate(lens):
            doc[b, n - q_len:n] = 0
    elif kind == "shared":
        doc[:, :70] = -1
        doc[:, ::611] = -1
    elif kind == "blocks":
        doc = np.broadcast_to((np.arange(st, dtype=np.int32) // 32 % 3) * 2, (B, st)).copy()
    elif kind == "hidden":
        doc[:] = 5
        for b, n in enumerate(lens):
            doc[b, n - q_len:n] = 6
    elif kind == "seen":
        doc[:] = 2
    elif kind in ("window", "all"):
        more = dict(key_pos=lr.gaps(5, B, st), window=150, prefix_lens=np.full(B, 40, np.int32))
        if kind == "window":
            doc = None
        else:
            more.update(softcap=20.0, slopes=lr.slopes(H))
    check(cuda_lib, s, lr.Rules(key_doc=doc, **more), nsplit=nsplit)


@pytest.mark.parametrize("B", [20, 50, 130])
def test_keys_that_no_draft_sees_of_many_streams(cuda_lib, B):
    lens = [8200 + 37 * (i % 5) if i % 4 == 0 else 40 + i for i in range(B)]
    s = lr.Step(37, lens, 1, 1)
    check(cuda_lib, s, lr.Rules(key_doc=packed(lens, s.stride, (0.2, 0.9))), nsplit=8)


def test_slots_of_keys_that_no_draft_sees(cuda_lib):
    """What lies in the middle of a long run of another document's keys is not looked at."""
    s = lr.Step(31, [9000, 6000], 4, 2)
    rules = lr.Rules(key_doc=packed([9000, 6000], s.stride, (0.25, 0.75)))
    want = check(cuda_lib, s, rules, nsplit=2)
    args = list(s.on("cuda"))
    table = args[4].clone()
    table[:, 2500:4200] = -1
    args[4] = table
    out, lse = cuda_lib.verify_attn_fp8_rules(*args, SCALE, **rules.on("cuda"), nsplit=2)
    assert cuda_lib.device_status() == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_wide_table_many_streams_and_a_stream(cuda_lib):
    """More streams than the balanced split takes, a table wider than any, another stream, out and lse given."""
    lens = [4 + 7 * (i % 30) for i in range(70)]
    s = lr.Step(23, lens, 4, 4, stride=400)
    out = torch.empty((70, 4, 4, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((70, 4, 4), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = check(cuda_lib, s, lr.Rules(window=64, slopes=lr.slopes(4)), out=out, lse=lse, stream=side)
    assert a is out and b is lse


def test_bad_lengths_and_slots(cuda_lib):
    mv = cuda_lib
    s = lr.Step(25, [100, 60, 80], 4, 4)
    rules = lr.Rules(window=30, prefix_lens=np.array([3, 3, 3], np.int32), slopes=lr.slopes(4))
    q, lat, sc, rope, table, seq, _ = s.on("cuda")
    seq[0], seq[1] = 3, s.stride + 1
    out, lse = mv.verify_attn_fp8_rules(q, lat, sc, rope, table, seq, None, SCALE, **rules.on("cuda"))
    assert mv.device_status() == 2
    assert torch.isnan(lse[:2]).all() and (out[:2] == 0).all() and torch.isfinite(lse[2]).all()
    seq.copy_(torch.from_numpy(s.seq))
    table[1, 58] = s.lat.shape[0]
    table[2, 79] = -1
    mv.verify_attn_fp8_rules(q, lat, sc, rope, table, seq, None, SCALE, **rules.on("cuda"))
    assert mv.device_status() == 1


def test_captured(cuda_lib):
    """Captured once, replayed on other lengths and rules' contents."""
    mv = cuda_lib
    s = lr.Step(27, [300, 200], 5, 8)
    args = s.on("cuda")
    rules = lr.Rules(softcap=20.0, slopes=lr.slopes(8), window=100, prefix_lens=np.array([5, 9], np.int32))
    dev = rules.on("cuda")
    out, lse = torch.empty((2, 5, 8, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 5, 8), device="cuda")
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    call = lambda: mv.verify_attn_fp8_rules(*args, SCALE, **dev, out=out, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens, prefix in (([300, 200], [5, 9]), ([120, 7], [60, 0])):
        s.seq[:] = lens
        args[5].copy_(torch.from_numpy(s.seq))
        rules.prefix_lens = np.array(prefix, np.int32)
        dev["prefix_lens"].copy_(torch.from_numpy(rules.prefix_lens))
        g.replay()
        torch.cuda.synchronize()
        o, l, t_out, t_lse = lr.attention(ref.f64(s.q), s.keys_of, s.seq, None, SCALE, rules)
        assert np.all(np.abs(ref.f64(out) - o) <= t_out) and np.all(np.abs(ref.f64(lse) - l) <= t_lse)


def test_captured_search(cuda_lib):
    """A captured call looks for hidden keys anew at each replay: other documents, other lengths."""
    mv = cuda_lib
    s = lr.Step(53, [900, 700], 3, 4)
    rules = lr.Rules(key_doc=packed([900, 700], s.stride, (0.4, 0.8)))
    args, on = s.on("cuda"), rules.on("cuda")
    call = lambda: mv.verify_attn_fp8_rules(*args, SCALE, **on, nsplit=1)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for cuts, lens in (((0.4, 0.8), (900, 700)), ((0.1, 0.2), (900, 650)), ((0.9, 0.95), (3, 700)), ((2.0, 2.0), (810, 333))):
        on["key_doc"].copy_(torch.from_numpy(packed([900, 700], s.stride, cuts)))
        args[5].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and mv.device_status() == 0
        s.seq = np.array(lens, np.int32)
        check(mv, s, lr.Rules(key_doc=packed([900, 700], s.stride, cuts)), nsplit=1)
