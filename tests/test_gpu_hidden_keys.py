"""The search for keys that no draft sees leaves out hidden keys and no others: inputs that count the keys
(counted_keys.py), in tables of every width class of the search (a cluster of eight, four and two CTAs a
stream, and one).  Queries are zero, so every score is: the attention's log-sum-exp is the logarithm of the
number of keys seen, and with a log-sum-exp of zero a key's weight is the number of rows that see it, a whole
number.  One key too few or too many shows."""
import numpy as np
import pytest
import torch

import long_ref as lr
import step_ref as ref
from counted_keys import Counted

pytestmark = pytest.mark.gpu


def docs(kind, c):
    """(key_doc, positions, window, prefix) by which streams hide their keys."""
    r = np.random.default_rng(5)
    B, st = c.table.shape
    doc = np.zeros((B, st), np.int32)
    for b, n in enumerate(c.seq):
        for i, share in enumerate((0.31, 0.63)):
            doc[b, int(share * n):] = i + 1
        if kind == "islands":                             # single shared keys within the hidden ones
            doc[b, r.integers(0, n, max(1, n // 1500))] = -1
        elif kind == "first":                             # the drafts go on with the first document
            doc[b, n - c.q_len:n] = 0
    if kind == "seen":
        doc[:] = 7
    if kind == "window":
        return None, lr.gaps(3, B, st), 400, r.integers(0, 200, B).astype(np.int32)
    return doc, None, 0, None


def expected_rows(c, rules):
    """Of each stream: bool [q_len, n], the keys that each draft sees."""
    return [np.stack([rules.seen(c.mask, b, t, int(n), c.q_len)[0] for t in range(c.q_len)]) for b, n in enumerate(c.seq)]


def cuda(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


# streams (the first one is the longest), rows of drafts, heads
BATCHES = [([20000], 2, 1), ([24000, 20011, 90], 3, 2), ([9000] + [40 + 97 * i for i in range(20)], 1, 8),
           ([8300, 8200] + [30 + 41 * i for i in range(45)], 2, 4), ([8250] + [33 + 19 * i for i in range(79)], 1, 4)]


@pytest.mark.parametrize("kind", ["last", "first", "islands", "seen", "window"])
@pytest.mark.parametrize("lens,q_len,H", BATCHES)
def test_attention(cuda_lib, lens, q_len, H, kind):
    mv = cuda_lib
    c = Counted(q_len, H, lens, seed=len(lens), mask=q_len > 1)
    doc, pos, window, prefix = docs(kind, c)
    rules = lr.Rules(key_doc=doc, key_pos=pos, window=window, prefix_lens=prefix)
    q = torch.zeros((c.B, q_len, H, 576), dtype=torch.bfloat16, device="cuda")
    args = (q, cuda(c.lat), cuda(c.scale), cuda(c.rope).to(torch.bfloat16), cuda(c.table), cuda(c.seq), cuda(c.mask), 1.0)
    rows = expected_rows(c, rules)
    for nsplit in (1, 0):
        out, lse = (ref.f64(x) for x in mv.verify_attn_fp8_rules(*args, **rules.on("cuda"), nsplit=nsplit))
        assert mv.device_status(clear=True) == 0
        for b in range(c.B):
            for t in range(q_len):
                s = c.table[b, :c.seq[b]][rows[b][t]]
                if len(s):
                    assert c.agree(out[b, t], lse[b, t], *c.expected(s)), (b, t, nsplit)
                else:
                    assert np.all(out[b, t] == 0) and np.all(np.isneginf(lse[b, t])), (b, t, nsplit)


def counts(c, rules, H, stride):
    """[B, stride]: the rows that see each key; -1 behind a stream's last."""
    want = np.full((c.B, stride), -1.0)
    for b, v in enumerate(expected_rows(c, rules)):
        want[b, :v.shape[1]] = v.sum(0) * H
    return want


def weights_call(mv, cache, c, H):
    q = torch.zeros((c.B, c.q_len, H, 576), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((c.B, c.q_len, H), device="cuda")
    table, seq, mask = cuda(c.table), cuda(c.seq), cuda(c.mask)
    if cache == "fp8":
        rows = (cuda(c.lat), cuda(c.scale), cuda(c.rope).to(torch.bfloat16))
        f = mv.key_weights_fp8
    else:
        rows = (torch.ones((len(c.lat), 576), dtype=torch.bfloat16, device="cuda"),)
        f = mv.key_weights
    need = mv.load().mla_key_weights_workspace_bytes(c.B, c.q_len, H, c.table.shape[1])
    room = torch.empty(need + 256 + 8 * c.B, dtype=torch.uint8, device="cuda")
    return seq, lambda out, rules: f(q, *rows, table, seq, mask, 1.0, lse, out=out, workspace=room, **rules)


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("kind", ["last", "first", "islands", "seen", "window"])
@pytest.mark.parametrize("lens,q_len,H", BATCHES + [([9000, 40], 17, 16)])
def test_key_weights(cuda_lib, lens, q_len, H, kind, cache):
    mv = cuda_lib
    c = Counted(q_len, H, lens, seed=len(lens), mask=q_len > 1)
    doc, pos, window, prefix = docs(kind, c)
    rules = lr.Rules(key_doc=doc, key_pos=pos, window=window, prefix_lens=prefix)
    _, call = weights_call(mv, cache, c, H)
    out = torch.full(c.table.shape, -1.0, device="cuda")
    call(out, rules.on("cuda"))
    assert np.array_equal(ref.f64(out), counts(c, rules, H, c.table.shape[1])) and mv.device_status() == 0


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("lens,q_len,H", [([20000, 9000], 2, 4), ([9000, 40], 17, 16)])
def test_key_weights_captured(cuda_lib, lens, q_len, H, cache):
    """Captured once, replayed on other documents and other lengths: the search runs anew each time."""
    mv = cuda_lib
    c = Counted(q_len, H, lens, seed=2, mask=True)
    doc = docs("last", c)[0]
    on = lr.Rules(key_doc=doc).on("cuda")
    seq, call = weights_call(mv, cache, c, H)
    out = torch.zeros(c.table.shape, device="cuda")
    call(out, on)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, on)
    for kind, now in (("last", lens), ("islands", lens), ("seen", [n - n // 3 for n in lens]), ("first", [lens[0] - 1, 33]),
                      ("last", [q_len, lens[1]])):
        c.seq[:] = now
        doc = docs(kind, c)[0]
        seq.copy_(torch.from_numpy(c.seq))
        on["key_doc"].copy_(torch.from_numpy(doc))
        out.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ref.f64(out), counts(c, lr.Rules(key_doc=doc), H, c.table.shape[1])), kind
        assert mv.device_status() == 0


def test_bad_lengths(cuda_lib):
    """Streams of bad lengths between others that are searched: reported and left alone, the others exact."""
    mv = cuda_lib
    q_len, H = 2, 4
    c = Counted(q_len, H, [9000, 8500, 8700, 400], seed=8, mask=True)
    doc = docs("last", c)[0]
    rules = lr.Rules(key_doc=doc)
    want = counts(c, rules, H, c.table.shape[1])
    seq, call = weights_call(mv, "fp8", c, H)
    seq[1], seq[2] = 1, 9001
    want[1:3] = -1
    out = torch.full(c.table.shape, -1.0, device="cuda")
    on = rules.on("cuda")
    call(out, on)
    assert np.array_equal(ref.f64(out), want) and mv.device_status(clear=True) == 2
    q = torch.zeros((c.B, q_len, H, 576), dtype=torch.bfloat16, device="cuda")
    for nsplit in (1, 0):
        o, lse = (ref.f64(x) for x in mv.verify_attn_fp8_rules(q, cuda(c.lat), cuda(c.scale), cuda(c.rope).to(torch.bfloat16),
                                                               cuda(c.table), seq, cuda(c.mask), 1.0, nsplit=nsplit, **on))
        assert mv.device_status(clear=True) == 2
        assert np.isnan(lse[1:3]).all() and np.all(o[1:3] == 0)
        for b in (0, 3):
            for t, see in enumerate(expected_rows(c, rules)[b]):
                s = c.table[b, :c.seq[b]][see]
                assert c.agree(o[b, t], lse[b, t], *c.expected(s)), (b, t, nsplit)
