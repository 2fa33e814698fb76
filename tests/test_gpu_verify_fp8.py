"""mla_verify_attn_fp8 against a float64 form, each element at the bound that the kernel's
roundings give (step_ref.attention)."""
import numpy as np
import pytest
import torch

import step_ref as ref
import workloads as w

pytestmark = pytest.mark.gpu


class Case:
    """One call's inputs: an fp8 cache with scattered slots, its unused rows poisoned with NaN."""

    def __init__(self, B, q_len, H, prefixes, *, seed, mask="chain", stride=None, spread=0.5, q_size=1.0,
                 fill=-1, extra=37):
        rng = np.random.default_rng(seed)
        self.B, self.q_len, self.H, self.scale = B, q_len, H, w.default_scale()
        self.seq = np.array([p + q_len for p in prefixes], np.int32)
        total = int(self.seq.sum())
        self.n_pool = total + extra
        perm = rng.permutation(self.n_pool).astype(np.int32)
        stride = int(self.seq.max()) if stride is None else stride
        self.table = np.full((B, stride), fill, np.int32)
        off = 0
        for b in range(B):
            self.table[b, :self.seq[b]] = perm[off:off + self.seq[b]]
            off += int(self.seq[b])
        x = rng.normal(size=(self.n_pool, 512)) * np.exp(spread * rng.normal(size=(self.n_pool, 1)))
        x = torch.from_numpy(x).to(torch.bfloat16)
        self.lat, self.kscale = ref.quantise(x.float().numpy())
        self.rope = torch.from_numpy(rng.normal(size=(self.n_pool, 64))).to(torch.bfloat16)
        unused = perm[off:]
        self.lat[unused] = 0x7F
        self.kscale[unused] = np.nan
        self.rope[torch.from_numpy(unused).long()] = float("nan")
        self.q = torch.from_numpy(q_size * rng.normal(size=(B, q_len, H, 576))).to(torch.bfloat16)
        par = w.tree_parents(seed, B, q_len)
        self.mask = {"chain": None, "none": None, "tree": w.tree_mask_from_parents(par),
                     "packed": w.tree_mask_from_parents(par),
                     "random": (rng.random((B, q_len, q_len)) < 0.4).astype(np.uint8)}[mask]
        self.packed = mask == "packed"

    def device(self):
        m = None
        if self.mask is not None:
            m = torch.from_numpy(w.pack_mask(self.mask).view(np.int64) if self.packed else self.mask).cuda()
        return (self.q.cuda(), torch.from_numpy(self.lat).cuda(), torch.from_numpy(self.kscale).cuda(),
                self.rope.cuda(), torch.from_numpy(self.table).cuda(), torch.from_numpy(self.seq).cuda(), m, self.scale)

    def keys_of(self, b):
        s = self.table[b, :self.seq[b]]
        return ref.dequantise_rows(self.lat[s], self.kscale[s], ref.f64(self.rope[torch.from_numpy(s).long()]))

    def expected(self):
        return ref.attention(ref.f64(self.q), self.keys_of, self.seq, self.mask, self.scale)


def agree(out, lse, want, what=""):
    o, l, t_out, t_lse = want
    go, gl = ref.f64(out), ref.f64(lse)
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(gl), empty), f"{what}: rows without a visible key differ"
    assert np.all(go[empty] == 0), f"{what}: rows without a visible key are zero"
    assert np.all(np.isfinite(go)) and np.all(np.isfinite(gl[~empty])), f"{what}: non-finite values"
    dl = np.abs(gl[~empty] - l[~empty])
    assert np.all(dl <= t_lse[~empty]), f"{what}: lse off by {np.max(dl):.3e}"
    d = np.abs(go - o) - t_out
    assert np.all(d <= 0), f"{what}: out off by {np.max(d):.3e} over its bound"


def check(mv, c, nsplit=0, what=""):
    out, lse = mv.verify_attn_fp8(*c.device(), nsplit=nsplit)
    torch.cuda.synchronize()
    assert out.dtype == torch.bfloat16 and lse.dtype == torch.float32
    agree(out, lse, c.expected(), what or f"nsplit {nsplit}")
    assert mv.device_status() == 0
    return out, lse


SHAPES = [  # B, q_len, H, prefixes, mask
    (1, 1, 1, [0], "chain"), (1, 1, 1, [1], "chain"), (1, 1, 8, [31], "chain"), (1, 9, 8, [0], "tree"),
    (1, 9, 8, [256], "chain"), (2, 9, 8, [63, 64], "packed"), (3, 5, 3, [1, 127, 128], "tree"),
    (1, 9, 64, [500], "tree"), (2, 1, 128, [129, 700], "none"), (4, 2, 20, [10, 300, 77, 0], "random"),
    (1, 64, 4, [200], "packed"), (2, 33, 5, [95, 33], "tree"), (5, 1, 64, [64, 1, 200, 33, 96], "chain"),
    (1, 17, 8, [1000], "random"), (1, 10, 8, [2100], "chain"), (1, 1, 80, [400], "chain"), (1, 1, 81, [90], "chain"),
    # row tiles beside two key stages: 73 to 96 rows, and two or three tiles of them
    (1, 1, 73, [300], "chain"), (2, 12, 8, [500, 96], "tree"), (1, 1, 89, [48], "chain"), (1, 10, 16, [700], "packed"),
    (2, 19, 10, [200, 49], "tree"), (1, 9, 64, [47], "random"),
]


@pytest.mark.parametrize("nsplit", [0, 1, 3])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"B{s[0]}q{s[1]}H{s[2]}n{max(s[3])}{s[4]}")
def test_shapes(cuda_lib, shape, nsplit):
    B, q_len, H, pre, mask = shape
    check(cuda_lib, Case(B, q_len, H, pre, seed=sum(pre) + 7 * q_len + H, mask=mask), nsplit)


def test_many_streams(cuda_lib):
    """More streams than the balanced split takes, of lengths from one to hundreds."""
    pre = [int(x) for x in np.random.default_rng(2).integers(0, 300, 70)]
    pre[3], pre[50] = 0, 0
    check(cuda_lib, Case(70, 2, 4, pre, seed=21, mask="tree"))


def test_long_stream(cuda_lib):
    check(cuda_lib, Case(2, 3, 4, [20000, 3], seed=22, mask="tree"))


@pytest.mark.parametrize("q_size,spread", [(12.0, 0.5), (1e-3, 0.5), (1.0, 3.0), (40.0, 2.0)])
def test_score_and_scale_ranges(cuda_lib, q_size, spread):
    """Peaked and flat softmax rows, key scales over several orders of magnitude."""
    check(cuda_lib, Case(2, 4, 8, [700, 90], seed=23, mask="tree", q_size=q_size, spread=spread))


def test_extreme_key_scales_and_queries(cuda_lib):
    """Zero rows (scale 0), tiny and huge scales in one stream, query rows of very different size."""
    c = Case(1, 4, 8, [300], seed=24)
    s = c.table[0]
    c.lat[s[5]], c.kscale[s[5]] = 0, 0.0
    c.kscale[s[20:40]] *= np.float32(1e-20)
    c.kscale[s[50]] = np.float32(1e-38)
    c.q[0, 1] *= 1e-4
    c.q[0, 2, 3] = 0
    c.q[0, 3, 0, 0] = 300.0
    for ns in (1, 4):
        check(cuda_lib, c, ns)


def test_all_keys_zero(cuda_lib):
    """A cache of zero rows: uniform probabilities over the rope scores, output zero."""
    c = Case(1, 2, 4, [40], seed=25)
    c.lat[c.table[0]], c.kscale[c.table[0]] = 0, 0.0
    out, _ = check(cuda_lib, c, 1)
    assert int(out.count_nonzero()) == 0


def test_rising_scores_rescale(cuda_lib):
    """Scores that climb along the keys, so that the running maximum moves again and again."""
    c = Case(1, 9, 8, [1500], seed=26, spread=0.0)
    s = c.table[0]
    c.kscale[s] = (c.kscale[s] * np.linspace(0.01, 6.0, len(s))).astype(np.float32)
    for ns in (1, 2, 0):
        check(cuda_lib, c, ns)


@pytest.mark.parametrize("part", ["codes", "scale", "rope", "inf scale", "one code"])
def test_nan_in_a_key(cuda_lib, part):
    """A key that holds NaN or an infinity makes NaN of the rows that see it, and of no other."""
    c = Case(1, 4, 8, [100], seed=27, mask="tree")
    c.mask[:] = 0
    c.mask[0, 1, 0] = c.mask[0, 3, 0] = c.mask[0, 3, 2] = 1    # draft 2 as a key: seen by draft 3 alone
    s = c.table[0, 102]
    if part == "codes":
        c.lat[s] = 0x7F
    elif part == "one code":
        c.lat[s, 301] = 0xFF
    elif part == "scale":
        c.kscale[s] = np.nan
    elif part == "inf scale":
        c.kscale[s] = np.inf
    else:
        c.rope[int(s)] = float("nan")
    c.mask[0, 3, 2] = 0
    want = c.expected()
    for ns in (1, 2):
        agree(*cuda_lib.verify_attn_fp8(*c.device(), nsplit=ns), want, what="unseen")
    c.mask[0, 3, 2] = 1
    for ns in (1, 2):
        out, lse = cuda_lib.verify_attn_fp8(*c.device(), nsplit=ns)
        agree(out[:, :3], lse[:, :3], [x[:, :3] for x in want], what="rows beside it")
        if part != "inf scale":                        # an infinite key is infinitely likely or impossible
            assert bool(torch.isnan(lse[:, 3]).all())


def test_no_visible_key(cuda_lib):
    c = Case(2, 3, 4, [0, 0], seed=28, mask="tree")
    c.mask[:] = 0
    c.mask[1, 1, 0] = 1
    for ns in (0, 1, 2):
        check(cuda_lib, c, ns)


def test_padded_table_and_partial_outputs(cuda_lib):
    """Table rows wider than the streams, filled with -1 behind them; given outputs are used."""
    mv = cuda_lib
    c = Case(3, 5, 8, [300, 40, 1], seed=29, mask="packed", stride=1111)
    out = torch.full((3, 5, 8, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 5, 8), 7.0, device="cuda")
    ws = torch.empty(mv.workspace_bytes(3, 5, 8, 8), dtype=torch.uint8, device="cuda")
    o, l = mv.verify_attn_fp8(*c.device(), out=out, lse=lse, workspace=ws, nsplit=8)
    torch.cuda.synchronize()
    assert o.data_ptr() == out.data_ptr() and l.data_ptr() == lse.data_ptr()
    agree(out, lse, c.expected())
    assert mv.device_status() == 0


def test_split_counts_agree_and_runs_repeat(cuda_lib):
    mv = cuda_lib
    c = Case(2, 9, 8, [900, 333], seed=30, mask="tree")
    dev, want = c.device(), c.expected()
    for ns in (1, 2, 5, 16, 64):
        a = mv.verify_attn_fp8(*dev, nsplit=ns)
        b = mv.verify_attn_fp8(*dev, nsplit=ns)
        torch.cuda.synchronize()
        agree(*a, want, what=f"nsplit {ns}")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_lengths_and_slots(cuda_lib):
    mv = cuda_lib
    c = Case(3, 4, 8, [100, 50, 60], seed=31, mask="tree")
    want = c.expected()
    c.seq[1] = 3                                       # fewer keys than drafts
    c.seq[2] = c.table.shape[1] + 1                    # longer than its table row
    for ns in (0, 1, 4):
        mv.device_status(clear=True)
        out, lse = mv.verify_attn_fp8(*c.device(), nsplit=ns)
        assert mv.device_status(clear=True) == mv.DEV_BAD_LEN
        agree(out[:1], lse[:1], [x[:1] for x in want])
        assert int(out[1:].count_nonzero()) == 0 and bool(torch.isnan(lse[1:]).all())
    c = Case(2, 4, 8, [100, 50], seed=32, mask="tree")
    want = c.expected()
    c.table[1, 7] = c.n_pool
    mv.device_status(clear=True)
    out, lse = mv.verify_attn_fp8(*c.device())
    assert mv.device_status(clear=True) == mv.DEV_BAD_SLOT
    agree(out[:1], lse[:1], [x[:1] for x in want])


def test_zero_streams(cuda_lib):
    c = Case(1, 2, 4, [5], seed=33)
    q, lat, sc, rope, table, seq, m, scale = c.device()
    out, lse = cuda_lib.verify_attn_fp8(q[:0], lat, sc, rope, table[:0], seq[:0], None, scale)
    assert out.shape == (0, 2, 4, 512) and lse.shape == (0, 2, 4)


def test_side_stream_and_graph(cuda_lib):
    """On a stream of its own, and captured: ten calls share one workspace, inputs change between replays."""
    mv = cuda_lib
    a = Case(2, 9, 8, [700, 200], seed=34, mask="tree")
    b = Case(2, 9, 8, [700, 200], seed=35, mask="tree")
    dev = a.device()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = mv.verify_attn_fp8(*dev, stream=s)
    s.synchronize()
    agree(out, lse, a.expected())
    ws = torch.empty(mv.workspace_bytes(2, 9, 8, 64), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for _ in range(10):
            mv.verify_attn_fp8(*dev, out=out, lse=lse, workspace=ws)
    for c in (b, a, b):
        for dst, src in zip(dev[:7], c.device()[:7]):
            dst.copy_(src)
        out.zero_()
        lse.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        agree(out, lse, c.expected())
    assert mv.device_status() == 0


def test_two_streams_at_once(cuda_lib):
    """Calls on two streams at the same time, each with a workspace of its own, over one cache."""
    mv = cuda_lib
    c = Case(2, 9, 8, [3000, 700], seed=36, mask="tree")
    dev, want = c.device(), c.expected()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for s in streams:
            got.append(mv.verify_attn_fp8(*dev, stream=s))
    torch.cuda.synchronize()
    for out, lse in got:
        agree(out, lse, want)
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


def test_same_cache_as_the_sparse_decode(cuda_lib):
    """One token a stream over all of its keys: the sparse decode with every key listed, whose keys are
    rounded to bf16 (a score moves by at most 2^-8 scale sum |q k|)."""
    mv = cuda_lib
    c = Case(3, 1, 16, [299, 299, 299], seed=37)
    q, lat, sc, rope, table, seq, _, scale = c.device()
    out, lse = mv.verify_attn_fp8(q, lat, sc, rope, table, seq, None, scale)
    o2, l2 = mv.sparse_fp8_decode(q[:, 0].contiguous(), lat, sc, rope, table, scale)
    torch.cuda.synchronize()
    want = c.expected()
    agree(out, lse, want)
    for b in range(3):
        k = c.keys_of(b)
        ds = 2.0 ** -8 * scale * (np.abs(ref.f64(c.q[b, 0])) @ np.abs(k).T).max(1)
        assert np.all(np.abs(ref.f64(l2[b]) - want[1][b, 0]) <= ds + want[3][b, 0])
        p = np.exp(scale * ref.f64(c.q[b, 0]) @ k.T - want[1][b, 0][:, None])
        size = p @ np.abs(k[:, :512])
        assert np.all(np.abs(ref.f64(o2[b]) - want[0][b, 0]) <= want[2][b, 0] + size * (2.2 * ds[:, None] + 2.0 ** -8))


def test_expired_wait_reports_timeout_and_context_survives(cuda_lib):
    """The gather withholds its first arrival (test hook): the bounded waits run out, the status says
    so, the outputs are finite, and the next call is exact again."""
    mv = cuda_lib
    c = Case(1, 9, 8, [200], seed=38, mask="tree")
    dev = c.device()
    mv.device_status(clear=True)
    assert mv.load().mla_debug_stall_next_launch() == 0
    out, _ = mv.verify_attn_fp8(*dev)
    torch.cuda.synchronize()
    assert mv.device_status(clear=True) & mv.DEV_TIMEOUT
    assert bool(torch.isfinite(out).all())
    check(mv, c)


def test_rescale_branch_runs(cuda_lib):
    """The rising scores of test_rising_scores_rescale really move the running maximum."""
    mv = cuda_lib
    c = Case(1, 9, 8, [1500], seed=39, spread=0.0, q_size=6.0)
    s = c.table[0]
    c.kscale[s] = (c.kscale[s] * np.linspace(0.01, 6.0, len(s))).astype(np.float32)
    mv.debug_rescale_count()
    check(mv, c, 1)
    assert mv.debug_rescale_count() > 0
