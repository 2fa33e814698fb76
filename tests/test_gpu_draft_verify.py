"""mla_draft_verify against the float64 walk (step_ref.accept): whole numbers, so equal."""
import numpy as np
import pytest
import torch

import step_ref as ref
import workloads as w

pytestmark = pytest.mark.gpu


def rows(rng, *shape, size=3.0):
    z = size * rng.normal(size=shape)
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def make(B, q_len, V, *, seed, tree, drafter=True, noise=1.0, size=3.0):
    rng = np.random.default_rng(seed)
    p = rows(rng, B, q_len, V, size=size)
    q = (p.astype(np.float64) ** 0.8) * np.exp(noise * rng.normal(size=p.shape))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    par = w.tree_parents(seed, B, q_len).astype(np.int32) if tree else None
    tok = np.zeros((B, q_len), np.int32)
    for b in range(B):
        for i in range(1, q_len):
            d = q[b, par[b, i] if tree else i - 1].astype(np.float64)
            tok[b, i] = min(int(np.searchsorted(np.cumsum(d), rng.random() * d.sum(), side="right")), V - 1)
    u = rng.random((B, q_len)).astype(np.float32)
    un = rng.random(B).astype(np.float32)
    return p, q if drafter else None, tok, par, u, un


def call(mv, c):
    t = [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in c]
    got = mv.draft_verify(*t)
    torch.cuda.synchronize()
    return [g.cpu().numpy() for g in got]


def check(mv, c, status=0):
    n, toks, path = call(mv, c)
    p, q, tok, par, u, un = c
    for b in range(p.shape[0]):
        en, et, ep = ref.accept(p[b], None if q is None else q[b], tok[b], None if par is None else par[b], u[b], un[b])
        assert n[b] == en and path[b].tolist() == ep, f"stream {b}: {n[b]} {path[b]} for {en} {ep}"
        assert toks[b].tolist() == et, f"stream {b}: {toks[b]} for {et}"
    assert mv.device_status(clear=True) == status
    return n, toks, path


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("B,q_len,V", [(1, 1, 1), (1, 1, 5), (3, 2, 2), (4, 9, 7), (2, 9, 1000), (1, 64, 130), (17, 5, 2049),
                                       (2, 4, 32000), (1, 3, 131072), (1, 2, 200003), (70, 3, 33)])
def test_against_float64(cuda_lib, B, q_len, V, tree, drafter):
    check(cuda_lib, make(B, q_len, V, seed=B + q_len + V, tree=tree, drafter=drafter, size=1.0 if V < 10 else 3.0))


def test_wide_tree_many_rejections(cuda_lib):
    """All nodes children of the root, drawn from a drafter far from the target: sum after sum."""
    rng = np.random.default_rng(1)
    B, q_len, V = 6, 33, 5000
    p, q, tok, _, u, un = make(B, q_len, V, seed=5, tree=False, noise=4.0)
    par = np.zeros((B, q_len), np.int32)
    for b in range(B):
        tok[b] = rng.choice(V, q_len, p=q[b, 0].astype(np.float64) / q[b, 0].astype(np.float64).sum())
    u[:] = 0.2 + 0.8 * u
    n, _, path = check(cuda_lib, (p, q, tok, par, u, un))
    assert (path[:, 0] > 3).any()                      # some stream went through several rejections
    check(cuda_lib, (p, None, tok, par, u, un))


def test_exact_borders(cuda_lib):
    """Dyadic probabilities, where every sum and product is exact: ties go by the definition."""
    V = 8
    p = np.full((1, 2, V), 0.125, np.float32)
    q = np.zeros((1, 2, V), np.float32)
    q[0, :, 3] = 0.5
    q[0, :, 4] = 0.5
    tok = np.array([[0, 3]], np.int32)
    for u, un in [(0.25, 0.0), (np.nextafter(np.float32(0.25), np.float32(0)), 0.5), (0.75, 0.5),
                  (0.5, 1 / 6), (0.9, 0.99999994), (0.0, 0.125), (0.0, 0.875), (0.0, 0.0)]:
        c = (p, q, tok, None, np.array([[0.0, u]], np.float32), np.array([un], np.float32))
        check(cuda_lib, c)
    n, toks, _ = call(cuda_lib, (p, q, tok, None, np.array([[0.0, 0.25]], np.float32), np.array([0.0], np.float32)))
    assert n[0] == 0 and toks[0].tolist() == [0, -1]   # u q = p: not accepted
    n, toks, _ = call(cuda_lib, (p, q, tok, None, np.array([[0.0, 0.2]], np.float32), np.array([0.5], np.float32)))
    assert n[0] == 1 and toks[0].tolist() == [3, 4]    # half of p's mass lies below token 4, and is passed


def test_identical_drafter_accepts_everything(cuda_lib):
    p, _, tok, _, u, un = make(5, 9, 999, seed=8, tree=False)
    q = p.copy()
    rng = np.random.default_rng(3)
    for b in range(5):
        for i in range(1, 9):
            d = q[b, i - 1].astype(np.float64)
            tok[b, i] = rng.choice(999, p=d / d.sum())
    n, _, _ = check(cuda_lib, (p, q, tok, None, u, un))
    assert (n == 8).all()


def test_nothing_left_falls_back_to_the_target(cuda_lib):
    """The drafter covers the target everywhere, and the draft is rejected all the same (its token
    has no probability): the next token is drawn from the target's row."""
    V = 64
    p = np.zeros((1, 2, V), np.float32)
    p[0, 0, 10:14] = 0.25
    q = p.copy()
    tok = np.array([[0, 50]], np.int32)
    for un in (0.0, 0.3, 0.6, 0.99):
        _, toks, _ = check(cuda_lib, (p, q, tok, None, np.zeros((1, 2), np.float32), np.array([un], np.float32)))
        assert 10 <= toks[0, 0] < 14


def test_same_token_twice_without_drafter(cuda_lib):
    p, _, tok, _, u, un = make(3, 6, 40, seed=9, tree=False)
    par = np.zeros((3, 6), np.int32)
    tok[:, 1:] = tok[:, 1:2]
    u[:, 1:] = 0.999
    u[:, 4] = 0.0                                      # zero: still no acceptance of a token taken out
    check(cuda_lib, (p, None, tok, par, u, un))


def test_absent_and_bad_nodes(cuda_lib):
    """-1 as a parent: the node is not there.  A parent that is not before its child, or a token
    outside the vocabulary: passed over, with a status bit, and without touching the residual."""
    c = make(4, 9, 500, seed=10, tree=True)
    par = c[3].copy()
    par[1, 4:] = -1
    par[2, 1:] = -1
    check(cuda_lib, (*c[:3], par, *c[4:]))
    par[0, 3] = 3
    par[3, 2] = -5
    check(cuda_lib, (*c[:3], par, *c[4:]), status=cuda_lib.DEV_BAD_DRAFT)
    tok = c[2].copy()
    tok[0, 1], tok[1, 2], tok[3, 1] = 500, -1, 2 ** 31 - 1
    check(cuda_lib, (c[0], c[1], tok, c[3], *c[4:]), status=cuda_lib.DEV_BAD_DRAFT)


def test_odd_probabilities(cuda_lib):
    """NaN, negative and huge entries count as 0, 0 and 1; a row without any gives -1 and a status."""
    c = make(3, 4, 300, seed=11, tree=False)
    p, q = c[0].copy(), c[1].copy()
    p[0, 0, ::7] = np.nan
    p[1, 0, ::5] = -0.3
    q[0, :, 3] = np.nan
    p[2, 0, 17] = 5.0
    check(cuda_lib, (p, q, *c[2:]))
    p[0] = 0.0
    p[1] = np.nan
    n, toks, path = check(cuda_lib, (p, q, *c[2:]), status=cuda_lib.DEV_BAD_DRAFT)
    assert toks[0].tolist() == [-1] * 4 and n[0] == 0


def test_tokens_follow_the_target(cuda_lib):
    """Over many streams the first token that comes out is distributed as the target's row, whatever
    the drafter: every frequency within five standard deviations (fixed seed)."""
    B, V = 40000, 6
    rng = np.random.default_rng(12)
    p1, q1 = rows(rng, V, size=1.0), rows(rng, V, size=1.5)
    p = np.broadcast_to(p1, (B, 4, V)).copy()
    q = np.broadcast_to(q1, (B, 4, V)).copy()
    par = np.broadcast_to(np.array([-1, 0, 0, 0], np.int32), (B, 4)).copy()   # three siblings
    tok = rng.choice(V, (B, 4), p=q1.astype(np.float64) / q1.astype(np.float64).sum()).astype(np.int32)
    u, un = rng.random((B, 4)).astype(np.float32), rng.random(B).astype(np.float32)
    _, toks, _ = call(cuda_lib, (p, q, tok, par, u, un))
    freq = np.bincount(toks[:, 0], minlength=V) / B
    assert np.all(np.abs(freq - p1) <= 5 * np.sqrt(p1 * (1 - p1) / B))


def test_graph_replay_and_given_outputs(cuda_lib):
    mv = cuda_lib
    a, b = make(3, 5, 5000, seed=13, tree=True), make(3, 5, 5000, seed=14, tree=True)
    dev = [torch.from_numpy(x).cuda() for x in a]
    outs = [torch.empty(3, dtype=torch.int32, device="cuda")] + [torch.empty((3, 5), dtype=torch.int32, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mv.draft_verify(*dev, n_accepted=outs[0], tokens=outs[1], path=outs[2], stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for _ in range(5):
            mv.draft_verify(*dev, n_accepted=outs[0], tokens=outs[1], path=outs[2])
    for c in (b, a):
        for d, x in zip(dev, c):
            d.copy_(torch.from_numpy(x))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in range(3):
            en, et, ep = ref.accept(c[0][k], c[1][k], c[2][k], c[3][k], c[4][k], c[5][k])
            assert (int(outs[0][k]), outs[1][k].tolist(), outs[2][k].tolist()) == (en, et, ep)


def test_many_streams_small_vocabulary(cuda_lib):
    """More streams than CTAs fit the GPU at once, one CTA a stream."""
    check(cuda_lib, make(700, 3, 70, seed=15, tree=True, size=1.5))


def test_two_streams_at_once(cuda_lib):
    mv = cuda_lib
    c = make(4, 9, 30000, seed=16, tree=True)
    dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in c]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [mv.draft_verify(*dev, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    want = check(mv, c)
    for g in got:
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(g, want))


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("V", [300001, 1 << 20])
def test_rows_that_are_no_distribution(cuda_lib, V, drafter):
    """Raw scores in place of probabilities: sums that 64 bits would not hold."""
    B, q_len = 2, 3
    p = torch.ones(B, q_len, V, device="cuda")
    q = torch.full_like(p, 2.0 ** -20) if drafter else None
    tok = torch.tensor([[0, 5, 7]] * B, dtype=torch.int32, device="cuda")
    u = torch.full((B, q_len), 0.5, device="cuda")
    for u_next in (0.0, 0.3, 0.999999):
        got = [torch.full(s, 123456789, dtype=torch.int32, device="cuda") for s in ((B,), (B, q_len), (B, q_len))]
        n, toks, path = cuda_lib.draft_verify(p, q, tok, None, u, torch.full((B,), u_next, device="cuda"),
                                              n_accepted=got[0], tokens=got[1], path=got[2])
        assert n.tolist() == [2] * B and path.tolist() == [[1, 2, -1]] * B
        assert toks[:, :2].tolist() == [[5, 7]] * B
        assert bool(((toks[:, 2] >= -1) & (toks[:, 2] < V)).all())
    cuda_lib.device_status(clear=True)
