"""kv_evict bit for bit against its plain form: budgets, ties, NaN and signed zeros, sinks and recent keys that
meet, in place and into other tables, one key to many, tables left alone past what is named."""
import numpy as np
import pytest
import torch

import long_ref as lr

pytestmark = pytest.mark.gpu
OUTS = ("table_out", "lens_out", "weights_out", "pos_out", "doc_out", "freed", "n_freed")


def make(seed, lens, stride, kind="spread", pos=True, doc=True):
    r = np.random.default_rng(seed)
    B = len(lens)
    weights = np.exp(2.5 * r.standard_normal((B, stride)) - 6).astype(np.float32)
    if kind == "ties":                                    # few values: many ties at the border
        weights = r.integers(-2, 3, (B, stride)).astype(np.float32)
        weights[weights == 0] *= np.where(r.random((weights == 0).sum()) < 0.5, np.float32(-1), np.float32(1))
    elif kind == "same":
        weights[:] = 0.25
    elif kind == "odd":                                   # NaN of both signs, infinities, zeros, denormals
        some = np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, -1e-40, 3.0], np.float32)
        weights = some[r.integers(0, 9, (B, stride))]
    elif kind == "close":                                 # numbers that differ in their last bits only
        weights = (np.float32(1.0).view(np.int32) + r.integers(0, 300, (B, stride)).astype(np.int32)).view(np.float32)
    table = r.permutation(B * stride).reshape(B, stride).astype(np.int32)
    return dict(table=table, seq=np.array(lens, np.int32), weights=weights,
                key_pos=lr.gaps(seed, B, stride) if pos else None,
                key_doc=r.integers(-1, 5, (B, stride)).astype(np.int32) if doc else None)


def same_bits(a, b):
    return np.array_equal(a.view(np.int32), b.view(np.int32))


def run(mv, x, budget, sink, recent, *, inplace, pos_out=True, status=0):
    shape = x["table"].shape
    put = lambda a: None if a is None else torch.from_numpy(a.copy()).cuda()
    t = {k: put(v) for k, v in x.items()}
    freed, n_freed = np.full(shape, -7, np.int32), np.full(shape[0], -7, np.int32)
    if inplace:
        outs = dict(table_out=x["table"], lens_out=x["seq"], weights_out=x["weights"], pos_out=x["key_pos"],
                    doc_out=x["key_doc"], freed=freed, n_freed=n_freed)
        given = dict(freed=put(freed), n_freed=put(n_freed))
    else:
        outs = dict(table_out=np.full(shape, -7, np.int32), lens_out=np.full(shape[0], -7, np.int32),
                    weights_out=np.full(shape, -7, np.float32), pos_out=np.full(shape, -7, np.int32) if pos_out else None,
                    doc_out=None if x["key_doc"] is None else np.full(shape, -7, np.int32), freed=freed, n_freed=n_freed)
        given = {k: put(v) for k, v in outs.items()}
    b = budget if np.isscalar(budget) else torch.from_numpy(budget).cuda()
    got = mv.kv_evict(t["table"], t["seq"], t["weights"], b, sink=sink, recent=recent, key_pos=t["key_pos"],
                      key_doc=t["key_doc"], **given)
    torch.cuda.synchronize()
    assert mv.device_status() == status
    want = lr.evict(x["table"], x["seq"], x["weights"], budget, sink, recent, x["key_pos"], x["key_doc"], outs)
    for name, g in zip(OUTS, got):
        if want[name] is None:
            assert g is None or (inplace and g is None)
            continue
        assert same_bits(g.cpu().numpy(), want[name]), (name, np.argwhere(g.cpu().numpy() != want[name])[:5])
    if not inplace:                                       # the inputs stay
        for k, v in x.items():
            assert v is None or same_bits(t[k].cpu().numpy(), v)
    return got


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "same", "odd", "close"])
@pytest.mark.parametrize("lens,stride,budget,sink,recent", [
    ([1], 1, 1, 0, 0), ([5, 0, 3], 7, 2, 1, 1), ([1000, 31, 32, 33, 999], 1003, 100, 4, 16), ([2500, 1024, 1025], 2600, 1024, 0, 0),
    ([9000, 8192, 8193, 100], 9001, 2048, 3, 64), ([40000], 40000, 5000, 4, 256)])
def test_evict(cuda_lib, lens, stride, budget, sink, recent, kind, inplace):
    run(cuda_lib, make(len(lens) + stride, lens, stride, kind), budget, sink, recent, inplace=inplace)


@pytest.mark.parametrize("budget", [0, 1, 4, 5, 6, 499, 500, 501, 2 ** 31 - 1])
def test_budgets(cuda_lib, budget):
    """Nothing but sinks and recent keys, one more, all but one, all, more than all."""
    for sink, recent in ((0, 0), (2, 3), (300, 300), (0, 500), (2 ** 31 - 1, 2 ** 31 - 1)):
        run(cuda_lib, make(3, [500, 12, 4], 500, "ties"), budget, sink, recent, inplace=True)


@pytest.mark.parametrize("inplace", [False, True])
def test_budget_of_each_stream(cuda_lib, inplace):
    x = make(5, [700, 300, 64, 2000, 50], 2100)
    run(cuda_lib, x, np.array([100, 300, -5, 1999, 0], np.int32), 2, 8, inplace=inplace)


def test_without_positions_and_documents(cuda_lib):
    """pos_out gets the kept keys' indices; without it nothing is written there."""
    x = make(7, [3000, 77], 3100, pos=False, doc=False)
    run(cuda_lib, x, 500, 4, 32, inplace=False)
    run(cuda_lib, x, 500, 4, 32, inplace=False, pos_out=False)
    run(cuda_lib, x, 500, 4, 32, inplace=True)


def test_long_streams(cuda_lib):
    """More keys than any on-chip memory holds, the border's ties far apart."""
    r = np.random.default_rng(1)
    n = 700001
    x = make(9, [n, 300000], n, "spread", doc=False)
    x["weights"][:, r.integers(0, n, n // 3)] = 0.01
    for inplace in (False, True):
        run(cuda_lib, x, 200000, 16, 1024, inplace=inplace)


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_short_streams_in_a_wide_table(cuda_lib, kind):
    """Streams of a few keys, of a round and of several beside a long one."""
    lens = [300000, 50, 0, 9000, 131072, 131073, 1]
    for inplace in (False, True):
        run(cuda_lib, make(19, lens, 300000, kind), 20000, 4, 64, inplace=inplace)
        run(cuda_lib, make(19, lens, 300000, kind), 30, 1, 2, inplace=inplace)


def test_no_choice_in_a_wide_table(cuda_lib):
    """Sinks and recent keys are the whole budget, in place, with more chunks than run at once: every one of them
    needs the length that is replaced."""
    lens = [1000000, 999999, 20, 0, 600000, 300000]
    for budget, sink, recent in ((0, 0, 0), (0, 200001, 200000), (64, 32, 32), (5, 1000000, 0)):
        run(cuda_lib, make(23, lens, 1000000, doc=False), budget, sink, recent, inplace=True)


def test_many_streams(cuda_lib):
    lens = [(37 * i) % 211 for i in range(700)]
    run(cuda_lib, make(11, lens, 211, "ties"), 64, 4, 8, inplace=True)


@pytest.mark.parametrize("inplace", [False, True])
def test_bad_lengths(cuda_lib, inplace):
    x = make(13, [100, 50, 30], 60)
    x["seq"][:] = [61, 50, -1]
    run(cuda_lib, x, 20, 2, 4, inplace=inplace, status=2)


def test_twice_is_once(cuda_lib):
    """A table that is within its budget stays as it is."""
    x = make(15, [900, 200], 900)
    a = run(cuda_lib, x, 128, 4, 32, inplace=True)
    b = cuda_lib.kv_evict(a.slot_table.clone(), a.seq_lens.clone(), a.weights.clone(), 128, sink=4, recent=32)
    assert torch.equal(a.slot_table, b.slot_table) and torch.equal(a.weights, b.weights) and (b.n_freed == 0).all()


def test_captured_and_streams(cuda_lib):
    """Captured once, replayed on other weights; two calls at once on two streams."""
    mv = cuda_lib
    x = make(17, [4000, 3000], 4000, doc=False)
    t = {k: torch.from_numpy(v).cuda() for k, v in x.items() if v is not None}
    sets = [{k: torch.full_like(v, -7) for k, v in dict(table_out=t["table"], lens_out=t["seq"], weights_out=t["weights"],
                                                        pos_out=t["key_pos"], freed=t["table"], n_freed=t["seq"]).items()}
            for _ in range(2)]
    call = lambda o: mv.kv_evict(t["table"], t["seq"], t["weights"], 700, sink=4, recent=60, key_pos=t["key_pos"], **o)
    call(sets[0])
    torch.cuda.synchronize()
    graphs = []
    for o in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for seed in (17, 18, 19):
        x["weights"] = make(seed, [4000, 3000], 4000)["weights"]
        t["weights"].copy_(torch.from_numpy(x["weights"]))
        before = [{k: v.cpu().numpy() for k, v in o.items()} for o in sets]
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, old in zip(sets, before):
            want = lr.evict(x["table"], x["seq"], x["weights"], 700, 4, 60, x["key_pos"], None, old)
            assert all(same_bits(v.cpu().numpy(), want[k]) for k, v in o.items())
