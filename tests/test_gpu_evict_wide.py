"""kv_evict in tables that are wider than its clusters take, right behind the kernels that leave its weights and
lengths: its kernels read weights, slots and lengths before they wait for the kernel ahead of them.  Eagerly
and replayed from a graph on changed inputs, into other tables and in place, bit for bit."""
import numpy as np
import pytest
import torch

import long_ref as lr
import step_ref as ref
from test_gpu_kv_evict import same_bits

pytestmark = pytest.mark.gpu
B, STRIDE, POOL, SINK, RECENT = 2, 300000, 5000, 4, 256
NAMES = ("table_out", "lens_out", "weights_out", "pos_out", "doc_out", "freed", "n_freed")


class Loop:
    """Weights of one query over rows that many keys share (so that many weights tie), then the eviction."""

    def __init__(self, mv, cache, inplace):
        g = torch.Generator().manual_seed(1)
        self.mv, self.inplace = mv, inplace
        rows = torch.randn((POOL, 576), generator=g).to(torch.bfloat16).cuda()
        if cache == "fp8":
            self.rows = (torch.zeros((POOL, 512), dtype=torch.uint8, device="cuda"), torch.zeros(POOL, device="cuda"),
                         torch.zeros((POOL, 64), dtype=torch.bfloat16, device="cuda"))
            mv.kv_append_quant(*self.rows, torch.arange(POOL, dtype=torch.int32, device="cuda"), rows)
        else:
            self.rows = (rows,)
        self.q = torch.zeros((B, 1, 2, 576), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((B, 1, 2), 9.0, device="cuda")
        new = lambda t=torch.int32: torch.zeros((B, STRIDE), dtype=t, device="cuda")
        self.t = dict(table=new(), seq=torch.zeros(B, dtype=torch.int32, device="cuda"), weights=new(torch.float32),
                      key_pos=new(), key_doc=new())
        self.budget = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.out = dict(freed=new(), n_freed=torch.zeros(B, dtype=torch.int32, device="cuda"))
        if not inplace:
            self.out.update(table_out=new(), lens_out=torch.zeros_like(self.budget), weights_out=new(torch.float32),
                            pos_out=new(), doc_out=new())

    def fill(self, seed, lens):
        """Other inputs in the same tensors; what the outputs hold otherwise stays."""
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.host = dict(table=r.integers(0, POOL, (B, STRIDE)).astype(np.int32), seq=np.array(lens, np.int32),
                         weights=(r.random((B, STRIDE)) * 1e-3 * (r.random((B, STRIDE)) < 0.3)).astype(np.float32),
                         key_pos=lr.gaps(seed, B, STRIDE), key_doc=r.integers(-1, 4, (B, STRIDE)).astype(np.int32))
        self.host_budget = r.integers(SINK + RECENT, STRIDE // 2, B).astype(np.int32)
        for k, v in self.host.items():
            self.t[k].copy_(torch.from_numpy(v))
        self.budget.copy_(torch.from_numpy(self.host_budget))
        self.q.copy_(torch.randn(self.q.shape, generator=g).to(torch.bfloat16))

    def weigh(self, out):
        f = self.mv.key_weights_fp8 if len(self.rows) == 3 else self.mv.key_weights
        return f(self.q, *self.rows, self.t["table"], self.t["seq"], None, 0.07, self.lse, weights=self.t["weights"], decay=0.9,
                 out=out)

    def __call__(self):
        t = self.t
        self.weigh(t["weights"])                         # in place; the eviction follows at once
        return self.mv.kv_evict(t["table"], t["seq"], t["weights"], self.budget, sink=SINK, recent=RECENT, key_pos=t["key_pos"],
                                key_doc=t["key_doc"], **self.out)

    def expected(self):
        """Bit for bit, from the weights that the same call leaves when it is alone."""
        w = self.t["weights"].clone()
        self.weigh(w)
        torch.cuda.synchronize()
        x = dict(self.host, weights=w.cpu().numpy())
        host = lambda t: t.cpu().numpy().copy()
        o = dict(freed=host(self.out["freed"]), n_freed=host(self.out["n_freed"]))
        if self.inplace:
            o.update(table_out=x["table"], lens_out=x["seq"], weights_out=x["weights"], pos_out=x["key_pos"], doc_out=x["key_doc"])
        else:
            o.update({k: host(self.out[k]) for k in NAMES[:5]})
        return lr.evict(x["table"], x["seq"], x["weights"], self.host_budget, SINK, RECENT, x["key_pos"], x["key_doc"], o)


INPUTS = [(1, (300000, 200001)), (2, (9000, 299999)), (3, (261, 300000)), (4, (300000, 1))]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("cache", ["fp8", "bf16"])
def test_behind_the_key_weights(cuda_lib, cache, inplace):
    mv = cuda_lib
    loop = Loop(mv, cache, inplace)
    assert mv.load().mla_kv_evict_workspace_bytes(B, STRIDE, int(inplace), mv.num_sms()) > 0   # the wide form
    loop.fill(0, (STRIDE, STRIDE))
    loop()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    loop.fill(0, (STRIDE, STRIDE))
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = loop()
    for how in ("eager", "replayed"):
        for seed, lens in INPUTS:
            loop.fill(seed, lens)
            want = loop.expected()
            got = loop() if how == "eager" else captured
            if how == "replayed":
                g.replay()
            torch.cuda.synchronize()
            assert mv.device_status() == 0
            for name, x in zip(NAMES, got):
                assert same_bits(x.cpu().numpy(), want[name]), (how, seed, name)


def test_lengths_written_just_before(cuda_lib):
    """Lengths and weights that a kernel of the same graph has just written, calls one behind the other on one
    workspace: each sees its own."""
    mv = cuda_lib
    loop = Loop(mv, "bf16", False)
    room = torch.empty(mv.load().mla_kv_evict_workspace_bytes(B, STRIDE, 0, mv.num_sms()), dtype=torch.uint8, device="cuda")
    loop.fill(7, (STRIDE, 250000))
    t, shorter = loop.t, torch.tensor([30000, 7], dtype=torch.int32, device="cuda")
    outs = [{k: torch.full_like(v, -7) for k, v in loop.out.items()} for _ in range(3)]

    def calls():
        for o in outs:
            mv.kv_evict(t["table"], t["seq"], t["weights"], loop.budget, sink=SINK, recent=RECENT, key_pos=t["key_pos"],
                        key_doc=t["key_doc"], workspace=room, **o)
            t["seq"].sub_(shorter)
            t["weights"].mul_(-1.0)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for seed in (7, 8):
        loop.fill(seed, (STRIDE, 250000))
        for o in outs:
            for v in o.values():
                v.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        x = dict(loop.host)
        for o in outs:
            old = {k: np.full(v.shape, -7, v.cpu().numpy().dtype) for k, v in o.items()}
            want = lr.evict(x["table"], x["seq"], x["weights"], loop.host_budget, SINK, RECENT, x["key_pos"], x["key_doc"], old)
            for name in NAMES:
                assert same_bits(o[name].cpu().numpy(), want[name]), (seed, name)
            x["seq"] = x["seq"] - np.array([30000, 7], np.int32)
            x["weights"] = -x["weights"]
    assert mv.device_status() == 0
