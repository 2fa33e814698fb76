"""Attention under rules, key weights and eviction captured in one graph, replayed on other queries, lengths,
documents, positions and former weights: what every replay leaves is what the same calls leave eagerly, bit for bit."""
import numpy as np
import pytest
import torch

import long_ref as lr
import workloads as w

pytestmark = pytest.mark.gpu
SCALE = w.default_scale()


@pytest.mark.parametrize("lens,q_len,H,stride", [((9000, 8400, 300), 3, 4, 9100), ((600, 20, 333), 2, 80, 700),
                                                 ((140000, 90000, 131073), 1, 8, 140500)])
def test_step_in_one_graph(cuda_lib, lens, q_len, H, stride):
    """Tables of the search's clusters and of one CTA, several row tiles, the eviction's wide form."""
    mv = cuda_lib
    B, pool = len(lens), 4000
    g0 = torch.Generator().manual_seed(2)
    lat, sc = torch.zeros((pool, 512), dtype=torch.uint8, device="cuda"), torch.zeros(pool, device="cuda")
    rope = torch.zeros((pool, 64), dtype=torch.bfloat16, device="cuda")
    mv.kv_append_quant(lat, sc, rope, torch.arange(pool, dtype=torch.int32, device="cuda"),
                       torch.randn((pool, 576), generator=g0).to(torch.bfloat16).cuda())
    slopes = torch.from_numpy(lr.slopes(H) * np.float32(1e-3)).cuda()
    zeros = lambda *shape, t=torch.int32: torch.zeros(shape, dtype=t, device="cuda")
    x = dict(q=zeros(B, q_len, H, 576, t=torch.bfloat16), table=zeros(B, stride), seq=zeros(B), weights=zeros(B, stride, t=torch.float32),
             pos=zeros(B, stride), doc=zeros(B, stride), prefix=zeros(B), budget=zeros(B))

    def fill(seed):
        r, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        put = lambda k, a: x[k].copy_(torch.from_numpy(np.ascontiguousarray(a)))
        n = np.array([max(q_len, m - int(r.integers(0, m // 2))) for m in lens], np.int32)
        doc = np.zeros((B, stride), np.int32)
        for b in range(B):
            for i, share in enumerate(np.sort(r.random(2))):
                doc[b, int(share * n[b]):] = i + 1
        x["q"].copy_(torch.randn(x["q"].shape, generator=g).to(torch.bfloat16))
        for k, a in (("table", r.integers(0, pool, (B, stride))), ("seq", n), ("weights", r.random((B, stride)) * 0.01),
                     ("pos", lr.gaps(seed, B, stride)), ("doc", doc), ("prefix", r.integers(0, 90, B)),
                     ("budget", r.integers(20, 200, B))):
            put(k, a.astype(np.float32 if k == "weights" else np.int32))

    def step(out):
        rules = dict(softcap=30.0, slopes=slopes, key_pos=x["pos"], window=stride // 2, prefix_lens=x["prefix"], key_doc=x["doc"])
        o, lse = mv.verify_attn_fp8_rules(x["q"], lat, sc, rope, x["table"], x["seq"], None, SCALE, **rules)
        mv.key_weights_fp8(x["q"], lat, sc, rope, x["table"], x["seq"], None, SCALE, lse, weights=x["weights"], decay=0.9, **rules)
        e = mv.kv_evict(x["table"], x["seq"], x["weights"], x["budget"], sink=4, recent=16, key_pos=x["pos"], key_doc=x["doc"], **out)
        return [o, lse, *e]

    out = dict(freed=zeros(B, stride), n_freed=zeros(B))
    fill(0)
    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(out)
    for seed in (1, 2, 3):
        fill(seed)
        out["freed"].fill_(-7)
        want = [t.clone() for t in step(out)]
        fill(seed)
        out["freed"].fill_(-7)
        out["n_freed"].fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert mv.device_status() == 0
        bits = lambda t: t.view(torch.int32 if t.element_size() == 4 else torch.int16)
        for i, (a, b) in enumerate(zip(captured, want)):
            assert torch.equal(bits(a), bits(b)), (seed, i)
        assert torch.isfinite(captured[1]).all() and (captured[8] > 0).any()
