"""A long-context serving loop: attention under rules, the keys' weights, eviction, the freed slots used again
for the next step's rows; every operator's output against its float64 form of what it was given."""
import numpy as np
import pytest
import torch

import long_ref as lr
import step_ref as ref
import workloads as w

pytestmark = pytest.mark.gpu
SCALE = w.default_scale()


def test_serving_loop(cuda_lib):
    """Four steps on one side stream without a synchronise: each appends a block of drafts, attends, keeps what
    was accepted, adds the weights up and evicts down to the budget."""
    mv = cuda_lib
    B, q_len, H, stride, budget = 3, 4, 8, 128, 60
    n0 = np.array([100, 75, 58], np.int32)
    g = torch.Generator().manual_seed(3)
    pool = B * stride
    table = torch.randperm(pool, generator=g).to(torch.int32).view(B, stride).cuda()
    rows = torch.randn((int(n0.sum()), 576), generator=g).to(torch.bfloat16)
    lat = torch.zeros((pool, 512), dtype=torch.uint8, device="cuda")
    sc, rope = torch.zeros(pool, device="cuda"), torch.zeros((pool, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(stride, dtype=torch.int32).expand(B, stride).contiguous().cuda()
    seq = torch.from_numpy(n0.copy()).cuda()
    weights = torch.zeros((B, stride), device="cuda")
    slope, prefix = torch.from_numpy(lr.slopes(H)).cuda(), torch.full((B,), 6, dtype=torch.int32, device="cuda")
    counted = torch.tensor([[1, 1, 0, 0], [1, 0, 0, 0], [1, 1, 1, 1]], dtype=torch.uint8).cuda()
    accepted = counted.sum(1).to(torch.int32)
    first = torch.cat([table[b, :n] for b, n in enumerate(n0.tolist())])
    rules = dict(softcap=25.0, slopes=slope, window=80, prefix_lens=prefix)
    s, kept = torch.cuda.Stream(), []
    s.wait_stream(torch.cuda.current_stream())
    b_at = torch.arange(B, device="cuda")[:, None]
    next_pos = seq.clone()
    with torch.cuda.stream(s):
        mv.kv_append_quant(lat, sc, rope, first, rows.cuda())
        for step in range(4):
            gs = torch.Generator().manual_seed(60 + step)
            # the drafts' rows go to the slots behind each stream's last key (freed ones after the first step)
            at = seq.long()[:, None] + torch.arange(q_len, device="cuda")
            new_pos = next_pos[:, None] + torch.arange(q_len, device="cuda", dtype=torch.int32)
            pos[b_at, at] = new_pos
            seq += q_len
            mv.kv_append_quant(lat, sc, rope, table[b_at, at].view(-1).contiguous(),
                               torch.randn((B * q_len, 576), generator=gs).to(torch.bfloat16).cuda())
            q = torch.randn((B, q_len, H, 576), generator=gs).to(torch.bfloat16).cuda()
            out, lse = mv.verify_attn_fp8_rules(q, lat, sc, rope, table, seq, None, SCALE, key_pos=pos, **rules)
            before = [x.clone() for x in (q, lat, sc, rope, table, seq, pos, weights)]
            mv.key_weights_fp8(q, lat, sc, rope, table, seq, None, SCALE, lse, key_pos=pos, weights=weights, decay=0.95,
                               counted=counted, **rules)
            seq -= q_len - accepted                       # the accepted drafts stay
            next_pos += accepted
            grown = [x.clone() for x in (table, seq, weights, pos)]
            ev = mv.kv_evict(table, seq, weights, budget, sink=4, recent=8, key_pos=pos)
            # the allocator puts the freed slots behind the kept ones
            j = torch.arange(stride, device="cuda")
            gone = (j >= seq[:, None]) & (j < (seq + ev.n_freed)[:, None])
            table[gone] = ev.freed[j < ev.n_freed[:, None]]
            kept.append((before, [out, lse, grown[2]], grown, [x.clone() for x in (table, seq, weights, pos)]))
    s.synchronize()
    assert mv.device_status() == 0
    cpu = lambda t: t.cpu().numpy()
    for before, (out, lse, weighed), (g_table, g_seq, g_weights, g_pos), after in kept:
        q, lat_, sc_, rope_, table_, seq_, pos_, weights_ = before
        n = cpu(seq_)
        keys = lambda b: (lambda at: ref.dequantise_rows(cpu(lat_)[at], cpu(sc_)[at], ref.f64(rope_)[at]))(cpu(table_)[b])
        r = lr.Rules(25.0, lr.slopes(H), cpu(pos_), 80, np.full(B, 6), None)
        o, l, t_out, t_lse = lr.attention(ref.f64(q), keys, n, None, SCALE, r)
        assert np.all(np.abs(ref.f64(out) - o) <= t_out) and np.all(np.abs(ref.f64(lse) - l) <= t_lse)
        want, tol = lr.key_weights(ref.f64(q), keys, n, None, SCALE, r, ref.f64(lse), cpu(counted), ref.f64(weights_),
                                   float(np.float32(0.95)), ref.f64(weights_))
        assert np.all(np.abs(ref.f64(weighed) - want) <= tol)
        outs = dict(table_out=cpu(g_table), lens_out=cpu(g_seq), weights_out=cpu(g_weights), pos_out=cpu(g_pos), doc_out=None,
                    freed=np.zeros((B, stride), np.int32), n_freed=np.zeros(B, np.int32))
        e = lr.evict(cpu(g_table), cpu(g_seq), cpu(g_weights), budget, 4, 8, cpu(g_pos), None, outs)
        for b in range(B):
            left, gone = int(e["lens_out"][b]), int(e["n_freed"][b])
            assert left <= budget and np.array_equal(cpu(after[1]), e["lens_out"])
            assert np.array_equal(cpu(after[0])[b, :left], e["table_out"][b, :left])
            assert np.array_equal(cpu(after[0])[b, left:left + gone], e["freed"][b, :gone])
            assert np.array_equal(cpu(after[2])[b, :left], e["weights_out"][b, :left])
            assert np.array_equal(cpu(after[3])[b, :left], e["pos_out"][b, :left])
            assert sorted(cpu(after[0])[b]) == sorted(cpu(g_table)[b])       # no slot is lost


def test_bf16_cache(cuda_lib):
    """The bf16 cache's attention, its weights, and an eviction whose kept keys the attention then reads."""
    mv = cuda_lib
    s = lr.Step(5, [300, 90], 5, 8, mask="tree", cache="bf16")
    q, kv, table, seq, mask = s.on("cuda")
    _, lse = mv.verify_attn(q, kv, table, seq, mask, SCALE)
    weights = mv.key_weights(q, kv, table, seq, mask, SCALE, lse)
    assert torch.allclose(weights.double().sum(1), torch.full((2,), 40.0, dtype=torch.float64, device="cuda"), rtol=1e-2)
    ev = mv.kv_evict(table, seq, weights, 80, recent=5)
    assert ev.slot_table is table and ev.seq_lens.tolist() == [80, 80] and ev.n_freed.tolist() == [220, 10]
    s.seq[:] = 80
    s.table = table.cpu()
    out, lse = mv.verify_attn(q, kv, table, seq, mask, SCALE)
    o, l, t_out, t_lse = ref.attention(ref.f64(s.q), s.keys_of, s.seq, s.mask, SCALE)
    # (the bf16 attention also rounds its probabilities to bf16: the bounds cover it)
    assert np.all(np.abs(ref.f64(out) - o) <= t_out + 1e-6) and np.all(np.abs(ref.f64(lse) - l) <= t_lse + 1e-6)
