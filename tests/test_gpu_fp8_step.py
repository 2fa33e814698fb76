"""One speculative-verify step over the fp8 cache, its operators in the order of use: norm and
rotation, quantising append, verify attention, acceptance."""
import numpy as np
import pytest
import torch

import step_ref as ref
import workloads as w

pytestmark = pytest.mark.gpu


def test_whole_step(cuda_lib):
    """Two steps in a row on one side stream without a synchronise in between; every operator's output
    against the float64 form of what it was given."""
    mv = cuda_lib
    B, q_len, H, V, n_pool = 3, 6, 8, 1000, 1200
    prefix = np.array([257, 40, 130], np.int32)
    g = torch.Generator().manual_seed(1)
    freq = (10000.0 ** (-torch.arange(0, 64, 2).double() / 64)).float()
    wq, wk = ((1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16) for _ in range(2))
    perm = torch.randperm(n_pool, generator=g).to(torch.int32)
    stride = int(prefix.max()) + q_len
    table = perm[:B * stride].view(B, stride).contiguous()
    lat = torch.full((n_pool, 512), 0x7F, dtype=torch.uint8, device="cuda")
    sc = torch.full((n_pool,), float("nan"), device="cuda")
    rope = torch.full((n_pool, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    par = torch.from_numpy(w.tree_parents(3, B, q_len)).to(torch.int32)
    mask = w.tree_mask_from_parents(par.numpy().astype(np.int64))
    depth = mask.sum(2) - 1
    seq = torch.from_numpy(prefix + q_len)
    head = torch.randn((H * 512, V), generator=g).cuda() * 0.02
    dev = {k: v.cuda() for k, v in dict(freq=freq, wq=wq, wk=wk, table=table, par=par, seq=seq.to(torch.int32),
                                        mask=torch.from_numpy(mask)).items()}
    # the prefixes' rows, quantised from a prompt pass
    rows = torch.randn((int(prefix.sum()), 576), generator=g).to(torch.bfloat16)
    slots = torch.cat([table[b, :prefix[b]] for b in range(B)])
    s = torch.cuda.Stream()
    kept = []
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mv.kv_append_quant(lat, sc, rope, slots.cuda(), rows.cuda())
        for step in range(2):
            gs = torch.Generator().manual_seed(50 + step)
            xq = torch.randn((B, q_len, H, 576), generator=gs).to(torch.bfloat16).cuda()
            xk = torch.randn((B, q_len, 576), generator=gs).to(torch.bfloat16).cuda()
            pos = torch.from_numpy(prefix[:, None] + depth).to(torch.int32).cuda()
            q, k = mv.qk_norm_rope(xq, xk, pos, dev["freq"], q_weight=dev["wq"], kv_weight=dev["wk"])
            new = torch.stack([dev["table"][b, prefix[b]:prefix[b] + q_len] for b in range(B)]).view(-1)
            mv.kv_append_quant(lat, sc, rope, new, k.view(-1, 576))
            out, lse = mv.verify_attn_fp8(q, lat, sc, rope, dev["table"], dev["seq"], dev["mask"], w.default_scale())
            p = torch.softmax(out.float().view(B, q_len, H * 512) @ head, -1)
            d = torch.softmax(torch.log(p) + 0.5 * torch.randn(p.shape, generator=gs).cuda(), -1)
            tok = torch.randint(0, V, (B, q_len), generator=gs, dtype=torch.int32).cuda()
            tok[:, 1:4] = p[:, 0].topk(3).indices.to(torch.int32)      # likely tokens, some accepted
            u, un = torch.rand((B, q_len), generator=gs).cuda(), torch.rand((B,), generator=gs).cuda()
            n, toks, path = mv.draft_verify(p, d, tok, dev["par"], u, un)
            back = mv.kv_read_fp8(lat, sc, rope, new)
            kept.append([x.clone() for x in (xq, xk, pos, q, k, lat, sc, rope, out, lse, p, d, tok, u, un, n, toks, path, back)])
    s.synchronize()
    assert mv.device_status() == 0
    for xq, xk, pos, q, k, l, c, r, out, lse, p, d, tok, u, un, n, toks, path, back in kept:
        args = (pos.cpu().numpy().reshape(-1).astype(np.float64), ref.f64(freq), float(np.float32(1e-6)), True)
        for got, x, wt in ((q, xq.view(B * q_len, H, 576), wq), (k, xk.view(B * q_len, 1, 576), wk)):
            want, tol = ref.norm_rope(ref.f64(x), ref.f64(wt), *args)
            assert np.all(np.abs(ref.f64(got).reshape(want.shape) - want) <= tol)
        code, scale = ref.quantise(k.view(-1, 576).float().cpu().numpy())
        at = np.concatenate([table[b, prefix[b]:prefix[b] + q_len].numpy() for b in range(B)])
        lat_np, sc_np = l.cpu().numpy(), c.cpu().numpy()
        assert np.array_equal(lat_np[at], code) and np.array_equal(sc_np[at], scale)
        rope_f = ref.f64(r)
        keys = lambda b: (lambda t: ref.dequantise_rows(lat_np[t], sc_np[t], rope_f[t]))(table[b, :prefix[b] + q_len].numpy())
        o, ll, t_out, t_lse = ref.attention(ref.f64(q), keys, prefix + q_len, mask, w.default_scale())
        assert np.all(np.abs(ref.f64(out) - o) <= t_out) and np.all(np.abs(ref.f64(lse) - ll) <= t_lse)
        deq = ref.dequantise_rows(code, scale, ref.f64(k.view(-1, 576))[:, 512:])
        assert np.all(np.abs(ref.f64(back) - deq) <= np.abs(deq) * (2.0 ** -8 + 2.0 ** -23))
        cp = lambda t: t.cpu().numpy()
        for b in range(B):
            en, et, ep = ref.accept(cp(p)[b], cp(d)[b], cp(tok)[b], par[b].numpy(), cp(u)[b], cp(un)[b])
            assert (int(n[b]), toks[b].tolist(), path[b].tolist()) == (en, et, ep)
