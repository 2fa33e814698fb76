"""The long-context operators' first calls, from several host threads on streams of their own at once, in a
process of their own: all get the same bits."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import threading
import torch
import mla_speculative_verify_attention_gb300 as mv

torch.manual_seed(0)
dev, N = "cuda", 10
B, q_len, H, n = 2, 3, 64, 9000
q = torch.randn(B, q_len, H, 576, device=dev).to(torch.bfloat16)
rows = torch.randn(B * n, 576, device=dev).to(torch.bfloat16)
slots = torch.arange(B * n, dtype=torch.int32, device=dev)
table, seq = slots.view(B, n), torch.full((B,), n, dtype=torch.int32, device=dev)
cache = (torch.empty(B * n, 512, dtype=torch.uint8, device=dev), torch.empty(B * n, device=dev),
         torch.empty(B * n, 64, dtype=torch.bfloat16, device=dev))
doc = (torch.arange(n, dtype=torch.int32, device=dev) // 4000).expand(B, n).contiguous()
wide = torch.rand(2, 600000, device=dev)
wide_table = torch.arange(1200000, dtype=torch.int32, device=dev).view(2, 600000)
wide_seq = torch.tensor([600000, 500001], dtype=torch.int32, device=dev)
gate, got, wrong = threading.Barrier(N), [None] * N, []

def work(k):
    try:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        rules = dict(softcap=20.0, key_doc=doc)
        gate.wait()
        with torch.cuda.stream(s):
            if k % 2:                                  # half of them meet in the eviction, half in the attention
                e = mv.kv_evict(wide_table.clone(), wide_seq.clone(), wide.clone(), 100000, sink=4, recent=64)
            o, lse = mv.verify_attn_fp8_rules(q, *cache, table, seq, None, 0.07, **rules, nsplit=4)
            w = mv.key_weights_fp8(q, *cache, table, seq, None, 0.07, lse, **rules)
            v = mv.key_weights(q, rows, table, seq, None, 0.07, lse, **rules)
            f = mv.kv_evict(table.clone(), seq.clone(), w.clone(), 2000, recent=64)
            if not k % 2:
                e = mv.kv_evict(wide_table.clone(), wide_seq.clone(), wide.clone(), 100000, sink=4, recent=64)
        s.synchronize()
        got[k] = [x.cpu() for x in (o, lse, w, v, f.seq_lens, f.slot_table, f.weights, e.seq_lens, e.slot_table, e.weights)]
    except BaseException as e:
        wrong.append(repr(e))

mv.kv_append_quant(*cache, slots, rows)
torch.cuda.synchronize()
threads = [threading.Thread(target=work, args=(k,)) for k in range(N)]
for t in threads: t.start()
for t in threads: t.join()
assert not wrong, wrong
for g in got:
    assert all(torch.equal(x, y) for x, y in zip(g, got[0]))
assert mv.device_status() == 0
print("same")
"""


def test_threads_meet_in_the_first_calls():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(2):
        r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
