"""The first calls on a device, from several host threads at once, in a process of their own: what the
library sets up once is complete before any of them uses it."""
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
dev, N = "cuda", 12
B, q_len, H, n, V = 3, 4, 8, 300, 5000
q = torch.randn(B, q_len, H, 576, device=dev).to(torch.bfloat16)
rows = torch.randn(B * n, 576, device=dev).to(torch.bfloat16)
slots = torch.arange(B * n, dtype=torch.int32, device=dev)
table, seq = slots.view(B, n), torch.full((B,), n, dtype=torch.int32, device=dev)
p = torch.softmax(torch.randn(B, q_len, V, device=dev), -1)
d = torch.softmax(torch.randn(B, q_len, V, device=dev), -1)
tok = torch.randint(0, V, (B, q_len), dtype=torch.int32, device=dev)
u, un = torch.rand(B, q_len, device=dev), torch.rand(B, device=dev)
torch.cuda.synchronize()
gate, got, wrong = threading.Barrier(N), [None] * N, []

def work(k):
    try:
        s = torch.cuda.Stream()
        gate.wait()
        with torch.cuda.stream(s):
            if k % 2:                                  # half of them meet in the acceptance, half in the append
                a = mv.draft_verify(p, d, tok, None, u, un)
            cache = (torch.empty(B * n, 512, dtype=torch.uint8, device=dev), torch.empty(B * n, device=dev),
                     torch.empty(B * n, 64, dtype=torch.bfloat16, device=dev))
            mv.kv_append_quant(*cache, slots, rows)
            o = mv.verify_attn_fp8(q, *cache, table, seq, None, 0.07)
            f = mv.verify_attn(q, rows, table, seq, None, 0.07)
            if not k % 2:
                a = mv.draft_verify(p, d, tok, None, u, un)
        s.synchronize()
        got[k] = [x.cpu() for x in (*a, *o, *f)]
    except BaseException as e:
        wrong.append(repr(e))

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
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
