"""The dense entries' first calls of a process: captured into a graph, and from
two host threads at once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import threading, torch
from block_sparse_attention_15_b200 import binding as B
gen = torch.Generator(device="cuda").manual_seed(3)
new = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
q, k, v, dout = new(8, 700, 64), new(2, 700, 64), new(2, 700, 64), new(8, 700, 64)
cu = [0, 130, 700]
qd, ks, vs = new(600, 8, 1, 64), new(600, 2, 50, 64), new(600, 2, 50, 64)
lens = torch.full((600,), 37, dtype=torch.int32, device="cuda")
def calls():
    out, lse = B.dense_attn_varlen(q, k, v, cu, cu, return_lse=True)
    return [out, lse, *B.dense_attn_varlen_backward(q, k, v, out, dout, lse, cu, cu),
            B.shared_prefix_attn(qd, k, v, ks, vs, lens)]
"""

CAPTURED = SETUP + """
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    first = calls()
graph.replay()
torch.cuda.synchronize()
B.check_device_status()
assert all(torch.equal(a, b) for a, b in zip(first, calls()))
print("same")
"""

THREADS = SETUP + """
torch.cuda.synchronize()
got, start = {}, threading.Barrier(4)
def work(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        got[i] = [calls() for _ in range(5)]
        torch.cuda.current_stream().synchronize()
threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
B.check_device_status()
want = calls()
assert len(got) == 4 and all(torch.equal(a, b) for r in got.values() for c in r for a, b in zip(c, want))
print("same")
"""


@pytest.mark.parametrize("script", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls(script):
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
