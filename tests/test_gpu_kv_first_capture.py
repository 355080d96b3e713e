"""The first call that a process makes may be one that is captured into a graph:
what the library looks up once does not fail the capture, nor any call after it."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys, torch
import gemm_epilogue_02_gb300 as tg
order = sys.argv[1].split(",")
k, v, tk, tv = (torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4))
c, to = tg.PagedCache(k, v), tg.PagedCache(tk, tv)
table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
x = torch.arange(1, 65, device="cuda").bfloat16().expand(1, 2, 64).contiguous()
n = torch.ones(1, dtype=torch.int32, device="cuda")
o = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
q = torch.ones_like(o)
w = torch.zeros(1, 2, 128, device="cuda")
ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
kept = torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda")
tl, tw = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, 4, device="cuda")
calls = dict(append=lambda: tg.kv_append(c, x, x, table, n, weights=w),
             attend=lambda: tg.attention_decode(q, c, table, n, o, weights=w, workspace=ws),
             evict=lambda: tg.kv_evict(c, table, n, w, to, table, kept, tl, tw))
torch.cuda.synchronize()
graphs = {}
for name in order:
    graphs[name] = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graphs[name]):
        calls[name]()
for name in ("append", "attend", "evict"):
    graphs[name].replay()
torch.cuda.synchronize()
assert torch.equal(o[0, 3], x[0, 0]) and torch.equal(tv[0, 0, 1], x[0, 1]) and tl.tolist() == [1]
assert w[0, :, 0].tolist() == [2.0, 2.0] and kept[0, 0].tolist() == [0, -1, -1, -1]
assert tg.tgemm_last_device_status() == 0
print("captured first")
"""


@pytest.mark.parametrize("order", ["append,attend,evict", "attend,evict,append", "evict,append,attend"])
def test_first_calls_are_captured(cuda_lib, order):
    done = subprocess.run([sys.executable, "-c", CHILD, order], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured first" in done.stdout, done.stdout[-1000:] + done.stderr[-3000:]
