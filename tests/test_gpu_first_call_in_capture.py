"""A process whose first calls of the newer operators are captured into a graph (no warm-up outside it)."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
sys.path[:0] = ["tests", "."]
import torch
import paged_kv_cache_275_gb300 as pkv
from plain64 import Pages

pages = Pages((300, 40, 700), 2, 128, 1, width=4000)
kc, vc, table, cl = pages.cuda()
q = pages.randn(3, 8, 128).cuda()
k, v = pages.randn(3, 2, 128).cuda(), pages.randn(3, 2, 128).cuda()
i32 = dict(dtype=torch.int32, device="cuda")
start, prefix, chunks = torch.tensor([0, 1], **i32), torch.tensor([160], **i32), torch.tensor([0, 1, 2, 3], **i32)
slots, pos = torch.full((3,), -1, dtype=torch.int64, device="cuda"), torch.arange(3, device="cuda")
cos_sin = torch.ones(8, 128, device="cuda")
outs = [torch.zeros_like(q) for _ in range(5)]

def calls():
    pkv.rope_append(q, k, v, pos, slots, cos_sin, kc, vc, outs[0])
    pkv.paged_window_decode_attention(q, kc, vc, table, cl, 0.09, outs[1], 64, 4)
    pkv.paged_window_decode_attention(q, kc, vc, table, cl, 0.09, outs[2], 64, 4, num_partitions=30)
    pkv.paged_window_prefill_attention(q, kc, vc, table, cl, chunks, 1, 0.09, outs[3], 64, 4)
    pkv.paged_prefix_decode_attention(q, kc, vc, table, cl, start, prefix, 0.09, outs[4])

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
torch.cuda.synchronize()
captured = [o.clone() for o in outs]
for o in outs:
    o.zero_()
calls()
torch.cuda.synchronize()
assert pkv.get_and_clear_device_error() == 0
assert all(torch.equal(a, b) for a, b in zip(captured, outs)), "captured and eager results differ"
print("same")
"""


def test_first_calls_may_be_captured():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=Path(__file__).resolve().parents[1], capture_output=True,
                       text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout[-500:] + r.stderr[-1500:]
