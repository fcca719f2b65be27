"""The first paged call of a process, where the kernels are set up: inside a graph capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import paged_ref as R
from deepseek_v4_sparse_ratio_gb300 import _binding as B

def job(lens, heads, seed):
    batch = R.make(lens, 32, seed=seed)
    q = torch.randn(sum(n for n, _ in lens), heads, 512,
                    generator=torch.Generator().manual_seed(seed)).bfloat16()
    gb = {{k: v.cuda() for k, v in batch.items()}}
    d = dict(batch=batch, q=q, gb=gb, qd=q.cuda(), out=torch.zeros_like(q, device="cuda"),
             work=torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return d

def call(d, stream=None):
    g = d["gb"]
    B.dsa_paged_attn(d["qd"], g["new_start"], g["seq_len"], g["page_table"], g["pages"], 0, 0.05,
                     d["work"], d["out"], g["cos_sin"], d["status"], stream)

def check(d):
    assert d["status"].item() == 0
    ref, tol, _ = R.attention(d["batch"], d["q"], 0, 0.05)
    assert bool(((d["out"].cpu().double() - ref).abs() <= tol).all())

jobs = [job([(1, 700), (1, 40)], 64, 1), job([(60, 300)], 64, 2)]
torch.cuda.synchronize()
"""

CAPTURE = COMMON + """
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for d in jobs:
        call(d)
graph.replay()
torch.cuda.synchronize()
for d in jobs:
    check(d)
"""

@pytest.mark.parametrize("script", [CAPTURE], ids=["capture"])
def test_first_call(dsa, script):
    r = subprocess.run([sys.executable, "-c", script.format(root=ROOT)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
