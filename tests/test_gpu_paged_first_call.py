"""The first paged call of a process, where the kernels are set up: inside a graph capture; and the
first call of a thread, several at once, each with a stream of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = """
import sys, threading
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

THREADS = COMMON + """
SECOND = {second}
if SECOND:      # every kernel is set up here; the threads' own first calls come after
    for d in jobs:
        call(d)
    torch.cuda.synchronize()
streams = [torch.cuda.Stream() for _ in range(6)]
more = [job([(1, 700), (1, 40)], 64, k) if k % 2 else job([(60, 300)], 64, k) for k in range(6)]
torch.cuda.synchronize()
failed = []
gate = threading.Barrier(6)

def work(k):
    try:
        gate.wait()
        for _ in range(20):
            call(more[k], streams[k])
    except Exception as e:
        failed.append(e)

threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
for d in more:
    check(d)
"""


# the library's other calls that encode tensor maps, in threads that made no CUDA call before
OTHERS = """
import sys, threading
sys.path.insert(0, {root!r})
import torch
from deepseek_v4_sparse_ratio_gb300 import _binding as B

T, off, k = 40, 400, 16
n = (off + T) // 4
g = torch.Generator().manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
q, raw, pooled, q_idx, ik = rnd(T, 64, 512), rnd(off + T, 512), rnd(n, 512), rnd(T, 64, 128), rnd(n, 128)
w = torch.randn(T, 64, generator=g).cuda()
scratch = torch.empty(B.dsa_score_scratch_bytes(T, n) // 4, device="cuda")

def both(stream, sel, out, scratch):
    B.dsa_index_score_topk(q_idx, w, ik, n, T, off, 4, k, T, scratch, sel, None, stream)
    B.dsa_window_sparse_attn(q, raw, 0, pooled, n, sel, k, T, off, 4, 128, 0.05, out, None, stream)

def buffers():
    return (torch.zeros(T, k, dtype=torch.int32, device="cuda"),
            torch.zeros(T, 64, 512, dtype=torch.bfloat16, device="cuda"),
            torch.empty_like(scratch))

first = buffers()
both(None, *first)
more = [(torch.cuda.Stream(), *buffers()) for _ in range(4)]
torch.cuda.synchronize()
failed = []

def work(k):
    try:
        both(*more[k])
    except Exception as e:
        failed.append(e)

threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
for m in more:
    assert torch.equal(m[1], first[0]) and torch.equal(m[2], first[1])
"""


@pytest.mark.parametrize("script,second", [(CAPTURE, False), (THREADS, False), (THREADS, True),
                                           (OTHERS, False)],
                         ids=["capture", "threads", "threads_after_set_up", "other_calls"])
def test_first_call(dsa, script, second):
    r = subprocess.run([sys.executable, "-c", script.format(root=ROOT, second=second)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
