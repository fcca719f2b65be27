"""The longest sequences of the 4-bit paged cache, and the first calls of a process and of threads."""
import os
import subprocess
import sys

import pytest
import torch

import q4_ref as Q
from deepseek_v4_sparse_ratio_gb300 import _binding as B

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LENGTH = B.MAX_PAGED_TOKENS


def signs(seed):
    return torch.where(torch.randn(512, generator=torch.Generator().manual_seed(seed)) > 0, 1.0, -1.0)


def row_of_signs(d, size):
    """The bytes of a row that stands for size * d, d of ones and minus ones, size a power of two:
    n = +-1, scales of 1 and the exponent's byte 137 + log2 size."""
    row = Q.pack((d * 7).bfloat16()[None])[0].clone()     # n = +-7: codes 15 and 1
    codes = row[32:256]
    codes = torch.where(codes >> 4 == 15, 0x90, 0x70) | torch.where(codes & 15 == 15, 9, 7)
    row[32:256] = codes.to(torch.uint8)
    row[:14] = row[16:30] = 0x38
    row[14] = row[30] = 137 + int(torch.log2(torch.tensor(float(size))).item())
    row[256:] = (d[448:] * size).bfloat16().view(torch.uint8)
    assert torch.equal(Q.decode(row), d.double() * size)
    return row


def no_turns():
    cos_sin = torch.zeros(LENGTH, 32, 2, device="cuda")
    cos_sin[..., 0] = 1.0
    return cos_sin


def attend(q, starts, lens, table, pages, window, sinks, cos_sin):
    out = torch.zeros_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    work = torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    B.dsa_paged_q4_attn(q, starts, lens, table, pages, window, sinks, 512 ** -0.5, work, out,
                        cos_sin, False, status)
    torch.cuda.synchronize()
    assert status.item() == B.DSA_OK
    return out.float()


@pytest.mark.parametrize("seqs,tokens", [(1, 608), (304, 1)])
def test_whole_units_of_the_longest_sequence(dsa, seqs, tokens):
    """Equal rows, 2^24 of them, 64 heads: every weight is 1, every sum a whole number up to 2^24,
    and the output the row, rounded once (2^-8). Waits for the next queries last for whole units."""
    d = signs(5)
    pages = row_of_signs(d, 1.0).expand(4, 1024, Q.ROW).contiguous().cuda()
    rows = seqs * tokens
    table = (torch.arange(LENGTH // 1024) % 4).int().expand(seqs, -1).contiguous().cuda()
    q = torch.randn(rows, 64, 512, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    starts = torch.arange(0, rows + 1, tokens, dtype=torch.int32, device="cuda")
    lens = torch.full((seqs,), LENGTH, dtype=torch.int32, device="cuda")
    out = attend(q, starts, lens, table, pages, 0, 0, no_turns())
    assert bool((out * d.cuda() - 1.0).abs().max() <= 2.0 ** -8)


@pytest.mark.parametrize("tokens,window,sinks", [(1, 128, 4), (1, 4096, 128), (70, 1000, 37),
                                                 (300, 128, 1)])
def test_first_tokens_and_a_window_far_apart(dsa, tokens, window, sinks):
    """Queries of zero: every weight is 1. The first page's rows are d, the last pages' 2 d, those
    between hold NaN; a token sees `sinks` and `window` of them, and its output is their mean: sums
    of whole numbers, one division (2^-23), one rounding to bf16 (2^-8)."""
    d, size = signs(7), 1024
    first, last = row_of_signs(d, 1.0), row_of_signs(d, 2.0)
    pages = torch.full((7, size, Q.ROW), 0xFF, dtype=torch.uint8)
    pages[0, :sinks] = first
    pages[2:].view(5 * size, Q.ROW)[5 * size - window - tokens + 1:] = last
    table = torch.ones(1, LENGTH // size, dtype=torch.int32)
    table[0, 0] = 0
    table[0, -5:] = torch.arange(2, 7)
    q = torch.zeros(tokens, 64, 512, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    lens = torch.tensor([LENGTH], dtype=torch.int32, device="cuda")
    out = attend(q, starts, lens, table.cuda(), pages.cuda(), window, sinks, no_turns())
    mean = (sinks + 2 * window) / (sinks + window)
    err = (out * d.cuda() - mean).abs().max().item()
    assert err <= mean * (2.0 ** -8 + 2.0 ** -22), err


def test_rows_of_the_last_positions(dsa):
    """The norm, the append and the read at positions up to 2^24 - 1."""
    n, size = 40, 64
    g = torch.Generator().manual_seed(8)
    kv = torch.randn(n, 512, generator=g).bfloat16()
    q = torch.randn(n, 2, 512, generator=g).bfloat16()
    cos_sin = torch.zeros(LENGTH, 32, 2)
    cos_sin[-n:] = Q.angles(n)
    table = torch.full((1, LENGTH // size), -1, dtype=torch.int32)
    table[0, -1] = 1
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([LENGTH], dtype=torch.int32, device="cuda")
    pages = torch.zeros(2, size, Q.ROW, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gcs, gt = cos_sin.cuda(), table.cuda()
    out, qo, ko = torch.zeros(n, 512).bfloat16().cuda(), torch.zeros_like(q).cuda(), \
        torch.zeros_like(kv).cuda()
    B.dsa_paged_q4_append(kv.cuda(), starts, lens, gt, pages, gcs, status)
    B.dsa_paged_q4_read(starts, lens, gt, pages, out, None, status)
    B.dsa_qk_norm_rope(q.cuda(), kv.cuda(), starts, lens, qo, ko, gcs, None, None, 1e-6, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    turned = torch.stack([Q.turn(kv[i].double(), cos_sin[i - n]) for i in range(n)])
    want = Q.pack(turned.bfloat16())
    assert torch.equal(pages[1, size - n:, :256].cpu(), want[:, :256])
    # rotated elements: fp32 products and a sum (3 * 2^-24 of their sizes), then one bf16 rounding
    bound = (Q.U + 2.0 ** -20) * kv.double().abs().max() * 1.5
    got = out.cpu().double()
    assert bool((got[:, 448:] - turned[:, 448:]).abs().max() <= bound)
    assert torch.equal(got[:, :448], Q.unpack(want)[:, :448])
    r = (kv.double().pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    err = (ko.cpu().double() - turned * r).abs()
    assert bool((err <= (Q.U + 2.0 ** -14) * 1.5 * (kv.double() * r).abs().max()).all())
    assert not bool(pages[0].any()) and not bool(pages[1, :size - n].any())


COMMON = """
import sys, threading
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import q4_ref as Q
from deepseek_v4_sparse_ratio_gb300 import _binding as B

def job(lens, heads, seed):
    batch = Q.make(lens, 32, seed=seed)
    n = sum(k for k, _ in lens)
    q = torch.randn(n, heads, 512, generator=torch.Generator().manual_seed(seed)).bfloat16()
    kv = torch.randn(n, 512, generator=torch.Generator().manual_seed(seed + 100)).bfloat16()
    gb = {{k: v.cuda() for k, v in batch.items()}}
    return dict(batch=batch, q=q, kv=kv, gb=gb, qd=q.cuda(), kvd=kv.cuda(),
                qn=torch.zeros_like(q, device="cuda"), kn=torch.zeros_like(kv, device="cuda"),
                spare=torch.zeros_like(gb["pages"]), back=torch.zeros_like(kv, device="cuda"),
                out=torch.zeros_like(q, device="cuda"),
                work=torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))

def call(d, stream=None):
    g = d["gb"]
    at = g["new_start"], g["seq_len"]
    B.dsa_paged_q4_attn(d["qd"], *at, g["page_table"], g["pages"], 0, 0, 0.05, d["work"], d["out"],
                        g["cos_sin"], False, d["status"], stream)
    B.dsa_qk_norm_rope(d["qd"], d["kvd"], *at, d["qn"], d["kn"], None, None, None, 1e-6, d["status"],
                       stream)
    B.dsa_paged_q4_append(d["kvd"], *at, g["page_table"], d["spare"], None, d["status"], stream)
    B.dsa_paged_q4_read(*at, g["page_table"], d["spare"], d["back"], None, d["status"], stream)

def check(d):
    assert d["status"].item() == 0
    ref, tol, _ = Q.attention(d["batch"], d["q"], 0, 0, 0.05, False)
    assert bool(((d["out"].cpu().double() - ref).abs() <= tol).all())
    assert torch.equal(d["back"].cpu().double(), Q.unpack(Q.pack(d["kv"])))
    x = d["q"].double()
    y = x * (x.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    assert bool(((d["qn"].cpu().double() - y).abs() <= (Q.U + 2.0 ** -14) * y.abs()).all())

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
streams = [torch.cuda.Stream() for _ in range(4)]
more = [job([(1, 700), (1, 40)], 64, k) if k % 2 else job([(60, 300)], 64, k) for k in range(4)]
torch.cuda.synchronize()
failed = []
gate = threading.Barrier(4)

def work(k):
    try:
        gate.wait()
        for _ in range(20):
            call(more[k], streams[k])
    except Exception as e:
        failed.append(e)

threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
for d in more:
    check(d)
"""


@pytest.mark.parametrize("script", [CAPTURE, THREADS], ids=["capture", "threads"])
def test_first_call(dsa, script):
    r = subprocess.run([sys.executable, "-c", script.format(root=ROOT)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
