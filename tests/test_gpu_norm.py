"""The norm of query heads and KV rows with their rotation, against its float64 form (q4_ref.py,
which derives the tolerances)."""
import pytest
import torch

import paged_ref as R
import q4_ref as Q
from deepseek_v4_sparse_ratio_gb300 import _binding as B

pytestmark = pytest.mark.gpu
EPS = 1e-6


def inputs(batch, heads, seed, pad=0, rows=None):
    g = torch.Generator().manual_seed(seed)
    n = (int(batch["new_start"][-1]) if rows is None else rows) + pad
    size = torch.exp(torch.randn(n, 1, 1, generator=g))
    q = (torch.randn(n, heads, 512, generator=g) * size).bfloat16()
    kv = (torch.randn(n, 512, generator=g) * size[:, 0]).bfloat16()
    return q, kv


def call(batch, q, kv, wq=None, wk=None, eps=EPS, status=None, in_place=False, stream=None):
    gb = {k: None if v is None else v.cuda() for k, v in batch.items()}
    q, kv = q.cuda(), kv.cuda()
    qo, ko = (q, kv) if in_place else (torch.full_like(q, 7.0), torch.full_like(kv, 7.0))
    B.dsa_qk_norm_rope(q, kv, gb["new_start"], gb["seq_len"], qo, ko, gb["cos_sin"],
                       None if wq is None else wq.cuda(), None if wk is None else wk.cuda(), eps,
                       status)
    torch.cuda.synchronize()
    return qo.cpu(), ko.cpu()


def check(batch, q, kv, got, wq=None, wk=None, eps=EPS, untouched=None):
    """Rows of a sequence are the norm, all others as they were. (A row that decreasing starts give
    to two sequences may have the position of either.)"""
    n = q.shape[0]
    limit = B.MAX_PAGED_TOKENS if batch["cos_sin"] is None else batch["cos_sin"].shape[0]
    positions = [[] for _ in range(n)]
    for s in range(len(batch["seq_len"])):
        r0, r1 = int(batch["new_start"][s]), int(batch["new_start"][s + 1])
        ln = int(batch["seq_len"][s])
        if 0 <= r0 <= r1 <= n and r1 - r0 <= ln <= limit:
            for r in range(r0, r1):
                positions[r].append(ln - r1 + r)
    for r in range(n):
        for x, w, y in ((q[r], wq, got[0][r]), (kv[r], wk, got[1][r])):
            if not positions[r]:
                assert torch.equal(y, x if untouched is None else torch.full_like(y, untouched))
                continue
            ok = False
            for p in positions[r]:
                cs = None if batch["cos_sin"] is None else batch["cos_sin"][p]
                ref, tol = Q.norm(x, w, eps, cs)
                ok |= bool(((y.double() - ref).abs() <= tol).all())
            assert ok, r


CASES = [  # (sequences (new, total), heads, rope, weights, padded rows)
    ([(1, 1)], 64, True, (False, True), 0),
    ([(1, 1)], 1, False, (False, False), 0),
    ([(3, 40), (0, 9), (1, 700), (17, 17)], 5, True, (True, True), 2),
    ([(33, 100)], 4, True, (True, False), 0),
    ([(2, 60), (5, 5)], 128, True, (False, True), 1),
    ([(1, 10 + i) for i in range(1100)], 3, True, (False, True), 3),
    ([(130, 300)], 16, False, (True, True), 0),
]


@pytest.mark.parametrize("lens,heads,rope,weights,pad", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_matches_the_formula(dsa, lens, heads, rope, weights, pad, in_place):
    batch = R.make(lens, 16, rope=rope, seed=heads)
    q, kv = inputs(batch, heads, 3, pad)
    g = torch.Generator().manual_seed(4)
    wq, wk = (1 + 0.3 * torch.randn(512, generator=g) if w else None for w in weights)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(batch, q, kv, wq, wk, status=status, in_place=in_place)
    assert status.item() == 0
    check(batch, q, kv, got, wq, wk, untouched=None if in_place else 7.0)


@pytest.mark.parametrize("size,eps", [(2.0 ** -60, 1e-6), (0.0, 1e-6), (2.0 ** 55, 1e-6),
                                      (1e-3, 1e-5), (1.0, 1e30), (2.0 ** -60, 1e-36)])
def test_small_and_large_rows(dsa, size, eps):
    batch = R.make([(3, 30)], 16, seed=1)
    q, kv = (torch.randn(*s, generator=torch.Generator().manual_seed(2)).mul(size).bfloat16()
             for s in ((3, 6, 512), (3, 512)))
    got = call(batch, q, kv, eps=eps)
    check(batch, q, kv, got, eps=eps, untouched=7.0)


def test_odd_values_stay_in_their_rows(dsa):
    """A NaN makes its row NaN; a sum of squares beyond fp32 makes its row zeros (0 * inf: NaN where
    the element itself is infinite)."""
    batch = R.make([(4, 30)], 16, rope=False, seed=1)
    q, kv = inputs(batch, 8, 5)
    clean = q.clone()
    q[1, 3, 7] = float("nan")
    q[2, 0, 450] = 2.0 ** 100
    q[3, 7, 9] = float("inf")
    got, _ = call(batch, q, kv)
    assert bool(got[1, 3].isnan().all()) and not got[2, 0].any() and bool(got[3, 7, 9].isnan())
    assert not got[3, 7, :9].any()
    for r, h in ((1, 3), (2, 0), (3, 7)):
        got[r, h], q[r, h] = 0, 0
        clean[r, h] = 0
    ref, tol = Q.norm(clean, None, EPS, None)
    assert bool(((got.double() - ref).abs() <= tol).all())


def test_sequences_that_cannot_be_are_left_and_reported(dsa):
    batch = R.make([(3, 20), (4, 40), (2, 30), (1, 60)], 16, seed=2)
    batch["seq_len"][1] = 3                                  # fewer than its four new tokens
    batch["cos_sin"] = batch["cos_sin"][:50].contiguous()    # too few for the last
    q, kv = inputs(batch, 8, 6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(batch, q, kv, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check(batch, q, kv, got, untouched=7.0)


@pytest.mark.parametrize("starts", [[0, 5, 2, 9], [-3, 2, 4, 9], [0, 4, 8, 20], [2, 5, 5, 7]])
def test_odd_starts(dsa, starts):
    batch = R.make([(3, 20), (3, 40), (3, 30)], 16, seed=4)
    batch["new_start"] = torch.tensor(starts, dtype=torch.int32)
    q, kv = inputs(batch, 8, 6, rows=9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(batch, q, kv, status=status)
    bad = any(not (0 <= a <= b <= 9 and b - a <= c) for a, b, c in
              zip(starts, starts[1:], batch["seq_len"].tolist()))
    assert status.item() == (B.DSA_ERR_BOUNDS if bad else 0)
    check(batch, q, kv, got, untouched=7.0)


def test_a_long_sequence_without_angles(dsa):
    """Without angles a sequence may be as long as any (positions are not looked up)."""
    batch = R.make([(2, 20)], 16, rope=False, seed=4)
    batch["seq_len"][0] = B.MAX_PAGED_TOKENS
    q, kv = inputs(batch, 2, 6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(batch, q, kv, call(batch, q, kv, status=status), untouched=7.0)
    assert status.item() == 0
    batch["seq_len"][0] = B.MAX_PAGED_TOKENS + 1
    got = call(batch, q, kv, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS and bool((got[0] == 7.0).all())


def test_positions_of_the_last_angles(dsa):
    """Angles of positions whose offsets pass 32 bits of bytes (2^24 of 256 bytes)."""
    n = 1 << 24
    cs = torch.zeros(n, 32, 2, device="cuda")
    tail = R.angles(8)
    cs[-8:] = tail.cuda()
    q, kv = inputs(dict(new_start=torch.tensor([0, 8])), 4, 7)
    out, rows = torch.empty_like(q, device="cuda"), torch.empty_like(kv, device="cuda")
    B.dsa_qk_norm_rope(q.cuda(), kv.cuda(), torch.tensor([0, 8], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), out, rows, cs)
    torch.cuda.synchronize()
    for r in range(8):
        ref, tol = Q.norm(q[r], None, EPS, tail[r])
        assert bool(((out[r].cpu().double() - ref).abs() <= tol).all())


def test_writes_stay_inside_the_buffers_and_odd_places(dsa):
    batch = R.make([(3, 20), (30, 40)], 16, seed=8)
    q, kv = inputs(batch, 7, 9)
    gb = {k: v.cuda() for k, v in batch.items()}
    guard = 4096 + 8                                          # 16 bytes off 32
    bufs = [torch.full((x.numel() + 2 * guard,), 5.0, dtype=torch.bfloat16, device="cuda")
            for x in (q, kv, q, kv)]
    qi, ki, qo, ko = (b[guard:-guard].view(x.shape) for b, x in zip(bufs, (q, kv, q, kv)))
    qi.copy_(q)
    ki.copy_(kv)
    B.dsa_qk_norm_rope(qi, ki, gb["new_start"], gb["seq_len"], qo, ko, gb["cos_sin"])
    torch.cuda.synchronize()
    check(batch, q, kv, (qo.cpu(), ko.cpu()))
    for b in bufs:
        assert bool((b[:guard] == 5).all()) and bool((b[-guard:] == 5).all())
    assert torch.equal(qi.cpu(), q) and torch.equal(ki.cpu(), kv)


def test_captured_call_replays_with_other_positions(dsa):
    batch = R.make([(0, 300), (0, 300)], 16, seed=8)
    gb = {k: v.cuda() for k, v in batch.items()}
    q = torch.zeros(9, 64, 512, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(9, 512, dtype=torch.bfloat16, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(kv)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        B.dsa_qk_norm_rope(q, kv, gb["new_start"], gb["seq_len"], qo, ko, gb["cos_sin"])
    for new, lens in (([1, 1], [300, 7]), ([0, 8], [0, 60])):
        b = dict(batch, seq_len=torch.tensor(lens, dtype=torch.int32),
                 new_start=torch.tensor([0] + new).cumsum(0).int())
        x, y = inputs(b, 64, sum(lens), rows=9)
        gb["seq_len"].copy_(b["seq_len"])
        gb["new_start"].copy_(b["new_start"])
        q.copy_(x)
        kv.copy_(y)
        qo.fill_(7.0)
        ko.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(b, x, y, (qo.cpu(), ko.cpu()), untouched=7.0)
