"""Behaviour of the kernel for chunks (more than 256 rows of q per sequence on average) where
test_gpu_paged.py has it for the kernel for few rows: pages left out, entries that must not be
read, sequences that cannot be, non-finite queries, maxima that rise in every block, replays with
other lengths. Every batch is asserted to go to that kernel, every call finds its workspace full
of NaN and, where a page is left out, shared memory full of what a call before left there."""
import math

import numpy as np
import pytest
import torch

import paged_ref as R
from deepseek_v4_sparse_ratio_gb300 import _binding as B

from test_gpu_paged import args, check_attn, queries, to_gpu

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(512)


@pytest.fixture(scope="module")
def workspace(dsa):
    return torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def for_chunks(batch, q):
    return q.shape[0] * q.shape[1] > 256 * batch["seq_len"].shape[0]


def run(batch, q, window, workspace, scale=SCALE, status=None):
    assert for_chunks(batch, q)
    gb, qd = to_gpu(batch), q.cuda()
    workspace.fill_(255)      # NaN in fp32
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    assert qd.data_ptr() % 32 == 0 and out.data_ptr() % 32 == 0
    B.dsa_paged_attn(qd, *args(gb), window, scale, workspace, out, gb["cos_sin"], status)
    torch.cuda.synchronize()
    return out.cpu()


def poison(workspace, value):
    """A call whose rows are all `value`: what its tiles leave in shared memory."""
    batch = R.make([(64, 512)] * 4, 64, rope=False)
    batch["pages"].fill_(value)
    run(batch, queries(batch, 64, 1), 0, workspace)


def zero_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("junk", [float("nan"), float("-inf"), 2.0])
@pytest.mark.parametrize("heads", [64, 24])
@pytest.mark.parametrize("page,left_out", [
    (16, [(0, 0), (0, 3), (0, 7), (0, 8), (1, 2), (1, 15), (2, 0), (2, 1), (2, 2)]),
    (64, [(0, 0), (1, 3), (2, 0)]), (128, [(0, 1), (2, 0)]), (256, [(1, 0), (2, 0)])])
def test_pages_left_out(dsa, workspace, junk, heads, page, left_out):
    """First, middle and last page of a block, several of one block, and every page of the third
    sequence, whose tokens see nothing."""
    batch = R.make([(40, 300), (33, 270), (20, 40), (25, 500)], page, seed=14)
    n_pages = batch["pages"].shape[0]
    for i, (s, j) in enumerate(left_out):
        batch["page_table"][s, j] = (n_pages, -1, 2 ** 31 - 1, -2 ** 31)[i % 4]
    q = queries(batch, heads, 7)
    poison(workspace, junk)
    status = zero_status()
    out = run(batch, q, 0, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check_attn(out, batch, q, 0)


@pytest.mark.parametrize("window", [1, 50, 130])
@pytest.mark.parametrize("page", [16, 128])
def test_entries_below_the_window_or_past_the_end_are_not_read(dsa, workspace, window, page):
    lens = [(40, 400), (30, 300), (25, 25)]
    batch = R.make(lens, page, seed=15, max_pages=64)
    for s, (n, c) in enumerate(lens):
        low = max(0, c - n - window + 1)
        batch["page_table"][s, :low // page] = -7
        batch["page_table"][s, -(-c // page):] = 2 ** 30
    q = queries(batch, 64, 8)
    poison(workspace, float("inf"))
    status = zero_status()
    out = run(batch, q, window, workspace, status=status)
    assert status.item() == 0
    check_attn(out, batch, q, window)


def test_a_sequence_longer_than_its_table_or_angles_is_skipped(dsa, workspace):
    batch = R.make([(20, 100), (30, 60), (33, 90)], 16, seed=16)
    batch["cos_sin"] = batch["cos_sin"][:95].contiguous()
    q = queries(batch, 64, 9)
    status = zero_status()
    out = run(batch, q, 0, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check_attn(out, batch, q, 0)
    assert bool((out[:20] == 7.0).all())


@pytest.mark.parametrize("starts", [[0, 50, 20, 110], [-3, 20, 40, 90], [0, 40, 80, 200],
                                    [50, 50, 50, 50], [40, 70, 10, 40], [0, 31, 31, 90]])
def test_bad_starts_cost_their_own_sequences_alone(dsa, workspace, starts):
    batch = R.make([(30, 60), (30, 90), (30, 75)], 16, seed=4)
    q = queries(batch, 64, 1)
    batch["new_start"] = torch.tensor(starts, dtype=torch.int32)
    bad = [s for s in range(3) if not R.valid(batch, s, 90)]
    rows = np.zeros(90, dtype=int)
    for s in set(range(3)) - set(bad):
        rows[starts[s]:starts[s + 1]] += 1
    assert rows.max() <= 1
    status = zero_status()
    out = run(batch, q, 0, workspace, status=status)
    assert status.item() == (B.DSA_ERR_BOUNDS if bad else 0)
    check_attn(out, batch, q, 0)


@pytest.mark.parametrize("at,start", [(20, -1), (20, 5000), (31, -5), (1, 400), (64, -2)])
def test_one_start_out_of_order_among_many(dsa, workspace, at, start):
    batch = R.make([(6, 20 + s) for s in range(65)], 16, seed=30)
    q = queries(batch, 64, 7)
    batch["new_start"][at] = start
    ok = [s for s in range(65) if R.valid(batch, s, 390)]
    taken = np.zeros(391, dtype=int)
    for s in ok:
        a, b = batch["new_start"][s:s + 2].tolist()
        taken[a:b] += 1
    assert 2 <= len(ok) < 65 and taken.max() == 1
    status = zero_status()
    out = run(batch, q, 0, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check_attn(out, batch, q, 0)


@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("heads", [16, 64])
def test_non_finite_queries_stay_in_their_rows(dsa, workspace, rope, heads):
    """In dims of shared memory (5), of TMEM (400) and of the rotation (500)."""
    batch = R.make([(40, 300)], 64, rope=rope, seed=13)
    q = queries(batch, heads, 6)
    clean = q.clone()
    bad = [(2, 5, 5, float("nan")), (4, 0, 400, float("inf")), (17, heads - 1, 500, float("nan")),
           (39, 3, 501, float("-inf"))]
    for t, h, dim, v in bad:
        q[t, h, dim] = v
    q[11, 7] = float("nan")
    out = run(batch, q, 0, workspace)
    ref, tol, _ = R.attention(batch, clean, 0, SCALE)
    ok = torch.ones(40, heads, dtype=torch.bool)
    for t, h, *_ in bad + [(11, 7)]:
        ok[t, h] = False
    assert bool(((out.double() - ref).abs() <= tol)[ok].all())
    assert bool(out[~ok].isnan().all())


@pytest.mark.parametrize("some", [None, 0, 5])
def test_rising_logits_rescale_every_block(dsa, workspace, some):
    """Keys whose logits grow block by block, for every row of q or for one head in eight."""
    lens = [(40, 1200), (64, 900)]
    batch = R.make(lens, 64, rope=False, seed=8)
    d = torch.randn(512, generator=torch.Generator().manual_seed(1))
    for s, (_, c) in enumerate(lens):
        for p in range(c):
            at = R.place(batch, s, p)
            batch["pages"][at] = (d * (0.2 + p / 400.0)
                                  + 0.1 * batch["pages"][at].float()).bfloat16()
    q = 0.1 * queries(batch, 16, 3).float()
    if some is None:
        q += d
    else:
        q[:, some::8] += d
    q = q.bfloat16()
    out = run(batch, q, 0, workspace)
    check_attn(out, batch, q, 0)


@pytest.mark.parametrize("window", [0, 100])
def test_captured_step_replays_with_other_lengths(dsa, workspace, window):
    """One graph of append + attention padded to 64 rows of 64 heads, three users."""
    batch = R.make([(0, 400), (0, 400), (0, 400)], 16, seed=23)
    g = torch.Generator().manual_seed(24)
    gb = to_gpu(batch)
    kv = torch.zeros(64, 512, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(64, 64, 512, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    assert for_chunks(batch, q)
    # (set up outside the capture, as a program's warm-up does)
    B.dsa_paged_attn(q, *args(gb), window, SCALE, workspace, out, gb["cos_sin"])
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        B.dsa_paged_append(kv, *args(gb), gb["cos_sin"])
        B.dsa_paged_attn(q, *args(gb), window, SCALE, workspace, out, gb["cos_sin"])
    for new, lens in [([60, 1, 3], [260, 9, 300]), ([1, 1, 1], [261, 10, 301]),
                      ([0, 64, 0], [0, 64, 5]), ([0, 0, 0], [1, 2, 3]), ([20, 20, 20], [20, 84, 400])]:
        b = dict(batch, pages=gb["pages"].cpu(), seq_len=torch.tensor(lens, dtype=torch.int32),
                 new_start=torch.tensor([0] + new).cumsum(0).int())
        kvh = torch.randn(64, 512, generator=g).bfloat16()
        qh = torch.randn(64, 64, 512, generator=g).bfloat16()
        kv.copy_(kvh)
        q.copy_(qh)
        out.fill_(7.0)
        workspace.fill_(255)
        gb["seq_len"].copy_(b["seq_len"])
        gb["new_start"].copy_(b["new_start"])
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        ref, tol = R.append(b, kvh)
        got = gb["pages"].cpu()
        assert bool(((got.double() - ref).abs() <= tol).all())
        b["pages"] = got
        check_attn(out.cpu(), b, qh, window)


@pytest.mark.parametrize("lens,heads,page,window", [
    ([(150, 700)], 64, 64, 0), ([(700, 900), (1, 33), (350, 350)], 16, 32, 100),
    ([(100, 100)] * 12 + [(90, 128)], 64, 32, 0)])
def test_nothing_of_the_workspace_is_read_before_it_is_written(dsa, workspace, lens, heads, page,
                                                              window):
    batch = R.make(lens, page, seed=heads + page)
    q = queries(batch, heads, 11)
    check_attn(run(batch, q, window, workspace), batch, q, window)


@pytest.mark.parametrize("lens,heads", [([(1, 5000)], 64), ([(1, 30 + 7 * i) for i in range(200)], 4),
                                        ([(3, 500), (5, 5)], 16), ([(1, 40000)], 64)])
def test_nor_by_the_kernel_for_few_rows(dsa, workspace, lens, heads):
    batch = R.make(lens, 64, seed=heads)
    q = queries(batch, heads, 11)
    assert not for_chunks(batch, q)
    gb = to_gpu(batch)
    workspace.fill_(255)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    B.dsa_paged_attn(q.cuda(), *args(gb), 0, SCALE, workspace, out, gb["cos_sin"])
    torch.cuda.synchronize()
    check_attn(out.cpu(), batch, q, 0)
