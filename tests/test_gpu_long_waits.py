"""The waits of the paged kernels that span whole units of work: their budget of about a second
counts from the last block of keys, so a long context on a slow machine does not run it out."""
import time

import pytest
import torch

from deepseek_v4_sparse_ratio_gb300 import _binding as B

pytestmark = pytest.mark.gpu


def _timed(mode):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    B.dsa_bounded_wait_selftest(mode, status)
    torch.cuda.synchronize()
    return status.item(), time.perf_counter() - t0


def test_a_wait_longer_than_its_budget_completes_while_blocks_move_on(dsa):
    """One and a half budgets of 2^31 cycles: at 2.07 GHz at most, 1.55 s at least."""
    code, dt = _timed(2)
    assert code == B.DSA_OK
    assert 1.5 < dt < 30.0, dt


def test_a_wait_without_progress_runs_out(dsa):
    code, dt = _timed(3)
    assert code == B.DSA_ERR_TIMEOUT
    assert dt < 30.0, dt


@pytest.mark.parametrize("seqs,tokens", [(1, 608), (304, 1)])
def test_whole_units_of_the_longest_sequence(dsa, seqs, tokens):
    """Equal rows, 2^24 of them, 64 heads: every weight is 1, every sum a whole number up to 2^24,
    and the output the row, rounded once (2^-8). Whole units for each of 152 SMs: 608 tokens of one
    sequence are four of 131,072 blocks, the queries of two shared, so that the wait for the next
    queries lasts half of the call; 304 sequences of one token (that share their pages) are two,
    the rotation of the second one's queries waits for the first."""
    d = torch.where(torch.randn(512, generator=torch.Generator().manual_seed(5)) > 0, 1.0, -1.0)
    pages = d.bfloat16().expand(4, 1024, 512).contiguous().cuda()
    length, rows = B.MAX_PAGED_TOKENS, seqs * tokens
    table = (torch.arange(length // 1024) % 4).int().expand(seqs, -1).contiguous().cuda()
    # angles of zero
    cos_sin = torch.zeros(length, 32, 2, device="cuda")
    cos_sin[..., 0] = 1.0
    q = torch.randn(rows, 64, 512, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    out = torch.zeros_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    work = torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    starts = torch.arange(0, rows + 1, tokens, dtype=torch.int32, device="cuda")
    lens = torch.full((seqs,), length, dtype=torch.int32, device="cuda")
    B.dsa_paged_attn(q, starts, lens, table, pages, 0, 512 ** -0.5, work, out, cos_sin, status)
    torch.cuda.synchronize()
    assert status.item() == B.DSA_OK
    assert bool((out.float() * d.cuda() - 1.0).abs().max() <= 2.0 ** -8)
