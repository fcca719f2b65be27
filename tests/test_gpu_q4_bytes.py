"""Rows of the 4-bit pages whose exponent byte no append writes (14 to 250 are written): bytes of
other programs, or of memory that was never written."""
import pytest
import q4_ref as Q
import torch
from deepseek_v4_sparse_ratio_gb300 import _binding as B
from test_gpu_q4 import SCALE, args, queries, run_attn, to_gpu, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def spoil(batch, p, byte):
    """Position p of the first sequence: the largest scales, with an exponent byte."""
    row = batch["pages"][Q.place(batch, 0, p)]
    row[0:14] = row[16:30] = 0x7E
    row[14] = row[30] = byte


@pytest.mark.parametrize("byte", [251, 253, 255])
@pytest.mark.parametrize("heads", [8, 16])
def test_a_later_tokens_row_stays_with_the_tokens_that_see_it(dsa, workspace, heads, byte):  # noqa: F811
    """Tokens of one unit of work: the first six do not see row 134, whose scales times its power
    of two are beyond what bf16 holds."""
    batch = Q.make([(12, 140)], 64, seed=10)
    q = queries(batch, heads, 5)
    ref, tol, _ = Q.attention(batch, q, 0, 0, SCALE)
    spoil(batch, 134, byte)
    out = run_attn(batch, q, 0, 0, workspace)
    assert bool(((out[:6].double() - ref[:6]).abs() <= tol[:6]).all())


@pytest.mark.parametrize("byte", [251, 255])
@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("heads", [8, 16])
def test_a_row_that_leaves_the_window_stays_behind(dsa, workspace, heads, sinks, byte):  # noqa: F811
    """Row 165 is seen by the first of six tokens (at 194) with a window of 30, and by no other."""
    batch = Q.make([(6, 200)], 64, seed=11)
    q = queries(batch, heads, 5)
    ref, tol, _ = Q.attention(batch, q, 30, sinks, SCALE)
    spoil(batch, 165, byte)
    out = run_attn(batch, q, 30, sinks, workspace)
    assert bool(((out[1:].double() - ref[1:]).abs() <= tol[1:]).all())


@pytest.mark.parametrize("of", ["read", "attention"])
def test_every_exponent_byte_stands_for_the_same(dsa, workspace, of):  # noqa: F811
    """A sequence of one row for every byte: bytes below 14 stand for 14 and those above 250 for 250,
    in both calls. A query of zeros gives its only row the weight 1, so the attention returns it:
    exactly, as n s 2^E is a bf16 (with scales of 1 and more a normal one)."""
    batch = Q.make([(1, 1)] * 256, 16, rope=False, seed=12)
    g = torch.Generator().manual_seed(13)
    want = torch.zeros(256, 512, dtype=torch.float64)
    for s in range(256):
        row = batch["pages"][Q.place(batch, s, 0)]
        row[32:256] = torch.randint(0, 256, (224,), generator=g)       # all codes, n = -8 among them
        least = 0x38 if of == "attention" else 0
        sign = torch.randint(0, 2, (30,), generator=g) * 128
        row[:30] = torch.randint(least, 0x7F, (30,), generator=g) + sign
        row[14] = row[30] = min(max(s, 14), 250)
        row[15] = row[31] = 0
        want[s] = Q.decode(row)
        row[14] = row[30] = s
    if of == "attention":
        q = torch.zeros(256, 4, 512, dtype=torch.bfloat16)
        out = run_attn(batch, q, 0, 0, workspace).double()
        assert torch.equal(out, want[:, None].expand(-1, 4, -1))
    else:
        gb = to_gpu(batch)
        out = torch.empty(256, 512, dtype=torch.bfloat16, device="cuda")
        B.dsa_paged_q4_read(*args(gb), out)
        assert torch.equal(out.cpu().double(), want)
