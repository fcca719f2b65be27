"""Rows of the 4-bit pages whose exponent byte no append writes (14 to 250 are written): bytes of
other programs, or of memory that was never written."""
import pytest
import q4_ref as Q
import torch
from test_gpu_q4 import SCALE, queries, run_attn, workspace  # noqa: F401

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
