"""Attention over pages with logits of any size that fp32 holds: the running maximum and the
exponent must come from the same difference, and a row's first maximum from its own logits.

Every case has an answer that does not depend on the logits' own rounding:
- equal rows in the cache: whatever the (equal) weights, the output is that row;
- two kinds of rows whose logits differ by thousands: the output is the row of the larger one.
Tolerance: the weights are equal and exactly representable sums of them at most n * 2^-24 off
(chains of fp32 additions over n keys, in the sum and in the products: 2 n 2^-24), one bf16
rounding of the output (2^-8)."""
import pytest
import torch

import paged_ref as R
from deepseek_v4_sparse_ratio_gb300 import _binding as B

pytestmark = pytest.mark.gpu

# (sequences (new, total), heads): single tokens (whole and cut into parts), chunks
BATCHES = [([(1, 1), (1, 130)], 64), ([(1, 4000)], 64), ([(1, 300)], 128),
           ([(20, 150), (70, 70)], 64), ([(40, 3000)], 16)]


def _call(batch, q, scale, window=0):
    g = {k: None if v is None else v.cuda() for k, v in batch.items()}
    work = torch.full((B.DSA_PAGED_WORKSPACE_BYTES,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_paged_attn(q.cuda(), g["new_start"], g["seq_len"], g["page_table"], g["pages"], window,
                     scale, work, out, None, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    return out.cpu().double()


def _rows(lens, heads):
    """A batch without angles, its queries' shape, and the direction all rows lie along."""
    batch = R.make(lens, 32, rope=False, seed=3)
    d = torch.where(torch.randn(512, generator=torch.Generator().manual_seed(5)) > 0, 1.0, -1.0)
    return batch, (sum(n for n, _ in lens), heads, 512), d


@pytest.mark.parametrize("lens,heads", BATCHES)
# q . row is 512 * size; times the scale: logits from 1e9 to 1e36, and a tiny and a huge scale
@pytest.mark.parametrize("size,scale", [(2.0 ** 22, 0.5), (1.5 * 2.0 ** 22, 0.9), (2.0 ** 24, 1.1),
                                        (2.0 ** 60, 0.7), (2.0 ** 110, 0.3), (1.0, 2.0e38),
                                        (2.0 ** 100, 3.0e-39), (2.0 ** 90, 1e-30)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_rows(dsa, lens, heads, size, scale, sign):
    batch, shape, d = _rows(lens, heads)
    batch["pages"][:] = d.bfloat16()
    # each head another size, so that the product's rounding differs from head to head
    f = 1.0 + torch.arange(heads) / 128.0
    q = (sign * size * f[None, :, None] * d).expand(shape).bfloat16()
    out = _call(batch, q, scale)
    n = max(c for _, c in lens)
    err = (out - d.double()).abs()
    assert bool((err <= R.U + 2 * n * 2.0 ** -24).all()), err.max()


@pytest.mark.parametrize("lens,heads", BATCHES)
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("window", [0, 77])
def test_the_larger_of_two_kinds_of_rows(dsa, lens, heads, size, sign, window):
    """Rows at even positions are d / 2, the others d (position 0 sees the even kind alone)."""
    batch, shape, d = _rows(lens, heads)
    for s, (_, c) in enumerate(lens):
        for p in range(c):
            at = R.place(batch, s, p)
            batch["pages"][at] = (d * (1.0 if p % 2 else 0.5)).bfloat16()
    q = (sign * size * d).expand(shape).bfloat16()
    out = _call(batch, q, 0.4, window)
    r = 0
    for n, c in lens:
        for i in range(n):
            t = c - n + i
            big = 1.0 if sign > 0 and t > 0 and window != 1 else 0.5
            err = (out[r] - big * d.double()).abs()
            assert bool((err <= R.U + 2 * c * 2.0 ** -24).all()), (t, err.max())
            r += 1
