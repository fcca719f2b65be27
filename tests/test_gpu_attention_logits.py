"""The window + selected attention at the largest logits that its description allows (1e9 in size):
with all rows equal the output is that row, whatever the logits' rounding. Tolerance: sums of n
equal weights in fp32 (2 n 2^-24) and one bf16 rounding of the output."""
import pytest
import torch

from deepseek_v4_sparse_ratio_gb300 import _binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 8, 200])        # a cluster per token, and one CTA per token
@pytest.mark.parametrize("window,k", [(1, 4), (128, 2048)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_rows_at_the_largest_logits(dsa, T, window, k, sign):
    off = 20000
    n = (off + T) // 4
    d = torch.where(torch.randn(512, generator=torch.Generator().manual_seed(5)) > 0, 1.0, -1.0)
    rows = lambda m: d.bfloat16().expand(m, 512).contiguous().cuda()  # noqa: E731
    # q . row = 512 * 2^21 * f, times the scale: 0.47e9 to 0.94e9
    f = 1.0 + torch.arange(64) / 64.0
    q = (sign * 2.0 ** 21 * f[None, :, None] * d).expand(T, 64, 512).bfloat16().cuda()
    scale = 0.4375
    sel = torch.arange(k, dtype=torch.int32, device="cuda").repeat(T, 1)
    out = torch.empty(T, 64, 512, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_window_sparse_attn(q, rows(window - 1 + T), off - window + 1, rows(n), n, sel, k, T, off,
                             4, window, scale, out, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    err = (out.cpu().double() - d.double()).abs()
    assert bool((err <= 2.0 ** -8 + 2 * (window + k) * 2.0 ** -24).all()), err.max()
