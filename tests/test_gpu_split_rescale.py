"""The split (few tokens) mode of the window + selected attention, where the running maximum of
one half of the heads rises in a CTA's later blocks and the other half's does not: each half
keeps its own maximum, and the merge of the cluster's partial results must take it from there."""
import math

import numpy as np
import pytest
import torch

import oracle
from deepseek_v4_sparse_ratio_gb300 import _binding as B

from parity import bf16_to_f64, check_attention

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(512)


@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("first", [896, 1920])
def test_one_half_of_the_heads_rises_alone(dsa, half, first):
    """128 window rows + 2048 selected ones = 17 blocks over 8 CTAs; pooled rows from `first` on
    carry a direction that one half of the heads looks along (logits of about 20)."""
    off, T, k = 20000, 1, 2048
    n = (off + T) // 4
    g = torch.Generator().manual_seed(11)
    d = torch.randn(512, generator=g)
    raw = (0.2 * torch.randn(128, 512, generator=g)).bfloat16()
    pooled = 0.2 * torch.randn(n, 512, generator=g)
    pooled[first:k] += 0.9 * d
    pooled = pooled.bfloat16()
    q = 0.1 * torch.randn(T, 64, 512, generator=g)
    q[:, 32 * half:32 * half + 32] += d
    q = q.bfloat16()
    sel = torch.arange(k, dtype=torch.int32).repeat(T, 1)
    out = torch.empty(T, 64, 512, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_window_sparse_attn(q.cuda(), raw.cuda(), off - 127, pooled.cuda(), n, sel.cuda(), k, T,
                             off, 4, 128, SCALE, out, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    ref = oracle.attention(q, off + np.arange(T), raw, off - 127, oracle.as_bf16_bits(pooled), n,
                           sel.numpy(), 128, SCALE)
    # each head on its own scale: one half's outputs are much larger than the other's
    got = bf16_to_f64(out)
    for h in range(64):
        check_attention(got[:, h:h + 1], ref[:, h:h + 1])
