"""Sizes and scales at the ends of what the paged calls take: refused by a code before anything is
enqueued (addresses that are never followed; no GPU needed)."""
import pytest

import deepseek_v4_sparse_ratio_gb300 as dsa
from deepseek_v4_sparse_ratio_gb300 import _binding as B

from test_paged_abi import APPEND, ATTN


@pytest.fixture(scope="module")
def lib():
    dsa.build()
    return B.load()


def attn(lib, **change):
    return lib.dsa_paged_attn(*{**ATTN, **change}.values())


def append(lib, **change):
    return lib.dsa_paged_append(*{**APPEND, **change}.values())


# ATTN's output lies in its workspace, which only a call with nothing else wrong gets to hear;
# 9 << 40 is apart from everything
APART = 9 << 40


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_a_scale_that_leaves_fp32_in_log2_units(lib, scale):
    """scale * log2(e) is the factor of every logit: infinite, it makes 0 * inf of the largest."""
    assert attn(lib, out=APART, scale=scale) == B.DSA_ERR_SHAPE


@pytest.mark.parametrize("n_seqs", [(1 << 30) + 1, (1 << 31) - 200, (1 << 31) - 1])
def test_more_sequences_than_the_kernels_can_count(lib, n_seqs):
    """Their loops step past n_seqs by up to a block of threads: the sum has to stay in 32 bits."""
    assert append(lib, n_seqs=n_seqs) == B.DSA_ERR_SHAPE
    assert attn(lib, n_seqs=n_seqs, out=APART) == B.DSA_ERR_SHAPE
