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


LONG = dict(page_size=1024, page_stride=1024 * 512, max_pages=1 << 14, cos_sin=None, out=APART)


@pytest.mark.parametrize("change", [
    dict(n_new=5_000_000, heads=33, n_seqs=1),            # two units per three tokens
    dict(n_new=2_600_000, heads=65, n_seqs=1),            # two per token
    dict(n_new=3_000_000, heads=1, n_seqs=3_000_000)])    # a unit per sequence
def test_more_blocks_than_a_cta_can_count(lib, change):
    """131,072 blocks for each of more than 2.5 million units: a 152nd passes 32 bits."""
    assert attn(lib, **LONG, **change) == B.DSA_ERR_SHAPE


@pytest.mark.parametrize("change", [
    dict(n_new=5_000_000, heads=33, n_seqs=1, window=4096),
    dict(n_new=1_000_000, heads=65, n_seqs=1),
    dict(n_new=3_000_000, heads=1, n_seqs=1)])
def test_long_work_that_can_be_counted_is_not_refused(lib, change):
    """It gets past the checks of the arguments: to the workspace's, here one byte short."""
    short = B.DSA_PAGED_WORKSPACE_BYTES - 1
    assert attn(lib, **LONG, **change, workspace_bytes=short) == B.DSA_ERR_SCRATCH


STRIDE = 3 * 64 * 512                     # two thirds of every stride is other data
PAGE, NEXT = 64 * 512 * 2, STRIDE * 2     # bytes of a page, and from one to the next
POOL = 5 << 40


@pytest.mark.parametrize("at,hit", [
    (POOL - 4 * 1024, False), (POOL - 4 * 1024 + 16, True), (POOL, True), (POOL + PAGE - 16, True),
    (POOL + PAGE, False), (POOL + NEXT - 4 * 1024, False), (POOL + NEXT - 16, True),
    (POOL + 9 * NEXT + PAGE - 16, True), (POOL + 9 * NEXT + PAGE, False),
    (POOL + 10 * NEXT, False), (POOL + (1 << 30), False)])
def test_rows_inside_the_pages_are_refused(lib, at, hit):
    """kv read while pages are written, out written while pages are read: whichever comes first.
    Between the pages, where another layer's may lie, either is fine (the call then gets to
    its workspace, which is missing: none of these reaches a GPU)."""
    pool = dict(pages=POOL, page_stride=STRIDE)
    code = B.DSA_ERR_ARG if hit else B.DSA_ERR_SCRATCH
    assert attn(lib, **pool, out=at, heads=1, workspace=None) == code
    if hit:
        assert append(lib, **pool, kv=at) == code


WORK = ATTN["workspace"]


@pytest.mark.parametrize("change", [
    dict(out=WORK), dict(out=WORK + B.DSA_PAGED_WORKSPACE_BYTES - 16),
    dict(out=APART, q=WORK + 4096), dict(out=APART, pages=WORK + 4096),
    dict(out=APART, pages=WORK - 9 * 64 * 1024 - 16)])
def test_a_workspace_that_holds_other_arguments_is_refused(lib, change):
    """Parts of cut units would be written over what other SMs still read or write."""
    assert attn(lib, **change) == B.DSA_ERR_ARG
