"""What the Python binding of the paged calls must not hand on (CPU tensors, no GPU needed)."""
import pytest
import torch

import deepseek_v4_sparse_ratio_gb300 as dsa
from deepseek_v4_sparse_ratio_gb300 import _binding as B


@pytest.fixture(scope="module")
def lib():
    dsa.build()
    return B.load()


def meta(*shape, dtype=torch.int32):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("n_seqs,max_pages,page,heads", [
    (2, (1 << 32) + 8, 64, 8), ((1 << 32) + 2, 8, 64, 8), (2, 8, (1 << 32) + 64, 8),
    (2, 8, 64, (1 << 32) + 8)])
def test_sizes_beyond_32_bits_are_refused(lib, monkeypatch, n_seqs, max_pages, page, heads):
    """ctypes would drop their upper bits and pass a table of 8 columns, 2 sequences, pages of 64
    rows or 8 heads on."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # where meta tensors are
    bf16 = torch.bfloat16
    common = (meta(n_seqs + 1), meta(n_seqs), meta(n_seqs, max_pages),
              meta(10, page, 512, dtype=bf16))
    kv, q = meta(3, 512, dtype=bf16), meta(3, heads, 512, dtype=bf16)
    work = meta(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8)

    def never(*a):
        raise AssertionError("the library was called")

    monkeypatch.setattr(B, "_lib", type("L", (), dict(
        dsa_paged_append=staticmethod(never), dsa_paged_attn=staticmethod(never),
        dsa_strerror=staticmethod(lib.dsa_strerror)))())
    if heads == 8:
        with pytest.raises(B.DsaError) as e:
            B.dsa_paged_append(kv, *common, stream=0)
        assert e.value.code == B.DSA_ERR_SHAPE
    with pytest.raises(B.DsaError) as e:
        B.dsa_paged_attn(q, *common, 0, 0.1, work, torch.empty_like(q), stream=0)
    assert e.value.code == B.DSA_ERR_SHAPE
