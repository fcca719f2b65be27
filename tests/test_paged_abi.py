"""Refusals of the paged calls, and that they come before anything is enqueued: the C entry
points with addresses that are never followed, the binding with CPU tensors (no GPU needed)."""
import pytest
import torch

import deepseek_v4_sparse_ratio_gb300 as dsa
from deepseek_v4_sparse_ratio_gb300 import _binding as B

import paged_ref as R

FAKE = 1 << 20
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    dsa.build()
    return B.load()


APPEND = dict(kv=FAKE, n_new=4, new_start=FAKE, seq_len=FAKE, n_seqs=2, page_table=FAKE,
              max_pages=8, pages=FAKE, n_pages=10, page_stride=64 * 512, page_size=64,
              cos_sin=FAKE, n_pos=512, dev_status=None, stream=None)
ATTN = dict(q=FAKE, heads=64, n_new=4, new_start=FAKE, seq_len=FAKE, n_seqs=2, page_table=FAKE,
            max_pages=8, pages=FAKE, n_pages=10, page_stride=64 * 512, page_size=64, cos_sin=FAKE,
            n_pos=512, window=0, scale=0.1, workspace=BIG,
            workspace_bytes=B.DSA_PAGED_WORKSPACE_BYTES, out=BIG, dev_status=None, stream=None)

SHARED = [
    (dict(new_start=None), B.DSA_ERR_ARG), (dict(seq_len=None), B.DSA_ERR_ARG),
    (dict(page_table=None), B.DSA_ERR_ARG), (dict(pages=None), B.DSA_ERR_ARG),
    (dict(n_new=0), B.DSA_ERR_ARG), (dict(n_new=-3), B.DSA_ERR_ARG),
    (dict(n_seqs=0), B.DSA_ERR_ARG), (dict(max_pages=0), B.DSA_ERR_ARG),
    (dict(n_pages=0), B.DSA_ERR_ARG), (dict(n_pos=0), B.DSA_ERR_ARG),
    (dict(pages=FAKE + 8), B.DSA_ERR_ARG), (dict(cos_sin=FAKE + 4), B.DSA_ERR_ARG),
    (dict(new_start=FAKE + 2), B.DSA_ERR_ARG), (dict(dev_status=FAKE + 1), B.DSA_ERR_ARG),
    (dict(page_size=8, page_stride=8 * 512), B.DSA_ERR_SHAPE),
    (dict(page_size=48), B.DSA_ERR_SHAPE),
    (dict(page_size=2048, page_stride=2048 * 512), B.DSA_ERR_SHAPE),
    (dict(page_size=0), B.DSA_ERR_SHAPE), (dict(page_size=-64), B.DSA_ERR_SHAPE),
    (dict(page_stride=64 * 512 - 8), B.DSA_ERR_SHAPE),
    (dict(page_stride=64 * 512 + 4), B.DSA_ERR_SHAPE),
    (dict(page_stride=1 << 39), B.DSA_ERR_SHAPE),
    (dict(n_new=1 << 31), B.DSA_ERR_SHAPE), (dict(n_pages=1 << 31), B.DSA_ERR_SHAPE),
    (dict(max_pages=1 << 25), B.DSA_ERR_SHAPE),
]


@pytest.mark.parametrize("change,code", SHARED + [
    (dict(kv=None), B.DSA_ERR_ARG), (dict(kv=FAKE + 8), B.DSA_ERR_ARG)])
def test_append_refuses(lib, change, code):
    assert lib.dsa_paged_append(*{**APPEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", SHARED + [
    (dict(q=None), B.DSA_ERR_ARG), (dict(out=None), B.DSA_ERR_ARG),
    (dict(q=FAKE + 8), B.DSA_ERR_ARG), (dict(out=BIG + 2), B.DSA_ERR_ARG),
    (dict(out=FAKE), B.DSA_ERR_ARG), (dict(out=FAKE + 4 * 64 * 1024 - 16), B.DSA_ERR_ARG),
    (dict(heads=0), B.DSA_ERR_SHAPE), (dict(heads=129), B.DSA_ERR_SHAPE),
    (dict(n_new=1 << 25, heads=64), B.DSA_ERR_SHAPE),
    (dict(window=-1), B.DSA_ERR_SHAPE), (dict(scale=0.0), B.DSA_ERR_SHAPE),
    (dict(scale=float("nan")), B.DSA_ERR_SHAPE), (dict(scale=float("inf")), B.DSA_ERR_SHAPE),
    (dict(workspace=None), B.DSA_ERR_SCRATCH), (dict(workspace=BIG + 8), B.DSA_ERR_SCRATCH),
    (dict(workspace_bytes=B.DSA_PAGED_WORKSPACE_BYTES - 1), B.DSA_ERR_SCRATCH)])
def test_attention_refuses(lib, change, code):
    assert lib.dsa_paged_attn(*{**ATTN, **change}.values()) == code


def test_limits_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                             "include", "dsa.h")).read()
    get = lambda n: int(re.search(rf"#define\s+{n}\s+(\d+)", text).group(1))  # noqa: E731
    assert get("DSA_ROPE_DIM") == B.ROPE_DIM
    assert get("DSA_MAX_PAGE_SIZE") == B.MAX_PAGE_SIZE
    assert get("DSA_MAX_PAGED_HEADS") == B.MAX_PAGED_HEADS
    m = re.search(r"#define\s+DSA_MAX_PAGED_TOKENS\s+\((\d+) << (\d+)\)", text)
    assert B.MAX_PAGED_TOKENS == int(m.group(1)) << int(m.group(2))
    m = re.search(r"#define\s+DSA_PAGED_WORKSPACE_BYTES\s+\(\(size_t\)(\d+)\s*<<\s*(\d+)\)", text)
    assert B.DSA_PAGED_WORKSPACE_BYTES == int(m.group(1)) << int(m.group(2))


def test_binding_refuses_tensors_of_another_kind(lib, monkeypatch):
    """CPU tensors, other types, strides and shapes: DsaError before the library is called."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    b = R.make([(2, 20), (1, 5)], 16)
    kv = torch.zeros(3, 512, dtype=torch.bfloat16)
    common = (b["new_start"], b["seq_len"], b["page_table"], b["pages"])
    with pytest.raises(B.DsaError) as e:
        B.dsa_paged_append(kv, *common, b["cos_sin"])
    assert e.value.code == B.DSA_ERR_ARG and "kv" in str(e.value)
    with pytest.raises(B.DsaError):
        B.dsa_paged_attn(torch.zeros(3, 64, 512, dtype=torch.bfloat16), *common, 0, 0.1,
                         torch.zeros(8), torch.zeros(3, 64, 512, dtype=torch.bfloat16))
    # shapes and types are looked at the same way on the device the tensors are said to be on
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    for bad in (kv.float(), kv[:, :256], torch.zeros(512, 3, dtype=torch.bfloat16).t()):
        with pytest.raises(B.DsaError, match="kv"):
            B.dsa_paged_append(bad, *common)
    with pytest.raises(B.DsaError, match="new_start"):
        B.dsa_paged_append(kv, b["new_start"][:2], *common[1:])
    with pytest.raises(B.DsaError, match="seq_len"):
        B.dsa_paged_append(kv, b["new_start"], b["seq_len"].long(), *common[2:])
    with pytest.raises(B.DsaError, match="page_table"):
        B.dsa_paged_append(kv, b["new_start"], b["seq_len"], b["page_table"].repeat(1, 2)[:, ::2],
                           b["pages"])
    with pytest.raises(B.DsaError, match="pages"):
        B.dsa_paged_append(kv, *common[:3], b["pages"].transpose(0, 1))
    with pytest.raises(B.DsaError, match="cos_sin"):
        B.dsa_paged_append(kv, *common, b["cos_sin"][:, :16])
    with pytest.raises(B.DsaError, match="cos_sin"):
        B.dsa_paged_append(kv, *common, torch.tensor(1.0))
    with pytest.raises(B.DsaError, match="page_table"):
        B.dsa_paged_append(kv, b["new_start"], b["seq_len"], b["page_table"][0], b["pages"])
    with pytest.raises(B.DsaError, match="dev_status"):
        B.dsa_paged_append(kv, *common, b["cos_sin"], torch.zeros(2, dtype=torch.int32))
    q = torch.zeros(3, 8, 512, dtype=torch.bfloat16)
    work = torch.zeros(4)
    for out in (q[:2], q.float(), torch.zeros(3, 512, 8, dtype=torch.bfloat16).transpose(1, 2)):
        with pytest.raises(B.DsaError, match="out"):
            B.dsa_paged_attn(q, *common, 0, 0.1, work, out)
    for window in (1 << 31, 1 << 40, -1):
        with pytest.raises(B.DsaError, match="window") as e:
            B.dsa_paged_attn(q, *common, window, 0.1, work, torch.zeros_like(q))
        assert e.value.code == B.DSA_ERR_SHAPE
    with pytest.raises(B.DsaError, match="workspace"):
        B.dsa_paged_attn(q, *common, 0, 0.1, torch.zeros(8, 8).t()[::2], torch.zeros_like(q))
