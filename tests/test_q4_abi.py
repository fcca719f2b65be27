"""Refusals of the norm with rotation and of the 4-bit paged calls, before anything is enqueued:
the C entry points with addresses that are never followed, the binding with CPU tensors."""
import os
import re

import pytest
import torch

import deepseek_v4_sparse_ratio_gb300 as dsa
from deepseek_v4_sparse_ratio_gb300 import _binding as B

import q4_ref as Q

FAKE = 1 << 20
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    dsa.build()
    return B.load()


NORM = dict(q=FAKE, heads=64, kv=BIG, n_new=4, new_start=FAKE, seq_len=FAKE, n_seqs=2,
            q_weight=None, kv_weight=FAKE, eps=1e-6, cos_sin=FAKE, n_pos=512, q_out=2 * BIG,
            kv_out=3 * BIG, dev_status=None, stream=None)
APPEND = dict(kv=BIG, n_new=4, new_start=FAKE, seq_len=FAKE, n_seqs=2, page_table=FAKE,
              max_pages=8, pages=FAKE, n_pages=10, page_stride=64 * 384, page_size=64,
              cos_sin=FAKE, n_pos=512, dev_status=None, stream=None)
READ = dict(new_start=FAKE, seq_len=FAKE, n_seqs=2, page_table=FAKE, max_pages=8, pages=FAKE,
            n_pages=10, page_stride=64 * 384, page_size=64, cos_sin=None, n_pos=0, out=BIG,
            n_new=4, dev_status=None, stream=None)
ATTN = dict(q=FAKE, heads=64, n_new=4, new_start=FAKE, seq_len=FAKE, n_seqs=2, page_table=FAKE,
            max_pages=8, pages=4 * BIG, n_pages=10, page_stride=64 * 384, page_size=64,
            cos_sin=FAKE, n_pos=512, window=0, sinks=0, q_turned=0, scale=0.1, workspace=BIG,
            workspace_bytes=B.DSA_PAGED_WORKSPACE_BYTES, out=3 * BIG, dev_status=None, stream=None)

BATCH = [
    (dict(new_start=None), B.DSA_ERR_ARG), (dict(seq_len=None), B.DSA_ERR_ARG),
    (dict(n_new=0), B.DSA_ERR_ARG), (dict(n_new=-3), B.DSA_ERR_ARG),
    (dict(n_seqs=0), B.DSA_ERR_ARG), (dict(cos_sin=FAKE, n_pos=0), B.DSA_ERR_ARG),
    (dict(cos_sin=FAKE + 4, n_pos=9), B.DSA_ERR_ARG), (dict(new_start=FAKE + 2), B.DSA_ERR_ARG),
    (dict(dev_status=FAKE + 1), B.DSA_ERR_ARG), (dict(n_new=1 << 31), B.DSA_ERR_SHAPE),
    (dict(n_seqs=(1 << 30) + 1), B.DSA_ERR_SHAPE),
]
PAGES = BATCH + [
    (dict(page_table=None), B.DSA_ERR_ARG), (dict(pages=None), B.DSA_ERR_ARG),
    (dict(max_pages=0), B.DSA_ERR_ARG), (dict(n_pages=0), B.DSA_ERR_ARG),
    (dict(pages=FAKE + 8), B.DSA_ERR_ARG), (dict(pages=FAKE + 16), B.DSA_ERR_ARG),
    (dict(page_size=8, page_stride=8 * 384), B.DSA_ERR_SHAPE),
    (dict(page_size=48), B.DSA_ERR_SHAPE),
    (dict(page_size=2048, page_stride=2048 * 384), B.DSA_ERR_SHAPE),
    (dict(page_stride=64 * 384 - 32), B.DSA_ERR_SHAPE),
    (dict(page_stride=64 * 384 + 8), B.DSA_ERR_SHAPE),
    (dict(page_stride=64 * 384 + 16), B.DSA_ERR_SHAPE),
    (dict(page_stride=1 << 39), B.DSA_ERR_SHAPE), (dict(n_pages=1 << 31), B.DSA_ERR_SHAPE),
    (dict(max_pages=1 << 25), B.DSA_ERR_SHAPE),
]


@pytest.mark.parametrize("change,code", BATCH + [
    (dict(q=None), B.DSA_ERR_ARG), (dict(kv=None), B.DSA_ERR_ARG), (dict(q_out=None), B.DSA_ERR_ARG),
    (dict(kv_out=None), B.DSA_ERR_ARG), (dict(q=FAKE + 8), B.DSA_ERR_ARG),
    (dict(kv_out=3 * BIG + 4), B.DSA_ERR_ARG), (dict(kv_weight=FAKE + 4), B.DSA_ERR_ARG),
    (dict(q_weight=FAKE + 8), B.DSA_ERR_ARG),
    (dict(heads=0), B.DSA_ERR_SHAPE), (dict(heads=129), B.DSA_ERR_SHAPE),
    (dict(n_new=1 << 25), B.DSA_ERR_SHAPE), (dict(eps=0.0), B.DSA_ERR_SHAPE),
    (dict(eps=-1e-6), B.DSA_ERR_SHAPE), (dict(eps=float("nan")), B.DSA_ERR_SHAPE),
    (dict(eps=float("inf")), B.DSA_ERR_SHAPE),
    # overlaps that are not "the same array"
    (dict(q_out=FAKE + 1024), B.DSA_ERR_ARG), (dict(kv_out=BIG + 1024), B.DSA_ERR_ARG),
    (dict(q_out=BIG), B.DSA_ERR_ARG), (dict(kv_out=FAKE), B.DSA_ERR_ARG),
    (dict(kv_out=2 * BIG + 4 * 64 * 1024 - 16), B.DSA_ERR_ARG)])
def test_norm_refuses(lib, change, code):
    assert lib.dsa_qk_norm_rope(*{**NORM, **change}.values()) == code


@pytest.mark.parametrize("change,code", PAGES + [
    (dict(kv=None), B.DSA_ERR_ARG), (dict(kv=BIG + 8), B.DSA_ERR_ARG),
    (dict(kv=FAKE), B.DSA_ERR_ARG), (dict(kv=FAKE + 9 * 64 * 384 + 16), B.DSA_ERR_ARG),
    (dict(kv=FAKE + 63 * 384, n_new=1, page_stride=64 * 384 + 4096), B.DSA_ERR_ARG)])
def test_append_refuses(lib, change, code):
    assert lib.dsa_paged_q4_append(*{**APPEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", PAGES + [
    (dict(out=None), B.DSA_ERR_ARG), (dict(out=BIG + 8), B.DSA_ERR_ARG),
    (dict(out=FAKE + 1024), B.DSA_ERR_ARG)])
def test_read_refuses(lib, change, code):
    assert lib.dsa_paged_q4_read(*{**READ, **change}.values()) == code


@pytest.mark.parametrize("change,code", PAGES + [
    (dict(q=None), B.DSA_ERR_ARG), (dict(out=None), B.DSA_ERR_ARG),
    (dict(q=FAKE + 8), B.DSA_ERR_ARG), (dict(out=3 * BIG + 2), B.DSA_ERR_ARG),
    (dict(out=FAKE), B.DSA_ERR_ARG), (dict(out=FAKE + 4 * 64 * 1024 - 16), B.DSA_ERR_ARG),
    (dict(out=4 * BIG), B.DSA_ERR_ARG), (dict(workspace=4 * BIG + 4096), B.DSA_ERR_ARG),
    (dict(workspace=3 * BIG), B.DSA_ERR_ARG),
    (dict(heads=0), B.DSA_ERR_SHAPE), (dict(heads=129), B.DSA_ERR_SHAPE),
    (dict(n_new=1 << 25), B.DSA_ERR_SHAPE), (dict(window=-1), B.DSA_ERR_SHAPE),
    (dict(sinks=-1), B.DSA_ERR_SHAPE), (dict(sinks=129), B.DSA_ERR_SHAPE),
    (dict(window=64, sinks=129), B.DSA_ERR_SHAPE),
    (dict(q_turned=2), B.DSA_ERR_SHAPE), (dict(q_turned=-1), B.DSA_ERR_SHAPE),
    (dict(scale=0.0), B.DSA_ERR_SHAPE), (dict(scale=float("nan")), B.DSA_ERR_SHAPE),
    (dict(scale=3e38), B.DSA_ERR_SHAPE), (dict(workspace=None), B.DSA_ERR_SCRATCH),
    (dict(workspace=BIG + 8), B.DSA_ERR_SCRATCH),
    (dict(workspace_bytes=B.DSA_PAGED_WORKSPACE_BYTES - 1), B.DSA_ERR_SCRATCH)])
def test_attention_refuses(lib, change, code):
    assert lib.dsa_paged_q4_attn(*{**ATTN, **change}.values()) == code


def test_limits_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                             "include", "dsa.h")).read()
    get = lambda n: int(re.search(rf"#define\s+{n}\s+(\d+)", text).group(1))  # noqa: E731
    assert get("DSA_Q4_ROW_BYTES") == B.Q4_ROW_BYTES == Q.ROW
    assert get("DSA_MAX_SINKS") == B.MAX_SINKS


def test_binding_refuses_tensors_of_another_kind(lib, monkeypatch):
    """Types, strides and shapes are looked at before the library is called."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)    # where CPU tensors are

    def never(*a):
        raise AssertionError("the library was called")

    monkeypatch.setattr(B, "_lib", type("L", (), dict(
        {n: staticmethod(never) for n in ("dsa_qk_norm_rope", "dsa_paged_q4_append",
                                          "dsa_paged_q4_read", "dsa_paged_q4_attn")},
        dsa_strerror=staticmethod(lib.dsa_strerror)))())
    b = Q.make([(2, 20), (1, 5)], 16)
    common = b["new_start"], b["seq_len"], b["page_table"], b["pages"]
    bf16 = torch.bfloat16
    kv, q, work = torch.zeros(3, 512, dtype=bf16), torch.zeros(3, 8, 512, dtype=bf16), torch.zeros(4)

    for bad in (kv.float(), kv[:, :256], torch.zeros(512, 3, dtype=bf16).t(), q):
        with pytest.raises(B.DsaError, match="kv"):
            B.dsa_paged_q4_append(bad, *common)
        with pytest.raises(B.DsaError, match="out"):
            B.dsa_paged_q4_read(*common, bad)
        with pytest.raises(B.DsaError, match="kv"):
            B.dsa_qk_norm_rope(q, bad, *common[:2], q, kv)
        with pytest.raises(B.DsaError, match="kv_out"):
            B.dsa_qk_norm_rope(q, kv, *common[:2], q, bad)
    for bad in (b["pages"].view(torch.int8), b["pages"][..., :376], b["pages"].transpose(0, 1),
                torch.zeros(4, 16, 512, dtype=bf16)):
        with pytest.raises(B.DsaError, match="pages"):
            B.dsa_paged_q4_append(kv, *common[:3], bad)
        with pytest.raises(B.DsaError, match="pages"):
            B.dsa_paged_q4_attn(q, *common[:3], bad, 0, 0, 0.1, work, torch.zeros_like(q))
    for bad in (q[:2], q.float(), torch.zeros(3, 512, 8, dtype=bf16).transpose(1, 2), kv):
        with pytest.raises(B.DsaError, match="out"):
            B.dsa_paged_q4_attn(q, *common, 0, 0, 0.1, work, bad)
        with pytest.raises(B.DsaError, match="q_out"):
            B.dsa_qk_norm_rope(q, kv, *common[:2], bad, kv)
    with pytest.raises(B.DsaError, match="q_weight"):
        B.dsa_qk_norm_rope(q, kv, *common[:2], q, kv, None, torch.zeros(512, dtype=bf16))
    with pytest.raises(B.DsaError, match="kv_weight"):
        B.dsa_qk_norm_rope(q, kv, *common[:2], q, kv, None, None, torch.zeros(64))
    with pytest.raises(B.DsaError, match="new_start"):
        B.dsa_qk_norm_rope(q, kv, b["new_start"][:2], b["seq_len"], q, kv)
    with pytest.raises(B.DsaError, match="cos_sin"):
        B.dsa_qk_norm_rope(q, kv, *common[:2], q, kv, b["cos_sin"].double())
    for window, sinks in ((1 << 31, 0), (-1, 0), (8, 1 << 32), (8, -1)):
        with pytest.raises(B.DsaError, match="window") as e:
            B.dsa_paged_q4_attn(q, *common, window, sinks, 0.1, work, torch.zeros_like(q))
        assert e.value.code == B.DSA_ERR_SHAPE
    with pytest.raises(B.DsaError, match="workspace"):
        B.dsa_paged_q4_attn(q, *common, 0, 0, 0.1, torch.zeros(8, 8).t()[::2], torch.zeros_like(q))
