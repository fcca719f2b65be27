"""The paged append and the paged attention against their float64 forms (paged_ref.py, which
derives the tolerances): lengths from one token on, page and head layouts, windows, rows that
must not be touched or seen, bad tables, streams, graphs and the two run together."""
import math

import numpy as np
import pytest
import torch

import paged_ref as R
from deepseek_v4_sparse_ratio_gb300 import _binding as B

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(512)


@pytest.fixture(scope="module")
def workspace(dsa):
    # NaN everywhere: nothing in it may be read before it is written
    return torch.full((B.DSA_PAGED_WORKSPACE_BYTES // 4,), float("nan"), device="cuda")


def to_gpu(batch):
    return {k: None if v is None else v.cuda() for k, v in batch.items()}


def args(gb):
    return gb["new_start"], gb["seq_len"], gb["page_table"], gb["pages"]


def queries(batch, heads, seed, pad=0):
    n = int(batch["new_start"][-1]) + pad
    return torch.randn(n, heads, 512, generator=torch.Generator().manual_seed(seed)).bfloat16()


def run_attn(batch, q, window, workspace, scale=SCALE, status=None, fill=7.0):
    gb = to_gpu(batch)
    out = torch.full(q.shape, fill, dtype=torch.bfloat16, device="cuda")
    B.dsa_paged_attn(q.cuda(), *args(gb), window, scale, workspace, out, gb["cos_sin"], status)
    torch.cuda.synchronize()
    return out.cpu()


def check_attn(out, batch, q, window, scale=SCALE, fill=7.0):
    ref, tol, written = R.attention(batch, q, window, scale)
    got = out.double()
    assert bool((got[~written] == fill).all()), "a row of no sequence was written"
    if not written.any():
        return
    ref, tol, got = ref[written], tol[written], got[written]
    err = (got - ref).abs()
    worst = (err - tol).max().item()
    assert bool((err <= tol).all()), f"worst excess {worst:.3g} (NaN: {got.isnan().any()})"
    # two independent bf16 roundings (probabilities, output), each at most U / sqrt(3) in the
    # mean square, over many elements; a quarter more for the rest
    if ref.numel() >= 4096:
        rel = (err.norm() / ref.norm()).item()
        assert rel <= 1.25 * math.sqrt(2.0 / 3.0) * R.U, f"relative error {rel:.3g}"


# --------------------------------------------------------------------------- append

APPEND = [  # (sequences (new, total), page size, rope)
    ([(1, 1)], 16, True), ([(1, 17)], 16, True), ([(5, 5), (0, 9), (1, 40), (33, 64)], 16, True),
    ([(130, 300), (1, 256), (2, 257)], 128, True), ([(7, 100), (64, 64)], 32, False),
    ([(1, 10 + i) for i in range(1100)], 16, True), ([(1000, 1025)], 1024, True),
]


@pytest.mark.parametrize("lens,page,rope", APPEND)
def test_append_matches_the_formula(dsa, lens, page, rope):
    batch = R.make(lens, page, rope=rope, seed=len(lens))
    n, pad = int(batch["new_start"][-1]), 3
    kv = torch.randn(n + pad, 512, generator=torch.Generator().manual_seed(5)).bfloat16()
    ref, tol = R.append(batch, kv)
    gb = to_gpu(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_paged_append(kv.cuda(), *args(gb), gb["cos_sin"], status)
    torch.cuda.synchronize()
    got = gb["pages"].cpu().double()
    assert status.item() == 0
    assert bool(((got - ref).abs() <= tol).all())


def test_append_leaves_out_what_cannot_be_and_reports_it(dsa):
    batch = R.make([(3, 20), (2, 40), (4, 30), (1, 16)], 16, seed=3)
    batch["page_table"][0, 1] = batch["pages"].shape[0]   # one past the last page
    batch["page_table"][1, 2] = -5
    batch["seq_len"][2] = 3                               # fewer than its four new tokens
    kv = torch.randn(10, 512, generator=torch.Generator().manual_seed(6)).bfloat16()
    ref, tol = R.append(batch, kv)
    gb = to_gpu(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_paged_append(kv.cuda(), *args(gb), gb["cos_sin"], status)
    torch.cuda.synchronize()
    assert status.item() == B.DSA_ERR_BOUNDS
    assert bool(((gb["pages"].cpu().double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("starts", [[0, 5, 2, 9], [-3, 2, 4, 9], [0, 4, 8, 20], [5, 5, 5, 5]])
def test_bad_starts_write_nothing_of_their_sequences(dsa, workspace, starts):
    batch = R.make([(3, 20), (3, 40), (3, 30)], 16, seed=4)
    batch["new_start"] = torch.tensor(starts, dtype=torch.int32)
    kv = torch.randn(9, 512, generator=torch.Generator().manual_seed(6)).bfloat16()
    gb = to_gpu(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_paged_append(kv.cuda(), *args(gb), gb["cos_sin"], status)
    torch.cuda.synchronize()
    bad = [s for s in range(3) if not R.valid(batch, s, 9)]
    assert status.item() == (B.DSA_ERR_BOUNDS if bad else 0)
    before, after = batch["pages"], gb["pages"].cpu()
    for s in bad:
        used = [e for e in batch["page_table"][s].tolist() if e >= 0]
        assert torch.equal(before[used], after[used])
    q = queries(R.make([(3, 20), (3, 40), (3, 30)], 16), 8, 1)
    status.zero_()
    out = run_attn(batch, q, 0, workspace, status=status)
    assert status.item() == (B.DSA_ERR_BOUNDS if bad else 0)
    rows = np.zeros(9, dtype=bool)
    for s in range(3):
        if s not in bad:
            rows[starts[s]:starts[s + 1]] = True
    assert bool((out[~rows] == 7.0).all())


@pytest.mark.parametrize("at,start", [(20, -1), (20, 500), (31, -5), (1, 40), (64, -2)])
def test_starts_that_decrease_cost_their_own_sequences_alone(dsa, workspace, at, start):
    """65 sequences of a row each, one start out of order: those whose numbers cannot be are
    skipped, all others are served (their rows belong to no other sequence)."""
    batch = R.make([(1, 20 + s) for s in range(65)], 16, seed=30)
    batch["new_start"][at] = start
    ok = [s for s in range(65) if R.valid(batch, s, 65)]
    spans = [tuple(batch["new_start"][s:s + 2].tolist()) for s in ok]
    taken = torch.zeros(66, dtype=torch.int32)
    for a, b in spans:
        taken[a:b] += 1
    assert 2 <= len(ok) < 65 and int(taken.max()) == 1
    kv = torch.randn(65, 512, generator=torch.Generator().manual_seed(6)).bfloat16()
    ref, tol = R.append(batch, kv)
    gb = to_gpu(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_paged_append(kv.cuda(), *args(gb), gb["cos_sin"], status)
    torch.cuda.synchronize()
    assert status.item() == B.DSA_ERR_BOUNDS
    assert bool(((gb["pages"].cpu().double() - ref).abs() <= tol).all())
    q = torch.randn(65, 16, 512, generator=torch.Generator().manual_seed(7)).bfloat16()
    out = run_attn(batch, q, 0, workspace)
    check_attn(out, batch, q, 0)


# --------------------------------------------------------------------------- attention

ATTN = [  # (sequences (new, total), heads, page, window, rope, padded rows)
    ([(1, 1)], 64, 16, 0, True, 0),
    ([(1, 1)], 1, 16, 0, False, 0),
    ([(1, 127), (1, 128), (1, 129), (1, 2)], 64, 64, 0, True, 0),
    ([(1, 300), (0, 50), (3, 3), (2, 257)], 64, 128, 0, True, 2),
    ([(1, 1000)], 128, 256, 0, True, 0),
    ([(1, 5000)], 64, 64, 0, True, 0),
    ([(1, 2100)], 16, 16, 0, True, 0),
    ([(70, 200)], 8, 32, 0, True, 1),
    ([(19, 19), (40, 333)], 5, 16, 0, True, 0),
    ([(9, 140), (130, 130)], 24, 64, 0, False, 0),
    ([(3, 500), (5, 5)], 96, 16, 0, True, 0),
    ([(33, 100)], 48, 1024, 0, True, 0),
    ([(40, 300), (1, 700)], 64, 64, 128, True, 0),
    ([(200, 400)], 16, 16, 1, True, 0),
    ([(150, 150), (1, 600)], 32, 32, 37, True, 0),
    ([(2, 900)], 64, 16, 129, False, 0),
    ([(64, 64), (1, 4096)], 7, 128, 5000, True, 0),
    ([(1, 30 + 7 * i) for i in range(200)], 4, 16, 0, True, 3),
    ([(150, 700)], 64, 64, 0, True, 0),
    # more than 64 heads where most sequences are idle; the same with every one at work
    ([(0, 10), (1, 300), (0, 5), (0, 7)], 128, 64, 0, True, 1),
    ([(0, 10), (0, 300), (1, 500), (0, 7)], 70, 16, 100, True, 0),
    ([(1, 260), (3, 300)], 65, 32, 0, True, 0),
    # a long prompt beside single tokens, on average few rows per sequence
    ([(40, 90)] + [(1, 20 + 30 * i) for i in range(60)], 16, 16, 0, True, 0),
    # units of 128 rows with odd head counts
    ([(120, 120), (200, 333)], 5, 16, 0, True, 2),
    ([(400, 450)], 1, 64, 200, True, 0),
    ([(5, 40), (9, 300)], 127, 32, 0, True, 0),
    # many units of one block per SM: a segment's end follows the one before at once
    ([(100, 100)] * 12 + [(90, 128)], 64, 32, 0, True, 0),
    ([(256, 256)] * 6, 64, 64, 3, True, 0),
    # many short units per SM, cut where a run ends
    ([(700, 900), (1, 33), (350, 350)], 16, 32, 100, True, 1),
    ([(600, 2000)], 64, 64, 128, True, 0),
    ([(900, 1200)], 8, 16, 0, True, 0),
]


@pytest.mark.parametrize("lens,heads,page,window,rope,pad", ATTN)
def test_attention_matches_the_formula(dsa, workspace, lens, heads, page, window, rope, pad):
    batch = R.make(lens, page, rope=rope, seed=heads + page)
    q = queries(batch, heads, 11, pad)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, window, workspace, status=status)
    assert status.item() == 0
    check_attn(out, batch, q, window)


@pytest.mark.parametrize("scale,amp", [(1.0, 1.0), (0.3, 4.0), (SCALE, 1e-3)])
def test_attention_with_sharp_and_flat_logits(dsa, workspace, scale, amp):
    """Logits of hundreds (one key takes all, the maximum rises late) and of nearly zero."""
    batch = R.make([(1, 1500), (40, 300)], 64, seed=2)
    q = (queries(batch, 16, 12).float() * amp).bfloat16()
    out = run_attn(batch, q, 0, workspace, scale=scale)
    ref, tol, _ = R.attention(batch, q, 0, scale)
    assert bool(((out.double() - ref).abs() <= tol).all())


def test_attention_rising_logits_rescale_every_block(dsa, workspace):
    """Keys whose logits grow block by block: the running maximum rises at every block."""
    batch = R.make([(1, 1200), (3, 900)], 64, rope=False, seed=8)
    d = torch.randn(512, generator=torch.Generator().manual_seed(1))
    for s in range(2):
        for p in range(int(batch["seq_len"][s])):
            e, r = R.place(batch, s, p)
            batch["pages"][e, r] = (d * (0.2 + p / 400.0)
                                    + 0.1 * batch["pages"][e, r].float()).bfloat16()
    q = (d[None, None] + 0.1 * queries(batch, 64, 3).float()).bfloat16()
    out = run_attn(batch, q, 0, workspace)
    check_attn(out, batch, q, 0)


@pytest.mark.parametrize("half", [0, 1])
def test_one_half_of_the_rows_rescales_alone(dsa, workspace, half):
    """Logits rise block by block for half of the heads only, in a unit cut into parts of
    several blocks: each half keeps its own running maximum."""
    batch = R.make([(1, 40000)], 64, rope=False, seed=19)
    d = torch.randn(512, generator=torch.Generator().manual_seed(2))
    at = torch.tensor([R.place(batch, 0, p) for p in range(40000)])
    rise = torch.arange(40000)[:, None] / 10000.0
    rows = batch["pages"][at[:, 0], at[:, 1]].float() * 0.2 + d * rise
    batch["pages"][at[:, 0], at[:, 1]] = rows.bfloat16()
    q = queries(batch, 64, 16).float() * 0.05
    q[:, 32 * half:32 * half + 32] += d
    q = q.bfloat16()
    out = run_attn(batch, q, 0, workspace)
    check_attn(out, batch, q, 0)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("heads,window", [(64, 0), (16, 0), (64, 40), (8, 40), (128, 0)])
def test_rows_that_are_not_seen_do_not_touch_the_output(dsa, workspace, junk, heads, window):
    lens = [(5, 150), (1, 131), (20, 60)]
    batch = R.make(lens, 64, seed=9)
    clean = {k: v.clone() for k, v in batch.items()}
    used = torch.zeros(batch["pages"].shape[:2], dtype=torch.bool)
    for s, (n, c) in enumerate(lens):
        for p in range(max(0, c - n - window + 1) if window else 0, c):
            used[R.place(batch, s, p)] = True
    batch["pages"][~used] = junk
    q = queries(batch, heads, 4)
    out = run_attn(batch, q, window, workspace)
    check_attn(out, clean, q, window)


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [8, 16, 64])
def test_a_later_tokens_bad_row_stays_with_the_tokens_that_see_it(dsa, workspace, junk, heads):
    """Token 6 of 12 has a non-finite row: the earlier tokens do not see it, the later do."""
    batch = R.make([(12, 140)], 64, seed=10)
    clean = {k: v.clone() for k, v in batch.items()}
    batch["pages"][R.place(batch, 0, 134)][3::7] = junk
    q = queries(batch, heads, 5)
    out = run_attn(batch, q, 0, workspace)
    ref, tol, _ = R.attention(clean, q, 0, SCALE)
    assert bool(((out[:6].double() - ref[:6]).abs() <= tol[:6]).all())
    assert bool(out[6:].isnan().any(-1).all())


def test_non_finite_queries_stay_in_their_rows(dsa, workspace):
    batch = R.make([(6, 200)], 64, seed=13)
    q = queries(batch, 16, 6)
    clean = q.clone()
    q[2, 5] = float("nan")
    q[4, 0, 17] = float("inf")
    out = run_attn(batch, q, 0, workspace)
    ref, tol, _ = R.attention(batch, clean, 0, SCALE)
    ok = torch.ones(6, 16, dtype=torch.bool)
    ok[2, 5] = ok[4, 0] = False
    assert bool(((out.double() - ref).abs() <= tol)[ok].all())
    assert bool(out[2, 5].isnan().all()) and bool(out[4, 0].isnan().all())


def test_bad_table_entries_are_left_out_and_reported(dsa, workspace):
    batch = R.make([(1, 200), (2, 70), (1, 16), (3, 100)], 16, seed=14)
    n_pages = batch["pages"].shape[0]
    batch["page_table"][0, 3] = n_pages
    batch["page_table"][1, 4] = -1
    batch["page_table"][2, 0] = 2 ** 31 - 1       # the only page: its token sees nothing
    q = queries(batch, 64, 7)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 0, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check_attn(out, batch, q, 0)


def test_entries_below_the_window_or_past_the_end_are_not_read(dsa, workspace):
    batch = R.make([(2, 400), (1, 300)], 16, seed=15, max_pages=64)
    for s, (n, c) in enumerate([(2, 400), (1, 300)]):
        low = c - n - 50 + 1
        batch["page_table"][s, :low // 16] = -7
        batch["page_table"][s, -(-c // 16):] = 2 ** 30
    q = queries(batch, 64, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 50, workspace, status=status)
    assert status.item() == 0
    check_attn(out, batch, q, 50)


def test_a_sequence_longer_than_its_table_or_angles_is_skipped(dsa, workspace):
    batch = R.make([(1, 100), (1, 60), (2, 90)], 16, seed=16)
    batch["cos_sin"] = batch["cos_sin"][:95].contiguous()
    q = queries(batch, 8, 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 0, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check_attn(out, batch, q, 0)          # rows of the first sequence stay as they were


def test_pages_far_apart_pass_32_bit_offsets(dsa, workspace):
    """Pages of one layer in a cache of many: element offsets beyond 2^32."""
    lens = [(3, 150), (1, 64)]
    batch = R.make(lens, 64, extra_pages=0, seed=17)
    n_pages = batch["pages"].shape[0]
    stride = (1 << 32) // (n_pages - 1) // 8 * 8 + 64 * 512
    store = torch.empty(n_pages * stride, dtype=torch.bfloat16, device="cuda")
    pages = store.as_strided((n_pages, 64, 512), (stride, 512, 1))
    pages.copy_(batch["pages"])
    gb = to_gpu(batch)
    q = queries(batch, 64, 10)
    kv = torch.randn(4, 512, generator=torch.Generator().manual_seed(3)).bfloat16()
    B.dsa_paged_append(kv.cuda(), gb["new_start"], gb["seq_len"], gb["page_table"], pages,
                       gb["cos_sin"])
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    B.dsa_paged_attn(q.cuda(), gb["new_start"], gb["seq_len"], gb["page_table"], pages, 0, SCALE,
                     workspace, out, gb["cos_sin"])
    torch.cuda.synchronize()
    ref, tol = R.append(batch, kv)
    got = pages.cpu()
    assert bool(((got.double() - ref).abs() <= tol).all())
    batch["pages"] = got
    check_attn(out.cpu(), batch, q, 0)


def _over_and_over(len_, n_new):
    """A sequence whose table names the same four pages of 1,024 rows over and over."""
    g = torch.Generator().manual_seed(31)
    pages = torch.randn(4, 1024, 512, generator=g).bfloat16()
    table = (torch.arange(-(-len_ // 1024)) % 4).int()[None]
    return dict(pages=pages, page_table=table, cos_sin=None,
                new_start=torch.tensor([0, n_new], dtype=torch.int32),
                seq_len=torch.tensor([len_], dtype=torch.int32))


@pytest.mark.parametrize("n_new,heads", [(1, 64), (3, 128)])
def test_the_longest_sequence(dsa, workspace, n_new, heads):
    """The largest length there is, each key at many positions. Beside the bounds of the module
    for few keys, every fp32 sum is a chain over a CTA's share of the keys (a 152nd, of all units;
    then 152 parts): 2^-24 a step."""
    length = B.MAX_PAGED_TOKENS - 5
    batch = _over_and_over(length, n_new)
    q = torch.randn(n_new, heads, 512, generator=torch.Generator().manual_seed(32)).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 0, workspace, status=status)
    assert status.item() == 0
    kv = batch["pages"].double().view(4096, 512)
    share = 2 * n_new * length / 152 + 152
    for i in range(n_new):
        seen = length - n_new + i + 1
        times = torch.full((4096,), float(seen // 4096), dtype=torch.float64)
        times[:seen % 4096] += 1
        qr = q[i].double()
        logits = SCALE * qr @ kv.T
        w = torch.softmax(logits + times.log(), -1)
        ref, big = w @ kv, w @ kv.abs()
        size = SCALE * (qr.abs() @ kv.abs().T).amax(-1)
        e = 512 * 2.0 ** -23 * size + 2.0 ** -22 * 1.45 * (logits.abs().amax(-1) + 16)
        spread = torch.expm1(2 * e) + 2.02 * R.U + 2.0 ** -20 + 2 * share * 2.0 ** -24
        err = (out[i].double() - ref).abs()
        assert bool((err <= R.U * ref.abs() + big * spread[:, None]).all())


def test_a_sequence_over_the_largest_length_is_skipped(dsa, workspace):
    batch = _over_and_over(B.MAX_PAGED_TOKENS + 1, 1)
    q = torch.randn(1, 64, 512, generator=torch.Generator().manual_seed(33)).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 0, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    assert bool((out == 7.0).all())
    gb = to_gpu(batch)
    status.zero_()
    B.dsa_paged_append(q[:, 0].contiguous().cuda(), *args(gb), None, status)
    torch.cuda.synchronize()
    assert status.item() == B.DSA_ERR_BOUNDS
    assert torch.equal(gb["pages"].cpu(), batch["pages"])


def test_writes_stay_inside_the_buffers(dsa):
    """Canaries around the output, the workspace and the pages."""
    guard = 4096
    lens = [(1, 900), (3, 129), (40, 77)]
    batch = R.make(lens, 32, seed=18)
    gb = to_gpu(batch)
    q = queries(batch, 24, 11)

    def guarded(n, dtype):
        buf = torch.full((n + 2 * guard,), 5, dtype=dtype, device="cuda")
        return buf, buf[guard:guard + n]

    ob, out = guarded(q.numel(), torch.bfloat16)
    wb, work = guarded(B.DSA_PAGED_WORKSPACE_BYTES, torch.uint8)
    pb, pages = guarded(batch["pages"].numel(), torch.bfloat16)
    pages = pages.view(batch["pages"].shape)
    pages.copy_(batch["pages"])
    kv = torch.randn(q.shape[0], 512, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    a = (gb["new_start"], gb["seq_len"], gb["page_table"], pages)
    B.dsa_paged_append(kv, *a, gb["cos_sin"])
    B.dsa_paged_attn(q.cuda(), *a, 0, SCALE, work, out.view(q.shape), gb["cos_sin"])
    torch.cuda.synchronize()
    for buf in (ob, wb, pb):
        assert bool((buf[:guard] == 5).all()) and bool((buf[-guard:] == 5).all())


@pytest.mark.parametrize("off_q,off_out,off_work", [(8, 8, 16), (0, 8, 0), (0, 0, 16), (8, 0, 48)])
@pytest.mark.parametrize("lens", [[(1, 900), (1, 40)], [(300, 700), (40, 40)]])
def test_buffers_on_odd_multiples_of_16_bytes(dsa, lens, off_q, off_out, off_work):
    """Every tensor 16 bytes into its allocation (queries, output: elements; workspace: bytes),
    with single tokens and with chunks, whose units are cut into parts."""
    batch = R.make(lens, 32, seed=34)
    gb = to_gpu(batch)
    q = queries(batch, 32, 19)
    n = q.numel()

    def at(offset, size, dtype, fill):
        buf = torch.full((offset + size + 64,), fill, dtype=dtype, device="cuda")
        return buf, buf[offset:offset + size]

    _, qd = at(off_q, n, torch.bfloat16, 0.0)
    ob, out = at(off_out, n, torch.bfloat16, 7.0)
    wb, work = at(off_work, B.DSA_PAGED_WORKSPACE_BYTES, torch.uint8, 5)
    _, pages = at(8, batch["pages"].numel(), torch.bfloat16, 0.0)
    pages = pages.view(batch["pages"].shape).copy_(batch["pages"])
    assert out.data_ptr() % 32 == 2 * off_out % 32 and pages.data_ptr() % 32 == 16
    qd = qd.view(q.shape).copy_(q)
    B.dsa_paged_attn(qd, gb["new_start"], gb["seq_len"], gb["page_table"], pages, 0, SCALE, work,
                     out.view(q.shape), gb["cos_sin"])
    torch.cuda.synchronize()
    check_attn(out.view(q.shape).cpu(), batch, q, 0)
    assert bool((ob[:off_out] == 7.0).all()) and bool((ob[off_out + n:] == 7.0).all())
    assert bool((wb[:off_work] == 5).all()) and bool((wb[-64:] == 5).all())


@pytest.mark.parametrize("heads", [8, 64])
def test_sequences_that_share_pages(dsa, workspace, heads):
    """A common prefix of whole pages in three sequences, one of them twice in the batch."""
    batch = R.make([(1, 200), (30, 260), (1, 200), (2, 150)], 16, seed=27)
    for s in (1, 2, 3):
        batch["page_table"][s, :8] = batch["page_table"][0, :8]
    batch["page_table"][2] = batch["page_table"][0]
    q = queries(batch, heads, 17)
    out = run_attn(batch, q, 0, workspace)
    check_attn(out, batch, q, 0)


def test_thousands_of_sequences(dsa, workspace):
    lens = [(1 if i % 3 else 0, 1 + i % 40) for i in range(3000)]
    batch = R.make(lens, 16, seed=28)
    q = queries(batch, 2, 18, pad=1)
    out = run_attn(batch, q, 0, workspace)
    check_attn(out, batch, q, 0)


def test_rows_before_the_first_sequence_are_left(dsa, workspace):
    batch = R.make([(3, 20), (2, 40)], 16, seed=29)
    batch["new_start"] = torch.tensor([2, 5, 7], dtype=torch.int32)
    kv = torch.randn(8, 512, generator=torch.Generator().manual_seed(6)).bfloat16()
    ref, tol = R.append(batch, kv)
    gb = to_gpu(batch)
    B.dsa_paged_append(kv.cuda(), *args(gb), gb["cos_sin"])
    torch.cuda.synchronize()
    assert bool(((gb["pages"].cpu().double() - ref).abs() <= tol).all())
    q = torch.randn(8, 16, 512, generator=torch.Generator().manual_seed(7)).bfloat16()
    out = run_attn(batch, q, 0, workspace)
    check_attn(out, batch, q, 0)


# --------------------------------------------------------------------------- how it is used

def _serve(batch, steps, heads, window, workspace, stream=None):
    """Grow every sequence by `steps` (lists of new counts) and check each step's attention."""
    g = torch.Generator().manual_seed(21)
    gb = to_gpu(batch)
    lens = [0] * batch["page_table"].shape[0]
    for new in steps:
        lens = [a + b for a, b in zip(lens, new)]
        n = sum(new)
        batch["seq_len"] = torch.tensor(lens, dtype=torch.int32)
        batch["new_start"] = torch.tensor([0] + new).cumsum(0).int()
        gb["seq_len"], gb["new_start"] = batch["seq_len"].cuda(), batch["new_start"].cuda()
        kv = torch.randn(n, 512, generator=g).bfloat16()
        q = torch.randn(n, heads, 512, generator=g).bfloat16()
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        kd, qd = kv.cuda(), q.cuda()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        B.dsa_paged_append(kd, *args(gb), gb["cos_sin"], stream=stream)
        B.dsa_paged_attn(qd, *args(gb), window, SCALE, workspace, out, gb["cos_sin"],
                         stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        ref, tol = R.append(batch, kv)
        torch.cuda.synchronize()
        got = gb["pages"].cpu()
        assert bool(((got.double() - ref).abs() <= tol).all())
        batch["pages"] = got
        check_attn(out.cpu(), batch, q, window)


@pytest.mark.parametrize("window", [0, 128])
@pytest.mark.parametrize("own_stream", [False, True])
def test_prompts_then_single_tokens(dsa, workspace, window, own_stream):
    """Three users: prompt chunks, then decode steps, then a new prompt beside them."""
    batch = R.make([(0, 400), (0, 400), (0, 400)], 32, seed=20)
    stream = torch.cuda.Stream() if own_stream else None
    _serve(batch, [[100, 33, 0], [50, 1, 0], [1, 1, 0], [1, 4, 70], [1, 1, 1]], 16, window,
           workspace, stream)


def test_window_agrees_with_the_window_sparse_attention(dsa, workspace):
    """The window alone over pages equals the library's window attention over packed rows."""
    T, off = 40, 300
    batch = R.make([(T, off + T)], 64, rope=False, seed=22)
    raw = torch.stack([batch["pages"][R.place(batch, 0, p)] for p in range(off + T)])
    q = queries(batch, 64, 13)
    out = run_attn(batch, q, 128, workspace)
    sel = torch.full((T, 8), -1, dtype=torch.int32, device="cuda")
    ref = torch.empty(T, 64, 512, dtype=torch.bfloat16, device="cuda")
    B.dsa_window_sparse_attn(q.cuda(), raw.cuda(), 0, None, 0, sel, 8, T, off, 4, 128, SCALE, ref)
    torch.cuda.synchronize()
    _, tol, _ = R.attention(batch, q, 128, SCALE)
    assert bool(((out.double() - ref.cpu().double()).abs() <= 2 * tol).all())


def test_captured_step_replays_with_other_lengths(dsa):
    """One graph of append + attention, padded to 12 rows; lengths change between replays.
    Two graphs with a workspace each run at the same time on two streams."""
    batch = R.make([(0, 300), (0, 300), (0, 300)], 16, seed=23)
    g = torch.Generator().manual_seed(24)
    graphs = []
    for _ in range(2):
        gb = to_gpu(batch)
        st = dict(gb=gb, kv=torch.zeros(12, 512, dtype=torch.bfloat16, device="cuda"),
                  q=torch.zeros(12, 64, 512, dtype=torch.bfloat16, device="cuda"),
                  out=torch.zeros(12, 64, 512, dtype=torch.bfloat16, device="cuda"),
                  work=torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"),
                  stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())
        with torch.cuda.graph(st["graph"], stream=st["stream"]):
            B.dsa_paged_append(st["kv"], *args(gb), gb["cos_sin"])
            B.dsa_paged_attn(st["q"], *args(gb), 0, SCALE, st["work"], st["out"], gb["cos_sin"])
        graphs.append(st)
    for new, lens in [([1, 1, 1], [250, 9, 300]), ([0, 10, 2], [0, 10, 200]), ([4, 0, 8], [44, 3, 8])]:
        want = []
        for st in graphs:
            b = {k: v for k, v in batch.items()}
            b["pages"] = st["gb"]["pages"].cpu()
            b["seq_len"] = torch.tensor(lens, dtype=torch.int32)
            b["new_start"] = torch.tensor([0] + new).cumsum(0).int()
            kv = torch.randn(12, 512, generator=g).bfloat16()
            q = torch.randn(12, 64, 512, generator=g).bfloat16()
            st["kv"].copy_(kv)
            st["q"].copy_(q)
            st["out"].fill_(7.0)
            st["gb"]["seq_len"].copy_(b["seq_len"])
            st["gb"]["new_start"].copy_(b["new_start"])
            want.append((b, kv, q))
        torch.cuda.synchronize()
        for st in graphs:
            with torch.cuda.stream(st["stream"]):
                st["graph"].replay()
        torch.cuda.synchronize()
        for st, (b, kv, q) in zip(graphs, want):
            ref, tol = R.append(b, kv)
            got = st["gb"]["pages"].cpu()
            assert bool(((got.double() - ref).abs() <= tol).all())
            b["pages"] = got
            check_attn(st["out"].cpu(), b, q, 0)


def test_calls_on_two_streams_at_once(dsa, workspace):
    """Chunks on one stream and single tokens on another, a workspace each, with nothing between
    them: the bits of the calls made one after the other."""
    work = torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    jobs = []
    for lens, seed, w in (([(300, 900), (200, 200)], 35, workspace), ([(1, 5000), (1, 70)], 36, work)):
        batch = R.make(lens, 64, seed=seed)
        gb, q = to_gpu(batch), queries(batch, 64, seed).cuda()
        want = torch.empty_like(q)
        B.dsa_paged_attn(q, *args(gb), 0, SCALE, w, want, gb["cos_sin"])
        jobs.append((gb, q, w, want, [torch.zeros_like(q) for _ in range(8)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for k in range(8):
        for gb, q, w, want, outs, stream in jobs:
            B.dsa_paged_attn(q, *args(gb), 0, SCALE, w, outs[k], gb["cos_sin"], stream=stream)
    torch.cuda.synchronize()
    for gb, q, w, want, outs, stream in jobs:
        assert all(torch.equal(want, o) for o in outs)


def test_same_call_twice_gives_the_same_bits(dsa, workspace):
    batch = R.make([(1, 3000), (30, 500), (1, 64)], 64, seed=25)
    q = queries(batch, 64, 14)
    a = run_attn(batch, q, 0, workspace)
    for _ in range(3):
        assert torch.equal(a, run_attn(batch, q, 0, workspace))


def test_a_token_gets_the_same_answer_in_any_batch(dsa, workspace):
    """Alone or beside others (where its keys are split differently): within the tolerance."""
    batch = R.make([(2, 700), (1, 900), (64, 64)], 32, seed=26)
    q = queries(batch, 64, 15)
    whole = run_attn(batch, q, 0, workspace)
    _, tol, _ = R.attention(batch, q, 0, SCALE)
    r0 = 0
    for s, n in enumerate([2, 1, 64]):
        one = dict(batch, page_table=batch["page_table"][s:s + 1].contiguous(),
                   seq_len=batch["seq_len"][s:s + 1].contiguous(),
                   new_start=torch.tensor([0, n], dtype=torch.int32))
        alone = run_attn(one, q[r0:r0 + n], 0, workspace)
        d = (alone.double() - whole[r0:r0 + n].double()).abs()
        assert bool((d <= 2 * tol[r0:r0 + n]).all())
        r0 += n
