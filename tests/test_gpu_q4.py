"""The 4-bit paged cache: rows written, read back and attended over, against the float64 forms
(q4_ref.py, which derives the tolerances)."""
import math

import numpy as np
import pytest
import torch

import q4_ref as Q
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


def rows_of(n, seed):
    return torch.randn(n, 512, generator=torch.Generator().manual_seed(seed)).bfloat16()


def run_attn(batch, q, window, sinks, workspace, scale=SCALE, status=None, fill=7.0,
             q_turned=False):
    gb = to_gpu(batch)
    out = torch.full(q.shape, fill, dtype=torch.bfloat16, device="cuda")
    B.dsa_paged_q4_attn(q.cuda(), *args(gb), window, sinks, scale, workspace, out, gb["cos_sin"],
                        q_turned, status)
    torch.cuda.synchronize()
    return out.cpu()


def check_attn(out, batch, q, window, sinks, scale=SCALE, fill=7.0, q_turned=False):
    ref, tol, written = Q.attention(batch, q, window, sinks, scale, q_turned)
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
        assert rel <= 1.25 * math.sqrt(2.0 / 3.0) * Q.U, f"relative error {rel:.3g}"


def check_pages(got, ref, tol):
    """All bytes but the rotated dims are equal; those are bf16 values within tol."""
    assert torch.equal(got[..., :256], ref[..., :256])
    a, b = (x[..., 256:].contiguous().view(torch.bfloat16).double() for x in (got, ref))
    same = (got[..., 256:] == ref[..., 256:]).view(*got.shape[:-1], -1, 2).all(-1)
    assert bool((same | ((a - b).abs() <= tol)).all())


# --------------------------------------------------------------------------- append and read

ROWS = [  # (sequences (new, total), page size, rope)
    ([(1, 1)], 16, True), ([(1, 17)], 16, True), ([(5, 5), (0, 9), (1, 40), (33, 64)], 16, True),
    ([(130, 300), (1, 256), (2, 257)], 128, True), ([(7, 100), (64, 64)], 32, False),
    ([(1, 10 + i) for i in range(300)], 16, True), ([(200, 1025)], 1024, True),
]


@pytest.mark.parametrize("lens,page,rope", ROWS)
def test_append_and_read_match_the_formula(dsa, lens, page, rope):
    batch = Q.make(lens, page, rope=rope, seed=len(lens))
    n, pad = int(batch["new_start"][-1]), 3
    kv = rows_of(n + pad, 5)
    # rows of all sizes, small and large groups, ties, zeros
    g = torch.Generator().manual_seed(6)
    kv *= torch.exp2(torch.randint(-20, 20, (n + pad, 1), generator=g)).bfloat16()
    kv[::3, :64] *= 2.0 ** -15
    kv[::5, 64:128] = 0
    kv[1::4, :16] = torch.tensor([7, 3.5, 2.5, -1.5, .5, -.5, 1, 2, 3, 4, 5, 6, 6.5, -6.5, -7,
                                  0.]).bfloat16()
    ref, tol = Q.append(batch, kv)
    gb = to_gpu(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_paged_q4_append(kv.cuda(), *args(gb), gb["cos_sin"], status)
    out = torch.full((n + pad, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    back = out.clone()
    B.dsa_paged_q4_read(*args(gb), out, None, status)
    B.dsa_paged_q4_read(*args(gb), back, gb["cos_sin"], status)
    torch.cuda.synchronize()
    assert status.item() == 0
    check_pages(gb["pages"].cpu(), ref, tol)
    values = Q.unpack(gb["pages"].cpu())
    out, back = out.cpu(), back.cpu()
    assert bool((out[n:] == 7.0).all()) and bool((back[n:] == 7.0).all())
    r = 0
    for s, (new, total) in enumerate(lens):
        for p in range(total - new, total):
            v = values[Q.place(batch, s, p)]
            assert torch.equal(out[r].double(), v)
            if rope:
                pair = v[448:].abs().view(-1, 2).sum(-1).repeat_interleave(2)
                w = Q.turn(v, batch["cos_sin"][p], -1.0)
                err = (back[r].double() - w).abs()
                assert not err[:448].any()
                assert bool((err[448:] <= Q.U * w[448:].abs() + 4 * 2.0 ** -24 * pair).all())
            r += 1


@pytest.mark.parametrize("top", [-133, -126, -118, -113, -112, -100, 0, 60, 120, 123])
def test_rows_of_every_size(dsa, top):
    """Elements from bf16's smallest to 2^124."""
    batch = Q.make([(40, 40)], 16, rope=False, seed=1)
    g = torch.Generator().manual_seed(top + 200)
    x = torch.rand(40, 512, generator=g).double() + 1.0
    x *= torch.exp2(top - torch.randint(0, 20, (40, 512), generator=g)).double()
    kv = (x * torch.where(torch.rand(40, 512, generator=g) < 0.5, -1.0, 1.0)).bfloat16()
    kv = kv.clamp(-2.0 ** 124 * (1 - 2.0 ** -8), 2.0 ** 124 * (1 - 2.0 ** -8))
    ref, tol = Q.append(batch, kv)
    gb = to_gpu(batch)
    B.dsa_paged_q4_append(kv.cuda(), *args(gb))
    out = torch.empty(40, 512, dtype=torch.bfloat16, device="cuda")
    B.dsa_paged_q4_read(*args(gb), out)
    torch.cuda.synchronize()
    check_pages(gb["pages"].cpu(), ref, tol)
    want = torch.stack([Q.decode(ref[Q.place(batch, 0, p)]) for p in range(40)])
    assert torch.equal(out.cpu().double(), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 2.0 ** 124, 3e38])
def test_odd_elements_spoil_their_group_alone(dsa, bad):
    batch = Q.make([(6, 6)], 16, rope=False, seed=1)
    kv = rows_of(6, 8)
    kv[1, 40], kv[3, 0], kv[3, 447], kv[4, :448], kv[5, 500] = bad, bad, -bad, bad, bad
    ref, tol = Q.append(batch, kv)
    gb = to_gpu(batch)
    B.dsa_paged_q4_append(kv.cuda(), *args(gb))
    out = torch.empty(6, 512, dtype=torch.bfloat16, device="cuda")
    B.dsa_paged_q4_read(*args(gb), out)
    torch.cuda.synchronize()
    got = gb["pages"].cpu()
    check_pages(got, ref, tol)
    out = out.cpu()
    assert torch.equal(out[:, 448:].view(torch.int16), kv[:, 448:].view(torch.int16))
    for i in range(6):
        want = Q.decode(ref[Q.place(batch, 0, i)])[:448]
        assert torch.equal(out[i, :448].double().nan_to_num(12345.0), want.nan_to_num(12345.0))
    assert bool(out[1, 32:48].isnan().all()) and bool(out[4, :448].isnan().all())


def test_what_cannot_be_is_left_out_and_reported(dsa):
    batch = Q.make([(3, 20), (2, 40), (4, 30), (1, 16)], 16, seed=3)
    batch["page_table"][0, 1] = batch["pages"].shape[0]   # one past the last page
    batch["page_table"][1, 2] = -5
    batch["seq_len"][2] = 3                               # fewer than its four new tokens
    kv = rows_of(10, 6)
    ref, tol = Q.append(batch, kv)
    gb = to_gpu(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_paged_q4_append(kv.cuda(), *args(gb), gb["cos_sin"], status)
    torch.cuda.synchronize()
    assert status.item() == B.DSA_ERR_BOUNDS
    check_pages(gb["pages"].cpu(), ref, tol)
    status.zero_()
    out = torch.full((10, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    B.dsa_paged_q4_read(*args(gb), out, None, status)
    torch.cuda.synchronize()
    assert status.item() == B.DSA_ERR_BOUNDS
    rows = [(s, p) for s, (n, c) in enumerate([(3, 20), (2, 40), (4, 30), (1, 16)])
            for p in range(c - n, c)]
    for r, (s, p) in enumerate(rows):
        at = Q.place(batch, s, p) if s != 2 else None
        want = torch.full((512,), 7.0).double() if at is None else Q.decode(gb["pages"][at].cpu())
        assert torch.equal(out[r].cpu().double(), want)


@pytest.mark.parametrize("starts", [[0, 5, 2, 9], [-3, 2, 4, 9], [0, 4, 8, 20], [5, 5, 5, 5],
                                    [2, 5, 7, 8]])
def test_odd_starts_touch_nothing_of_their_sequences(dsa, workspace, starts):
    batch = Q.make([(3, 20), (3, 40), (3, 30)], 16, seed=4)
    batch["new_start"] = torch.tensor(starts, dtype=torch.int32)
    kv = rows_of(9, 6)
    ref, tol = Q.append(batch, kv)
    gb = to_gpu(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((9, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    code = B.DSA_OK if all(Q.valid(batch, s, 9) for s in range(3)) else B.DSA_ERR_BOUNDS
    q = torch.randn(9, 8, 512, generator=torch.Generator().manual_seed(1)).bfloat16()
    B.dsa_paged_q4_append(kv.cuda(), *args(gb), gb["cos_sin"], status)
    torch.cuda.synchronize()
    assert status.item() == code
    # (a row that decreasing starts give to two sequences may go to either)
    got, claims = gb["pages"].cpu(), [[] for _ in range(9)]
    for s in range(3):
        if Q.valid(batch, s, 9):
            for r in range(starts[s], starts[s + 1]):
                claims[r].append(Q.place(batch, s, int(batch["seq_len"][s]) - starts[s + 1] + r))
    for places in claims:
        done = [at for at in places if torch.equal(got[at][:256], ref[at][:256])]
        assert bool(done) or not places
        for at in places:
            if at not in done:
                ref[at] = batch["pages"][at]
    check_pages(got, ref, tol)
    status.zero_()
    B.dsa_paged_q4_read(*args(gb), out, None, status)
    torch.cuda.synchronize()
    assert status.item() == code
    taken = torch.zeros(9, dtype=torch.bool)
    for s in range(3):
        if Q.valid(batch, s, 9):
            taken[starts[s]:starts[s + 1]] = True
    assert bool((out.cpu()[~taken] == 7.0).all()) and not bool((out.cpu()[taken] == 7.0).all(-1).any())
    status.zero_()
    got = run_attn(batch, q, 0, 0, workspace, status=status)
    assert status.item() == code
    assert bool((got[~taken] == 7.0).all())


# --------------------------------------------------------------------------- attention

ATTN = [  # (sequences (new, total), heads, page, window, sinks, rope, padded rows)
    ([(1, 1)], 64, 16, 0, 0, True, 0),
    ([(1, 1)], 1, 16, 0, 0, False, 0),
    ([(1, 127), (1, 128), (1, 129), (1, 2)], 64, 64, 0, 0, True, 0),
    ([(1, 300), (0, 50), (3, 3), (2, 257)], 64, 128, 0, 0, True, 2),
    ([(1, 1000)], 128, 256, 0, 0, True, 0),
    ([(1, 5000)], 64, 64, 0, 0, True, 0),
    ([(1, 2100)], 16, 16, 0, 0, True, 0),
    ([(70, 200)], 8, 32, 0, 0, True, 1),
    ([(19, 19), (40, 333)], 5, 16, 0, 0, True, 0),
    ([(9, 140), (130, 130)], 24, 64, 0, 0, False, 0),
    ([(3, 500), (5, 5)], 96, 16, 0, 0, True, 0),
    ([(33, 100)], 48, 1024, 0, 0, True, 0),
    ([(40, 300), (1, 700)], 64, 64, 128, 0, True, 0),
    ([(200, 400)], 16, 16, 1, 0, True, 0),
    ([(150, 150), (1, 600)], 32, 32, 37, 0, True, 0),
    ([(2, 900)], 64, 16, 129, 0, False, 0),
    ([(64, 64), (1, 4096)], 7, 128, 5000, 4, True, 0),
    ([(1, 30 + 7 * i) for i in range(200)], 4, 16, 0, 0, True, 3),
    ([(150, 700)], 64, 64, 0, 0, True, 0),
    ([(0, 10), (1, 300), (0, 5), (0, 7)], 128, 64, 0, 0, True, 1),
    ([(1, 260), (3, 300)], 65, 32, 0, 0, True, 0),
    ([(40, 90)] + [(1, 20 + 30 * i) for i in range(60)], 16, 16, 0, 0, True, 0),
    # a window and the first tokens
    ([(1, 1)], 64, 16, 1, 128, True, 0),
    ([(1, 2), (1, 5), (3, 6)], 64, 16, 1, 1, True, 0),
    ([(1, 700), (1, 128), (1, 129), (1, 257), (1, 40)], 64, 16, 64, 4, True, 1),
    ([(40, 300), (1, 700), (200, 200)], 64, 64, 128, 4, True, 0),
    ([(200, 400)], 16, 16, 1, 1, True, 0),
    ([(150, 150), (1, 600), (9, 1000)], 32, 32, 37, 128, True, 0),
    ([(300, 300)], 64, 64, 100, 100, True, 0),
    ([(2, 900), (2, 130)], 128, 16, 129, 127, False, 0),
    ([(1, 1500)], 64, 128, 300, 16, True, 0),
    ([(500, 900)], 8, 16, 200, 17, True, 0),
    ([(1, 200 + 5 * i) for i in range(180)], 64, 32, 70, 3, True, 2),
    ([(0, 10), (0, 300), (1, 500), (0, 7)], 70, 16, 100, 9, True, 0),
    # many units of few blocks per SM
    ([(100, 100)] * 12 + [(90, 128)], 64, 32, 0, 0, True, 0),
    ([(256, 256)] * 6, 64, 64, 3, 2, True, 0),
    ([(700, 900), (1, 33), (350, 350)], 16, 32, 100, 5, True, 1),
    ([(600, 2000)], 64, 64, 128, 4, True, 0),
]


@pytest.mark.parametrize("lens,heads,page,window,sinks,rope,pad", ATTN)
def test_attention_matches_the_formula(dsa, workspace, lens, heads, page, window, sinks, rope, pad):
    batch = Q.make(lens, page, rope=rope, seed=heads + page)
    q = queries(batch, heads, 11, pad)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, window, sinks, workspace, status=status)
    assert status.item() == 0
    check_attn(out, batch, q, window, sinks)


@pytest.mark.parametrize("heads,window", [(64, 0), (5, 40)])
def test_queries_that_come_turned(dsa, workspace, heads, window):
    batch = Q.make([(20, 150), (1, 400)], 32, seed=7)
    q = queries(batch, heads, 5)
    out = run_attn(batch, q, window, 4, workspace, q_turned=True)
    check_attn(out, batch, q, window, 4, q_turned=True)
    # without angles nothing is turned, whatever q_turned says
    batch["cos_sin"] = None
    a, b = (run_attn(batch, q, window, 4, workspace, q_turned=t) for t in (False, True))
    assert torch.equal(a, b)


def test_sinks_without_a_window_mean_nothing(dsa, workspace):
    batch = Q.make([(3, 300)], 32, seed=7)
    q = queries(batch, 16, 5)
    assert torch.equal(run_attn(batch, q, 0, 0, workspace), run_attn(batch, q, 0, 128, workspace))


@pytest.mark.parametrize("scale,amp", [(1.0, 1.0), (0.3, 4.0), (SCALE, 1e-3)])
def test_attention_with_sharp_and_flat_logits(dsa, workspace, scale, amp):
    """Logits of hundreds (one key takes all, the maximum rises late) and of nearly zero."""
    batch = Q.make([(1, 1500), (40, 300)], 64, seed=2)
    q = (queries(batch, 16, 12).float() * amp).bfloat16()
    out = run_attn(batch, q, 0, 0, workspace, scale=scale)
    ref, tol, _ = Q.attention(batch, q, 0, 0, scale)
    assert bool(((out.double() - ref).abs() <= tol).all())


def test_attention_rising_logits_rescale_every_block(dsa, workspace):
    """Keys whose logits grow block by block: the running maximum rises at every block."""
    batch = Q.make([(1, 1200), (3, 900)], 64, rope=False, seed=8)
    d = torch.randn(512, generator=torch.Generator().manual_seed(1))
    for s in range(2):
        p = torch.arange(int(batch["seq_len"][s]))
        at = torch.tensor([Q.place(batch, s, int(x)) for x in p])
        noise = rows_of(len(p), 40 + s).float()
        batch["pages"][at[:, 0], at[:, 1]] = Q.pack(
            (d * (0.2 + p / 400.0)[:, None] + 0.1 * noise).bfloat16())
    q = (d[None, None] + 0.1 * queries(batch, 64, 3).float()).bfloat16()
    out = run_attn(batch, q, 0, 0, workspace)
    check_attn(out, batch, q, 0, 0)


@pytest.mark.parametrize("half", [0, 1])
def test_one_half_of_the_rows_rescales_alone(dsa, workspace, half):
    """Logits rise block by block for half of the heads only."""
    n = 20000
    batch = Q.make([(1, n)], 64, rope=False, seed=19)
    d = torch.randn(512, generator=torch.Generator().manual_seed(2))
    at = torch.tensor([Q.place(batch, 0, p) for p in range(n)])
    rise = torch.arange(n)[:, None] / 5000.0
    batch["pages"][at[:, 0], at[:, 1]] = Q.pack((rows_of(n, 3).float() * 0.2 + d * rise).bfloat16())
    q = queries(batch, 64, 16).float() * 0.05
    q[:, 32 * half:32 * half + 32] += d
    q = q.bfloat16()
    out = run_attn(batch, q, 0, 0, workspace)
    check_attn(out, batch, q, 0, 0)


@pytest.mark.parametrize("rows", ["tiny", "huge", "mixed"])
def test_rows_of_other_sizes(dsa, workspace, rows):
    """Rows of 2^-60, of 2^60, and of sizes that differ from row to row and group to group."""
    batch = Q.make([(2, 300), (1, 90)], 16, seed=21)
    g = torch.Generator().manual_seed(22)
    shape = batch["pages"].shape[:2]
    x = torch.randn(*shape, 512, generator=g)
    if rows == "mixed":
        x *= torch.exp2(torch.randint(-8, 3, (*shape, 1), generator=g))
        x[..., :448] *= torch.exp2(torch.randint(-12, 1, (*shape, 28, 1), generator=g)).expand(
            *shape, 28, 16).reshape(*shape, 448)
        scale, amp = SCALE, 1.0
    else:
        x *= 2.0 ** (60 if rows == "huge" else -60)
        scale, amp = SCALE, 2.0 ** (-60 if rows == "huge" else 60)
    batch["pages"] = Q.pack(x.bfloat16())
    q = (queries(batch, 64, 4).float() * amp).bfloat16()
    out = run_attn(batch, q, 0, 0, workspace, scale=scale)
    check_attn(out, batch, q, 0, 0, scale=scale)


@pytest.mark.parametrize("junk", [0xFF, 0x7F, 0x00, 0xA5])
@pytest.mark.parametrize("heads,window,sinks", [(64, 0, 0), (16, 0, 0), (64, 40, 3), (8, 40, 0),
                                                (128, 20, 20), (128, 0, 0)])
def test_rows_that_are_not_seen_do_not_touch_the_output(dsa, workspace, junk, heads, window, sinks):
    """Rows past a sequence's end, between the first tokens and the window, of other pages: bytes
    of any value (scales and bf16 of NaN among them)."""
    lens = [(5, 350), (1, 131), (20, 60), (1, 300)]
    batch = Q.make(lens, 64, seed=9)
    clean = {k: v.clone() for k, v in batch.items()}
    used = torch.zeros(batch["pages"].shape[:2], dtype=torch.bool)
    for s, (n, c) in enumerate(lens):
        for t in range(c - n, c):
            for p in Q.visible(t, window, sinks):
                used[Q.place(batch, s, p)] = True
    batch["pages"][~used] = junk
    q = queries(batch, heads, 4)
    out = run_attn(batch, q, window, sinks, workspace)
    check_attn(out, clean, q, window, sinks)


@pytest.mark.parametrize("where", ["scale", "rope", "inf"])
@pytest.mark.parametrize("heads", [8, 16, 64])
def test_a_later_tokens_bad_row_stays_with_the_tokens_that_see_it(dsa, workspace, where, heads):
    """Token 6 of 12 has a non-finite row: the earlier tokens do not see it, the later do."""
    batch = Q.make([(12, 140)], 64, seed=10)
    clean = {k: v.clone() for k, v in batch.items()}
    row = batch["pages"][Q.place(batch, 0, 134)]
    if where == "scale":
        row[3] = 0x7F
    else:
        row[300:302] = torch.tensor([0xC0 if where == "rope" else 0x80, 0x7F], dtype=torch.uint8)
    q = queries(batch, heads, 5)
    out = run_attn(batch, q, 0, 0, workspace)
    ref, tol, _ = Q.attention(clean, q, 0, 0, SCALE)
    assert bool(((out[:6].double() - ref[:6]).abs() <= tol[:6]).all())
    if where != "inf":     # (an infinity with a logit of -inf gives its key no weight)
        assert bool(out[6:].isnan().any(-1).all())


def test_a_bad_row_between_sinks_and_window_touches_no_one(dsa, workspace):
    """Six tokens of a window of 30 with four sinks, in one unit of work; rows that only some of
    them see are NaN for the others' sake too."""
    batch = Q.make([(6, 200)], 64, seed=11)
    clean = {k: v.clone() for k, v in batch.items()}
    for p in (4, 50, 100, 164):               # (164 is just before the first token's window)
        batch["pages"][Q.place(batch, 0, p)] = 0xFF
    batch["pages"][Q.place(batch, 0, 166)] = 0xFF      # seen by the first two tokens alone
    q = queries(batch, 8, 5)
    out = run_attn(batch, q, 30, 4, workspace)
    ref, tol, _ = Q.attention(clean, q, 30, 4, SCALE)
    assert bool(((out[2:].double() - ref[2:]).abs() <= tol[2:]).all())
    assert bool(out[:2].isnan().any(-1).all())


def test_non_finite_queries_stay_in_their_rows(dsa, workspace):
    batch = Q.make([(6, 200)], 64, seed=13)
    q = queries(batch, 16, 6)
    clean = q.clone()
    q[2, 5] = float("nan")
    q[4, 0, 17] = float("inf")
    out = run_attn(batch, q, 0, 0, workspace)
    ref, tol, _ = Q.attention(batch, clean, 0, 0, SCALE)
    ok = torch.ones(6, 16, dtype=torch.bool)
    ok[2, 5] = ok[4, 0] = False
    assert bool(((out.double() - ref).abs() <= tol)[ok].all())
    assert bool(out[2, 5].isnan().all()) and bool(out[4, 0].isnan().all())


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 8)])
def test_bad_table_entries_are_left_out_and_reported(dsa, workspace, window, sinks):
    batch = Q.make([(1, 200), (2, 70), (1, 16), (3, 100)], 16, seed=14)
    n_pages = batch["pages"].shape[0]
    batch["page_table"][0, 11] = n_pages
    batch["page_table"][1, 4] = -1
    batch["page_table"][2, 0] = 2 ** 31 - 1       # the only page: its token sees nothing
    batch["page_table"][3, 0] = -9                # the first tokens of the last sequence
    q = queries(batch, 64, 7)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, window, sinks, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check_attn(out, batch, q, window, sinks)


@pytest.mark.parametrize("sinks", [0, 5, 40])
def test_entries_that_no_token_needs_are_not_read(dsa, workspace, sinks):
    batch = Q.make([(2, 400), (1, 300)], 16, seed=15, max_pages=64)
    for s, (n, c) in enumerate([(2, 400), (1, 300)]):
        low = c - n - 50 + 1
        batch["page_table"][s, -(-sinks // 16):low // 16] = -7
        batch["page_table"][s, -(-c // 16):] = 2 ** 30
    q = queries(batch, 64, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 50, sinks, workspace, status=status)
    assert status.item() == 0
    check_attn(out, batch, q, 50, sinks)


def test_a_sequence_longer_than_its_table_or_angles_is_skipped(dsa, workspace):
    batch = Q.make([(1, 100), (1, 60), (2, 90)], 16, seed=16)
    batch["cos_sin"] = batch["cos_sin"][:95].contiguous()
    q = queries(batch, 8, 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 0, 0, workspace, status=status)
    assert status.item() == B.DSA_ERR_BOUNDS
    check_attn(out, batch, q, 0, 0)


def test_pages_far_apart_pass_32_bit_offsets(dsa, workspace):
    """Pages of one layer in a cache of many: byte offsets beyond 2^33."""
    lens = [(3, 150), (1, 64)]
    batch = Q.make(lens, 64, extra_pages=0, seed=17)
    n_pages = batch["pages"].shape[0]
    stride = (1 << 33) // (n_pages - 1) // 32 * 32 + 64 * 384
    store = torch.empty(n_pages * stride, dtype=torch.uint8, device="cuda")
    pages = store.as_strided((n_pages, 64, 384), (stride, 384, 1))
    pages.copy_(batch["pages"])
    gb = to_gpu(batch)
    q, kv = queries(batch, 64, 10), rows_of(4, 3)
    a = gb["new_start"], gb["seq_len"], gb["page_table"], pages
    B.dsa_paged_q4_append(kv.cuda(), *a, gb["cos_sin"])
    out, rows = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in (q.shape, kv.shape))
    B.dsa_paged_q4_read(*a, rows)
    B.dsa_paged_q4_attn(q.cuda(), *a, 0, 0, SCALE, workspace, out, gb["cos_sin"])
    torch.cuda.synchronize()
    ref, tol = Q.append(batch, kv)
    got = pages.cpu()
    check_pages(got, ref, tol)
    batch["pages"] = got
    check_attn(out.cpu(), batch, q, 0, 0)
    assert torch.equal(rows[3].cpu().double(), Q.decode(got[Q.place(batch, 1, 63)]))


def test_writes_stay_inside_the_buffers(dsa):
    """Canaries around the outputs, the workspace and the pages, each 16 bytes off 32 (the pages 32
    off 64)."""
    batch = Q.make([(1, 900), (3, 129), (40, 77)], 32, seed=18)
    gb = to_gpu(batch)
    q = queries(batch, 24, 11)

    def guarded(shape, dtype, guard=4096 + 16):
        n = math.prod(shape) * dtype.itemsize
        buf = torch.full((n + 2 * guard,), 5, dtype=torch.uint8, device="cuda")
        return buf, buf[guard:guard + n].view(dtype).view(shape)

    ob, out = guarded(q.shape, torch.bfloat16)
    rb, rows = guarded((q.shape[0], 512), torch.bfloat16)
    wb, work = guarded((B.DSA_PAGED_WORKSPACE_BYTES,), torch.uint8)
    pb, pages = guarded(batch["pages"].shape, torch.uint8, 4096 + 32)
    kb, kv = guarded((q.shape[0], 512), torch.bfloat16)
    qb, qd = guarded(q.shape, torch.bfloat16)
    qd.copy_(q)
    pages.copy_(batch["pages"])
    kv.copy_(rows_of(q.shape[0], 4))
    a = (gb["new_start"], gb["seq_len"], gb["page_table"], pages)
    B.dsa_paged_q4_append(kv, *a, gb["cos_sin"])
    B.dsa_paged_q4_read(*a, rows)
    B.dsa_paged_q4_attn(qd, *a, 0, 0, SCALE, work, out, gb["cos_sin"])
    torch.cuda.synchronize()
    for buf in (ob, rb, wb, pb, kb, qb):
        assert bool((buf[:4112] == 5).all()) and bool((buf[-4112:] == 5).all())
    ref, tol = Q.append(batch, kv.cpu())
    check_pages(pages.cpu(), ref, tol)
    batch["pages"] = pages.cpu()
    check_attn(out.cpu(), batch, q, 0, 0)


@pytest.mark.parametrize("heads", [8, 64])
def test_sequences_that_share_pages(dsa, workspace, heads):
    """A common prefix of whole pages in three sequences, one of them twice in the batch."""
    batch = Q.make([(1, 200), (30, 260), (1, 200), (2, 150)], 16, seed=27)
    for s in (1, 2, 3):
        batch["page_table"][s, :8] = batch["page_table"][0, :8]
    batch["page_table"][2] = batch["page_table"][0]
    q = queries(batch, heads, 17)
    out = run_attn(batch, q, 0, 0, workspace)
    check_attn(out, batch, q, 0, 0)


def test_thousands_of_sequences(dsa, workspace):
    lens = [(1 if i % 3 else 0, 1 + i % 40) for i in range(3000)]
    batch = Q.make(lens, 16, seed=28)
    q = queries(batch, 2, 18, pad=1)
    out = run_attn(batch, q, 20, 3, workspace)
    check_attn(out, batch, q, 20, 3)


# --------------------------------------------------------------------------- how it is used

@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
@pytest.mark.parametrize("own_stream", [False, True])
def test_a_layer_step_by_step(dsa, workspace, window, sinks, own_stream):
    """Norm with rotation, append in 4 bits, attention over the pages and rows read back, for
    prompts and single tokens of three users; each step against float64."""
    batch = Q.make([(0, 400), (0, 400), (0, 400)], 32, seed=20)
    g = torch.Generator().manual_seed(21)
    gb = to_gpu(batch)
    lens, heads = [0] * 3, 16
    wk = 1 + 0.2 * torch.randn(512, generator=g)
    wd = wk.cuda()
    stream = torch.cuda.Stream() if own_stream else None
    for new in [[100, 33, 0], [50, 1, 0], [1, 1, 0], [1, 4, 70], [1, 1, 1]]:
        lens = [a + b for a, b in zip(lens, new)]
        n = sum(new)
        batch["seq_len"] = torch.tensor(lens, dtype=torch.int32)
        batch["new_start"] = torch.tensor([0] + new).cumsum(0).int()
        gb["seq_len"], gb["new_start"] = batch["seq_len"].cuda(), batch["new_start"].cuda()
        kv = (3 * torch.randn(n, 512, generator=g)).bfloat16()
        q = (3 * torch.randn(n, heads, 512, generator=g)).bfloat16()
        kd, qd = kv.cuda(), q.cuda()
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        rows = torch.full(kv.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kw = dict(stream=stream)
        B.dsa_qk_norm_rope(qd, kd, gb["new_start"], gb["seq_len"], qd, kd, gb["cos_sin"], None, wd,
                           **kw)
        B.dsa_paged_q4_append(kd, *args(gb), **kw)
        B.dsa_paged_q4_attn(qd, *args(gb), window, sinks, SCALE, workspace, out, gb["cos_sin"],
                            True, **kw)
        B.dsa_paged_q4_read(*args(gb), rows, **kw)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        qn, kn = qd.cpu(), kd.cpu()
        r = 0
        for s in range(3):
            for p in range(lens[s] - new[s], lens[s]):
                for x, w, y in ((q[r], None, qn[r]), (kv[r], wk, kn[r])):
                    ref, tol = Q.norm(x, w, 1e-6, batch["cos_sin"][p])
                    assert bool(((y.double() - ref).abs() <= tol).all())
                r += 1
        ref, tol = Q.append(dict(batch, cos_sin=None), kn)      # the rows as the norm gave them
        got = gb["pages"].cpu()
        assert torch.equal(got, ref)
        batch["pages"] = got
        check_attn(out.cpu(), batch, qn, window, sinks, q_turned=True)
        r = 0
        for s in range(3):
            for p in range(lens[s] - new[s], lens[s]):
                assert torch.equal(rows[r].cpu().double(), Q.decode(got[Q.place(batch, s, p)]))
                r += 1


def test_rows_read_back_serve_the_window_sparse_attention(dsa, workspace):
    """The rows of a chunk and the window before it, read back, in the library's window attention:
    the same as the attention over the 4-bit pages with that window."""
    T, off, window = 40, 300, 128
    batch = Q.make([(T, off + T)], 64, rope=False, seed=22)
    gb = to_gpu(batch)
    first = off - window + 1
    raw = torch.empty(off + T - first, 512, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, raw.shape[0]], dtype=torch.int32, device="cuda")
    B.dsa_paged_q4_read(start, gb["seq_len"], gb["page_table"], gb["pages"], raw)
    q = queries(batch, 64, 13)
    out = run_attn(batch, q, window, 0, workspace)
    sel = torch.full((T, 8), -1, dtype=torch.int32, device="cuda")
    ref = torch.empty(T, 64, 512, dtype=torch.bfloat16, device="cuda")
    B.dsa_window_sparse_attn(q.cuda(), raw, first, None, 0, sel, 8, T, off, 4, window, SCALE, ref)
    torch.cuda.synchronize()
    _, tol, _ = Q.attention(batch, q, window, 0, SCALE)
    assert bool(((out.double() - ref.cpu().double()).abs() <= 2 * tol).all())


def test_captured_step_replays_with_other_lengths(dsa):
    """One graph of append + attention + read, padded to 12 rows; lengths change between replays.
    Two graphs with a workspace each run at the same time on two streams."""
    batch = Q.make([(0, 300), (0, 300), (0, 300)], 16, seed=23)
    g = torch.Generator().manual_seed(24)
    graphs = []
    for _ in range(2):
        gb = to_gpu(batch)
        st = dict(gb=gb, kv=torch.zeros(12, 512, dtype=torch.bfloat16, device="cuda"),
                  q=torch.zeros(12, 64, 512, dtype=torch.bfloat16, device="cuda"),
                  out=torch.zeros(12, 64, 512, dtype=torch.bfloat16, device="cuda"),
                  rows=torch.zeros(12, 512, dtype=torch.bfloat16, device="cuda"),
                  work=torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"),
                  stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())
        with torch.cuda.graph(st["graph"], stream=st["stream"]):
            B.dsa_paged_q4_append(st["kv"], *args(gb), gb["cos_sin"])
            B.dsa_paged_q4_attn(st["q"], *args(gb), 90, 4, SCALE, st["work"], st["out"],
                                gb["cos_sin"])
            B.dsa_paged_q4_read(*args(gb), st["rows"])
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
            st["rows"].fill_(7.0)
            st["gb"]["seq_len"].copy_(b["seq_len"])
            st["gb"]["new_start"].copy_(b["new_start"])
            want.append((b, kv, q))
        torch.cuda.synchronize()
        for st in graphs:
            with torch.cuda.stream(st["stream"]):
                st["graph"].replay()
        torch.cuda.synchronize()
        for st, (b, kv, q) in zip(graphs, want):
            ref, tol = Q.append(b, kv)
            got = st["gb"]["pages"].cpu()
            check_pages(got, ref, tol)
            b["pages"] = got
            check_attn(st["out"].cpu(), b, q, 90, 4)
            n = sum(new)
            assert bool((st["rows"][n:] == 7.0).all())
            assert not bool((st["rows"][:n] == 7.0).all(-1).any())


def test_calls_on_two_streams_at_once(dsa, workspace):
    """Chunks on one stream and single tokens on another, a workspace each, with nothing between
    them: the bits of the calls made one after the other."""
    work = torch.empty(B.DSA_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    jobs = []
    for lens, seed, w in (([(300, 900), (200, 200)], 35, workspace), ([(1, 5000), (1, 70)], 36, work)):
        batch = Q.make(lens, 64, seed=seed)
        gb, q = to_gpu(batch), queries(batch, 64, seed).cuda()
        want = torch.empty_like(q)
        B.dsa_paged_q4_attn(q, *args(gb), 200, 4, SCALE, w, want, gb["cos_sin"])
        jobs.append((gb, q, w, want, [torch.zeros_like(q) for _ in range(8)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for k in range(8):
        for gb, q, w, want, outs, stream in jobs:
            B.dsa_paged_q4_attn(q, *args(gb), 200, 4, SCALE, w, outs[k], gb["cos_sin"],
                                stream=stream)
    torch.cuda.synchronize()
    for gb, q, w, want, outs, stream in jobs:
        assert all(torch.equal(want, o) for o in outs)


def test_both_caches_in_turn_share_a_workspace(dsa, workspace):
    """Layers of bf16 pages and of 4-bit pages one after the other on one stream and one workspace."""
    import paged_ref as R
    lens = [(1, 3000), (2, 500)]
    q4, bf = Q.make(lens, 64, seed=37), R.make(lens, 64, seed=38)
    g4, gb = to_gpu(q4), to_gpu(bf)
    q = queries(q4, 64, 39).cuda()
    outs = [torch.empty_like(q) for _ in range(6)]
    for k in range(0, 6, 2):
        B.dsa_paged_attn(q, *args(gb), 0, SCALE, workspace, outs[k], gb["cos_sin"])
        B.dsa_paged_q4_attn(q, *args(g4), 0, 0, SCALE, workspace, outs[k + 1], g4["cos_sin"])
    torch.cuda.synchronize()
    for k in range(2, 6):
        assert torch.equal(outs[k], outs[k % 2])
    check_attn(outs[1].cpu(), q4, q.cpu(), 0, 0)


def test_same_call_twice_gives_the_same_bits(dsa, workspace):
    batch = Q.make([(1, 3000), (30, 500), (1, 64)], 64, seed=25)
    q = queries(batch, 64, 14)
    a = run_attn(batch, q, 0, 0, workspace)
    for _ in range(3):
        assert torch.equal(a, run_attn(batch, q, 0, 0, workspace))


def test_a_token_gets_the_same_answer_in_any_batch(dsa, workspace):
    """Alone or beside others (where its keys are split differently): within the tolerance."""
    batch = Q.make([(2, 700), (1, 900), (64, 64)], 32, seed=26)
    q = queries(batch, 64, 15)
    whole = run_attn(batch, q, 0, 0, workspace)
    _, tol, _ = Q.attention(batch, q, 0, 0, SCALE)
    r0 = 0
    for s, n in enumerate([2, 1, 64]):
        one = dict(batch, page_table=batch["page_table"][s:s + 1].contiguous(),
                   seq_len=batch["seq_len"][s:s + 1].contiguous(),
                   new_start=torch.tensor([0, n], dtype=torch.int32))
        alone = run_attn(one, q[r0:r0 + n], 0, 0, workspace)
        d = (alone.double() - whole[r0:r0 + n].double()).abs()
        assert bool((d <= 2 * tol[r0:r0 + n]).all())
        r0 += n


# --------------------------------------------------------------------------- logits of any size

BATCHES = [([(1, 1), (1, 130)], 64), ([(1, 4000)], 64), ([(1, 300)], 128),
           ([(20, 150), (70, 70)], 64), ([(40, 3000)], 16)]


@pytest.mark.parametrize("lens,heads", BATCHES)
@pytest.mark.parametrize("size,scale", [(2.0 ** 22, 0.5), (2.0 ** 60, 0.7), (2.0 ** 110, 0.3),
                                        (1.0, 2.0e38), (2.0 ** 100, 3.0e-39)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_rows_whatever_the_logits(dsa, workspace, lens, heads, size, scale, sign):
    """The output is the row: weights are equal (sums of them 2 n 2^-24 off), one rounding."""
    batch = Q.make(lens, 32, rope=False, seed=3)
    d = torch.where(torch.randn(512, generator=torch.Generator().manual_seed(5)) > 0, 1.0, -1.0)
    batch["pages"][:] = Q.pack(d.bfloat16())
    f = 1.0 + torch.arange(heads) / 128.0
    q = (sign * size * f[None, :, None] * d).expand(sum(n for n, _ in lens), heads, 512).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, 0, 0, workspace, scale=scale, status=status).double()
    assert status.item() == 0
    n = max(c for _, c in lens)
    err = (out - Q.decode(batch["pages"][0, 0])).abs()
    assert bool((err <= Q.U + 2 * n * 2.0 ** -24).all()), err.max()


@pytest.mark.parametrize("lens,heads", BATCHES)
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("window,sinks", [(0, 0), (77, 2)])
def test_the_larger_of_two_kinds_of_rows(dsa, workspace, lens, heads, size, sign, window, sinks):
    """Rows at even positions are d / 2, the others d (position 0 sees the even kind alone)."""
    batch = Q.make(lens, 32, rope=False, seed=3)
    d = torch.where(torch.randn(512, generator=torch.Generator().manual_seed(5)) > 0, 1.0, -1.0)
    kinds = [Q.pack((d * x).bfloat16()) for x in (0.5, 1.0)]
    values = [Q.decode(k) for k in kinds]
    for s, (_, c) in enumerate(lens):
        for p in range(c):
            batch["pages"][Q.place(batch, s, p)] = kinds[p % 2]
    q = (sign * size * d).expand(sum(n for n, _ in lens), heads, 512).bfloat16()
    out = run_attn(batch, q, window, sinks, workspace, scale=0.4).double()
    r = 0
    for n, c in lens:
        for i in range(n):
            t = c - n + i
            want = values[1 if sign > 0 and t > 0 else 0]
            err = (out[r] - want).abs()
            assert bool((err <= Q.U + 2 * c * 2.0 ** -24).all()), (t, err.max())
            r += 1


@pytest.mark.parametrize("page,sinks", [(16, 1), (16, 16), (16, 37), (32, 16), (32, 65), (64, 4),
                                        (64, 100), (128, 8), (256, 8), (16, 128)])
@pytest.mark.parametrize("lens,heads,window", [
    ([(1, 129 + 9 * i) for i in range(45)], 64, 90),      # windows that begin everywhere in a block
    ([(330, 700), (1, 300)], 16, 130),                    # four tokens a unit
    ([(150, 420)], 64, 1), ([(140, 600)], 5, 257), ([(90, 500), (3, 260)], 128, 128)])
def test_first_tokens_in_the_places_before_a_window(dsa, workspace, page, sinks, lens, heads, window):
    """The first tokens' pages lie in the window's first block where it has room for them, and in a
    block of their own where it has not."""
    batch = Q.make(lens, page, seed=page + sinks)
    # rows that no token sees: NaN
    pages, table = batch["pages"], batch["page_table"]
    for s, (n, c) in enumerate(lens):
        pos = torch.arange(c)
        gone = pos[(pos >= sinks) & (pos <= c - n - window)]
        pages[table[s, gone // page].long(), gone % page] = 0xFF
    q = queries(batch, heads, 21)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_attn(batch, q, window, sinks, workspace, status=status)
    assert status.item() == 0
    check_attn(out, batch, q, window, sinks)
