"""The 4-bit row's definition: known values, its two plain forms against each other, its size of
error, and the stated limits (CPU)."""
import numpy as np
import torch

import q4_ref as Q


def test_e4m3_table_is_the_type():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), Q.E4M3)
    v = torch.rand(2000, generator=torch.Generator().manual_seed(1)) * 300
    v = torch.cat([v, torch.from_numpy((Q.E4M3[:-1] + Q.E4M3[1:]) / 2).float()])   # and the ties
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).tolist()
    assert [Q.nearest_e4m3(x) for x in v.double().tolist()] == want


def test_known_row():
    x = torch.zeros(512, dtype=torch.float64)
    x[:16] = torch.tensor([7, 3.5, 2.5, -1.5, .5, -.5, 1, 2, 3, 4, 5, 6, 6.5, -6.5, -7, 0.])
    x[448:] = torch.arange(64)
    row = Q.encode(x)
    # A = 7: E = 2 - 10; s = 1 / 2^-8 = 256 = 1.0 * 2^8 -> exponent 15, mantissa 0
    assert row[14] == row[30] == 2 + 127 and row[0] == 0x78 and row[1] == 0
    got = Q.decode(row)
    assert got[:16].tolist() == [7, 4, 2, -2, 0, 0, 1, 2, 3, 4, 5, 6, 6, -6, -7, 0]
    assert got[448:].tolist() == list(range(64)) and not got[16:448].any()


def test_both_forms_agree_and_the_error_is_as_stated():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(400, 512, generator=g).bfloat16()
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -100
    x[3, :448] = 0
    x[4, :64] *= 2.0 ** -17
    x[5] *= 2.0 ** -124
    rows = Q.pack(x)
    for i in range(12):
        assert torch.equal(rows[i], Q.encode(x[i].double()))
        assert torch.equal(Q.unpack(rows[i]), Q.decode(rows[i]))
    v = Q.unpack(rows)
    assert torch.equal(v.bfloat16().double(), v)                   # exact in bf16
    err = (v - x.double())[6:, :448].square().mean().sqrt().item()
    assert 0.08 < err < 0.09
    # a step is at most a seventh of the group's largest, and that is off by 2^-4 at most
    top = x.double()[6:, :448].view(-1, 28, 16).abs().amax(-1, keepdim=True)
    off = (v - x.double())[6:, :448].view(-1, 28, 16).abs()
    assert bool((off <= top / 14 * (1 + 2.0 ** -4) + top * 0.0).all())


def test_odd_groups_read_as_nan_and_leave_the_others():
    x = torch.randn(512, generator=torch.Generator().manual_seed(3)).bfloat16().double()
    plain = Q.decode(Q.encode(x))
    for bad in (float("nan"), float("inf"), -float("inf"), 2.0 ** 124, -3e38):
        y = x.clone()
        y[40] = bad
        got = Q.decode(Q.encode(y))
        assert got[32:48].isnan().all()
        keep = torch.ones(512, dtype=torch.bool)
        keep[32:48] = False
        y[32:48] = 0
        assert torch.equal(got[keep], Q.decode(Q.encode(y))[keep])
    assert plain.isfinite().all()
