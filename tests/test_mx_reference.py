"""The 64-bit reference of microscaled matrices against values worked out by hand and by brute force."""
import math

import pytest
import torch

from tests import mx_reference as M


def test_grids():
    assert M.GRID["e2m1"] == [0, .5, 1, 1.5, 2, 3, 4, 6]
    assert len(M.GRID["e4m3"]) == 127 and M.GRID["e4m3"][-1] == 448 and M.GRID["e4m3"][8] == 2.0 ** -6
    codes = torch.arange(127, dtype=torch.uint8)
    assert torch.equal(codes.view(torch.float8_e4m3fn).double(), torch.tensor(M.GRID["e4m3"], dtype=M.F64))


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_scales(form):
    v = torch.zeros((8, 32), dtype=M.F64)
    for i, top in enumerate((1.0, 1.99, 2.0, 0.0, 2.0 ** -140, 3e38, math.inf, math.nan)):
        v[i, 5] = -top
    e = M.EMAX[form]
    want = [127 - e, 127 - e, 128 - e, 0, 0, 127 - e + 127, 255, 255]
    assert M.scale_bytes(v, form)[:, 0].tolist() == want
    assert M.scale_bytes(v, form)[:, 1:].tolist() == [[0, 0, 0]] * 8    # wholly padded blocks


def test_ties_go_to_even_and_large_values_saturate():
    v = torch.zeros((1, 32), dtype=M.F64)
    v[0, :15] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.25, -0.75, 0.2501, 4.99, 5.01, -6.5])
    c, s = M.quantize(v, "e2m1")
    assert s[0, 0] == 127
    got = M.values(c, s, "e2m1", 15)[0].tolist()
    assert got == [4, 0, 1, 1, 2, 2, 4, 4, 6, -0.0, -1, .5, 4, 6, -6]
    assert math.copysign(1, got[9]) == -1


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_nearest_by_brute_force(form):
    g = torch.Generator().manual_seed(1)
    v = torch.randn((20, 200), generator=g, dtype=M.F64) * torch.exp(3 * torch.randn((20, 1), generator=g, dtype=M.F64))
    c, s = M.quantize(v, form)
    got = M.values(c, s, form, 200)
    power = torch.exp2(s.double() - 127).repeat_interleave(32, 1)[:, :200, None]
    every = torch.tensor(M.GRID[form], dtype=M.F64)
    every = torch.cat((every, -every)) * power
    assert torch.equal((got - v).abs(), (every - v[..., None]).abs().amin(-1))
    assert torch.equal(M.rounded(got, form), got)                       # a fixed point
    assert c.shape == (20, 256 if form == "e4m3" else 128) and s.shape == (20, 8)
    full = M.values(c, s, form, 256)
    assert torch.equal(full[:, 200:], torch.zeros((20, 56), dtype=M.F64))


def test_low_four_bits_hold_the_even_element():
    v = torch.zeros((1, 4), dtype=M.F64)
    v[0] = torch.tensor([6.0, -0.5, 1.5, 0.0])
    c, s = M.quantize(v, "e2m1")
    assert c[0, :2].tolist() == [0x97, 0x03] and s[0, 0] == 127
