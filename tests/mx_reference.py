"""Microscaled matrices in 64 bits: blocks of 32 elements with a power of two, written out from the
definition (the nearest of the elements there are, found by search), and the operators that read them."""
import math

import torch

from tests import block_reference as R

F64 = torch.float64
EMAX = {"e4m3": 8, "e2m1": 2}
GRID = {"e2m1": [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0],
        "e4m3": [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]}


def steps(cols):
    return -(-cols // 128)


def _blocks(v):
    rows, cols = v.shape
    full = torch.zeros((rows, steps(cols) * 128), dtype=F64)
    full[:, :cols] = v
    return full.view(rows, -1, 32)


def scale_bytes(v, form):
    """[rows][S * 4] of v (any float type, on the CPU)."""
    top = _blocks(v.to(F64)).abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(torch.where(torch.isfinite(top), top, 1.0)).exponent - 1 - EMAX[form], -127)
    return torch.where(torch.isfinite(top), e.clamp(min=-127) + 127, 255).to(torch.uint8)


def elements(v, scales, form):
    """Codes of v's elements under these scales, [rows][S * 128], unpacked; 0 in NaN blocks."""
    b, s = _blocks(v.to(F64)), scales[..., None].to(F64)
    grid = torch.tensor(GRID[form], dtype=F64)
    a = torch.where(s < 255, b.abs() * torch.exp2(127 - s), 0.0)
    between = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(a, between), torch.bucketize(a, between, right=True)
    code = torch.where(low % 2 == 0, low, high)
    sign = (torch.signbit(b) & (s < 255)).long()
    return (code + sign * (128 if form == "e4m3" else 8)).view(v.shape[0], -1)


def pack(codes, form):
    c = codes.to(torch.uint8)
    return c if form == "e4m3" else c[:, ::2] | c[:, 1::2] << 4


def quantize(v, form):
    """(codes, scales) as bytes."""
    s = scale_bytes(v, form)
    return pack(elements(v, s, form), form), s


def values(codes, scales, form, cols):
    """The 64-bit values of codes and scales."""
    codes = codes.cpu().long()
    if form == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(1)
    half = 128 if form == "e4m3" else 8
    grid = torch.tensor((GRID[form] + [math.nan])[:half], dtype=F64)
    s = scales.cpu().to(F64)
    power = torch.where(s == 255, math.nan, torch.exp2(s - 127)).repeat_interleave(32, 1)
    return (torch.cat((grid, -grid))[codes] * power)[:, :cols]


def rounded(v, form):
    """v's values in the form."""
    return values(*quantize(v, form), form, v.shape[1])


def linear(x, w, bias=None, residual=None, act="none"):
    return R.linear(x, w, bias, residual, act)


def ffn(x, w, residual=None, act="silu", form="e4m3"):
    mid = R.act(act, x @ w["w_gate"].T) * (x @ w["w_up"].T)
    y = rounded(mid, form) @ w["w_down"].T
    return y if residual is None else y + residual


def sums(dtype, cols, form):
    """Relative error of a contraction's sums.  A matrix instruction adds four block sums and the sum so far,
    each aligned to the largest and cut off, by less than 2^-22 of it (all in one direction), and rounds by
    2^-24; sums of eight waves or two halves are joined, and bias, activation and residual round once more
    each.  Block sums are exact, but for 8-bit operands where the output is bfloat16: there each product is
    cut off 2^-13 below its group's largest power of two, which for normal values is up to four times the
    typical product, uniformly and independently."""
    err = steps(cols) * (4 * 2.0 ** -22 + 2.0 ** -24) + 12 * 2.0 ** -24
    return err + (4 * 2.0 ** -13 / math.sqrt(3) if dtype == "bf16" and form == "e4m3" else 0)


def tolerance(dtype, cols, form):
    """Of a product of contraction `cols`, as block_reference.worst measures it: its sums, and the rounding
    of a bfloat16 output."""
    return sums(dtype, cols, form) + (2.0 ** -8 if dtype == "bf16" else 0)


def flips(dtype, cols, form):
    """What a middle of contraction `cols` adds to the error of a feed-forward block: an element nearer to
    the border of two codes than its own error may take the other.  Steps are 2^-4 to 2^-3 of a value (4
    bits: 2^-2 to 2^-1, and as much below the smallest normal one): a share of 2 error / step, each off by a
    step.  The element's error is that of two sums."""
    low = 2.0 ** (-4 if form == "e4m3" else -2)
    return math.sqrt(2 * 2 * sums(dtype, cols, form) / low) * 2 * low
