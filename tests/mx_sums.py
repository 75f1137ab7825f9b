"""Products of microscaled operands whose sums show every part that is left out: inputs and a model of what
one matrix instruction adds up.

Every eight elements begin with a pair of equal large ones whose weights are c and -c, so their products
cancel, and hold others that are 2^-13 and less of them.  A sum of eight that keeps 13 bits below its largest
product loses these others, which are all that is left of the sum; in three parts by magnitude nothing is
lost.  All values are multiples of 2^-10 (the block's 2^-16) and sums of whole groups of eight stay below 2^24
of these: float32 holds them in any order, and the operators' results have to be equal."""
import torch

from tests import mx_reference as M

F64 = torch.float64
LARGE = 256.0
ONE = 2.0 ** -6        # the element that an up projection's rows take: the block's middle is 2^-6 of the gate's


def _pick(gen, values, *shape):
    return torch.tensor(values, dtype=F64)[torch.randint(0, len(values), shape, generator=gen)]


def matrix(v, form):
    """(codes, scales) of values that are elements of the form as they are (scale 1)."""
    s = torch.full((v.shape[0], M.steps(v.shape[1]) * 4), 127, dtype=torch.uint8)
    codes = M.pack(M.elements(v, s, form), form)
    assert torch.equal(M.values(codes, s, form, v.shape[1]), v)
    return codes, s


def tokens(T, K, seed):
    """Of every eight: two large, ONE, two of 0.25 to 1, three of 2^-6 to 2^-4; all E4M3 elements, positive."""
    gen = torch.Generator().manual_seed(seed)
    grid = [g for g in M.GRID["e4m3"] if g > 0]
    v = _pick(gen, [g for g in grid if 2.0 ** -6 <= g < 2.0 ** -4], T, K)
    medium = _pick(gen, [g for g in grid if 0.25 <= g < 1], T, K)
    at = torch.arange(K) % 8
    v = torch.where((at == 3) | (at == 4), medium, v)
    v[:, at == 2] = ONE
    v[:, at < 2] = LARGE
    if K % 8 == 1:
        v[:, -1] = 1.0                                  # a large one without its pair
    return v


def _pairs(gen, rows, cols):
    """Zeros but for c, -c at the large pair of every eight."""
    w = torch.zeros((rows, cols), dtype=F64)
    c = _pick(gen, [1.0, 1.5, 2.0, -1.0, -1.5, -2.0], rows, (cols + 7) // 8)
    w[:, 0::8] = c
    if cols % 8 == 1:
        w[:, -1] = 1.0
    w[:, 1::8] = -c[:, : w[:, 1::8].shape[1]]
    return w


def weights(N, K, seed):
    """Pairs that cancel, any of 0, 0.5 and 1 with a sign elsewhere."""
    gen = torch.Generator().manual_seed(seed)
    rest = _pick(gen, [0.0, 0.5, -0.5, 1.0, -1.0], N, K)
    at = torch.arange(K) % 8
    return torch.where((at < 2)[None], _pairs(gen, N, K), rest)


def block(H, I, seed, alone=False):
    """Weights of a gated block for `tokens`, K = H >= 8: row j of the gate takes one element (a large one
    for the first two of every eight j) and that of the up projection ONE, so with relu the middle is on
    codes (scale 2^-6) and is `tokens`-like itself; `weights` bring it down.  alone: no pair is beside ONE, so
    one instruction has the up projection's sums too, and some of the gate's."""
    gen = torch.Generator().manual_seed(seed)
    gate, up = _pairs(gen, I, H), _pairs(gen, I, H)
    groups, at = H // 8, torch.arange(I) % 8
    rows = torch.arange(I)
    k = torch.randint(0, groups, (I,), generator=gen) * 8
    other = k + torch.randint(3, 8, (I,), generator=gen)
    large = at < 2
    gate[rows[large], k[large]], gate[rows[large], k[large] + 1] = 1.0, 0.0
    gate[rows[~large], other[~large]] = 1.0
    k = torch.randint(0, groups, (I,), generator=gen) * 8
    up[rows, k + 2] = 1.0
    if alone:
        up[rows, k] = up[rows, k + 1] = 0.0
    if H % 8 == 1:
        gate[:, -1] = up[:, -1] = 0.0
    down = weights(H, I, seed + 1)
    if I % 8 == 1:
        down[:, -1] = 0.5
    return {"w_gate": gate, "w_up": up, "w_down": down}


def _groups(x, w):
    """Products of E4M3 and E2M1 elements by groups of 8, [T][N][groups][8], and what a group's are cut off
    at: 2^-13 of the largest power of two, that of an element being its exponent's (the least there is, -6 and
    0, for the ones below it), of the products that are not zero."""
    pad = -x.shape[1] % 8
    x, w = (torch.nn.functional.pad(t, (0, pad)) for t in (x, w))
    p = (x[:, None] * w[None]).view(x.shape[0], w.shape[0], -1, 8)
    power = (torch.frexp(x).exponent - 1).clamp(min=-6)[:, None] + (torch.frexp(w).exponent - 1).clamp(min=0)[None]
    most = torch.where(p != 0, power.view(p.shape), -99).amax(-1, keepdim=True)
    return p, torch.exp2(most.to(F64) - 13)


def one_instruction(x, w, scale=None):
    """x w^T as one instruction for every step adds up elements: of each group of 8, products cut off towards
    zero; scale: of each element's block of x, [T][K]."""
    p, step = _groups(x, w)
    sums = (torch.trunc(p / step) * step).sum(-1)
    return (sums if scale is None else sums * scale[:, None, ::8]).sum(-1)


def lost(x, w):
    """Bound on what one instruction a step loses of x w^T: of seven of each eight products (the one of the
    largest power loses nothing) less than a step.  Products are multiples of 2^-10, so what loses has a largest
    power of 4 at least, its element of x is none of the smallest and its product at least 2^-1 of that power
    (weights of 0.5): less than 7 * 2^-12 of the largest product."""
    p, step = _groups(x, w)
    assert (7 * step <= 7 * 2.0 ** -12 * p.abs().amax(-1, keepdim=True)).logical_or(step <= 2.0 ** -10).all()
    return 7 * torch.where(step > 2.0 ** -10, step, 0.0).sum((-1, -2))


def three_parts(x, w, scale=None):
    """The elements of x in three parts by magnitude, an instruction each."""
    a = x.abs()
    return sum(one_instruction(torch.where(part, x, 0.0), w, scale)
               for part in (a < 2.0 ** -4, (a >= 2.0 ** -4) & (a < 8), a >= 8))


def exact(x, w, scale=None):
    return (x if scale is None else x * scale) @ w.T


def through(x, w, product):
    """The gated block (relu) with `product` for its sums: the middle, and what comes down from it in E4M3."""
    mid = torch.relu(product(x, w["w_gate"])) * product(x, w["w_up"])
    c, s = M.quantize(mid, "e4m3")
    scale = torch.exp2(s.to(F64) - 127).repeat_interleave(32, 1)[:, : mid.shape[1]]
    return mid, product(M.values(c, s, "e4m3", mid.shape[1]) / scale, w["w_down"], scale)
