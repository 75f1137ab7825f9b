"""The operators with microscaled operands on the GPU against plain 64-bit forms, through the C ABI's
binding: sizes from one token and one column on, sizes and strides that nothing divides, both forms and
types; blocks of zeros, infinities and NaN; exact sums; determinism, streams and graph replays."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests import block_reference as R
from tests import mx_reference as M
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FORMS = ["e4m3", "e2m1"]
F64 = torch.float64


def say(msg):
    print(msg, flush=True)


def _rand(dtype, *shape, seed=0, scale=1.0, shift=0.0):
    v = torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32)
    return (v * scale + shift).to(TYPES[dtype]).to(DEV)


def _rows(dtype, T, cols, pad, seed, scale=1.0):
    """[T][cols], the columns of a wider tensor whose others are NaN."""
    t = torch.full((T, cols + pad), float("nan"), dtype=TYPES[dtype], device=DEV)
    t[:, :cols] = _rand(dtype, T, cols, seed=seed, scale=scale)
    return t[:, :cols]


def _out(dtype, T, cols, pad=0):
    return torch.full((T, cols + pad), float("nan"), dtype=TYPES[dtype], device=DEV)[:, :cols]


def _pads_kept(t):
    base = t._base
    return base is None or base.shape[1] == t.shape[1] or bool(torch.isnan(base[:, t.shape[1]:]).all())


def _lift(v):
    return None if v is None else v.detach().cpu().double()


def _lifted(d):
    return {k: _lift(v) for k, v in d.items()}


class Guarded:
    """Room for a microscaled matrix, every byte 0xa5, with 64 rows more behind it that stay so."""

    def __init__(self, rows, cols, form):
        full = moe.alloc_mx(rows + 64, cols, form, DEV)
        full.codes.fill_(0xa5)
        full.scales.fill_(0xa5)
        self.full, self.rows = full, rows
        self.m = moe.MxMatrix(full.codes[:rows], full.scales[:rows], form, cols)

    def kept(self):
        return all(bool((t[self.rows:] == 0xa5).all()) for t in (self.full.codes, self.full.scales))


def _upload(v, form):
    """A 64-bit matrix in microscaled form on the GPU, and its values."""
    c, s = M.quantize(v, form)
    return moe.MxMatrix(c.to(DEV), s.to(DEV), form, v.shape[1]), M.values(c, s, form, v.shape[1])


def _matrix(rows, cols, form, seed, scale=1.0):
    """Normal values whose rows and blocks differ in size by powers of two."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((rows, cols), generator=g, dtype=F64) * scale
    v *= torch.exp2(torch.randint(-2, 3, (rows, 1), generator=g).double())
    v *= torch.exp2(torch.randint(-1, 2, (1, M.steps(cols) * 4), generator=g).double()).repeat_interleave(32, 1)[:, :cols]
    return _upload(v, form)


# ---------------------------------------------------------------- quantisation

SHAPES = [(1, 1, 0), (1, 31, 0), (3, 32, 0), (2, 33, 1), (5, 127, 3), (4, 128, 8), (3, 129, 0), (70, 40, 0),
          (17, 1001, 5), (9, 2048, 0), (5, 2056, 8), (3, 7168, 0), (300, 520, 0), (2, 131072, 0)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_quantize(rows, cols, pad, dtype, form):
    say(f"quantize {form} {dtype} {rows} x {cols} + {pad}")
    x = _rows(dtype, rows, cols, pad, seed=cols, scale=3.0)
    x[:, ::7] *= 100
    x[rows // 2, : min(cols, 64)] = 0                                   # blocks of zeros
    out = Guarded(rows, cols, form)
    moe.mx_quantize(x, out.m)
    c, s = M.quantize(_lift(x), form)
    assert torch.equal(out.m.scales.cpu(), s) and torch.equal(out.m.codes.cpu(), c) and out.kept()
    for to in TYPES:
        y = _out(to, rows, cols, pad)
        moe.mx_dequantize(out.m, y)
        assert torch.equal(y.cpu().double(), M.values(c, s, form, cols)) and _pads_kept(y)


@pytest.mark.parametrize("form", FORMS)
def test_quantize_borders_and_extremes(form):
    grid = torch.tensor(M.GRID[form], dtype=torch.float32)
    mid = (grid[1:] + grid[:-1]) / 2
    near = torch.cat((mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1), grid,
                      grid[-1] * torch.tensor([1.03, 1.06, 1.1, 1.14])))
    near = torch.cat((near, -near))
    near = torch.cat((near, torch.zeros(-len(near) % 31))).view(-1, 31)
    rows = torch.cat((torch.full((len(near), 1), 2.0 ** M.EMAX[form]), near), 1)       # the block's scale is 1
    scaled = [rows * 2.0 ** e for e in (0, 5, -100, -118, 100, 119 if form == "e4m3" else 125)]
    tiny = torch.tensor([[2.0 ** -149, 2.0 ** -140, 2.0 ** -126, -2.0 ** -130] * 8, [2.0 ** -135] * 32, [0.0] * 32])
    huge = torch.full((1, 32), torch.finfo(torch.float32).max)
    x = torch.cat((*scaled, tiny, huge)).to(DEV)
    out = Guarded(x.shape[0], 32, form)
    moe.mx_quantize(x, out.m)
    c, s = M.quantize(_lift(x), form)
    assert torch.equal(out.m.scales.cpu(), s) and torch.equal(out.m.codes.cpu(), c) and out.kept()


@pytest.mark.parametrize("form", FORMS)
def test_quantize_not_finite(form):
    x = _rand("f32", 6, 256, seed=3)
    x[0, 3], x[1, 40], x[2, 255], x[4, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[4, 1] = float("inf")
    out, y = Guarded(6, 256, form), _out("f32", 6, 256)
    moe.mx_quantize(x, out.m)
    c, s = M.quantize(_lift(x), form)
    assert torch.equal(out.m.scales.cpu(), s) and torch.equal(out.m.codes.cpu(), c)
    moe.mx_dequantize(out.m, y)
    bad = torch.isnan(y).view(6, 8, 32)
    assert bad[0, 0].all() and bad[1, 1].all() and bad[2, 7].all() and bad[4, 0].all() and bad.sum() == 4 * 32


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("to", ["bf16", "f32"])
def test_dequantize_every_code_and_scale(form, to):
    cols = 256 if form == "e4m3" else 512
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).to(DEV)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, cols // 32).to(DEV)
    y = _out(to, 256, cols)
    moe.mx_dequantize(moe.MxMatrix(codes, scales, form, cols), y)
    want = M.values(codes, scales, form, cols).to(TYPES[to])
    assert torch.equal(torch.isnan(y).cpu(), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=0.0), torch.nan_to_num(want, nan=0.0))


# ---------------------------------------------------------------- norm

NORM = [  # T, hidden, pad, rows of the gate (0: none)
    (1, 1, 0, 0), (1, 7168, 0, 1), (2, 31, 1, 2), (5, 64, 0, 0), (7, 130, 3, 7), (300, 512, 0, 0), (3, 520, 8, 1),
    (50, 1001, 5, 25), (33, 1024, 0, 33), (4, 1032, 0, 2), (3, 1030, 0, 3), (9, 4096, 8, 9), (2, 8200, 0, 0),
    (2, 9001, 0, 1), (2, 16384, 0, 2),
]


def _norm_inputs(dtype, T, H, pad, gate_rows, kind):
    r, f = _rows(dtype, T, H, pad, 1, 2.0), _rows(dtype, T, H, pad, 2, 0.5)
    p = {"w_post": _rand(dtype, H, seed=3, scale=0.1, shift=1), "w_pre": _rand(dtype, H, seed=4, scale=0.1, shift=1)}
    if kind == "layer":
        p["b_post"], p["b_pre"] = _rand(dtype, H, seed=5, scale=0.1), _rand(dtype, H, seed=6, scale=0.1)
    if gate_rows:
        p["gate"] = _rand(dtype, T // gate_rows, H, seed=7, scale=0.3, shift=0.5)
    return r, f, p


def _between(m, want, form, off):
    """m's codes and scales are those of values within `off` (relative to each row's typical size) of want."""
    off = off * want.square().mean(1, keepdim=True).sqrt()
    top = torch.nn.functional.pad(want, (0, M.steps(want.shape[1]) * 128 - want.shape[1])).view(want.shape[0], -1, 32)
    top = top.abs().amax(-1)
    byte = lambda t: M.scale_bytes(torch.nn.functional.pad(t[..., None], (0, 31)).flatten(1), form)  # noqa: E731
    s = m.scales.cpu()
    assert (s >= byte(torch.where(top > 0, top - off, 0.0).clamp(min=0))).all()
    assert (s <= byte(torch.where(top > 0, top + off, 0.0))).all()
    got = M.values(m.codes, s, form, want.shape[1])
    # by its own scales each code is that of a value no further off
    lo, hi = (M.values(M.pack(M.elements(v, s, form), form), s, form, want.shape[1]) for v in (want - off, want + off))
    assert ((got >= lo) & (got <= hi)).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,pad,gate_rows", NORM)
def test_norm(T, H, pad, gate_rows, dtype, form):
    for kind in ("rms", "layer"):
        say(f"norm {kind} {form} {dtype} T={T} H={H} pad={pad} gate={gate_rows}")
        r, f, p = _norm_inputs(dtype, T, H, pad, gate_rows, kind)
        cfg = moe.make_norm_cfg(H, dtype, kind, gate_rows, 1e-6, 0.75)
        out, u, h = Guarded(T, H, form), _out(dtype, T, H, pad), _out(dtype, T, H, pad)
        moe.norm_mx_forward(cfg, r, f, p, u, out.m, h=h)
        u2, h2 = _out(dtype, T, H), _out(dtype, T, H)
        moe.norm_forward(cfg, r, f, p, u2, h2)
        assert torch.equal(u, u2) and torch.equal(h, h2) and _pads_kept(u) and _pads_kept(h) and out.kept()
        wu, wh = R.norm(_lift(r), _lift(f), _lifted(p), kind, 1e-6, 0.75)
        # float32 sums of two norms in a row and a row's few operations, each element by itself: the
        # sums' share is the same for a row, the operations round 8 times
        _between(out.m, wh, form, 2 * R.tolerance("f32", 1, H) + 8 * 2.0 ** -24 * (1 + float(wh.abs().max())))
        alone = Guarded(T, H, form)
        moe.norm_mx_forward(cfg, r, f, p, None, alone.m)                # neither u nor h
        assert torch.equal(alone.m.codes, out.m.codes) and torch.equal(alone.m.scales, out.m.scales)
        # padding: codes 0, wholly padded blocks are blocks of zeros
        c = out.m.codes.cpu()
        assert not c[:, H if form == "e4m3" else (H + 1) // 2:].any() and not out.m.scales[:, -(-H // 32):].any()


def test_norm_rows_beyond_the_workers():
    T, H = 9000, 72                                                     # more rows than waves on the chip
    for form in FORMS:
        r, f, p = _norm_inputs("bf16", T, H, 0, 0, "rms")
        cfg, out, h = moe.make_norm_cfg(H, "bf16"), Guarded(T, H, form), _out("bf16", T, H)
        moe.norm_mx_forward(cfg, r, None, {"w_pre": p["w_pre"]}, None, out.m, h=h)
        _, wh = R.norm(_lift(r), None, {"w_pre": _lift(p["w_pre"])})
        _between(out.m, wh, form, 2 * R.tolerance("f32", 1, H) + 8 * 2.0 ** -24 * (1 + float(wh.abs().max())))
        assert out.kept()


@pytest.mark.parametrize("H", [256, 250, 2000, 2001])
def test_norm_not_finite(H):
    r, f, p = _norm_inputs("f32", 5, H, 0, 0, "rms")
    r[1, 3], f[3, H - 1] = float("nan"), float("inf")
    for form in FORMS:
        out, y = Guarded(5, H, form), _out("f32", 5, H)
        moe.norm_mx_forward(moe.make_norm_cfg(H, "f32"), r, f, p, None, out.m)
        moe.mx_dequantize(out.m, y)
        bad = torch.isnan(y).all(1)
        assert bad.tolist() == [False, True, False, True, False] and torch.isfinite(y[[0, 2, 4]]).all()
        c = out.m.codes
        assert not c[:, H if form == "e4m3" else (H + 1) // 2:].any() and (out.m.scales[:, -(-H // 32):] == 0).all()


def test_norm_in_place():
    T, H = 37, 1536
    r, f, p = _norm_inputs("bf16", T, H, 0, T, "rms")
    cfg = moe.make_norm_cfg(H, "bf16", "rms", T, 1e-6, 0.5)
    a, b, u, h = Guarded(T, H, "e4m3"), Guarded(T, H, "e4m3"), _out("bf16", T, H), _out("bf16", T, H)
    moe.norm_mx_forward(cfg, r, f, p, u, a.m, h=h)
    moe.norm_mx_forward(cfg, r, f, p, r, b.m, h=f)
    assert torch.equal(r, u) and torch.equal(f, h)
    assert torch.equal(a.m.codes, b.m.codes) and torch.equal(a.m.scales, b.m.scales)


# ---------------------------------------------------------------- linear

LINEAR = [  # T, in, out, pad
    (1, 1, 1, 0), (1, 128, 16, 0), (1, 1001, 777, 3), (3, 7, 1030, 0), (7, 256, 130, 8), (16, 2048, 640, 0),
    (17, 130, 33, 1), (33, 1000, 264, 0), (48, 1152, 96, 0), (64, 512, 256, 8), (65, 72, 8, 0), (100, 4096, 40, 0),
    (128, 64, 128, 0), (129, 1033, 257, 5), (257, 640, 300, 0), (300, 1024, 256, 0), (513, 384, 1100, 1),
    (1000, 200, 520, 2), (2100, 520, 2050, 0),
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,pad", LINEAR)
def test_linear(T, K, N, pad, dtype, form):
    x, xv = _matrix(T, K, form, 1)
    w, wv = _matrix(N, K, "e2m1", 2, K ** -0.5)
    for i, (act, bias, res) in enumerate((("none", False, False), ("gelu", True, True), ("silu", True, False),
                                          ("relu", False, True))):
        say(f"linear {form} {dtype} T={T} K={K} N={N} pad={pad} {act}")
        b = _rand(dtype, N, seed=20 + i) if bias else None
        r = _rows(dtype, T, N, pad, 30 + i) if res else None
        cfg = moe.make_mx_linear_cfg(K, N, act, dtype, form)
        y, ws = _out(dtype, T, N, pad), moe.alloc_mx_linear_workspace(cfg, T, DEV)
        moe.mx_linear_forward(cfg, x, w, y, ws, bias=b, residual=r)
        want = M.linear(xv, wv, _lift(b), _lift(r), act)
        assert R.worst(y, want) <= M.tolerance(dtype, K, form), (act, R.worst(y, want))
        assert _pads_kept(y)


# products large enough for every tile, and contractions that are split: whole and ragged tiles, with
# residuals that the largest tile can copy as they lie (rows of whole 16 bytes) and cannot
LARGE = [(130, 4100, 40, 0, 0), (200, 130, 4100, 3, 0), (333, 7168, 512, 0, 0), (700, 2050, 3000, 5, 0),
         (1100, 1500, 2048, 0, 0), (3000, 2600, 4100, 0, 0), (2816, 2600, 4352, 0, 8), (2817, 2304, 4353, 1, 1),
         (4096, 2304, 4096, 0, 0)]


def _on_gpu(v):
    return None if v is None else v.detach().to(DEV, F64)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,K,N,pad,pad_residual", LARGE)
def test_linear_large(T, K, N, pad, pad_residual, form):
    x, xv = _matrix(T, K, form, 1)
    w, wv = _matrix(N, K, "e2m1", 2, K ** -0.5)
    xg, wg = _on_gpu(xv), _on_gpu(wv)
    for i, (dtype, act, bias, res) in enumerate((("bf16", "none", False, True), ("bf16", "silu", True, False),
                                                 ("f32", "gelu", True, True))):
        say(f"linear large {form} {dtype} T={T} K={K} N={N} pad={pad} {act}")
        b = _rand(dtype, N, seed=20 + i) if bias else None
        r = _rows(dtype, T, N, pad_residual, 30 + i) if res else None
        cfg = moe.make_mx_linear_cfg(K, N, act, dtype, form)
        y, ws = _out(dtype, T, N, pad), moe.alloc_mx_linear_workspace(cfg, T, DEV)
        moe.mx_linear_forward(cfg, x, w, y, ws, bias=b, residual=r)
        want = M.linear(xg, wg, _on_gpu(b), _on_gpu(r), act).cpu()
        assert R.worst(y, want) <= M.tolerance(dtype, K, form), (act, R.worst(y, want))
        assert _pads_kept(y)
        if res:                                                         # into the residual itself
            moe.mx_linear_forward(cfg, x, w, r, ws, bias=b, residual=r)
            assert torch.equal(r, y)


def _whole(rows, cols, form, seed, most):
    """Whole numbers up to `most` at scale 1 (their blocks' scales say so where a block holds an element of
    2^emax): sums of their products are exact in float32."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-most, most + 1, (rows, cols), generator=g).double()
    codes = M.pack(M.elements(v, torch.full((rows, M.steps(cols) * 4), 127, dtype=torch.uint8), form), form)
    scales = torch.full((rows, M.steps(cols) * 4), 127, dtype=torch.uint8)
    m = moe.MxMatrix(codes.to(DEV), scales.to(DEV), form, cols)
    assert torch.equal(M.values(codes, scales, form, cols), v)
    return m, v


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,K,N", [(1, 7168, 200), (5, 999, 70), (33, 1500, 100), (64, 7168, 48), (70, 600, 65),
                                   (200, 2000, 300), (600, 1300, 900)])
def test_linear_sums_are_whole(T, K, N, form):
    say(f"whole sums {form} T={T} K={K} N={N}")
    (x, xv), (w, wv) = _whole(T, K, form, 1, 16 if form == "e4m3" else 4), _whole(N, K, "e2m1", 2, 4)
    cfg = moe.make_mx_linear_cfg(K, N, "none", "f32", form)
    y, ws = _out("f32", T, N), moe.alloc_mx_linear_workspace(cfg, T, DEV)
    moe.mx_linear_forward(cfg, x, w, y, ws)
    assert torch.equal(y.cpu().double(), xv @ wv.T)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,K,N", [(1, 300, 20), (40, 1000, 70), (70, 300, 65), (300, 640, 260)])
def test_linear_not_finite(T, K, N, form):
    x, xv = _matrix(T, K, form, 1)
    w, wv = _matrix(N, K, "e2m1", 2, K ** -0.5)
    x.scales[T - 1, 1] = 255                                            # a block of NaN in a token's row
    w.scales[3, K // 32 - 1] = 255                                      # and in a weight's
    if form == "e4m3" and T > 1:
        x.codes[0, 5] = 0x7f                                            # an element that is NaN
    cfg = moe.make_mx_linear_cfg(K, N, "relu", "bf16", form)
    y, ws = _out("bf16", T, N), moe.alloc_mx_linear_workspace(cfg, T, DEV)
    moe.mx_linear_forward(cfg, x, w, y, ws)
    bad = torch.zeros((T, N), dtype=torch.bool)
    bad[T - 1] = bad[:, 3] = True
    if form == "e4m3" and T > 1:
        bad[0] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    want = M.linear(xv, wv, None, None, "relu")
    assert ((y.cpu().double() - want).abs()[~bad] <= 2.0 ** -8 * want.abs()[~bad] + M.sums("bf16", K, form) * 4 * float((xv @ wv.T).std())).all()


def test_linear_scales_of_every_size():
    # rows whose scales are far apart, and products of scales that leave float32's range: 2^-127 2^-127 is
    # 0, 2^127 2^127 an infinity
    K = 128
    ones = torch.full((1, K), 0x38, dtype=torch.uint8)
    for form in FORMS:
        sx = torch.tensor([0, 1, 60, 100, 127, 150, 200, 254], dtype=torch.uint8)
        sw = torch.tensor([0, 27, 127, 200, 254], dtype=torch.uint8)
        x = moe.MxMatrix((ones if form == "e4m3" else torch.full((1, 64), 0x22, dtype=torch.uint8)).repeat(8, 1).to(DEV),
                         sx[:, None].repeat(1, 4).to(DEV), form, K)
        w = moe.MxMatrix(torch.full((5, 64), 0x22, dtype=torch.uint8).to(DEV), sw[:, None].repeat(1, 4).to(DEV), "e2m1", K)
        cfg = moe.make_mx_linear_cfg(K, 5, "none", "f32", form)
        y = _out("f32", 8, 5)
        moe.mx_linear_forward(cfg, x, w, y, moe.alloc_mx_linear_workspace(cfg, 8, DEV))
        want = (128 * torch.exp2(sx.double()[:, None] + sw.double()[None] - 254)).float()
        # a product below float32's smallest step, 2^-149, counts as 0: 128 of them are off by at most that
        assert torch.equal(torch.isinf(y).cpu(), torch.isinf(want))
        fine = torch.isfinite(want)
        assert ((y.cpu() - want).abs()[fine] <= 128 * 2.0 ** -149).all() and (want[fine] > 2.0 ** -100).sum() >= 10


def test_linear_in_place_and_alone():
    T, K, N = 90, 384, 136
    x, _ = _matrix(T, K, "e4m3", 1)
    w, _ = _matrix(N, K, "e2m1", 2, K ** -0.5)
    cfg = moe.make_mx_linear_cfg(K, N, "gelu", "bf16", "e4m3")
    ws = moe.alloc_mx_linear_workspace(cfg, T, DEV)
    r, y = _rand("bf16", T, N, seed=4), _out("bf16", T, N)
    moe.mx_linear_forward(cfg, x, w, y, ws, residual=r)
    moe.mx_linear_forward(cfg, x, w, r, ws, residual=r)
    assert torch.equal(r, y)


# ---------------------------------------------------------------- ffn

FFN = [  # T, hidden, inter, pad
    (1, 1, 1, 0), (1, 256, 512, 0), (2, 1001, 777, 3), (16, 640, 130, 0), (17, 130, 33, 1), (50, 1024, 264, 0),
    (64, 512, 256, 8), (65, 72, 8, 0), (129, 1033, 257, 5), (300, 1024, 256, 0), (520, 384, 1100, 1),
]


FFN_LARGE = [(200, 2600, 40, 0), (129, 7168, 300, 0), (1500, 1500, 2000, 3), (1500, 2600, 4100, 0), (2049, 2304, 3300, 0),
             (5, 300, 5000, 0), (16, 2048, 4097, 1)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,I,pad", FFN_LARGE)
def test_ffn_large(T, H, I, pad, form):
    say(f"ffn large {form} T={T} H={H} I={I} pad={pad}")
    x, xv = _matrix(T, H, form, 1)
    w, wv = _ffn_weights(H, I, 2)
    g = {k: _on_gpu(v) for k, v in wv.items()}
    for dtype in TYPES:
        r = _rows(dtype, T, H, pad, 30)
        cfg = moe.make_mx_ffn_cfg(H, I, "silu", dtype, form)
        y, ws = _out(dtype, T, H, pad), moe.alloc_mx_ffn_workspace(cfg, T, DEV)
        moe.mx_ffn_forward(cfg, x, w, y, ws, residual=r)
        mid = R.act("silu", _on_gpu(xv) @ g["w_gate"].T) * (_on_gpu(xv) @ g["w_up"].T)
        want = (_on_gpu(M.rounded(mid.cpu(), form)) @ g["w_down"].T).cpu() + _lift(r)
        assert R.worst(y, want) <= M.tolerance(dtype, I, form) + M.flips(dtype, H, form), R.worst(y, want)
        assert _pads_kept(y)


def _ffn_weights(H, I, seed):
    m = {k: _matrix(rows, cols, "e2m1", seed + i, cols ** -0.5)
         for i, (k, rows, cols) in enumerate((("w_gate", I, H), ("w_up", I, H), ("w_down", H, I)))}
    return {k: v[0] for k, v in m.items()}, {k: v[1] for k, v in m.items()}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,pad", FFN)
def test_ffn(T, H, I, pad, dtype, form):
    x, xv = _matrix(T, H, form, 1)
    w, wv = _ffn_weights(H, I, 2)
    for i, (act, res) in enumerate((("silu", True), ("gelu", False), ("relu", True))):
        say(f"ffn {form} {dtype} T={T} H={H} I={I} pad={pad} {act}")
        r = _rows(dtype, T, H, pad, 30 + i) if res else None
        cfg = moe.make_mx_ffn_cfg(H, I, act, dtype, form)
        y, ws = _out(dtype, T, H, pad), moe.alloc_mx_ffn_workspace(cfg, T, DEV)
        moe.mx_ffn_forward(cfg, x, w, y, ws, residual=r)
        want = M.ffn(xv, wv, _lift(r), act, form)
        assert R.worst(y, want) <= M.tolerance(dtype, I, form) + M.flips(dtype, H, form), (act, R.worst(y, want))
        assert _pads_kept(y)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,I", [(1, 7168, 256), (5, 300, 70), (40, 1500, 200), (64, 512, 2048), (70, 600, 65),
                                   (300, 1000, 400), (520, 256, 384)])
def test_ffn_whole_sums(T, H, I, form):
    # whole numbers and relu: the middle's values are exact, and so are their codes and the sums (up to the
    # middle's own scales, powers of two: products of 3 significant bits over a range of 2^12)
    say(f"ffn whole sums {form} T={T} H={H} I={I}")
    x, xv = _whole(T, H, form, 1, 2)
    ws_, wv = {}, {}
    for i, (k, rows, cols) in enumerate((("w_gate", I, H), ("w_up", I, H), ("w_down", H, I))):
        ws_[k], wv[k] = _whole(rows, cols, "e2m1", 2 + i, 1)
    cfg = moe.make_mx_ffn_cfg(H, I, "relu", "f32", form)
    y, work = _out("f32", T, H), moe.alloc_mx_ffn_workspace(cfg, T, DEV)
    moe.mx_ffn_forward(cfg, x, ws_, y, work)
    want = M.ffn(xv, wv, None, "relu", form)
    # the largest sum is below 2^24 smallest steps in 4 bits; in 8 bits sums of elements 2^-9 of the
    # largest may round
    assert (y.cpu().double() - want).abs().max() <= (0 if form == "e2m1" else M.tolerance("f32", I, form) * want.abs().max())


# ---------------------------------------------------------------- all


def _together(dtype, form, T, H, I):
    """A block's feed-forward half on microscaled operands, as a function that writes its outputs."""
    r, f, p = _norm_inputs(dtype, T, H, 0, T, "rms")
    ncfg = moe.make_norm_cfg(H, dtype, "rms", T)
    lcfg, fcfg = moe.make_mx_linear_cfg(H, H, "none", dtype, form), moe.make_mx_ffn_cfg(H, I, "silu", dtype, form)
    raw = {k: _rand("bf16", *s, seed=9 + i, scale=s[1] ** -0.5)
           for i, (k, s) in enumerate((("w_o", (H, H)), ("w_gate", (I, H)), ("w_up", (I, H)), ("w_down", (H, I))))}
    w = {k: moe.alloc_mx(*v.shape, "e2m1", DEV) for k, v in raw.items()}
    for k, v in raw.items():
        moe.mx_quantize(v, w[k])
    attn, hq = moe.alloc_mx(T, H, form, DEV), moe.alloc_mx(T, H, form, DEV)
    proj, u, y = (_out(dtype, T, H) for _ in range(3))
    lws, fws = moe.alloc_mx_linear_workspace(lcfg, T, DEV), moe.alloc_mx_ffn_workspace(fcfg, T, DEV)

    def run(stream=None):
        moe.mx_quantize(f, attn, stream=stream)
        moe.mx_linear_forward(lcfg, attn, w["w_o"], proj, lws, stream=stream)
        moe.norm_mx_forward(ncfg, r, proj, p, u, hq, stream=stream)
        moe.mx_ffn_forward(fcfg, hq, w, y, fws, residual=u, stream=stream)

    return run, [attn.codes, attn.scales, proj, u, hq.codes, hq.scales, y], (r, f, p, w, attn, hq)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,T,H,I", [("bf16", 1, 1024, 512), ("f32", 50, 520, 200), ("bf16", 300, 1001, 264)])
def test_together(dtype, T, H, I, form):
    say(f"together {form} {dtype} T={T} H={H} I={I}")
    run, (_, _, proj, u, _, _, y), (r, f, p, w, attn, hq) = _together(dtype, form, T, H, I)
    run()
    val = lambda m: M.values(m.codes, m.scales, m.form, m.cols)  # noqa: E731
    # each stage from what the stage before stored
    assert torch.equal(val(attn), M.rounded(_lift(f), form))
    wv = {k: val(m) for k, m in w.items()}
    assert R.worst(proj, val(attn) @ wv["w_o"].T) <= M.tolerance(dtype, H, form)
    wu, wh = R.norm(_lift(r), _lift(proj), _lifted(p))
    assert R.worst(u, wu) <= R.tolerance(dtype, 1, H)
    _between(hq, wh, form, 2 * R.tolerance("f32", 1, H) + 8 * 2.0 ** -24 * (1 + float(wh.abs().max())))
    want = M.ffn(val(hq), wv, _lift(u), "silu", form)
    assert R.worst(y, want) <= M.tolerance(dtype, I, form) + M.flips(dtype, H, form)


@pytest.mark.parametrize("T", [1, 50, 300])
@pytest.mark.parametrize("form", FORMS)
def test_repeats_streams_and_graphs_agree(form, T):
    run, outs, _ = _together("bf16", form, T, 1024, 264)
    run()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.fill_(77)
    side.wait_stream(torch.cuda.current_stream())
    run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in outs:
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))


@pytest.mark.parametrize("form", FORMS)
def test_a_large_workspace_serves_smaller_batches(form):
    H, I, most = 640, 300, 600
    lcfg, fcfg = moe.make_mx_linear_cfg(H, I, "silu", "bf16", form), moe.make_mx_ffn_cfg(H, I, "silu", "bf16", form)
    lws, fws = moe.alloc_mx_linear_workspace(lcfg, most, DEV), moe.alloc_mx_ffn_workspace(fcfg, most, DEV)
    w, _ = _ffn_weights(H, I, 2)
    for T in (600, 1, 17, 64, 65, 130, 400):
        x, _ = _matrix(T, H, form, T)
        own = moe.alloc_mx_linear_workspace(lcfg, T, DEV), moe.alloc_mx_ffn_workspace(fcfg, T, DEV)
        y, z = [_out("bf16", T, I) for _ in range(2)], [_out("bf16", T, H) for _ in range(2)]
        for k, (a, b) in enumerate(((lws, fws), own)):
            a.fill_(255)
            b.fill_(255)
            moe.mx_linear_forward(lcfg, x, w["w_gate"], y[k], a)
            moe.mx_ffn_forward(fcfg, x, w, z[k], b)
        assert torch.equal(y[0], y[1]) and torch.equal(z[0], z[1]) and torch.isfinite(z[0]).all()


def test_no_tokens():
    for form in FORMS:
        x, y = moe.alloc_mx(0, 64, form, DEV), torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
        w, _ = _ffn_weights(64, 64, 2)
        lcfg, fcfg = moe.make_mx_linear_cfg(64, 64, form=form), moe.make_mx_ffn_cfg(64, 64, form=form)
        moe.mx_quantize(y, x)
        moe.mx_dequantize(x, y)
        moe.norm_mx_forward(moe.make_norm_cfg(64), y, y, {"w_pre": _rand("bf16", 64)}, y, x)
        moe.mx_linear_forward(lcfg, x, w["w_gate"], y, moe.alloc_mx_linear_workspace(lcfg, 0, DEV))
        moe.mx_ffn_forward(fcfg, x, w, y, moe.alloc_mx_ffn_workspace(fcfg, 0, DEV))


# ---------------------------------------------------------------- past 32 bits

def _tiled(base, times):
    return base.expand(times, *base.shape).reshape(times * base.shape[0], -1)


def test_more_threads_than_a_grid_has():
    rows, times, cols = 1024, 1 << 14, 1032                             # a workgroup a row, 2^24 of them
    base = _rand("bf16", rows, cols, seed=5)
    small = Guarded(rows, cols, "e2m1")
    moe.mx_quantize(base, small.m)
    values = _out("bf16", rows, cols)
    moe.mx_dequantize(small.m, values)
    x = _tiled(base, times)
    out = moe.alloc_mx(rows * times, cols, "e2m1", DEV)
    out.codes.fill_(0xa5)
    moe.mx_quantize(x, out)
    assert bool((out.codes.view(times, rows, -1) == small.m.codes).all())
    assert bool((out.scales.view(times, rows, -1) == small.m.scales).all())
    x.zero_()
    moe.mx_dequantize(out, x)
    assert bool((x.view(times, rows, cols) == values).all())
    del x, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form", FORMS)
def test_offsets_past_32_bits(form):
    big = 16 if form == "e4m3" else 4
    # an output of 2.4e9 elements
    (x, xv), (w, wv) = _whole(1000, 128, form, 1, big), _whole(4100, 128, "e2m1", 2, 4)
    cfg = moe.make_mx_linear_cfg(128, 4100, "none", "bf16", form)
    full = moe.MxMatrix(_tiled(x.codes, 600), _tiled(x.scales, 600), form, 128)
    y = _out("bf16", 600000, 4100)
    moe.mx_linear_forward(cfg, full, w, y, moe.alloc_mx_linear_workspace(cfg, 600000, DEV))
    assert bool((y.view(600, 1000, 4100) == (xv @ wv.T).bfloat16().to(DEV)).all())
    del y, full
    # operands of 5e9 bytes
    T = 40000 if form == "e4m3" else 80000
    (x, xv), (w, wv) = _whole(100, 131072, form, 1, 4), _whole(24, 131072, "e2m1", 2, 4)
    cfg = moe.make_mx_linear_cfg(131072, 24, "none", "f32", form)
    full = moe.MxMatrix(_tiled(x.codes, T // 100), _tiled(x.scales, T // 100), form, 131072)
    y = _out("f32", T, 24)
    moe.mx_linear_forward(cfg, full, w, y, moe.alloc_mx_linear_workspace(cfg, T, DEV))
    assert bool((y.view(T // 100, 100, 24) == (xv @ wv.T).float().to(DEV)).all())
    del y, full
    # a middle, and a norm's output, of 5e9 elements
    (x, _), (w, _) = _whole(1000, 128, form, 1, big), _ffn_weights(128, 16384, 2)
    cfg = moe.make_mx_ffn_cfg(128, 16384, "silu", "bf16", form)
    full = moe.MxMatrix(_tiled(x.codes, 300), _tiled(x.scales, 300), form, 128)
    y = _out("bf16", 300000, 128)
    moe.mx_ffn_forward(cfg, full, w, y, moe.alloc_mx_ffn_workspace(cfg, 300000, DEV))
    assert bool((y.view(300, 1000, 128) == y[:1000]).all()) and bool(torch.isfinite(y[:1000]).all())
    r, params = _rand("bf16", 1000, 16384, seed=3), {"w_pre": _rand("bf16", 16384, seed=4)}
    cfg, small = moe.make_norm_cfg(16384), moe.alloc_mx(1000, 16384, form, DEV)
    moe.norm_mx_forward(cfg, r, None, params, None, small)
    out = moe.alloc_mx(300000, 16384, form, DEV)
    moe.norm_mx_forward(cfg, _tiled(r, 300), None, params, None, out)
    assert bool((out.codes.view(300, 1000, -1) == small.codes).all())
    assert bool((out.scales.view(300, 1000, -1) == small.scales).all())
    del out, y, full
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form", FORMS)
def test_two_streams_at_once(form):
    # each with a workspace of its own, the operands shared
    T, H, I = 80, 1500, 700
    x, _ = _matrix(T, H, form, 1)
    w, _ = _ffn_weights(H, I, 2)
    cfg = moe.make_mx_ffn_cfg(H, I, "silu", "bf16", form)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [moe.alloc_mx_ffn_workspace(cfg, T, DEV) for _ in range(3)]
    y = [_out("bf16", T, H) for _ in range(3)]
    moe.mx_ffn_forward(cfg, x, w, y[2], ws[2])
    torch.cuda.synchronize()
    for _ in range(20):
        for k, s in enumerate(streams):
            moe.mx_ffn_forward(cfg, x, w, y[k], ws[k], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[2]) and torch.equal(y[1], y[2])


def test_two_graphs_share_a_workspace():
    # replayed one after the other on a stream, as calls that share a workspace are ordered
    H, I, form = 640, 300, "e4m3"
    w, _ = _ffn_weights(H, I, 2)
    cfg = moe.make_mx_ffn_cfg(H, I, "silu", "bf16", form)
    ws = moe.alloc_mx_ffn_workspace(cfg, 300, DEV)
    runs = []
    for T in (300, 9):
        x, _ = _matrix(T, H, form, T)
        y, want = _out("bf16", T, H), _out("bf16", T, H)
        moe.mx_ffn_forward(cfg, x, w, want, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.mx_ffn_forward(cfg, x, w, y, ws)
        runs.append((g, x, y, want))
    for _ in range(3):
        for g, _, y, _ in runs:
            y.fill_(77)
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for _, _, y, want in runs)
