"""The operators around the expert layer on the GPU against plain 64-bit forms, through the C ABI's
binding: sizes from one token and one column on, sizes and strides that nothing divides, absent
parts, every activation and type; determinism, overwritten outputs and graph replays."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests import block_reference as R
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


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
    """What lies between the rows of an output that is a slice was not written."""
    base = t._base
    return base is None or base.shape[1] == t.shape[1] or bool(torch.isnan(base[:, t.shape[1]:]).all())


def _lift(v):
    return None if v is None else v.detach().cpu().double()


def _lifted(d):
    return {k: _lift(v) for k, v in d.items()}


# ---------------------------------------------------------------- linear

LINEAR = [  # T, in, out, pad
    (1, 1, 1, 0), (1, 64, 16, 0), (1, 1001, 777, 3), (3, 7, 1030, 0), (7, 256, 130, 8), (16, 2048, 640, 0),
    (17, 130, 33, 1), (33, 1000, 264, 0), (64, 512, 256, 8), (65, 72, 8, 0), (128, 64, 128, 0), (129, 1033, 257, 5),
    (300, 1024, 256, 0), (1000, 200, 520, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,pad", LINEAR)
def test_linear_forward(dtype, T, K, N, pad):
    for i, (act, bias, res) in enumerate((("none", False, False), ("gelu", True, True), ("silu", True, False),
                                          ("relu", False, True))):
        say(f"linear {dtype} T={T} K={K} N={N} pad={pad} {act}")
        x, w = _rows(dtype, T, K, pad, i), _rand(dtype, N, K, seed=10 + i, scale=K ** -0.5)
        b = _rand(dtype, N, seed=20 + i) if bias else None
        r = _rows(dtype, T, N, pad, 30 + i) if res else None
        cfg = moe.make_linear_cfg(K, N, act, dtype)
        y, ws = _out(dtype, T, N, pad), moe.alloc_linear_workspace(cfg, T, DEV)
        moe.linear_forward(cfg, x, w, y, ws, bias=b, residual=r)
        want = R.linear(_lift(x), _lift(w), _lift(b), _lift(r), act)
        assert R.worst(y, want) <= R.tolerance(dtype, 1, K), (act, R.worst(y, want))
        assert _pads_kept(y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,pad", LINEAR)
def test_linear_backward(dtype, T, K, N, pad):
    for i, (act, bias) in enumerate((("none", False), ("gelu", True), ("silu", False))):
        say(f"linear backward {dtype} T={T} K={K} N={N} pad={pad} {act}")
        x, w = _rows(dtype, T, K, pad, i), _rand(dtype, N, K, seed=10 + i, scale=K ** -0.5)
        b, dy = (_rand(dtype, N, seed=20 + i) if bias else None), _rows(dtype, T, N, pad, 40 + i)
        cfg = moe.make_linear_cfg(K, N, act, dtype)
        ws = moe.alloc_linear_backward_workspace(cfg, T, DEV)
        dx, dw, db = _out(dtype, T, K, pad), _out(dtype, N, K), _out(dtype, 1, N)[0]
        moe.linear_backward(cfg, x, w, dy, ws, bias=b, dx=dx, dw=dw, dbias=db)
        want = R.linear_grads(_lift(x), _lift(w), _lift(b), _lift(dy), act)
        for name, got, terms in (("dx", dx, K + N), ("dw", dw, K + T), ("dbias", db, K + T)):
            assert R.worst(got, want[name]) <= R.tolerance(dtype, 2, terms), (act, name, R.worst(got, want[name]))
        assert _pads_kept(dx)
        # each gradient alone
        for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
            alone = torch.full_like(got, float("nan"))
            moe.linear_backward(cfg, x, w, dy, ws, bias=b, **{name: alone})
            assert torch.equal(alone, got), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_relu_backward(dtype):
    # sums of small whole numbers are exact, so both sides see the same signs (zeros included)
    T, K, N = 70, 24, 40
    gen = torch.Generator().manual_seed(5)
    x = torch.randint(-2, 3, (T, K), generator=gen).to(TYPES[dtype]).to(DEV)
    w = torch.randint(-2, 3, (N, K), generator=gen).to(TYPES[dtype]).to(DEV)
    dy = _rand(dtype, T, N, seed=6)
    cfg = moe.make_linear_cfg(K, N, "relu", dtype)
    dx, dw, db = _out(dtype, T, K), _out(dtype, N, K), _out(dtype, 1, N)[0]
    moe.linear_backward(cfg, x, w, dy, moe.alloc_linear_backward_workspace(cfg, T, DEV), dx=dx, dw=dw, dbias=db)
    want = R.linear_grads(_lift(x), _lift(w), None, _lift(dy), "relu")
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
        assert R.worst(got, want[name]) <= R.tolerance(dtype, 2, T), name


def test_linear_of_unaligned_tensors():
    # rows whose first element is aligned to itself alone
    T, K, N = 40, 64, 48
    cfg = moe.make_linear_cfg(K, N)
    flat = _rand("bf16", T * K + N * K + 3, seed=1)
    x, w = flat[1:1 + T * K].view(T, K), flat[3 + T * K:].view(N, K)
    y = _out("bf16", T, N)
    moe.linear_forward(cfg, x, w, y, moe.alloc_linear_workspace(cfg, T, DEV))
    assert R.worst(y, R.linear(_lift(x), _lift(w))) <= R.tolerance("bf16", 1, K)


def test_linear_into_its_residual():
    T, K, N = 150, 512, 256
    cfg = moe.make_linear_cfg(K, N)
    x, w, r = _rand("bf16", T, K), _rand("bf16", N, K, seed=1, scale=K ** -0.5), _rand("bf16", T, N, seed=2)
    want = R.linear(_lift(x), _lift(w), None, _lift(r))
    moe.linear_forward(cfg, x, w, r, moe.alloc_linear_workspace(cfg, T, DEV), residual=r)
    assert R.worst(r, want) <= R.tolerance("bf16", 1, K)


def test_linear_extreme_values():
    # the largest and smallest values of the type pass through every part of the split unharmed
    K, N = 64, 16
    cfg = moe.make_linear_cfg(K, N, "none", "f32")
    x = torch.zeros((2, K), device=DEV)
    x[0, 3], x[1, 5] = 3.0e38, 1.1754944e-30
    w = torch.zeros((N, K), device=DEV)
    w[:, 3], w[:, 5] = 1.0, 3.0
    y = _out("f32", 2, N)
    moe.linear_forward(cfg, x, w, y, moe.alloc_linear_workspace(cfg, 2, DEV))
    want = R.linear(_lift(x), _lift(w))
    assert torch.allclose(y.cpu().double(), want, rtol=2 ** -22, atol=0)


# ---------------------------------------------------------------- ffn

FFN = [  # T, hidden, inter, pad
    (1, 1, 1, 0), (1, 256, 128, 0), (1, 1001, 333, 3), (2, 64, 520, 0), (9, 130, 66, 1), (16, 1024, 256, 0),
    (31, 96, 200, 8), (64, 512, 192, 0), (100, 1033, 129, 5), (300, 1024, 256, 0), (520, 136, 264, 8),
]


def _ffn_weights(dtype, H, I, seed):
    return {"w_gate": _rand(dtype, I, H, seed=seed, scale=H ** -0.5),
            "w_up": _rand(dtype, I, H, seed=seed + 1, scale=H ** -0.5),
            "w_down": _rand(dtype, H, I, seed=seed + 2, scale=I ** -0.5)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,pad", FFN)
def test_ffn_forward(dtype, T, H, I, pad):
    for i, (act, res) in enumerate((("silu", True), ("gelu", False), ("relu", True))):
        say(f"ffn {dtype} T={T} H={H} I={I} pad={pad} {act}")
        x, w = _rows(dtype, T, H, pad, i), _ffn_weights(dtype, H, I, 50 + 3 * i)
        r = _rows(dtype, T, H, pad, 30 + i) if res else None
        cfg = moe.make_ffn_cfg(H, I, act, dtype)
        y = _out(dtype, T, H, pad)
        moe.ffn_forward(cfg, x, w, y, moe.alloc_ffn_workspace(cfg, T, DEV), residual=r)
        want = R.ffn(_lift(x), _lifted(w), _lift(r), act)
        assert R.worst(y, want) <= R.tolerance(dtype, 2, H + I), (act, R.worst(y, want))
        assert _pads_kept(y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,pad", FFN)
def test_ffn_backward(dtype, T, H, I, pad):
    for i, act in enumerate(("silu", "gelu")):
        say(f"ffn backward {dtype} T={T} H={H} I={I} pad={pad} {act}")
        x, dy, w = _rows(dtype, T, H, pad, i), _rows(dtype, T, H, pad, 7 + i), _ffn_weights(dtype, H, I, 50 + 3 * i)
        cfg = moe.make_ffn_cfg(H, I, act, dtype)
        dx = _out(dtype, T, H, pad)
        dw = {k: torch.full_like(v, float("nan")) for k, v in w.items()}
        moe.ffn_backward(cfg, x, w, dy, dx, dw["w_gate"], dw["w_up"], dw["w_down"],
                         moe.alloc_ffn_backward_workspace(cfg, T, DEV))
        want = R.ffn_grads(_lift(x), _lifted(w), _lift(dy), act)
        for name, got in (("dx", dx), *dw.items()):
            err = R.worst(got, want[name])
            assert err <= R.tolerance(dtype, 2, 2 * H + I + T), (act, name, err)
        assert _pads_kept(dx)


def test_ffn_with_one_unaligned_projection():
    T, H, I = 20, 64, 72
    cfg = moe.make_ffn_cfg(H, I)
    w = _ffn_weights("bf16", H, I, 3)
    moved = torch.empty(I * H + 1, dtype=torch.bfloat16, device=DEV)[1:].view(I, H)
    x = _rand("bf16", T, H)
    want = R.ffn(_lift(x), _lifted(w))
    for name in ("w_gate", "w_up"):
        moved.copy_(w[name])
        y = _out("bf16", T, H)
        moe.ffn_forward(cfg, x, {**w, name: moved}, y, moe.alloc_ffn_workspace(cfg, T, DEV))
        assert R.worst(y, want) <= R.tolerance("bf16", 2, H + I), name


# ---------------------------------------------------------------- norm

NORM = [  # T, hidden, pad, gate_rows
    (1, 1, 0, 1), (1, 64, 0, 0), (5, 3, 1, 5), (9, 512, 0, 3), (40, 513, 3, 1), (64, 1000, 8, 16), (30, 1024, 0, 30),
    (33, 1025, 0, 11), (700, 1030, 2, 7), (600, 2048, 0, 200), (300, 7168, 0, 300), (515, 4100, 4, 103),
    (20, 8192, 0, 4), (7, 8200, 1, 7), (6, 16384, 0, 2), (21, 256, 3, 7), (12, 1536, 5, 4), (1100, 72, 1, 1100),
]


def _norm_inputs(dtype, T, H, pad, gate_rows, kind, seed=0, post=True, outliers=True):
    r, f = _rows(dtype, T, H, pad, seed, 2.0), _rows(dtype, T, H, pad, seed + 1, 0.5)
    if outliers:
        r[:, H // 2] *= 16
    p = {"w_pre": _rand(dtype, H, seed=seed + 2, scale=0.1, shift=1.0)}
    if post:
        p["w_post"] = _rand(dtype, H, seed=seed + 3, scale=0.1, shift=1.0)
    if kind == "layer":
        p["b_pre"] = _rand(dtype, H, seed=seed + 4)
        if post:
            p["b_post"] = _rand(dtype, H, seed=seed + 5)
    if gate_rows:
        p["gate"] = _rand(dtype, T // gate_rows, H, seed=seed + 6)
    return r, f, p


def _norm_tol(dtype, H):
    # float32: sums of H terms, 8 a thread and then tree-wise, twice over
    return R.tolerance("bf16", 1, H) if dtype == "bf16" else 64 * 2.0 ** -24


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,pad,gate_rows", NORM)
def test_norm_forward(dtype, kind, T, H, pad, gate_rows):
    if kind == "layer" and H == 1:
        pytest.skip("a row of one is its own mean")
    for post in (True, False):
        say(f"norm {dtype} {kind} T={T} H={H} pad={pad} gate_rows={gate_rows} post={post}")
        r, f, p = _norm_inputs(dtype, T, H, pad, gate_rows, kind, post=post)
        cfg = moe.make_norm_cfg(H, dtype, kind, gate_rows, 1e-6, 0.75)
        u, h = _out(dtype, T, H, pad), _out(dtype, T, H, pad)
        moe.norm_forward(cfg, r, f, p, u, h)
        wu, wh = R.norm(_lift(r), _lift(f), _lifted(p), kind, 1e-6, 0.75)
        assert R.worst(u, wu) <= _norm_tol(dtype, H), ("u", R.worst(u, wu))
        assert R.worst(h, wh) <= _norm_tol(dtype, H), ("h", R.worst(h, wh))
        assert _pads_kept(u) and _pads_kept(h)
    # parts left out
    u2, h2 = torch.empty_like(u), torch.empty_like(h)
    moe.norm_forward(cfg, r, f, p, u2, None)
    moe.norm_forward(cfg, r, f, p, None, h2)
    assert torch.equal(u2, u) and torch.equal(h2, h)
    cfg = moe.make_norm_cfg(H, dtype, kind)
    moe.norm_forward(cfg, r, None, {k: v for k, v in p.items() if k.endswith("_pre")}, u, h)
    wu, wh = R.norm(_lift(r), None, _lifted(p), kind)
    assert torch.equal(u, r) and R.worst(h, wh) <= _norm_tol(dtype, H)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,pad,gate_rows", NORM)
def test_norm_backward(dtype, kind, T, H, pad, gate_rows):
    if H == 1:
        pytest.skip("the unit of a row of one is constant: its gradient is rounding alone")
    for post, use_du, use_dh in ((True, True, True), (False, True, True), (True, False, True), (True, True, False)):
        say(f"norm backward {dtype} {kind} T={T} H={H} pad={pad} gate_rows={gate_rows} post={post} {use_du}{use_dh}")
        r, f, p = _norm_inputs(dtype, T, H, pad, gate_rows, kind, post=post)
        du = _rows(dtype, T, H, pad, 80) if use_du else None
        dh = _rows(dtype, T, H, pad, 81) if use_dh else None
        cfg = moe.make_norm_cfg(H, dtype, kind, gate_rows, 1e-6, 0.75)
        g = {k: torch.full_like(v, float("nan")) for k, v in p.items() if use_dh or not k.endswith("_pre")}
        g["residual"], g["branch"] = _out(dtype, T, H, pad), _out(dtype, T, H, pad)
        ws = moe.alloc_norm_backward_workspace(cfg, T, DEV)
        moe.norm_backward(cfg, r, f, p, du, dh, g, ws)
        want = R.norm_grads(_lift(r), _lift(f), _lifted(p), _lift(du), _lift(dh), kind, 1e-6, 0.75)
        for k, got in g.items():
            err = R.worst(got, want[k])
            assert err <= _norm_tol(dtype, H) * (1 if dtype == "bf16" else 4), (k, err)
        assert _pads_kept(g["residual"]) and _pads_kept(g["branch"])
        again = {k: torch.empty_like(v) for k, v in g.items()}
        moe.norm_backward(cfg, r, f, p, du, dh, again, ws)
        assert all(torch.equal(again[k], g[k]) for k in g)


def test_norm_of_zero_and_offset_rows():
    # an all-zero row stays zero; a row far from zero keeps its layer norm
    H = 1024
    r = torch.zeros((3, H), device=DEV)
    r[1] = 1000.0 + torch.linspace(-1, 1, H, device=DEV)
    cfg = moe.make_norm_cfg(H, "f32", "layer", eps=1e-6)
    p = {"w_pre": torch.ones(H, device=DEV)}
    h = _out("f32", 3, H)
    moe.norm_forward(cfg, r, None, p, None, h)
    _, want = R.norm(_lift(r), None, _lifted(p), "layer", 1e-6)
    assert torch.equal(h[0], torch.zeros_like(h[0])) and torch.equal(h[2], h[0])
    # the row's own float32 spacing is 6e-5 of its deviations: 2^-24 * 1000 / 0.58 for the mean
    assert R.worst(h, want) <= 2 * 2.0 ** -24 * 1000 / 0.58


def test_norm_in_place():
    T, H = 37, 1536
    cfg = moe.make_norm_cfg(H, "bf16", "rms", T, 1e-6, 0.5)
    r, f, p = _norm_inputs("bf16", T, H, 0, T, "rms")
    u, h = _out("bf16", T, H), _out("bf16", T, H)
    moe.norm_forward(cfg, r, f, p, u, h)
    r2, f2 = r.clone(), f.clone()
    moe.norm_forward(cfg, r2, f2, p, r2, f2)
    assert torch.equal(r2, u) and torch.equal(f2, h)
    du, dh = _rand("bf16", T, H, seed=8), _rand("bf16", T, H, seed=9)
    g = {"residual": _out("bf16", T, H), "branch": _out("bf16", T, H)}
    ws = moe.alloc_norm_backward_workspace(cfg, T, DEV)
    moe.norm_backward(cfg, r, f, p, du, dh, g, ws)
    moe.norm_backward(cfg, r, f, p, du, dh, {"residual": du, "branch": dh}, ws)
    assert torch.equal(du, g["residual"]) and torch.equal(dh, g["branch"])


# ---------------------------------------------------------------- all


def _block(dtype, T, H, I):
    """One call of each operator, as a function of nothing that writes its outputs."""
    r, f, p = _norm_inputs(dtype, T, H, 0, T, "rms")
    ncfg, fcfg, lcfg = moe.make_norm_cfg(H, dtype, "rms", T), moe.make_ffn_cfg(H, I, "silu", dtype), \
        moe.make_linear_cfg(H, I, "gelu", dtype)
    fw, lw = _ffn_weights(dtype, H, I, 4), _rand(dtype, I, H, seed=8, scale=H ** -0.5)
    u, h, y = (_out(dtype, T, H) for _ in range(3))
    z = _out(dtype, T, I)
    fws, lws = moe.alloc_ffn_workspace(fcfg, T, DEV), moe.alloc_linear_workspace(lcfg, T, DEV)
    bws = moe.alloc_ffn_backward_workspace(fcfg, T, DEV)
    dx, dw = _out(dtype, T, H), {k: torch.empty_like(v) for k, v in fw.items()}

    def run(stream=None):
        moe.norm_forward(ncfg, r, f, p, u, h, stream=stream)
        moe.ffn_forward(fcfg, h, fw, y, fws, residual=u, stream=stream)
        moe.linear_forward(lcfg, y, lw, z, lws, stream=stream)
        moe.ffn_backward(fcfg, h, fw, y, dx, dw["w_gate"], dw["w_up"], dw["w_down"], bws, stream=stream)

    return run, [u, h, y, z, dx, *dw.values()]


@pytest.mark.parametrize("T", [1, 50, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_streams_and_graphs_agree(dtype, T):
    run, outs = _block(dtype, T, 1024, 264)
    run()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in outs:
        t.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))


def test_no_tokens():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = _rand("bf16", 64, 64)
    lcfg, fcfg, ncfg = moe.make_linear_cfg(64, 64), moe.make_ffn_cfg(64, 64), moe.make_norm_cfg(64)
    fw = {"w_gate": w, "w_up": w, "w_down": w}
    moe.linear_forward(lcfg, x, w, x, moe.alloc_linear_workspace(lcfg, 0, DEV))
    moe.ffn_forward(fcfg, x, fw, x, moe.alloc_ffn_workspace(fcfg, 0, DEV))
    moe.norm_forward(ncfg, x, x, {"w_pre": w[0]}, x, x)
    keep = w.clone()
    moe.linear_backward(lcfg, x, w, x, moe.alloc_linear_backward_workspace(lcfg, 0, DEV), dw=keep)
    assert torch.equal(keep, w)
