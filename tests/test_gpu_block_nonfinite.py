"""NaN in the operands of projections and feed-forward blocks: it comes out where float32 arithmetic has it
and nowhere else, whatever the activation, on the streaming route, on whole and ragged tiles and behind a
split contraction."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")
SIZES = [  # T, in, out: streamed; small tiles, split and ragged; small tiles; large tiles, ragged
    (5, 200, 40), (70, 512, 48), (300, 64, 256), (2050, 136, 1034), (4096, 64, 4096),
]
ACTS = ["none", "relu", "silu", "gelu"]


def say(msg):
    print(msg, flush=True)


def _rand(dtype, *shape, seed, scale=1.0):
    v = torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    # no element so small that its products vanish
    v = torch.where(v < 0, v - 0.1, v + 0.1) * scale
    return v.to(TYPES[dtype]).to(DEV)


def _linear(dtype, T, K, N, act, x, w, b=None, r=None):
    cfg = moe.make_linear_cfg(K, N, act, dtype)
    y = torch.empty((T, N), dtype=TYPES[dtype], device=DEV)
    moe.linear_forward(cfg, x, w, y, moe.alloc_linear_workspace(cfg, T, DEV), bias=b, residual=r)
    return y


def _at(*places, shape):
    m = torch.zeros(shape, dtype=torch.bool, device=DEV)
    for p in places:
        m[p] = True
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_nan_passes_every_activation(dtype, act, T, K, N):
    say(f"NaN through linear {dtype} {act} T={T} K={K} N={N}")
    x, w, b = _rand(dtype, T, K, seed=1), _rand(dtype, N, K, seed=2, scale=K ** -0.5), _rand(dtype, N, seed=3)
    clean = _linear(dtype, T, K, N, act, x, w, b)
    assert torch.isfinite(clean).all()
    x[3, 5] = NAN
    w[17, 7] = NAN
    b[N - 1] = NAN
    y = _linear(dtype, T, K, N, act, x, w, b)
    bad = _at(3, (slice(None), 17), (slice(None), N - 1), shape=(T, N))
    assert torch.isnan(y[bad]).all()
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("T,K,N", SIZES)
def test_nan_with_low_bits_alone(T, K, N):
    # a NaN whose upper half is infinity's
    x, w = _rand("f32", T, K, seed=1), _rand("f32", N, K, seed=2, scale=K ** -0.5)
    x.view(torch.int32)[2, 1] = 0x7f800001
    w.view(torch.int32)[1, 0] = -0x7fffff  # the same, negative
    y = _linear("f32", T, K, N, "relu", x, w)
    bad = _at(2, (slice(None), 1), shape=(T, N))
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("T,H,I", [(5, 200, 40), (70, 512, 48), (2050, 136, 1034)])
def test_ffn_nan_in_a_gate_weight(dtype, act, T, H, I):
    say(f"NaN through ffn {dtype} {act} T={T} H={H} I={I}")
    x, cfg = _rand(dtype, T, H, seed=1), moe.make_ffn_cfg(H, I, act, dtype)
    w = {"w_gate": _rand(dtype, I, H, seed=2, scale=H ** -0.5), "w_up": _rand(dtype, I, H, seed=3, scale=H ** -0.5),
         "w_down": _rand(dtype, H, I, seed=4, scale=I ** -0.5)}
    w["w_gate"][33, 7] = NAN
    y = torch.empty_like(x)
    moe.ffn_forward(cfg, x, w, y, moe.alloc_ffn_workspace(cfg, T, DEV))
    assert torch.isnan(y).all()
    dx, dw = torch.empty_like(x), {k: torch.empty_like(v) for k, v in w.items()}
    moe.ffn_backward(cfg, x, w, y.fill_(1.0), dx, *dw.values(), moe.alloc_ffn_backward_workspace(cfg, T, DEV))
    assert torch.isnan(dx).all() and torch.isnan(dw["w_gate"][33]).all() and torch.isnan(dw["w_down"][:, 33]).all()
    assert torch.isfinite(dw["w_gate"][:33]).all() and torch.isfinite(dw["w_down"][:, :33]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_nan_passes_the_slope_of_relu(dtype, T, K, N):
    say(f"NaN through linear backward {dtype} T={T} K={K} N={N}")
    x, w, b = _rand(dtype, T, K, seed=1), _rand(dtype, N, K, seed=2, scale=K ** -0.5), _rand(dtype, N, seed=3)
    dy, cfg = _rand(dtype, T, N, seed=4), moe.make_linear_cfg(K, N, "relu", dtype)
    b[17] = NAN
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    moe.linear_backward(cfg, x, w, dy, moe.alloc_linear_backward_workspace(cfg, T, DEV), bias=b, dx=dx, dw=dw,
                        dbias=db)
    assert torch.isnan(dx).all() and torch.isnan(dw[17]).all() and torch.isnan(db[17])
    keep = torch.arange(N, device=DEV) != 17
    assert torch.isfinite(dw[keep]).all() and torch.isfinite(db[keep]).all()
