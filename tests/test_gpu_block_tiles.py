"""Projections and the gated feed-forward block at sizes where a product has more tiles than the chip
has compute units, so that the larger tiles run: whole tiles and ragged ones, every epilogue, both
types, against the plain forms in 64 bits."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests import block_reference as R
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [  # T, in, out
    (2050, 1034, 2050), (4096, 520, 8192), (4100, 2056, 7001),
]


def say(msg):
    print(msg, flush=True)


def _rand(dtype, *shape, seed, scale=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(TYPES[dtype])


def _rows(t, pad):
    """The same rows as columns of a wider tensor whose others are NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _nan_like(t):
    return torch.full(t.shape, float("nan"), dtype=t.dtype, device=DEV)


def _lift(v):
    return None if v is None else v.double()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear_forward_of_many_tiles(dtype, T, K, N):
    x, w = _rand(dtype, T, K, seed=1), _rand(dtype, N, K, seed=2, scale=K ** -0.5)
    b, r = _rand(dtype, N, seed=3), _rows(_rand(dtype, T, N, seed=4), 6)
    for act, bias, res in (("none", None, r), ("gelu", b, r), ("silu", b, None), ("none", None, None)):
        say(f"linear {dtype} T={T} K={K} N={N} {act} bias={bias is not None} residual={res is not None}")
        cfg = moe.make_linear_cfg(K, N, act, dtype)
        y = torch.full((T, N), float("nan"), dtype=TYPES[dtype], device=DEV)
        moe.linear_forward(cfg, x, w, y, moe.alloc_linear_workspace(cfg, T, DEV), bias=bias, residual=res)
        want = R.linear(_lift(x), _lift(w), _lift(bias), _lift(res), act)
        err = R.worst(y, want)
        assert err <= R.tolerance(dtype, 1, K), (act, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear_backward_of_many_tiles(dtype, T, K, N):
    x, w = _rand(dtype, T, K, seed=1), _rand(dtype, N, K, seed=2, scale=K ** -0.5)
    b, dy = _rand(dtype, N, seed=3), _rows(_rand(dtype, T, N, seed=4), 6)
    for act, bias in (("none", None), ("silu", b)):
        say(f"linear backward {dtype} T={T} K={K} N={N} {act}")
        cfg = moe.make_linear_cfg(K, N, act, dtype)
        dx, dw, db = _nan_like(x), _nan_like(w), _nan_like(b)
        moe.linear_backward(cfg, x, w, dy, moe.alloc_linear_backward_workspace(cfg, T, DEV), bias=bias, dx=dx, dw=dw,
                            dbias=db)
        want = R.linear_grads(_lift(x), _lift(w), _lift(bias), _lift(dy), act)
        for name, got, terms in (("dx", dx, K + N), ("dw", dw, K + T), ("dbias", db, K + T)):
            err = R.worst(got, want[name])
            assert err <= R.tolerance(dtype, 2, terms), (act, name, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", [(2050, 1034, 520), (4100, 2056, 2049)])
def test_ffn_of_many_tiles(dtype, T, H, I):
    x, dy = _rand(dtype, T, H, seed=1), _rand(dtype, T, H, seed=2)
    w = {"w_gate": _rand(dtype, I, H, seed=3, scale=H ** -0.5), "w_up": _rand(dtype, I, H, seed=4, scale=H ** -0.5),
         "w_down": _rand(dtype, H, I, seed=5, scale=I ** -0.5)}
    lifted = {k: _lift(v) for k, v in w.items()}
    cfg = moe.make_ffn_cfg(H, I, "silu", dtype)
    say(f"ffn {dtype} T={T} H={H} I={I}")
    y = _nan_like(x)
    moe.ffn_forward(cfg, x, w, y, moe.alloc_ffn_workspace(cfg, T, DEV), residual=dy)
    err = R.worst(y, R.ffn(_lift(x), lifted, _lift(dy), "silu"))
    assert err <= R.tolerance(dtype, 2, H + I), err
    say(f"ffn backward {dtype} T={T} H={H} I={I}")
    dx, dw = _nan_like(x), {k: _nan_like(v) for k, v in w.items()}
    moe.ffn_backward(cfg, x, w, dy, dx, dw["w_gate"], dw["w_up"], dw["w_down"],
                     moe.alloc_ffn_backward_workspace(cfg, T, DEV))
    want = R.ffn_grads(_lift(x), lifted, _lift(dy), "silu")
    for name, got in (("dx", dx), *dw.items()):
        err = R.worst(got, want[name])
        assert err <= R.tolerance(dtype, 2, 2 * H + I + T), (name, err)
