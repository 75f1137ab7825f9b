"""Infinities and the largest values in the operands of projections and feed-forward blocks: sums come out
infinite with the sign that float32 arithmetic gives them, tokens and columns without one as ever."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests.conftest import gpu_available
from tests.test_gpu_block_nonfinite import ACTS, DEV, SIZES, _at, _linear, _rand, say

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

INF = float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_infinity_passes(dtype, act, T, K, N):
    say(f"infinity through linear {dtype} {act} T={T} K={K} N={N}")
    x, w = _rand(dtype, T, K, seed=1), _rand(dtype, N, K, seed=2, scale=K ** -0.5)
    clean = _linear(dtype, T, K, N, act, x, w)
    x[3, 5] = INF
    x[4, 6] = -INF
    w[17, 7] = INF
    y = _linear(dtype, T, K, N, act, x, w)
    bad = _at(3, 4, (slice(None), 17), shape=(T, N))
    assert torch.equal(y[~bad], clean[~bad])
    sign = torch.zeros((T, N), device=DEV)  # of the sums before the activation
    sign[3], sign[4] = torch.sign(w[:, 5].float()), -torch.sign(w[:, 6].float())
    sign[:, 17] = torch.sign(x[:, 7].float())
    bad[3:5, 17] = False  # infinities of both operands meet the other's sign there
    assert torch.isinf(y[bad & (sign > 0)]).all() and (y[bad & (sign > 0)] > 0).all()
    below = y[bad & (sign < 0)]
    if act == "none":
        assert torch.equal(below, torch.full_like(below, -INF))
    elif act == "relu":
        assert torch.equal(below, torch.zeros_like(below))


@pytest.mark.parametrize("T,K,N", SIZES)
def test_nan_with_low_bits_beside_an_infinity(T, K, N):
    x, w = _rand("f32", T, K, seed=1), _rand("f32", N, K, seed=2, scale=K ** -0.5)
    x.view(torch.int32)[2, 1] = 0x7f800001
    x[3, 2] = INF
    y = _linear("f32", T, K, N, "none", x, w)
    assert torch.isnan(y[2]).all() and torch.equal(y[3], torch.sign(w[:, 2]) * INF)
    bad = _at(2, 3, shape=(T, N))
    assert torch.isfinite(y[~bad]).all()


def test_largest_values():
    # above the largest bfloat16 value, where rounding its leading part up would overflow
    big = torch.finfo(torch.float32).max
    for T in (4, 100):
        x, w = torch.zeros((T, 64), device=DEV), torch.zeros((32, 64), device=DEV)
        x[:, 9], x[1, 9], x[2, 9] = big, -big, 3.3961e38
        w[:, 9] = 0.5
        y = _linear("f32", T, 64, 32, "none", x, w)
        want = x.double() @ w.double().t()
        assert torch.allclose(y.double(), want, rtol=2 ** -22, atol=0), T
        y = _linear("f32", T, 32, 64, "none", w[:1].repeat(T, 1)[:, :32].contiguous(), x[:1, :32].repeat(64, 1))
        assert torch.allclose(y.double(), torch.full_like(y, big).double() * 0.5, rtol=2 ** -22, atol=0), T


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", [(5, 200, 40), (70, 512, 48), (2050, 136, 1034)])
def test_ffn_infinity_in_a_gate_weight(dtype, T, H, I):
    # through a ReLU, tokens on its other side are as finite as ever
    x, cfg = _rand(dtype, T, H, seed=1), moe.make_ffn_cfg(H, I, "relu", dtype)
    w = {"w_gate": _rand(dtype, I, H, seed=2, scale=H ** -0.5), "w_up": _rand(dtype, I, H, seed=3, scale=H ** -0.5),
         "w_down": _rand(dtype, H, I, seed=4, scale=I ** -0.5)}
    w["w_gate"][33, 7] = INF
    y, ws = torch.empty_like(x), moe.alloc_ffn_workspace(cfg, T, DEV)
    moe.ffn_forward(cfg, x, w, y, ws)
    on = x[:, 7] > 0
    up = (x.double() @ w["w_up"][33].double())[on]
    # (an up projection this near zero may have either sign)
    clear = up.abs() > 1e-3
    want = torch.sign(up[clear])[:, None] * torch.sign(w["w_down"][:, 33].double()) * INF
    assert torch.equal(y[on][clear].double(), want)
    w["w_gate"][33, 7] = 0.0
    w["w_down"][:, 33] = 0.0
    other = torch.empty_like(x)
    moe.ffn_forward(cfg, x, w, other, ws)
    assert torch.equal(y[~on], other[~on])
