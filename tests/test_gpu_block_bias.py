"""Bias gradients of projections with an activation: sums, and no operands of a later product, so nothing
in them is rounded to bfloat16 before the end."""
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


# The sum of T float32 values, rounded once: half a unit of the result (2^-8 of it at most) and what float32
# itself loses.  That is: z's sums are off by at most K 2^-24 of about 1, the slope and the product by some
# 2^-22 of theirs, and sums over the rows (in pieces of at most some hundred) by 2^-17, all together below
# 1e-4 of the terms' 2-norm.  Rounding every term to bfloat16 first is off by 1.6e-3 of it.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,K,N", [(3, 40, 24), (70, 512, 48), (300, 64, 256), (520, 1024, 320), (2050, 136, 1034),
                                   (4096, 512, 256), (4096, 64, 8192), (8191, 72, 2050)])
def test_bias_gradient_is_rounded_once(dtype, act, T, K, N):
    say(f"bias gradient {dtype} {act} T={T} K={K} N={N}")
    g = torch.Generator(DEV).manual_seed(T + K)
    rand = lambda *shape, scale=1.0: (torch.randn(shape, generator=g, device=DEV) * scale).to(TYPES[dtype])  # noqa: E731
    x, w, b, dy = rand(T, K), rand(N, K, scale=K ** -0.5), rand(N, scale=0.5), rand(T, N)
    cfg = moe.make_linear_cfg(K, N, act, dtype)
    ws = moe.alloc_linear_backward_workspace(cfg, T, DEV)
    for bias in (b, None):
        db = torch.full((N,), float("nan"), dtype=TYPES[dtype], device=DEV)
        moe.linear_backward(cfg, x, w, dy, ws, bias=bias, dbias=db)
        z = x.double() @ w.double().t() + (0 if bias is None else bias.double())
        dz = dy.double() * R.act_slope(act, z)
        want, size = dz.sum(0), dz.square().sum(0).sqrt()
        off = (db.double() - want).abs()
        assert (off <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * want.abs() + 1e-4 * size).all()
        # the same beside the other gradients, and again
        dx, dw, again = torch.empty_like(x), torch.empty_like(w), torch.empty_like(db)
        moe.linear_backward(cfg, x, w, dy, ws, bias=bias, dx=dx, dw=dw, dbias=again)
        assert torch.equal(again, db)
