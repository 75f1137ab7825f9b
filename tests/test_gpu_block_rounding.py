"""How many bits float32 products keep whose operands fill all of their split parts."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda"


def say(msg):
    print(msg, flush=True)


# A contraction of one element: the split's parts (8 bits each, rounded to nearest) leave out two pairs of
# at most 2^-25 of the product each, and of its six terms, added smallest first, only the last sum is of
# the product's own size: 2^-24 + 2^-23 if that sum is truncated, and less than 2^-22 in all.
@pytest.mark.parametrize("T,N", [(4, 40), (100, 80), (2050, 2050)])
def test_float32_products_of_full_parts(T, N):
    say(f"single float32 products T={T} N={N}")
    g = torch.Generator().manual_seed(T)
    # values just below and above a multiple of the first part's unit, of the second's and of both, and any
    base = torch.tensor([1 + 2 ** -7 - 2 ** -23, 1 + 2 ** -8 + 2 ** -9 - 2 ** -23, 1 + 2 ** -8 - 2 ** -23,
                         1 + 2 ** -8 + 2 ** -16 + 2 ** -17 - 2 ** -23, 2 - 2 ** -23, 1 + 2 ** -16 - 2 ** -23,
                         1 + 2 ** -15 - 2 ** -23], dtype=torch.float32)

    def column(n):
        v = base[torch.randint(0, len(base), (n,), generator=g)]
        v[::3] = 1 + torch.rand(v[::3].shape, generator=g)
        e = torch.randint(-12, 13, (n,), generator=g).float()
        s = torch.randint(0, 2, (n,), generator=g).float() * 2 - 1
        return (v * torch.exp2(e) * s)[:, None].to(DEV)

    x, w = column(T), column(N)
    cfg = moe.make_linear_cfg(1, N, "none", "f32")
    y = torch.empty((T, N), device=DEV)
    moe.linear_forward(cfg, x, w, y, moe.alloc_linear_workspace(cfg, T, DEV))
    want = x.double() @ w.double().t()
    assert ((y.double() - want) / want).abs().max().item() < 2.0 ** -22
