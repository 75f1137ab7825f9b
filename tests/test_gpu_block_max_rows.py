"""A projection of 2^24 tokens, the most that are accepted, whose rows have to be laid out anew: more pieces of
work than one dimension of a grid has threads, and offsets far past 32 bits."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests import block_reference as R
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_linear_of_the_most_tokens():
    T, K, N = 1 << 24, 2047, 4
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of free device memory")
    print(f"linear bf16 T={T} K={K} N={N}", flush=True)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    cfg = moe.make_linear_cfg(K, N)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.linear_forward(cfg, x, w, y, moe.alloc_linear_workspace(cfg, T, "cuda"))
    rows = torch.cat([torch.arange(64), torch.randint(0, T, (2048,), generator=torch.Generator().manual_seed(2)),
                      torch.arange((1 << 22) - 32, (1 << 22) + 32), torch.arange(T - 64, T)])
    rows = rows.to("cuda")
    assert R.worst(y[rows], R.linear(x[rows].double(), w.double()).cpu()) <= R.tolerance("bf16", 1, K)
    assert torch.isfinite(y).all()
    del x, y
    torch.cuda.empty_cache()
