"""Workspace sizes of the operators around the expert layer (host code, no GPU needed): a workspace made
for a batch serves every smaller one."""
import os

import pytest

import sparse_moe_layer_group_amd as moe

pytestmark = pytest.mark.skipif(not os.path.exists(moe.lib_path()),
                                reason="library not built (python -m sparse_moe_layer_group_amd.build)")

LINEAR = (moe.linear_workspace_bytes, moe.linear_backward_workspace_bytes)
FFN = (moe.ffn_workspace_bytes, moe.ffn_backward_workspace_bytes)


def _never_falls(f, cfg, batches):
    most = 0
    for T in batches:
        n = f(cfg, T)
        assert n >= most, (T, n, most)
        most = n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("K,N", [(256, 256), (7168, 7168), (7168, 2048), (1001, 777), (64, 16)])
def test_linear_sizes_never_fall(dtype, act, K, N):
    for f in LINEAR:
        _never_falls(f, moe.make_linear_cfg(K, N, act, dtype), range(3000))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,I", [(256, 128), (7168, 2048), (1033, 129)])
def test_ffn_sizes_never_fall(dtype, H, I):
    for f in FFN:
        _never_falls(f, moe.make_ffn_cfg(H, I, "silu", dtype), range(3000))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes_of_large_batches_never_fall(dtype):
    batches = [n + d for k in range(12, 24) for n in (1 << k, 3 << (k - 1)) for d in (-65, -1, 0, 1, 63, 64)]
    batches = sorted(b for b in batches if b <= 1 << 24) + [1 << 24]
    for K, N in ((1, 1), (131072, 1), (1, 131072), (4096, 64), (131072, 131072)):
        for f in LINEAR:
            _never_falls(f, moe.make_linear_cfg(K, N, "gelu", dtype), batches)
        for f in FFN:
            _never_falls(f, moe.make_ffn_cfg(K, N, "gelu", dtype), batches)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,gate_rows", [("rms", 0), ("layer", 1)])
def test_norm_sizes_never_fall(dtype, kind, gate_rows):
    for H in (72, 1000, 7168, 16384):
        _never_falls(moe.norm_backward_workspace_bytes, moe.make_norm_cfg(H, dtype, kind, gate_rows), range(3000))


@pytest.mark.parametrize("dtype,most", [("bf16", 16), ("f32", 64)])
@pytest.mark.parametrize("K,N", [(7168, 7168), (1001, 777)])
def test_few_tokens_need_no_copies_of_the_weights(dtype, most, K, N):
    # up to `most` tokens the weights are read where they lie; a block keeps its middle alone
    size = 2 if dtype == "bf16" else 4
    for T in (1, most):
        assert 0 < moe.linear_workspace_bytes(moe.make_linear_cfg(K, N, "gelu", dtype), T) <= 256
        assert 0 < moe.ffn_workspace_bytes(moe.make_ffn_cfg(K, N, "gelu", dtype), T) <= T * N * size + 256
    assert moe.linear_workspace_bytes(moe.make_linear_cfg(K, N, "gelu", dtype), most + 1) > K * N * 2
