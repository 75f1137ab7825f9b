"""Buffers of the operators around the expert layer that were made for the largest batch, used by smaller
ones."""
import pytest
import torch

import sparse_moe_layer_group_amd as moe
import synthetic as S
from tests import block_reference as R
from tests import test_gpu_block_example as E
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(msg):
    print(msg, flush=True)


def _rand(dtype, *shape, seed, scale=1.0):
    v = torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    return (v * scale).to(TYPES[dtype]).to(DEV)


@pytest.mark.parametrize("name,batch,smaller", [("tiny", 192, (183, 64, 1)), ("mid", 300, (70, 3))])
def test_example_runs_smaller_batches(name, batch, smaller):
    c = S.get_config(name)
    half = E.example.FeedForwardHalf(c, batch)
    for T in smaller:
        say(f"feed-forward half made for {batch} tokens: {name} T={T}")
        attn, stream = (_rand(c.act_dtype, T, c.hidden, seed=s) for s in (7, 8))
        out, s = half.forward(attn, stream)
        assert torch.isfinite(out).all()
        proj = R.linear(attn.cpu().double(), half.w_o.cpu().double())
        assert R.worst(s["proj"], proj) <= R.tolerance(c.act_dtype, 1, c.hidden)
        want = R.ffn(s["h1"].cpu().double(), {k: w.cpu().double() for k, w in half.ffn_w.items()})
        assert R.worst(s["f"], want) <= R.tolerance(c.act_dtype, 2, c.hidden + c.inter)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspace_of_the_largest_batch(dtype):
    # the sizes that each of these batches needs by itself do not rise with the batch
    K, N = 2048, 1024
    lin, ffn = moe.make_linear_cfg(K, N, "silu", dtype), moe.make_ffn_cfg(K, N, "silu", dtype)
    w = _rand(dtype, N, K, seed=1, scale=K ** -0.5)
    fw = {"w_gate": w, "w_up": _rand(dtype, N, K, seed=2, scale=K ** -0.5),
          "w_down": _rand(dtype, K, N, seed=3, scale=N ** -0.5)}
    top = 1500
    lws, lbws = moe.alloc_linear_workspace(lin, top, DEV), moe.alloc_linear_backward_workspace(lin, top, DEV)
    fws, fbws = moe.alloc_ffn_workspace(ffn, top, DEV), moe.alloc_ffn_backward_workspace(ffn, top, DEV)
    for T in (1, 16, 17, 63, 64, 65, 127, 128, 255, 256, 257, 320, 511, 640, 768, 1023, 1024, 1500):
        say(f"batch of {T} in workspaces for {top}, {dtype}")
        x, dy, dz = _rand(dtype, T, K, seed=T), _rand(dtype, T, K, seed=T + 1), _rand(dtype, T, N, seed=T + 2)
        z, y, dx = torch.empty_like(dz), torch.empty_like(x), torch.empty_like(x)
        dw, db, dfw = torch.empty_like(w), torch.empty_like(w[:, 0]), {k: torch.empty_like(v) for k, v in fw.items()}

        def run(a, b, c, d):
            moe.linear_forward(lin, x, w, z, a)
            moe.linear_backward(lin, x, w, dz, b, dx=dx, dw=dw, dbias=db)
            moe.ffn_forward(ffn, x, fw, y, c)
            outs = [v.clone() for v in (z, dx, dw, db, y)]
            moe.ffn_backward(ffn, x, fw, dy, dx, *dfw.values(), d)
            return outs + [v.clone() for v in (dx, *dfw.values())]

        got = run(lws, lbws, fws, fbws)
        want = run(moe.alloc_linear_workspace(lin, T, DEV), moe.alloc_linear_backward_workspace(lin, T, DEV),
                   moe.alloc_ffn_workspace(ffn, T, DEV), moe.alloc_ffn_backward_workspace(ffn, T, DEV))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
