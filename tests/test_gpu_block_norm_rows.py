"""Norms of more rows than there are workers (waves or workgroups that take a range of rows each): rows that
follow each other in one worker, sums over them, gate rows that end inside a worker's range or span several,
for every width's form, whole and ragged, both kinds and types.  The plain forms run on the device."""
import math

import pytest
import torch

import sparse_moe_layer_group_amd as moe
from tests import block_reference as R
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# hidden, T, gate_rows.  Workers, forward and backward: up to hidden 512 8192 and 2048, to 1024 8192 and 1024,
# 1030 4096 and 1024, 7168 1024 and 256, 8200 1536 and 256, 16384 1024 and 256.
CASES = [(72, 20010, (0, 667, 6)), (513, 20010, (20010, 345, 10)), (1000, 9000, (9000, 75, 8)), (1030, 9000, (0, 75, 8)),
         (7168, 2500, (2500, 125, 4)), (7001, 2500, (625, 2)), (8200, 3200, (3200, 128, 5)), (8201, 3200, (0, 100)),
         (16384, 2100, (700, 21, 3))]


def say(msg):
    print(msg, flush=True)


def _rows(g, dtype, T, H, pad, scale=1.0):
    t = torch.full((T, H + pad), float("nan"), dtype=TYPES[dtype], device=DEV)
    t[:, :H] = torch.randn((T, H), generator=g, device=DEV) * scale
    return t[:, :H]


def _vec(g, dtype, *shape, scale, shift=0.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale + shift).to(TYPES[dtype])


def _worst(got, want):
    """The comparison of block_reference.worst, on the device."""
    got = got.double()
    if want.dim() == 1:
        got, want = got[None], want[None]
    assert torch.isfinite(got).all(), "not finite"
    rms, most = want.square().mean().sqrt(), 0.0
    for dim in (1, 0):
        n = want.shape[dim]
        err = (got - want).square().sum(dim).sqrt()
        ref = torch.maximum(want.square().sum(dim).sqrt(), rms * math.sqrt(n))
        most = max(most, torch.where(err > 0, err / ref, torch.zeros_like(err)).max().item() / (1 + 4 / math.sqrt(n)))
    return most


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,T,gates", CASES)
def test_norms_of_many_rows(dtype, kind, H, T, gates):
    # as for few rows: one rounding to the type; float32 sums of the row's terms, 8 a thread and then tree-wise
    tol = R.tolerance("bf16", 1, H) if dtype == "bf16" else 64 * 2.0 ** -24
    g = torch.Generator(DEV).manual_seed(H + T)
    pad = H % 3
    r, f = _rows(g, dtype, T, H, pad, 2.0), _rows(g, dtype, T, H, pad, 0.5)
    du, dh = _rows(g, dtype, T, H, pad), _rows(g, dtype, T, H, pad)
    r[:, H // 2] *= 16
    p = {k: _vec(g, dtype, H, scale=0.1, shift=1.0) for k in ("w_post", "w_pre")}
    if kind == "layer":
        p.update({k: _vec(g, dtype, H, scale=1.0) for k in ("b_post", "b_pre")})
    lift = lambda d: {k: v.double() for k, v in d.items()}  # noqa: E731
    for rows in gates:
        say(f"norm {dtype} {kind} T={T} H={H} gate_rows={rows}")
        if rows:
            p["gate"] = _vec(g, dtype, T // rows, H, scale=0.3, shift=0.5)
        cfg = moe.make_norm_cfg(H, dtype, kind, rows, 1e-6, 0.75)
        u, h = (torch.full((T, H), float("nan"), dtype=TYPES[dtype], device=DEV) for _ in range(2))
        moe.norm_forward(cfg, r, f, p, u, h)
        wu, wh = R.norm(r.double(), f.double(), lift(p), kind, 1e-6, 0.75)
        assert _worst(u, wu) <= tol and _worst(h, wh) <= tol
        del u, h, wu, wh
        grads = {k: torch.full_like(v, float("nan")) for k, v in p.items()}
        grads.update({k: torch.full((T, H), float("nan"), dtype=TYPES[dtype], device=DEV)
                      for k in ("residual", "branch")})
        ws = moe.alloc_norm_backward_workspace(cfg, T, DEV)
        moe.norm_backward(cfg, r, f, p, du, dh, grads, ws)
        want = R.norm_grads(r.double(), f.double(), lift(p), du.double(), dh.double(), kind, 1e-6, 0.75)
        for k, got in grads.items():
            err = _worst(got, want[k])
            assert err <= tol * (1 if dtype == "bf16" else 4), (k, err)
        del want
        again = {k: torch.empty_like(v) for k, v in grads.items()}
        moe.norm_backward(cfg, r, f, p, du, dh, again, ws)
        assert all(torch.equal(again[k], grads[k]) for k in grads)
        p.pop("gate", None)
