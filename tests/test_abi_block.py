"""Argument checks of the operators around the expert layer: bad calls return status codes (or raise
in the binding) before any GPU work.  No compute call is made here (no GPU needed)."""
import ctypes
import os

import pytest
import torch

import sparse_moe_layer_group_amd as moe

pytestmark = pytest.mark.skipif(not os.path.exists(moe.lib_path()),
                                reason="library not built (python -m sparse_moe_layer_group_amd.build)")

OK, NULL, SHAPE, DTYPE, WS = 0, -1, -2, -3, -4
P = ctypes.c_void_p(1 << 20)   # never followed: every call here ends in its checks
BIG = 1 << 50


def _norm(cfg=None, T=4, residual=P, ldr=64, branch=P, ldb=64, params=None, u=P, ldu=64, h=P, ldh=64):
    cfg = moe.make_norm_cfg(64) if cfg is None else cfg
    params = moe._NormParams(w_post=1 << 20, w_pre=1 << 20) if params is None else params
    return moe.lib().moe_norm_forward(cfg, T, residual, ldr, branch, ldb, params, u, ldu, h, ldh, None)


@pytest.mark.parametrize("kw,want", [
    (dict(hidden=0), SHAPE), (dict(hidden=16385), SHAPE), (dict(hidden=64, kind=2), SHAPE),
    (dict(hidden=64, dtype="e4m3"), DTYPE), (dict(hidden=64, dtype=7), DTYPE), (dict(hidden=64, eps=-1e-6), SHAPE),
    (dict(hidden=64, eps=float("nan")), SHAPE), (dict(hidden=64, eps=float("inf")), SHAPE),
    (dict(hidden=64, res_scale=float("nan")), SHAPE), (dict(hidden=64, gate_rows=3), SHAPE),
    (dict(hidden=64, gate_rows=-1), SHAPE),
])
def test_norm_configurations(kw, want):
    cfg = moe.make_norm_cfg(**kw)
    assert _norm(cfg) == want
    assert moe.norm_backward_workspace_bytes(cfg, 4) == 0


def test_norm_arguments():
    Q = moe._NormParams
    a = 1 << 20
    assert moe.lib().moe_norm_forward(None, 4, P, 64, P, 64, None, P, 64, P, 64, None) == NULL
    assert _norm(residual=None) == NULL
    assert _norm(u=None, h=None) == NULL
    assert _norm(params=Q(w_post=a)) == NULL                              # h without w_pre
    assert _norm(params=Q(w_post=a, w_pre=a, b_pre=a)) == SHAPE           # a bias with RMS
    assert _norm(params=Q(w_post=a, w_pre=a, gate=a)) == SHAPE            # a gate without its rows
    assert _norm(moe.make_norm_cfg(64, gate_rows=4)) == NULL              # rows without a gate
    assert _norm(branch=None) == NULL                                     # w_post without a branch
    assert _norm(moe.make_norm_cfg(64, kind="layer"), params=Q(w_pre=a, b_post=a)) == NULL
    for kw in (dict(ldr=63), dict(ldb=63), dict(ldu=1), dict(ldh=0), dict(ldr=1 << 22)):
        assert _norm(**kw) == SHAPE, kw
    assert _norm(T=-1) == SHAPE and _norm(T=(1 << 24) + 1) == SHAPE
    assert _norm(T=0, residual=None, u=None, h=None) == OK


def _norm_back(cfg=None, T=4, params=None, branch=P, du=P, dh=P, grads=None, ws=P, n=BIG, ldd=64):
    cfg = moe.make_norm_cfg(64) if cfg is None else cfg
    a = 1 << 20
    params = moe._NormParams(w_post=a, w_pre=a) if params is None else params
    grads = moe._NormGrads(d_residual=a, ld_d_residual=64) if grads is None else grads
    return moe.lib().moe_norm_backward(cfg, T, P, 64, branch, 64, params, du, ldd, dh, 64, grads, ws, n, None)


def test_norm_backward_arguments():
    G, Q, a = moe._NormGrads, moe._NormParams, 1 << 20
    assert _norm_back(du=None, dh=None) == NULL
    assert _norm_back(grads=G(db_post=a)) == NULL and _norm_back(grads=G(db_pre=a)) == NULL
    assert _norm_back(grads=G(dgate=a)) == NULL
    assert _norm_back(grads=G(dw_pre=a), dh=None) == NULL
    assert _norm_back(grads=G(dw_post=a), params=Q(w_pre=a)) == NULL
    assert _norm_back(grads=G(d_branch=a, ld_d_branch=64), branch=None, params=Q(w_pre=a)) == NULL
    assert _norm_back(grads=G(d_residual=a, ld_d_residual=63)) == SHAPE
    assert _norm_back(ldd=3) == SHAPE
    need = moe.norm_backward_workspace_bytes(moe.make_norm_cfg(64), 4)
    assert need > 0
    assert _norm_back(ws=None) == WS and _norm_back(n=need - 1) == WS
    assert _norm_back(ws=ctypes.c_void_p((1 << 20) + 8)) == WS
    assert _norm_back(T=0, ws=None, n=0) == OK


def _linear(cfg=None, T=4, x=P, ldx=64, w=P, res=P, ldr=32, y=P, ldy=32, ws=P, n=BIG):
    cfg = moe.make_linear_cfg(64, 32) if cfg is None else cfg
    return moe.lib().moe_linear_forward(cfg, T, x, ldx, w, None, res, ldr, y, ldy, ws, n, None)


def _linear_back(cfg=None, T=4, x=P, ldx=64, w=P, dy=P, ldy=32, dx=P, lddx=64, ws=P, n=BIG):
    cfg = moe.make_linear_cfg(64, 32) if cfg is None else cfg
    return moe.lib().moe_linear_backward(cfg, T, x, ldx, w, None, dy, ldy, dx, lddx, None, None, ws, n, None)


@pytest.mark.parametrize("call", [_linear, _linear_back])
def test_linear_arguments(call):
    for kw, want in ((dict(in_dim=0, out_dim=8), SHAPE), (dict(in_dim=8, out_dim=131073), SHAPE),
                     (dict(in_dim=8, out_dim=8, act=4), SHAPE), (dict(in_dim=8, out_dim=8, act=-1), SHAPE),
                     (dict(in_dim=8, out_dim=8, dtype="e4m3"), DTYPE)):
        cfg = moe.make_linear_cfg(**kw)
        assert call(cfg) == want, kw
        assert moe.linear_workspace_bytes(cfg, 4) == 0 and moe.linear_backward_workspace_bytes(cfg, 4) == 0
    assert call(x=None) == NULL and call(w=None) == NULL
    assert call(ldx=63) == SHAPE and call(ldy=31) == SHAPE and call(ldx=1 << 22) == SHAPE
    assert call(T=-1) == SHAPE and call(T=(1 << 24) + 1) == SHAPE
    assert call(ws=None) == WS and call(n=16) == WS and call(ws=ctypes.c_void_p((1 << 20) + 4)) == WS
    assert call(T=0, x=None, w=None, ws=None, n=0) == OK


def test_linear_more_arguments():
    assert moe.lib().moe_linear_forward(None, 4, P, 8, P, None, None, 0, P, 8, P, BIG, None) == NULL
    assert moe.lib().moe_linear_backward(None, 4, P, 8, P, None, P, 8, P, 8, P, P, P, BIG, None) == NULL
    assert _linear(y=None) == NULL and _linear(ldr=31) == SHAPE
    assert _linear_back(dy=None) == NULL and _linear_back(lddx=63) == SHAPE
    assert _linear_back(dx=None) == OK             # no gradient wanted: nothing to do


def _ffn(cfg=None, T=4, x=P, ldx=64, wd=P, ldr=64, y=P, ldy=64, ws=P, n=BIG):
    cfg = moe.make_ffn_cfg(64, 32) if cfg is None else cfg
    return moe.lib().moe_ffn_forward(cfg, T, x, ldx, P, P, wd, P, ldr, y, ldy, ws, n, None)


def _ffn_back(cfg=None, T=4, x=P, ldx=64, wd=P, ldr=64, y=P, ldy=64, ws=P, n=BIG):
    cfg = moe.make_ffn_cfg(64, 32) if cfg is None else cfg
    return moe.lib().moe_ffn_backward(cfg, T, x, ldx, P, P, wd, P, ldr, y, ldy, P, P, P, ws, n, None)


@pytest.mark.parametrize("call", [_ffn, _ffn_back])
def test_ffn_arguments(call):
    for kw, want in ((dict(hidden=0, inter=8), SHAPE), (dict(hidden=8, inter=0), SHAPE),
                     (dict(hidden=131073, inter=8), SHAPE), (dict(hidden=8, inter=8, act="none"), SHAPE),
                     (dict(hidden=8, inter=8, act=4), SHAPE), (dict(hidden=8, inter=8, dtype="e4m3"), DTYPE)):
        cfg = moe.make_ffn_cfg(**kw)
        assert call(cfg) == want, kw
        assert moe.ffn_workspace_bytes(cfg, 4) == 0 and moe.ffn_backward_workspace_bytes(cfg, 4) == 0
    assert call(x=None) == NULL and call(wd=None) == NULL and call(y=None) == NULL
    assert call(ldx=63) == SHAPE and call(ldy=63) == SHAPE and call(ldr=63) == SHAPE
    assert call(T=-1) == SHAPE and call(T=(1 << 24) + 1) == SHAPE
    assert call(ws=None) == WS and call(n=16) == WS
    assert call(T=0, x=None, wd=None, y=None, ws=None, n=0) == OK


def test_workspaces_grow_with_the_batch():
    lin, ffn = moe.make_linear_cfg(7168, 2048), moe.make_ffn_cfg(7168, 2048)
    for f, cfg in ((moe.linear_workspace_bytes, lin), (moe.linear_backward_workspace_bytes, lin),
                   (moe.ffn_workspace_bytes, ffn), (moe.ffn_backward_workspace_bytes, ffn)):
        assert f(cfg, 0) == 0 < f(cfg, 4096) < f(cfg, 1 << 24)
    assert moe.ffn_workspace_bytes(ffn, 8192) >= 8192 * 2048 * 2
    # the largest sizes accepted do not wrap
    wide = moe.make_ffn_cfg(131072, 131072, dtype="f32")
    assert moe.ffn_backward_workspace_bytes(wide, 1 << 24) > 3 * (1 << 24) * 131072 * 6


def test_binding_refusals():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((32, 64), dtype=torch.bfloat16)
    y = torch.zeros((4, 32), dtype=torch.bfloat16)
    cfg = moe.make_linear_cfg(64, 32)
    with pytest.raises(ValueError, match="device tensor"):
        moe.linear_forward(cfg, x, w, y, None)
    with pytest.raises(ValueError, match="shape"):
        moe.linear_forward(cfg, x[:, :63], w, y, None)
    with pytest.raises(ValueError, match="dtype"):
        moe.linear_forward(cfg, x.float(), w, y, None)
    with pytest.raises(ValueError, match="required"):
        moe.linear_forward(cfg, None, w, y, None)
    with pytest.raises(ValueError, match="required"):
        moe.norm_forward(moe.make_norm_cfg(64), None, x, {"w_pre": w[0]}, x, x)
    with pytest.raises(ValueError, match="required"):
        moe._ffn_weights(moe.make_ffn_cfg(64, 32), x.dtype, {"w_up": w, "w_down": w})
    with pytest.raises(ValueError, match="contiguous"):
        moe._rows(torch.empty((64, 4), dtype=x.dtype, device="meta").T, "x", x.dtype, 4, 64)
    with pytest.raises(moe.MoeError):
        moe.alloc_ffn_workspace(moe.make_ffn_cfg(64, 32, "none"), 4, "cpu")
