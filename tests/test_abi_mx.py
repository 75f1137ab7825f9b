"""Argument checks of the operators with microscaled operands: bad calls return status codes (or raise
in the binding) before any GPU work.  No compute call is made here (no GPU needed)."""
import ctypes
import os

import pytest
import torch

import sparse_moe_layer_group_amd as moe

pytestmark = pytest.mark.skipif(not os.path.exists(moe.lib_path()),
                                reason="library not built (python -m sparse_moe_layer_group_amd.build)")

OK, NULL, SHAPE, DTYPE, WS = 0, -1, -2, -3, -4
A = 1 << 20                    # never followed: every call here ends in its checks
P = ctypes.c_void_p(A)
BIG = 1 << 50


def test_sizes():
    code, scale = moe.lib().moe_mx_code_bytes, moe.lib().moe_mx_scale_bytes
    assert code(0, 3, 128) == 384 and code(1, 3, 128) == 192 and code(0, 3, 129) == 768 and code(1, 1, 1) == 64
    assert scale(3, 128) == 12 and scale(3, 129) == 24 and scale(0, 5) == 0
    assert code(2, 3, 128) == code(-1, 3, 128) == code(0, -1, 128) == code(0, 3, 0) == code(0, 3, 131073) == 0
    assert code(0, 1 << 24, 131072) == 1 << 41 and scale(1 << 24, 131072) == 1 << 36
    for form, bytes_ in (("e4m3", 256), ("e2m1", 128)):
        m = moe.alloc_mx(5, 130, form, "cpu")
        assert m.codes.shape == (5, bytes_) and m.scales.shape == (5, 8) and m.rows == 5 and m.cols == 130


def _quantize(form=0, dtype=1, rows=4, cols=64, x=P, ld=64, c=P, s=P):
    return moe.lib().moe_mx_quantize(form, dtype, rows, cols, x, ld, c, s, None)


def _dequantize(form=0, dtype=1, rows=4, cols=64, x=P, ld=64, c=P, s=P):
    return moe.lib().moe_mx_dequantize(form, dtype, rows, cols, c, s, x, ld, None)


@pytest.mark.parametrize("call", [_quantize, _dequantize])
def test_quantisation_arguments(call):
    assert call(form=2) == DTYPE and call(form=-1) == DTYPE and call(dtype=2) == DTYPE
    assert call(rows=-1) == SHAPE and call(rows=(1 << 24) + 1) == SHAPE and call(cols=0) == SHAPE
    assert call(cols=131073, ld=131073) == SHAPE and call(ld=63) == SHAPE and call(ld=1 << 22) == SHAPE
    assert call(x=None) == NULL and call(c=None) == NULL and call(s=None) == NULL
    assert call(c=ctypes.c_void_p(A + 8)) == SHAPE and call(s=ctypes.c_void_p(A + 2)) == SHAPE
    assert call(rows=0, x=None, c=None, s=None) == OK


def _norm(cfg=None, form=0, T=4, residual=P, ldr=64, branch=P, ldb=64, params=None, u=P, ldu=64, h=P, ldh=64, c=P, s=P):
    cfg = moe.make_norm_cfg(64) if cfg is None else cfg
    params = moe._NormParams(w_post=A, w_pre=A) if params is None else params
    return moe.lib().moe_norm_mx_forward(cfg, form, T, residual, ldr, branch, ldb, params, u, ldu, h, ldh, c, s, None)


def test_norm_arguments():
    Q = moe._NormParams
    assert moe.lib().moe_norm_mx_forward(None, 0, 4, P, 64, P, 64, None, P, 64, P, 64, P, P, None) == NULL
    assert _norm(form=2) == DTYPE and _norm(moe.make_norm_cfg(64, dtype=7)) == DTYPE
    assert _norm(moe.make_norm_cfg(0)) == SHAPE and _norm(moe.make_norm_cfg(16385)) == SHAPE
    assert _norm(c=None) == NULL and _norm(s=None) == NULL and _norm(residual=None) == NULL
    assert _norm(params=Q(w_post=A)) == NULL and _norm(params=Q(w_post=A), h=None) == NULL   # codes need w_pre
    assert _norm(params=Q(w_post=A, w_pre=A, b_pre=A)) == SHAPE and _norm(params=Q(w_post=A, w_pre=A, gate=A)) == SHAPE
    assert _norm(branch=None) == NULL and _norm(moe.make_norm_cfg(64, gate_rows=3)) == SHAPE
    for kw in (dict(ldr=63), dict(ldb=63), dict(ldu=1), dict(ldh=0), dict(ldr=1 << 22)):
        assert _norm(**kw) == SHAPE, kw
    assert _norm(c=ctypes.c_void_p(A + 8)) == SHAPE and _norm(s=ctypes.c_void_p(A + 1)) == SHAPE
    assert _norm(T=-1) == SHAPE and _norm(T=(1 << 24) + 1) == SHAPE
    assert _norm(T=0, residual=None, u=None, h=None, c=None, s=None) == OK


def _m(codes=A, scales=A):
    return moe._Mx(codes, scales)


def _linear(cfg=None, T=4, x=_m(), w=_m(), res=P, ldr=32, y=P, ldy=32, ws=P, n=BIG):
    cfg = moe.make_mx_linear_cfg(64, 32) if cfg is None else cfg
    return moe.lib().moe_mx_linear_forward(cfg, T, x, w, None, res, ldr, y, ldy, ws, n, None)


def _ffn(cfg=None, T=4, x=_m(), w=_m(), res=P, ldr=64, y=P, ldy=64, ws=P, n=BIG):
    cfg = moe.make_mx_ffn_cfg(64, 32) if cfg is None else cfg
    return moe.lib().moe_mx_ffn_forward(cfg, T, x, _m(), _m(), w, res, ldr, y, ldy, ws, n, None)


@pytest.mark.parametrize("call,make,query", [
    (_linear, lambda **k: moe.make_mx_linear_cfg(**{"in_dim": 64, "out_dim": 32, **k}), moe.mx_linear_workspace_bytes),
    (_ffn, lambda **k: moe.make_mx_ffn_cfg(**{"hidden": 64, "inter": 32, **k}), moe.mx_ffn_workspace_bytes)])
def test_product_arguments(call, make, query):
    first = "in_dim" if call is _linear else "hidden"
    for kw, want in (({first: 0}, SHAPE), ({first: 131073}, SHAPE), (dict(act=4), SHAPE), (dict(act=-1), SHAPE),
                     (dict(dtype="e4m3"), DTYPE), (dict(dtype=7), DTYPE), (dict(form=2), DTYPE), (dict(form=-1), DTYPE)):
        cfg = make(**kw)
        assert call(cfg) == want, kw
        assert query(cfg, 4) == 0
    assert call(x=None) == NULL and call(w=None) == NULL and call(y=None) == NULL
    assert call(x=_m(codes=0)) == NULL and call(w=_m(scales=0)) == NULL
    assert call(x=_m(codes=A + 8)) == SHAPE and call(w=_m(scales=A + 2)) == SHAPE
    assert call(ldy=31) == SHAPE and call(ldr=31) == SHAPE and call(ldy=1 << 22) == SHAPE
    assert call(T=-1) == SHAPE and call(T=(1 << 24) + 1) == SHAPE
    need = query(make(), 4)
    assert need > 0 and call(ws=None) == WS and call(n=need - 1) == WS and call(ws=ctypes.c_void_p(A + 4)) == WS
    assert call(T=0, x=None, w=None, y=None, ws=None, n=0) == OK
    assert call(cfg=make(act="none")) == SHAPE if call is _ffn else query(make(act="none"), 4) > 0


def test_workspaces_serve_every_smaller_batch():
    for query, cfg in ((moe.mx_linear_workspace_bytes, moe.make_mx_linear_cfg(7168, 2048)),
                       (moe.mx_ffn_workspace_bytes, moe.make_mx_ffn_cfg(7168, 2048))):
        sizes = [query(cfg, T) for T in range(1, 700)] + [query(cfg, T) for T in (4096, 8192, 1 << 24)]
        assert query(cfg, 0) == 0 < sizes[0] and sizes == sorted(sizes)


def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    m = moe.alloc_mx(4, 64, "e4m3", "cpu")
    with pytest.raises(ValueError, match="device tensor"):
        moe.mx_quantize(x, m)
    with pytest.raises(ValueError, match="device tensor"):
        moe.mx_dequantize(m, x)
    with pytest.raises(ValueError, match="dtype"):
        moe.mx_quantize(x.half(), m)
    with pytest.raises(ValueError, match="form"):
        moe.mx_quantize(x, m._replace(form="e5m2"))
    with pytest.raises(ValueError, match="form"):
        moe.mx_quantize(x, None)
    with pytest.raises(ValueError, match="matrix"):
        moe.mx_quantize(x[0], m)
    y, cfg = torch.zeros((4, 32), dtype=torch.bfloat16), moe.make_mx_linear_cfg(64, 32)
    w = moe.alloc_mx(32, 64, "e2m1", "cpu")
    with pytest.raises(ValueError, match="expected 64 of e4m3"):
        moe.mx_linear_forward(cfg, w, w, y, None)
    with pytest.raises(ValueError, match="columns"):
        moe.mx_linear_forward(cfg, m._replace(cols=63), w, y, None)
    with pytest.raises(ValueError, match="shape"):
        moe.mx_linear_forward(cfg, moe.alloc_mx(5, 64, "e4m3", "cpu"), w, y, None)
    with pytest.raises(ValueError, match="required"):
        moe.mx_linear_forward(cfg, None, w, y, None)
    with pytest.raises(ValueError, match="required"):
        moe._mx({}.get("w_gate"), "w_gate", 32, 64, 1)
    with pytest.raises(ValueError, match="required"):
        moe.norm_mx_forward(moe.make_norm_cfg(64), None, x, {"w_pre": x[0]}, x, m)
    with pytest.raises(moe.MoeError):
        moe.alloc_mx_ffn_workspace(moe.make_mx_ffn_cfg(64, 32, "none"), 4, "cpu")
