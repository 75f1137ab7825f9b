"""The 64-bit forms of the operators around the expert layer: gradients against central
differences, and closed forms."""
import pytest
import torch

from tests import block_reference as R

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def _check(f, leaves, grads, seed=99):
    """Directional derivatives of the scalar f(leaves) along random directions."""
    for k, (name, v) in enumerate(leaves.items()):
        d = _rand(*v.shape, seed=seed + k)
        h = 1e-5
        up, down = f({**leaves, name: v + h * d}), f({**leaves, name: v - h * d})
        num, want = (up - down) / (2 * h), (grads[name] * d).sum()
        assert abs(num - want) <= 1e-6 * max(1.0, abs(want)), (name, float(num), float(want))


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_linear_gradients(act):
    x, w, b, dy = _rand(5, 7), _rand(6, 7, seed=1), _rand(6, seed=2), _rand(5, 6, seed=3)
    g = R.linear_grads(x, w, b, dy, act)
    _check(lambda v: (R.linear(v["dx"], v["dw"], v["dbias"], name=act) * dy).sum(),
           {"dx": x, "dw": w, "dbias": b}, g)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_ffn_gradients(act):
    leaves = {"dx": _rand(4, 6), "w_gate": _rand(5, 6, seed=1), "w_up": _rand(5, 6, seed=2),
              "w_down": _rand(6, 5, seed=3)}
    dy = _rand(4, 6, seed=4)
    _check(lambda v: (R.ffn(v["dx"], v, name=act) * dy).sum(), leaves,
           R.ffn_grads(leaves["dx"], leaves, dy, act))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gates,post,use_du,use_dh", [(0, True, True, True), (1, True, True, True),
                                                      (3, True, True, True), (6, False, True, True),
                                                      (2, True, False, True), (2, True, True, False)])
def test_norm_gradients(kind, gates, post, use_du, use_dh):
    T, H = 6, 5
    leaves = {"residual": _rand(T, H), "branch": _rand(T, H, seed=1), "w_pre": _rand(H, seed=2)}
    if post:
        leaves["w_post"] = _rand(H, seed=3)
    if kind == "layer":
        leaves["b_pre"] = _rand(H, seed=4)
        if post:
            leaves["b_post"] = _rand(H, seed=5)
    if gates:
        leaves["gate"] = _rand(gates, H, seed=6)
    du, dh = (_rand(T, H, seed=7) if use_du else None), (_rand(T, H, seed=8) if use_dh else None)

    def total(v):
        u, h = R.norm(v["residual"], v["branch"], v, kind, 1e-3, 0.7)
        return (0 if du is None else (u * du).sum()) + (0 if dh is None else (h * dh).sum())

    g = R.norm_grads(leaves["residual"], leaves["branch"], leaves, du, dh, kind, 1e-3, 0.7)
    if not use_dh:
        leaves = {k: v for k, v in leaves.items() if not k.endswith("_pre")}
    _check(total, leaves, g)


def test_norm_of_a_constant_row():
    v = torch.full((2, 8), 3.0, dtype=F64)
    ones = {"w_pre": torch.ones(8, dtype=F64)}
    _, h = R.norm(v, None, ones, "rms", 0.0)
    assert torch.allclose(h, torch.ones_like(v))
    _, h = R.norm(v, None, ones, "layer", 1e-6)
    assert torch.equal(h, torch.zeros_like(v))


def test_ffn_of_one_unit_by_hand():
    one = lambda v: torch.tensor([[v]], dtype=F64)  # noqa: E731
    y = R.ffn(one(2.0), {"w_gate": one(0.5), "w_up": one(3.0), "w_down": one(-1.0)}, one(10.0))
    assert abs(float(y) - (10 - 6 / (1 + 2.718281828459045 ** -1))) < 1e-12


def test_comparison_sees_one_wrong_element():
    want = _rand(64, 257)
    got = want.clone()
    assert R.worst(got, want) == 0
    got[13, 256] += 1
    assert R.worst(got, want) > R.tolerance("bf16", 3, 1024)
