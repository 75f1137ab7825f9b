"""Plain 64-bit implementations of the operators around the expert layer (norms with the residual
stream, projections, the dense gated feed-forward block), values and gradients written out from
their formulas, and the comparison that the GPU tests use."""
import math

import torch

F64 = torch.float64


# ---------------------------------------------------------------- activations


def act(name, z):
    if name == "none":
        return z.clone()
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))


def act_slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


# ---------------------------------------------------------------- linear


def linear(x, w, bias=None, residual=None, name="none"):
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(name, z)
    return y if residual is None else y + residual


def linear_grads(x, w, bias, dy, name="none"):
    z = x @ w.T
    if bias is not None:
        z = z + bias
    dz = dy * act_slope(name, z)
    return {"dx": dz @ w, "dw": dz.T @ x, "dbias": dz.sum(0)}


# ---------------------------------------------------------------- ffn


def ffn(x, w, residual=None, name="silu"):
    y = (act(name, x @ w["w_gate"].T) * (x @ w["w_up"].T)) @ w["w_down"].T
    return y if residual is None else y + residual


def ffn_grads(x, w, dy, name="silu"):
    g, u = x @ w["w_gate"].T, x @ w["w_up"].T
    dm = dy @ w["w_down"]
    dg, du = dm * u * act_slope(name, g), dm * act(name, g)
    return {"dx": dg @ w["w_gate"] + du @ w["w_up"], "w_gate": dg.T @ x, "w_up": du.T @ x,
            "w_down": dy.T @ (act(name, g) * u)}


# ---------------------------------------------------------------- norm


def unit(v, kind, eps):
    m = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    c = v - m
    inv = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    return c * inv, inv


def gate_per_token(gate, T):
    return gate.repeat_interleave(T // gate.shape[0], 0)


def norm(residual, branch, p, kind="rms", eps=1e-6, scale=1.0):
    u = scale * residual
    if branch is not None:
        n = branch
        if p.get("w_post") is not None:
            n = unit(branch, kind, eps)[0] * p["w_post"]
            if p.get("b_post") is not None:
                n = n + p["b_post"]
        if p.get("gate") is not None:
            n = n * gate_per_token(p["gate"], n.shape[0])
        u = u + n
    h = None
    if p.get("w_pre") is not None:
        h = unit(u, kind, eps)[0] * p["w_pre"]
        if p.get("b_pre") is not None:
            h = h + p["b_pre"]
    return u, h


def norm_grads(residual, branch, p, du, dh, kind="rms", eps=1e-6, scale=1.0):
    T = residual.shape[0]
    u, _ = norm(residual, branch, p, kind, eps, scale)
    e = torch.zeros_like(u) if du is None else du.clone()
    out = {}

    def back(d, q, inv):
        m = d.mean(1, keepdim=True) if kind == "layer" else 0.0
        return inv * (d - m - q * (d * q).mean(1, keepdim=True))

    if dh is not None:
        q, inv = unit(u, kind, eps)
        out["w_pre"], out["b_pre"] = (dh * q).sum(0), dh.sum(0)
        e = e + back(dh * p["w_pre"], q, inv)
    out["residual"] = scale * e
    if branch is not None:
        post = p.get("w_post") is not None
        q, inv = unit(branch, kind, eps) if post else (branch, None)
        n = q * p["w_post"] if post else q
        if p.get("b_post") is not None:
            n = n + p["b_post"]
        if p.get("gate") is not None:
            out["gate"] = (e * n).reshape(p["gate"].shape[0], -1, n.shape[1]).sum(1)
            e = e * gate_per_token(p["gate"], T)
        if post:
            out["w_post"], out["b_post"] = (e * q).sum(0), e.sum(0)
            e = back(e * p["w_post"], q, inv)
        out["branch"] = e
    return out


# ---------------------------------------------------------------- comparison


def worst(got, want):
    """The largest over rows and columns of |got - want| / max(|want|, typical |want|), 2-norms,
    divided by the allowance 1 + 4 / sqrt(n) for the fluctuation of a norm of n values."""
    got, want = got.detach().to("cpu", F64), want.to("cpu", F64)
    assert got.shape == want.shape, (got.shape, want.shape)
    if want.dim() == 1:
        got, want = got[None], want[None]
    assert torch.isfinite(got).all(), "not finite"
    rms = want.square().mean().sqrt()
    most = 0.0
    for dim in (1, 0):
        n = want.shape[dim]
        err = (got - want).square().sum(dim).sqrt()
        ref = torch.maximum(want.square().sum(dim).sqrt(), rms * math.sqrt(n))
        rel = torch.where(err > 0, err / ref, torch.zeros_like(err)).max().item()
        most = max(most, rel / (1 + 4 / math.sqrt(n)))
    return most


def tolerance(dtype, roundings, terms):
    """Relative tolerance of an output after `roundings` roundings to the type on its path and sums
    of `terms` products.  bfloat16: each rounding is at most 2^-8 of its value and they are
    independent.  float32: sums go through one accumulation for every 16 products of each of six
    partial products, each off by at most 2^-24 of the partial sum; four times their random walk,
    once for every stage."""
    if dtype == "bf16":
        return 2.0 ** -8 * math.sqrt(roundings)
    return roundings * 4 * math.sqrt(6 * terms / 16 + 16) * 2.0 ** -24
