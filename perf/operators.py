"""The operators around the expert layer, as cases to be timed and compared.

Three operators, each forward and backward:

* ``norm``: ``u = s * residual + gate * post(branch)``, ``h = pre(u)``, the norms after one block
  and before the next with the gate and the residual scale between them;
* ``ffn``: ``y = residual + (act(x Wg^T) * (x Wu^T)) Wd^T``, the dense gated feed-forward block;
* ``linear``: ``y = residual + act(x W^T + b)``.

``own = False`` computes them from elementary torch operations in 32 bits, rounded once at the end;
``own = True`` calls this package's entry points.  ``exact`` is the 64-bit value, gradients by
automatic differentiation of the definition.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
RES_SCALE = 0.75      # depth-scaled residual streams use values like this one
H, I = 7168, 2048     # the layer's hidden and expert widths


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one token of a serving loop between two blocks: pure latency
        _norm("norm one token", 1, H),
        # a long prompt, per-channel gate (layer scale)
        _norm("norm prompt", 8192, H, gate_rows=8192),
        # a training step's token batch
        _norm("norm backward", 4096, H, back=True, gate_rows=4096),
        # three sequences with a gate row each (conditioned gates), layer norms with biases, and a
        # width that no vector load divides
        _norm("norm backward odd layer", 777, 1001, back=True, kind="layer", gate_rows=259, dtype="f32"),
        # serving: one token, and a ragged batch of them, through a dense block of the shared
        # expert's size
        _ffn("ffn one token", 1, H, I),
        _ffn("ffn small batch", 50, H, I),
        # a prompt (the prefill batch), and a training step
        _ffn("ffn prompt", 8192, H, I),
        _ffn("ffn backward", 4096, H, I, back=True),
        # full-precision training at the reduced width
        _ffn("ffn backward f32", 300, 1024, 256, back=True, act="gelu", dtype="f32"),
        # a projection with sizes that no tile divides, reading columns of a wider tensor
        _linear("linear odd", 333, 1001, 777, act="gelu", pad=23),
        # a square projection into the residual stream
        _linear("linear prompt", 4096, H, H),
        # a training step of an activated projection
        _linear("linear backward", 4096, H, I, act="silu", back=True),
    ]


def _norm(name, T, hidden, back=False, kind="rms", gate_rows=0, dtype="bf16", pad=0):
    c = {"op": "norm", "T": T, "hidden": hidden, "back": back, "kind": kind, "gate_rows": gate_rows,
         "dtype": dtype, "pad": pad}
    return c if name is None else dict(c, name=name)


def _ffn(name, T, hidden, inter, act="silu", back=False, dtype="bf16", pad=0):
    c = {"op": "ffn", "T": T, "hidden": hidden, "inter": inter, "act": act, "back": back,
         "dtype": dtype, "pad": pad}
    return c if name is None else dict(c, name=name)


def _linear(name, T, n_in, n_out, act="none", back=False, dtype="bf16", pad=0):
    c = {"op": "linear", "T": T, "n_in": n_in, "n_out": n_out, "act": act, "back": back,
         "dtype": dtype, "pad": pad}
    return c if name is None else dict(c, name=name)


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: two of three are multiples of 64 or 8, the third is whatever it is."""
    w, kind = _log(rng, lo, hi), rng.randrange(3)
    step = (64, 8, 1)[kind]
    return max(step, w // step * step)


def draw(rng):
    op = rng.choice(("norm", "ffn", "linear"))
    back = rng.random() < 0.5
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    pad = rng.choice((0, 0, 8, 5))
    if op == "norm":
        hidden = _width(rng, 64, 8192)
        T = _log(rng, 1, max(1, 8192 * H // 2 // hidden) if back else max(1, 8192 * H // hidden))
        T = min(T, 30000)
        rows = rng.choice((0, T, 1, T))
        if rng.random() < 0.3 and T >= 8:
            rows = max(1, T // 4)
            T = 4 * rows
        return _norm(None, T, hidden, back, rng.choice(("rms", "rms", "layer")), rows, dtype, pad)
    most = 4096 * H * I if back or dtype == "f32" else 8192 * H * I
    if dtype == "f32":
        most //= 8
    a, b = _width(rng, 128, H), _width(rng, 64, H)
    T = _log(rng, 1, max(1, min(16384, most // (a * b))))
    # the slope of relu jumps at zero, where two right sums of different order fall on either side:
    # its gradient cannot be compared element by element, so it is drawn forward only
    acts = ("silu", "gelu") if back else ("silu", "gelu", "relu")
    if op == "ffn":
        return _ffn(None, T, a, b, rng.choice(acts), back, dtype, pad)
    return _linear(None, T, a, b, rng.choice(("none",) + acts), back, dtype, pad)


# ---------------------------------------------------------------- inputs


def _rand(gen, dtype, *shape, scale=1.0, shift=0.0):
    v = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return (v * scale + shift).to(dtype)


def _rows(gen, dtype, T, cols, pad, scale=1.0):
    """[T][cols] activations; with `pad`, the columns of a wider tensor."""
    return _rand(gen, dtype, T, cols + pad, scale=scale)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt, T, back, pad = TYPES[case["dtype"]], case["T"], case["back"], case["pad"]
    s = {"case": case}
    if case["op"] == "norm":
        h = case["hidden"]
        layer = case["kind"] == "layer"
        s["residual"] = _rows(g, dt, T, h, pad, scale=2.0)
        # a residual stream has a few channels far larger than the others
        s["residual"][:, torch.randint(0, h, (max(1, h // 500),), generator=g, device=DEV)] *= 16
        s["branch"] = _rows(g, dt, T, h, pad, scale=0.5)
        p = {"w_post": _rand(g, dt, h, scale=0.1, shift=1.0), "w_pre": _rand(g, dt, h, scale=0.1, shift=1.0)}
        p["b_post"] = _rand(g, dt, h, scale=0.1) if layer else None
        p["b_pre"] = _rand(g, dt, h, scale=0.1) if layer else None
        n = case["gate_rows"]
        p["gate"] = _rand(g, dt, T // n, h, scale=0.3, shift=0.5) if n else None
        s["params"] = p
        if back:
            s["du"], s["dh"] = _rows(g, dt, T, h, pad), _rows(g, dt, T, h, pad)
            s["grads"] = {k: torch.empty_like(v) for k, v in p.items() if v is not None}
            s["grads"]["residual"] = torch.empty((T, h), dtype=dt, device=DEV)
            s["grads"]["branch"] = torch.empty((T, h), dtype=dt, device=DEV)
        else:
            s["u"], s["h"] = (torch.empty((T, h), dtype=dt, device=DEV) for _ in range(2))
    elif case["op"] == "ffn":
        h, i = case["hidden"], case["inter"]
        s["x"] = _rows(g, dt, T, h, pad)
        s["w"] = {"w_gate": _rand(g, dt, i, h, scale=h ** -0.5), "w_up": _rand(g, dt, i, h, scale=h ** -0.5),
                  "w_down": _rand(g, dt, h, i, scale=i ** -0.5)}
        if back:
            s["dy"] = _rows(g, dt, T, h, pad)
            s["dx"] = torch.empty((T, h), dtype=dt, device=DEV)
            s["dw"] = {k: torch.empty_like(v) for k, v in s["w"].items()}
        else:
            s["residual"] = _rows(g, dt, T, h, pad)
            s["y"] = torch.empty((T, h), dtype=dt, device=DEV)
    else:
        k, n = case["n_in"], case["n_out"]
        s["x"] = _rows(g, dt, T, k, pad)
        s["w"] = _rand(g, dt, n, k, scale=k ** -0.5)
        s["bias"] = _rand(g, dt, n, scale=0.2)
        if back:
            s["dy"] = _rows(g, dt, T, n, pad)
            s["dx"] = torch.empty((T, k), dtype=dt, device=DEV)
            s["dw"], s["dbias"] = torch.empty_like(s["w"]), torch.empty_like(s["bias"])
        else:
            s["residual"] = _rows(g, dt, T, n, pad)
            s["y"] = torch.empty((T, n), dtype=dt, device=DEV)
    if own:
        # the configuration and the workspace that a program makes once for its layers
        s["cfg"], s["ws"] = _own_plan(case)
    return s


def _own_plan(c):
    import sparse_moe_layer_group_amd as moe

    if c["op"] == "norm":
        cfg = moe.make_norm_cfg(c["hidden"], c["dtype"], c["kind"], c["gate_rows"], EPS, RES_SCALE)
        return cfg, moe.alloc_norm_backward_workspace(cfg, c["T"], DEV) if c["back"] else None
    if c["op"] == "ffn":
        cfg = moe.make_ffn_cfg(c["hidden"], c["inter"], c["act"], c["dtype"])
        return cfg, (moe.alloc_ffn_backward_workspace if c["back"] else moe.alloc_ffn_workspace)(cfg, c["T"], DEV)
    cfg = moe.make_linear_cfg(c["n_in"], c["n_out"], c["act"], c["dtype"])
    return cfg, (moe.alloc_linear_backward_workspace if c["back"] else moe.alloc_linear_workspace)(cfg, c["T"], DEV)


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    if own:
        return _own_run(s, c)
    plain = {"norm": (_plain_norm, _plain_norm_back), "ffn": (_plain_ffn, _plain_ffn_back),
             "linear": (_plain_linear, _plain_linear_back)}
    return plain[c["op"]][c["back"]](s, c, TYPES[c["dtype"]])


def _own_run(s, c):
    import sparse_moe_layer_group_amd as moe

    if c["op"] == "norm":
        if c["back"]:
            moe.norm_backward(s["cfg"], s["residual"], s["branch"], s["params"], s["du"], s["dh"], s["grads"], s["ws"])
            return s["grads"]
        moe.norm_forward(s["cfg"], s["residual"], s["branch"], s["params"], s["u"], s["h"])
        return {"u": s["u"], "h": s["h"]}
    if c["op"] == "ffn":
        if c["back"]:
            moe.ffn_backward(s["cfg"], s["x"], s["w"], s["dy"], s["dx"], s["dw"]["w_gate"], s["dw"]["w_up"],
                             s["dw"]["w_down"], s["ws"])
            return {"dx": s["dx"], **s["dw"]}
        moe.ffn_forward(s["cfg"], s["x"], s["w"], s["y"], s["ws"], residual=s["residual"])
        return {"y": s["y"]}
    if c["back"]:
        moe.linear_backward(s["cfg"], s["x"], s["w"], s["dy"], s["ws"], bias=s["bias"], dx=s["dx"], dw=s["dw"],
                            dbias=s["dbias"])
        return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}
    moe.linear_forward(s["cfg"], s["x"], s["w"], s["y"], s["ws"], bias=s["bias"], residual=s["residual"])
    return {"y": s["y"]}


# ---------------------------------------------------------------- plain forms, 32 bits


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))


def _act_slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        e = 1 / (1 + torch.exp(-z))
        return e * (1 + z * (1 - e))
    return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _unit(v, kind):
    """The rows of v, centred where `kind` says so, over their root mean square; and its inverse."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    inv = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * inv, inv


def _unit_back(d, unit, inv, kind):
    """Gradient at the rows whose unit rows are `unit`, from d at those."""
    if kind == "layer":
        d = d - d.mean(-1, keepdim=True)
    return inv * (d - unit * (d * unit).mean(-1, keepdim=True))


def _gate_rows(gate, T):
    return gate.repeat_interleave(T // gate.shape[0], 0)


def _norm_mid(s, c):
    """The unit rows after the branch, the normed branch, the gate's rows and the stream."""
    p = {k: v.float() for k, v in s["params"].items() if v is not None}
    unit, inv = _unit(s["branch"].float(), c["kind"])
    normed = unit * p["w_post"]
    if "b_post" in p:
        normed = normed + p["b_post"]
    gate = _gate_rows(p["gate"], c["T"]) if "gate" in p else None
    u = RES_SCALE * s["residual"].float() + (normed if gate is None else normed * gate)
    return p, unit, inv, normed, gate, u


def _plain_norm(s, c, dt):
    p, _, _, _, _, u = _norm_mid(s, c)
    h = _unit(u, c["kind"])[0] * p["w_pre"]
    if "b_pre" in p:
        h = h + p["b_pre"]
    return {"u": u.to(dt), "h": h.to(dt)}


def _plain_norm_back(s, c, dt):
    p, unit, inv, normed, gate, u = _norm_mid(s, c)
    unit2, inv2 = _unit(u, c["kind"])
    dh = s["dh"].float()
    du = s["du"].float() + _unit_back(dh * p["w_pre"], unit2, inv2, c["kind"])
    dn = du if gate is None else du * gate
    g = {"w_pre": (dh * unit2).sum(0), "w_post": (dn * unit).sum(0), "residual": RES_SCALE * du,
         "branch": _unit_back(dn * p["w_post"], unit, inv, c["kind"])}
    if "b_pre" in p:
        g["b_pre"], g["b_post"] = dh.sum(0), dn.sum(0)
    if gate is not None:
        g["gate"] = (du * normed).view(c["T"] // c["gate_rows"], c["gate_rows"], -1).sum(1)
    return {k: v.to(dt) for k, v in g.items()}


def _plain_ffn(s, c, dt):
    x, w = s["x"].float(), {k: v.float() for k, v in s["w"].items()}
    mid = _act(x @ w["w_gate"].t(), c["act"]) * (x @ w["w_up"].t())
    return {"y": (s["residual"].float() + mid @ w["w_down"].t()).to(dt)}


def _plain_ffn_back(s, c, dt):
    x, dy, w = s["x"].float(), s["dy"].float(), {k: v.float() for k, v in s["w"].items()}
    gate, up = x @ w["w_gate"].t(), x @ w["w_up"].t()
    soft = _act(gate, c["act"])
    dmid = dy @ w["w_down"]
    dgate, dup = dmid * up * _act_slope(gate, c["act"]), dmid * soft
    g = {"dx": dgate @ w["w_gate"] + dup @ w["w_up"], "w_gate": dgate.t() @ x, "w_up": dup.t() @ x,
         "w_down": dy.t() @ (soft * up)}
    return {k: v.to(dt) for k, v in g.items()}


def _plain_linear(s, c, dt):
    z = s["x"].float() @ s["w"].float().t() + s["bias"].float()
    return {"y": (s["residual"].float() + _act(z, c["act"])).to(dt)}


def _plain_linear_back(s, c, dt):
    x, w, dz = s["x"].float(), s["w"].float(), s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(x @ w.t() + s["bias"].float(), c["act"])
    return {"dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt), "dbias": dz.sum(0).to(dt)}


# ---------------------------------------------------------------- work


def work(case):
    T, b = case["T"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        h, n = case["hidden"], case["gate_rows"]
        params = h * ((4 if case["kind"] == "layer" else 2) + (T // n if n else 0))
        # forward: residual and branch in, u and h out; backward: du and dh too, and the gradients
        if case["back"]:
            return {"bytes": b * (6 * T * h + 2 * params), "flops": 40.0 * T * h}
        return {"bytes": b * (4 * T * h + params), "flops": 14.0 * T * h}
    if case["op"] == "ffn":
        h, i = case["hidden"], case["inter"]
        if case["back"]:  # gate, up, their gradient, and two products for each of three matrices
            return {"bytes": b * (3 * T * h + 6 * h * i), "flops": 16.0 * T * h * i}
        return {"bytes": b * (3 * T * h + 3 * h * i), "flops": 6.0 * T * h * i}
    k, n = case["n_in"], case["n_out"]
    if case["back"]:
        products = 2 if case["act"] == "none" else 3
        return {"bytes": b * (2 * T * k + T * n + 2 * n * k + 2 * n), "flops": 2.0 * products * T * k * n}
    return {"bytes": b * (T * k + 2 * T * n + n * k + n), "flops": 2.0 * T * k * n}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    """The definitions in 64 bits; gradients of <upstream, outputs> by automatic differentiation."""
    s = prepare(case, seed)
    need = case["back"]
    lift = lambda t: None if t is None else t.double().requires_grad_(need)  # noqa: E731
    act = {"none": lambda z: z, "relu": torch.relu, "silu": lambda z: z * torch.sigmoid(z),
           "gelu": lambda z: z * 0.5 * torch.erfc(-z / math.sqrt(2.0))}
    with torch.set_grad_enabled(need):
        if case["op"] == "norm":
            leaf = {k: lift(v) for k, v in s["params"].items() if v is not None}
            leaf["residual"], leaf["branch"] = lift(s["residual"]), lift(s["branch"])

            def norm(v, w, b):
                if case["kind"] == "layer":
                    var, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
                    return (v - mean) * torch.rsqrt(var + EPS) * w + b
                return v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + EPS) * w

            f = norm(leaf["branch"], leaf["w_post"], leaf.get("b_post"))
            if "gate" in leaf:
                f = (f.view(leaf["gate"].shape[0], -1, f.shape[1]) * leaf["gate"][:, None, :]).view(f.shape)
            u = f + leaf["residual"] * RES_SCALE
            h = norm(u, leaf["w_pre"], leaf.get("b_pre"))
            if not need:
                return {"u": u, "h": h}
            total = (u * s["du"].double()).sum() + (h * s["dh"].double()).sum()
            return dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
        if case["op"] == "ffn":
            leaf = {k: lift(v) for k, v in s["w"].items()}
            leaf["dx"] = lift(s["x"])
            a = torch.nn.functional.linear(leaf["dx"], leaf["w_gate"])
            b = torch.nn.functional.linear(leaf["dx"], leaf["w_up"])
            y = torch.nn.functional.linear(act[case["act"]](a) * b, leaf["w_down"])
        else:
            leaf = {"dx": lift(s["x"]), "dw": lift(s["w"]), "dbias": lift(s["bias"])}
            y = act[case["act"]](torch.nn.functional.linear(leaf["dx"], leaf["dw"], leaf["dbias"]))
        if not need:
            return {"y": y + s["residual"].double()}
        return dict(zip(leaf, torch.autograd.grad(y, list(leaf.values()), grad_outputs=s["dy"].double())))
