"""The operators with microscaled operands, as cases to be timed and compared.

A microscaled matrix has blocks of 32 consecutive elements of a row that share a power of two: value =
element * 2^e, e = floor(log2(largest magnitude)) - emax, elements E4M3 (8 bits, emax 8) or E2M1
(4 bits, emax 2), rounded to nearest even and saturated.

* ``quantize``: a matrix to that form, and its values back;
* ``norm``: ``u = s * residual + gate * post(branch)``, ``h = pre(u)`` with h in that form;
* ``linear``: ``y = residual + act(x W^T + b)``, x in either form, W in 4 bits;
* ``ffn``: ``y = residual + m Wd^T``, ``m = act(x Wg^T) * (x Wu^T)`` in x's form.

``own = False`` computes them from elementary torch operations in 32 bits, rounded once at the end;
``own = True`` calls this package's entry points.  ``exact`` is the 64-bit value.  What is held in 8
or 4 bits is returned as its values, which bfloat16 holds exactly.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
RES_SCALE = 0.75      # depth-scaled residual streams use values like this one
H, I = 7168, 2048     # the layer's hidden and expert widths

EMAX = {"e4m3": 8, "e2m1": 2}
MOST = {"e4m3": 448.0, "e2m1": 6.0}
LOWEST = {"e4m3": -6, "e2m1": 0}      # exponent of the smallest normal element
MANTISSA = {"e4m3": 3, "e2m1": 1}
# magnitudes by code
GRID = {"e2m1": [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0],
        "e4m3": [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # an up projection's weights, laid out when a model is loaded
        _quantize("quantize weights", I, H, "e2m1"),
        # activations that are columns of a wider tensor, of sizes that nothing divides
        _quantize("quantize odd", 777, 1001, "e4m3", dtype="f32", pad=23),
        # one token of a serving loop between two blocks: pure latency
        _norm("norm one token", 1, H, "e4m3"),
        # a long prompt, per-channel gate (layer scale)
        _norm("norm prompt", 8192, H, "e4m3", gate_rows=8192),
        # three sequences with a gate row each, layer norms with biases, 4-bit output, an odd width
        _norm("norm odd layer", 777, 1001, "e2m1", kind="layer", gate_rows=259, dtype="f32"),
        # one token through a square projection into the residual stream
        _linear("linear one token", 1, H, H, "e4m3"),
        # sizes that no tile divides, both operands in 4 bits
        _linear("linear odd", 333, 1001, 777, "e2m1", act="gelu", pad=23),
        # a prompt through a square projection, 8-bit activations
        _linear("linear prompt", 4096, H, H, "e4m3"),
        # a prompt, both operands in 4 bits
        _linear("linear prompt 4 bit", 8192, H, I, "e2m1", act="silu"),
        # serving: one token, and a ragged batch of them, through a dense block of the shared
        # expert's size; and a prompt (the prefill batch)
        _ffn("ffn one token", 1, H, I, "e4m3"),
        _ffn("ffn small batch", 50, H, I, "e4m3"),
        _ffn("ffn prompt", 8192, H, I, "e4m3"),
    ]


def _named(name, case):
    return case if name is None else dict(case, name=name)


def _quantize(name, rows, cols, form, dtype="bf16", pad=0):
    return _named(name, {"op": "quantize", "T": rows, "cols": cols, "form": form, "dtype": dtype, "pad": pad})


def _norm(name, T, hidden, form, kind="rms", gate_rows=0, dtype="bf16", pad=0):
    return _named(name, {"op": "norm", "T": T, "hidden": hidden, "form": form, "kind": kind, "gate_rows": gate_rows,
                         "dtype": dtype, "pad": pad})


def _linear(name, T, n_in, n_out, form, act="none", dtype="bf16", pad=0):
    return _named(name, {"op": "linear", "T": T, "n_in": n_in, "n_out": n_out, "form": form, "act": act,
                         "dtype": dtype, "pad": pad})


def _ffn(name, T, hidden, inter, form, act="silu", dtype="bf16", pad=0):
    return _named(name, {"op": "ffn", "T": T, "hidden": hidden, "inter": inter, "form": form, "act": act,
                         "dtype": dtype, "pad": pad})


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: two of three are multiples of 64 or 8, the third is whatever it is."""
    w, kind = _log(rng, lo, hi), rng.randrange(3)
    step = (64, 8, 1)[kind]
    return max(step, w // step * step)


def draw(rng):
    op = rng.choice(("quantize", "norm", "linear", "ffn"))
    form = rng.choice(("e4m3", "e2m1"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    pad = rng.choice((0, 0, 8, 5))
    if op == "quantize":
        cols = _width(rng, 32, 16384)
        return _quantize(None, min(30000, _log(rng, 1, max(1, 8192 * H // cols))), cols, form, dtype, pad)
    if op == "norm":
        hidden = _width(rng, 64, 8192)
        T = min(30000, _log(rng, 1, max(1, 8192 * H // hidden)))
        rows = rng.choice((0, T, 1, T))
        if rng.random() < 0.3 and T >= 8:
            rows = max(1, T // 4)
            T = 4 * rows
        return _norm(None, T, hidden, form, rng.choice(("rms", "rms", "layer")), rows, dtype, pad)
    a, b = _width(rng, 128, H), _width(rng, 64, H)
    T = _log(rng, 1, max(1, min(16384, 8192 * H * I // (a * b))))
    acts = ("silu", "gelu", "relu")
    if op == "ffn":
        # an element of the middle whose sums fall on either side of the border between two codes moves
        # by a whole step in one of two right computations: more than a float32 result may be off
        return _ffn(None, T, a, b, form, rng.choice(acts), "bf16", pad)
    return _linear(None, T, a, b, form, rng.choice(("none",) + acts), dtype, pad)


# ---------------------------------------------------------------- the form, 32 bits


def _power(e):
    """2^e as float32 for integers -126 <= e <= 127, and 2^-127."""
    return torch.where(e >= -126, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _blocks(v):
    """[rows][cols] float32 with zeros up to the next multiple of 128 columns, as blocks of 32."""
    rows, cols = v.shape
    full = torch.zeros((rows, (cols + 127) // 128 * 128), dtype=torch.float32, device=v.device)
    full[:, :cols] = v
    return full.view(rows, -1, 32)


def _scaled(v, form):
    """The blocks' elements, rounded, and their exponents."""
    blocks = _blocks(v)
    amax = blocks.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent.to(torch.int64) - 1 - EMAX[form], -127).clamp(min=-127)
    a = (blocks * _power(-e)).abs().clamp(max=MOST[form])
    least = torch.frexp(a).exponent.to(torch.int64) - 1
    step = _power(torch.where(a > 0, least, -200).clamp(min=LOWEST[form]) - MANTISSA[form])
    return torch.copysign(torch.round(a / step) * step, blocks), e


def _values(v, form):
    """The values that v has in microscaled form, float32."""
    q, e = _scaled(v, form)
    return (q * _power(e)).view(q.shape[0], -1)[:, :v.shape[1]]


def _encode(v, form):
    """(codes, scales) of v: bytes, rows padded to a multiple of 128 columns, low four bits first."""
    q, e = _scaled(v, form)
    rows = q.shape[0]
    grid = torch.tensor(GRID[form], device=q.device)
    sign = torch.signbit(q).to(torch.uint8)
    code = torch.searchsorted(grid, q.abs()).to(torch.uint8)
    if form == "e4m3":
        codes = code | sign << 7
    else:
        code = (code | sign << 3).view(rows, -1, 2)
        codes = code[..., 0] | code[..., 1] << 4
    return codes.view(rows, -1).contiguous(), (e + 127).to(torch.uint8).view(rows, -1).contiguous()


def _tables(form):
    """The elements by code, and 2^e by scale byte."""
    grid = torch.tensor(GRID[form] + [math.nan] * (form == "e4m3"), device=DEV)
    return torch.cat((grid, -grid)), _power(torch.arange(-127, 128, device=DEV))


def _decode(m, cols, tables):
    """The float32 values of codes and scales."""
    codes, scales, form = m
    elements, powers = tables[form]
    rows = codes.shape[0]
    if form == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).view(rows, -1)
    v = elements[codes.int()].view(rows, -1, 32) * powers[scales.int()].view(rows, -1, 1)
    return v.view(rows, -1)[:, :cols]


# ---------------------------------------------------------------- inputs


def _rand(gen, dtype, *shape, scale=1.0, shift=0.0):
    v = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return (v * scale + shift).to(dtype)


def _rows(gen, dtype, T, cols, pad, scale=1.0):
    """[T][cols] activations; with `pad`, the columns of a wider tensor."""
    return _rand(gen, dtype, T, cols + pad, scale=scale)[:, :cols]


def _stream(gen, dtype, T, cols, pad, scale=2.0):
    """Rows of a residual stream, which has a few channels far larger than the others."""
    v = _rows(gen, dtype, T, cols, pad, scale)
    v[:, torch.randint(0, cols, (max(1, cols // 500),), generator=gen, device=DEV)] *= 16
    return v


def _matrix(gen, rows, cols, form, scale):
    """A weight, or normed activations, in microscaled form: (codes, scales, form)."""
    return (*_encode(_rand(gen, torch.float32, rows, cols, scale=scale), form), form)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt, T, pad, form = TYPES[case["dtype"]], case["T"], case["pad"], case["form"]
    s = {"case": case, "tables": {k: _tables(k) for k in GRID}}
    if case["op"] == "quantize":
        s["x"] = _stream(g, dt, T, case["cols"], pad)
        s["values"] = torch.empty((T, case["cols"]), dtype=dt, device=DEV)
    elif case["op"] == "norm":
        h = case["hidden"]
        layer = case["kind"] == "layer"
        s["residual"], s["branch"] = _stream(g, dt, T, h, pad), _rows(g, dt, T, h, pad, scale=0.5)
        p = {"w_post": _rand(g, dt, h, scale=0.1, shift=1.0), "w_pre": _rand(g, dt, h, scale=0.1, shift=1.0)}
        p["b_post"] = _rand(g, dt, h, scale=0.1) if layer else None
        p["b_pre"] = _rand(g, dt, h, scale=0.1) if layer else None
        n = case["gate_rows"]
        p["gate"] = _rand(g, dt, T // n, h, scale=0.3, shift=0.5) if n else None
        s["params"] = p
        s["u"] = torch.empty((T, h), dtype=dt, device=DEV)
        s["values"] = torch.empty((T, h), dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "linear":
        k, n = case["n_in"], case["n_out"]
        s["x"], s["w"] = _matrix(g, T, k, form, 1.0), _matrix(g, n, k, "e2m1", k ** -0.5)
        s["bias"], s["residual"] = _rand(g, dt, n, scale=0.2), _rows(g, dt, T, n, pad)
        s["y"] = torch.empty((T, n), dtype=dt, device=DEV)
    else:
        h, i = case["hidden"], case["inter"]
        s["x"] = _matrix(g, T, h, form, 1.0)
        s["w"] = {"w_gate": _matrix(g, i, h, "e2m1", h ** -0.5), "w_up": _matrix(g, i, h, "e2m1", h ** -0.5),
                  "w_down": _matrix(g, h, i, "e2m1", i ** -0.5)}
        s["residual"] = _rows(g, dt, T, h, pad)
        s["y"] = torch.empty((T, h), dtype=dt, device=DEV)
    if own:
        _own_plan(s, case)
    return s


def _own_plan(s, c):
    """The configuration, buffers and workspace that a program makes once for its layers."""
    import sparse_moe_layer_group_amd as moe

    T, form = c["T"], c["form"]
    if c["op"] == "quantize":
        s["mx"] = moe.alloc_mx(T, c["cols"], form, DEV)
    elif c["op"] == "norm":
        s["cfg"] = moe.make_norm_cfg(c["hidden"], c["dtype"], c["kind"], c["gate_rows"], EPS, RES_SCALE)
        s["mx"] = moe.alloc_mx(T, c["hidden"], form, DEV)
    elif c["op"] == "linear":
        s["cfg"] = moe.make_mx_linear_cfg(c["n_in"], c["n_out"], c["act"], c["dtype"], form)
        s["mx"], s["mw"] = moe.MxMatrix(*s["x"], c["n_in"]), moe.MxMatrix(*s["w"], c["n_in"])
        s["ws"] = moe.alloc_mx_linear_workspace(s["cfg"], T, DEV)
    else:
        h, i = c["hidden"], c["inter"]
        s["cfg"] = moe.make_mx_ffn_cfg(h, i, c["act"], c["dtype"], form)
        s["mx"] = moe.MxMatrix(*s["x"], h)
        s["mw"] = {k: moe.MxMatrix(*v, i if k == "w_down" else h) for k, v in s["w"].items()}
        s["ws"] = moe.alloc_mx_ffn_workspace(s["cfg"], T, DEV)


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    if own:
        return _own_run(s, c)
    plain = {"quantize": _plain_quantize, "norm": _plain_norm, "linear": _plain_linear, "ffn": _plain_ffn}
    return plain[c["op"]](s, c, TYPES[c["dtype"]])


def _own_run(s, c):
    import sparse_moe_layer_group_amd as moe

    if c["op"] == "quantize":
        moe.mx_quantize(s["x"], s["mx"])
        moe.mx_dequantize(s["mx"], s["values"])
        return {"values": s["values"]}
    if c["op"] == "norm":
        moe.norm_mx_forward(s["cfg"], s["residual"], s["branch"], s["params"], s["u"], s["mx"])
        moe.mx_dequantize(s["mx"], s["values"])
        return {"u": s["u"], "h": s["values"]}
    if c["op"] == "linear":
        moe.mx_linear_forward(s["cfg"], s["mx"], s["mw"], s["y"], s["ws"], bias=s["bias"], residual=s["residual"])
    else:
        moe.mx_ffn_forward(s["cfg"], s["mx"], s["mw"], s["y"], s["ws"], residual=s["residual"])
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


def _unit(v, kind):
    """The rows of v, centred where `kind` says so, over their root mean square."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def _plain_quantize(s, c, dt):
    return {"values": _values(s["x"].float(), c["form"]).to(dt)}


def _plain_norm(s, c, dt):
    p = {k: v.float() for k, v in s["params"].items() if v is not None}
    n = _unit(s["branch"].float(), c["kind"]) * p["w_post"]
    if "b_post" in p:
        n = n + p["b_post"]
    if "gate" in p:
        n = n * p["gate"].repeat_interleave(c["gate_rows"], 0)
    u = RES_SCALE * s["residual"].float() + n
    h = _unit(u, c["kind"]) * p["w_pre"]
    if "b_pre" in p:
        h = h + p["b_pre"]
    return {"u": u.to(dt), "h": _values(h, c["form"]).to(torch.bfloat16)}


def _plain_linear(s, c, dt):
    k, tables = c["n_in"], s["tables"]
    z = _decode(s["x"], k, tables) @ _decode(s["w"], k, tables).t() + s["bias"].float()
    return {"y": (s["residual"].float() + _act(z, c["act"])).to(dt)}


def _plain_ffn(s, c, dt):
    h, w, tables = c["hidden"], s["w"], s["tables"]
    x = _decode(s["x"], h, tables)
    mid = _act(x @ _decode(w["w_gate"], h, tables).t(), c["act"]) * (x @ _decode(w["w_up"], h, tables).t())
    y = _values(mid, c["form"]) @ _decode(w["w_down"], c["inter"], tables).t()
    return {"y": (s["residual"].float() + y).to(dt)}


# ---------------------------------------------------------------- work


def _bytes(rows, cols, form):
    """Of a matrix in microscaled form: its codes and a byte for each block."""
    return rows * cols * ({"e4m3": 1.0, "e2m1": 0.5}[form] + 1 / 32)


def work(case):
    T, b, form = case["T"], 4 if case["dtype"] == "f32" else 2, case["form"]
    if case["op"] == "quantize":
        return {"bytes": 2 * b * T * case["cols"], "flops": 8.0 * T * case["cols"]}
    if case["op"] == "norm":
        h, n = case["hidden"], case["gate_rows"]
        params = h * ((4 if case["kind"] == "layer" else 2) + (T // n if n else 0))
        # residual and branch in, u and the values of h out
        return {"bytes": b * (3 * T * h + params) + 2 * T * h, "flops": 22.0 * T * h}
    if case["op"] == "ffn":
        h, i = case["hidden"], case["inter"]
        return {"bytes": _bytes(T, h, form) + 3 * _bytes(h, i, "e2m1") + 2 * b * T * h, "flops": 6.0 * T * h * i}
    k, n = case["n_in"], case["n_out"]
    return {"bytes": _bytes(T, k, form) + _bytes(n, k, "e2m1") + b * (2 * T * n + n), "flops": 2.0 * T * k * n}


# ---------------------------------------------------------------- 64 bits


def _nearest(v, form):
    """v's values in the form, 64 bits: the nearest of the elements there are, by the places between them."""
    rows, cols = v.shape
    pad = torch.nn.functional.pad(v, (0, -cols % 32)).view(rows, -1, 32)
    top = pad.abs().max(-1, keepdim=True).values
    scale = torch.exp2(torch.clamp(torch.floor(torch.log2(top)) - EMAX[form], min=-127))
    grid = torch.tensor(GRID[form], dtype=torch.float64, device=v.device)
    between = (grid[1:] + grid[:-1]) / 2
    a = pad.abs() / scale
    low, high = torch.bucketize(a, between), torch.bucketize(a, between, right=True)
    code = torch.where(low % 2 == 0, low, high)  # they differ where a lies between two elements
    return (torch.sign(pad) * grid[code] * scale).view(rows, -1)[:, :cols]


def _wide(m, cols):
    """The values of codes and scales, from the bits' meaning."""
    codes, scales, form = m
    if form == "e4m3":
        v = codes.view(torch.float8_e4m3fn).double()
    else:
        c = torch.stack((codes % 16, codes // 16), -1).flatten(1).double()
        sign, c = torch.where(c < 8, 1.0, -1.0).double(), c % 8
        v = sign * torch.where(c < 2, c / 2, (2 + c % 2) * torch.exp2(torch.floor(c / 2) - 2))
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1))[:, :cols]


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    f = torch.nn.functional
    act = {"none": lambda z: z, "relu": torch.relu, "silu": lambda z: z * torch.sigmoid(z),
           "gelu": lambda z: z * 0.5 * torch.erfc(-z / math.sqrt(2.0))}
    if case["op"] == "quantize":
        return {"values": _nearest(s["x"].double(), case["form"])}
    if case["op"] == "norm":
        p = {k: v.double() for k, v in s["params"].items() if v is not None}

        def norm(v, w, b):
            if case["kind"] == "layer":
                var, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
                return (v - mean) * torch.rsqrt(var + EPS) * w + b
            return v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + EPS) * w

        n = norm(s["branch"].double(), p["w_post"], p.get("b_post"))
        if "gate" in p:
            n = (n.view(p["gate"].shape[0], -1, n.shape[1]) * p["gate"][:, None, :]).view(n.shape)
        u = n + s["residual"].double() * RES_SCALE
        return {"u": u, "h": _nearest(norm(u, p["w_pre"], p.get("b_pre")), case["form"])}
    if case["op"] == "linear":
        y = f.linear(_wide(s["x"], case["n_in"]), _wide(s["w"], case["n_in"]), s["bias"].double())
        return {"y": s["residual"].double() + act[case["act"]](y)}
    h, w = case["hidden"], s["w"]
    x = _wide(s["x"], h)
    mid = act[case["act"]](f.linear(x, _wide(w["w_gate"], h))) * f.linear(x, _wide(w["w_up"], h))
    return {"y": s["residual"].double() + f.linear(_nearest(mid, case["form"]), _wide(w["w_down"], case["inter"]))}
