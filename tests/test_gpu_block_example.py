"""examples/feed_forward_half.py against the 64-bit forms of its operators, each stage from the tensors
that the stage before stored (so that every stage is held to its own roundings)."""
import importlib.util
import os

import pytest
import torch

import oracle as O
import synthetic as S
from tests import block_reference as R
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("feed_forward_half", os.path.join(ROOT, "examples", "feed_forward_half.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def _lift(v):
    return v.detach().cpu().double()


def _lifted(d):
    return {k: _lift(v) for k, v in d.items()}


@pytest.mark.parametrize("name,T", [("tiny", 64), ("tiny", 1), ("mid", 70), ("mid", 5)])
def test_feed_forward_half(name, T):
    c = S.get_config(name)
    H, I, dt = c.hidden, c.inter, c.act_dtype
    print(f"feed-forward half: {name} T={T}", flush=True)
    half = example.FeedForwardHalf(c, T)
    gen = torch.Generator().manual_seed(7)
    attn, stream, du, dh = (torch.randn((T, H), generator=gen).to(half.dtype).to("cuda") for _ in range(4))
    out, s = half.forward(attn, stream)
    tol = lambda roundings, terms: R.tolerance(dt, roundings, terms)  # noqa: E731
    v = _lifted(s)
    assert R.worst(s["proj"], R.linear(v["attn"], _lift(half.w_o))) <= tol(1, H)
    for res, branch, u, h, p in (("stream", "proj", "u1", "h1", 0), ("u1", "f", "u2", "h2", 1)):
        wu, wh = R.norm(v[res], v[branch], _lifted(half.norms[p]))
        assert R.worst(s[u], wu) <= tol(1, H) and R.worst(s[h], wh) <= tol(1, H), u
    assert R.worst(s["f"], R.ffn(v["h1"], _lifted(half.ffn_w))) <= tol(2, H + I)
    # the expert layer, with the stream as its residual
    ex = {k: w.cpu() for k, w in half.experts.items()}
    ref = O.forward(O.lift(s["h2"].cpu()), O.lift(half.router.cpu()), half.bias.cpu().numpy(),
                    lambda e: {k: w[e] for k, w in ex.items()}, n_groups=c.n_groups, topk_groups=c.topk_groups,
                    topk=c.topk, group_topn=c.group_topn, n_shared=c.n_shared)
    ok = torch.from_numpy(~ref.routing.flagged)
    want = v["u2"] + torch.from_numpy(ref.y)
    assert R.worst(out.cpu()[ok], want[ok]) <= (2e-2 if dt == "bf16" else 1e-5)
    # a training step's way back through the dense block
    g = half.backward(s, du, dh)
    w1 = R.norm_grads(v["u1"], v["f"], _lifted(half.norms[1]), _lift(du), _lift(dh))
    for k, got in g["norms"][1].items():
        assert R.worst(got, w1[k]) <= 4 * tol(1, H), ("second norms", k)
    wf = R.ffn_grads(v["h1"], _lifted(half.ffn_w), _lift(g["norms"][1]["branch"]))
    for k, got in g["ffn"].items():
        assert R.worst(got, wf[k]) <= tol(2, 2 * H + I + T), k
    # (the stage between, dh1, is the example's own; from the exact one the first norms are within its roundings)
    w0 = R.norm_grads(v["stream"], v["proj"], _lifted(half.norms[0]), _lift(g["norms"][1]["residual"]), wf["dx"])
    for k, got in g["norms"][0].items():
        assert R.worst(got, w0[k]) <= 4 * tol(3, 3 * H), ("first norms", k)
    wl = R.linear_grads(v["attn"], _lift(half.w_o), None, _lift(g["norms"][0]["branch"]))
    assert R.worst(g["attn"], wl["dx"]) <= tol(1, 2 * H) and R.worst(g["w_o"], wl["dw"]) <= tol(1, H + T)
    assert torch.equal(g["stream"], g["norms"][0]["residual"])
