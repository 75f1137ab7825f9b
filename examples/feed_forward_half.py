"""The feed-forward half of two decoder blocks, a dense one and an expert one, on one GPU.

What follows attention in a block, for a batch of tokens: the output projection of what attention
gave, the norms after it and before the feed-forward part with the residual stream between them,
the feed-forward part, and the norms to the next block.  The first block's feed-forward part is
dense, the second's is the expert layer.  ``backward`` is a training step's way back through the
dense block.

    python examples/feed_forward_half.py            # hidden 7168, a prompt and one token
"""
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sparse_moe_layer_group_amd as moe  # noqa: E402
import synthetic as S  # noqa: E402


class FeedForwardHalf:
    """Weights of a dense block (projection, gated norms, feed-forward block) and of the expert layer
    after it, for batches of up to ``T`` tokens; buffers are made once."""

    def __init__(self, c, T, device="cuda", seed=0):
        self.c, self.T, self.dev = c, T, device
        H, I = c.hidden, c.inter
        self.dtype = torch.float32 if c.act_dtype == "f32" else torch.bfloat16
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, scale, shift=0.0):
            v = torch.randn(shape, generator=g, device=device, dtype=torch.float32)
            return (v * scale + shift).to(self.dtype)

        self.w_o = rand(H, H, scale=H ** -0.5)
        self.ffn_w = {"w_gate": rand(I, H, scale=H ** -0.5), "w_up": rand(I, H, scale=H ** -0.5),
                      "w_down": rand(H, I, scale=I ** -0.5)}
        # around the projection and around the feed-forward part: norm after, gate, norm before the next
        self.norms = [{"w_post": rand(H, scale=0.1, shift=1.0), "w_pre": rand(H, scale=0.1, shift=1.0),
                       "gate": rand(1, H, scale=0.1, shift=0.5)} for _ in range(2)]
        self.moe_cfg = moe.cfg_from(c.with_(T=T))
        self.router = S.gen_router(c, device=device)
        self.bias = S.gen_bias(c, device=device)
        self.experts = S.gen_experts(c, device=device)
        self.lin = moe.make_linear_cfg(H, H, "none", c.act_dtype)
        self.ffn = moe.make_ffn_cfg(H, I, "silu", c.act_dtype)
        self.lin_ws = moe.alloc_linear_workspace(self.lin, T, device)
        self.ffn_ws = moe.alloc_ffn_workspace(self.ffn, T, device)
        self.moe_ws = moe.alloc_workspace(self.moe_cfg, T, device)

    def _norm_cfg(self, T):
        return moe.make_norm_cfg(self.c.hidden, self.c.act_dtype, "rms", gate_rows=T)

    def _new(self, T):
        return torch.empty((T, self.c.hidden), dtype=self.dtype, device=self.dev)

    def forward(self, attn, stream):
        """(stream after both blocks, what ``backward`` needs) for attention's output and the stream."""
        T = attn.shape[0]
        n = self._norm_cfg(T)
        proj, u1, h1, f, u2, h2, out = (self._new(T) for _ in range(7))
        moe.linear_forward(self.lin, attn, self.w_o, proj, self.lin_ws)
        moe.norm_forward(n, stream, proj, self.norms[0], u1, h1)
        moe.ffn_forward(self.ffn, h1, self.ffn_w, f, self.ffn_ws)
        moe.norm_forward(n, u1, f, self.norms[1], u2, h2)
        moe.forward(self.moe_cfg, h2, self.router, self.bias, self.experts, out, self.moe_ws, residual=u2)
        return out, {"attn": attn, "stream": stream, "proj": proj, "u1": u1, "h1": h1, "f": f, "u2": u2, "h2": h2}

    def backward(self, saved, du2, dh2):
        """Gradients of <du2, u2> + <dh2, h2> through the dense block: inputs, weights and norms."""
        T = du2.shape[0]
        n = self._norm_cfg(T)
        ws = moe.alloc_norm_backward_workspace(n, T, self.dev)
        like = torch.empty_like
        g1 = {k: like(v) for k, v in self.norms[1].items()}
        g1.update(residual=self._new(T), branch=self._new(T))
        moe.norm_backward(n, saved["u1"], saved["f"], self.norms[1], du2, dh2, g1, ws)
        dh1, dw = self._new(T), {k: like(v) for k, v in self.ffn_w.items()}
        moe.ffn_backward(self.ffn, saved["h1"], self.ffn_w, g1["branch"], dh1, dw["w_gate"], dw["w_up"], dw["w_down"],
                         moe.alloc_ffn_backward_workspace(self.ffn, T, self.dev))
        g0 = {k: like(v) for k, v in self.norms[0].items()}
        g0.update(residual=self._new(T), branch=self._new(T))
        moe.norm_backward(n, saved["stream"], saved["proj"], self.norms[0], g1["residual"], dh1, g0, ws)
        dattn, dw_o = self._new(T), like(self.w_o)
        moe.linear_backward(self.lin, saved["attn"], self.w_o, g0["branch"],
                            moe.alloc_linear_backward_workspace(self.lin, T, self.dev), dx=dattn, dw=dw_o)
        return {"attn": dattn, "stream": g0["residual"], "w_o": dw_o, "ffn": dw, "norms": [g0, g1]}


def _ms(f, reps):
    f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(reps):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / reps * 1e3


def main():
    c = S.get_config("decode")
    for T in (1, 2048):
        half = FeedForwardHalf(c, T)
        attn, stream, du, dh = (torch.randn((T, c.hidden), device="cuda").to(half.dtype) for _ in range(4))
        _, saved = half.forward(attn, stream)
        print(f"T={T}: both blocks forward {_ms(lambda: half.forward(attn, stream), 5):.3f} ms, "
              f"dense block backward {_ms(lambda: half.backward(saved, du, dh), 5):.3f} ms", flush=True)
        del half, saved
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
