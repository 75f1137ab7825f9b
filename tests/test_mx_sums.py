"""The inputs that pin the sums of 8-bit products: what is left out shows in them, by far (planted here, in
the model of the instruction), and the tolerances of the general tests would not show it."""
import pytest
import torch

from tests import block_reference as R
from tests import mx_reference as M
from tests import mx_sums as S


@pytest.mark.parametrize("T,K,N", [(1, 128, 16), (3, 999, 40), (2, 1000, 33), (4, 9, 5)])
def test_products_in_parts_are_exact_and_one_instruction_is_not(T, K, N):
    x, w = S.tokens(T, K, 1), S.weights(N, K, 2)
    want = S.exact(x, w)
    assert torch.equal(S.three_parts(x, w), want)
    one = S.one_instruction(x, w)
    assert (one != want).double().mean() > (0.9 if K > 100 else 0)
    assert ((one - want).abs() <= S.lost(x, w)).all()
    # float32 holds every sum of whole groups: multiples of 2^-10 below 2^24 of them, a single large product too
    rest = torch.arange(K) % 8 >= 2
    assert ((x[:, rest] @ w[:, rest].abs().T + 512) * 2 ** 10).max() < 2 ** 24
    assert torch.equal(want * 2 ** 10, (want * 2 ** 10).round())
    assert torch.equal(want.float().double(), want)


@pytest.mark.parametrize("T,H,I", [(1, 128, 64), (3, 300, 130), (2, 136, 257)])
def test_the_block_shows_a_product_in_one_instruction(T, H, I):
    x, w = S.tokens(T, H, 1), S.block(H, I, 2)
    mid, want = S.through(x, w, S.exact)
    assert torch.equal(M.rounded(mid, "e4m3"), mid) and (mid > 0).all()
    assert torch.equal(want.float().double(), want)
    _, parts = S.through(x, w, S.three_parts)
    assert torch.equal(parts, want)
    up_only = torch.relu(S.one_instruction(x, w["w_gate"])) * S.one_instruction(x, w["w_up"])
    assert (up_only != mid).double().mean() > 0.7            # the up projection's loss alone shows
    down_only = S.one_instruction(mid * 64, w["w_down"], torch.full_like(mid, 1 / 64))
    assert (down_only != want).double().mean() > 0.5         # and the down projection's


def test_general_tolerances_do_not_show_it():
    # random operands as the general tests have them: a float32 block whose products take one instruction a
    # step stays within the tolerance there
    g = torch.Generator().manual_seed(1)
    T, H, I = 17, 130, 33

    def values(rows, cols, form, scale):
        v = torch.randn((rows, cols), generator=g, dtype=M.F64) * scale
        return v, M.quantize(v, form)

    def apart(c, s, form, cols):
        return M.values(c, s, form, cols), torch.exp2(s.to(M.F64) - 127).repeat_interleave(32, 1)[:, :cols]

    def product(x, sx, w, sw):
        # blocks one after the other, with the weights' scales
        at = [slice(k, k + 32) for k in range(0, x.shape[1], 32)]
        return sum(S.one_instruction(x[:, b] / sx[:, b], w[:, b] / sw[:, b], sx[:, b]) * sw[None, :, b.start] for b in at)

    x = apart(*values(T, H, "e4m3", 1.0)[1], "e4m3", H)
    w = {k: apart(*values(r, c, "e2m1", c ** -0.5)[1], "e2m1", c)
         for k, r, c in (("w_gate", I, H), ("w_up", I, H), ("w_down", H, I))}
    mid = R.act("silu", product(*x, *w["w_gate"])) * product(*x, *w["w_up"])
    c, s = M.quantize(mid, "e4m3")
    got = product(*apart(c, s, "e4m3", I), *w["w_down"])
    want = M.ffn(x[0], {k: v[0] for k, v in w.items()}, None, "silu", "e4m3")
    assert 0 < R.worst(got, want) <= M.tolerance("f32", I, "e4m3") + M.flips("f32", H, "e4m3")
