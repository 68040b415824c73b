"""The group scales of a trellis layer made from weights of any size (needs a B200)."""
import pytest
import torch

import bcjr_inputs as I

pytestmark = pytest.mark.gpu

L, K, N, ROWS, COLS = 8, 2, 64, 12, 256


@pytest.mark.parametrize("group", [0, 64, 16, 128])
@pytest.mark.parametrize("ckind", [None, torch.bfloat16])
def test_groups_of_zeros_stay_zeros(group, ckind):
    from differentiable_bcjr_b200.linear import TrellisLinear
    w, c, x = I.normal((ROWS, COLS), 1).cuda(), I.codebook(1 << L).cuda(), I.normal((5, COLS), 2).cuda()
    w[3] = 0
    w[7, :128] = 0  # whole groups of every size but the row's
    layer = TrellisLinear.from_weight(w, c, L, K, N, group, ckind)
    assert (layer.scales[:, 3] == 0).all() and (layer(x)[:, 3] == 0).all()
    x[:, 128:] = 0
    if group:
        assert (layer(x)[:, 7] == 0).all()
    assert (layer(x)[:, [0, 1, 2, 4]] != 0).all()


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -70, 1e-6, 1e10, 2.0 ** 80])
def test_weights_whose_squares_leave_the_range(group, size):
    import differentiable_bcjr_b200 as B
    from differentiable_bcjr_b200.linear import TrellisLinear
    w, c, x = I.normal((ROWS, COLS), 1).cuda() * size, I.codebook(1 << L).cuda(), I.normal((3, COLS), 2).cuda()
    layer = TrellisLinear.from_weight(w, c, L, K, N, group)
    parts = w.double().view(ROWS, -1, group or COLS)
    rms = parts.square().mean(2).sqrt()
    # a sum of 256 squares in float32, each addition off by 2^-24 at most, and its root by half of that
    assert ((layer.scales.double().t() - rms).abs() <= rms * 130 * 2 ** -24).all()
    wide = layer.scales.t().repeat_interleave(group or COLS, 1)
    _, hard = B.viterbi_decode((w / wide).view(-1, N), c, L, K)
    used = hard.view(ROWS, COLS).double() * wide.double()
    # three roundings of every product, and no more than 64 sums on a value's way
    assert ((layer(x).double() - x.double() @ used.t()).abs() <= x.double().abs() @ used.abs().t() * 67 * 2 ** -24).all()
