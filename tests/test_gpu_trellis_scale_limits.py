"""Scales that are not finite, through every form of the trellis product (needs a B200)."""
import pytest
import torch

import bcjr_inputs as I
import layer_ref as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("L", [8, 16])
@pytest.mark.parametrize("kind,ckind", [(BF16, BF16), (F16, F16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_infinite_and_nan_scales(L, kind, ckind):
    for n, group in ((50, 50), (50, 100), (64, 16), (64, 64), (64, 0)):
        for tokens in (1, 3, 9, 17):
            _check(L, kind, ckind, n, group, tokens)


def _check(L, kind, ckind, n, group, tokens):
    import differentiable_bcjr_b200 as B
    k, rows, per_row = 2, 30, 4
    cols = per_row * n
    packed = B.trellis_pack(R.random_path(rows * per_row, n, L, k, 5).cuda(), L, k)
    c = (I.codebook(1 << L).abs() + 0.1).to(ckind).cuda()  # of one sign: sums are not 0
    x = (torch.rand(tokens, cols, generator=torch.Generator().manual_seed(1)) + 0.1).to(kind).cuda()
    x[-1] = -x[-1]
    groups = cols // group if group else 1
    scales = torch.ones(groups, rows, device="cuda")
    scales[0, 3] = scales[-1, 4] = float("inf")
    scales[groups // 2, 20] = float("nan")
    y = B.trellis_matmul(x, packed, c, L, k, n, scales, group).float()
    sign = torch.ones(tokens, 1, device="cuda")
    sign[-1] = -1
    assert (y[:, 3:5] * sign == float("inf")).all() and torch.isnan(y[:, 20]).all()
    rest = [r for r in range(rows) if r not in (3, 4, 20)]
    assert torch.isfinite(y[:, rest]).all()
    want = B.trellis_matmul(x, packed, c, L, k, n, torch.ones_like(scales), group).float()
    assert torch.equal(y[:, rest], want[:, rest])
