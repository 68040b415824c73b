"""4-bit quantisation of groups whose scales are at the ends of their type's range (needs a B200)."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TINY = {F32: 2.0 ** -149, F16: 2.0 ** -24, BF16: 2.0 ** -133}  # steps of the smallest values


def _check(w, group, zero, scale):
    import differentiable_bcjr_b200 as B
    rows, cols = w.shape
    packed, scales, zeros = B.int4_quantize(w, group, zero, scale)
    g = torch.arange(cols, device="cuda") // (group or cols)
    parts = [w.double()[:, g == i] for i in range(int(g[-1]) + 1)]
    lo, hi = (torch.stack([f(p) for p in parts]) for f in (lambda p: p.amin(1).clamp(max=0), lambda p: p.amax(1).clamp(min=0)))
    want = (hi - lo) / 15 if zero else torch.maximum(hi, -lo) / 7
    # three roundings to float32 and one to the scale's type, by half a step each (of the smallest values where those are meant)
    assert ((scales.double() - want).abs() <= want * (3 * 2 ** -24 + torch.finfo(scale).eps / 2) + 3 * 2.0 ** -150 + TINY[scale] / 2).all()
    s = scales.double()
    held = s > 0
    per = torch.where(held, s, torch.ones_like(s))
    z = torch.where(held, -lo / per, torch.zeros_like(s)).clamp(0, 15) if zero else torch.full_like(s, 8)
    if zero:
        # next to a tie either integer
        assert ((zeros.double() - z).abs() <= 0.5 + 2 ** -18).all()
        z = zeros.double()
    t = torch.where(held[g].t(), w.double() / per[g].t(), torch.zeros_like(w, dtype=torch.float64)) + z[g].t()
    got = R.unpack_int4(packed, rows, cols)
    assert ((got - t.clamp(0, 15)).abs() <= 0.5 + 2 ** -18).all()
    assert (got[w == 0] == z[g].t()[w == 0]).all()
    full = R.unpack_int4(packed, packed.shape[0] * 16, packed.shape[1] * 128)
    full[:rows, :cols] = 8
    assert (full == 8).all()
    return packed, scales, zeros


def _rows_of_all_sizes(cols, kind, lowest, highest):
    """Rows whose largest magnitudes run over the powers of two between the exponents, random, with zeros and both signs."""
    n = highest - lowest + 1
    w = torch.rand(n, cols, generator=torch.Generator().manual_seed(6)).double() * 2 - 1
    w[:, 0], w[:, 1], w[:, 2] = 1, -1, 0
    w[1::3] = w[1::3].abs()
    w[2::3, 3:] *= 0.1
    return (w * 2.0 ** torch.arange(lowest, highest + 1).double()[:, None]).to(kind).cuda()


@pytest.mark.parametrize("cols,group", [(32, 32), (100, 32), (192, 64), (300, 128), (700, 256), (515, 0)])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("kind,scale", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
def test_tiny_groups(cols, group, zero, kind, scale):
    import differentiable_bcjr_b200 as B
    w = _rows_of_all_sizes(cols, kind, -148, -118)
    packed, scales, zeros = _check(w, group, zero, scale)
    # what a product makes of the codes is what they stand for: identity columns leave one product each, of an integer
    # of up to 4 bits and a 24-bit mantissa, whose 28 bits float32 rounds once (exact where it is subnormal)
    x = torch.eye(cols, device="cuda")[::7].contiguous()
    y = B.int4_matmul(x, packed, scales, zeros, group)
    want = R.int4_weights(packed, scales, zeros, *w.shape, group)[:, ::7].t()
    assert ((y.double() - want).abs() <= want.abs() * 2 ** -24).all()


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("kind", [F32, F16])
@pytest.mark.parametrize("group", [32, 0])
def test_subnormal_half_scales(zero, kind, group):
    _check(_rows_of_all_sizes(96, kind, -24, -8), group, zero, F16)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("scale", [F32, BF16])
def test_huge_groups(zero, scale):
    _check(_rows_of_all_sizes(96, F32, 100, 126), 32, zero, scale)
