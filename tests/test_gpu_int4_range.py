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


@pytest.mark.parametrize("tokens", [1, 2, 3, 7, 12])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 0])
@pytest.mark.parametrize("rows", [40, 5000])
def test_float32_tokens_under_an_infinite_scale(tokens, group, rows):
    import differentiable_bcjr_b200 as B
    # float32 tokens are multiplied in parts, some of them zero: 0 times infinity must not reach the sum
    cols = 300
    gen = torch.Generator().manual_seed(tokens)
    groups = -(-cols // group) if group else 1
    packed = (torch.randint(0, 256, (-(-rows // 16), 3, 1024), generator=gen, dtype=torch.uint8) | 0x88).cuda()  # codes 8..15
    scales = (0.004 + 0.01 * torch.rand(groups, rows, generator=gen)).cuda()
    zeros = torch.ones(groups, rows, dtype=torch.uint8, device="cuda")
    scales[0, 3] = scales[-1, 7] = float("inf")
    scales[groups // 2, 11] = float("nan")
    x = torch.rand(tokens, cols, generator=gen).cuda() + 0.5
    x[0] = 1.0  # one part holds all of it
    x[-1] = x[-1].neg().half().float() if tokens > 1 else x[-1]  # two parts do
    want = x.double() @ R.int4_weights(packed, scales, zeros, rows, cols, group).t()
    y = B.int4_matmul(x, packed, scales, zeros, group).double()
    assert torch.isinf(want[:, [3, 7]]).all() and torch.isnan(want[:, 11]).all()
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(y), torch.isinf(want))
    assert torch.equal(y[torch.isinf(y)], want[torch.isinf(want)])
    fine = torch.isfinite(want)
    # positive codes and tokens of one sign: the size of the sum is the sum
    assert ((y[fine] - want[fine]).abs() <= want[fine].abs() * 64 * 2 ** -23).all()


@pytest.mark.parametrize("tokens", [1, 4, 9])
def test_nan_tokens_of_every_payload(tokens):
    import differentiable_bcjr_b200 as B
    packed = torch.full((1, 2, 1024), 0x99, dtype=torch.uint8, device="cuda")  # codes 9: ones
    x = torch.ones(tokens, 256, device="cuda")
    for bits in (0x7F800001, 0x7FC00000, 0x7F80FFFF, 0x7F810000, -1):
        x.view(torch.int32)[-1, 77] = bits
        for s in (1.0, float("inf")):
            y = B.int4_matmul(x, packed, torch.full((1, 16), s, device="cuda"), None, 0)
            assert torch.isnan(y[-1]).all() and (y[:-1] == 256 * s).all()


@pytest.mark.parametrize("tokens", [1, 3, 10])
@pytest.mark.parametrize("exponent", [-149, -143, -140, -135, -131, -126, -120, -113, -107, -100, 0, 100, 119])
def test_float32_tokens_of_every_size_are_multiplied_exactly(tokens, exponent):
    import differentiable_bcjr_b200 as B
    rows, cols = 64, 256
    gen = torch.Generator().manual_seed(tokens)
    packed = torch.randint(0, 256, (4, 2, 1024), generator=gen, dtype=torch.uint8).cuda()
    scales = torch.ones(1, rows, device="cuda")
    w = R.int4_weights(packed, scales, None, rows, cols, 0)
    x = ((torch.rand(tokens, cols, generator=gen).double() + 1) * 2.0 ** exponent * (1 - 2 * torch.randint(0, 2, (tokens, cols), generator=gen))).float().cuda()
    y = B.int4_matmul(x, packed, scales, None, 0).double()
    want, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    # exact products; no more than 64 float32 sums on a value's way, each off by 2^-23 of it or half a smallest number
    assert ((y - want).abs() <= size * 64 * 2 ** -23 + 64 * 2.0 ** -150).all()
    # one token value at a time: its product alone, rounded once (28 bits; parts are at most two sums more)
    x = torch.zeros_like(x)
    x[:, 77] = (1 + 2.0 ** -23) * 2.0 ** exponent
    x[-1, 77] = -(2 - 2.0 ** -23) * 2.0 ** exponent
    y, want = B.int4_matmul(x, packed, scales, None, 0).double(), x.double() @ w.t()
    assert ((y - want).abs() <= want.abs() * 3 * 2 ** -24).all()
