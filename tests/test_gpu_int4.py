"""4-bit quantisation and products against their definitions in 64 bits (needs a B200)."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _w(rows, cols, dtype, seed):
    return (torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)) * 0.02).to(dtype).cuda()


@pytest.mark.parametrize("rows,cols,group", [(1, 1, 0), (16, 128, 128), (17, 129, 128), (33, 300, 32), (5, 64, 64), (40, 1000, 64),
                                             (100, 1024, 256), (3, 2050, 384), (20, 700, 0), (64, 96, 128), (257, 515, 32)])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("kind,scale", [(F32, F32), (BF16, BF16), (F16, F32), (F32, BF16), (F32, F16)])
def test_quantize_matches_the_definition(rows, cols, group, zero, kind, scale):
    import differentiable_bcjr_b200 as B
    w = _w(rows, cols, kind, rows + cols)
    packed, scales, zeros = B.int4_quantize(w, group, zero, scale)
    codes, s, z = R.quantize(w, group, zero, scale)
    # the extreme values' difference is rounded once before the division: a last place of float32, which
    # may become one of the scale's type
    assert ((scales.double() - s.double()).abs() <= s.double() * torch.finfo(scale).eps * 1.01 + (1e-7 if scale == F16 else 0)).all()
    # a code may differ where the quotient is next to a tie, and by one
    g = torch.arange(cols, device="cuda") // (group or cols)
    got = R.unpack_int4(packed, rows, cols)
    assert (got - codes).abs().max() <= 1
    zz = zeros.double()[g].t() if zero else 8.0
    t = w.double() / scales.double()[g].t() + zz
    assert (((got - t).abs() <= 0.5 + 2 ** -18) | (got == 0) | (got == 15)).all()
    if zero:
        assert (zeros.long() - z.long()).abs().max() <= 1
    # the tiles' padding holds eights
    full = R.unpack_int4(packed, packed.shape[0] * 16, packed.shape[1] * 128)
    full[:rows, :cols] = 8
    assert (full == 8).all()


def test_quantize_of_zeros_and_non_finite_weights():
    import differentiable_bcjr_b200 as B
    w = _w(20, 256, F32, 1)
    w[3, :128] = 0
    w[4, 7], w[5, 200] = float("nan"), float("inf")
    for zero in (False, True):
        packed, scales, zeros = B.int4_quantize(w, 128, zero)
        assert scales[0, 3] == 0 and not torch.isfinite(scales[0, 4]) and not torch.isfinite(scales[1, 5])
        assert torch.isfinite(scales).sum() == 38
        q = R.unpack_int4(packed, 20, 256)
        assert (q[3, :128] == (zeros[0, 3] if zero else 8)).all()


def test_quantize_of_unaligned_weights():
    import differentiable_bcjr_b200 as B
    for kind in (F32, BF16):
        flat = torch.zeros(1 + 40 * 256, dtype=kind, device="cuda")
        w = flat[1:].view(40, 256)
        w.copy_(_w(40, 256, kind, 3))
        a, b = B.int4_quantize(w, 64), B.int4_quantize(w.clone(), 64)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _layer(rows, cols, group, zero, scale, seed):
    gen = torch.Generator().manual_seed(seed)
    groups = -(-cols // group) if group else 1
    packed = torch.randint(0, 256, (-(-rows // 16), -(-cols // 128), 1024), generator=gen, dtype=torch.uint8).cuda()
    scales = (0.004 + 0.01 * torch.rand(groups, rows, generator=gen)).to(scale).cuda()
    zeros = torch.randint(0, 16, (groups, rows), generator=gen, dtype=torch.uint8).cuda() if zero else None
    return packed, scales, zeros


def _tolerance(x, w, group, dtype):
    """Half a step of y's type, and 2^-23 of the sum of magnitudes for each float32 sum on a value's way: the mma
    of a scaling's columns, the scalings of a warp's blocks, eight warps, eight CTAs, three parts."""
    blocks = -(-x.shape[-1] // 128)
    depth = 16 + -(-blocks // 8) * (4 if group == 32 else 2 if group == 64 else 1) + 8 + 8 + 3
    size = x.double().abs() @ w.abs().t()
    y = x.double() @ w.t()
    return y, y.abs() * torch.finfo(dtype).eps / 2 + size * depth * 2 ** -23 + (2.0 ** -25 if dtype == F16 else 0)


@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8, 9, 16, 17, 33, 70])
@pytest.mark.parametrize("rows,cols,group", [(16, 128, 128), (50, 300, 32), (17, 1000, 64), (257, 2176, 256), (5, 77, 0), (2048, 512, 128),
                                             (33, 8192, 0)])
@pytest.mark.parametrize("kind,scale", [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32)])
def test_matmul_matches_the_definition(tokens, rows, cols, group, kind, scale):
    import differentiable_bcjr_b200 as B
    zero = (tokens + rows) % 2 == 0
    packed, scales, zeros = _layer(rows, cols, group, zero, scale, rows + tokens)
    x = torch.randn(tokens, cols, generator=torch.Generator().manual_seed(7)).to(kind).cuda()
    y = B.int4_matmul(x, packed, scales, zeros, group)
    want, tol = _tolerance(x, R.int4_weights(packed, scales, zeros, rows, cols, group), group, kind)
    assert y.dtype == kind and y.shape == (tokens, rows)
    assert ((y.double() - want).abs() <= tol).all(), ((y.double() - want).abs() / tol).max()


def test_matmul_shapes_views_and_outputs():
    import differentiable_bcjr_b200 as B
    packed, scales, zeros = _layer(40, 256, 64, True, F32, 1)
    w = R.int4_weights(packed, scales, zeros, 40, 256, 64)
    flat = torch.randn(1 + 6 * 256, device="cuda").bfloat16()
    x = flat[1:].view(2, 3, 256)  # not 16-byte aligned
    out = torch.empty(2, 3, 40, dtype=BF16, device="cuda")
    assert B.int4_matmul(x, packed, scales, zeros, 64, out=out) is out
    want, tol = _tolerance(x.view(6, 256), w, 64, BF16)
    assert ((out.double().view(6, 40) - want).abs() <= tol).all()
    assert torch.equal(B.int4_matmul(x.clone(), packed, scales, zeros, 64), out)
    one = B.int4_matmul(x[1, 2].clone(), packed, scales, zeros, 64)
    assert one.shape == (40,) and torch.equal(one, out[1, 2])
    assert B.int4_matmul(x[:0].clone(), packed, scales, zeros, 64).shape == (0, 3, 40)


def test_an_output_over_its_input_is_refused():
    import differentiable_bcjr_b200 as B
    packed, scales, _ = _layer(256, 256, 64, False, F32, 1)
    buf = torch.randn(2 * 256 + 5, device="cuda")
    x = buf[:256].view(1, 256)
    before = buf.clone()
    for out in (x, buf[5:261].view(1, 256), buf[255:511].view(1, 256)):
        with pytest.raises(ValueError):
            B.int4_matmul(x, packed, scales, None, 64, out=out)
    assert torch.equal(buf, before)
    B.int4_matmul(x, packed, scales, None, 64, out=buf[256:512].view(1, 256))
    assert torch.equal(buf[:256], before[:256]) and torch.equal(buf[512:], before[512:])


def test_matmul_of_infinite_and_nan_inputs():
    import differentiable_bcjr_b200 as B
    packed, scales, zeros = _layer(40, 256, 64, False, F32, 2)
    w = R.int4_weights(packed, scales, zeros, 40, 256, 64)
    for kind in (F32, F16, BF16):
        x = torch.randn(4, 256, device="cuda").to(kind)
        x[1, 5], x[2, 100] = float("inf"), float("nan")
        want = x.double() @ w.t()
        y = B.int4_matmul(x, packed, scales, zeros, 64).double()
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.isnan(y[2]).all()
        fine = ~torch.isnan(want)
        assert torch.equal(torch.isinf(y[fine]), torch.isinf(want[fine]))
        assert torch.equal(y[1][torch.isinf(want[1])], want[1][torch.isinf(want[1])])
        assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()


@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 0])
def test_matmul_with_an_infinite_scale(tokens, group):
    import differentiable_bcjr_b200 as B
    # codes above the zero point and positive inputs: an infinite scale gives infinity, also in a short last group
    packed, scales, zeros = _layer(40, 300, group, True, F32, 2)
    packed |= 0x88
    zeros.fill_(1)
    scales[0, 3] = scales[-1, 7] = float("inf")
    x = torch.rand(tokens, 300, device="cuda").bfloat16() + 0.5
    y = B.int4_matmul(x, packed, scales, zeros, group)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[3] = bad[7] = True
    assert (y[:, bad] == float("inf")).all() and torch.isfinite(y[:, ~bad]).all()


@pytest.mark.parametrize("tokens", [1, 3, 7, 20, 33])
@pytest.mark.parametrize("rows,cols,group", [(4, 40, 0), (132, 1100, 128), (20, 2300, 256), (44, 700, 32), (300, 129, 64)])
@pytest.mark.parametrize("scale", [F32, F16, BF16])
def test_matmul_of_unaligned_scales(tokens, rows, cols, group, scale):
    import differentiable_bcjr_b200 as B
    packed, scales, zeros = _layer(rows, cols, group, True, scale, rows)
    x = torch.randn(tokens, cols, device="cuda").bfloat16()
    y = B.int4_matmul(x, packed, scales, zeros, group)
    want, tol = _tolerance(x, R.int4_weights(packed, scales, zeros, rows, cols, group), group, BF16)
    assert ((y.double() - want).abs() <= tol).all()
    # the same values one element behind an aligned address
    apart = [torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape) for t in (scales, zeros)]
    assert all(t.data_ptr() % (4 * t.element_size()) for t in apart)
    assert torch.equal(B.int4_matmul(x, packed, apart[0], apart[1], group), y)
    assert torch.equal(B.int4_matmul(x, packed, scales, apart[1], group), y)


def test_float32_inputs_are_not_rounded():
    import differentiable_bcjr_b200 as B
    # one column in use: the products of a 24-bit mantissa and a 4-bit code, a single rounding away
    packed, scales, _ = _layer(64, 128, 128, False, F32, 3)
    scales.fill_(1.0)
    w = R.int4_weights(packed, scales, None, 64, 128, 128)
    x = torch.zeros(2, 128, device="cuda")
    for v in (1.0 + 2.0 ** -23, 3.4028234e38 / 8, -1.9999999, 1.2345678e-30):
        x[0, 77] = v
        y = B.int4_matmul(x, packed, scales, None, 128).double()
        want = x.double() @ w.t()
        assert ((y - want).abs() <= want.abs() * 2 ** -22).all()


def test_quantise_then_multiply_in_a_graph_and_on_another_stream():
    import differentiable_bcjr_b200 as B
    w = _w(100, 640, BF16, 5)
    x = torch.randn(3, 640, device="cuda").bfloat16()
    eager = B.int4_matmul(x, *B.int4_quantize(w, 64, True), 64)
    static = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = B.int4_matmul(static, *B.int4_quantize(w, 64, True), 64)
    static.copy_(x)
    graph.replay()
    assert torch.equal(y, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = B.int4_matmul(x, *B.int4_quantize(w, 64, True), 64)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, eager)


def test_refusals():
    import differentiable_bcjr_b200 as B
    packed, scales, zeros = _layer(40, 256, 64, True, F32, 1)
    x = torch.randn(2, 256, device="cuda")
    bad = [lambda: B.int4_matmul(x.cpu(), packed, scales, zeros, 64),
           lambda: B.int4_matmul(x.double(), packed, scales, zeros, 64),
           lambda: B.int4_matmul(x.t(), packed, scales, zeros, 64),
           lambda: B.int4_matmul(x, packed[:2], scales, zeros, 64),
           lambda: B.int4_matmul(x, packed.view(torch.int8), scales, zeros, 64),
           lambda: B.int4_matmul(x, packed, scales[:3].contiguous(), zeros, 64),
           lambda: B.int4_matmul(x, packed, scales, zeros[:3].contiguous(), 64),
           lambda: B.int4_matmul(x, packed, scales, zeros, 96),
           lambda: B.int4_matmul(x, packed, scales, zeros, -128),
           lambda: B.int4_matmul(x, packed, scales.double(), zeros, 64),
           lambda: B.int4_matmul(x, packed, scales, zeros, 64, out=torch.empty(2, 41, device="cuda")),
           lambda: B.int4_quantize(x.cpu()),
           lambda: B.int4_quantize(x, 48),
           lambda: B.int4_quantize(x.double()),
           lambda: B.int4_quantize(x[0].contiguous()),
           lambda: B.int4_quantize(x, scale_dtype=torch.float64)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
