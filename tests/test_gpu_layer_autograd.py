"""What autograd sees of the calls around a quantised layer (needs a B200)."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu


def test_a_parameter_left_alone_keeps_its_graph():
    import differentiable_bcjr_b200 as B
    for bits in (8, 32):
        a, b = (torch.ones(300, device="cuda", requires_grad=True) for _ in range(2))
        y, z = (a * a).sum(), (b * b).sum()
        first, second, scales = B.adamw_state([a, b], bits)
        version = a._version, b._version
        B.adamw_step([a, b], [None, torch.ones(300, device="cuda")], first, second, 1, scales=scales)
        assert a._version == version[0] and b._version > version[1]
        y.backward()
        assert (a.grad == 2).all()
        with pytest.raises(RuntimeError):
            z.backward()
        B.adamw_step([a, b], [None, None], first, second, 2, scales=scales)
        assert a._version == version[0]


def _products():
    """(function of an input, which of its tensors may want gradients) of both products."""
    import differentiable_bcjr_b200 as B
    w = torch.randn(40, 128, generator=torch.Generator().manual_seed(1)).cuda()
    packed, scales, _ = B.int4_quantize(w, 64)
    stream = B.trellis_pack(R.random_path(80, 64, 8, 2, 1).cuda(), 8, 2)
    codebook, wide = torch.randn(256, device="cuda"), torch.ones(1, 40, device="cuda")
    return [(lambda x, scales=scales, **kw: B.int4_matmul(x, packed, scales, None, 64, **kw), {"scales": scales}),
            (lambda x, codebook=codebook, scales=wide, **kw: B.trellis_matmul(x, stream, codebook, 8, 2, 64, scales, 0, **kw),
             {"codebook": codebook, "scales": wide})]


def test_products_do_not_drop_a_gradient_silently():
    for f, weights in _products():
        x = torch.randn(3, 128, device="cuda")
        want = f(x)
        live = x.clone().requires_grad_()
        for call in [lambda: f(live), lambda: f(live * 2), lambda: f(x, out=torch.empty_like(want, requires_grad=True))] + \
                    [lambda name=name, t=t: f(x, **{name: t.clone().requires_grad_()}) for name, t in weights.items()]:
            with pytest.raises(RuntimeError, match="no gradient"):
                call()
            with torch.no_grad():
                call()
        with torch.no_grad():
            assert torch.equal(f(live), want)
        assert torch.equal(f(live.detach()), want)
        with torch.inference_mode():
            assert torch.equal(f(live), want)


def test_an_output_that_autograd_has_saved_is_missed():
    for f, _ in _products():
        x = torch.randn(3, 128, device="cuda")
        out = torch.ones(3, 40, device="cuda")
        a = torch.ones(3, 40, device="cuda", requires_grad=True)
        y = (a * out).sum()
        f(x, out=out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
