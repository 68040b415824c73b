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
