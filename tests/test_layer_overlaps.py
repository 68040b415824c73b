"""Arguments of the calls of bcjr_layer.h that share memory and may not (CPU only: refused before any CUDA call)."""
import ctypes

import pytest
import torch

P, I = ctypes.c_void_p, ctypes.c_int
INVALID = 1


class Tensor(ctypes.Structure):
    _fields_ = [("param", P), ("grad", P), ("numel", ctypes.c_int64)]


class Options(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64), ("step_ptr", P), ("grad_scale", P), ("seed", ctypes.c_uint32)]


@pytest.mark.parametrize("bits", [8, 32])
def test_states_of_an_adamw_step(bits):
    from differentiable_bcjr_b200 import build
    f = ctypes.CDLL(build.build()).bcjr_adamw_step
    f.restype, f.argtypes = I, [P, I, I, I, I, P, P, P, P, P]
    size = 1024 if bits == 8 else 4096  # bytes of a state: four blocks of 256 elements

    def call(tensors=((1 << 20, 2 << 20, 1000),), first=1 << 16, second=1 << 17, scales=1 << 18):
        ts = (Tensor * len(tensors))(*[Tensor(*t) for t in tensors])
        o = Options(1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None, 0)
        return f(ctypes.addressof(ts), len(tensors), 0, 0, bits, first, second, scales if bits == 8 else None, ctypes.addressof(o), None)

    assert call(second=1 << 16) == INVALID  # one array for both
    assert call(second=(1 << 16) + size - 16) == INVALID and call(second=(1 << 16) - size + 16) == INVALID
    p = 1 << 20
    assert call(first=p) == INVALID and call(second=p) == INVALID
    assert call(first=p + 3984) == INVALID and call(first=p - size + 16) == INVALID  # the parameter's last 16 bytes, its first
    g = 2 << 20
    assert call(first=g) == INVALID and call(second=g + 3984) == INVALID  # a gradient
    if bits == 8:
        assert call(scales=1 << 16) == INVALID and call(scales=(1 << 17) + 1020) == INVALID and call(scales=p + 3996) == INVALID
        assert call(scales=(1 << 17) - 28) == INVALID  # 2 x 4 scales of 4 bytes
    two = ((1 << 20, 2 << 20, 600), (3 << 20, 2 << 20, 10))  # (a gradient of two parameters is read only)
    assert call(tensors=two, first=3 << 20) == INVALID and call(tensors=two, second=(3 << 20) + 32) == INVALID


class Fake(torch.Tensor):
    """A CPU tensor that says it is on the first GPU."""

    def get_device(self):
        return 0


def test_outputs_of_the_products(monkeypatch):
    import differentiable_bcjr_b200 as B
    from differentiable_bcjr_b200 import layer
    calls = []
    monkeypatch.setattr(layer, "_call", lambda *a: calls.append(a[0]))

    def fake(t):
        return t.as_subclass(Fake)

    # all in one buffer, one after the other: an output may touch but not cover any of them
    buf = torch.zeros(1 << 16)
    x, out = fake(buf[:256].view(2, 128)), fake(buf[4096:4096 + 32].view(2, 16))
    scales, packed = fake(buf[1024:1040].view(1, 16)), fake(buf[2048:2304].view(torch.uint8).view(1, 1, 1024))
    zeros = fake(buf[1536:1540].view(torch.uint8).view(1, 16))
    stream, codebook = fake(buf[2560:2560 + 16 * 9].view(torch.int32).view(16, 9)), fake(buf[8192:8192 + 256])

    def int4(out):
        return B.int4_matmul(x, packed, scales, zeros, 0, out=out)

    def trellis(out):
        return B.trellis_matmul(x, stream, codebook, 8, 2, 128, scales, 0, out=out)

    for f, others in ((int4, (x, packed, scales, zeros)), (trellis, (x, stream, codebook, scales))):
        assert f(out) is out
        for t in others:
            at = (t.data_ptr() - buf.data_ptr()) // 4
            end = at + t.numel() * t.element_size() // 4
            for start in (at, end - 1, max(0, at - 31)):
                with pytest.raises(ValueError, match="must not overlap"):
                    f(fake(buf[start:start + 32].view(2, 16)))
            f(fake(buf[end:end + 32].view(2, 16)))
    assert calls and set(calls) == {"bcjr_int4_matmul", "bcjr_trellis_matmul"}
