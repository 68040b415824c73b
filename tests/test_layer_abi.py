"""The calls of bcjr_layer.h reject bad arguments on the host before touching
the GPU, and the Python binding rejects CPU tensors (CPU only)."""
import ctypes

import pytest
import torch

P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from differentiable_bcjr_b200 import build
    return ctypes.CDLL(build.build())


class Tensor(ctypes.Structure):
    _fields_ = [("param", P), ("grad", P), ("numel", ctypes.c_int64)]


class Options(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64), ("step_ptr", P), ("grad_scale", P), ("seed", ctypes.c_uint32)]


def test_adamw_arguments(lib):
    f = lib.bcjr_adamw_step
    f.restype, f.argtypes = I, [P, I, I, I, I, P, P, P, P, P]

    # fake, never-dereferenced device addresses: every call here must be rejected before any CUDA call
    def call(tensors=((4096, 8192, 100),), p=0, g=0, bits=32, first=65536, second=131072, scales=None, **o):
        ts = (Tensor * max(1, len(tensors)))(*[Tensor(*t) for t in tensors])
        opt = Options(1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None, 0)
        for name, v in o.items():
            setattr(opt, name, v)
        return f(ctypes.addressof(ts), len(tensors), p, g, bits, first, second, scales, ctypes.addressof(opt), None)

    assert f(None, 1, 0, 0, 32, 65536, 131072, None, None, None) == INVALID
    assert call(p=3) == INVALID and call(g=-1) == INVALID
    assert call(bits=16) == UNSUPPORTED
    assert call(p=1, g=2) == UNSUPPORTED and call(p=2, g=1) == UNSUPPORTED
    assert call(first=None) == INVALID and call(second=None) == INVALID and call(first=65544) == INVALID
    assert call(bits=8) == INVALID and call(scales=4096) == INVALID  # scales belong to 8 bits alone
    assert call(bits=8, scales=4098) == INVALID
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(beta2=float("nan")), dict(eps=-1e-8),
                dict(eps=float("inf")), dict(weight_decay=-1.0), dict(step=0), dict(grad_scale=4098), dict(step_ptr=4100)):
        assert call(**bad) == INVALID, bad
    assert call(tensors=((None, 8192, 4),)) == INVALID
    assert call(tensors=((4098, 8192, 4),)) == INVALID  # a float32 off its alignment
    assert call(tensors=((4096, 8194, 4),)) == INVALID
    assert call(tensors=((4096, 8192, -1),)) == INVALID
    assert call(tensors=((4096, 8192, 100), (4096, 16384, 100))) == INVALID  # the same tensor twice
    assert call(tensors=((4096, 1 << 20, 100), (4492, 1 << 20, 100))) == INVALID  # 396 bytes apart: they share one element
    many = [(1 << 30 | i << 12, 1 << 20, 100) for i in range(600)]
    assert call(tensors=tuple(many + [(many[77][0] + 396, 1 << 20, 100)])) == INVALID
    assert call(tensors=()) == 0 and call(tensors=((None, None, 0),)) == 0


def test_int4_arguments(lib):
    f = lib.bcjr_int4_matmul
    f.restype, f.argtypes = I, [P, I, I, I, I, P, P, I, P, I, P, P]

    def call(x=4096, xd=0, tokens=2, rows=40, cols=256, packed=8192, scales=12288, sd=0, zeros=None, group=64, y=16384):
        return f(x, xd, tokens, rows, cols, packed, scales, sd, zeros, group, y, None)

    assert call(xd=3) == INVALID and call(sd=-1) == INVALID
    assert call(tokens=-1) == INVALID and call(rows=-1) == INVALID and call(cols=0) == INVALID and call(group=-64) == INVALID
    assert call(group=96) == UNSUPPORTED and call(group=16) == UNSUPPORTED and call(group=100) == UNSUPPORTED
    assert call(x=None) == INVALID and call(packed=None) == INVALID and call(scales=None) == INVALID and call(y=None) == INVALID
    assert call(packed=8200) == INVALID and call(x=4098) == INVALID and call(xd=2, x=4097) == INVALID and call(y=16386) == INVALID
    assert call(tokens=1 << 20) == UNSUPPORTED and call(cols=1 << 28) == UNSUPPORTED
    assert call(tokens=0) == 0 and call(rows=0) == 0
    q = lib.bcjr_int4_quantize
    q.restype, q.argtypes = I, [P, I, I, I, I, P, P, I, P, P]

    def quantize(w=4096, wd=0, rows=40, cols=256, group=64, packed=8192, scales=12288, sd=0, zeros=None):
        return q(w, wd, rows, cols, group, packed, scales, sd, zeros, None)

    assert quantize(wd=7) == INVALID and quantize(sd=3) == INVALID and quantize(rows=-1) == INVALID and quantize(cols=0) == INVALID
    assert quantize(group=48) == UNSUPPORTED and quantize(rows=(1 << 30) + 1) == UNSUPPORTED
    assert quantize(w=None) == INVALID and quantize(packed=None) == INVALID and quantize(scales=None) == INVALID
    assert quantize(w=4097, wd=1) == INVALID and quantize(packed=8196) == INVALID
    assert quantize(rows=0) == 0


def test_trellis_arguments(lib):
    f = lib.bcjr_trellis_matmul
    f.restype, f.argtypes = I, [P, I, I, I, I, P, P, I, I, I, I, P, I, P, P]

    def call(x=4096, xd=0, tokens=2, rows=3, cols=128, packed=8192, c=12288, cd=0, L=8, k=2, n=64, scales=None, group=0, y=16384):
        return f(x, xd, tokens, rows, cols, packed, c, cd, L, k, n, scales, group, y, None)

    assert call(xd=3) == INVALID and call(cd=3) == INVALID and call(tokens=-1) == INVALID and call(rows=-1) == INVALID
    assert call(k=0) == INVALID and call(L=2, k=3) == INVALID and call(n=0) == INVALID and call(cols=100) == INVALID
    assert call(k=5) == UNSUPPORTED and call(L=17) == UNSUPPORTED and call(tokens=1 << 20) == UNSUPPORTED
    assert call(scales=4096, group=24) == UNSUPPORTED and call(scales=4096, group=8) == UNSUPPORTED
    assert call(scales=4096, group=192) == UNSUPPORTED  # does not divide the columns
    assert call(scales=4096, group=-1) == INVALID
    assert call(x=None) == INVALID and call(packed=None) == INVALID and call(c=None) == INVALID and call(y=None) == INVALID
    assert call(packed=8193) == INVALID and call(c=12289, cd=1) == INVALID and call(scales=4097) == INVALID
    assert call(tokens=0) == 0 and call(rows=0) == 0
    p = lib.bcjr_trellis_pack
    p.restype, p.argtypes = I, [P, I, I, I, I, P, P, P]
    assert p(4096, 8, 0, 4, 2, 8192, None, None) == INVALID and p(4096, 3, 4, 4, 2, 8192, None, None) == INVALID
    assert p(4096, 8, 2, 0, 2, 8192, None, None) == INVALID and p(4096, 8, 2, 4, -1, 8192, None, None) == INVALID
    assert p(4096, 17, 2, 4, 2, 8192, None, None) == UNSUPPORTED and p(4096, 8, 5, 4, 2, 8192, None, None) == UNSUPPORTED
    assert p(None, 8, 2, 4, 2, 8192, None, None) == INVALID and p(4096, 8, 2, 4, 2, None, None, None) == INVALID
    assert p(4096, 8, 2, 4, 2, 8192, 4098, None) == INVALID and p(None, 8, 2, 4, 0, None, None, None) == 0


def test_cpu_tensors_are_refused():
    import differentiable_bcjr_b200 as B
    x = torch.ones(2, 256)
    with pytest.raises(ValueError):
        B.int4_quantize(x)
    with pytest.raises(ValueError):
        B.int4_matmul(x, torch.zeros(1, 2, 1024, dtype=torch.uint8), torch.ones(2, 16))
    with pytest.raises(ValueError):
        B.trellis_pack(torch.zeros(2, 4, dtype=torch.int32), 8, 2)
    with pytest.raises(ValueError):
        B.trellis_matmul(x, torch.zeros(2, 17, dtype=torch.int32), torch.ones(256), 8, 2, 256)
    with pytest.raises(ValueError):
        B.adamw_step([x], [x], torch.zeros(512), torch.zeros(512), 1)


def test_words_of_a_sequence():
    import differentiable_bcjr_b200 as B
    assert B.trellis_words(16, 2, 256) == 17 and B.trellis_words(8, 2, 1) == 1 and B.trellis_words(4, 4, 8) == 1
    assert B.trellis_words(16, 4, 5) == 1 and B.trellis_words(16, 4, 6) == 2
    for bad in ((17, 2), (8, 5), (3, 4), (8, 0)):
        with pytest.raises(ValueError):
            B.trellis_words(*bad, 10)
