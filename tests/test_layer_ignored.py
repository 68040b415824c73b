"""Arguments of the calls of bcjr_layer.h that the header says are ignored (CPU only: nothing is launched without rows)."""
import ctypes

P, I = ctypes.c_void_p, ctypes.c_int


def test_a_group_size_without_scales():
    from differentiable_bcjr_b200 import build
    f = ctypes.CDLL(build.build()).bcjr_trellis_matmul
    f.restype, f.argtypes = I, [P, I, I, I, I, P, P, I, I, I, I, P, I, P, P]

    def call(scales, group):
        return f(4096, 0, 2, 0, 128, 8192, 12288, 0, 8, 2, 64, scales, group, 16384, None)

    for group in (-1, -128, 7, 24, 192):
        assert call(None, group) == 0 and call(4096, group) != 0
    for group in (0, 16, 32, 64, 128):
        assert call(None, group) == 0 and call(4096, group) == 0
