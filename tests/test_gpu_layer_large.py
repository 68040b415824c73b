"""The calls of bcjr_layer.h where offsets pass 32 bits (needs a B200; 15 to 45 GB a test)."""
import gc

import pytest
import torch

import bcjr_inputs as I
import layer_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_int4_weights_beyond_4_gib():
    import differentiable_bcjr_b200 as B
    rows, cols = 66000, 140032  # 4.6 GB packed; 9.2 G codes
    gen = torch.Generator(device="cuda").manual_seed(1)
    packed = torch.randint(0, 256, (rows // 16, cols // 128, 1024), generator=gen, device="cuda", dtype=torch.uint8)
    assert packed.numel() > 2 ** 32
    scales = 0.01 + torch.rand(1, rows, generator=gen, device="cuda")
    for tokens in (1, 12):
        x = torch.randn(tokens, cols, generator=gen, device="cuda").bfloat16()
        y = B.int4_matmul(x, packed, scales, None, 0)
        for lo in (0, rows - 48):
            w = R.int4_weights(packed[lo // 16:lo // 16 + 3], scales[:, lo:lo + 48], None, 48, cols, 0)
            want = x.double() @ w.t()
            # a bf16 rounding, and 2^-23 of the magnitudes for each of about 1100 / 16 + 32 sums on a value's way
            tol = want.abs() * 2 ** -9 + (x.double().abs() @ w.abs().t()) * 180 * 2 ** -23
            assert ((y[:, lo:lo + 48].double() - want).abs() <= tol).all()


def test_quantise_beyond_4_gib():
    import differentiable_bcjr_b200 as B
    rows, cols = 40000, 65600  # 2.6 G weights, 5.2 GB
    w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    for group in (128, 0):
        packed, scales, _ = B.int4_quantize(w, group)
        for lo in (0, rows - 32):
            part = B.int4_quantize(w[lo:lo + 32].clone(), group)
            assert torch.equal(packed[lo // 16:lo // 16 + 2], part[0]) and torch.equal(scales[:, lo:lo + 32], part[1])


def test_trellis_beyond_4_gib():
    import differentiable_bcjr_b200 as B
    L, k, n, cols = 8, 4, 256, 8192
    rows = 140000
    seqs = rows * cols // n
    gen = torch.Generator(device="cuda").manual_seed(3)
    last = R.random_path(64, n, L, k, 5).cuda()  # the last two rows
    states = torch.zeros(seqs, n, dtype=torch.int32, device="cuda")  # 4.6 GB; state 0 follows itself
    states[-64:] = last
    packed = B.trellis_pack(states, L, k, check=True)
    assert torch.equal(packed[-64:].cpu(), R.pack_states(last.cpu(), L, k)) and (packed[:-64] == 0).all()
    del states
    many = packed.repeat(8, 1)  # 1.1 M rows: 4.7 GB of words
    assert many.numel() * 4 > 2 ** 32
    c = I.codebook(1 << L).cuda()
    x = torch.randn(1, cols, generator=gen, device="cuda")
    y = B.trellis_matmul(x, many, c, L, k, n)
    w = c.double()[last.long()].view(2, cols)
    want = x.double() @ w.t()
    size = x.double().abs() @ w.abs().t()
    for end in (rows, 8 * rows):
        assert ((y[:, end - 2:end].double() - want).abs() <= size * 64 * 2 ** -24).all()
    rest = x.double().sum() * c[0].double()
    assert ((y[:, -10:-2].double() - rest).abs() <= x.double().abs().sum() * c[0].abs() * 64 * 2 ** -24).all()


def test_adamw_beyond_4_g_elements():
    import differentiable_bcjr_b200 as B
    n = 2 ** 32 + 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = torch.Generator(device="cuda").manual_seed(4)
    g[-5000:] = torch.randn(5000, generator=tail, device="cuda").bfloat16()
    small = torch.ones(77, dtype=torch.bfloat16, device="cuda")
    first, second, scales = B.adamw_state([p, small], 8)
    B.adamw_step([p, small], [g, small], first, second, 1, lr=0.5, scales=scales)
    want, m, v = R.adamw(torch.zeros(5000, device="cuda"), g[-5000:], 0 * g[-5000:], 0 * g[-5000:], 1, 0.5, 0.9, 0.999, 1e-8, 0.0)
    assert ((p[-5000:].double() - want).abs() <= want.abs() * 2 ** -8).all() and (p[:-5000] == 0).all()
    assert (small.double() - 0.5).abs().max() <= 2 ** -9
    at = n - 5000
    block = torch.arange(at, n, device="cuda") // 256
    got = first[at:n].float().double() * scales[0].double()[block]
    # a code is at most an eighth of its value off, or a step of the smallest codes
    assert ((got - m).abs() <= m.abs() / 8 + scales[0].double()[block] * 2 ** -9).all()
    root = second[at:n].float().double() * scales[1].double()[block]
    assert ((root - v.sqrt()).abs() <= v.sqrt() / 8 + scales[1].double()[block] * 2 ** -9).all()
