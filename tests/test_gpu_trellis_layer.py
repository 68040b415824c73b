"""Packed trellis states and products with them against their definitions in 64 bits (needs a B200)."""
import pytest
import torch

import bcjr_inputs as I
import layer_ref as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("L,k", [(4, 4), (1, 1), (5, 1), (8, 2), (11, 3), (16, 1), (16, 2), (16, 3), (16, 4), (7, 4)])
@pytest.mark.parametrize("n_seq,n", [(1, 1), (3, 2), (5, 16), (2, 33), (40, 77), (7, 256)])
def test_pack_matches_the_stream(L, k, n_seq, n):
    import differentiable_bcjr_b200 as B
    states = R.random_path(n_seq, n, L, k, L * 100 + n)
    got = B.trellis_pack(states.cuda(), L, k, check=True)
    assert torch.equal(got.cpu(), R.pack_states(states, L, k))


def test_pack_tells_states_that_are_no_path():
    import differentiable_bcjr_b200 as B
    good = R.random_path(9, 50, 10, 2, 1).cuda()
    for seq, t in ((0, 0), (3, 1), (8, 49), (4, 20)):
        s = good.clone()
        s[seq, t] ^= 1 << 9
        if t == 0 and ((good[seq, 0] ^ (1 << 9)) >> 0) >= 0:
            s[seq, 0] = 1 << 10  # out of range
        with pytest.raises(ValueError):
            B.trellis_pack(s, 10, 2, check=True)
    B.trellis_pack(good, 10, 2, check=True)
    assert B.trellis_pack(good[:0].contiguous(), 10, 2, check=True).shape == (0, 4)


def _want(x, states, c, scales, group, rows):
    w = c.double()[states.long()].view(rows, -1)
    if scales is not None:
        w = w * scales.double().t().repeat_interleave(group or w.shape[1], 1)
    y = x.double() @ w.t()
    return y, x.double().abs() @ w.abs().t()


def _check(y, want, size, tiles):
    # a lane's 16 products, the scale, 5 steps of the butterfly, the warp's tiles, both halves of a codebook, 16
    # warps: each rounds once
    depth = 16 + 1 + 5 + tiles + 2 + 16
    tol = want.abs() * torch.finfo(y.dtype).eps / 2 + size * depth * 2 ** -24 + (2.0 ** -25 if y.dtype == F16 else 0)
    assert ((y.double() - want).abs() <= tol).all(), ((y.double() - want).abs() / tol).max()


@pytest.mark.parametrize("L,k,n,per_row,rows,group", [
    (4, 4, 64, 2, 5, 64), (8, 2, 64, 3, 33, 16), (6, 1, 1, 7, 9, 0), (10, 2, 100, 5, 20, 100), (12, 3, 77, 4, 50, 154), (16, 2, 256, 32, 40, 0),
    (16, 4, 256, 8, 300, 256), (16, 1, 40, 1, 3, 0), (16, 3, 512, 2, 17, 128), (15, 3, 33, 20, 11, 33), (13, 2, 2048, 9, 4, 2048),
    (9, 4, 17, 300, 6, 0), (14, 1, 256, 4, 700, 512)])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 8, 11])
@pytest.mark.parametrize("kind,ckind", [(BF16, F32), (F32, BF16), (F16, F16)])
def test_matmul_matches_the_definition(L, k, n, per_row, rows, group, tokens, kind, ckind):
    import differentiable_bcjr_b200 as B
    states = R.random_path(rows * per_row, n, L, k, L + n).cuda()
    packed = B.trellis_pack(states, L, k)
    c = I.codebook(1 << L).to(ckind).cuda()
    cols = per_row * n
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(tokens, cols, generator=gen).to(kind).cuda()
    for scales in (None, (0.5 + torch.rand(cols // group if group else 1, rows, generator=gen)).cuda()):
        y = B.trellis_matmul(x, packed, c, L, k, n, scales, group)
        assert y.dtype == kind and y.shape == (tokens, rows)
        _check(y, *_want(x, states, c, scales, group, rows), -(-per_row * -(-n // 16) // 32))


# Inputs and codewords of one 16-bit type are summed by the tensor core: exact products, at most 16 added at a time
# to a float32 sum of 4 instructions, each cutting what lies 2^-23 below its largest term (four times at worst), then
# the scale, a warp's other columns and 16 warps.  That is no more than the depth of _check counts.
@pytest.mark.parametrize("L,k,n,per_row,rows,group", [
    (4, 4, 64, 2, 5, 64), (8, 2, 64, 3, 33, 16), (6, 1, 1, 7, 9, 0), (10, 2, 100, 5, 20, 100), (12, 3, 77, 4, 50, 154), (16, 2, 256, 32, 40, 0),
    (16, 4, 256, 8, 3000, 256), (16, 1, 40, 1, 3, 0), (16, 3, 512, 2, 17, 128), (15, 3, 33, 20, 1300, 33), (13, 2, 2048, 9, 4, 2048),
    (9, 4, 17, 300, 6, 0), (14, 1, 256, 4, 700, 512), (1, 1, 48, 2, 8, 48), (11, 2, 16, 1, 20000, 16),
    (10, 2, 100, 40, 20, 100), (12, 3, 64, 64, 9, 64), (16, 4, 1024, 4, 600, 256)])
@pytest.mark.parametrize("tokens", [1, 3, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("kind", [BF16, F16])
def test_matmul_of_one_16_bit_type(L, k, n, per_row, rows, group, tokens, kind):
    import differentiable_bcjr_b200 as B
    states = R.random_path(rows * per_row, n, L, k, L + n).cuda()
    packed = B.trellis_pack(states, L, k)
    c = I.codebook(1 << L).to(kind).cuda()
    cols = per_row * n
    gen = torch.Generator().manual_seed(3)
    flat = torch.randn(1 + tokens * cols, generator=gen).to(kind).cuda()
    x = flat[1:].view(tokens, cols)  # not 16-byte aligned
    for scales in (None, (0.5 + torch.rand(cols // group if group else 1, rows, generator=gen)).cuda()):
        y = B.trellis_matmul(x, packed, c, L, k, n, scales, group)
        _check(y, *_want(x, states, c, scales, group, rows), -(-per_row * -(-n // 16) // 32))
        assert torch.equal(B.trellis_matmul(x.clone(), packed, c, L, k, n, scales, group), y)
        moved = torch.cat([c[:1], c])[1:]
        assert torch.equal(B.trellis_matmul(x, packed, moved, L, k, n, scales, group), y)


@pytest.mark.parametrize("L", [8, 16])
@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("tokens", [3, 11])
def test_non_finite_values_of_one_16_bit_type(L, kind, tokens):
    import differentiable_bcjr_b200 as B
    k, n, rows = 2, 50, 30  # sequences end inside a chunk
    states = R.random_path(rows * 2, n, L, k, 5).cuda()
    states[3] = 0  # a path of the codeword that is infinite below
    packed = B.trellis_pack(states, L, k, check=True)
    c = I.codebook(1 << L).to(kind).cuda()
    x = torch.randn(tokens, 2 * n, device="cuda").to(kind)
    x[1, 60], x[2, 7] = float("inf"), float("nan")
    for _ in range(2):
        want, _ = _want(x, states, c, None, 0, rows)
        y = B.trellis_matmul(x, packed, c, L, k, n).double()
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(y), torch.isinf(want))
        assert torch.equal(y[torch.isinf(y)], want[torch.isinf(want)]) and torch.isfinite(want[0]).any()
        # the padding behind a sequence's end reads as state 0, whose codeword must not be met there
        c[0] = float("inf")


@pytest.mark.parametrize("L", [8, 16])
@pytest.mark.parametrize("kind,ckind", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("tokens", [1, 4, 9])
def test_infinite_codewords_of_whole_chunks(L, kind, ckind, tokens):
    import differentiable_bcjr_b200 as B
    k, n, rows = 2, 256, 40  # no padding anywhere
    states = R.random_path(rows * 2, n, L, k, 5).cuda()
    states[3] = 0
    packed = B.trellis_pack(states, L, k, check=True)
    c = I.codebook(1 << L).to(ckind).cuda()
    c[0] = float("inf")
    c[(1 << L) - 1] = -float("inf")
    x = torch.rand(tokens, 2 * n, device="cuda").to(kind) + 0.5
    for _ in range(2):
        want, _ = _want(x, states, c, None, 0, rows)
        y = B.trellis_matmul(x, packed, c, L, k, n).double()
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(y), torch.isinf(want))
        assert torch.equal(y[torch.isinf(y)], want[torch.isinf(want)]) and not torch.isfinite(y[0, 1])
        x[0, 300] = float("inf")


@pytest.mark.parametrize("L,ckind", [(8, F32), (16, F32), (16, BF16), (16, F16)])
def test_matmul_of_non_finite_inputs_and_codewords(L, ckind):
    import differentiable_bcjr_b200 as B
    k, n, rows = 2, 50, 30  # sequences end inside a chunk
    states = R.random_path(rows * 2, n, L, k, 5).cuda()
    states[3] = 0  # a path of the codeword that is infinite below
    packed = B.trellis_pack(states, L, k, check=True)
    c = I.codebook(1 << L).to(ckind).cuda()
    x = torch.randn(3, 2 * n, device="cuda")
    x[1, 60] = float("inf")
    x[2, 7] = float("nan")
    want, _ = _want(x, states, c, None, 0, rows)
    y = B.trellis_matmul(x, packed, c, L, k, n).double()
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(y), torch.isinf(want))
    assert torch.equal(y[1].sign(), want[1].sign())
    c[0] = float("inf")
    x = torch.randn(1, 2 * n, device="cuda")
    want, size = _want(x, states, c, None, 0, rows)
    y = B.trellis_matmul(x, packed, c, L, k, n).double()
    # the padding behind a sequence's end reads as state 0, whose codeword must not be met there
    assert torch.equal(torch.isfinite(y), torch.isfinite(want)) and torch.isfinite(want).any() and not torch.isfinite(y[0, 1])


@pytest.mark.parametrize("L", [8, 16])
def test_matmul_with_an_infinite_scale(L):
    import differentiable_bcjr_b200 as B
    k, n, rows = 2, 50, 30
    packed = B.trellis_pack(R.random_path(rows * 2, n, L, k, 5).cuda(), L, k)
    c = I.codebook(1 << L).abs().cuda() + 0.1
    x = torch.rand(2, 2 * n, device="cuda") + 0.1
    scales = torch.ones(2, rows, device="cuda")
    scales[0, 3] = scales[1, 4] = float("inf")
    y = B.trellis_matmul(x, packed, c, L, k, n, scales, n)
    assert (y[:, 3:5] == float("inf")).all() and torch.isfinite(y[:, :3]).all() and torch.isfinite(y[:, 5:]).all()


def test_decode_pack_and_multiply_as_a_program_does():
    import differentiable_bcjr_b200 as B
    L, k, n, rows, cols = 10, 2, 64, 24, 256
    w = I.normal((rows, cols), seed=4).cuda()
    c = I.codebook(1 << L).cuda()
    states, hard = B.viterbi_decode(w.view(-1, n), c, L, k)
    packed = B.trellis_pack(states, L, k, check=True)
    x = I.normal((2, 3, cols), seed=5).cuda()
    y = B.trellis_matmul(x, packed, c, L, k, n)
    assert y.shape == (2, 3, rows)
    want = x.view(6, cols).double() @ hard.view(rows, cols).double().t()
    _check(y.view(6, rows), want, x.view(6, cols).double().abs() @ hard.view(rows, cols).double().abs().t(), 1)


def test_matmul_in_a_graph_on_a_stream_and_into_a_given_output():
    import differentiable_bcjr_b200 as B
    L, k, n, rows = 16, 2, 256, 60
    packed = B.trellis_pack(R.random_path(rows * 4, n, L, k, 5).cuda(), L, k)
    c = I.codebook(1 << L).cuda()
    x = torch.randn(2, 4 * n, device="cuda")
    eager = B.trellis_matmul(x, packed, c, L, k, n)
    out = torch.full_like(eager, float("nan"))
    assert B.trellis_matmul(x, packed, c, L, k, n, out=out) is out and torch.equal(out, eager)
    static = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = B.trellis_matmul(static, packed, c, L, k, n)
    static.copy_(x)
    graph.replay()
    assert torch.equal(y, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = B.trellis_matmul(x, packed, c, L, k, n)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, eager)
    assert B.trellis_matmul(x[:0].contiguous(), packed, c, L, k, n).shape == (0, rows)


def test_refusals():
    import differentiable_bcjr_b200 as B
    L, k, n = 8, 2, 64
    packed = B.trellis_pack(R.random_path(6, n, L, k, 5).cuda(), L, k)
    c = I.codebook(1 << L).cuda()
    x = torch.randn(2, 2 * n, device="cuda")
    s = torch.ones(2, 3, device="cuda")
    bad = [lambda: B.trellis_matmul(x.cpu(), packed, c, L, k, n),
           lambda: B.trellis_matmul(x.double(), packed, c, L, k, n),
           lambda: B.trellis_matmul(x[:, :100].contiguous(), packed, c, L, k, n),
           lambda: B.trellis_matmul(x, packed[:5], c, L, k, n),
           lambda: B.trellis_matmul(x, packed[:, :3].contiguous(), c, L, k, n),
           lambda: B.trellis_matmul(x, packed.float(), c, L, k, n),
           lambda: B.trellis_matmul(x, packed, c[:100], L, k, n),
           lambda: B.trellis_matmul(x, packed, c.double(), L, k, n),
           lambda: B.trellis_matmul(x, packed, c, L, 5, n),
           lambda: B.trellis_matmul(x, packed, c, 17, k, n),
           lambda: B.trellis_matmul(x, packed, c, L, k, n, s, 0),
           lambda: B.trellis_matmul(x, packed, c, L, k, n, s, 24),
           lambda: B.trellis_matmul(x, packed, c, L, k, n, s.half(), n),
           lambda: B.trellis_matmul(x, packed, c, L, k, n, out=torch.empty(2, 4, device="cuda")),
           lambda: B.trellis_matmul(x, packed, c, L, k, n, out=x.view(-1)[100:106].view(2, 3)),
           lambda: B.trellis_pack(packed[0], L, k),
           lambda: B.trellis_pack(packed.float(), L, k),
           lambda: B.trellis_pack(packed.cpu(), L, k),
           lambda: B.trellis_pack(packed, 3, 4)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
