"""The AdamW step of many tensors against the formula in 64 bits (needs a B200).

Rounding counted in the tolerances: a float32 operation is off by at most
2^-24 of its result, sqrt.approx and the approximate division by 2^-22; a
parameter is rounded once to its type (half a step)."""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

LR, BETAS, EPS = 1e-2, (0.9, 0.99), 1e-8
SIZES = {"one": [1], "block": [256], "ragged": [255, 257, 1, 0, 1000, 256, 4099], "many": [1 + 37 * i % 901 for i in range(300)],
         "wide": [2048 * 70 + 3], "over a table": [3 + i % 5 for i in range(1100)]}


def _tensors(sizes, dtype, seed, scale, tight=False, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    data = [torch.randn(n, generator=gen) * scale for n in sizes]
    if not tight:
        return [d.to(dtype).to(device) for d in data]
    flat = torch.cat([torch.zeros(1)] + data).to(dtype).to(device)  # one element in: nothing is aligned
    out, at = [], 1
    for n in sizes:
        out.append(flat[at:at + n])
        at += n
    return out


def _check_p(got, want, dtype, step_size):
    # lr * m / denominator comes out of about eight float32 operations, two of them approximate
    half = torch.finfo(dtype).eps / 2
    tol = want.abs() * (half + 2 ** -22) + step_size * 2 ** -20 + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() / tol.clamp(min=1e-300)).max()


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("kind,gkind", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.float32, torch.float16),
                                        (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
                                        (torch.float16, torch.float32)])
def test_32_bit_states_follow_the_formula(sizes, kind, gkind):
    import differentiable_bcjr_b200 as B
    sizes = SIZES[sizes]
    tight = kind == gkind
    params = _tensors(sizes, kind, 1, 0.5, tight)
    state = B.adamw_state(params, 32)
    gs = torch.full((1,), 0.25, device="cuda")
    ref = [(p.double(), torch.zeros(p.numel(), device="cuda").double(), torch.zeros(p.numel(), device="cuda").double()) for p in params]
    offsets, _ = R.flat_offsets(sizes)
    for step in (1, 2, 3):
        grads = _tensors(sizes, gkind, 10 + step, 1e-2, tight)
        before = [p.clone() for p in params]
        B.adamw_step(params, grads, state[0], state[1], step, LR, BETAS, EPS, 0.1, grad_scale=gs)
        for i, (p, g, b, at) in enumerate(zip(params, grads, before, offsets)):
            _, m, v = ref[i]
            want, m, v = R.adamw(b, g, m, v, step, LR, *BETAS, EPS, 0.1, 0.25)
            ref[i] = (want, m, v)
            n = p.numel()
            # three roundings a step of values that are at most the running maxima
            top_m = (g.double().abs() * 0.25).max() if n else 0
            assert n == 0 or ((state[0][at:at + n].double() - m).abs() <= step * 2 ** -22 * (m.abs() + top_m)).all()
            assert n == 0 or ((state[1][at:at + n].double() - v).abs() <= step * 2 ** -22 * v).all()
            # the states' own rounding reaches p through m / sqrt(v), which is at most about 1 / sqrt(1 - beta2)
            _check_p(p, want, kind, LR * 10)


def test_padding_of_the_states_stays_zero():
    import differentiable_bcjr_b200 as B
    for bits in (32, 8):
        params, grads = _tensors([5, 300], torch.float32, 1, 1.0), _tensors([5, 300], torch.float32, 2, 1.0)
        a, b, s = B.adamw_state(params, bits)
        B.adamw_step(params, grads, a, b, 1, scales=s)
        pad = torch.ones(768, dtype=torch.bool, device="cuda")
        pad[:5] = False
        pad[256:556] = False
        for t in (a, b):
            assert (t.view(torch.uint8).view(768, -1)[pad] == 0).all()


@pytest.mark.parametrize("kind,gkind", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
@pytest.mark.parametrize("sizes", ["ragged", "wide"])
@pytest.mark.parametrize("tight", [False, True])
def test_8_bit_states_follow_the_formula_and_its_rounding(kind, gkind, sizes, tight):
    import differentiable_bcjr_b200 as B
    sizes = SIZES[sizes]
    params = _tensors(sizes, kind, 1, 0.5, tight)
    first, second, scales = B.adamw_state(params, 8)
    offsets, total = R.flat_offsets(sizes)
    seed = 5
    for step in (1, 2, 7):
        grads = _tensors(sizes, gkind, 20 + step, 1e-2, tight)
        before = [p.clone() for p in params]
        wide = scales.double().repeat_interleave(R.BLOCK, 1)
        m0, r0 = first.float().double() * wide[0], second.float().double() * wide[1]
        B.adamw_step(params, grads, first, second, step, LR, BETAS, EPS, 0.1, scales=scales, seed=seed)
        new = torch.zeros(2, total, dtype=torch.float64, device="cuda")
        for p, g, b, at in zip(params, grads, before, offsets):
            n = p.numel()
            want, m, v = R.adamw(b, g, m0[at:at + n], r0[at:at + n] ** 2, step, LR, *BETAS, EPS, 0.1)
            _check_p(p, want, kind, LR * 10)
            new[0, at:at + n], new[1, at:at + n] = m, v.sqrt()
        bits = R.hash16(total, step, seed, "cuda")
        for k, codes in enumerate((first, second)):
            x = new[k].view(-1, R.BLOCK)
            top = x.abs().amax(1)
            assert ((scales[k].double() - top / 448).abs() <= top / 448 * 2 ** -20).all()
            t = x.abs() * (448 / top.clamp(min=1e-300))[:, None]
            # in units of the code's step: 2^(e - 3) for t in [2^e, 2^(e+1)), 2^-9 under 2^-6
            least = t.clamp(min=2.0 ** -6)
            unit = least / torch.frexp(least).mantissa / 16  # the mantissa lies in [1/2, 1): exact
            part = t / unit - torch.floor(t / unit)
            up = part * 2 ** 20 + bits[k].view(-1, R.BLOCK) * 16 + 8 >= 2 ** 20
            want = (torch.floor(t / unit) + up) * unit
            if k == 1:
                want = torch.where((x > 0) & (want == 0), torch.full_like(want, 2.0 ** -9), want)
            got = codes.float().double().view(-1, R.BLOCK)
            if k == 0:
                assert ((got < 0) <= (x < 0)).all()
            # the float32 forms of t are off by less than 2^-19, which decides only next to the threshold
            near = ((part * 2 ** 20 + bits[k].view(-1, R.BLOCK) * 16 + 8) / 2 ** 20 - 1).abs() <= 16 * 2.0 ** -18
            near |= (part < 2.0 ** -14) | (part > 1 - 2.0 ** -14)
            assert ((got.abs() == want.clamp(max=448)) | near).all()
            assert ((got.abs() - t).abs() <= unit * (1 + 2.0 ** -14))[want > 2.0 ** -9].all()


def test_8_bit_rounding_is_unbiased():
    import differentiable_bcjr_b200 as B
    # a constant gradient of two sizes: over many seeds the mean of a code is the value it stands for
    n = 256 * 64
    g = torch.full((n,), 0.0123, device="cuda")
    g[::256] = 1.0
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    seeds = 200
    for seed in range(seeds):
        p = torch.zeros(n, device="cuda")
        a, b, s = B.adamw_state([p], 8)
        B.adamw_step([p], [g], a, b, 1, betas=(0.9, 0.99), scales=s, seed=seed)
        total += a.float().double() * s[0].double().repeat_interleave(256)
    mean = (total / seeds)[torch.arange(n, device="cuda") % 256 != 0].mean().item()
    # a code's step there is at most 2^-3 of the value, so one rounding's deviation is at most half of that, over all draws
    assert abs(mean / (0.1 * 0.0123) - 1) <= 5 * 2 ** -4 / math.sqrt(seeds * n * 255 / 256)


def test_a_missing_gradient_leaves_its_tensor_alone():
    import differentiable_bcjr_b200 as B
    for bits in (32, 8):
        params = _tensors([300, 700], torch.float32, 1, 1.0)
        a, b, s = B.adamw_state(params, bits)
        B.adamw_step(params, _tensors([300, 700], torch.float32, 2, 1.0), a, b, 1, scales=s)
        keep = params[0].clone(), a[:512].view(torch.uint8).clone(), b[:512].view(torch.uint8).clone()
        moved = params[1].clone()
        B.adamw_step(params, [None, torch.ones(700, device="cuda")], a, b, 2, scales=s)
        assert torch.equal(params[0], keep[0]) and not torch.equal(params[1], moved)
        assert torch.equal(a[:512].view(torch.uint8), keep[1]) and torch.equal(b[:512].view(torch.uint8), keep[2])


def test_zero_and_non_finite_gradients():
    import differentiable_bcjr_b200 as B
    for bits in (32, 8):
        p = torch.ones(600, device="cuda")
        a, b, s = B.adamw_state([p], bits)
        B.adamw_step([p], [torch.zeros(600, device="cuda")], a, b, 1, scales=s)
        assert (p == 1).all() and (a.float() == 0).all() and (b.float() == 0).all()
        g = torch.ones(600, device="cuda")
        g[3], g[300] = float("nan"), float("inf")
        B.adamw_step([p], [g], a, b, 2, scales=s)
        bad = ~torch.isfinite(p)
        assert bad[3] and bad[300] and bad.sum() == 2
        if bits == 8:
            assert not torch.isfinite(s[:, :2]).any() and torch.isfinite(s[:, 2]).all()


def test_step_count_on_the_device_and_in_a_graph():
    import differentiable_bcjr_b200 as B
    for bits in (32, 8):
        sizes = [1000, 70000, 3]
        params, again = _tensors(sizes, torch.float32, 1, 1.0), _tensors(sizes, torch.float32, 1, 1.0)
        s1, s2 = B.adamw_state(params, bits), B.adamw_state(again, bits)
        static = [torch.zeros_like(p) for p in params]
        count = torch.zeros(1, dtype=torch.int64, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            count += 1
            B.adamw_step(params, static, s1[0], s1[1], count, scales=s1[2], seed=3)
        for step in (1, 2, 3):
            grads = _tensors(sizes, torch.float32, 50 + step, 1e-2)
            for a, g in zip(static, grads):
                a.copy_(g)
            graph.replay()
            B.adamw_step(again, grads, s2[0], s2[1], step, scales=s2[2], seed=3)
            # the device's pow may differ from the host's in the last place of a double
            for a, b in zip(params, again):
                assert torch.allclose(a, b, rtol=2 ** -20, atol=1e-3 * 2 ** -20)
        with pytest.raises(ValueError):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                B.adamw_step(params, static, s1[0], s1[1], 4, scales=s1[2])


def test_another_stream_and_repeatability():
    import differentiable_bcjr_b200 as B
    out = []
    for _ in range(2):
        params = _tensors([5000, 77], torch.bfloat16, 1, 1.0)
        grads = _tensors([5000, 77], torch.bfloat16, 2, 1.0)
        st = B.adamw_state(params, 8)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for step in range(1, 5):
                B.adamw_step(params, grads, st[0], st[1], step, scales=st[2])
        torch.cuda.current_stream().wait_stream(side)
        out.append(params + [st[0].view(torch.uint8), st[1].view(torch.uint8), st[2]])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_autograd_sees_the_change():
    import differentiable_bcjr_b200 as B
    p = torch.ones(10, device="cuda", requires_grad=True)
    y = (p * p).sum()
    st = B.adamw_state([p])
    B.adamw_step([p], [torch.ones(10, device="cuda")], st[0], st[1], 1)
    with pytest.raises(RuntimeError):
        y.backward()


def test_refusals():
    import differentiable_bcjr_b200 as B
    p, g = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    a, b, _ = B.adamw_state([p])
    bad = [lambda: B.adamw_step([p], [], a, b, 1),
           lambda: B.adamw_step([p], [g[:10]], a, b, 1),
           lambda: B.adamw_step([p], [g.cpu()], a, b, 1),
           lambda: B.adamw_step([p.double()], [g], a, b, 1),
           lambda: B.adamw_step([p.half()], [g.bfloat16()], a, b, 1),
           lambda: B.adamw_step([p], [g.repeat_interleave(2)[::2]], a, b, 1),
           lambda: B.adamw_step([p, p], [g, g], *B.adamw_state([p, p])[:2], 1),
           lambda: B.adamw_step([p[:200], p[100:]], [g[:200], g[100:]], *B.adamw_state([p[:200], p[100:]])[:2], 1),
           lambda: B.adamw_step([p], [g], a[:256], b, 1),
           lambda: B.adamw_step([p], [g], a.half(), b, 1),
           lambda: B.adamw_step([p], [g], a, b, 1, scales=torch.ones(2, 2, device="cuda")),
           lambda: B.adamw_step([p], [g], a, b, torch.ones(1, device="cuda")),
           lambda: B.adamw_step([p], [g], a, b, 1, grad_scale=torch.ones(2, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for kw in ({"lr": -1.0}, {"lr": float("nan")}, {"betas": (1.0, 0.9)}, {"betas": (0.9, -0.1)}, {"eps": -1.0}, {"weight_decay": float("inf")}):
        with pytest.raises(B.BCJRError):
            B.adamw_step([p], [g], a, b, 1, **kw)
    with pytest.raises(B.BCJRError):
        B.adamw_step([p], [g], a, b, 0)
    assert (p == 1).all() and (a == 0).all()
