"""The AdamW step with 8-bit states over the whole range of float32 (needs a B200): second moments that are
subnormal or overflow, the root that becomes a code, scales from the smallest to the largest.

Rounding counted: a second moment v = b2 r^2 + (1 - b2) g^2 takes at most four float32 operations, each off by 2^-24
of its result or, where that is subnormal, by 2^-150; so v lies within v (1 +- 2^-22) +- 2^-148, and its root
between the roots of these bounds."""
import math

import numpy as np
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

BETAS = (0.9, 0.999)


def _root_bounds(v):
    return (v * (1 - 2 ** -22) - 2.0 ** -148).clamp(min=0).sqrt(), (v * (1 + 2 ** -22) + 2.0 ** -148).sqrt()


def _states(first, second, scales):
    wide = scales.double().repeat_interleave(R.BLOCK, 1)
    return first.float().double() * wide[0], second.float().double() * wide[1]


@pytest.mark.parametrize("size", [1e-16, 3e-18, 1e-18, 1e-19, 1e-20, 2e-21])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-20, 1e-8])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_tiny_gradients(size, eps, kind):
    import differentiable_bcjr_b200 as B
    n, lr = 1000, 0.5
    gen = torch.Generator().manual_seed(1)
    p = torch.zeros(n, dtype=kind, device="cuda")
    first, second, scales = B.adamw_state([p], 8)
    for step in (1, 2, 3):
        # magnitudes within a factor of two: their squares do not vanish
        g = ((1 + torch.rand(n, generator=gen)) * size * (1 - 2 * torch.randint(0, 2, (n,), generator=gen))).to(kind).cuda()
        m0, r0 = _states(first, second, scales)
        before = p.double()
        B.adamw_step([p], [g], first, second, step, lr, BETAS, eps, scales=scales)
        m = BETAS[0] * m0[:n] + (1 - BETAS[0]) * g.double()
        v = BETAS[1] * r0[:n] ** 2 + (1 - BETAS[1]) * g.double() ** 2
        lo, hi = _root_bounds(v)
        inv = 1 / math.sqrt(1 - BETAS[1] ** step)
        scale = lr / (1 - BETAS[0] ** step)
        # m is off by three roundings of values that are at most the block's largest; the quotient by 2^-21 of itself
        off = 2.0 ** -22 * (m.abs() + g.double().abs())
        least, most = (scale * (m.abs() + s * off) / (r * inv + eps) for s, r in ((-1, hi), (1, lo)))
        moved = (before - p.double()) * m.sign()
        half = before.abs().add(most) * torch.finfo(kind).eps / 2
        assert (moved <= most * (1 + 2 ** -20) + half).all() and (moved >= least.clamp(min=0) * (1 - 2 ** -20) - half).all()
        for b in range(4):
            part = slice(b * 256, min((b + 1) * 256, n))
            got = scales[1, b].item() * 448
            assert lo[part].max().item() * (1 - 2 ** -20) <= got <= hi[part].max().item() * (1 + 2 ** -20)
        # codes are at most one of their steps off: an eighth of the value, or the smallest code
        _, r1 = _states(first, second, scales)
        least_code = scales[1].double().repeat_interleave(R.BLOCK)[:n] * 2.0 ** -9
        assert (r1[:n] <= hi * 1.126 + least_code).all() and (r1[:n] >= lo * 0.874 - least_code).all() and (r1[:n] > 0).all()


def test_tiny_gradients_beside_large_ones():
    import differentiable_bcjr_b200 as B
    # what the tiny ones move by is right although their block's scale belongs to the large one
    for eps, tiny in ((0.0, 1e-19), (1e-25, 1e-19), (1e-14, 1e-18), (1e-8, 1e-18)):
        p = torch.zeros(600, device="cuda")
        g = torch.full((600,), tiny, device="cuda")
        g[::256] = 1.0
        first, second, scales = B.adamw_state([p], 8)
        B.adamw_step([p], [g], first, second, 1, 1.0, (0.9, 0.9999), eps, scales=scales)
        lo, hi = _root_bounds(1e-4 * g.double() ** 2)
        near, far = g.double() / (hi * 100 + eps), g.double() / (lo * 100 + eps)
        assert ((-p.double() >= near * (1 - 2 ** -19)) & (-p.double() <= far * (1 + 2 ** -19))).all()
        assert (second.float()[:600] > 0).all()


@pytest.mark.parametrize("kind,gkind", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_a_gradient_whose_square_overflows(kind, gkind):
    import differentiable_bcjr_b200 as B
    out = {}
    for bits in (32, 8):
        p = torch.ones(600, dtype=kind, device="cuda")
        g = torch.ones(600, dtype=gkind, device="cuda")
        g[3], g[599] = 1e25, -1e30
        a, b, s = B.adamw_state([p], bits)
        B.adamw_step([p], [g], a, b, 1, lr=0.125, eps=0.0, scales=s)
        out[bits] = p.clone()
        if bits == 8:
            # that step is the 32-bit one: the second moment is infinite, so these two stay
            assert torch.equal(out[8], out[32]) and p[3] == 1 and p[599] == 1 and (p[4:599] < 1).all()
            assert not torch.isfinite(s[1, 0]) and not torch.isfinite(s[1, 2]) and torch.isfinite(s[:, 1]).all()
            B.adamw_step([p], [torch.ones_like(g)], a, b, 2, lr=0.125, eps=0.0, scales=s)
            assert torch.isnan(p[:256]).all() and torch.isnan(p[512:]).all() and torch.isfinite(p[256:512]).all()


def test_the_root_against_the_correctly_rounded_one():
    import differentiable_bcjr_b200 as B
    # one gradient a block and no averaging: the second scale is root(fl(g^2)) times 1/448, in float32
    blocks = 1 << 18
    gen = torch.Generator().manual_seed(3)
    bits = torch.randint(127 - 74, 127 + 64, (blocks,), generator=gen) << 23 | torch.randint(0, 1 << 23, (blocks,), generator=gen)
    bits[:2000] = (torch.arange(2000) % 138 + 127 - 74) << 23  # powers of two, and those next to them
    bits[1000:2000] -= 1
    g = bits.to(torch.int32).view(torch.float32)
    p = torch.zeros(blocks * 256, device="cuda")
    a, b, s = B.adamw_state([p], 8)
    B.adamw_step([p], [g.cuda().repeat_interleave(256)], a, b, 1, betas=(0.0, 0.0), scales=s)
    with np.errstate(under="ignore"):
        v = g.numpy() * g.numpy()
        want = np.sqrt(v) * (np.float32(1) / np.float32(448))
    assert want.dtype == np.float32 and np.isfinite(v).all() and (v > 0).all()
    got = s[1].cpu().numpy()
    apart = np.abs(got.view(np.int32) - want.view(np.int32))
    assert apart.max() <= 1 and (apart != 0).sum() <= 2  # a case in millions


@pytest.mark.parametrize("size", [1e-15, 1e-9, 1e-3, 3e3, 1e5, 1e6, 3e8, 1e12, 1e17])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_codes_of_every_size(size, kind):
    import differentiable_bcjr_b200 as B
    n, seed = 256 * 40 + 77, 9
    gen = torch.Generator().manual_seed(4)
    p = torch.zeros(n, dtype=kind, device="cuda")
    first, second, scales = B.adamw_state([p], 8)
    total = first.numel()
    for step in (1, 2, 3):
        g = (torch.randn(n, generator=gen) * size).to(kind).cuda()
        m0, r0 = _states(first, second, scales)
        B.adamw_step([p], [g], first, second, step, 1e-3, (0.9, 0.99), 0.0, scales=scales, seed=seed)
        new = torch.zeros(2, total, dtype=torch.float64, device="cuda")
        _, m, v = R.adamw(p, g, m0[:n], r0[:n] ** 2, step, 1e-3, 0.9, 0.99, 0.0, 0.0)
        new[0, :n], new[1, :n] = m, v.sqrt()
        bits = R.hash16(total, step, seed, "cuda")
        for k, codes in enumerate((first, second)):
            x = new[k].view(-1, R.BLOCK)
            top = x.abs().amax(1)
            assert ((scales[k].double() - top / 448).abs() <= top / 448 * 2 ** -20).all()
            t = x.abs() * (448 / top)[:, None]
            least = t.clamp(min=2.0 ** -6)
            unit = least / torch.frexp(least).mantissa / 16
            part = t / unit - torch.floor(t / unit)
            threshold = (part * 2 ** 20 + bits[k].view(-1, R.BLOCK) * 16 + 8) / 2 ** 20
            want = (torch.floor(t / unit) + (threshold >= 1)) * unit
            if k == 1:
                want = torch.where((x > 0) & (want == 0), torch.full_like(want, 2.0 ** -9), want)
            got = codes.float().double().view(-1, R.BLOCK)
            # the float32 forms of t are off by less than 2^-19 of it, 16 units at most, which decides next to a threshold
            near = ((threshold - 1).abs() <= 16 * 2.0 ** -18) | (part < 2.0 ** -14) | (part > 1 - 2.0 ** -14)
            assert ((got.abs() == want.clamp(max=448)) | near).all()
    assert torch.isfinite(p).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [1e-37, 1e-38, 1e-40, 1e-45, 1e-60, 5e-324])
def test_an_eps_below_float32s_normal_numbers(bits, eps):
    import differentiable_bcjr_b200 as B
    p = torch.ones(600, device="cuda")
    first, second, scales = B.adamw_state([p], bits)
    m = v = torch.zeros(600, dtype=torch.float64, device="cuda")
    for step in (1, 2):
        g = torch.linspace(-1, 1, 600, device="cuda")
        g[::3] = 0  # moments of 0: a step of 0 / eps
        before = p.clone()
        if bits == 8:
            m, r = (t[:600] for t in _states(first, second, scales))
            v = r * r
        B.adamw_step([p], [g], first, second, step, 0.25, (0.9, 0.99), eps, scales=scales)
        want, m, v = R.adamw(before, g, m, v, step, 0.25, 0.9, 0.99, eps, 0.0)
        assert (p[::3] == 1).all()
        # a step is at most 0.25 / sqrt(1 - beta2), of ten roundings; the parameter one more
        assert ((p.double() - want).abs() <= 2.5 * 2 ** -20 + want.abs() * 2 ** -23).all()
