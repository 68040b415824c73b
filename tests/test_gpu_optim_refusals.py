"""A refused optimiser step leaves everything as it was: parameters, states and counts (needs a B200)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _params(kinds, seed=0):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for k in kinds:
        for n in (300, 77):
            p = torch.randn(n, generator=gen).to(k).cuda()
            p.grad_dtype = None
            out.append(p)
    return out


def _grads(ps, seed):
    gen = torch.Generator().manual_seed(seed)
    for p in ps:
        p.grad = torch.randn(p.numel(), generator=gen).to(p.dtype).cuda()


def _all(opt, ps):
    states = [t for bs in opt._buckets for b in bs for t in b["state"] if t is not None]
    return [t.detach().view(torch.uint8).clone() for t in ps + states], [int(b["step"]) for bs in opt._buckets for b in bs]


def _good_steps(opt, ps, seeds):
    for s in seeds:
        _grads(ps, s)
        opt.step()


def _bad_scale(opt, ps):
    opt.step(grad_scale=torch.ones(2, device="cuda"))


def _bad_type(opt, ps):
    # bfloat16 parameters: the gradients of their own type come first, the others are refused
    ps[-1].grad = ps[-1].grad.to(F16)
    opt.step()


def _bad_lr(opt, ps):
    old, opt.param_groups[-1]["lr"] = opt.param_groups[-1]["lr"], float("nan")
    try:
        opt.step()
    finally:
        opt.param_groups[-1]["lr"] = old


def _bad_beta(opt, ps):
    old, opt.param_groups[-1]["betas"] = opt.param_groups[-1]["betas"], (0.9, 1.0)
    try:
        opt.step()
    finally:
        opt.param_groups[-1]["betas"] = old


def _not_contiguous(opt, ps):
    data = ps[-1].data
    ps[-1].data = data.repeat_interleave(2)[::2]
    try:
        opt.step()
    finally:
        ps[-1].data = data


@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [_bad_scale, _bad_type, _bad_lr, _bad_beta, _not_contiguous])
@pytest.mark.parametrize("groups", [1, 2])
def test_a_refused_step_changes_nothing(capturable, bits, bad, groups):
    import differentiable_bcjr_b200 as B
    from differentiable_bcjr_b200.optim import AdamW
    mine, other = _params([F32, BF16]), _params([F32, BF16])
    cut = (lambda ps: [{"params": ps}]) if groups == 1 else (lambda ps: [{"params": ps[:3]}, {"params": ps[3:], "lr": 1e-2}])
    a, b = (AdamW(cut(ps), state_bits=bits, seed=3, capturable=capturable) for ps in (mine, other))
    _good_steps(a, mine, (1, 2))
    _good_steps(b, other, (1, 2))
    _grads(mine, 3)
    before = _all(a, mine)
    with pytest.raises((ValueError, B.BCJRError)):
        bad(a, mine)
    after = _all(a, mine)
    assert after[1] == before[1] and all(torch.equal(x, y) for x, y in zip(after[0], before[0]))
    _good_steps(a, mine, (3, 4))
    _good_steps(b, other, (3, 4))
    x, y = _all(a, mine), _all(b, other)
    assert x[1] == y[1] and all(torch.equal(p, q) for p, q in zip(x[0], y[0]))


def test_gradients_of_two_types_in_one_step():
    from differentiable_bcjr_b200.optim import AdamW
    # the same numbers as gradients of one type
    mine, other = _params([F32]), _params([F32])
    a, b = AdamW(mine), AdamW(other)
    for s in (1, 2):
        _grads(mine, s)
        _grads(other, s)
        other[1].grad = other[1].grad.bfloat16().float()
        mine[1].grad = mine[1].grad.bfloat16()
        a.step()
        b.step()
    assert all(torch.equal(p, q) for p, q in zip(mine, other)) and a._buckets[0][0]["step"] == 2


def test_parameters_over_one_another_are_refused_at_once():
    from differentiable_bcjr_b200.optim import AdamW
    flat = torch.zeros(400, device="cuda")
    with pytest.raises(ValueError):
        AdamW([flat[:300], flat[200:]])
    AdamW([flat[:200], flat[200:]])
