"""The optimiser class, the quantised layers and the QAT loop that uses them, together (needs a B200)."""
import math

import pytest
import torch

import bcjr_inputs as I

pytestmark = pytest.mark.gpu


def _model(kinds, seed=0):
    gen = torch.Generator().manual_seed(seed)
    shapes = [(33, 17), (300,), (1, 1), (64, 64)]
    return [torch.nn.Parameter(torch.randn(s, generator=gen).to(k).cuda()) for k in kinds for s in shapes]


def test_optimiser_follows_torch_with_32_bits():
    from differentiable_bcjr_b200.optim import AdamW
    mine, theirs = _model([torch.float32]), _model([torch.float32])
    groups = lambda ps: [{"params": ps[:2], "lr": 3e-3}, {"params": ps[2:], "weight_decay": 0.2}]  # noqa: E731
    a = AdamW(groups(mine), lr=1e-2, weight_decay=0.05)
    b = torch.optim.AdamW(groups(theirs), lr=1e-2, weight_decay=0.05)
    for step in range(6):
        gen = torch.Generator().manual_seed(step)
        for p, q in zip(mine, theirs):
            g = torch.randn(p.shape, generator=gen).cuda()
            p.grad, q.grad = g.clone(), g
        a.step()
        b.step()
        a.zero_grad()
        assert all(p.grad is None for p in mine)
    for p, q in zip(mine, theirs):
        # a step is at most about ten roundings of float32 off in either, and a step's size is at most lr * 3.2
        assert ((p - q).abs() <= q.abs() * 2 ** -22 * 6 + 6 * 1e-2 * 3.2 * 2 ** -20).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_optimiser_state_moves_to_another(bits):
    from differentiable_bcjr_b200.optim import AdamW
    kinds = [torch.float32, torch.bfloat16, torch.float16]
    first, second = _model(kinds), _model(kinds)

    def run(opt, ps, steps):
        for step in steps:
            gen = torch.Generator().manual_seed(100 + step)
            for p in ps:
                p.grad = torch.randn(p.shape, generator=gen).to(p.dtype).cuda()
            opt.step()

    a = AdamW(first, lr=1e-3, state_bits=bits, seed=4)
    run(a, first, range(5))
    b = AdamW(second, lr=9.0, state_bits=bits, capturable=True)
    with torch.no_grad():
        for p, q in zip(first, second):
            q.copy_(p)
    b.load_state_dict(a.state_dict())
    run(a, first, range(5, 8))
    run(b, second, range(5, 8))
    for p, q in zip(first, second):
        # the step count on the device goes through the device's pow, a last place of a double away
        assert torch.allclose(p, q, rtol=2 * torch.finfo(p.dtype).eps, atol=1e-3 * 2 ** -18)
    with pytest.raises(ValueError):
        AdamW(first[:2], state_bits=bits).load_state_dict(a.state_dict())
    with pytest.raises(ValueError):
        AdamW(first, state_bits=40 - bits).load_state_dict(a.state_dict())


def test_optimiser_without_some_gradients_and_refusals():
    from differentiable_bcjr_b200.optim import AdamW
    ps = _model([torch.float32])
    opt = AdamW(ps)
    before = [p.detach().clone() for p in ps]
    opt.step()
    ps[1].grad = torch.ones_like(ps[1]).expand(300)
    opt.step()
    assert [torch.equal(p, q) for p, q in zip(ps, before)] == [True, False, True, True]
    for bad in ([], [ps[0], ps[0]], [ps[0].cpu()], [ps[0].t()], [ps[0].double()]):
        with pytest.raises(ValueError):
            AdamW(bad)


def test_a_captured_training_step_replays():
    # a quantised-weight training step, backward and optimiser included, as one graph
    import differentiable_bcjr_b200 as B
    from differentiable_bcjr_b200.optim import AdamW
    L, k, n = 8, 2, 32
    c = I.codebook(1 << L).cuda()
    w0, x = I.normal((8, n), 3).cuda(), I.normal((16, n), 4).cuda()

    def step(v, opt):
        loss = ((x @ (w0 - B.soft_quantize(v, c, 0.1, L, k)).T) ** 2).mean()
        loss.backward()
        opt.step()
        opt.zero_grad(set_to_none=False)
        return loss.detach()

    eager, captured = w0.clone().requires_grad_(), w0.clone().requires_grad_()
    a, b = AdamW([eager], lr=0.02), AdamW([captured], lr=0.02, capturable=True)
    losses = [step(eager, a) for _ in range(5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [step(captured, b).clone() for _ in range(2)]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step(captured, b)
    for _ in range(3):
        graph.replay()
        got.append(loss.clone())
    # five steps of float32 arithmetic whose bias corrections differ by a last place
    assert torch.allclose(torch.stack(got), torch.stack(losses), rtol=1e-4)
    assert torch.allclose(captured, eager, rtol=0, atol=5 * 0.02 * 2 ** -12)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("zero", [False, True])
def test_int4_layer_is_near_its_weight(kind, zero):
    from differentiable_bcjr_b200.linear import Int4Linear
    w, x = I.normal((100, 320), 1).to(kind).cuda(), I.normal((2, 5, 320), 2).to(kind).cuda()
    bias = I.normal((100,), 3).to(kind).cuda()
    layer = Int4Linear.from_weight(w, 64, zero, bias=bias)
    with torch.no_grad():
        y = layer(x)
    want = x.double() @ w.double().t() + bias.double()
    # a weight is at most half a code off, a code a seventh (fifteenth of the range) of the group's largest
    part = w.double().view(100, 5, 64)
    reach = torch.where(torch.tensor(zero), (part.amax(2).clamp(min=0) - part.amin(2).clamp(max=0)) / 30, part.abs().amax(2) / 14).cuda()
    off = (x.double().abs().view(2, 5, 5, 64).sum(3) @ reach.t()) * 1.02
    assert y.shape == (2, 5, 100) and ((y.double() - want).abs() <= off + want.abs() * 2 ** -7 + 2.0 ** -7).all()
    again = Int4Linear(layer.packed, layer.scales, layer.zeros, 320, 64, bias)
    again.load_state_dict(layer.state_dict())
    assert torch.equal(again(x), y)
    assert layer(x.transpose(0, 1)).shape == (5, 2, 100)  # made contiguous
    with pytest.raises(RuntimeError):
        layer(x.clone().requires_grad_())
    with pytest.raises(ValueError):
        layer(x[..., :319])


@pytest.mark.parametrize("group", [None, 0, 64, 16])
@pytest.mark.parametrize("ckind", [None, torch.bfloat16])
def test_trellis_layer_multiplies_what_it_decoded(group, ckind):
    import differentiable_bcjr_b200 as B
    from differentiable_bcjr_b200.linear import TrellisLinear
    L, k, n, rows, cols = 10, 2, 64, 20, 256
    w, c, x = I.normal((rows, cols), 1).cuda() * 3, I.codebook(1 << L).cuda(), I.normal((3, cols), 2).cuda()
    layer = TrellisLinear.from_weight(w, c, L, k, n, group, ckind)
    assert layer.out_features == rows and layer.packed.shape == (rows * cols // n, 5)  # 64 steps of 2 bits and 8 more: 136 bits
    scale = torch.ones(rows, cols, device="cuda")
    if group is not None:
        scale = w.view(rows, -1, group or cols).square().mean(2).sqrt().repeat_interleave(group or cols, 1)
    _, hard = B.viterbi_decode((w / scale).view(-1, n), c, L, k)
    used = (hard.to(ckind) if ckind else hard).view(rows, cols).double() * scale.double()
    y = layer(x).double()
    want = x.double() @ used.t()
    size = x.double().abs() @ used.abs().t()
    assert ((y - want).abs() <= size * 64 * 2 ** -24).all()
    # converted as a whole: codebook and scales lose half a step of the type each, the output one
    got = layer.half()(x.half()).double()
    want = x.half().double() @ used.t()
    assert ((got - want).abs() <= size * 1.01 * (2 ** -11 * 2 + 2 ** -9 * (ckind is not None)) + want.abs() * 2 ** -11 + 2.0 ** -24).all()


@pytest.mark.parametrize("optimizer", ["adamw", "adamw8"])
def test_qat_runs_with_the_fused_step_and_serves_its_result(optimizer):
    from differentiable_bcjr_b200.qat import layer_reconstruction_qat
    L, k, n, R, C = 8, 4, 64, 16, 256
    W, X, c = I.normal((R, C), 71).cuda(), I.normal((32, C), 72).cuda(), I.codebook(1 << L, 73).cuda()
    res = layer_reconstruction_qat(W, X, c, L, k, n, [0.3, 0.1], steps_per_temperature=3, lr=0.02, train_codebook=True,
                                   optimizer=optimizer, pack=True, int4_group_size=128)
    assert all(math.isfinite(v) for v in res["history"]) and len(res["history"]) == 6
    assert not torch.equal(res["preimage"], W) and not torch.equal(res["codebook"], c)
    y = res["linear"](X).double()
    want = X.double() @ res["w_qat"].double().t()
    assert ((y - want).abs() <= X.double().abs() @ res["w_qat"].double().abs().t() * 64 * 2 ** -24).all()
    # rounding to a seventh of a group's largest of 128 normal weights: between a third and once its uniform error
    step = W.view(R, 2, 128).abs().amax(2).mean().item() / 7
    assert 0.3 * step ** 2 / 12 * C < res["mse_int4"] < 1.5 * step ** 2 / 12 * C
    with pytest.raises(ValueError):
        layer_reconstruction_qat(W, X, c, L, k, n, [0.3], optimizer="sgd")


def test_qat_of_the_fused_step_follows_torch():
    from differentiable_bcjr_b200.qat import layer_reconstruction_qat
    L, k, n, R, C = 8, 2, 64, 8, 128
    W, X, c = I.normal((R, C), 71).cuda(), I.normal((32, C), 72).cuda(), I.codebook(1 << L, 73).cuda()
    a, b = (layer_reconstruction_qat(W, X, c, L, k, n, [0.3], steps_per_temperature=2, optimizer=o) for o in ("adam", "adamw"))
    # the first step is the same but for roundings; the second's gradient is taken there
    assert abs(a["history"][0] - b["history"][0]) <= 1e-6 * a["history"][0]
    assert abs(a["history"][1] - b["history"][1]) <= 1e-3 * a["history"][1]
