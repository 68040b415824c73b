"""The layer that QAT packs, with its codebook in the type that it is served in (needs a B200)."""
import pytest
import torch

import bcjr_inputs as I

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
def test_qat_packs_a_codebook_of_the_activations_type(kind):
    import differentiable_bcjr_b200 as B
    from differentiable_bcjr_b200.qat import layer_reconstruction_qat
    L, k, n, R, C = 8, 2, 64, 16, 256
    W, X, c = I.normal((R, C), 71).cuda(), I.normal((32, C), 72).cuda(), I.codebook(1 << L, 73).cuda()
    args = dict(steps_per_temperature=2, lr=0.02, train_codebook=True, optimizer="adamw", pack=True)
    res = layer_reconstruction_qat(W, X, c, L, k, n, [0.3], pack_codebook_dtype=kind, **args)
    layer = res["linear"]
    # decoded with the codebook as it was trained, kept in the type asked for
    assert layer.codebook.dtype == kind and torch.equal(layer.codebook, res["codebook"].to(kind))
    states, hard = B.viterbi_decode(res["preimage"].view(-1, n), res["codebook"], L, k)
    assert torch.equal(layer.packed, B.trellis_pack(states, L, k)) and torch.equal(hard.view(R, C), res["w_qat"])
    used = layer.codebook.double()[states.long()].view(R, C)
    x = X.to(kind)
    for tokens in (1, 8, 32):
        y, want = layer(x[:tokens]).double(), x[:tokens].double() @ used.t()
        size = x[:tokens].double().abs() @ used.abs().t()
        # exact products; no more than 64 float32 sums on a value's way, each cutting or rounding 2^-23; then y's type
        assert ((y - want).abs() <= want.abs() * torch.finfo(kind).eps / 2 + size * 64 * 2 ** -23 + 2.0 ** -25).all()
    assert layer_reconstruction_qat(W, X, c, L, k, n, [0.3], **args)["linear"].codebook.dtype == torch.float32


def test_a_codebook_type_that_no_layer_keeps_is_refused_before_training():
    from differentiable_bcjr_b200.qat import layer_reconstruction_qat
    with pytest.raises(ValueError, match="codebook"):
        layer_reconstruction_qat(torch.ones(4, 64), torch.ones(2, 64), torch.zeros(256), 8, 2, 32, [0.3], pack=True,
                                 pack_codebook_dtype=torch.float64)
