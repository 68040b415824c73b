"""What the layers and the QAT loop refuse, before any work is done (CPU only)."""
import pytest
import torch

L, K, N = 8, 2, 32


def _qat(W=None, **kw):
    from differentiable_bcjr_b200.qat import layer_reconstruction_qat
    W = torch.ones(4, 64) if W is None else W
    args = {"state_bits": L, "k": K, "seq_len": N, **kw}
    return layer_reconstruction_qat(W, torch.ones(2, W.shape[1]), torch.zeros(1 << args["state_bits"]), temperatures=[0.3], **args)


@pytest.mark.parametrize("group", [96, -128, 16, 100])
def test_qat_refuses_a_group_size_before_it_trains(group):
    with pytest.raises(ValueError, match="group_size must be"):
        _qat(int4_group_size=group)


@pytest.mark.parametrize("state_bits,k", [(8, 5), (17, 2), (3, 4)])
def test_qat_refuses_codes_that_cannot_be_packed_before_it_trains(state_bits, k):
    with pytest.raises(ValueError, match="packed trellis codes need"):
        _qat(state_bits=state_bits, k=k, pack=True)


def test_qat_refuses_rows_that_are_no_sequences_before_it_trains():
    with pytest.raises(ValueError, match="whole sequences"):
        _qat(W=torch.ones(4, 40), pack=True)


@pytest.mark.parametrize("group", [24, 48, -32, 128, 8])
def test_a_trellis_layer_that_could_not_multiply_is_not_made(group):
    # 96 columns in sequences of 32: 24 and 8 are no multiples of 16, 48 divides no sequence, 128 no row
    from differentiable_bcjr_b200.linear import TrellisLinear
    with pytest.raises(ValueError, match="group_size must be"):
        TrellisLinear.from_weight(torch.ones(4, 96), torch.zeros(1 << L), L, K, N, group)


def test_a_trellis_layer_that_could_not_be_packed_is_not_decoded():
    from differentiable_bcjr_b200.linear import TrellisLinear
    with pytest.raises(ValueError, match="packed trellis codes need"):
        TrellisLinear.from_weight(torch.ones(4, 96), torch.zeros(1 << L), L, 5, N)


@pytest.mark.parametrize("kind", [torch.float64, torch.int8])
def test_a_trellis_layer_of_a_codebook_that_no_product_takes_is_not_made(kind):
    from differentiable_bcjr_b200.linear import TrellisLinear
    with pytest.raises(ValueError, match="codebook"):
        TrellisLinear.from_weight(torch.ones(4, 96), torch.zeros(1 << L), L, K, N, codebook_dtype=kind)
