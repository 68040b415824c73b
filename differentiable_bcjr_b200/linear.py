"""Linear layers with quantised weights, for serving what QAT or plain
rounding gives: `TrellisLinear` keeps hard-decoded trellis codes at k bits a
weight, `Int4Linear` 4-bit codes with group scales.  Both multiply a few
tokens at a time by the library's own kernels; neither has a gradient.
"""
from __future__ import annotations

import torch

from . import int4_matmul, int4_quantize, trellis_matmul, trellis_pack, trellis_words, viterbi_decode
from .layer import _trellis_groups


def _frozen(x):
    if torch.is_grad_enabled() and x.requires_grad:
        raise RuntimeError("a quantised layer has no gradient: call it under torch.no_grad()")
    return x.contiguous()


def check_codebook_dtype(dtype):
    """Raises if a layer cannot keep its codebook in `dtype` (None: as it is)."""
    if dtype not in (None, torch.float32, torch.float16, torch.bfloat16):
        raise ValueError(f"a layer keeps its codebook in float32, float16 or bfloat16, not {dtype}")


class Int4Linear(torch.nn.Module):
    """y = x W^T + bias with W in 4 bits (see `int4_quantize` for the forms).

        layer = Int4Linear.from_weight(w, group_size=128)
    """

    def __init__(self, packed, scales, zeros, in_features, group_size=128, bias=None):
        super().__init__()
        self.in_features, self.out_features, self.group_size = int(in_features), scales.shape[1], int(group_size)
        for name, t in (("packed", packed), ("scales", scales), ("zeros", zeros), ("bias", bias)):
            self.register_buffer(name, t)

    @classmethod
    def from_weight(cls, w, group_size=128, zero_point=False, scale_dtype=None, bias=None):
        """Rounds w [out_features][in_features] to 4 bits."""
        packed, scales, zeros = int4_quantize(w.detach().contiguous(), group_size, zero_point, scale_dtype)
        return cls(packed, scales, zeros, w.shape[1], group_size, bias)

    def forward(self, x):
        if x.shape[-1] != self.in_features:
            raise ValueError(f"x must be [..., {self.in_features}]")
        y = int4_matmul(_frozen(x), self.packed, self.scales, self.zeros, self.group_size)
        return y if self.bias is None else y + self.bias


class TrellisLinear(torch.nn.Module):
    """y = x W^T + bias with W hard-decoded on a bitshift trellis and kept at k bits a weight.

        layer = TrellisLinear.from_weight(preimage, codebook, state_bits=16, k=2, seq_len=256)
    """

    def __init__(self, packed, codebook, state_bits, k, seq_len, in_features, scales=None, group_size=0, bias=None):
        super().__init__()
        self.state_bits, self.k, self.seq_len = int(state_bits), int(k), int(seq_len)
        self.in_features, self.group_size = int(in_features), int(group_size)
        self.out_features = packed.shape[0] * self.seq_len // self.in_features
        for name, t in (("packed", packed), ("codebook", codebook), ("scales", scales), ("bias", bias)):
            self.register_buffer(name, t)

    @classmethod
    def from_weight(cls, w, codebook, state_bits, k, seq_len, group_size=None, codebook_dtype=None, bias=None):
        """Hard-decodes w [out_features][in_features] (float32; rows are whole
        sequences of `seq_len`).  With group_size None the codebook is that of
        the weights themselves; otherwise each group of columns (0: each row)
        is divided by its root mean square first, which becomes its scale.
        `codebook_dtype`: what the layer keeps the codebook in (the decoding
        uses it as it is)."""
        rows, cols = w.shape
        if cols % seq_len:
            raise ValueError("a row must be whole sequences")
        # what the packing or the product refuses is not decoded first
        trellis_words(state_bits, k, seq_len)
        check_codebook_dtype(codebook_dtype)
        w = w.detach().contiguous()
        scales = None
        if group_size is not None:
            parts = w.view(rows, _trellis_groups(cols, seq_len, group_size), -1)
            rms = parts.square().mean(2).sqrt()
            # squares that leave float32's range are those of parts of the largest; a group of zeros has the scale 0
            top = parts.abs().amax(2)
            far = top * (parts / top.clamp(min=2.0 ** -149)[:, :, None]).square().mean(2).sqrt()
            rms = torch.where((rms > 2.0 ** -60) & (rms < 2.0 ** 60), rms, far)
            w = (parts / torch.where(rms > 0, rms, torch.ones_like(rms))[:, :, None]).view(rows, cols)
            scales = rms.t().contiguous()
        states, _ = viterbi_decode(w.view(-1, seq_len), codebook, state_bits, k)
        kept = codebook if codebook_dtype is None else codebook.to(codebook_dtype)
        return cls(trellis_pack(states, state_bits, k), kept.detach().clone(), state_bits, k, seq_len, cols, scales,
                   group_size or 0, bias)

    def forward(self, x):
        if x.shape[-1] != self.in_features:
            raise ValueError(f"x must be [..., {self.in_features}]")
        scales = self.scales  # float32, unless the module was converted as a whole
        if scales is not None and scales.dtype != torch.float32:
            scales = scales.float()
        y = trellis_matmul(_frozen(x), self.packed, self.codebook, self.state_bits, self.k, self.seq_len, scales,
                           self.group_size)
        return y if self.bias is None else y + self.bias
