"""Per-layer reconstruction-MSE QAT on synthetic data.

"BCJR-QAT: A Differentiable Relaxation of Trellis-Coded Weight Quantization",
OLMoE experiment: greedy per-layer QAT that minimises the layer's
reconstruction mean squared error (a proxy objective), compared with the
hard-decoded post-training quantisation of the same weights.

Here: a layer W [R][C] (rows split into trellis sequences of `seq_len`
weights) and inputs X [B][C].  The preimage V starts at W; at each
temperature of an annealing schedule, a few optimiser steps minimise
mean((X W^T - X W_hat(V)^T)^2) with W_hat the BCJR soft codeword of V (the
library's forward and backward calls through autograd).  At the end V is
hard-decoded with the Viterbi call and compared with decoding W directly.
The matrix products are ordinary PyTorch; every trellis step runs in the
library's kernels, and on request the optimiser step (`optimizer="adamw"` or
"adamw8"), the packed layer that the result is served as (`pack`) and the
4-bit rounding it is compared with (`int4_group_size`).
"""
from __future__ import annotations

import torch

from . import soft_quantize, trellis_words, viterbi_decode
from .layer import _groups
from .linear import Int4Linear, TrellisLinear, check_codebook_dtype
from .optim import AdamW


def _recon_mse(X, W_ref, W_q):
    return ((X @ (W_ref - W_q).T) ** 2).mean()


def layer_reconstruction_qat(W: torch.Tensor, X: torch.Tensor, codebook: torch.Tensor, state_bits: int, k: int,
                             seq_len: int, temperatures, steps_per_temperature: int = 10, lr: float = 0.02,
                             train_codebook: bool = False, optimizer: str = "adam", pack: bool = False,
                             int4_group_size: int | None = None, pack_codebook_dtype: torch.dtype | None = None):
    """Returns a dict with the loss history, the hard-decoded reconstruction MSE
    after QAT (`mse_qat`), that of decoding W directly (`mse_ptq`), and the
    quantised weights.

    optimizer: "adam" is torch.optim.Adam; "adamw" and "adamw8" are the
    library's fused step (without weight decay, the same update) with moments
    in 32 and 8 bits.  pack: the result also holds `linear`, the trained layer
    packed at k bits a weight (rows must be whole sequences), with its codebook
    in `pack_codebook_dtype` (as it was trained if None; in a 16-bit type,
    several tokens of that type go through the tensor core).  int4_group_size:
    it also holds `mse_int4`, the error of rounding W to 4 bits in groups of
    that many columns."""
    if W.numel() % seq_len:
        raise ValueError("the layer must split into whole sequences")
    if optimizer not in ("adam", "adamw", "adamw8"):
        raise ValueError("optimizer must be adam, adamw or adamw8")
    if pack and W.shape[1] % seq_len:
        raise ValueError("to be packed, the layer's rows must be whole sequences")
    # what would only be refused at the end, with the training lost
    if pack:
        trellis_words(state_bits, k, seq_len)
        check_codebook_dtype(pack_codebook_dtype)
    if int4_group_size is not None:
        _groups(W.shape[1], int4_group_size)
    V = W.detach().clone().requires_grad_(True)
    cb = codebook.detach().clone().requires_grad_(train_codebook)
    params = [V] + ([cb] if train_codebook else [])
    if optimizer == "adam":
        opt = torch.optim.Adam(params, lr=lr)
    else:
        opt = AdamW(params, lr=lr, state_bits=8 if optimizer == "adamw8" else 32)
    history = []
    for T in temperatures:
        for _ in range(steps_per_temperature):
            W_hat = soft_quantize(V.view(-1, seq_len), cb, float(T), state_bits, k).view_as(W)
            loss = _recon_mse(X, W, W_hat)
            opt.zero_grad(set_to_none=True)
            loss.backward()
            opt.step()
            history.append(loss.detach())
    with torch.no_grad():
        _, w_qat = viterbi_decode(V.detach().view(-1, seq_len).contiguous(), cb.detach(), state_bits, k)
        _, w_ptq = viterbi_decode(W.detach().view(-1, seq_len).contiguous(), codebook, state_bits, k)
        w_qat = w_qat.view_as(W)
        w_ptq = w_ptq.view_as(W)
        mse_qat = float(_recon_mse(X, W, w_qat))
        mse_ptq = float(_recon_mse(X, W, w_ptq))
        result = {"history": [float(h) for h in history], "mse_qat": mse_qat, "mse_ptq": mse_ptq,
                  "w_qat": w_qat, "w_ptq": w_ptq, "preimage": V.detach(), "codebook": cb.detach()}
        if pack:
            result["linear"] = TrellisLinear.from_weight(V, cb.detach(), state_bits, k, seq_len, codebook_dtype=pack_codebook_dtype)
        if int4_group_size is not None:
            int4 = Int4Linear.from_weight(W, int4_group_size)
            result["mse_int4"] = float(((X @ W.T - int4(X.contiguous())) ** 2).mean())
    return result
