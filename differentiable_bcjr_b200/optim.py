"""AdamW over the library's fused step (`adamw_step`), for the preimages and
codebooks of quantisation-aware training or any other float parameters.

One launch updates every parameter of a device and type; the moments are kept
in 32 bits, or in 8 bits with a scale for every 256 of them.
"""
from __future__ import annotations

import torch

from . import adamw_state
from .layer import _adamw_check, _adamw_plan, _adamw_run


class AdamW:
    """AdamW (decoupled weight decay) with its moments in `state_bits` = 32 or 8 bits.

        opt = AdamW([preimage, codebook], lr=0.02, state_bits=8)
        loss.backward(); opt.step(); opt.zero_grad()

    `params` is an iterable of tensors, or of dicts with "params" and any of
    lr, betas, eps and weight_decay; `param_groups` holds those dicts, and a
    step uses what they hold then.  Parameters must be contiguous CUDA tensors
    of float32, float16 or bfloat16.  Parameters without a gradient are left
    as they are; the step count is one for all parameters of a group with the
    same device and type.  `seed` is that of the 8-bit states' rounding.
    With `capturable` the count lives on the GPU, so that `step` can be
    captured into a CUDA graph (whose replays keep the hyperparameters that
    were captured).
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=32, seed=0,
                 capturable=False):
        params = list(params)
        if not params:
            raise ValueError("there are no parameters")
        groups = params if isinstance(params[0], dict) else [{"params": params}]
        self.state_bits, self.seed, self.capturable = state_bits, int(seed), bool(capturable)
        self.param_groups = []
        self._buckets = []  # of each group: {"params", "state", "step"} for each device and type
        seen = set()
        for g in groups:
            tensors = [g["params"]] if isinstance(g["params"], torch.Tensor) else list(g["params"])
            self.param_groups.append({"params": tensors, "lr": g.get("lr", lr), "betas": tuple(g.get("betas", betas)),
                                      "eps": g.get("eps", eps), "weight_decay": g.get("weight_decay", weight_decay)})
            buckets = {}
            for t in tensors:
                if id(t) in seen:
                    raise ValueError("a parameter appears twice")
                seen.add(id(t))
                if not t.is_cuda or not t.is_contiguous() or t.dtype not in (torch.float32, torch.float16, torch.bfloat16):
                    raise ValueError("parameters must be contiguous CUDA tensors of float32, float16 or bfloat16")
                buckets.setdefault((t.device, t.dtype), []).append(t)
            for ts in buckets.values():
                spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in ts if t.numel())
                if any(end > start for (_, end), (start, _) in zip(spans, spans[1:])):
                    raise ValueError("parameters must not overlap")
            self._buckets.append([{"params": ts, "state": adamw_state(ts, state_bits),
                                   "step": torch.zeros(1, dtype=torch.int64, device=d) if capturable else 0}
                                  for (d, _), ts in buckets.items()])

    @torch.no_grad()
    def step(self, grad_scale=None):
        """One step; `grad_scale` (a float32 CUDA tensor of one element) multiplies every gradient.
        All groups are checked before the first launch, so that a step which is refused changes nothing."""
        todo = []
        for group, buckets in zip(self.param_groups, self._buckets):
            for b in buckets:
                grads = [p.grad for p in b["params"]]
                kinds = {g.dtype for g in grads if g is not None}
                if not kinds:
                    continue
                step = b["step"] if self.capturable else b["step"] + 1
                first, second, scales = b["state"]
                plans = []
                for kind in sorted(kinds, key=str):
                    own = grads if len(kinds) == 1 else [g if g is not None and g.dtype == kind else None for g in grads]
                    own = [g if g is None or g.is_contiguous() else g.contiguous() for g in own]
                    # (the plan holds addresses, so `own` is kept until the launch)
                    plans.append((_adamw_plan(b["params"], own, first, second, step, group["lr"], group["betas"], group["eps"],
                                              group["weight_decay"], scales, grad_scale, self.seed), own))
                todo.append((b, plans))
        if sum(len(plans) for _, plans in todo) > 1:  # (one launch is refused as a whole anyway)
            for _, plans in todo:
                for plan, _ in plans:
                    _adamw_check(plan)
        for b, plans in todo:
            if self.capturable:
                b["step"].add_(1)
            try:
                for plan, _ in plans:
                    _adamw_run(plan)
            except Exception:
                if self.capturable:
                    b["step"].sub_(1)
                raise
            if not self.capturable:
                b["step"] += 1

    def zero_grad(self, set_to_none=True):
        for group in self.param_groups:
            for p in group["params"]:
                if set_to_none:
                    p.grad = None
                elif p.grad is not None:
                    p.grad.zero_()

    def state_dict(self):
        """Hyperparameters and states (the states' own tensors, not copies)."""
        return {"state_bits": self.state_bits, "seed": self.seed,
                "groups": [{k: v for k, v in g.items() if k != "params"} for g in self.param_groups],
                "states": [[{"state": b["state"], "step": b["step"]} for b in buckets] for buckets in self._buckets]}

    def load_state_dict(self, saved):
        """Takes over what `state_dict` gave for parameters of the same shapes, types and order (copied)."""
        if saved["state_bits"] != self.state_bits:
            raise ValueError(f"the states have {saved['state_bits']} bits, not {self.state_bits}")
        shape = [[[None if t is None else (t.shape, t.dtype) for t in b["state"]] for b in buckets] for buckets in self._buckets]
        if shape != [[[None if t is None else (t.shape, t.dtype) for t in b["state"]] for b in buckets] for buckets in saved["states"]]:
            raise ValueError("the states are those of other parameters")
        self.seed = saved["seed"]
        for group, g in zip(self.param_groups, saved["groups"]):
            group.update(g)
        for buckets, others in zip(self._buckets, saved["states"]):
            for b, o in zip(buckets, others):
                for mine, theirs in zip(b["state"], o["state"]):
                    if mine is not None:
                        mine.view(torch.uint8).copy_(theirs.view(torch.uint8))
                if self.capturable:
                    b["step"].fill_(int(o["step"]))
                else:
                    b["step"] = int(o["step"])
