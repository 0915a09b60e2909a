"""AdamW over named tensors: states, masters and the step (moe_adamw_step).

What learns beside a layer of quantized experts is small and many: the router,
the shared expert, norms, adapters.  One step is one launch for the fp32 tensors
and one for the bf16 ones; its count lives on the device, so a captured graph
goes on counting.
"""
from __future__ import annotations

from typing import Dict, Optional, Union

import torch

from . import binding as B
from ._lib import ADAMW_BLOCK


class AdamW:
    """AdamW with fp32 or 8-bit states over a dict of fp32 and bf16 tensors.

    ``params`` are dense CUDA tensors of one device, updated in place; bf16 ones
    get fp32 masters unless ``masters`` is False (updates below half a bf16 step
    are then lost).  ``lr`` is a number or an fp32 tensor of one element on the
    device (which a captured graph reads anew); ``weight_decay`` a number or a
    dict by name (names it lacks: 0).  ``state_bits`` 32 or 8: int8 and uint8
    codes with a scale per ADAMW_BLOCK elements."""

    def __init__(self, params: Dict[str, torch.Tensor], lr: Union[float, torch.Tensor] = 1e-3,
                 betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: Union[float, Dict[str, float]] = 0.0, state_bits: int = 32,
                 masters: bool = True):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if not params:
            raise ValueError("no tensors to optimize")
        if isinstance(weight_decay, dict) and not set(weight_decay) <= set(params):
            raise ValueError(f"weight_decay names no tensor: {sorted(set(weight_decay) - set(params))}")
        self.lr, self.betas, self.eps, self.state_bits = lr, tuple(betas), float(eps), state_bits
        self._groups = []
        for dtype in (torch.float32, torch.bfloat16):
            names = [n for n, p in params.items() if p.dtype == dtype]
            if not names:
                continue
            ps = [params[n] for n in names]
            dev = ps[0].device
            g = dict(names=names, params=ps, masters=None, exp_avg_scales=None,
                     exp_avg_sq_scales=None,
                     step=torch.zeros(2, dtype=torch.int32, device=dev),
                     decay=[float(weight_decay.get(n, 0.0) if isinstance(weight_decay, dict)
                                  else weight_decay) for n in names])
            if dtype == torch.bfloat16 and masters:
                g["masters"] = [p.float() for p in ps]
            kinds = (torch.float32,) * 2 if state_bits == 32 else (torch.int8, torch.uint8)
            for key, kind in zip(("exp_avg", "exp_avg_sq"), kinds):
                g[key] = [torch.zeros(p.shape, dtype=kind, device=dev) for p in ps]
                if state_bits == 8:
                    g[key + "_scales"] = [torch.zeros(-(-p.numel() // ADAMW_BLOCK), device=dev)
                                          for p in ps]
            self._groups.append(g)
        known = sum(len(g["names"]) for g in self._groups)
        if known != len(params):
            raise ValueError("tensors must be float32 or bfloat16")

    def step(self, grads: Dict[str, torch.Tensor], grad_scale: Optional[torch.Tensor] = None,
             stream=None) -> None:
        """One step with the gradients by name (all of a type's tensors fp32 or all
        bf16).  grad_scale (fp32, one element on the device) multiplies them; one
        that is not finite skips the step.  Gradients that are refused leave every
        tensor as it was."""
        names = {n for g in self._groups for n in g["names"]}
        if set(grads) != names:
            raise ValueError(f"gradients must be those of {sorted(names)}, got {sorted(grads)}")
        lists = [[grads[n] for n in g["names"]] for g in self._groups]
        for g, gs in zip(self._groups[1:], lists[1:]):  # a later launch is not refused behind an earlier one
            B.native().adamw_check(g["params"], gs)
        for g, gs in zip(self._groups, lists):
            B.moe_adamw_step(
                g["params"], gs, g["exp_avg"], g["exp_avg_sq"],
                g["step"], self.lr, self.betas[0], self.betas[1], self.eps, g["decay"],
                g["masters"], g["exp_avg_scales"], g["exp_avg_sq_scales"], grad_scale, stream)

    def state_dict(self) -> dict:
        """The states by name, masters among them, and the steps done (references,
        not copies)."""
        out = {}
        for g in self._groups:
            for i, n in enumerate(g["names"]):
                out[n] = {k: g[k][i] for k in ("exp_avg", "exp_avg_sq", "exp_avg_scales",
                                               "exp_avg_sq_scales", "masters") if g[k] is not None}
                out[n]["step"] = g["step"]
        return out

    def load_state_dict(self, state: dict) -> None:
        """Copy states of state_dict() of the same tensors, types and bits into
        place, and masters to their tensors."""
        mine = self.state_dict()
        if {n: sorted(s) for n, s in state.items()} != {n: sorted(s) for n, s in mine.items()}:
            raise ValueError("the states belong to other tensors or another kind of state")
        for n, s in mine.items():
            for k, t in s.items():
                if state[n][k].shape != t.shape or state[n][k].dtype != t.dtype:
                    raise ValueError(f"{k} of {n} does not fit")
        for n, s in mine.items():
            for k, t in s.items():
                t.copy_(state[n][k])
        for g in self._groups:
            for p, m in zip(g["params"], g["masters"] or ()):
                p.copy_(m)
