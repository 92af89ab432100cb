"""AdamW over many tensors at once, behind the gradient buckets.

``GradBuckets`` (ddp.py) leaves averaged bf16 gradients in flat buckets with a
view per parameter; ``AdamW`` takes those views as its gradients, updates fp32
(or bf16) parameters in place and can write a bf16 copy beside them, in one
launch for up to 440 tensors.  Its two moments are held in fp32, or in 8 bits
with a scale per 128 elements (see ``ccl_adamw_step`` in include/ccl.h).

All arithmetic runs in libccl's kernels; this module allocates the states with
torch and counts the steps.
"""
from __future__ import annotations

from typing import Sequence

import torch

from . import ccl

STATE_BLOCK = 128  # elements that share a scale in an 8-bit state


class AdamW:
    """AdamW over params[i] with gradients grads[i].

    params      fp32 or bf16 CUDA tensors, updated in place.
    grads       fp32 or bf16 CUDA tensors, read at every step: the caller
                writes the next gradients into the same tensors.
    state_bits  32 or 8.
    states      the moments to go on from, as ``state_dict()["states"]`` gives
                them; default: zeros.
    copies      bf16 tensors that receive the rounded fp32 parameters.
    step        steps already taken.
    """

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], lr: float = 1e-3,
                 betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, states: dict[str, Sequence[torch.Tensor]] | None = None,
                 copies: Sequence[torch.Tensor] | None = None, step: int = 0):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.steps = step
        params = list(params)
        if states is None:
            kind = torch.float32 if state_bits == 32 else torch.uint8
            states = {name: [torch.zeros(p.numel(), dtype=kind, device=p.device) for p in params]
                      for name in ("exp_avg", "exp_avg_sq")}
            if state_bits == 8:
                states = {name: [v.view(torch.float8_e4m3fn) for v in ts] for name, ts in states.items()}
                states |= {f"{name}_scale": [torch.ones(-(-p.numel() // STATE_BLOCK), device=p.device) for p in params]
                           for name in ("exp_avg", "exp_avg_sq")}
        self.table = ccl.AdamWTable(params, grads, copies=copies, **states)
        if self.table.state_bits != state_bits:
            raise ValueError(f"states are {self.table.state_bits}-bit, state_bits is {state_bits}")

    def step(self, lr: float | None = None, grad_scale: torch.Tensor | None = None, stream=None) -> None:
        """One step on the gradients as they are now; grad_scale (one fp32 number
        on the GPU) multiplies them, so that clipping needs no host wait."""
        ccl.ccl_adamw_step(self.table, self.steps + 1, self.lr if lr is None else lr, self.betas, self.eps,
                           self.weight_decay, grad_scale, stream)
        self.steps += 1

    def moments(self, i: int) -> tuple[torch.Tensor, torch.Tensor]:
        """The values that parameter i's two moments stand for, fp32."""
        t = self.table.tensors
        m, v = t["exp_avg"][i].reshape(-1), t["exp_avg_sq"][i].reshape(-1)
        if self.table.state_bits == 32:
            return m, v

        def value(codes, scales):
            return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(STATE_BLOCK)[:codes.numel()]

        return value(m, t["exp_avg_scale"][i]), value(v, t["exp_avg_sq_scale"][i]).square()

    def state_dict(self) -> dict:
        """Copies of the moments as they are held, and the step count."""
        names = [n for n in self.table.tensors if n.startswith("exp_avg")]
        return {"step": self.steps, "states": {n: [t.clone() for t in self.table.tensors[n]] for n in names}}

    def load_state_dict(self, state: dict) -> None:
        """Takes over moments and step count of an AdamW over tensors of the same sizes."""
        mine = {n: ts for n, ts in self.table.tensors.items() if n.startswith("exp_avg")}
        if set(state["states"]) != set(mine):
            raise ValueError(f"states hold {sorted(state['states'])}, expected {sorted(mine)}")
        # all of it is looked at before any of it is taken
        codes = (torch.float8_e4m3fn, torch.uint8)
        for name, ts in mine.items():
            if [t.numel() for t in ts] != [t.numel() for t in state["states"][name]]:
                raise ValueError(f"{name}: other sizes")
            for i, (to, got) in enumerate(zip(ts, state["states"][name])):
                if got.dtype != to.dtype and not (got.dtype in codes and to.dtype in codes):
                    raise ValueError(f"{name}[{i}] is {got.dtype}, expected {to.dtype}")
        for name, ts in mine.items():
            for to, got in zip(ts, state["states"][name]):
                to.copy_(got.view(to.dtype).reshape(to.shape))
        self.steps = state["step"]
