"""AdamW over libzs: one launch for all tensors of a type, states in 32 or 8 bits."""
from __future__ import annotations

import torch

from . import zs


class AdamW:
    """AdamW (decoupled weight decay, bias correction) over CUDA parameters.

    params: tensors, each contiguous, float32, bfloat16 or float16, on one device;
    every call of ``step`` uses their ``.grad`` (a missing one counts as skipped:
    the parameter and its states stay).  state_bits 32 keeps both moments in
    float32, 8 as float8_e4m3fn codes with a scale for each 256 elements (the
    second one as its root): 2.06 bytes a parameter instead of 8.
    """

    def __init__(self, params, lr: float = 1e-3, betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        self.lr, self.betas, self.eps, self.weight_decay, self.state_bits = lr, betas, eps, weight_decay, state_bits
        self.steps = 0
        dtype = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        self.state = []
        for p in self.params:
            s = {k: torch.zeros(p.shape, dtype=torch.float32, device=p.device).to(dtype) for k in ("exp_avg", "exp_avg_sq")}
            if state_bits == 8:
                blocks = -(-p.numel() // zs.ADAMW_BLOCK)
                s |= {k: torch.zeros(blocks, device=p.device) for k in ("exp_avg_scale", "exp_avg_sq_scale")}
            self.state.append(s)
        self._plans: list[tuple[list[int], zs.AdamWPlan]] = []

    def _plan(self, live: list[int], grads: list[torch.Tensor]):
        """Plans over the parameters with gradients, one for each type; kept while the set stays."""
        if [i for group, _ in self._plans for i in group] != live:
            self._plans = []
            for dtype in dict.fromkeys(self.params[i].dtype for i in live):
                group = [i for i in live if self.params[i].dtype == dtype]
                scales = [[self.state[i][k] for i in group] for k in ("exp_avg_scale", "exp_avg_sq_scale")] \
                    if self.state_bits == 8 else [None, None]
                self._plans.append((group, zs.AdamWPlan([self.params[i].detach() for i in group],
                                                        [grads[live.index(i)] for i in group],
                                                        *([self.state[i][k] for i in group] for k in ("exp_avg", "exp_avg_sq")),
                                                        *scales)))
            return
        at = dict(zip(live, grads))
        for group, plan in self._plans:
            new = [at[i] for i in group]
            if any(p.data_ptr() != self.params[i].data_ptr() for p, i in zip(plan.params, group)):
                raise RuntimeError("a parameter has moved since the optimiser was built")
            if not plan.has_grads(new):   # by where they are: p.grad.data = other keeps the tensor
                plan.set_grads(new)

    @torch.no_grad()
    def step(self, grad_scale: torch.Tensor | None = None) -> None:
        """One step; grad_scale: one float32 element on the device that multiplies every gradient."""
        order = sorted(range(len(self.params)), key=lambda i: str(self.params[i].dtype))
        live = [i for i in order if self.params[i].grad is not None]
        if not live:
            return
        self._plan(live, [self.params[i].grad.contiguous() for i in live])
        self.steps += 1
        for group, plan in self._plans:
            zs.zs_adamw_step(plan, self.steps, lr=self.lr, beta1=self.betas[0], beta2=self.betas[1], eps=self.eps,
                             weight_decay=self.weight_decay, grad_scale=grad_scale)
            torch.autograd.graph.increment_version([self.params[i] for i in group])

    def zero_grad(self, set_to_none: bool = True) -> None:
        for p in self.params:
            if p.grad is not None:
                p.grad = None if set_to_none else p.grad.zero_()

    def state_dict(self) -> dict:
        return {"steps": self.steps, "state_bits": self.state_bits, "state": [{k: v.clone() for k, v in s.items()} for s in self.state]}

    def load_state_dict(self, d: dict) -> None:
        if d["state_bits"] != self.state_bits or len(d["state"]) != len(self.state):
            raise ValueError("the state is of another optimiser: other bits or another number of parameters")
        for mine, theirs in zip(self.state, d["state"]):
            for k, v in mine.items():
                if theirs[k].shape != v.shape:
                    raise ValueError(f"{k} has shape {tuple(theirs[k].shape)}, the parameter needs {tuple(v.shape)}")
                v.copy_(theirs[k])
        self.steps = d["steps"]
