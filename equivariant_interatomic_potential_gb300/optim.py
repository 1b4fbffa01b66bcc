"""AdamW over libzs: one launch for all tensors of a type, states in 32 or 8 bits."""
from __future__ import annotations

import torch

from . import zs


class AdamW:
    """AdamW (decoupled weight decay, bias correction) over CUDA parameters.

    params: tensors, each contiguous, float32, bfloat16 or float16, on one device;
    every call of ``step`` uses their ``.grad`` (a missing one counts as skipped: the
    parameter and its states stay, and its bias correction counts its own steps).  One
    launch for the parameters of a type that have had as many steps.  state_bits 32
    keeps both moments in float32, 8 as float8_e4m3fn codes with a scale for each 256
    elements (the second one as its root): 2.06 bytes a parameter instead of 8.
    """

    def __init__(self, params, lr: float = 1e-3, betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        self.lr, self.betas, self.eps, self.weight_decay, self.state_bits = lr, betas, eps, weight_decay, state_bits
        self.steps = [0] * len(self.params)   # that each parameter has had
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
        """Plans over the parameters with gradients, one for each type and number of steps; kept while the sets stay."""
        groups: dict[tuple, list[int]] = {}
        for i in live:
            groups.setdefault((self.params[i].dtype, self.steps[i]), []).append(i)
        kept = {tuple(group): plan for group, plan in self._plans}
        at = dict(zip(live, grads))
        self._plans = []
        for group in groups.values():
            new, plan = [at[i] for i in group], kept.get(tuple(group))
            if plan is None:
                scales = [[self.state[i][k] for i in group] for k in ("exp_avg_scale", "exp_avg_sq_scale")] \
                    if self.state_bits == 8 else [None, None]
                plan = zs.AdamWPlan([self.params[i].detach() for i in group], new,
                                    *([self.state[i][k] for i in group] for k in ("exp_avg", "exp_avg_sq")), *scales)
            elif any(p.data_ptr() != self.params[i].data_ptr() for p, i in zip(plan.params, group)):
                raise RuntimeError("a parameter has moved since the optimiser was built")
            elif not plan.has_grads(new):   # by where they are: p.grad.data = other keeps the tensor
                plan.set_grads(new)
            self._plans.append((group, plan))

    @torch.no_grad()
    def step(self, grad_scale: torch.Tensor | None = None) -> None:
        """One step; grad_scale: one float32 element on the device that multiplies every gradient."""
        live = [i for i, p in enumerate(self.params) if p.grad is not None]
        if not live:
            return
        self._plan(live, [self.params[i].grad.contiguous() for i in live])
        for group, plan in self._plans:
            zs.zs_adamw_step(plan, self.steps[group[0]] + 1, lr=self.lr, beta1=self.betas[0], beta2=self.betas[1], eps=self.eps,
                             weight_decay=self.weight_decay, grad_scale=grad_scale)
            for i in group:
                self.steps[i] += 1
            torch.autograd.graph.increment_version([self.params[i] for i in group])

    def zero_grad(self, set_to_none: bool = True) -> None:
        for p in self.params:
            if p.grad is not None:
                p.grad = None if set_to_none else p.grad.zero_()

    def state_dict(self) -> dict:
        return {"steps": list(self.steps), "state_bits": self.state_bits, "state": [{k: v.clone() for k, v in s.items()} for s in self.state]}

    def load_state_dict(self, d: dict) -> None:
        if d["state_bits"] != self.state_bits or len(d["state"]) != len(self.state):
            raise ValueError("the state is of another optimiser: other bits or another number of parameters")
        for mine, theirs in zip(self.state, d["state"]):
            for k, v in mine.items():
                if theirs[k].shape != v.shape:
                    raise ValueError(f"{k} has shape {tuple(theirs[k].shape)}, the parameter needs {tuple(v.shape)}")
                v.copy_(theirs[k])
        steps = d["steps"]   # one number where every parameter has had as many
        self.steps = [steps] * len(self.params) if isinstance(steps, int) else list(steps)
