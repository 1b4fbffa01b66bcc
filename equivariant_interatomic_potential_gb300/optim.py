"""AdamW over libzs: one launch for the tensors of a type, states in 32 or 8 bits."""
from __future__ import annotations

from itertools import chain

import torch

from . import zs

_HYPER = ("lr", "betas", "eps", "weight_decay")


def _of_groups(name: str) -> property:
    """A hyper-parameter of the first group; setting it sets every group's."""
    def put(self, value):
        for group in self.param_groups:
            group[name] = value

    return property(lambda self: self.param_groups[0][name], put)


class AdamW(torch.optim.Optimizer):
    """AdamW (decoupled weight decay, bias correction) over CUDA parameters.

    params: tensors, or groups of them with options of their own, each contiguous,
    float32, bfloat16 or float16, on one device; every call of ``step`` uses their
    ``.grad`` (a missing one counts as skipped: the parameter and its states stay, and
    its bias correction counts its own steps).  One launch for the parameters of a type
    that share their options and have had as many steps.  state_bits 32 keeps both
    moments in float32, 8 as float8_e4m3fn codes with a scale for each 256 elements (the
    second one as its root): 2.06 bytes a parameter instead of 8.
    """

    def __init__(self, params, lr: float = 1e-3, betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, seed: int = 0):
        params = list(params)
        if not params:
            raise ValueError("AdamW needs at least one parameter")
        self._plans: dict[tuple, zs.AdamWPlan] = {}
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits, seed=seed))

    lr, betas, eps, weight_decay = map(_of_groups, _HYPER)

    def __setstate__(self, state):
        super().__setstate__(state)
        self._plans = {}

    def add_param_group(self, param_group: dict) -> None:
        bits = param_group.get("state_bits", self.defaults["state_bits"])
        if bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {bits}")
        super().add_param_group(param_group)
        params = self.param_groups[-1]["params"]
        if len(set(params)) != len(params):
            self.param_groups.pop()
            raise ValueError("a parameter is given twice")
        dtype = torch.float32 if bits == 32 else torch.float8_e4m3fn
        for p in params:
            s = self.state[p]
            s["step"] = 0
            for k in ("exp_avg", "exp_avg_sq"):
                s[k] = torch.zeros(p.shape, dtype=torch.float32, device=p.device).to(dtype)
                if bits == 8:
                    s[k + "_scale"] = torch.zeros(-(-p.numel() // zs.ADAMW_BLOCK), device=p.device)

    def _plan(self, params: list[torch.Tensor], states: list[dict], grads: list[torch.Tensor], bits: int) -> zs.AdamWPlan:
        """The plan over these tensors; kept from the last step where they are the same."""
        plan = self._plans.get(tuple(map(id, params)))
        if plan is None or any(s["exp_avg"] is not m or s["exp_avg_sq"] is not v
                               for s, m, v in zip(states, plan.exp_avg, plan.exp_avg_sq)):
            names = ("exp_avg", "exp_avg_sq") + (("exp_avg_scale", "exp_avg_sq_scale") if bits == 8 else ())
            return zs.AdamWPlan([p.detach() for p in params], grads, *([s[k] for s in states] for k in names))
        if not plan.has_params(params):
            raise RuntimeError("a parameter has moved since the optimiser was built")
        if not plan.has_grads(grads):   # by where they are: p.grad.data = other keeps the tensor
            plan.set_grads(grads)
        return plan

    @torch.no_grad()
    def step(self, closure=None, grad_scale: torch.Tensor | None = None):
        """One step.  closure: evaluates the loss again, which is returned.  grad_scale: one
        float32 element on the device that multiplies every gradient (also taken in the
        closure's place).  Not while a graph is captured: the step's number, rates and
        addresses would be those of the capture in every replay."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("an optimiser step cannot be captured: its number, rates and addresses would stay those of the capture")
        loss = None
        if isinstance(closure, torch.Tensor):
            closure, grad_scale = None, closure
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # parameters, states and gradients of each set of options, type and number of steps
        alike: dict[tuple, tuple[list, list, list]] = {}
        for group in self.param_groups:
            options = (float(group["lr"]), *map(float, group["betas"]), group["eps"], group["weight_decay"],
                       group["state_bits"], group["seed"])
            last = into = None
            for p in group["params"]:
                g = p.grad
                if g is None:
                    continue
                s = self.state[p]
                kind = (p.dtype, s["step"])
                if kind != last:
                    last, into = kind, alike.setdefault((options, *kind), ([], [], []))
                into[0].append(p)
                into[1].append(s)
                into[2].append(g if g.is_contiguous() else g.contiguous())
        plans = {tuple(map(id, params)): self._plan(params, states, grads, options[5])
                 for (options, _, _), (params, states, grads) in alike.items()}   # what is refused is, before any launch
        self._plans = plans
        for i, (((lr, beta1, beta2, eps, decay, _, seed), _, steps), (params, states, _)) in enumerate(alike.items()):
            zs.zs_adamw_step(plans[tuple(map(id, params))], steps + 1, lr=lr, beta1=beta1, beta2=beta2, eps=eps,
                             weight_decay=decay, grad_scale=grad_scale, seed=seed + i)   # each launch has random bits of its own
            for s in states:
                s["step"] = steps + 1
            torch.autograd.graph.increment_version(params)
        return loss

    def state_dict(self) -> dict:
        """The base class's form, with copies of the states: later steps leave it as it is."""
        d = super().state_dict()
        d["state"] = {i: {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.items()} for i, s in d["state"].items()}
        return d

    def load_state_dict(self, state_dict: dict) -> None:
        d = dict(state_dict)
        mine, params = self.state, list(chain.from_iterable(g["params"] for g in self.param_groups))
        if "steps" in d:   # the form without groups
            steps = d["steps"] if isinstance(d["steps"], list) else [d["steps"]] * len(d["state"])
            if len(steps) != len(params):
                raise ValueError(f"the state is of {len(steps)} parameters, the optimiser of {len(params)}")
            groups = super().state_dict()["param_groups"]
            for g in groups:
                g["state_bits"] = d["state_bits"]
            d = {"state": {i: {**s, "step": n} for i, (s, n) in enumerate(zip(d["state"], steps))}, "param_groups": groups}
        bits = [(g["state_bits"], h.get("state_bits", 32)) for g, h in zip(self.param_groups, d["param_groups"])]
        if any(a != b for a, b in bits):
            raise ValueError("the state is of an optimiser with other state_bits")
        theirs = [d["state"].get(i, {}) for i in chain.from_iterable(g["params"] for g in d["param_groups"])]
        for p, s in zip(params, theirs):
            for k, v in mine[p].items():
                if s and k != "step" and s[k].shape != v.shape:
                    raise ValueError(f"{k} has shape {tuple(s[k].shape)}, the parameter needs {tuple(v.shape)}")
        # the groups are the base class's to check and take over; it would cast the states to the parameters' types
        super().load_state_dict({**d, "state": {}, "param_groups": [{"state_bits": 32, "seed": 0, **g} for g in d["param_groups"]]})
        self.state = mine
        for p, s in zip(params, theirs):
            for k, v in mine[p].items():
                if k == "step":
                    mine[p][k] = int(s.get(k, 0))
                else:
                    v.copy_(s[k]) if s else v.zero_()
