"""Train a small species-resolved block on top of the zonal scatter.

A seeded graph's radial features and couplings go through the degree-normalised
zonal scatter; the invariants of each degree, times the weights of each atom's
species, pass a block with residual norms and a gate; a readout by species gives
atomic energies.  A student learns the energies of a teacher with other weights,
with AdamW in 32 or 8 bits.

  python examples/species_block.py [--steps 200] [--state-bits 8] [--dtype bf16]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from equivariant_interatomic_potential_gb300 import AdamW, autograd as ops, workloads  # noqa: E402

DEGREES = ((1, 4), (4, 9), (9, 16))   # node rows of degrees 1, 2 and 3
SPECIES, WIDTH = 5, 64


class Block(torch.nn.Module):
    """Invariants (N, 96) -> atomic energies (N,), weights by species."""

    def __init__(self, features: int, dtype: torch.dtype, seed: int):
        super().__init__()
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weights(rows, cols):
            w = torch.randn(SPECIES, rows, cols, generator=gen, device="cuda") * cols ** -0.5
            return torch.nn.Parameter(w.to(dtype))

        def vector(value):
            return torch.nn.Parameter(torch.full((WIDTH,), value, device="cuda"))

        self.embed, self.inner, self.gate = weights(WIDTH, features), weights(WIDTH, WIDTH), weights(WIDTH, WIDTH)
        self.readout = weights(1, WIDTH)
        self.norms = torch.nn.ParameterList(vector(v) for v in (1.0, 0.5, 1.0) * 2)

    def forward(self, invariants, row_ptr, perm):
        linear = lambda x, w: ops.grouped_matmul(x, w, row_ptr, perm)  # noqa: E731
        x = linear(invariants, self.embed)
        y, u, _ = ops.norm_gate_residual(x, torch.zeros_like(x), None, *self.norms[:3])
        _, u, _ = ops.norm_gate_residual(linear(u, self.inner), y, linear(u, self.gate), *self.norms[3:])
        return linear(u, self.readout)[:, 0].float()


def train(steps: int = 100, state_bits: int = 32, dtype: torch.dtype = torch.float32, nodes: int = 1000,
          edges: int = 30000) -> list[float]:
    """The student's mean squared error at each step."""
    w = workloads.make_random(nodes, edges, 32, seed=11)
    coup, rad, dst = (torch.from_numpy(a).cuda() for a in (w.coup, w.rad, w.dst))
    degree = torch.bincount(dst, minlength=nodes).clamp_min(1)
    out = ops.degree_normalised_scatter(coup, rad, dst, degree.rsqrt(), nodes)
    invariants = torch.cat([out[:, a:b].square().mean(1) for a, b in DEGREES], 1).to(dtype)
    species = torch.randint(0, SPECIES, (nodes,), generator=torch.Generator().manual_seed(2)).int().cuda()
    row_ptr, perm = ops.build_csr(species, SPECIES)
    with torch.no_grad():
        target = Block(invariants.shape[1], dtype, seed=1)(invariants, row_ptr, perm)
    model = Block(invariants.shape[1], dtype, seed=3)
    opt = AdamW(model.parameters(), lr=3e-3, weight_decay=0.0, state_bits=state_bits)
    losses = []
    for _ in range(steps):
        loss = (model(invariants, row_ptr, perm) - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    losses = train(a.steps, a.state_bits, torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:5d}  mean squared error {losses[i]:.5f}")
    print(f"step {a.steps - 1:5d}  mean squared error {losses[-1]:.5f}")


if __name__ == "__main__":
    main()
