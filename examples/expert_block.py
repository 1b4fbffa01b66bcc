"""Train a small block whose atoms choose their own weights.

Where species_block.py multiplies an atom's features by the weights of its species, here
a router picks a few experts for each atom.  A seeded graph's invariants from the zonal
scatter are added to an embedding of the species; residual norms go around a layer of
experts and dropout; a readout by species gives atomic energies.  A student learns the
energies of a teacher with other weights, with AdamW in 32 or 8 bits.

  python examples/expert_block.py [--steps 200] [--state-bits 8] [--dtype bf16]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from equivariant_interatomic_potential_gb300 import AdamW, autograd as ops, workloads  # noqa: E402

DEGREES = ((1, 4), (4, 9), (9, 16))   # node rows of degrees 1, 2 and 3
SPECIES, WIDTH, HIDDEN = 5, 64, 96
EXPERTS, CHOICES, GROUPS, OPEN_GROUPS = 16, 2, 4, 2
DROPOUT, SEED = 0.05, 2024


class Block(torch.nn.Module):
    """Invariants (N, 96) and species (N,) -> atomic energies (N,)."""

    def __init__(self, features: int, dtype: torch.dtype, seed: int):
        super().__init__()
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape):
            w = torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5
            return torch.nn.Parameter(w.to(dtype))

        def vector(value):
            return torch.nn.Parameter(torch.full((WIDTH,), value, device="cuda"))

        self.species, self.inner = weights(SPECIES, WIDTH), weights(SPECIES, WIDTH, features)
        self.router = weights(1, EXPERTS, WIDTH)
        self.w_in, self.w_out = weights(EXPERTS, HIDDEN, WIDTH), weights(EXPERTS, WIDTH, HIDDEN)
        self.readout = weights(SPECIES, 1, WIDTH)
        self.norms = torch.nn.ParameterList(vector(v) for v in (1.0, 0.5, 1.0) * 2)
        self.register_buffer("balance", torch.zeros(EXPERTS, device="cuda"))

    def forward(self, invariants, species, row_ptr, perm, all_rows, step=None):
        """``step``: one int64 element on the device that counts the steps; None: no dropout."""
        x = ops.grouped_matmul(invariants, self.inner, row_ptr, perm)
        y, u, _ = ops.norm_gate_residual(x, ops.species_embedding(species, self.species, WIDTH ** 0.5), None, *self.norms[:3])
        logits = ops.grouped_matmul(u, self.router, all_rows)
        h = ops.expert_block(u, logits, self.w_in, self.w_out, CHOICES, self.balance, "sigmoid", GROUPS, OPEN_GROUPS, group_top=2)
        if step is not None:
            h = ops.dropout(h, DROPOUT, SEED, call=0, step_at=step)
        _, u, _ = ops.norm_gate_residual(h, y, None, *self.norms[3:])
        return ops.grouped_matmul(u, self.readout, row_ptr, perm)[:, 0].float()


def data(nodes: int, edges: int, dtype: torch.dtype):
    """A seeded graph's invariants, its species, their CSR, and the CSR of one group of all rows."""
    w = workloads.make_random(nodes, edges, 32, seed=11)
    coup, rad, dst = (torch.from_numpy(a).cuda() for a in (w.coup, w.rad, w.dst))
    degree = torch.bincount(dst, minlength=nodes).clamp_min(1)
    out = ops.degree_normalised_scatter(coup, rad, dst, degree.rsqrt(), nodes)
    invariants = torch.cat([out[:, a:b].square().mean(1) for a, b in DEGREES], 1).to(dtype)
    species = torch.randint(0, SPECIES, (nodes,), generator=torch.Generator().manual_seed(2)).int().cuda()
    all_rows = torch.tensor([0, nodes], dtype=torch.int32, device="cuda")
    return invariants, species, *ops.build_csr(species, SPECIES), all_rows


def train(steps: int = 100, state_bits: int = 32, dtype: torch.dtype = torch.float32, nodes: int = 1000,
          edges: int = 30000) -> list[float]:
    """The student's mean squared error at each step."""
    given = data(nodes, edges, dtype)
    with torch.no_grad():
        target = Block(given[0].shape[1], dtype, seed=1)(*given)
    model = Block(given[0].shape[1], dtype, seed=3)
    opt = AdamW(model.parameters(), lr=3e-3, weight_decay=0.0, state_bits=state_bits)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    losses = []
    for _ in range(steps):
        loss = (model(*given, step) - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        step += 1
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
