"""The training operators as a user has them: torch.library operators with
autograd, the optimiser, and the example that runs them together."""
import importlib.util
import os

import numpy as np
import pytest
import torch
from torch.fx.experimental.proxy_tensor import make_fx

from equivariant_interatomic_potential_gb300 import AdamW, autograd as ag, zs
from train_refs import csr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_operators_registered():
    for name in ("grouped_matmul", "grouped_matmul_backward", "grouped_matmul_dx", "norm_gate_residual",
                 "norm_gate_residual_backward"):
        assert hasattr(torch.ops.zs_gie, name)


def test_cpu_tensors_rejected():
    with pytest.raises(ValueError, match="CUDA tensors only"):
        ag.grouped_matmul(torch.zeros(3, 4), torch.zeros(2, 5, 4), torch.zeros(3, dtype=torch.int32))
    h, w = torch.zeros(3, 4), torch.ones(4)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        ag.norm_gate_residual(h, h, None, w, w, w)
    with pytest.raises(ValueError, match="state_bits"):
        AdamW([torch.zeros(3)], state_bits=16)
    with pytest.raises(ValueError, match="at least one"):
        AdamW([])


def test_fake_tracing():
    # traced with fake tensors: the fake implementations give every shape, no kernel runs
    def f(x, w, species, gate, vec, g):
        y = ag.species_linear(x, w, species)
        y, u, _ = ag.norm_gate_residual(y, x, gate, vec, vec, vec)
        return torch.autograd.grad(u + y, (x, w, gate, vec), g)

    M, C, G = 7, 8, 3
    x, w = torch.randn(M, C, requires_grad=True), torch.randn(G, C, C, requires_grad=True)
    gate, vec = torch.randn(M, 1, requires_grad=True), torch.ones(C, requires_grad=True)
    gm = make_fx(f, tracing_mode="fake")(x, w, torch.zeros(M, dtype=torch.int32), gate, vec, torch.randn(M, C))
    outs = [n for n in gm.graph.nodes if n.op == "output"][0].args[0]
    assert [tuple(o.meta["val"].shape) for o in outs] == [(M, C), (G, C, C), (M, 1), (C,)]


@pytest.mark.gpu
@pytest.mark.parametrize("needs", [(True, True), (True, False), (False, True)])
def test_grouped_autograd(needs):
    rng = np.random.default_rng(3)
    group = rng.integers(0, 4, 300)
    species = torch.from_numpy(group.astype(np.int32)).cuda()
    x, w = torch.randn(300, 48, device="cuda"), torch.randn(4, 40, 48, device="cuda")
    dy = torch.randn(300, 40, device="cuda")
    xr, wr = x.clone().requires_grad_(needs[0]), w.clone().requires_grad_(needs[1])
    y = ag.species_linear(xr, wr, species)
    y.backward(dy)
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group, 4))
    assert torch.equal(y, zs.zs_grouped_matmul(x, w, row_ptr, perm))
    dx, dw = zs.zs_grouped_matmul_backward(dy, x, w, row_ptr, perm)
    assert torch.equal(xr.grad, dx) if needs[0] else xr.grad is None
    assert torch.equal(wr.grad, dw) if needs[1] else wr.grad is None


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["full", "row", "none"])
def test_norm_autograd(gate):
    M, C = 200, 96
    gen = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ops = [rnd(M, C), rnd(M, C), {"full": rnd(M, C), "row": rnd(M, 1), "none": None}[gate], rnd(C), rnd(C), rnd(C)]
    leaves = [None if t is None else t.clone().requires_grad_() for t in ops]
    dy, du = rnd(M, C), rnd(M, C)
    y, u, _ = ag.norm_gate_residual(*leaves, kind="layer")
    torch.autograd.backward((y, u), (dy, du))
    yy, uu, stats = zs.zs_norm_gate_residual(*ops, kind="layer")
    assert torch.equal(y, yy) and torch.equal(u, uu)
    for leaf, g in zip(leaves, zs.zs_norm_gate_residual_backward(dy, du, *ops, stats, kind="layer")):
        assert (leaf is None) == (g is None) and (g is None or torch.equal(leaf.grad, g))


@pytest.mark.gpu
def test_optimiser_against_torch():
    # fp32 rounding of a few operations a step: 1e-6 of the parameters' size after five
    gen = torch.Generator(device="cuda").manual_seed(5)
    shapes = [(300, 7), (64,), (5, 5, 5)]
    mine = [torch.randn(s, generator=gen, device="cuda").requires_grad_() for s in shapes]
    theirs = [p.detach().clone().requires_grad_() for p in mine]
    a = AdamW(mine, lr=1e-2, weight_decay=0.1)
    b = torch.optim.AdamW(theirs, lr=1e-2, weight_decay=0.1)
    for _ in range(5):
        for p, q in zip(mine, theirs):
            p.grad = torch.randn(p.shape, generator=gen, device="cuda")
            q.grad = p.grad.clone()
        before = mine[0]._version
        a.step()
        b.step()
        assert mine[0]._version > before          # autograd sees the change
    for p, q in zip(mine, theirs):
        assert float((p - q).abs().max()) <= 1e-6 * float(q.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_optimiser_state_and_missing_gradients(bits):
    gen = torch.Generator(device="cuda").manual_seed(6)
    make = lambda: [torch.full((700,), 1.0, device="cuda"), torch.full((33,), 1.0, device="cuda", dtype=torch.bfloat16)]  # noqa: E731
    one, two = make(), make()
    a, b = AdamW(one, state_bits=bits), AdamW(two, state_bits=bits)
    grads = [[torch.randn(p.shape, generator=gen, device="cuda").to(p.dtype) for p in one] for _ in range(4)]

    def run(opt, params, which):
        for i in which:
            for p, g in zip(params, grads[i]):
                p.grad = g
            opt.step()

    run(a, one, (0, 1))
    two[0].copy_(one[0])
    two[1].copy_(one[1])
    b.load_state_dict(a.state_dict())
    run(a, one, (2, 3))
    run(b, two, (2, 3))
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    kept = one[1].clone()
    one[1].grad = None
    a.step()
    assert torch.equal(one[1], kept) and not torch.equal(one[0], two[0])
    a.zero_grad()
    assert all(p.grad is None for p in one)
    with pytest.raises(ValueError):
        a.load_state_dict(AdamW(make()[:1], state_bits=bits).state_dict())


@pytest.mark.gpu
@pytest.mark.parametrize("missing", [lambda t, i: i == 1 and t < 30, lambda t, i: (t + i) % 3 == 0,
                                     lambda t, i: i > 0 and t % 7 != i], ids=["late", "in_turn", "seldom"])
def test_optimiser_skipped_steps_against_torch(missing):
    # a parameter that misses steps has the bias correction of its own steps; tolerance as above, for 40 steps
    gen = torch.Generator(device="cuda").manual_seed(7)
    shapes = [(300, 7), (64,), (1000,)]
    mine = [torch.randn(s, generator=gen, device="cuda") for s in shapes]
    theirs = [p.clone().requires_grad_() for p in mine]
    a = AdamW(mine, lr=1e-2, weight_decay=0.1)
    b = torch.optim.AdamW(theirs, lr=1e-2, weight_decay=0.1)
    for t in range(40):
        for i, (p, q) in enumerate(zip(mine, theirs)):
            g = torch.randn(p.shape, generator=gen, device="cuda")
            p.grad, q.grad = (None, None) if missing(t, i) else (g, g.clone())
        if t == 25:    # the counts travel with the state
            state = a.state_dict()
            a = AdamW(mine, lr=1e-2, weight_decay=0.1)
            a.load_state_dict(state)
        a.step()
        b.step()
        for p, q in zip(mine, theirs):
            assert float((p - q.detach()).abs().max()) <= 4e-6 * float(q.detach().abs().max()), t


def spoil(n):
    """Takes freed blocks of n floats and overwrites them."""
    return [torch.full((n,), 3.0, device="cuda") for _ in range(8)]


@pytest.mark.gpu
def test_optimiser_gradient_memory_replaced():
    # p.grad stays the same tensor while its memory is another (p.grad.data = clipped): each step reads the present one
    gen = torch.Generator(device="cuda").manual_seed(12)
    rnd = lambda: torch.randn(5000, generator=gen, device="cuda")  # noqa: E731
    p, q = torch.ones(5000, device="cuda"), torch.ones(5000, device="cuda").requires_grad_()
    a, b = AdamW([p], lr=1e-2, weight_decay=0.1), torch.optim.AdamW([q], lr=1e-2, weight_decay=0.1)
    p.grad = rnd()
    for _ in range(4):
        p.grad.data = rnd()
        kept = spoil(5000)
        q.grad = p.grad.clone()
        a.step()
        b.step()
        del kept
    # a gradient of another shape in the same place is refused, not read past its end
    assert float((p - q).abs().max()) <= 1e-6 * float(q.detach().abs().max())
    p.grad.data = p.grad.data[:100]
    with pytest.raises(ValueError, match="shape"):
        a.step()


@pytest.mark.gpu
def test_plan_holds_the_memory():
    make = lambda: [torch.full((4000,), v, device="cuda") for v in (1.0, 0.5, 0.1, 0.2)]  # noqa: E731
    want, mine = make(), make()
    plans = [zs.AdamWPlan(*([t] for t in ts)) for ts in (want, mine)]
    kept = mine[0].detach()
    for t in mine:
        t.data = torch.zeros(4000, device="cuda")
    spoil(4000)
    for plan in plans:
        zs.zs_adamw_step(plan, 1, lr=1e-2)
    assert torch.equal(kept, want[0]) and not bool(mine[0].any())


@pytest.mark.gpu
@pytest.mark.parametrize("bits,dtype", [(32, torch.float32), (8, torch.float32), (8, torch.bfloat16)])
def test_example_learns(bits, dtype):
    spec = importlib.util.spec_from_file_location("species_block", os.path.join(ROOT, "examples", "species_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=60, state_bits=bits, dtype=dtype)
    assert all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]
    torch.cuda.synchronize()
    zs.zs_check_timeouts()
