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


def test_gradients_nobody_asked_for_are_not_formed(monkeypatch):
    # traced with fake tensors: which operators the backward calls
    def backward_of(needs):
        x, w = (torch.randn(s, requires_grad=n) for s, n in zip(((7, 8), (3, 5, 8)), needs))
        f = lambda x, w: torch.autograd.grad(ag.species_linear(x, w, torch.zeros(7, dtype=torch.int32)).sum(),  # noqa: E731
                                             [t for t in (x, w) if t.requires_grad])
        nodes = make_fx(f, tracing_mode="fake")(x, w).graph.nodes
        return sorted(str(n.target) for n in nodes if "grouped_matmul_" in str(n.target))

    dx, dw, both = (f"zs_gie.grouped_matmul_{n}.default" for n in ("dx", "dw", "backward"))
    assert backward_of((True, False)) == [dx] and backward_of((False, True)) == [dw] and backward_of((True, True)) == [both]


@pytest.mark.gpu
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("needs", [(True, True), (True, False), (False, True)])
def test_grouped_second_derivatives(needs, gathered):
    """A loss of an energy and its gradients (the forces' loss), against the same in 64 bits from plain products.
    Each result is a sum of at most three chains of products: 1e-5 of the magnitude of its largest element."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    M, K, N, G = 300, 48, 40, 4
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    group = torch.randint(0, G, (M,), generator=gen, device="cuda")
    group = group if gathered else group.sort()[0]
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group.cpu().numpy(), G))
    values = rnd(M, K), rnd(G, N, K) * K ** -0.5, rnd(M, N), rnd(M, K), rnd(G, N, K)

    def grads(dtype):
        x, w, c, a, b = (v.to(dtype) for v in values)
        x.requires_grad_(needs[0]), w.requires_grad_(needs[1])
        y = ag.grouped_matmul(x, w, row_ptr, perm if gathered else None) if dtype == torch.float32 else \
            torch.einsum("mnk,mk->mn", w[group], x)
        energy = (torch.tanh(y) * c).sum()       # not linear: the cotangent of y wants a gradient too
        at = [t for t in (x, w) if t.requires_grad]
        first = torch.autograd.grad(energy, at, create_graph=True)
        loss = energy + sum((g.square() * (a if g.dim() == 2 else b)).sum() for g in first)
        return torch.autograd.grad(loss, at)

    for got, want in zip(grads(torch.float32), grads(torch.float64)):
        assert float((got - want).abs().max()) <= 1e-5 * float(want.abs().max())


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


@pytest.mark.parametrize("which", ["y", "u"])
def test_cotangents_that_are_not_there(which):
    # traced with fake tensors: no matrix of zeros in a cotangent's place
    def f(h, x, vec):
        y, u, _ = ag.norm_gate_residual(h, x, None, vec, vec, vec)
        return torch.autograd.grad((y if which == "y" else u).sum(), (h, x, vec))

    h, x, vec = (torch.randn(s, requires_grad=True) for s in ((7, 8), (7, 8), (8,)))
    nodes = list(make_fx(f, tracing_mode="fake")(h, x, vec).graph.nodes)
    call, = [n for n in nodes if "norm_gate_residual_backward" in str(n.target)]
    assert (call.args[0] is None, call.args[1] is None) == (which == "u", which == "y")
    assert not any("zeros" in str(n.target) for n in nodes)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["y", "u"])
def test_norm_autograd_of_one_output(which):
    M, C = 300, 96
    gen = torch.Generator(device="cuda").manual_seed(14)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ops, d = [rnd(M, C), rnd(M, C), rnd(M, C), rnd(C), rnd(C), rnd(C)], rnd(M, C)
    leaves = [t.clone().requires_grad_() for t in ops]
    y, u, _ = ag.norm_gate_residual(*leaves)
    (y if which == "y" else u).backward(d)
    stats = zs.zs_norm_gate_residual(*ops)[2]
    want = zs.zs_norm_gate_residual_backward(d if which == "y" else None, d if which == "u" else None, *ops, stats)
    assert all(torch.equal(leaf.grad, g) for leaf, g in zip(leaves, want))


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


def test_optimiser_is_one_of_torchs(tmp_path):
    # groups with options of their own, schedulers, hooks, and states that are kept as they are (on the CPU: no step)
    p, q = torch.zeros(300), torch.zeros(33, dtype=torch.bfloat16)
    opt = AdamW([{"params": [p], "weight_decay": 0.0}, {"params": [q], "state_bits": 8}], lr=0.5, betas=(0.8, 0.9))
    assert isinstance(opt, torch.optim.Optimizer) and opt.lr == 0.5 and opt.betas == (0.8, 0.9)
    torch.optim.lr_scheduler.StepLR(opt, 1)
    opt.lr = 0.25
    assert [g["lr"] for g in opt.param_groups] == [0.25, 0.25] and [g["weight_decay"] for g in opt.param_groups] == [0.0, 0.01]
    for s in opt.state.values():   # values that the parameters' types could not hold
        for k, v in s.items():
            if k != "step":
                v.copy_(torch.rand(v.shape) + 0.1)
        s["step"] = 7
    torch.save(opt.state_dict(), tmp_path / "state")
    other = AdamW([{"params": [p.clone()]}, {"params": [q.clone()], "state_bits": 8}])
    other.load_state_dict(torch.load(tmp_path / "state"))
    assert other.lr == 0.25 and other.param_groups[0]["weight_decay"] == 0.0 and other.betas == (0.8, 0.9)
    for a, b in zip(opt.state.values(), other.state.values()):
        assert a.keys() == b.keys() and a["step"] == b["step"] == 7
        assert all(a[k].dtype == b[k].dtype and torch.equal(a[k].float(), b[k].float()) for k in a if k != "step")
    with pytest.raises(ValueError, match="state_bits"):
        AdamW([{"params": [p]}, {"params": [q]}]).load_state_dict(opt.state_dict())
    with pytest.raises(ValueError, match="shape"):
        AdamW([{"params": [p[:5]]}, {"params": [q], "state_bits": 8}]).load_state_dict(opt.state_dict())
    with pytest.raises(ValueError, match="state_bits must be"):
        opt.add_param_group({"params": [torch.zeros(3)], "state_bits": 4})


def test_optimiser_state_dict_is_a_snapshot():
    opt = AdamW([torch.zeros(5)])
    d = opt.state_dict()
    for s in opt.state.values():
        s["step"] = 3
        s["exp_avg"].fill_(1.0)
    assert d["state"][0]["step"] == 0 and not bool(d["state"][0]["exp_avg"].any())
    opt.load_state_dict(d)
    assert opt.state[opt.param_groups[0]["params"][0]]["step"] == 0


def test_optimiser_loads_the_form_without_groups():
    state = [{"exp_avg": torch.full((5,), 0.5), "exp_avg_sq": torch.full((5,), 0.25)},
             {"exp_avg": torch.full((2,), 0.1), "exp_avg_sq": torch.full((2,), 0.2)}]
    for steps in (11, [11, 4]):
        opt = AdamW([torch.zeros(5), torch.zeros(2)], lr=0.3)
        opt.load_state_dict({"steps": steps, "state_bits": 32, "state": state})
        a, b = opt.state.values()
        assert a["step"] == 11 and b["step"] == (11 if steps == 11 else 4) and opt.lr == 0.3
        assert torch.equal(a["exp_avg"], state[0]["exp_avg"]) and torch.equal(b["exp_avg_sq"], state[1]["exp_avg_sq"])
        with pytest.raises(ValueError, match="state_bits"):
            opt.load_state_dict({"steps": steps, "state_bits": 8, "state": state})
        with pytest.raises(ValueError, match="parameters"):
            opt.load_state_dict({"steps": steps if steps == 11 else [3], "state_bits": 32, "state": state[:1]})


@pytest.mark.gpu
def test_optimiser_groups_and_schedule_against_torch():
    # groups, a scheduler of rates and betas, a closure, and torch's own state taken over half way
    gen = torch.Generator(device="cuda").manual_seed(8)
    first = [torch.randn(s, generator=gen, device="cuda") for s in ((300, 7), (64,), (1000,))]

    def build(cls, values):
        ps = [v.clone().requires_grad_() for v in values]
        opt = cls([{"params": ps[:1], "weight_decay": 0.0, "eps": 1e-6}, {"params": ps[1:], "lr": 3e-3}], lr=1e-2, weight_decay=0.1)
        return ps, opt, torch.optim.lr_scheduler.OneCycleLR(opt, max_lr=[2e-2, 1e-2], total_steps=40)

    (mine, a, sa), (theirs, b, sb) = build(AdamW, first), build(torch.optim.AdamW, first)
    for t in range(30):
        if t == 15:
            state = b.state_dict()
            a.load_state_dict(state)
        for p, q in zip(mine, theirs):
            p.grad = torch.randn(p.shape, generator=gen, device="cuda")
            q.grad = p.grad.clone()
        assert float(a.step(lambda: torch.tensor(5.0))) == 5.0
        b.step()
        sa.step()
        sb.step()
        for p, q in zip(mine, theirs):
            assert float((p - q).abs().max()) <= 3e-6 * float(q.detach().abs().max()), t
    scale = torch.full((1,), 0.0, device="cuda")
    a.lr = 0.0
    before = [p.detach().clone() for p in mine]
    a.step(scale)   # in the closure's place
    assert all(torch.equal(p, q) for p, q in zip(mine, before))


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_optimiser_step_is_not_captured():
    p = torch.ones(100, device="cuda")
    p.grad = torch.ones(100, device="cuda")
    opt = AdamW([p])
    opt.step()
    before, s = p.clone(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        with pytest.raises(RuntimeError, match="captured"):
            opt.step()
    torch.cuda.synchronize()
    assert torch.equal(p, before) and opt.state[p]["step"] == 1
    opt.step()
    assert not torch.equal(p, before)


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
def test_optimiser_refuses_before_it_steps():
    # one gradient of a wrong shape: no parameter moves, of whatever launch
    p, q = torch.ones(50, device="cuda"), torch.ones(60, device="cuda", dtype=torch.bfloat16)
    opt = AdamW([p, q])
    p.grad, q.grad = torch.ones_like(p), torch.ones_like(q)
    opt.step()
    before = p.clone(), q.clone()
    q.grad.data = torch.ones(30, device="cuda", dtype=torch.bfloat16)
    for _ in range(2):
        with pytest.raises(ValueError, match="shape"):
            opt.step()
    assert torch.equal(p, before[0]) and torch.equal(q, before[1]) and opt.state[p]["step"] == opt.state[q]["step"] == 1
    q.grad = torch.ones_like(q)
    opt.step()
    assert not torch.equal(p, before[0]) and opt.state[p]["step"] == opt.state[q]["step"] == 2


@pytest.mark.filterwarnings("ignore:optimizer contains a parameter group with duplicate")
def test_parameters_given_twice():
    # threads of one launch would read and write them at the same time
    p, q = torch.zeros(5), torch.zeros(3)
    with pytest.raises(ValueError, match="twice"):
        AdamW([p, q, p])
    opt = AdamW([p])
    with pytest.raises(ValueError, match="twice"):
        opt.add_param_group({"params": [q, q]})
    with pytest.raises(ValueError):
        opt.add_param_group({"params": [p]})
    assert len(opt.param_groups) == 1


@pytest.mark.gpu
def test_plan_of_overlapping_memory():
    a = torch.zeros(1000, device="cuda")
    make = lambda n, k=1: [torch.zeros(n, device="cuda") for _ in range(k)]  # noqa: E731
    with pytest.raises(ValueError, match="overlap"):
        zs.AdamWPlan([a[:600], a[599:]], [*make(600), *make(401)], [*make(600), *make(401)], [*make(600), *make(401)])
    m = make(600)
    with pytest.raises(ValueError, match="overlap"):
        zs.AdamWPlan([a[:600]], make(600), m, m)
    zs.AdamWPlan([a[:600], a[600:]], [*make(600), *make(400)], [*make(600), *make(400)], [*make(600), *make(400)])


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
