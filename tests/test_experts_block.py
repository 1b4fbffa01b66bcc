"""Embedding, routing, the exchange with experts and dropout as a user has them: torch.library
operators with autograd, run together, on streams, on several devices, in captured graphs."""
import importlib.util
import os

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx

import expert_refs as ref
from equivariant_interatomic_potential_gb300 import autograd as ag, zs
from test_devices import Machine, on
from test_streams import BUSY, each

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_operators_registered():
    for name in ("embedding", "embedding_backward", "route", "route_backward", "dispatch", "combine", "combine_backward", "dropout"):
        assert hasattr(torch.ops.zs_gie, name)


def test_cpu_tensors_rejected():
    x, i = torch.zeros(4, 8), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: ag.embedding(x, i), lambda: ag.route(x, 2), lambda: ag.dispatch(x, i, i, 2),
                 lambda: ag.combine(x, i.view(4, 2), None, i, i), lambda: ag.dropout(x, 0.5, 1)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()


def test_fake_tracing():
    # traced with fake tensors: the fake implementations give every shape, no kernel runs
    def f(w, species, logits, w_in, w_out, bias, g):
        x = ag.species_embedding(species, w, 2.0)
        y = ag.expert_block(x, logits, w_in, w_out, 3, bias, "sigmoid", 2, 1, 2)
        y = ag.dropout(y, 0.1, 7, 1, 2, None, x)
        return torch.autograd.grad(y, (w, logits, w_in, w_out), g)

    M, C, E, H = 7, 8, 6, 5
    given = [torch.randn(s, requires_grad=True) for s in ((4, C), (M, E), (E, H, C), (E, C, H))]
    gm = make_fx(f, tracing_mode="fake")(given[0], torch.zeros(M, dtype=torch.int32), *given[1:], torch.zeros(E), torch.randn(M, C))
    outs = [n for n in gm.graph.nodes if n.op == "output"][0].args[0]
    assert [tuple(o.meta["val"].shape) for o in outs] == [(4, C), (M, E), (E, H, C), (E, C, H)]


def rnd(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=gen, device="cuda")


@pytest.mark.gpu
def test_each_operator_with_autograd():
    r = rnd(1)
    ids = torch.randint(-1, 6, (200,), generator=torch.Generator().manual_seed(2)).int().cuda()
    w, dy = r(6, 24).requires_grad_(), r(200, 24)
    y = ag.embedding(w, ids, 3.0)
    y.backward(dy)
    row_ptr, perm, _ = zs.zs_build_csr(ids, 6)
    assert torch.equal(y, zs.zs_embedding(w.detach(), ids, 3.0)) and torch.equal(w.grad, zs.zs_embedding_backward(dy, row_ptr, perm, 3.0))

    z, g = r(200, 16).requires_grad_(), r(200, 3)
    chosen, weights = ag.route(z, 3, None, "sigmoid", 4, 2, 2, False, 1.5)
    weights.backward(g)
    want = zs.zs_route(z.detach(), 3, None, "sigmoid", 4, 2, 2, False, 1.5)
    assert torch.equal(chosen, want[0]) and torch.equal(weights, want[1]) and not chosen.requires_grad
    assert torch.equal(z.grad, zs.zs_route_backward(g, z.detach(), chosen, "sigmoid", False, 1.5))

    row_ptr, perm = ag.build_csr(chosen.view(-1), 16)
    x, dxs = r(200, 24).requires_grad_(), r(600, 24)
    xs, slot = ag.dispatch(x, row_ptr, perm, 3)
    xs.backward(dxs)
    assert torch.equal(x.grad, zs.zs_combine(dxs, slot)) and not slot.requires_grad
    h, cw = r(600, 24).requires_grad_(), r(200, 3).requires_grad_()
    y = ag.combine(h, slot, cw, row_ptr, perm)
    y.backward(dy)
    want = zs.zs_combine_backward(dy, h.detach(), slot, cw.detach(), row_ptr)
    assert torch.equal(y, zs.zs_combine(h.detach(), slot, cw.detach())) and torch.equal(h.grad, want[0]) and torch.equal(cw.grad, want[1])

    a, b = r(200, 24).requires_grad_(), r(200, 24).requires_grad_()
    y = ag.dropout(a, 0.3, 5, 6, 7, None, b)
    y.backward(dy)
    assert torch.equal(y, zs.zs_dropout(a.detach(), 0.3, 5, 6, 7, b.detach()))
    assert torch.equal(a.grad, zs.zs_dropout(dy, 0.3, 5, 6, 7)) and torch.equal(b.grad, dy)


@pytest.mark.gpu
def test_second_derivatives_of_the_linear_ones():
    # each is linear: the loss of a square of its gradient has the operator itself, or its adjoint, as a derivative
    r = rnd(3)
    ids = torch.randint(-1, 6, (100,), generator=torch.Generator().manual_seed(4)).int().cuda()
    row_ptr, perm = ag.build_csr(torch.randint(0, 5, (200,), generator=torch.Generator().manual_seed(5)).int().cuda(), 5)
    slot = zs.zs_dispatch(r(100, 16), row_ptr, perm, 2)[1]
    for f, shape, out in ((lambda t: ag.embedding(t, ids, 2.0), (6, 16), (100, 16)),
                          (lambda t: ag.dispatch(t, row_ptr, perm, 2)[0], (100, 16), (200, 16)),
                          (lambda t: ag.combine(t, slot, None, row_ptr, perm), (200, 16), (100, 16)),
                          (lambda t: ag.dropout(t, 0.5, 9), (100, 16), (100, 16))):
        t, c = r(*shape).requires_grad_(), r(*out).requires_grad_()
        first, = torch.autograd.grad((f(t) * c).sum(), t, create_graph=True)
        second, = torch.autograd.grad(first.square().sum(), c)
        want = f(2.0 * first.detach())
        assert torch.equal(second, want)


@pytest.mark.gpu
def test_a_weighted_combine_has_no_second_derivative():
    r = rnd(6)
    row_ptr, perm = ag.build_csr(torch.zeros(20, dtype=torch.int32, device="cuda"), 1)
    slot = zs.zs_dispatch(r(10, 8), row_ptr, perm, 2)[1]
    h, w = r(20, 8).requires_grad_(), r(10, 2).requires_grad_()
    first, = torch.autograd.grad(ag.combine(h, slot, w, row_ptr, perm).square().sum(), h, create_graph=True)
    with pytest.raises(RuntimeError):
        first.sum().backward()


def plain_experts(x, logits, w_in, w_out, k, bias, score, groups, top_groups, group_top, renormalise, scale):
    """The layer of experts in 64 bits: every expert's answer for every row, and the choice by the reference."""
    z = logits.detach().cpu().numpy()
    ids, _ = ref.route(z, k, None if bias is None else bias.cpu().double().numpy(), score, groups, top_groups, group_top, renormalise, scale)
    ids = torch.from_numpy(ids).cuda()
    s = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)
    w = torch.where(ids < 0, 0.0, torch.gather(s, 1, ids.clamp_min(0)))
    if renormalise:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    full = torch.zeros_like(logits).scatter_add(1, ids.clamp_min(0), w * scale)
    h = torch.nn.functional.silu(torch.einsum("ehc,mc->meh", w_in, x))
    return torch.einsum("me,meh,enh->mn", full, h, w_out)


@pytest.mark.gpu
@pytest.mark.parametrize("M,C,H,N,E,k,groups,top_groups,score", [
    (300, 64, 96, 64, 16, 2, 1, 1, "softmax"), (257, 33, 40, 17, 12, 3, 4, 2, "sigmoid"), (1, 64, 32, 64, 64, 6, 8, 3, "softmax"),
    (1000, 128, 64, 128, 8, 8, 1, 1, "sigmoid")])
def test_experts_together(M, C, H, N, E, k, groups, top_groups, score):
    """The whole layer and its gradients in fp32 against 64 bits: two products in a row, the weights and a sum, each
    known to about sqrt(C) half ulps: 1e-5 of the largest element."""
    r = rnd(M)
    given = [r(M, C), r(M, E), r(E, H, C) * C ** -0.5, r(E, N, H) * H ** -0.5]
    bias, dy = r(E) * 0.1 if groups > 1 else None, r(M, N)
    how = (k, bias, score, groups, top_groups, 2, True, 2.0)
    results = []
    for f, dtype in ((ag.expert_block, torch.float32), (plain_experts, torch.float64)):
        leaves = [t.to(dtype).requires_grad_() for t in given]
        y = f(*leaves, *how)
        results.append((y.detach(), *torch.autograd.grad(y, leaves, dy.to(dtype))))
    for name, got, want in zip(("y", "dx", "dlogits", "dw_in", "dw_out"), *results):
        assert float((got - want).abs().max()) <= 1e-5 * float(want.abs().max()), name


@pytest.mark.gpu
def test_experts_closed_to_all_rows():
    # rows that no expert is open to give zeros and pass nothing back
    r = rnd(8)
    x, logits, w_in, w_out = (t.requires_grad_() for t in (r(40, 32), r(40, 8), r(8, 16, 32), r(8, 32, 16)))
    closed = logits.detach().clone()
    closed[10:20] = -float("inf")
    closed.requires_grad_()
    y = ag.expert_block(x, closed, w_in, w_out, 2)
    dx, dz = torch.autograd.grad(y.square().sum(), (x, closed))
    assert not bool(y[10:20].any()) and not bool(dx[10:20].any()) and not bool(dz[10:20].any())
    assert bool(y[:10].any(1).all()) and all(bool(torch.isfinite(t).all()) for t in (y, dx, dz))


def step_fn(r, M=256, C=64, E=8):
    """A training step's forward and backward with all operators, as a function of the step's count on the device."""
    table, w_in, w_out = r(5, C).requires_grad_(), (r(E, 32, C) * 0.1).requires_grad_(), (r(E, C, 32) * 0.1).requires_grad_()
    router, vec = (r(1, E, C) * 0.1).requires_grad_(), torch.ones(C, device="cuda")
    species = torch.randint(0, 5, (M,), generator=torch.Generator().manual_seed(1)).int().cuda()
    noise, all_rows = r(M, C), torch.tensor([0, M], dtype=torch.int32, device="cuda")

    def step(count):
        x = ag.species_embedding(species, table, 2.0) + noise
        h = ag.expert_block(x, ag.grouped_matmul(x, router, all_rows), w_in, w_out, 2)
        y, u, _ = ag.norm_gate_residual(ag.dropout(h, 0.2, 77, 1, 0, count), x, None, vec, vec, vec)
        return (y.detach(), *torch.autograd.grad((y * u).sum(), (table, w_in, w_out, router)))

    return step


@pytest.mark.gpu
def test_captured_steps_draw_new_masks():
    step = step_fn(rnd(9))
    counts = [torch.tensor([i], device="cuda") for i in range(3)]
    want = [[t.clone() for t in step(c)] for c in counts]
    assert not torch.equal(want[0][0], want[1][0])
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(count)
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):                      # two graphs of the same step: no memory of one is the other's
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(count)
        graphs.append((g, got))
    for i in (0, 2, 1):
        count.fill_(i)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


@pytest.mark.gpu
def test_a_step_that_moves_on_before_the_backward_pass_is_refused():
    h = torch.randn(8, 8, device="cuda", requires_grad=True)
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    y = ag.dropout(h, 0.5, 1, 0, 0, count)
    count += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with pytest.raises(ValueError, match="step and step_at"):
        ag.dropout(h, 0.5, 1, 0, 3, count)


def calls_on_streams():
    r = rnd(10)
    M, C, E, k = 3000, 129, 12, 3
    ids = torch.randint(-1, 700, (M,), generator=torch.Generator().manual_seed(1)).int().cuda()
    row_ptr, perm, _ = zs.zs_build_csr(ids, 700)
    w, dy, z = r(700, C), r(M, C), r(M, E)
    chosen, weights = zs.zs_route(z, k)
    rp, pm, _ = zs.zs_build_csr(chosen.view(-1), E)
    xs, slot = zs.zs_dispatch(dy, rp, pm, k)
    count = torch.ones(1, dtype=torch.int64, device="cuda")
    return {"csr": lambda **kw: zs.zs_build_csr(ids, 700, **kw),
            "embedding": lambda **kw: zs.zs_embedding(w, ids, 2.0, **kw),
            "embedding backward": lambda **kw: zs.zs_embedding_backward(dy, row_ptr, perm, 2.0, **kw),
            "route": lambda **kw: zs.zs_route(z, k, **kw),
            "route backward": lambda **kw: zs.zs_route_backward(weights, z, chosen, **kw),
            "dispatch": lambda **kw: zs.zs_dispatch(dy, rp, pm, k, **kw),
            "combine": lambda **kw: zs.zs_combine(xs, slot, weights, **kw),
            "combine backward": lambda **kw: zs.zs_combine_backward(dy, xs, slot, weights, rp, **kw),
            "dropout": lambda **kw: zs.zs_dropout(dy, 0.3, 4, 5, 6, **kw),
            "dropout at": lambda **kw: zs.zs_dropout(dy, 0.3, 4, 5, count, residual=dy, **kw)}


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True], ids=["object", "handle"])
def test_memory_stays_the_streams(handle):
    # the stream is kept busy while the call is made; the current stream then takes as much memory and fills it
    s = torch.cuda.Stream()
    for name, call in calls_on_streams().items():
        want = each(call())
        sizes = {t.numel() * t.element_size() for t in want}
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        call()
        sizes.add(torch.cuda.max_memory_allocated() - before)
        torch.cuda.empty_cache()
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        got = each(call(stream=s.cuda_stream if handle else s))
        taken = [torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")
                 for n in sorted(sizes) + [1 << 12, 1 << 16, 1 << 20, 1 << 22] for _ in range(4)]
        torch.cuda.synchronize()
        assert taken and all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.gpu
def test_calls_at_once():
    # the same calls on two streams at a time, several in flight: results of one do not depend on the other
    calls = calls_on_streams()
    want = {n: each(c()) for n, c in calls.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for n, c in calls.items():
            for s in streams:
                got.append((n, each(c(stream=s))))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for n, g in got for a, b in zip(g, want[n]))


@pytest.mark.gpu
def test_results_without_the_extension(monkeypatch):
    calls = calls_on_streams()
    want = {n: each(c()) for n, c in calls.items()}
    monkeypatch.setattr(zs, "_fast", type("None", (), {"__getattr__": lambda self, n: lambda *a: NotImplemented})())
    for n, c in calls.items():
        got = each(c())
        assert len(got) == len(want[n]) and all(torch.equal(a, b) and a.dtype == b.dtype for a, b in zip(got, want[n])), n


@pytest.fixture
def machine(monkeypatch):
    if torch.cuda.is_available() and torch.cuda.device_count() < 2:
        pytest.skip("a fake tensor's device has to exist where there is a GPU")
    with FakeTensorMode():
        yield Machine(monkeypatch)


def device_calls(d):
    i32, i64 = dict(dtype=torch.int32), dict(dtype=torch.int64)
    return [(zs.zs_embedding, (on(d, 5, 8), on(d, 6, **i32))),
            (zs.zs_embedding_backward, (on(d, 6, 8), on(d, 6, **i32), on(d, 6, **i32))),
            (lambda z, b: zs.zs_route(z, 2, b), (on(d, 6, 8), on(d, 8))),
            (zs.zs_route_backward, (on(d, 6, 2), on(d, 6, 8), on(d, 6, 2, **i32))),
            (lambda x, rp, pm: zs.zs_dispatch(x, rp, pm, 2), (on(d, 6, 8), on(d, 4, **i32), on(d, 12, **i32))),
            (zs.zs_combine, (on(d, 12, 8), on(d, 6, 2, **i32), on(d, 6, 2))),
            (zs.zs_combine_backward, (on(d, 6, 8), on(d, 12, 8), on(d, 6, 2, **i32), on(d, 6, 2), on(d, 4, **i32))),
            (lambda h, r, at: zs.zs_dropout(h, 0.5, 1, 0, at, r), (on(d, 6, 8), on(d, 6, 8), on(d, 1, **i64)))]


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
@pytest.mark.parametrize("device", [0, 1])
def test_launched_on_the_operands_device(machine, device):
    for fn, operands in device_calls(device):
        machine.seen.clear()
        fn(*operands)
        assert [d for _, d in machine.seen] == [device] and machine.current == 0, machine.seen


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_mixed_devices_refused(machine):
    for fn, operands in device_calls(0):
        for i, t in enumerate(operands):
            other = list(operands)
            other[i] = on(1, *t.shape, dtype=t.dtype)
            with pytest.raises(ValueError, match="one device, got cuda:0 and cuda:1"):
                fn(*other)
    assert not machine.seen


def example():
    spec = importlib.util.spec_from_file_location("expert_block", os.path.join(ROOT, "examples", "expert_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.bfloat16, 8)])
def test_example_runs(dtype, bits):
    losses = example().train(3, bits, dtype, nodes=200, edges=3000)
    assert len(losses) == 3 and np.isfinite(losses).all()


@pytest.mark.gpu
def test_example_gradients_against_differences():
    """The example's loss along a random direction of each parameter, with every expert chosen (a choice is a step, which
    has no slope).  A step moves a parameter by at most about 1 % of its size: 1e-4 of the slope's terms are of third order;
    the loss, a sum of 200 terms known to about 1e-6, is off by 1e-4, the slope by 0.1: both below 1e-2 of the terms."""
    m = example()
    m.CHOICES, m.OPEN_GROUPS = m.EXPERTS, m.GROUPS
    given = m.data(200, 3000, torch.float32)
    block = m.Block(given[0].shape[1], torch.float32, seed=3)
    target = torch.randn(200, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    count = torch.zeros(1, dtype=torch.int64, device="cuda")

    def loss():
        return ((block(*given, count).double() - target) * target).sum()

    names, params = zip(*block.named_parameters())
    grads = torch.autograd.grad(loss(), params)
    for i, (name, p, g) in enumerate(zip(names, params, grads)):
        v = torch.randn(p.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        with torch.no_grad():
            p += 1e-3 * v
            up = loss()
            p -= 2e-3 * v
            down = loss()
            p += 1e-3 * v
        slope, terms = float(up - down) / 2e-3, g.double() * v.double()
        assert abs(slope - float(terms.sum())) <= 1e-2 * float(terms.abs().sum()), name


@pytest.mark.parametrize("logits,w_in,w_out", [(6, 5, 5), (5, 6, 6), (6, 6, 5), (5, 5, 6)])
def test_numbers_of_experts_that_differ_are_refused(logits, w_in, w_out):
    # assignments to experts that have no weights would be dropped, after the weights were renormalised over them
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match=f"{logits} experts, w_in of {w_in} and w_out of {w_out}"):
        ag.expert_block(x, torch.zeros(4, logits), torch.zeros(w_in, 16, 8), torch.zeros(w_out, 8, 16), 2)
