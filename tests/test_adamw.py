"""The AdamW step.  Its arithmetic is documented operation by operation, so
parameters, states, codes and scales are compared bit for bit with the same
operations in numpy's float32, and the 32-bit step with the update in 64
bits (fp32 rounding of six operations: 1e-6 relative)."""
import ctypes

import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import zs
from train_refs import E4M3, TORCH, adamw, f64, quantise, to_e4m3

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def same(got, ref, what):
    got, ref = np.asarray(got), np.asarray(ref)
    assert got.shape == ref.shape, what
    eq = (got == ref) | (np.isnan(got) & np.isnan(ref))
    assert eq.all(), f"{what}: {(~eq).sum()} of {eq.size} differ"


class Host:
    """The tensors of a step on the CPU, as float32 values."""

    def __init__(self, sizes, dtype, eight, seed):
        rng = np.random.default_rng(seed)
        self.dtype, self.eight = dtype, eight
        rnd = lambda n, s: torch.from_numpy((rng.standard_normal(n) * s).astype(np.float32))  # noqa: E731
        self.p = [rnd(n, 0.02).to(TORCH[dtype]).float().numpy() for n in sizes]
        self.g = [rnd(n, 0.01).to(TORCH[dtype]).float().numpy() for n in sizes]
        self.m = [rnd(n, 0.003).numpy() for n in sizes]
        self.v = [np.abs(rnd(n, 0.01).numpy()) for n in sizes]     # the root when eight
        if eight:
            self.hold()
        else:
            self.v = [a * a for a in self.v]

    def hold(self):
        self.mc, self.ms = zip(*[quantise(a, False) for a in self.m])
        self.vc, self.vs = zip(*[quantise(a, True) for a in self.v])

    def plan(self, place):
        """An AdamWPlan over copies on the GPU; `place` puts a tensor somewhere."""
        dt = TORCH[self.dtype]
        up = lambda lst, d: [place(torch.from_numpy(np.asarray(a, np.float32)).to(d)) for a in lst]  # noqa: E731
        if not self.eight:
            return zs.AdamWPlan(up(self.p, dt), up(self.g, dt), up(self.m, torch.float32), up(self.v, torch.float32))
        return zs.AdamWPlan(up(self.p, dt), up(self.g, dt), up(self.mc, torch.float8_e4m3fn),
                            up(self.vc, torch.float8_e4m3fn), up(self.ms, torch.float32), up(self.vs, torch.float32))

    def step(self, t, grad_scale=1.0, **kw):
        h = {**HYPER, **kw}
        for i, g in enumerate(self.g):
            m, v = self.m[i], self.v[i]
            if self.eight:
                s = lambda sc, n: np.repeat(sc, 256)[:n]  # noqa: E731
                m = self.mc[i].astype(np.float32) * s(self.ms[i], len(g))
                v = self.vc[i].astype(np.float32) * s(self.vs[i], len(g))
            p, self.m[i], self.v[i] = adamw(self.p[i], g, m, v, t, h["lr"], h["beta1"], h["beta2"], h["eps"],
                                            h["weight_decay"], grad_scale, self.eight)
            self.p[i] = torch.from_numpy(p).to(TORCH[self.dtype]).float().numpy()
        if self.eight:
            self.hold()

    def compare(self, plan):
        for i in range(len(self.p)):
            same(plan.params[i].float().cpu().numpy(), self.p[i], f"param {i}")
            if self.eight:
                same(plan.exp_avg[i].float().cpu().numpy(), self.mc[i].astype(np.float32), f"first moment's codes {i}")
                same(plan.exp_avg_sq[i].float().cpu().numpy(), self.vc[i].astype(np.float32), f"root's codes {i}")
                same(plan.scales[0][i].cpu().numpy(), self.ms[i], f"first moment's scales {i}")
                same(plan.scales[1][i].cpu().numpy(), self.vs[i], f"root's scales {i}")
            else:
                same(plan.exp_avg[i].cpu().numpy(), self.m[i], f"first moment {i}")
                same(plan.exp_avg_sq[i].cpu().numpy(), self.v[i], f"second moment {i}")


def cuda(t):
    return t.cuda()


def shifted(t):
    """On the GPU, one element off the allocator's alignment."""
    base = torch.zeros(t.numel() + 1, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
    view = base[1:].view(t.dtype)
    view.copy_(t)
    return view


SIZES = [[1], [255, 256, 257], [2047, 2048, 2049, 0, 7], [100003], [5] * 40, [int(n) for n in range(1, 600)]]


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", SIZES, ids=["one", "blocks", "chunks", "long", "short_table", "long_tables"])
def test_steps(sizes, dtype, eight):
    host = Host(sizes, dtype, eight, seed=len(sizes) + sum(sizes))
    plan = host.plan(cuda)
    scale = torch.full((1,), 0.25, device="cuda")
    for t in (1, 2, 1000):
        host.step(t, 0.25)
        zs.zs_adamw_step(plan, t, grad_scale=scale, **HYPER)
        host.compare(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_any_alignment(dtype, eight):
    host = Host([1, 300, 4099], dtype, eight, 5)
    plan = host.plan(shifted)
    host.step(7)
    zs.zs_adamw_step(plan, 7, **HYPER)
    host.compare(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_zero_and_extreme_gradients(eight):
    # blocks of zeros, of values below the held range, of one huge value, and of NaN and infinity: each stays its own
    host = Host([256 * 6 + 100], "f32", eight, 9)
    g = host.g[0]
    for a in (host.m, host.v):
        a[0][:512] = 0
        a[0][256 * 5:] = 0
    g[:256] = 0
    g[256:512] = 1e-36
    g[512:768] = 1e-12
    g[600] = 1e6
    g[800], g[801] = np.nan, np.inf
    g[1100] = 3e38
    if eight:
        host.hold()
    plan = host.plan(cuda)
    for t in (1, 2, 3):
        host.step(t)
        zs.zs_adamw_step(plan, t, **HYPER)
        host.compare(plan)
    p = plan.params[0]
    sick = torch.isnan(p).nonzero().flatten().tolist()
    assert set(sick) <= {800, 801, 1100} and 800 in sick


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(weight_decay=0.0), dict(beta1=0.0), dict(beta2=0.0), dict(lr=0.0), dict(eps=1e-3)])
def test_hyper_parameters(kw):
    host = Host([3000, 17], "f32", False, 4)
    plan = host.plan(cuda)
    for t in (1, 5):
        host.step(t, **kw)
        zs.zs_adamw_step(plan, t, **{**HYPER, **kw})
        host.compare(plan)


@pytest.mark.gpu
def test_step_against_64_bits():
    host = Host([20000], "f32", False, 3)
    p, g, m, v = (a[0].astype(np.float64) for a in (host.p, host.g, host.m, host.v))
    plan = host.plan(cuda)
    zs.zs_adamw_step(plan, 10, **HYPER)
    m = 0.9 * m + 0.1 * g
    v = 0.999 * v + 0.001 * g * g
    p = p * (1 - 1e-5) - 1e-3 * (m / (1 - 0.9 ** 10)) / (np.sqrt(v / (1 - 0.999 ** 10)) + 1e-8)
    for got, ref in ((plan.params[0], p), (plan.exp_avg[0], m), (plan.exp_avg_sq[0], v)):
        assert np.abs(f64(got) - ref).max() <= 1e-6 * np.abs(ref).max()


@pytest.mark.gpu
def test_new_gradients_and_streams():
    host = Host([5000, 600], "bf16", True, 11)
    plan = host.plan(cuda)
    host.step(1)
    zs.zs_adamw_step(plan, 1, **HYPER)
    host.g = [np.ascontiguousarray(a[::-1]) for a in host.g]
    plan.set_grads([torch.from_numpy(a).to(torch.bfloat16).cuda() for a in host.g])
    host.step(2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    zs.zs_adamw_step(plan, 2, stream=s, **HYPER)
    torch.cuda.synchronize()
    host.compare(plan)


def test_reference_code_rounding():
    # the reference's e4m3 rounding against torch's conversion, every tie among them
    mid = (E4M3[:-1] + E4M3[1:]) / 2
    q = np.concatenate([E4M3, mid, np.nextafter(mid.astype(np.float32), 0), np.random.default_rng(0).random(4000) * 448])
    q = np.concatenate([q, -q]).astype(np.float32)
    same(to_e4m3(q.astype(np.float64)), torch.from_numpy(q).to(torch.float8_e4m3fn).double().numpy(), "codes")


def test_argument_checks():
    lib = zs.load()

    def call(bits=32, dtype=0, count=1, table=True, hyper=True, **kw):
        t = (zs._AdamWTensor * 1)()
        t[0].param = t[0].grad = t[0].exp_avg = t[0].exp_avg_sq = t[0].exp_avg_scale = t[0].exp_avg_sq_scale = FAKE
        t[0].numel = 10
        h = zs._AdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0.01, 1)
        for k, v in kw.items():
            setattr(t[0] if hasattr(t[0], k) else h, k, v)
        return lib.zs_adamw_step(ctypes.addressof(t) if table else None, count, dtype, bits,
                                 ctypes.addressof(h) if hyper else None, None, None)

    for kw in (dict(bits=16), dict(bits=0), dict(dtype=3)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(count=-1), dict(table=False), dict(hyper=False), dict(numel=-1), dict(param=None), dict(grad=None),
               dict(exp_avg=None), dict(exp_avg_sq=None), dict(bits=8, exp_avg_scale=None), dict(param=FAKE + 2),
               dict(exp_avg=FAKE + 1), dict(dtype=1, grad=FAKE + 1), dict(bits=8, exp_avg_sq_scale=FAKE + 2), dict(step=0),
               dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan")), dict(weight_decay=float("inf"))):
        assert call(**kw) == INVALID, kw
    assert call(count=0, table=False) == 0 and call(numel=0, param=None) == 0


def test_plan_refusals():
    t = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        zs.AdamWPlan([t], [t], [t], [t])
    with pytest.raises(ValueError, match="at least one"):
        zs.AdamWPlan([], [], [], [])
    with pytest.raises(ValueError, match="scales"):
        zs.AdamWPlan([t], [t], [t], [t], [t], None)
    with pytest.raises(ValueError, match="has 0 tensors"):
        zs.AdamWPlan([t], [t], [], [t])
