"""8-bit states whose codes are rounded at random.

The random numbers follow from the arguments, so one step is compared bit for
bit with the same operations in numpy, as the step rounded to nearest is.  Over
some thousand steps the states are compared with 32-bit ones: the second moment
of gradients that have become small has to fall."""
import ctypes

import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import AdamW, zs
from test_adamw import FAKE, HYPER, SIZES, UNSUPPORTED, INVALID, Host, cuda, same, shifted
from train_refs import E4M3, adamw, quantise

f, u32 = np.float32, np.uint32


def random_bits(c, seed, step):
    """32 bits of each element number c (int64)."""
    mask = (1 << 64) - 1
    key = (seed ^ (step * 0x9e3779b97f4a7c15)) & mask
    for _ in range(2):
        key = (key ^ (key >> 32)) * 0xd6e8feb86659fd93 & mask
    key ^= key >> 32
    lo, hi = u32(key & 0xffffffff), u32(key >> 32)
    with np.errstate(over="ignore"):
        x = (c & 0xffffffff).astype(u32) ^ (lo + (c >> 32).astype(u32) * u32(0x9e3779b9))
        x = (x ^ (x >> u32(16))) * u32(0x7feb352d)
        x = ((x ^ (x >> u32(15))) + hi) * u32(0x846ca68b)
    return x ^ (x >> u32(16))


def round_at_random(q, bits16):
    a = np.abs(q).astype(f)
    off = np.where(a < f(2.0 ** -6), f(2.0 ** -6), f(0))
    t = ((a + off).view(u32) + (bits16.astype(u32) << u32(4)) + u32(8)) & u32(0xfff00000)
    return np.copysign(np.minimum(t.view(f) - off, f(448)), q)


def quantise_at_random(v, root, bits16):
    """As train_refs.quantise, rounded at random."""
    codes, scales = quantise(v, root)
    for b in range(0, len(v), 256):
        x = v[b:b + 256].astype(f)
        fin = np.isfinite(x)
        top = f(np.abs(x[fin]).max()) if fin.any() else f(0)
        inv = f(f(f(1) / top) * f(448)) if top >= f(1e-30) else f(0)
        c = round_at_random((np.where(fin, x, 0) * inv).astype(f), bits16[b:b + 256])
        if root and inv > 0:
            c = np.where(x > 0, np.maximum(c, f(2.0 ** -9)), c)
        codes[b:b + 256] = np.where(fin, c, np.nan)
    return codes, scales


class Seeded(Host):
    now = None   # (seed, step): rounded at random from then on

    def hold(self):
        if self.now is None:
            return super().hold()
        at, bits = 0, []
        for a in self.m:
            bits.append(random_bits(np.arange(at, at + len(a), dtype=np.int64), *self.now))
            at += -(-len(a) // 2048) * 2048
        self.mc, self.ms = zip(*[quantise_at_random(a, False, x & u32(0xffff)) for a, x in zip(self.m, bits)])
        self.vc, self.vs = zip(*[quantise_at_random(a, True, x >> u32(16)) for a, x in zip(self.v, bits)])

    def seeded_step(self, t, seed, grad_scale=1.0):
        self.now = (seed, t)
        self.step(t, grad_scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", SIZES, ids=["one", "blocks", "chunks", "long", "short_table", "long_tables"])
def test_steps(sizes, dtype):
    host = Seeded(sizes, dtype, True, seed=len(sizes) + sum(sizes))
    plan = host.plan(cuda)
    scale = torch.full((1,), 0.25, device="cuda")
    for t, seed in ((1, 0), (2, 1), (3, 1), (1000, (1 << 64) - 1)):
        host.seeded_step(t, seed, 0.25)
        zs.zs_adamw_step(plan, t, grad_scale=scale, seed=seed, **HYPER)
        host.compare(plan)


@pytest.mark.gpu
def test_any_alignment_and_extremes():
    host = Seeded([1, 256 * 6 + 100, 4099], "f32", True, 5)
    g = host.g[1]
    for a in (host.m, host.v):
        a[1][:512] = 0
    host.hold()
    g[:256], g[256:512], g[512:768] = 0, 1e-36, 1e-12
    g[600], g[800], g[801], g[1100] = 1e6, np.nan, np.inf, 3e38
    plan = host.plan(shifted)
    for t in (7, 8):
        host.seeded_step(t, 3)
        zs.zs_adamw_step(plan, t, seed=3, **HYPER)
        host.compare(plan)


@pytest.mark.gpu
def test_32_bit_states_have_no_codes():
    host = Host([3000], "f32", False, 1)
    plan = host.plan(cuda)
    host.step(1)
    zs.zs_adamw_step(plan, 1, seed=9, **HYPER)
    host.compare(plan)


@pytest.mark.gpu
def test_class_against_32_bit_states():
    """Half of each block's gradients shrink 100-fold after 500 steps.  The root of that
    half has to follow the one held in 32 bits: its expectation does up to the curvature
    of the root over a code's width (an eighth at most), 2048 of them average out all but
    some percent of the codes' noise: within a quarter.  Held to nearest it stays
    seventeen times too large."""
    n, gen = 4096, torch.Generator(device="cuda").manual_seed(3)
    quiet = (torch.arange(n, device="cuda") % 256) < 128
    params = [torch.zeros(n, device="cuda") for _ in range(2)]
    opts = [AdamW([p], lr=1e-3, weight_decay=0.0, state_bits=b) for p, b in zip(params, (32, 8))]
    for t in range(6000):
        g = torch.randn(n, generator=gen, device="cuda") * 0.01
        if t >= 500:
            g[quiet] *= 0.01
        for p, opt in zip(params, opts):
            p.grad = g
            opt.step()
        if t % 1000 == 999:
            s32, s8 = opts[0].state[params[0]], opts[1].state[params[1]]
            want = s32["exp_avg_sq"].sqrt()
            root = s8["exp_avg_sq"].float() * s8["exp_avg_sq_scale"].repeat_interleave(256)
            m = s8["exp_avg"].float() * s8["exp_avg_scale"].repeat_interleave(256)
            for half in (quiet, ~quiet):
                assert abs(float(root[half].mean() / want[half].mean()) - 1) <= 0.25, t
                assert float((m - s32["exp_avg"])[half].square().mean().sqrt()) <= 0.25 * float(
                    s32["exp_avg"].square().mean().sqrt()), t
    assert float(want[quiet].mean() / want[~quiet].mean()) < 0.05


def test_rounding_of_the_reference():
    # what is a code stays one, others go to a neighbour, and on average nowhere
    rng = np.random.default_rng(0)
    for bits in (0, 1, 0x7fff, 0xffff):
        k = np.full(len(E4M3), bits, u32)
        same(round_at_random(E4M3.astype(f), k), E4M3.astype(f), "codes")
        same(round_at_random(-E4M3.astype(f), k), -E4M3.astype(f), "codes")
    every = np.arange(65536, dtype=u32)
    for q in np.concatenate([np.exp(rng.uniform(np.log(1e-4), np.log(448), 40)), [2.0 ** -9 * 1.5, 2.0 ** -6 * 0.999]]).astype(f):
        got = round_at_random(np.full(65536, q, f), every).astype(np.float64)
        i = np.searchsorted(E4M3, q)
        assert set(got) <= {E4M3[i - 1], E4M3[i]}
        # 65536 equal chances, and 24 bits of the sum with 2^-6
        assert abs(got.mean() - q) <= (E4M3[i] - E4M3[i - 1]) * 2.0 ** -15


def test_second_moment_held_to_nearest_stands_still():
    # why: a root half as large as its block's largest, and no gradient: 3000 steps leave its code, at random it falls
    held = {}
    for name in ("nearest", "random"):
        v = np.r_[np.full(64, 0.5), np.ones(64)].astype(f)
        g = np.r_[np.zeros(64), np.ones(64)].astype(f)
        for t in range(1, 3001):
            _, _, v = adamw(v, g, v, v, t, 0.0, 0.9, 0.999, 1e-8, 0.0, 1.0, True)
            bits = random_bits(np.arange(128, dtype=np.int64), 0, t) >> u32(16)
            codes, scales = quantise(v, True) if name == "nearest" else quantise_at_random(v, True, bits)
            v = (codes.astype(f) * scales[0]).astype(f)
        held[name] = v[:64].mean()
    assert abs(held["nearest"] - 0.5) < 0.04 and abs(held["random"] / (0.5 * 0.999 ** 1500) - 1) < 0.25


def test_argument_checks():
    lib = zs.load()
    t = (zs._AdamWTensor * 1)()
    t[0].param = t[0].grad = t[0].exp_avg = t[0].exp_avg_sq = FAKE
    t[0].numel = 10
    h = zs._AdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0.01, 1)
    call = lambda bits, dtype=0: lib.zs_adamw_step_seeded(ctypes.addressof(t), 1, dtype, bits, ctypes.addressof(h), 5, None, None)  # noqa: E731
    assert call(16) == UNSUPPORTED and b"zs_adamw_step_seeded" in lib.zs_last_error() and call(8, 3) == UNSUPPORTED
    assert call(8) == INVALID      # no scales
