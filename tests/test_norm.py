"""The residual norms with a gate, against the plain implementation in 64 bits.

Tolerances, fixed before the first run.  An element of an output is a sum of
at most six products, each of a few factors known to about 16 ulps of fp32
(the row sums add sqrt(C) of half an ulp): 1e-5 of the output's largest
magnitude, plus the one rounding to its type.  A gradient's magnitude is that
of the terms its formula adds, which may cancel; the column sums over M rows
are held to 1e-5 of the sum of theirs."""
import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import zs
from train_refs import HALF_ULP, STEP, f64, held, norm_backward, norm_forward

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20
EPS = 1e-6
TOL = 1e-5
NAMES = ("dh", "dx", "dgate", "dw_post", "dscale", "dw_pre")


def close(got, ref, dtype, what, mag=None):
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.size == 0:
        return
    bound = TOL * (np.abs(ref).max() if mag is None else mag) + HALF_ULP[dtype] * (1 + 1e-3) * np.abs(ref) + STEP[dtype]
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / bound):.2f} x the bound"


def draw(M, C, gate, dtype, seed):
    rng = np.random.default_rng(seed)
    rows = {"full": C, "row": 1}
    big = [held(rng.standard_normal((M, C)), dtype), held(rng.standard_normal((M, C)) * 2 + 0.1, dtype),
           (None, None) if gate == "none" else held(rng.standard_normal((M, rows[gate])) * 3, dtype)]
    small = [held(rng.standard_normal(C) * s + b, "f32") for s, b in ((0.1, 1), (0.3, 0), (0.1, 1))]
    cot = [held(rng.standard_normal((M, C)), dtype) for _ in range(2)]
    return [t for t, _ in big + small], [d for _, d in big + small], [t for t, _ in cot], [d for _, d in cot]


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


def check(t, d, ct, cd, dtype, kind):
    t, ct = cuda(t), cuda(ct)
    y, u, stats = zs.zs_norm_gate_residual(*t, eps=EPS, kind=kind)
    f = norm_forward(*d, EPS, kind)
    close(y, f["y"], dtype, "y")
    close(u, f["u"], dtype, "u")
    grads = zs.zs_norm_gate_residual_backward(*ct, *t, stats, kind=kind)
    dy, du = (np.zeros_like(d[0]) if c is None else c for c in cd)
    ref, mags = norm_backward(dy, du, *d, EPS, kind)
    for name, g in zip(NAMES, grads):
        if g is None:
            assert name not in ref
            continue
        of_rows = name in NAMES[:3]
        close(g, ref[name], dtype if of_rows else "f32", name, mags[name].max(initial=0.0) if of_rows else mags[name])
    return (y, u) + tuple(grads)


SHAPES = [(1, 1), (1, 32), (64, 32), (3, 8), (130, 20), (77, 64), (500, 128), (33, 200), (9, 512), (1000, 512), (5, 1024),
          (40, 1031), (7, 2048), (3, 4096), (2, 4100), (700, 4104), (4, 8192), (3, 8191), (257, 33), (2000, 7), (19, 255)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,C", SHAPES)
def test_forward_and_backward(M, C, dtype):
    for kind, gate in (("rms", "full"), ("layer", "row"), ("rms", "row"), ("layer", "none")):
        if C == 1 and gate == "full":
            continue
        check(*draw(M, C, gate, dtype, M + C), dtype, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [32, 37])
def test_one_cotangent_only(C):
    t, d, ct, cd = draw(90, C, "full", "f32", 4)
    check(t, d, [ct[0], None], [cd[0], None], "f32", "rms")
    check(t, d, [None, ct[1]], [None, cd[1]], "f32", "layer")


@pytest.mark.gpu
def test_no_rows():
    t, _, ct, _ = draw(0, 32, "full", "f32", 1)
    y, u, stats = zs.zs_norm_gate_residual(*cuda(t))
    grads = zs.zs_norm_gate_residual_backward(*cuda(ct), *cuda(t), stats)
    assert y.shape == (0, 32) and all(bool((g == 0).all()) for g in grads) and grads[3].shape == (32,)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("C", [64, 65])
def test_rows_of_zeros_and_large_gates(kind, C):
    # a row of zeros has norm 0 whatever eps; gates of +-200 are 1 and 0 without overflow
    t, d, ct, cd = draw(40, C, "full", "f32", 2)
    for a in (t[0], d[0]):
        a[5] = 0
    for a in (t[2], d[2]):
        a[7], a[8] = 200, -200
    out = check(t, d, ct, cd, "f32", kind)
    assert all(bool(torch.isfinite(o).all()) for o in out)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [48, 51, 700])
def test_rows_do_not_mix(C):
    # NaN in one row stays there, in the forward and in the gradients of rows
    t, d, ct, cd = draw(60, C, "full", "bf16", 3)
    want = [o.clone() for o in check(t, d, ct, cd, "bf16", "layer")]
    t[0][11] = float("nan")
    t = cuda(t)
    y, u, stats = zs.zs_norm_gate_residual(*t, eps=EPS, kind="layer")
    grads = zs.zs_norm_gate_residual_backward(*cuda(ct), *t, stats, kind="layer")
    for got, ref in zip((y, u) + grads[:3], want):
        keep = torch.arange(60, device="cuda") != 11
        assert torch.equal(got[keep], ref[keep])
    assert bool(torch.isnan(y[11]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (5, 1)])
def test_row_strides_and_alignment(pad, shift, dtype):
    M, C = 70, 96
    t, d, ct, cd = draw(M, C, "full", dtype, 13)

    def wide(a):
        base = torch.full((a.shape[0], a.shape[1] + pad + shift), float("nan"), dtype=a.dtype, device="cuda")
        base[:, shift:shift + a.shape[1]] = a.cuda()
        return base[:, shift:shift + a.shape[1]]

    check([wide(a) for a in t[:3]] + t[3:], d, [wide(a) for a in ct], cd, dtype, "rms")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,C", [("f32", 20000, 96), ("bf16", 5000, 512), ("f16", 900, 77)])
def test_run_to_run_bits(dtype, M, C):
    t, _, ct, _ = draw(M, C, "row", dtype, 6)
    t, ct = cuda(t), cuda(ct)

    def once():
        y, u, stats = zs.zs_norm_gate_residual(*t, eps=EPS)
        return (y, u, stats) + zs.zs_norm_gate_residual_backward(*ct, *t, stats)

    first = once()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(once(), first))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_against_differences(kind):
    # a step of 1e-2 leaves a truncation error of about 1e-4 of the slope's terms
    t, _, ct, _ = draw(200, 40, "full", "f32", 8)
    t, (dy, du) = cuda(t), cuda(ct)
    y, u, stats = zs.zs_norm_gate_residual(*t, eps=EPS, kind=kind)
    grads = zs.zs_norm_gate_residual_backward(dy, du, *t, stats, kind=kind)

    def loss(ops):
        y, u, _ = zs.zs_norm_gate_residual(*ops, eps=EPS, kind=kind)
        return float((y.double() * dy.double()).sum() + (u.double() * du.double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, g in enumerate(grads):
        v = torch.randn(t[i].shape, generator=gen, device="cuda")
        slope = (loss(t[:i] + [t[i] + 1e-2 * v] + t[i + 1:]) - loss(t[:i] + [t[i] - 1e-2 * v] + t[i + 1:])) / 2e-2
        terms = g.double() * v.double()
        assert abs(slope - float(terms.sum())) <= 1e-3 * float(terms.abs().sum()), NAMES[i]


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(5)
    for kind, cols in (("rms", 6), ("layer", 1)):
        ops = [rng.standard_normal(s) for s in ((4, 6), (4, 6), (4, cols), (6,), (6,), (6,))]
        dy, du = rng.standard_normal((4, 6)), rng.standard_normal((4, 6))
        grads, _ = norm_backward(dy, du, *ops, 1e-3, kind)

        def loss():
            f = norm_forward(*ops, 1e-3, kind)
            return (f["y"] * dy).sum() + (f["u"] * du).sum()

        for at, name in zip(ops, NAMES):
            for i in np.ndindex(at.shape):
                old, e = at[i], 1e-5
                at[i] = old + e
                up = loss()
                at[i] = old - e
                down = loss()
                at[i] = old
                assert abs((up - down) / (2 * e) - grads[name][i]) < 1e-6, (kind, name, i)


def test_argument_checks():
    lib = zs.load()
    ok = dict(dtype=0, kind=0, h=FAKE, h_ld=32, x=FAKE, gate=FAKE, gate_ld=32, cols=32, w=FAKE, eps=1e-6, M=4, C=32, y=FAKE,
              stats=FAKE)

    def fwd(**kw):
        a = {**ok, **kw}
        return lib.zs_norm_gate_residual(a["dtype"], a["kind"], a["h"], a["h_ld"], a["x"], a["C"], a["gate"], a["gate_ld"],
                                         a["cols"], a["w"], a["w"], a["w"], a["eps"], a["M"], a["C"], a["y"], a["y"],
                                         a["stats"], None)

    for kw in (dict(dtype=5), dict(kind=2), dict(C=8193, h_ld=8193, cols=0, gate=None)):
        assert fwd(**kw) == UNSUPPORTED, kw
    for kw in (dict(M=-1), dict(C=0), dict(h=None), dict(x=None), dict(y=None), dict(w=None), dict(cols=7), dict(cols=0),
               dict(gate=None), dict(h_ld=31), dict(gate_ld=31), dict(eps=-1.0), dict(eps=float("nan")), dict(stats=FAKE + 4),
               dict(h=FAKE + 2), dict(dtype=1, y=FAKE + 1)):
        assert fwd(**kw) == INVALID, kw
    assert fwd(M=0, h=None, x=None, y=None) == 0

    ok |= dict(dy=FAKE, dh=FAKE, dgate=FAKE, dw=FAKE, ws=FAKE, bytes=1 << 30)

    def bwd(**kw):
        a = {**ok, **kw}
        return lib.zs_norm_gate_residual_backward(
            a["dtype"], a["kind"], a["dy"], a["C"], a["dy"], a["C"], a["h"], a["h_ld"], a["x"], a["C"], a["gate"],
            a["gate_ld"], a["cols"], a["w"], a["w"], a["w"], a["stats"], a["M"], a["C"], a["dh"], a["dh"], a["dgate"],
            a["dw"], a["dw"], a["dw"], a["ws"], a["bytes"], None)

    need = lib.zs_norm_gate_residual_backward_workspace_bytes(4, 32)
    assert need == 4 * 2 * 32 * 4
    assert lib.zs_norm_gate_residual_backward_workspace_bytes(0, 32) == 0
    for kw in (dict(dh=None), dict(dgate=None), dict(dw=None), dict(stats=None), dict(bytes=need - 1), dict(ws=None),
               dict(ws=FAKE + 16), dict(h_ld=3), dict(M=-2), dict(dy=FAKE + 1)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(kind=-1) == UNSUPPORTED


def test_binding_refusals():
    h, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_norm_gate_residual(h, h, None, w, w, w)
    with pytest.raises(ValueError, match="kind"):
        zs.zs_norm_gate_residual(h, h, None, w, w, w, kind="batch")
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_norm_gate_residual(w, h, None, w, w, w)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["full", "row"])
def test_gates_in_32_bits(gate):
    # With x = 0 and h = 1, y is the gate.  An exponential known to 2 ulps, a sum, a reciprocal, a root known to 2 and
    # three products: 2^-20 of the result, for gates far below zero too.
    C = 96
    z = torch.linspace(-80.0, 20.0, 64 * C).reshape(64, C)
    z = z if gate == "full" else z[:, :1].contiguous()
    ones, zeros, vec = torch.ones(64, C), torch.zeros(64, C), torch.ones(C)
    y, _, _ = zs.zs_norm_gate_residual(*cuda([ones, zeros, z, vec, vec, vec]), eps=0.0)
    want = 1.0 / (1.0 + np.exp(-f64(z)))
    assert (np.abs(f64(y) - want) <= 2.0 ** -20 * want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", [(70, 700), (33, 2048), (9, 4100), (5, 8191), (2, 8192)])
def test_operands_at_different_phases(M, C, dtype):
    # each operand starts at another element offset, so that rows go element by element, over clusters where they are wide
    for kind, gate in (("rms", "full"), ("layer", "row")):
        t, d, ct, cd = draw(M, C, gate, dtype, C + M)

        def at(a, shift):
            base = torch.full((a.numel() + 8,), float("nan"), dtype=a.dtype, device="cuda")
            view = base[shift:shift + a.numel()].view(a.shape)
            view.copy_(a.cuda())
            return view

        check([at(a, i + 1) for i, a in enumerate(t[:3])] + t[3:], d, [at(a, i + 4) for i, a in enumerate(ct)], cd, dtype, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["full", "none"])
def test_infinite_cotangents_stay_infinite(gate):
    """dy of +infinity in one column, whose norm(h) are all positive: its sums over the rows
    are +-infinity by the formula, however many rows the last round of the grid lacks.  A
    row's slots are taken again every few rounds, so there are several of them."""
    for M in (20000, 40000, 61003):
        t, _, (dy, du), _ = draw(M, 32, gate, "f32", 3)
        t[0][:, 5] = t[0][:, 5].abs() + 0.1
        dy[:, 5] = float("inf")
        du.zero_()
        t = cuda(t)
        stats = zs.zs_norm_gate_residual(*t, eps=EPS)[2]
        dw_post, dscale = zs.zs_norm_gate_residual_backward(dy.cuda(), du.cuda(), *t, stats)[3:5]
        assert float(dw_post[5]) == float("inf") * float(t[4][5].sign()), M
        assert float(dscale[5]) == float("inf") * float(t[3][5].sign()), M
        keep = torch.arange(32, device="cuda") != 5
        assert bool(torch.isfinite(dw_post[keep]).all())
