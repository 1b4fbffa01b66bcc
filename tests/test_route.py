"""Routing to experts, against the plain implementation in 64 bits.

The ids have to be those of the scores in 64 bits.  Tolerances, fixed before the first
run: a score is an exponential of a difference known to 2^-24 of itself (below 16 for the
logits drawn here: 2^-20), itself known to 2 ulps, and a sum of at most 1024 terms added up
in 5 + 32 steps: with a quotient and two products 2^-17 of it.  A gradient is a sum of a
product with each of the row's cotangents, each known as well: 2^-16 of the magnitude of its
terms, and the rounding to its type."""
import itertools

import numpy as np
import pytest
import torch

import expert_refs as ref
from equivariant_interatomic_potential_gb300 import zs
from train_refs import HALF_ULP, STEP, f64, held

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20


def check(z, zd, k, bias, score, groups, top_groups, group_top, renormalise, scale, dtype, rng):
    """z on the device, zd its values."""
    b = None if bias is None else torch.from_numpy(bias).cuda()
    how = dict(score=score, renormalise=renormalise, scale=scale)
    ids, w = zs.zs_route(z, k, b, groups=groups, top_groups=top_groups, group_top=group_top, **how)
    bd = None if bias is None else bias.astype(np.float64)
    want_ids, want_w = ref.route(zd, k, bd, score, groups, top_groups, group_top, renormalise, scale)
    got = ids.cpu().numpy()
    assert ids.dtype == torch.int32 and np.array_equal(got, want_ids), np.argwhere(got != want_ids)[:5]
    assert (np.abs(f64(w) - want_w) <= 2.0 ** -17 * np.abs(want_w) + 2.0 ** -140).all()
    g = rng.standard_normal(want_w.shape).astype(np.float32)
    dz = zs.zs_route_backward(torch.from_numpy(g).cuda(), z, ids, **how)
    want, mag = ref.route_backward(g.astype(np.float64), zd, want_ids, score, renormalise, scale)
    assert (np.abs(f64(dz) - want) <= 2.0 ** -16 * mag + HALF_ULP[dtype] * 1.001 * np.abs(want) + STEP[dtype]).all()
    return ids, w, dz


# E, k, groups, top_groups
SIZES = [(1, 1, 1, 1), (2, 1, 1, 1), (8, 2, 1, 1), (8, 8, 1, 1), (60, 4, 4, 2), (61, 3, 1, 1), (64, 6, 8, 3), (160, 6, 8, 3), (256, 8, 8, 4),
         (255, 16, 5, 3), (384, 32, 1, 1), (512, 16, 16, 4), (800, 12, 25, 7), (1024, 32, 32, 32), (1024, 9, 2, 1), (96, 12, 32, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,k,groups,top_groups", SIZES)
def test_choice_weights_and_gradients(E, k, groups, top_groups, dtype):
    rng = np.random.default_rng(E + k)
    for i, (score, biased, renormalise) in enumerate(itertools.product(("softmax", "sigmoid"), (False, True), (False, True))):
        M = (1, 7, 130, 33, 300, 65, 8, 1000)[i]
        z, zd = held(rng.standard_normal((M, E)) * 1.5, dtype)
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if biased else None
        check(z.cuda(), zd, k, bias, score, groups, top_groups, 1 + i % 2, renormalise, 2.5, dtype, rng)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_closed_experts(groups, top_groups, dtype):
    # from none to all experts of a row closed; a group without open experts is behind all others
    rng = np.random.default_rng(11)
    E, M = 32, 400
    share = np.linspace(0, 1, M)[:, None]
    for score, biased, renormalise in itertools.product(("softmax", "sigmoid"), (False, True), (False, True)):
        a = rng.standard_normal((M, E))
        a[rng.random((M, E)) < share] = -np.inf
        a[::50, :24] = -np.inf
        a[-1] = -np.inf
        z, zd = held(a, dtype)
        bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if biased else None
        ids, w, dz = check(z.cuda(), zd, 6, bias, score, groups, top_groups, 2, renormalise, 1.0, dtype, rng)
        none = ids < 0
        assert bool(none[-1].all()) and bool((w[none] == 0).all()) and not bool(dz[-1].any())
        assert not bool(torch.isnan(w).any()) and not bool(torch.isnan(dz).any())
        if biased:                     # a bias of -infinity closes an expert to all rows
            bias[[3, 17]] = -np.inf
            got, _ = zs.zs_route(z.cuda(), 6, torch.from_numpy(bias).cuda(), score, groups, top_groups, 2, renormalise)
            assert not bool(((got == 3) | (got == 17)).any())


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_ties_go_to_the_lowest_index(score, groups):
    rng = np.random.default_rng(12)
    z, zd = held(rng.integers(0, 3, (500, 64)), "bf16")
    for bias in (None, np.zeros(64, np.float32), np.repeat(np.float32([0.5, 0.25]), 32)):
        check(z.cuda(), zd, 8, bias, score, groups, max(groups // 2, 1), 2, True, 1.0, "bf16", rng)
    same = torch.zeros(5, 64, device="cuda")
    ids, w = zs.zs_route(same, 8, score=score)
    assert bool((ids == torch.arange(8, device="cuda")).all()) and bool((w == 0.125).all())
    ids, _ = zs.zs_route(torch.tensor([[0.0, -0.0, 0.0, -0.0]], device="cuda"), 4, score=score)
    assert ids.tolist() == [[0, 1, 2, 3]]


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_closer_than_32_bits(score):
    """Rows whose scores with a bias differ by less than fp32 tells apart, in an order that only 64 bits know: a bias
    that takes away what the logit adds, up to a few 2^-27."""
    rng = np.random.default_rng(13)
    M, E = 300, 48
    z = rng.standard_normal((1, E)).astype(np.float32).repeat(M, 0)
    s = ref.scores(z.astype(np.float64), score)
    bias = (0.5 - s[0]).astype(np.float32)                      # score + bias: 0.5 up to the bias's rounding
    ids, _ = zs.zs_route(torch.from_numpy(z).cuda(), 12, torch.from_numpy(bias).cuda(), score)
    a = s + bias.astype(np.float64)
    assert np.abs(a - 0.5).max() < 2.0 ** -24
    assert np.array_equal(ids.cpu().numpy(), np.argsort(-a, axis=1, kind="stable")[:, :12])
    for group_top in (1, 2):                                    # and groups of them
        ids, _ = zs.zs_route(torch.from_numpy(z).cuda(), 12, torch.from_numpy(bias).cuda(), score, 8, 3, group_top)
        want, _ = ref.route(z.astype(np.float64), 12, bias.astype(np.float64), score, 8, 3, group_top, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top_groups", [(256, 8, 8, 4), (1024, 8, 32, 5), (96, 4, 32, 4), (40, 3, 20, 9)])
def test_groups_that_are_alike(score, E, k, groups, top_groups):
    """Rows of one logit (a router that has learnt nothing), with a few that stand out, and groups that are alike but for
    one logit's last bit: the border goes by the groups' numbers, or by what only 64 bits tell."""
    rng = np.random.default_rng(16)
    M, per = 64, E // groups
    z = np.zeros((M, E), np.float32)
    for i in range(M):
        stand_out = rng.permutation(groups)[: i % top_groups]
        z[i, stand_out * per] = 1.0                                            # some groups are in for sure
        if i % 3 == 0:
            z[i] += np.tile((np.arange(per) * 0.01).astype(np.float32), groups)     # groups alike, experts not
        if i % 5 == 0:
            at = rng.permutation(groups)[: groups // 2] * per + per - 1
            z[i, at] = np.nextafter(z[i, at], np.float32(2))
    for bias in (None, np.zeros(E, np.float32), np.tile((rng.standard_normal(per) * 0.01).astype(np.float32), groups)):
        for group_top in (1, 2):
            check(torch.from_numpy(z).cuda(), z.astype(np.float64), k, bias, score, groups, top_groups, group_top, True, 1.0, "f32", rng)


@pytest.mark.gpu
@pytest.mark.parametrize("renormalise", [True, False])
def test_far_logits(renormalise):
    # logits whose scores leave fp32's range: renormalised weights are ratios all the same
    z = torch.tensor([[-300.0, -301.0, -400.0, -1000.0], [200.0, 100.0, -100.0, 0.0], [-90.0, -95.0, -104.0, -3e38], [3e38, -3e38, 0.0, 1.0]],
                     device="cuda")
    zd = f64(z)
    for score in ("softmax", "sigmoid"):
        ids, w = zs.zs_route(z, 3, score=score, renormalise=renormalise)
        chosen = np.take_along_axis(zd, ids.cpu().numpy(), 1)
        assert np.array_equal(ids.cpu().numpy(), np.argsort(-zd, 1, kind="stable")[:, :3])
        log = -np.logaddexp(0, -chosen) if score == "sigmoid" else chosen - np.logaddexp.reduce(zd, 1)[:, None]
        if renormalise:
            log = log - np.logaddexp.reduce(log, 1)[:, None]
        # an exponent of up to 300 is known to 2^-24 of itself
        assert (np.abs(f64(w) - np.exp(log)) <= 2.0 ** -15 * np.exp(log) + 2.0 ** -126).all()
        dz = zs.zs_route_backward(torch.ones_like(w), z, ids, score, renormalise)
        assert bool(torch.isfinite(dz).all())


@pytest.mark.gpu
def test_lowest_values():
    # a mask of the type's lowest value instead of -infinity leaves experts open, behind all others
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        z = torch.full((3, 6), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        z[0, 4] = 1.0
        z[1, 2:4] = -5.0
        for score in ("softmax", "sigmoid"):
            ids, w = zs.zs_route(z, 3, score=score)
            assert ids.tolist() == [[4, 0, 1], [2, 3, 0], [0, 1, 2]]
            assert torch.allclose(w.cpu(), torch.tensor([[1.0, 0, 0], [0.5, 0.5, 0], [1 / 3] * 3]), atol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
def test_nan_is_the_largest(bias):
    z = torch.randn(20, 40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    b = torch.zeros(40, device="cuda") if bias else None
    want = zs.zs_route(z, 5, b, "sigmoid")
    z[3, 17] = float("nan")
    z[4] = float("nan")
    z[5, 2] = -float("nan")
    ids, w = zs.zs_route(z, 5, b, "sigmoid")
    assert int(ids[3, 0]) == 17 and ids[4].tolist() == [0, 1, 2, 3, 4] and int(ids[5, 0]) == 2
    assert bool(torch.isnan(w[3:6]).all())
    keep = [i for i in range(20) if i not in (3, 4, 5)]
    assert torch.equal(ids[keep], want[0][keep]) and torch.equal(w[keep], want[1][keep])
    z[6, 1] = float("inf")
    ids, w = zs.zs_route(z, 5, b, "sigmoid", renormalise=False)
    assert int(ids[6, 0]) == 1 and float(w[6, 0]) == 1.0
    half = torch.randn(9, 40, device="cuda").bfloat16()    # 16-bit logits, whose keys are exact
    half[3, 17], half[5] = float("nan"), float("nan")
    ids, w = zs.zs_route(half, 5, b, "sigmoid")
    assert int(ids[3, 0]) == 17 and ids[5].tolist() == [0, 1, 2, 3, 4] and bool(torch.isnan(w[[3, 5]]).all())
    assert not bool(torch.isnan(w[[0, 1, 2, 4, 6, 7, 8]]).any())
    for score in ("softmax", "sigmoid"):           # ids stay those of experts, each once
        ids, _ = zs.zs_route(z, 5, b, score, 4, 2, 2)
        assert bool(((ids >= 0) & (ids < 40)).all()) and all(len(set(r)) == 5 for r in ids.tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (5, 1)])
def test_row_strides_and_alignment(pad, shift, dtype):
    rng = np.random.default_rng(14)
    z, zd = held(rng.standard_normal((90, 64)), dtype)
    base = torch.full((90, 64 + pad + shift), float("nan"), dtype=z.dtype, device="cuda")
    base[:, shift:shift + 64] = z.cuda()
    check(base[:, shift:shift + 64], zd, 6, (rng.standard_normal(64) * 0.1).astype(np.float32), "sigmoid", 8, 4, 2, True, 1.0, dtype, rng)


@pytest.mark.gpu
def test_ids_named_twice_or_outside():
    # a choice that is not the router's: gradients of an expert named twice add up, ids outside add nothing
    z = torch.randn(4, 10, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    ids = torch.tensor([[1, 1, 3], [-1, 10, 4], [2 ** 31 - 1, -(2 ** 31), 0], [9, 9, 9]], dtype=torch.int32, device="cuda")
    g = torch.randn(4, 3, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    zd, gd = f64(z), f64(g)
    kept = np.where((f64(ids) >= 0) & (f64(ids) < 10), f64(ids), -1).astype(np.int64)
    for score, renormalise in itertools.product(("softmax", "sigmoid"), (False, True)):
        dz = zs.zs_route_backward(g, z, ids, score, renormalise, 2.0)
        want, mag = ref.route_backward(gd, zd, kept, score, renormalise, 2.0)
        assert (np.abs(f64(dz) - want) <= 2.0 ** -16 * mag).all()


@pytest.mark.gpu
def test_run_to_run_bits():
    z = torch.randn(5000, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    b = torch.randn(256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)) * 0.1

    def once():
        ids, w = zs.zs_route(z, 8, b, "sigmoid", 8, 4, 2)
        return ids, w, zs.zs_route_backward(w, z, ids, "sigmoid")

    first = once()
    for _ in range(4):
        assert all(torch.equal(a, c) for a, c in zip(first, once()))


def test_reference_gradient_against_differences():
    rng = np.random.default_rng(15)
    for kind, renormalise in itertools.product(("softmax", "sigmoid"), (False, True)):
        z, g = rng.standard_normal((3, 7)), rng.standard_normal((3, 3))
        z[1, 4] = -np.inf
        ids, _ = ref.route(z, 3, None, kind, 1, 1, 1, renormalise, 2.0)
        ids[2, 2] = -1
        got, _ = ref.route_backward(g, z, ids, kind, renormalise, 2.0)
        for i in np.ndindex(z.shape):
            if np.isneginf(z[i]):
                assert got[i] == 0
                continue
            up, down = z.copy(), z.copy()
            up[i] += 1e-6
            down[i] -= 1e-6
            loss = [(ref.route_weights(a, ids, kind, renormalise, 2.0) * g).sum() for a in (up, down)]
            assert abs((loss[0] - loss[1]) / 2e-6 - got[i]) < 1e-7


@pytest.mark.gpu
def test_no_rows():
    ids, w = zs.zs_route(torch.zeros(0, 8, device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2)
    assert zs.zs_route_backward(w, torch.zeros(0, 8, device="cuda"), ids).shape == (0, 8)


def test_argument_checks():
    lib = zs.load()
    ok = dict(dtype=0, score=0, z=FAKE, ld=64, bias=None, M=4, E=64, k=4, groups=8, top=2, group_top=2, scale=1.0, ids=FAKE, w=FAKE)

    def fwd(**kw):
        a = {**ok, **kw}
        return lib.zs_route(a["dtype"], a["score"], a["z"], a["ld"], a["bias"], a["M"], a["E"], a["k"], a["groups"], a["top"], a["group_top"], 1,
                            a["scale"], a["ids"], a["w"], None)

    for kw in (dict(dtype=4), dict(score=2), dict(E=1025, ld=1025, groups=1, top=1), dict(E=66, k=33, groups=1, top=1, ld=66),
               dict(groups=64, top=64, k=4), dict(E=1023, ld=1023, groups=3, top=2)):
        assert fwd(**kw) == UNSUPPORTED, kw
    for kw in (dict(M=-1), dict(E=0), dict(k=0), dict(k=65), dict(k=17), dict(groups=0), dict(groups=7), dict(top=0), dict(top=9), dict(group_top=3),
               dict(group_top=0), dict(z=None), dict(ids=None), dict(w=None), dict(ld=63), dict(z=FAKE + 2), dict(bias=FAKE + 1),
               dict(scale=float("nan")), dict(dtype=1, z=FAKE + 1), dict(M=1 << 31)):
        assert fwd(**kw) == INVALID, kw
    assert fwd(M=0, z=None, ids=None, w=None) == 0
    ok |= dict(g=FAKE, dz=FAKE)

    def bwd(**kw):
        a = {**ok, **kw}
        return lib.zs_route_backward(a["dtype"], a["score"], a["g"], a["z"], a["ld"], a["ids"], a["M"], a["E"], a["k"], 1, a["scale"], a["dz"], None)

    assert bwd(score=-1) == UNSUPPORTED
    for kw in (dict(g=None), dict(ids=None), dict(dz=None), dict(z=None), dict(k=0), dict(ld=1), dict(dz=FAKE + 2), dict(g=FAKE + 2)):
        assert bwd(**kw) == INVALID, kw


def test_binding_refusals():
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="score"):
        zs.zs_route(z, 2, score="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_route(z, 2)
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_route(z[0], 2)
    with pytest.raises(ValueError, match="score"):
        zs.zs_route_backward(z, z, z, score="tanh")


@pytest.mark.gpu
def test_refusals_on_the_device():
    z = torch.zeros(4, 64, device="cuda")
    for kw in (dict(k=0), dict(k=65), dict(k=1 << 32), dict(k=2, groups=0), dict(k=2, groups=1 << 33), dict(k=2, group_top=3),
               dict(k=2, top_groups=-1, groups=4), dict(k=2, bias=torch.zeros(63, device="cuda")), dict(k=2, bias=torch.zeros(64).double())):
        with pytest.raises(ValueError):
            zs.zs_route(z, **kw)
    for kw in (dict(k=33), dict(k=2, groups=5), dict(k=20, groups=4, top_groups=1), dict(k=2, groups=4, top_groups=5), dict(k=2, scale=float("inf"))):
        with pytest.raises(zs.ZsError):
            zs.zs_route(z, **kw)
    with pytest.raises(TypeError):
        zs.zs_route(z, 2.0)
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="dweights"):
        zs.zs_route_backward(torch.zeros(4, 3, device="cuda"), z, ids)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (3, 3), (4, 2), (8, 2), (8, 8), (13, 4), (16, 16), (17, 4)])
def test_many_rows_of_few_experts(E, k, dtype):
    # closed experts, ties, NaN, rows at strides and views off 16-byte boundaries among them
    rng = np.random.default_rng(E + 7 * k)
    M = 4099
    a = rng.standard_normal((M, E)) * 1.5
    a[rng.random((M, E)) < np.linspace(0, 0.5, M)[:, None]] = -np.inf
    a[-1] = -np.inf
    a[5:400] = rng.integers(0, 3, (395, E))
    z, zd = held(a, dtype)
    z = z.cuda()
    for score, biased, renormalise in itertools.product(("softmax", "sigmoid"), (False, True), (False, True)):
        bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if biased else None
        ids, w, dz = check(z, zd, k, bias, score, 1, 1, 1, renormalise, 2.5, dtype, rng)
        assert bool((ids[-1] == -1).all()) and not bool(w[-1].any()) and not bool(dz[-1].any())
        wide = torch.full((M, E + 3), float("nan"), dtype=z.dtype, device="cuda")
        wide[:, 1:1 + E] = z
        view = wide[:, 1:1 + E]
        how = dict(score=score, renormalise=renormalise, scale=2.5)
        again = zs.zs_route(view, k, None if bias is None else torch.from_numpy(bias).cuda(), **how)
        assert torch.equal(again[0], ids) and torch.equal(again[1], w)
        g = torch.ones_like(w)
        assert torch.equal(zs.zs_route_backward(g, view, ids, **how), zs.zs_route_backward(g, z, ids, **how))
        # a row of NaN is its own affair, and so is one of infinity
        bad = z.clone()
        bad[77] = float("nan")
        bad[78, 0] = float("inf")
        got, gw = zs.zs_route(bad, k, None if bias is None else torch.from_numpy(bias).cuda(), **how)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[77:79] = False
        assert torch.equal(got[keep], ids[keep]) and torch.equal(gw[keep], w[keep])
        assert got[77].tolist() == list(range(k)) and bool(torch.isnan(gw[77]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_few_experts_closer_than_32_bits(score):
    # as above, a thread's row: rows that 64 bits have to tell, beside others that they need not
    rng = np.random.default_rng(17)
    M, E, k = 4200, 12, 5
    z = rng.standard_normal((M, E)).astype(np.float32)
    z[::3] = z[0]
    s = ref.scores(z[:1].astype(np.float64), score)
    bias = (0.5 - s[0]).astype(np.float32)
    ids, _ = zs.zs_route(torch.from_numpy(z).cuda(), k, torch.from_numpy(bias).cuda(), score)
    a = ref.scores(z.astype(np.float64), score) + bias.astype(np.float64)
    assert np.array_equal(ids.cpu().numpy(), np.argsort(-a, axis=1, kind="stable")[:, :k])


@pytest.mark.gpu
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_few_experts_named_twice(score, renormalise):
    # the gradient of ids that hold an expert twice, or none: cotangents of the same expert add up, as for few rows
    torch.manual_seed(3)
    z, g = torch.randn(4100, 8, device="cuda"), torch.randn(4100, 3, device="cuda")
    ids = torch.randint(-1, 8, (4100, 3), device="cuda", dtype=torch.int32)
    many = zs.zs_route_backward(g, z, ids, score, renormalise)
    few = torch.cat([zs.zs_route_backward(g[i:i + 100], z[i:i + 100], ids[i:i + 100], score, renormalise) for i in range(0, 4100, 100)])
    assert bool(((many - few).abs() <= 2.0 ** -18 * (1 + g.abs().sum(1, keepdim=True))).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E", [(15, 13), (5000, 13), (300, 64), (70, 1000)])
def test_only_choice(M, E, score, dtype):
    # the renormalised weight of the only choice is 1, whatever its score, and the logits have no gradient: exactly
    z = (torch.randn(M, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) * 3).to(dtype)
    ids, w = zs.zs_route(z, 1, score=score, scale=2.5)
    assert bool((w == 2.5).all())
    g = torch.randn(M, 1, device="cuda")
    assert not bool(zs.zs_route_backward(g, z, ids, score, True, 2.5).any())
    z[:, 1:] = -float("inf")                       # and of the only one that is open
    ids, w = zs.zs_route(z, 4, score=score, scale=2.5)
    assert bool((w[:, 0] == 2.5).all()) and not bool(w[:, 1:].any())
    assert not bool(zs.zs_route_backward(torch.randn(M, 4, device="cuda"), z, ids, score, True, 2.5).any())


@pytest.mark.gpu
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,k,groups,top_groups", [(8, 3, 4, 2), (64, 6, 8, 3), (256, 8, 8, 4), (96, 4, 32, 6)])
def test_groups_of_one_small_score_with_few_open(E, k, groups, top_groups, group_top):
    """Scores that are alike and so small that 32 bits do not tell one from the sum of two: a group with a single open
    expert is behind those with two.  Beside them closed groups and such that are in for sure."""
    rng = np.random.default_rng(E + group_top)
    M, per = 96, E // groups
    z = np.zeros((M, groups, per), np.float32)
    for i in range(M):
        open_one = rng.permutation(groups)[: 1 + i % (groups - 1)]
        for g in open_one:
            z[i, g, rng.permutation(per)[1:]] = -np.inf
        if i % 4 == 1:
            z[i, rng.integers(groups)] = -np.inf
    low, high = z.copy(), z.copy()
    low[np.isfinite(z)] = -30.0                                  # a sigmoid of 2^-43
    for i in range(M):
        high[i, i % groups] = 20.0                               # the others' softmax is below 2^-28
    some = (rng.standard_normal(E) * 0.01).astype(np.float32)
    for score, a in (("softmax", high), ("sigmoid", low)):
        a = a.reshape(M, E)
        for bias in (None, np.zeros(E, np.float32), some):
            for renormalise in (True, False):
                check(torch.from_numpy(a).cuda(), a.astype(np.float64), k, bias, score, groups, top_groups, group_top, renormalise, 1.0,
                      "f32", rng)


@pytest.mark.gpu
def test_a_single_open_expert_against_two():
    z = torch.tensor([[20.0, 20.0, 0.0, -float("inf"), 0.0, 0.0, 0.0, 0.0]], device="cuda")
    ids, _ = zs.zs_route(z, 3, torch.zeros(8, device="cuda"), "softmax", 4, 2, 2)
    assert ids.tolist() == [[0, 1, 4]]


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(64, 1), (96, 4), (260, 8), (1000, 32)])
def test_more_alike_than_are_looked_at(E, k):
    """Most experts of a row are alike, and a few behind them are larger by what only 64 bits tell, or the logits' last bits."""
    rng = np.random.default_rng(E)
    M = 40
    z = np.full((M, E), -30.0, np.float32)
    for i in range(1, M):
        at = rng.permutation(E)[:i % 7]
        z[i, at] = np.nextafter(z[i, at], np.float32(0))
    check(torch.from_numpy(z).cuda(), z.astype(np.float64), k, None, "sigmoid", 1, 1, 1, True, 1.0, "f32", rng)
    check(torch.from_numpy(z).cuda(), z.astype(np.float64), k, np.zeros(E, np.float32), "softmax", 1, 1, 1, True, 1.0, "f32", rng)
    high = np.full((M, E), 18.5, np.float32)                     # sigmoids of 1 but for 2^-27
    for i in range(1, M):
        high[i, rng.permutation(E)[:i % 7]] = 27.25
    for groups, top in ((1, 1), (4, 2)):
        check(torch.from_numpy(high).bfloat16().cuda(), high.astype(np.float64), k, np.zeros(E, np.float32), "sigmoid", groups, top, 1, False,
              1.0, "bf16", rng)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(11, 1), (16, 3), (8, 7), (3, 1)])
def test_few_experts_alike_behind_the_choice(E, k):
    """A thread's row: behind the choice several scores that 32 bits do not tell from its last one, the larger not first."""
    rng = np.random.default_rng(E)
    M = 4200
    a = np.where(rng.random((M, E)) < 0.4, 18.5, -3.0)           # sigmoids of 1 but for 2^-27
    a[rng.random((M, E)) < 0.2] = 27.25
    a[1::7, 1:] = 18.5
    a[2::7] = -30.0
    a[2::7, E - 1] = -29.5
    z, zd = held(a, "bf16")
    for bias in (np.zeros(E, np.float32), np.full(E, 0.75, np.float32)):
        check(z.cuda(), zd, k, bias, "sigmoid", 1, 1, 1, False, 1.0, "bf16", rng)
    peak = np.where(a > 0, 20.0, a)
    peak[:, 0] = 60.0                                            # a softmax below 2^-57 for the others
    z, zd = held(peak, "bf16")
    check(z.cuda(), zd, k, np.zeros(E, np.float32), "softmax", 1, 1, 1, False, 1.0, "bf16", rng)


@pytest.mark.gpu
@pytest.mark.parametrize("per", [2, 10])
def test_groups_far_below_the_largest_logit(per):
    """Scores that are 0 in 64 bits, beside a logit that is 746 or more larger, are alike whatever their logits; so are those
    that a division by the row's sum makes alike (2^-1074 and three times that over eight)."""
    rng = np.random.default_rng(per)
    for far in (1000.0, 746.0):
        z = np.zeros((1, 4, per), np.float32)
        z[0, 0] = far
        z[0, 2] = 1.0 if far == 1000.0 else 0.25
        z = z.reshape(1, -1)
        for group_top in (1, 2):
            check(torch.from_numpy(z).cuda(), z.astype(np.float64), per + 1, None, "softmax", 4, 2, group_top, True, 1.0, "f32", rng)
    unit = np.float32(1074 * np.log(2))                          # exp(-unit): 2^-1074
    z = np.zeros((40, 4, 8), np.float32)                         # a sum of eight and a little
    for i in range(40):
        z[i, 1:] = -(unit - np.log(rng.integers(1, 4, (3, 8))).astype(np.float32))
    z = z.reshape(40, 32)
    assert np.array_equal(np.unique(np.exp(z[:, 8:].astype(np.float64))), np.array([1, 2, 3]) * 2.0 ** -1074)
    for top_groups, k in ((1, 8), (2, 16), (3, 20)):
        for group_top in (1, 2):
            check(torch.from_numpy(z).cuda(), z.astype(np.float64), k, None, "softmax", 4, top_groups, group_top, False, 1.0, "f32", rng)
