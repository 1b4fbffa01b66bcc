"""The way of rows to several experts and back, against the plain implementation in 64 bits.

Copies are exact.  Tolerances of the rest, fixed before the first run: a combined row is a
sum of k products in fp32, k + 1 half ulps of the sum of their magnitudes, then rounded; a
weight's gradient is a sum of C products in some order: 1e-5 of the sum of their magnitudes;
dh is one product, rounded in fp32 and to its type."""
import numpy as np
import pytest
import torch

import expert_refs as ref
from equivariant_interatomic_potential_gb300 import zs
from train_refs import HALF_ULP, STEP, f64, held

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20


def draw_ids(rng, M, k, E, dropped=0.1):
    """k different experts a row, some dropped, some of a number that is none."""
    ids = np.argsort(rng.random((M, E)) + rng.standard_normal(E) * 0.3, axis=1)[:, :k] if M else np.zeros((0, k), np.int64)
    out = rng.random((M, k))
    ids = np.where(out < dropped, -1, ids)
    return np.where(out > 1 - dropped / 4, E + 3, ids)


def close(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off"


def check(ids, E, x, xd, h, hd, dy, dyd, wd, dtype):
    M, k = ids.shape
    half, step = HALF_ULP[dtype] * 1.001, STEP[dtype]
    flat = torch.from_numpy(ids.astype(np.int32)).cuda()
    row_ptr, perm, _ = zs.zs_build_csr(flat.view(-1), E)
    weights = torch.from_numpy(wd.astype(np.float32)).cuda()
    wd = f64(weights)
    xs, slot = zs.zs_dispatch(x, row_ptr, perm, k)
    want, want_slot = ref.dispatch(xd, ids, E)
    assert np.array_equal(f64(xs), want) and np.array_equal(slot.cpu().numpy(), want_slot)
    y = zs.zs_combine(h, slot, weights)
    want, mag = ref.combine(hd, want_slot, wd)
    close(y, want, (k + 1) * 2.0 ** -24 * mag + half * np.abs(want) + step, "y")
    dx = zs.zs_combine(h, slot)
    want, mag = ref.combine(hd, want_slot)
    close(dx, want, (k + 1) * 2.0 ** -24 * mag + half * np.abs(want) + step, "dx")
    dh, dw = zs.zs_combine_backward(dy, h, slot, weights, row_ptr)
    want, want_dw, mag = ref.combine_backward(dyd, hd, want_slot, wd)
    close(dh, want, (half + 2.0 ** -24) * np.abs(want) + step, "dh")
    close(dw, want_dw, 1e-5 * mag, "dweights")
    return xs, slot, y, dx, dh, dw


def draw(M, k, E, C, dtype, seed, dropped=0.1):
    rng = np.random.default_rng(seed)
    ids = draw_ids(rng, M, k, E, dropped)
    (x, xd), (h, hd), (dy, dyd) = (held(rng.standard_normal((n, C)), dtype) for n in (M, M * k, M))
    return ids, E, x.cuda(), xd, h.cuda(), hd, dy.cuda(), dyd, rng.standard_normal((M, k))


SHAPES = [(1, 1, 1, 1), (1, 8, 256, 4096), (7, 2, 3, 33), (64, 3, 8, 32), (1000, 8, 64, 96), (257, 9, 16, 40), (33, 20, 32, 1031), (4097, 3, 37, 301),
          (300, 1, 5, 2048), (2, 12, 400, 8200), (5000, 2, 4, 8), (40, 31, 31, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,k,E,C", SHAPES)
def test_there_and_back(M, k, E, C, dtype):
    for dropped in (0.0, 0.2, 1.0):
        check(*draw(M, k, E, C, dtype, M + k + C, dropped), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,k,E,C", [(3000, 8, 64, 256), (5001, 2, 16, 600), (9000, 4, 300, 129)])
def test_more_than_the_small_calls(M, k, E, C, dtype):
    # rows of xs of 8 MB and more: x is read once for all of a row's choices
    check(*draw(M, k, E, C, dtype, M, 0.1), dtype)


@pytest.mark.gpu
def test_no_rows():
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    row_ptr, perm, _ = zs.zs_build_csr(none, 4)
    xs, slot = zs.zs_dispatch(torch.zeros(0, 8, device="cuda"), row_ptr, perm, 2)
    assert xs.shape == (0, 8) and slot.shape == (0, 2)
    w = torch.zeros(0, 2, device="cuda")
    assert zs.zs_combine(xs, slot, w).shape == (0, 8)
    dh, dw = zs.zs_combine_backward(xs, xs, slot, w, row_ptr)
    assert dh.shape == (0, 8) and dw.shape == (0, 2)
    y = zs.zs_combine(xs, torch.zeros(3, 2, dtype=torch.int32, device="cuda"))      # slots of no row
    assert y.shape == (3, 8) and not bool(y.any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (5, 1), (3, 0)])
def test_row_strides_and_alignment(pad, shift, dtype):
    ids, E, x, xd, h, hd, dy, dyd, wd = draw(120, 4, 9, 96, dtype, 3)

    def wide(a):
        base = torch.full((a.shape[0], a.shape[1] + pad + shift), float("nan"), dtype=a.dtype, device="cuda")
        base[:, shift:shift + a.shape[1]] = a
        return base[:, shift:shift + a.shape[1]]

    check(ids, E, wide(x), xd, wide(h), hd, wide(dy), dyd, wd, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 77])
def test_rows_behind_the_last_expert_are_not_read(C):
    # NaN in h behind the last expert's rows, in weights and rows of dropped assignments: no trace of them
    ids, E, x, xd, h, hd, dy, dyd, wd = draw(300, 3, 7, C, "f32", 5, 0.3)
    want = check(ids, E, x, xd, h, hd, dy, dyd, wd, "f32")
    row_ptr, _, slot = ref.slots(ids, E)
    h = h.clone()
    h[int(row_ptr[E]):] = float("nan")
    wd = np.where(slot < 0, np.nan, wd)
    flat = torch.from_numpy(ids.astype(np.int32)).cuda()
    rp, perm, _ = zs.zs_build_csr(flat.view(-1), E)
    weights = torch.from_numpy(wd.astype(np.float32)).cuda()
    _, slot = zs.zs_dispatch(x, rp, perm, 3)
    got = (zs.zs_combine(h, slot, weights), zs.zs_combine(h, slot), *zs.zs_combine_backward(dy, h, slot, weights, rp))
    assert all(torch.equal(a, b) for a, b in zip(got, want[2:]))


@pytest.mark.gpu
def test_slots_and_positions_that_are_none():
    # slots outside h add nothing; a perm or row_ptr that no CSR is reads nothing outside the operands
    h = torch.randn(20, 40, device="cuda")
    slot = torch.tensor([[3, -1], [20, 19], [2 ** 31 - 1, -(2 ** 31)], [5, 5]], dtype=torch.int32, device="cuda")
    y = zs.zs_combine(h, slot, torch.ones(4, 2, device="cuda"))
    assert torch.equal(y[0], h[3]) and torch.equal(y[1], h[19]) and not bool(y[2].any()) and torch.equal(y[3], h[5] + h[5])
    x = torch.randn(50, 40, device="cuda")
    gen = torch.Generator().manual_seed(1)
    for lo, hi in ((-(2 ** 31), 2 ** 31 - 1), (0, 130)):
        row_ptr, perm = (torch.randint(lo, hi, (n,), generator=gen).int().cuda() for n in (6, 100))
        assert zs.zs_dispatch(x, row_ptr, perm, 2)[0].shape == (100, 40)
        row_ptr[-1] = lo
        hh = torch.randn(100, 40, device="cuda")
        slot = torch.arange(100, dtype=torch.int32, device="cuda").view(50, 2)
        assert zs.zs_combine_backward(x, hh, slot, torch.ones(50, 2, device="cuda"), row_ptr)[0].shape == (100, 40)
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,k,E,C", [("f32", 3000, 4, 16, 96), ("bf16", 2000, 8, 64, 1024), ("f16", 999, 3, 7, 301)])
def test_run_to_run_bits(dtype, M, k, E, C):
    ids, E, x, _, h, _, dy, _, wd = draw(M, k, E, C, dtype, 6)
    flat = torch.from_numpy(ids.astype(np.int32)).cuda().view(-1)
    weights = torch.from_numpy(wd.astype(np.float32)).cuda()

    def once():
        row_ptr, perm, _ = zs.zs_build_csr(flat, E)
        xs, slot = zs.zs_dispatch(x, row_ptr, perm, k)
        return xs, slot, zs.zs_combine(h, slot, weights), *zs.zs_combine_backward(dy, h, slot, weights, row_ptr)

    first = once()
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


@pytest.mark.gpu
def test_gradients_against_differences():
    ids, E, x, _, h, _, dy, _, wd = draw(200, 3, 8, 48, "f32", 8)
    flat = torch.from_numpy(ids.astype(np.int32)).cuda()
    row_ptr, perm, _ = zs.zs_build_csr(flat.view(-1), E)
    w = torch.from_numpy(wd.astype(np.float32)).cuda()
    _, slot = zs.zs_dispatch(x, row_ptr, perm, 3)
    dh, dw = zs.zs_combine_backward(dy, h, slot, w, row_ptr)
    gen = torch.Generator(device="cuda").manual_seed(9)
    vh, vw, vx = (torch.randn(t.shape, device="cuda", generator=gen) for t in (h, w, x))
    loss = lambda hh, ww: float((zs.zs_combine(hh, slot, ww).double() * dy.double()).sum())  # noqa: E731  (linear in each)
    scale = float((dy.double().abs().sum()))
    assert abs(loss(h + vh, w) - loss(h, w) - float((dh.double() * vh.double()).sum())) <= 1e-5 * scale
    assert abs(loss(h, w + vw) - loss(h, w) - float((dw.double() * vw.double()).sum())) <= 1e-5 * scale
    spread = lambda xx: float((zs.zs_dispatch(xx, row_ptr, perm, 3)[0].double() * h.double()).sum())  # noqa: E731
    dx = zs.zs_combine(h, slot)
    held_h = h.double()[: int(row_ptr[-1])]
    assert abs(spread(x + vx) - spread(x) - float((dx.double() * vx.double()).sum())) <= 1e-5 * float(held_h.abs().sum())


@pytest.mark.gpu
def test_rows_past_2_31_elements():
    # M * k * C above 2^31 elements: the last rows travel like the first
    M, k, C = 2 ** 17 + 3, 8, 2056
    x = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    x[-2:] = torch.randn(2, C, device="cuda").to(torch.bfloat16)
    ids = torch.full((M, k), 1, dtype=torch.int32, device="cuda")
    ids[:, 0] = 0
    row_ptr, perm, _ = zs.zs_build_csr(ids.view(-1), 2)
    xs, slot = zs.zs_dispatch(x, row_ptr, perm, k)
    assert torch.equal(xs[-k + 1:], x[-1:].expand(k - 1, C)) and torch.equal(xs[M - 2:M], x[-2:])
    assert int(slot[-1, -1]) == M * k - 1
    w = torch.zeros(M, k, device="cuda")
    w[:, 1] = 1.0
    y = zs.zs_combine(xs, slot, w)
    assert torch.equal(y[-2:], x[-2:]) and not bool(y[:-2].any())
    del y
    dh, dw = zs.zs_combine_backward(x, xs, slot, w, row_ptr)
    assert torch.equal(dh[int(slot[-1, 1])], x[-1]) and not bool(dh[-1].any())
    norm = x[-2:].double().square().sum(1)
    assert bool(((dw[-2:].double() - norm[:, None]).abs() <= 1e-5 * norm[:, None]).all()) and not bool(dw[:-2].any())


def test_argument_checks():
    lib = zs.load()
    ok = dict(dtype=0, x=FAKE, ld=32, rp=FAKE, perm=FAKE, M=4, k=2, G=3, C=32, xs=FAKE, slot=FAKE, R=8, w=FAKE, y=FAKE, y_ld=32, dw=FAKE)

    def there(**kw):
        a = {**ok, **kw}
        return lib.zs_dispatch(a["dtype"], a["x"], a["ld"], a["rp"], a["perm"], a["M"], a["k"], a["G"], a["C"], a["xs"], a["slot"], None)

    def back(**kw):
        a = {**ok, **kw}
        return lib.zs_combine(a["dtype"], a["x"], a["ld"], a["slot"], a["w"], a["M"], a["k"], a["R"], a["C"], a["y"], a["y_ld"], None)

    def grad(**kw):
        a = {**ok, **kw}
        return lib.zs_combine_backward(a["dtype"], a["y"], a["y_ld"], a["x"], a["ld"], a["slot"], a["w"], a["rp"], a["M"], a["k"], a["G"], a["C"],
                                       a["xs"], a["dw"], None)

    for f in (there, back, grad):
        assert f(dtype=3) == UNSUPPORTED
        for kw in (dict(M=-1), dict(k=0), dict(C=0), dict(x=None), dict(ld=31), dict(x=FAKE + 2), dict(slot=None), dict(slot=FAKE + 1),
                   dict(M=1 << 30, k=2, R=4), dict(M=1 << 31)):
            assert f(**kw) == INVALID, (f.__name__, kw)
        assert f(M=0, x=None, xs=None, slot=None, y=None, w=None, rp=None, perm=None, dw=None, R=0) == 0
    for f in (there, grad):
        for kw in (dict(G=-1), dict(rp=None), dict(xs=None), dict(rp=FAKE + 2), dict(xs=FAKE + 1)):
            assert f(**kw) == INVALID, kw
    assert there(perm=None) == INVALID
    for kw in (dict(y=None), dict(y_ld=31), dict(R=-1), dict(w=FAKE + 2)):
        assert back(**kw) == INVALID, kw
    for kw in (dict(w=None), dict(dw=None), dict(y=None), dict(y_ld=3), dict(dw=FAKE + 2)):
        assert grad(**kw) == INVALID, kw


def test_binding_refusals():
    x, i = torch.zeros(4, 8), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_dispatch(x, i, i, 2)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_combine(x, i.view(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_combine_backward(x[:2], x, i[:4].view(2, 2), torch.zeros(2, 2), i)
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_combine(x, i)


@pytest.mark.gpu
def test_refusals_on_the_device():
    x, i = torch.zeros(4, 8, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    for call in (lambda: zs.zs_dispatch(x, i, i, 3), lambda: zs.zs_dispatch(x, i, i, 0), lambda: zs.zs_dispatch(x, i, i, 1 << 33),
                 lambda: zs.zs_dispatch(x, i.long(), i, 2), lambda: zs.zs_dispatch(x, i[:0], i, 2),
                 lambda: zs.zs_combine(x, i.view(4, 2), torch.zeros(4, 3, device="cuda")),
                 lambda: zs.zs_combine(x, i.view(4, 2).long()), lambda: zs.zs_combine(x, i.view(4, 2), x[:, :2].half()),
                 lambda: zs.zs_combine(x, i[:0].view(4, 0)),
                 lambda: zs.zs_combine_backward(x, x, i.view(4, 2), torch.zeros(4, 2, device="cuda"), i)):
        with pytest.raises(ValueError):
            call()
