"""Embedding and its gradient by sorted ids, against the plain implementation in 64 bits.

Tolerances, fixed before the first run.  An element of y is one product of two values of
fp32 (the factor itself rounded), then rounded to its type: 2^-23 of it and half an ulp.
An element of dw is a sum in fp32 in some order, of which no term passes more than about
1500 additions: in earnest the square root of that many half ulps of the sum of the terms'
magnitudes, 1e-5 of it with room, and the result's rounding."""
import numpy as np
import pytest
import torch

import expert_refs as ref
from equivariant_interatomic_potential_gb300 import zs
from train_refs import HALF_ULP, STEP, f64, held

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20


def close(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off"


def check(w, wd, ids, dy, dyd, scale, dtype):
    """w, dy on the device, wd, dyd their values."""
    V, C = wd.shape
    idt = torch.from_numpy(ids.astype(np.int32)).cuda()
    y = zs.zs_embedding(w, idt, scale)
    want = ref.embedding(wd, ids, scale)
    close(y, want, (HALF_ULP[dtype] * 1.001 + 2.0 ** -23) * np.abs(want) + STEP[dtype], "y")
    row_ptr, perm, _ = zs.zs_build_csr(idt, V)
    dw = zs.zs_embedding_backward(dy, row_ptr, perm, scale)
    want, mag = ref.embedding_backward(dyd, ids, V, scale)
    close(dw, want, 1e-5 * mag + HALF_ULP[dtype] * 1.001 * np.abs(want) + STEP[dtype], "dw")
    return y, dw


def draw_ids(rng, M, V, how):
    if how == "one":
        return np.full(M, V // 2)
    if how == "skewed":
        return np.minimum(rng.zipf(1.3, M) - 1, V - 1)
    if how == "outside":
        return rng.choice([-1, -2 ** 31, V, 2 ** 31 - 1, 0, V - 1], M)
    return rng.integers(0, V, M)


def draw(M, V, C, how, dtype, seed):
    rng = np.random.default_rng(seed)
    w, wd = held(rng.standard_normal((V, C)), dtype)
    dy, dyd = held(rng.standard_normal((M, C)), dtype)
    return w.cuda(), wd, draw_ids(rng, M, V, how), dy.cuda(), dyd


SHAPES = [(1, 1, 1), (1, 1000, 4096), (2, 3, 8), (33, 5, 7), (64, 89, 32), (700, 3, 33), (4096, 89, 32), (5000, 700, 96), (20, 3000, 64),
          (3001, 50, 301), (257, 129, 1030), (130, 40, 2056), (9, 6000, 16), (40000, 7, 8), (2500, 4, 1), (1000, 300, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,V,C", SHAPES)
def test_forward_and_backward(M, V, C, dtype):
    for i, how in enumerate(("uniform", "skewed", "one", "outside")):
        check(*draw(M, V, C, how, dtype, M + V + C + i), scale=(1.0, 8.0, 0.3, -2.5)[i], dtype=dtype)


@pytest.mark.gpu
def test_nothing_to_do():
    w = torch.randn(5, 8, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert zs.zs_embedding(w, none).shape == (0, 8)
    row_ptr, perm, _ = zs.zs_build_csr(none, 5)
    dw = zs.zs_embedding_backward(torch.zeros(0, 8, device="cuda"), row_ptr, perm)
    assert dw.shape == (5, 8) and bool((dw == 0).all())
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = zs.zs_embedding(torch.zeros(0, 8, device="cuda"), ids)
    assert y.shape == (3, 8) and bool((y == 0).all())
    row_ptr, perm, _ = zs.zs_build_csr(ids, 0)
    assert zs.zs_embedding_backward(y, row_ptr, perm).shape == (0, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (5, 1), (3, 0)])
def test_row_strides_and_alignment(pad, shift, dtype):
    w, wd, ids, dy, dyd = draw(900, 60, 96, "skewed", dtype, 3)

    def wide(a):
        base = torch.full((a.shape[0], a.shape[1] + pad + shift), float("nan"), dtype=a.dtype, device="cuda")
        base[:, shift:shift + a.shape[1]] = a
        return base[:, shift:shift + a.shape[1]]

    check(wide(w), wd, ids, wide(dy), dyd, 1.5, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 65])
def test_rows_do_not_mix(C):
    # NaN and infinities stay with their ids, and rows of no id (NaN too) are not used
    w, wd, ids, dy, dyd = draw(3000, 40, C, "skewed", "f32", 5)
    ids = ids.copy()
    ids[100:200] = -1
    _, want = check(w, wd, ids, dy, dyd, 1.0, "f32")
    dy = dy.clone()
    dy[100:200] = float("nan")
    at = int(ids[7])
    dy[7, 3] = float("nan")
    row_ptr, perm, _ = zs.zs_build_csr(torch.from_numpy(ids.astype(np.int32)).cuda(), 40)
    dw = zs.zs_embedding_backward(dy, row_ptr, perm)
    bad = torch.zeros_like(dw, dtype=torch.bool)
    bad[at, 3] = True
    assert torch.equal(torch.isnan(dw), bad) and torch.equal(dw[~bad], want[~bad])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,V,C", [("f32", 60000, 7921, 96), ("bf16", 9000, 20011, 256), ("f16", 30011, 3, 77)])
def test_run_to_run_bits(dtype, M, V, C):
    w, _, ids, dy, _ = draw(M, V, C, "skewed", dtype, 6)
    row_ptr, perm, _ = zs.zs_build_csr(torch.from_numpy(ids.astype(np.int32)).cuda(), V)
    first = zs.zs_embedding_backward(dy, row_ptr, perm, 2.0)
    for _ in range(5):
        assert torch.equal(zs.zs_embedding_backward(dy, row_ptr, perm, 2.0), first)


@pytest.mark.gpu
def test_positions_that_are_none():
    # a perm or a row_ptr that no CSR is gives some sums, and reads and writes nothing outside the operands
    dy = torch.randn(500, 40, device="cuda")
    gen = torch.Generator().manual_seed(1)
    for lo, hi in ((-(2 ** 31), 2 ** 31 - 1), (0, 600)):
        row_ptr = torch.randint(lo, hi, (301,), generator=gen).int().cuda()
        perm = torch.randint(lo, hi, (500,), generator=gen).int().cuda()
        assert zs.zs_embedding_backward(dy, row_ptr, perm).shape == (300, 40)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_gradient_against_differences():
    w, _, ids, dy, _ = draw(600, 30, 24, "skewed", "f32", 8)
    idt = torch.from_numpy(ids.astype(np.int32)).cuda()
    row_ptr, perm, _ = zs.zs_build_csr(idt, 30)
    g = zs.zs_embedding_backward(dy, row_ptr, perm, 3.0).double()
    v = torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    loss = lambda u: float((zs.zs_embedding(u, idt, 3.0).double() * dy.double()).sum())  # noqa: E731
    slope = (loss(w + 0.5 * v) - loss(w - 0.5 * v))
    assert abs(slope - float((g * v.double()).sum())) <= 1e-5 * float((dy.abs().double() * 3).sum())


@pytest.mark.gpu
def test_rows_far_into_a_table():
    # a table of more than 2^31 elements: the last rows are those
    V, C = 2 ** 21 + 5, 1032
    w = torch.zeros(V, C, dtype=torch.bfloat16, device="cuda")
    w[-3:] = torch.arange(3 * C, device="cuda").view(3, C).to(torch.bfloat16)
    ids = torch.tensor([V - 1, 0, V - 3, V], dtype=torch.int32, device="cuda")
    y = zs.zs_embedding(w, ids)
    assert torch.equal(y[0], w[-1]) and torch.equal(y[2], w[-3]) and not bool(y[1].any()) and not bool(y[3].any())
    del w
    row_ptr, perm, _ = zs.zs_build_csr(ids, V)
    dy = torch.randn(4, C, device="cuda").to(torch.bfloat16)
    dw = zs.zs_embedding_backward(dy, row_ptr, perm)
    assert torch.equal(dw[V - 1], dy[0]) and torch.equal(dw[V - 3], dy[2]) and torch.equal(dw[0], dy[1])
    assert int(dw.ne(0).any(1).sum()) == 3


def test_argument_checks():
    lib = zs.load()
    ok = dict(dtype=0, w=FAKE, ld=32, ids=FAKE, M=4, V=9, C=32, scale=1.0, y=FAKE, y_ld=32)

    def fwd(**kw):
        a = {**ok, **kw}
        return lib.zs_embedding(a["dtype"], a["w"], a["ld"], a["ids"], a["M"], a["V"], a["C"], a["scale"], a["y"], a["y_ld"], None)

    assert fwd(dtype=3) == UNSUPPORTED
    for kw in (dict(M=-1), dict(V=-1), dict(C=0), dict(w=None), dict(ids=None), dict(y=None), dict(ld=31), dict(y_ld=31), dict(w=FAKE + 2),
               dict(ids=FAKE + 2), dict(dtype=1, y=FAKE + 1), dict(scale=float("nan")), dict(scale=float("inf")), dict(M=1 << 31)):
        assert fwd(**kw) == INVALID, kw
    assert fwd(M=0, ids=None, y=None) == 0
    need = lib.zs_embedding_backward_workspace_bytes(0, 4, 9, 32)
    assert need > 0 and lib.zs_embedding_backward_workspace_bytes(7, 4, 9, 32) == 0
    ok |= dict(bytes=need, ws=FAKE)

    def bwd(**kw):
        a = {**ok, **kw}
        return lib.zs_embedding_backward(a["dtype"], a["w"], a["ld"], a["ids"], a["ids"], a["M"], a["V"], a["C"], a["scale"], a["y"], a["ws"],
                                         a["bytes"], None)

    assert bwd(dtype=-1) == UNSUPPORTED and bwd(C=(1 << 23) + 1, ld=1 << 24) == UNSUPPORTED
    for kw in (dict(M=-1), dict(C=-4), dict(w=None), dict(ids=None), dict(y=None), dict(ld=3), dict(ws=None), dict(bytes=need - 1),
               dict(ws=FAKE + 8), dict(y=FAKE + 2), dict(scale=float("nan"))):
        assert bwd(**kw) == INVALID, kw
    assert bwd(V=0, ws=None, bytes=0) == 0


def test_binding_refusals():
    w, ids = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_embedding(w, ids)
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_embedding(w[0], ids)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        zs.zs_embedding(w.double(), ids)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_embedding_backward(w, ids, ids)


@pytest.mark.gpu
def test_refusals_on_the_device():
    w, ids = torch.zeros(4, 8, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="torch.int32"):
        zs.zs_embedding(w, ids.long())
    with pytest.raises(ValueError, match="shape"):
        zs.zs_embedding(w, ids.view(3, 1))
    with pytest.raises(zs.ZsError, match="scale"):
        zs.zs_embedding(w, ids, float("nan"))
    with pytest.raises(ValueError, match="contiguous rows"):
        zs.zs_embedding(torch.zeros(8, 4, device="cuda").T, ids)
    with pytest.raises(ValueError, match="perm"):
        zs.zs_embedding_backward(w, ids, ids)


@pytest.mark.gpu
@pytest.mark.parametrize("E,N", [(1, 50021), (173, 32624), (257, 200000), (16384, 50021), (200000, 70000), (131073, 66000), (140001, 70000),
                                 (513, 65536), (300, 1 << 24), (40000, (1 << 24) + 3), (131072, 100000), (262145, 30000), (600001, 70000),
                                 (819201, 9000), (1048577, 6000), (1025, 1023), (5000, 37), (16384, 900), (12289, 1), (4097, 1024)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "last", "outside"])
def test_order_of_ids_with_gaps(E, N, kind):
    # row_ptr is exact however far apart the ids are: few ids of many, all of one, and none
    u = torch.rand(E, device="cuda", dtype=torch.float64)
    ids = {"uniform": u * N, "skewed": u**9 * N, "one": torch.full_like(u, N // 3), "last": torch.full_like(u, N - 1),
           "outside": torch.where(u < 0.3, -1.0, N + 5.0)}[kind].floor().int()
    row_ptr, perm, bad = zs.zs_build_csr(ids, N)
    held = (ids >= 0) & (ids < N)
    count = torch.bincount(ids[held].long(), minlength=N)
    want = torch.cat([count.new_zeros(1), count.cumsum(0)])
    assert torch.equal(row_ptr.long(), want)
    assert int(bad) == int((~held).sum())
    order = torch.where(held, ids, N).long().sort(stable=True)[1]
    assert torch.equal(perm.long(), order)
