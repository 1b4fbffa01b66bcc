"""Dropout from a counter-based generator, against the plain implementation in 64 bits.

The mask has to be the very one of the counters.  An element that is kept is a product with
a rounded factor, or one fused multiply and add, then rounded to its type: 2^-24 of the
product and half an ulp of the result (twice that in fp32, where both are one)."""
import numpy as np
import pytest
import torch

import expert_refs as ref
from equivariant_interatomic_potential_gb300 import zs
from train_refs import HALF_ULP, STEP, f64, held

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20


def check(y, hd, rd, p, seed, call, step, dtype):
    gain = ref.dropout_gain(hd.size, p, seed, call, step).reshape(hd.shape)
    part = np.where(gain > 0, hd, 0.0) * gain
    want = part + (0.0 if rd is None else rd)
    got = f64(y)
    assert got.shape == want.shape
    bound = HALF_ULP[dtype] * 1.001 * np.abs(want) + 2.0 ** -23 * np.abs(part) + STEP[dtype]
    assert (np.abs(got - want) <= bound).all()
    if rd is None:
        assert (got[gain == 0] == 0).all()
        assert dtype == "f16" or (got[(gain > 0) & (hd != 0)] != 0).all()


def test_generator_against_its_published_answers():
    # the generator's known answers: all bits clear, all bits set, digits of pi
    full = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((full,) * 4, (full,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(v) for v in ref.philox(np.array([counter], np.uint64), key)[0]) == want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,C", [(1, 1), (1, 8), (64, 32), (3, 7), (130, 20), (9, 1031), (1000, 512), (5, 8192), (77, 64)])
def test_against_the_formula(M, C, dtype):
    rng = np.random.default_rng(M + C)
    (h, hd), (r, rd) = (held(rng.standard_normal((M, C)), dtype) for _ in range(2))
    h, r = h.cuda(), r.cuda()
    for p, seed, call, step in ((0.1, 7, 0, 0), (0.5, 2 ** 63 - 1, 2 ** 32 - 1, 2 ** 32 + 5), (0.0, 3, 1, 2), (1.0, 3, 1, 2), (0.999, 12345678901, 4, 9)):
        check(zs.zs_dropout(h, p, seed, call, step), hd, None, p, seed, call, step, dtype)
        check(zs.zs_dropout(h, p, seed, call, step, residual=r), hd, rd, p, seed, call, step, dtype)
        at = torch.tensor([step], device="cuda")
        check(zs.zs_dropout(h, p, seed, call, at, residual=r), hd, rd, p, seed, call, step, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_elements(dtype):
    # more blocks than a thread each has room for, the last one short
    M, C = 3001, 2049
    rng = np.random.default_rng(5)
    (h, hd), (r, rd) = (held(rng.standard_normal((M, C)), dtype) for _ in range(2))
    h, r = h.cuda(), r.cuda()
    check(zs.zs_dropout(h, 0.1, 99, 1, 2), hd, None, 0.1, 99, 1, 2, dtype)
    check(zs.zs_dropout(h, 0.1, 99, 1, 2, residual=r, out=h), hd, rd, 0.1, 99, 1, 2, dtype)


@pytest.mark.gpu
def test_other_seeds_and_signs():
    h = torch.ones(64, 64, device="cuda")
    for seed in (-1, 2 ** 64 - 1, 1 << 63):
        check(zs.zs_dropout(h, 0.5, seed), np.ones((64, 64)), None, 0.5, seed & (1 << 64) - 1, 0, 0, "f32")
    masks = [zs.zs_dropout(h, 0.5, *a) > 0 for a in ((1, 0, 0), (2, 0, 0), (1, 1, 0), (1, 0, 1), (1 << 32, 0, 0))]
    for i, a in enumerate(masks):
        for b in masks[:i]:
            assert 0.4 < float((a == b).float().mean()) < 0.6      # 4096 coins: eight deviations from a half are 0.0625


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(), (5,), (3, 4, 5), (2, 3, 1, 8)])
def test_shapes(shape):
    rng = np.random.default_rng(2)
    (h, hd), (r, rd) = (held(rng.standard_normal(shape), "bf16") for _ in range(2))
    check(zs.zs_dropout(h.cuda(), 0.3, 5, residual=r.cuda()), hd, rd, 0.3, 5, 0, 0, "bf16")


@pytest.mark.gpu
def test_nothing_to_do():
    for shape in ((0, 8), (8, 0), (0,), (2, 0, 3)):
        assert zs.zs_dropout(torch.zeros(shape, device="cuda"), 0.5, 1).shape == shape


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift,C", [(8, 0, 96), (8, 8, 96), (5, 1, 96), (3, 0, 33), (0, 1, 33), (2, 0, 5)])
def test_row_strides_and_alignment(pad, shift, C, dtype):
    rng = np.random.default_rng(3)
    (h, hd), (r, rd) = (held(rng.standard_normal((70, C)), dtype) for _ in range(2))

    def wide(a):
        base = torch.full((a.shape[0], a.shape[1] + pad + shift), float("nan"), dtype=a.dtype, device="cuda")
        base[:, shift:shift + a.shape[1]] = a.cuda()
        return base[:, shift:shift + a.shape[1]]

    for hh, rr in ((wide(h), wide(r)), (h.cuda(), wide(r)), (wide(h), r.cuda())):
        check(zs.zs_dropout(hh, 0.2, 9, 1, 2, residual=rr), hd, rd, 0.2, 9, 1, 2, dtype)
    out = wide(h)
    around = out._base.clone() if out._base is not None else None
    y = zs.zs_dropout(out, 0.2, 9, 1, 2, residual=wide(r), out=out)      # in place, in rows of a wider array
    check(y, hd, rd, 0.2, 9, 1, 2, dtype)
    if around is not None and around.shape != out.shape:
        keep = torch.ones_like(around, dtype=torch.bool)
        keep[:, shift:shift + C] = False
        assert bool(torch.isnan(out._base[keep]).all())


@pytest.mark.gpu
def test_in_place():
    rng = np.random.default_rng(4)
    (h, hd), (r, rd) = (held(rng.standard_normal((33, 40)), "f32") for _ in range(2))
    a, b = h.cuda(), r.cuda()
    check(zs.zs_dropout(a, 0.5, 1, residual=b, out=a), hd, rd, 0.5, 1, 0, 0, "f32")
    a = h.cuda()
    check(zs.zs_dropout(a, 0.5, 1, residual=b, out=b), hd, rd, 0.5, 1, 0, 0, "f32")
    assert b is zs.zs_dropout(a, 0.0, 1, out=b) and torch.equal(a, b)


@pytest.mark.gpu
def test_what_is_dropped_counts_as_zero():
    # NaN and infinities that are dropped leave no trace; all is dropped at p = 1
    h = torch.full((50, 40), float("nan"), device="cuda")
    h[::2] = float("inf")
    r = torch.randn(50, 40, device="cuda")
    assert torch.equal(zs.zs_dropout(h, 1.0, 3, residual=r), r) and not bool(zs.zs_dropout(h, 1.0, 3).any())
    kept = torch.from_numpy(ref.dropout_gain(2000, 0.5, 3, 0, 0).reshape(50, 40) > 0).cuda()
    y = zs.zs_dropout(h, 0.5, 3, residual=r)
    assert torch.equal(y[~kept], r[~kept]) and not bool(torch.isfinite(y[kept]).any())


@pytest.mark.gpu
def test_share_and_mean():
    # 2^22 elements: a deviation of the kept share is 0.00015 at p = 0.1, of their mean 0.00016
    h = torch.ones(2048, 2048, device="cuda")
    y = zs.zs_dropout(h, 0.1, 42, 5, 6)
    assert abs(float((y > 0).double().mean()) - 0.9) < 1e-3 and abs(float(y.double().mean()) - 1.0) < 1.1e-3


@pytest.mark.gpu
def test_gradient_is_the_same_call():
    h, dy = (torch.randn(300, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)) for i in (1, 2))
    y, dh = zs.zs_dropout(h, 0.3, 11, 2, 3), zs.zs_dropout(dy, 0.3, 11, 2, 3)
    terms = y.double() * dy.double()
    assert abs(float(terms.sum() - (h.double() * dh.double()).sum())) <= 2.0 ** -22 * float(terms.abs().sum())


def test_argument_checks():
    lib = zs.load()
    ok = dict(dtype=0, h=FAKE, h_ld=32, r=FAKE, r_ld=32, M=4, C=32, p=0.5, at=FAKE, y=FAKE, y_ld=32)

    def call(**kw):
        a = {**ok, **kw}
        return lib.zs_dropout(a["dtype"], a["h"], a["h_ld"], a["r"], a["r_ld"], a["M"], a["C"], a["p"], 1, 2, 3, a["at"], a["y"], a["y_ld"], None)

    assert call(dtype=9) == UNSUPPORTED
    for kw in (dict(M=-1), dict(C=0), dict(h=None), dict(y=None), dict(h_ld=31), dict(r_ld=31), dict(y_ld=31), dict(p=-0.1), dict(p=1.5),
               dict(p=float("nan")), dict(at=FAKE + 4), dict(h=FAKE + 2), dict(r=FAKE + 1), dict(M=1 << 31), dict(M=1 << 30, C=1 << 11, h_ld=1 << 11)):
        assert call(**kw) == INVALID, kw
    assert call(M=0, h=None, y=None) == 0


def test_binding_refusals():
    h = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_dropout(h, 0.5, 1)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        zs.zs_dropout(h.int(), 0.5, 1)


@pytest.mark.gpu
def test_refusals_on_the_device():
    h = torch.zeros(4, 8, device="cuda")
    for kw in (dict(call=-1), dict(call=1 << 32), dict(step=1 << 63), dict(residual=torch.zeros(4, 9, device="cuda")),
               dict(residual=h.half()), dict(step=torch.zeros(1)), dict(step=torch.zeros(2, dtype=torch.int64, device="cuda")),
               dict(step=torch.zeros(1, device="cuda")), dict(out=torch.zeros(8, 4, device="cuda").T)):
        with pytest.raises(ValueError):
            zs.zs_dropout(h, 0.5, 1, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        zs.zs_dropout(torch.zeros(2, 3, 4, device="cuda").transpose(0, 1), 0.5, 1)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(zs.ZsError, match="p="):
            zs.zs_dropout(h, p, 1)
    with pytest.raises(TypeError):
        zs.zs_dropout(h, 0.5, 1.5)
