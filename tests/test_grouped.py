"""Products grouped by a CSR, against the plain implementation in 64 bits.

Tolerance, fixed before the first run: a product of n terms summed in fp32
(in any order, each addition off by at most an ulp) is off by at most
n 2^-23 sum|terms|, typically sqrt(n) 2^-24 sum|terms|; 1e-5 sum|terms| holds
for the lengths here, as for the zonal scatter.  The one rounding to the
output's type adds half an ulp of the result."""
import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import zs
from train_refs import HALF_ULP, STEP, TORCH, csr, f64, grouped, held

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20
TOL = 1e-5


def close(got, ref, absum, dtype, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    bound = TOL * absum + HALF_ULP[dtype] * (1 + 1e-3) * np.abs(ref) + STEP[dtype]
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / bound):.2f} x the bound"


def draw(M, K, N, G, dtype, seed, sizes="uniform", bad=0.0):
    rng = np.random.default_rng(seed)
    if sizes == "zipf":
        p = (np.arange(G) + 1.0) ** -1.5
        group = rng.permutation(G)[rng.choice(G, M, p=p / p.sum())]
    elif sizes == "one":
        group = np.full(M, G // 2)
    else:
        group = rng.integers(0, max(G, 1), M)
    if bad:
        group = np.where(rng.random(M) < bad, G + 3, group)
    x, xd = held(rng.standard_normal((M, K)), dtype)
    w, wd = held(rng.standard_normal((G, N, K)) / np.sqrt(K), dtype)
    dy, dyd = held(rng.standard_normal((M, N)), dtype)
    return group, (x, w, dy), (xd, wd, dyd)


def run(group, G, x, w, dy, ordered=False):
    row_ptr, perm = csr(group, G)
    rp, pm = torch.from_numpy(row_ptr).cuda(), None if ordered else torch.from_numpy(perm).cuda()
    y = zs.zs_grouped_matmul(x, w, rp, pm)
    dx, dw = zs.zs_grouped_matmul_backward(dy, x, w, rp, pm)
    torch.cuda.synchronize()
    zs.zs_check_timeouts()
    return y, dx, dw


def check_all(group, t, d, dtype, ordered=False):
    y, dx, dw = run(group, t[1].shape[0], *(a.cuda() for a in t), ordered=ordered)
    ry, ay, rdx, adx, rdw, adw = grouped(d[0], d[1], group, d[2])
    close(y, ry, ay, dtype, "y")
    close(dx, rdx, adx, dtype, "dx")
    close(dw, rdw, adw, dtype, "dw")
    return y, dx, dw


SHAPES = [
    (1, 32, 32, 1), (1, 1, 1, 1), (64, 32, 32, 4), (127, 32, 32, 5), (128, 64, 64, 1), (129, 64, 128, 3),
    (300, 48, 80, 7), (1000, 256, 256, 3), (513, 8, 520, 9), (700, 520, 8, 2), (257, 72, 264, 4),
    (400, 33, 65, 6), (333, 187, 301, 11), (50, 1, 300, 3), (50, 300, 1, 3), (2000, 7, 5, 40), (90, 130, 96, 120),
    (4100, 128, 384, 2), (260, 1100, 200, 2), (640, 200, 1030, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N,G", SHAPES)
def test_products_and_gradients(M, K, N, G, dtype):
    check_all(*draw(M, K, N, G, dtype, seed=M + 3 * K + 5 * N + G, sizes="zipf", bad=0.1 if M > 10 else 0.0), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", ["uniform", "one"])
def test_rows_in_order(sizes, dtype):
    # perm None: position p is row p; with every row in one group most groups are empty
    group, t, d = draw(1500, 96, 160, 8, dtype, 3, sizes)
    group = np.sort(group)
    check_all(group, t, d, dtype, ordered=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_no_rows_no_groups(dtype):
    dt = TORCH[dtype]
    e = lambda *s: torch.full(s, 7.0, dtype=dt, device="cuda")  # noqa: E731
    rp = torch.zeros(4, dtype=torch.int32, device="cuda")
    y = zs.zs_grouped_matmul(e(0, 32), e(3, 48, 32), rp)
    dx, dw = zs.zs_grouped_matmul_backward(e(0, 48), e(0, 32), e(3, 48, 32), rp)
    assert y.shape == (0, 48) and dx.shape == (0, 32) and dw.shape == (3, 48, 32) and bool((dw == 0).all())
    # no group at all, and no row in any group: every row is zero
    for G in (0, 3):
        y = zs.zs_grouped_matmul(e(70, 32), e(G, 48, 32), rp[:G + 1].contiguous())
        dx, dw = zs.zs_grouped_matmul_backward(e(70, 48), e(70, 32), e(G, 48, 32), rp[:G + 1].contiguous())
        assert bool((y == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all()) and dw.shape == (G, 48, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K,N", [(64, 64), (36, 44)])
def test_values_stay_in_their_group(K, N, dtype):
    # a row, or a group's weights, of NaN and infinities reach nothing beyond the row, or its group
    M, G = 900, 5
    group, t, d = draw(M, K, N, G, dtype, 9)
    x, w, dy = (a.clone() for a in t)
    sick = int(np.flatnonzero(group == 1)[3])
    x[sick, 0::2], x[sick, 1::2] = float("nan"), float("inf")
    dy[sick] = float("-inf")
    w[3] = float("nan")
    y, dx, dw = run(group, G, x.cuda(), w.cuda(), dy.cuda())
    ry, ay, rdx, adx, rdw, adw = grouped(d[0], d[1], group, d[2])
    keep = (np.arange(M) != sick) & (group != 3)
    close(y[keep], ry[keep], ay[keep], dtype, "y")
    close(dx[keep], rdx[keep], adx[keep], dtype, "dx")
    clean = np.arange(G) != 1
    close(dw[clean], rdw[clean], adw[clean], dtype, "dw")
    assert not bool(torch.isfinite(y[sick]).any()) and not bool(torch.isfinite(dw[1]).any())
    assert bool(torch.isnan(y[torch.from_numpy(group == 3).cuda()]).all())


@pytest.mark.gpu
def test_rows_of_no_group_are_not_read():
    # rows outside every group may hold anything; their results are zeros, and neighbours keep theirs
    group, t, d = draw(700, 64, 64, 4, "bf16", 21, bad=0.3)
    none = group >= 4
    x, w, dy = (a.clone() for a in t)
    x[torch.from_numpy(none)] = float("nan")
    dy[torch.from_numpy(none)] = float("inf")
    y, dx, dw = run(group, 4, x.cuda(), w.cuda(), dy.cuda())
    ry, ay, rdx, adx, rdw, adw = grouped(d[0], d[1], group, d[2])
    close(y, ry, ay, "bf16", "y")
    close(dx, rdx, adx, "bf16", "dx")
    close(dw, rdw, adw, "bf16", "dw")
    assert bool((y[torch.from_numpy(none).cuda()] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (8, 8), (3, 1), (24, 4)])
def test_row_strides_and_alignment(pad, shift, dtype):
    # x, dy and the results as column ranges of wider matrices, at any element offset; what lies around stays
    M, K, N, G = 517, 64, 96, 3
    group, (x, w, dy), d = draw(M, K, N, G, dtype, 5)
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group, G))

    def wide(a):
        base = torch.full((a.shape[0], a.shape[1] + pad + shift), 9.0, dtype=a.dtype, device="cuda")
        view = base[:, shift:shift + a.shape[1]]
        view.copy_(a.cuda())
        return base, view

    xv, dyv, wc = wide(x)[1], wide(dy)[1], w.cuda()
    (yb, yv), (dxb, dxv) = wide(torch.zeros(M, N, dtype=x.dtype)), wide(torch.zeros(M, K, dtype=x.dtype))
    zs.zs_grouped_matmul(xv, wc, row_ptr, perm, out=yv)
    zs.zs_grouped_matmul_dx(dyv, wc, row_ptr, perm, out=dxv)
    dw = zs.zs_grouped_matmul_dw(dyv, xv, row_ptr, perm)
    ry, ay, rdx, adx, rdw, adw = grouped(d[0], d[1], group, d[2])
    close(yv, ry, ay, dtype, "y")
    close(dxv, rdx, adx, dtype, "dx")
    close(dw, rdw, adw, dtype, "dw")
    for base, cols in ((yb, N), (dxb, K)):
        around = torch.ones(base.shape[1], dtype=torch.bool)
        around[shift:shift + cols] = False
        assert bool((base[:, around.cuda()] == 9.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_at_any_alignment(dtype):
    group, (x, w, dy), d = draw(300, 40, 56, 3, dtype, 12)
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group, 3))
    flat = torch.zeros(w.numel() + 1, dtype=w.dtype, device="cuda")
    wv = flat[1:].view(w.shape)
    wv.copy_(w.cuda())
    dwf = torch.full((w.numel() + 2,), 9.0, dtype=w.dtype, device="cuda")
    dwv = dwf[1:-1].view(w.shape)
    ry, ay, rdx, adx, rdw, adw = grouped(d[0], d[1], group, d[2])
    close(zs.zs_grouped_matmul(x.cuda(), wv, row_ptr, perm), ry, ay, dtype, "y")
    close(zs.zs_grouped_matmul_dx(dy.cuda(), wv, row_ptr, perm), rdx, adx, dtype, "dx")
    zs.zs_grouped_matmul_dw(dy.cuda(), x.cuda(), row_ptr, perm, out=dwv)
    close(dwv, rdw, adw, dtype, "dw")
    assert float(dwf[0]) == 9.0 and float(dwf[-1]) == 9.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_run_to_run_bits(dtype):
    group, t, _ = draw(5000, 96, 64, 5, dtype, 17, "zipf")
    t = [a.cuda() for a in t]
    first = run(group, 5, *t)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(group, 5, *t), first))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,scale", [("f32", 1e30), ("f32", 1e-30), ("bf16", 1e30)])
def test_large_and_small_magnitudes(dtype, scale):
    # products stay within fp32's range although an operand is near its ends
    group, (x, w, dy), _ = draw(200, 64, 32, 3, dtype, 8)
    x, xd = held(x.float().numpy() * scale, dtype)
    wd, dyd = f64(w), f64(dy)
    y, dx, dw = run(group, 3, x.cuda(), w.cuda(), dy.cuda())
    ry, ay, rdx, adx, rdw, adw = grouped(xd, wd, group, dyd)
    close(y, ry, ay, dtype, "y")
    close(dw, rdw, adw, dtype, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_skewed_and_long_sums(dtype):
    # one group holds nearly every row: its weight gradient is one sum of many thousand terms
    rng = np.random.default_rng(2)
    M, K, N, G = 60000, 32, 48, 6
    group = np.where(rng.random(M) < 0.97, 4, rng.integers(0, G, M))
    x, xd = held(rng.standard_normal((M, K)), dtype)
    w, wd = held(rng.standard_normal((G, N, K)), dtype)
    dy, dyd = held(rng.standard_normal((M, N)), dtype)
    check_all(group, (x, w, dy), (xd, wd, dyd), dtype)


@pytest.mark.gpu
def test_side_stream_and_graph():
    group, t, d = draw(800, 64, 64, 4, "bf16", 30)
    x, w, dy = (a.cuda() for a in t)
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group, 4))
    run(group, 4, x, w, dy)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        y = zs.zs_grouped_matmul(x, w, row_ptr, perm)
        dx, dw = zs.zs_grouped_matmul_backward(dy, x, w, row_ptr, perm)
    torch.cuda.synchronize()
    for seed in (31, 32):
        group, t2, d2 = draw(800, 64, 64, 4, "bf16", seed)
        rp, pm = csr(group, 4)
        for a, b in ((x, t2[0]), (w, t2[1]), (dy, t2[2]), (row_ptr, torch.from_numpy(rp)), (perm, torch.from_numpy(pm))):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        ry, ay, rdx, adx, rdw, adw = grouped(d2[0], d2[1], group, d2[2])
        close(y, ry, ay, "bf16", "y")
        close(dx, rdx, adx, "bf16", "dx")
        close(dw, rdw, adw, "bf16", "dw")


@pytest.mark.gpu
def test_gradients_against_differences():
    # y is linear in x and in w, so central differences have no truncation error
    group, t, _ = draw(400, 48, 40, 3, "f32", 6, bad=0.1)
    x, w, dy = (a.cuda() for a in t)
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group, 3))
    dx, dw = zs.zs_grouped_matmul_backward(dy, x, w, row_ptr, perm)
    loss = lambda a, b: (zs.zs_grouped_matmul(a, b, row_ptr, perm).double() * dy.double()).sum()  # noqa: E731
    for grad, at, call in ((dx, x, lambda e: loss(x + e, w)), (dw, w, lambda e: loss(x, w + e))):
        v = torch.randn_like(at)
        slope = (call(v) - call(-v)) / 2
        want = (grad.double() * v.double()).sum()
        # fp32 rounding of about 1e-6 in each of the 16000 terms of the loss
        assert abs(float(slope - want)) <= 1e-5 * float((grad.double() * v.double()).abs().sum())


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, w, dy = rng.standard_normal((9, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((9, 5))
    group = np.array([0, 2, 2, 0, 7, 0, 2, 0, 2])
    _, _, dx, _, dw, _ = grouped(x, w, group, dy)
    for at, grad in ((x, dx), (w, dw)):
        for i in np.ndindex(at.shape):
            old, e = at[i], 0.5
            at[i] = old + e
            up = (grouped(x, w, group)[0] * dy).sum()
            at[i] = old - e
            down = (grouped(x, w, group)[0] * dy).sum()
            at[i] = old
            assert abs((up - down) / (2 * e) - grad[i]) < 1e-12
    assert not dw[1].any() and not dx[4].any()


def test_argument_checks():
    lib = zs.load()
    ok = dict(dtype=0, x=FAKE, x_ld=32, w=FAKE, rp=FAKE, perm=FAKE, M=10, K=32, N=48, G=3, y=FAKE, y_ld=48)

    def fwd(**kw):
        a = {**ok, **kw}
        return lib.zs_grouped_matmul(a["dtype"], a["x"], a["x_ld"], a["w"], a["rp"], a["perm"], a["M"], a["K"], a["N"],
                                     a["G"], a["y"], a["y_ld"], None)

    def dx(**kw):
        a = {**ok, "x_ld": 48, "y_ld": 32, **kw}
        return lib.zs_grouped_matmul_dx(a["dtype"], a["x"], a["x_ld"], a["w"], a["rp"], a["perm"], a["M"], a["K"], a["N"],
                                        a["G"], a["y"], a["y_ld"], None)

    for call in (fwd, dx):
        assert call(dtype=3) == UNSUPPORTED and b"dtype" in lib.zs_last_error()
        for kw in (dict(M=-1), dict(M=1 << 31), dict(K=0), dict(N=0), dict(G=-1), dict(x=None), dict(w=None), dict(y=None),
                   dict(rp=None), dict(x_ld=31), dict(y_ld=31), dict(x=FAKE + 2), dict(dtype=1, y=FAKE + 1),
                   dict(perm=FAKE + 2)):
            assert call(**kw) == INVALID, kw
        assert call(M=0, x=None, y=None) == 0      # enqueues nothing

    def dw(**kw):
        a = {**ok, "ws": FAKE, "bytes": 1 << 40, **kw}
        return lib.zs_grouped_matmul_dw(a["dtype"], a["x"], 48, a["w"], 32, a["rp"], a["perm"], a["M"], a["K"], a["N"],
                                        a["G"], a["y"], a["ws"], a["bytes"], None)

    assert dw(dtype=-1) == UNSUPPORTED
    for kw in (dict(M=-1), dict(K=0), dict(N=-4), dict(x=None), dict(w=None), dict(y=None), dict(rp=None), dict(ws=FAKE + 8)):
        assert dw(**kw) == INVALID, kw
    need = lib.zs_grouped_matmul_dw_workspace_bytes(0, 10, 32, 48, 3)
    if need:
        assert dw(bytes=need - 1) == INVALID and dw(ws=None) == INVALID
    assert dw(G=0, y=None, w=None, x=None) == 0
    assert lib.zs_grouped_matmul_dw_workspace_bytes(0, -1, 32, 48, 3) == 0
    assert lib.zs_grouped_matmul_dw_workspace_bytes(9, 10, 32, 48, 3) == 0


def test_sizes_past_32_bits_refused():
    # positions, columns and units of work a tile or a range past the last one have to stay below 2^31; all of these
    # are refused before anything is launched
    lib, most = zs.load(), (1 << 31) - (1 << 16)

    def product(fn, M=10, K=32, N=48):
        return fn(1, FAKE, max(K, N), FAKE, FAKE, None, M, K, N, 1, FAKE, max(K, N), None)

    def dw(M=10, K=32, N=48):
        return lib.zs_grouped_matmul_dw(1, FAKE, N, FAKE, K, FAKE, None, M, K, N, 1, FAKE, FAKE, 1 << 40, None)

    for side in ("M", "K", "N"):
        for call in (lambda **kw: product(lib.zs_grouped_matmul, **kw), lambda **kw: product(lib.zs_grouped_matmul_dx, **kw), dw):
            assert call(**{side: most + 1}) == INVALID and call(**{side: (1 << 31) - 1}) == INVALID, side
    # 24601 tiles of 87202 units: fewer than 2^31 of them, but not with one range more
    assert dw(M=64 * 87200, K=337 * 256, N=73 * 128) == INVALID and b"units" in lib.zs_last_error()


def test_nothing_to_lay_out():
    # operands of whole 16-byte pieces, and a size that is refused after the laying out was looked at, before any
    # launch: on the way the host divided by the zero pieces of the matrix that is not there, which x86 traps
    assert zs.load().zs_grouped_matmul_dw(1, FAKE, 9344, FAKE, 86272, FAKE, None, 64 * 87200, 86272, 9344, 1, FAKE, FAKE,
                                          1 << 40, None) == INVALID


def test_binding_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(2, 6, 8)
    rp = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_grouped_matmul(x, w, rp)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        zs.zs_grouped_matmul(x, w.double(), rp)
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_grouped_matmul(x[0], w, rp)
    with pytest.raises(ValueError, match="shape"):
        zs.zs_grouped_matmul(x, w[0], rp)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K,N", [(41, 25), (217, 136), (136, 217), (7, 130), (1, 300), (263, 3)])
@pytest.mark.parametrize("shift", [0, 1, 5])
def test_rows_laid_out_anew(K, N, shift, dtype):
    # whether a workspace has room for both operands, for one, or there is none, the results are the same sums
    M, G = 777, 4
    group, (x, w, dy), d = draw(M, K, N, G, dtype, K + N, "zipf", bad=0.05)
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group, G))
    code, lib = {"f32": 0, "bf16": 1, "f16": 2}[dtype], zs.load()

    def exact_end(a):   # views that end where their allocation does, rows `shift` elements wider
        base = torch.full((a.numel() + (a.shape[0] - 1) * shift if a.dim() == 2 else a.numel(),), float("nan"),
                          dtype=a.dtype, device="cuda")
        view = base.as_strided(a.shape, (a.shape[1] + shift, 1)) if a.dim() == 2 else base.view(a.shape)
        view.copy_(a.cuda())
        return view

    xv, dyv, wv = exact_end(x), exact_end(dy), exact_end(w)
    need = lib.zs_grouped_matmul_workspace_bytes(code, M, K, N, G)
    assert need % 256 == 0 and need > 0
    ry, ay, rdx, adx, _, _ = grouped(d[0], d[1], group, d[2])
    for room in (need, max(need // 2 // 256 * 256, 256), 0):
        ws = torch.full((max(room, 256) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        y = torch.full((M, N), 9.0, dtype=x.dtype, device="cuda")
        dx = torch.full((M, K), 9.0, dtype=x.dtype, device="cuda")
        for fn, a, ld, out, cols in ((lib.zs_grouped_matmul_ws, xv, K + shift, y, N),
                                     (lib.zs_grouped_matmul_dx_ws, dyv, N + shift, dx, K)):
            assert fn(code, a.data_ptr(), ld, wv.data_ptr(), row_ptr.data_ptr(), perm.data_ptr(), M, K, N, G,
                      out.data_ptr(), cols, ws.data_ptr() if room else None, room,
                      torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        zs.zs_check_timeouts()
        assert bool((ws[room:] == 0xFF).all())
        close(y, ry, ay, dtype, "y")
        close(dx, rdx, adx, dtype, "dx")


def test_workspace_sizes_and_refusals():
    lib = zs.load()
    size = lib.zs_grouped_matmul_workspace_bytes
    assert size(1, 5000, 64, 128, 3) == 0          # rows of whole 16-byte pieces
    assert size(1, 5000, 17, 31, 3) == 0           # both at most 32: on other cores
    assert size(9, 5000, 65, 128, 3) == 0 and size(1, -1, 65, 128, 3) == 0 and size(1, 5000, 0, 128, 3) == 0
    up = lambda b: -(-b // 256) * 256  # noqa: E731
    assert size(1, 5000, 65, 128, 3) == up(3 * 128 * 72 * 2) + up(5000 * 72 * 2)
    assert size(0, 5000, 64, 129, 3) == up(5000 * 132 * 4)
    for fn in (lib.zs_grouped_matmul_ws, lib.zs_grouped_matmul_dx_ws):
        call = lambda ws, M: fn(1, FAKE, 65, FAKE, FAKE, FAKE, M, 65, 65, 3, FAKE, 65, ws, 1 << 30, None)  # noqa: E731
        assert call(FAKE + 8, 300) == INVALID and b"aligned" in lib.zs_last_error()
        assert call(FAKE, 0) == 0 and call(FAKE, -1) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,G,sizes,ordered", [
    (1500, 200, 256, 2, "uniform", False), (1100, 256, 136, 2, "uniform", True), (512, 64, 480, 1, "uniform", False),
    (513, 16, 1000, 1, "one", True), (9000, 264, 232, 5, "zipf", False), (40000, 768, 256, 3, "one", False),
    (7000, 1032, 984, 2, "zipf", True),
])
def test_tiles_of_two_ctas(M, K, N, G, sizes, ordered, dtype):
    # many rows a group and more than 128 columns: rows off the tiles' ends, columns in one CTA's half alone
    group, t, d = draw(M, K, N, G, dtype, M + N, sizes, bad=0.02 if not ordered else 0.0)
    if ordered:
        group = np.sort(group)
    check_all(group, t, d, dtype, ordered=ordered)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N,G", [(900, 72, 1300, 5), (900, 1288, 136, 3), (700, 1031, 1029, 2), (1300, 520, 1024, 4), (256, 1024, 1320, 1), (300, 2048, 1032, 2)])
def test_gathered_rows_put_in_order(M, K, N, G, dtype):
    # rows of no group, and one row of values that are not finite, which reach nothing beyond it and its group
    group, t, d = draw(M, K, N, G, dtype, M + K, "zipf", bad=0.1)
    x, w, dy = (a.clone() for a in t)
    sick = int(np.flatnonzero(group == 0)[0])
    x[sick], dy[sick] = float("nan"), float("inf")
    none = torch.from_numpy(group >= G)
    x[none], dy[none] = float("nan"), float("nan")
    y, dx, dw = run(group, G, x.cuda(), w.cuda(), dy.cuda())
    ry, ay, rdx, adx, rdw, adw = grouped(d[0], d[1], group, d[2])
    keep = np.arange(M) != sick
    close(y[keep], ry[keep], ay[keep], dtype, "y")
    close(dx[keep], rdx[keep], adx[keep], dtype, "dx")
    close(dw[1:], rdw[1:], adw[1:], dtype, "dw")
    assert not bool(torch.isfinite(y[sick]).any()) and not bool(torch.isfinite(dw[0]).any())
    assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
               for a, b in zip(run(group, G, x.cuda(), w.cuda(), dy.cuda()), (y, dx, dw)))


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(64, 96), (65, 131)])
def test_fp32_products_of_one_term(K, N):
    """fp32 on the tensor cores, sums of one term that is not zero: what is left of the
    three planes of 8 bits.  Planes rounded to nearest leave at most 2^-8 and 2^-17 of a
    value in [1, 2), so the products left out are below 2^-24 of the term, of either sign;
    the joining of the three partial sums rounds twice, the second time once at most."""
    M, rng = 700, np.random.default_rng(3)

    def some(*shape):
        bits = rng.integers(0x3f800000, 0x40000000, shape, dtype=np.uint32)
        hard = np.array([0x3f80ffff, 0x3f807f40, 0x3f837bbe, 0x3f8590c0, 0x3fffffff, 0x3f817fff], np.uint32)
        return np.where(rng.random(shape) < 0.3, rng.choice(hard, shape), bits).view(np.float32)

    def check(got, want, what):
        err = np.abs(f64(got) - want) / np.where(want == 0, 1, want)
        assert err.max() <= 2.2 * 2.0 ** -24, f"{what}: {err.max() * 2 ** 24:.2f} x 2^-24"

    one = lambda a: np.where(np.arange(a.shape[1]) == rng.integers(0, a.shape[1], (len(a), 1)), a, 0)  # noqa: E731
    x, dy, w = one(some(M, K)), one(some(M, N)), some(1, N, K)
    row_ptr = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    up = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    d = lambda a: a.astype(np.float64)  # noqa: E731
    check(zs.zs_grouped_matmul(up(x), up(w), row_ptr), d(x) @ d(w[0]).T, "y")
    check(zs.zs_grouped_matmul_dx(up(dy), up(w), row_ptr), d(dy) @ d(w[0]), "dx")
    x, dy = some(M, K), some(M, N)
    x[np.arange(M) != 333] = 0
    check(zs.zs_grouped_matmul_dw(up(dy), up(x), row_ptr)[0], d(dy).T @ d(x), "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(64, 96), (65, 131)])
def test_fp32_largest_values(K, N):
    # values that bf16 would round to infinity are cut off instead; an infinity and a NaN still reach only their rows
    M, top = 700, float(np.finfo(np.float32).max)
    x, w = torch.zeros(M, K), torch.zeros(1, N, K)
    x[:, 3], x[:, 5], w[0, :, 3] = top, -top, 0.75
    x[7, 3], x[9, 2], x[11, 3] = float("inf"), float("nan"), top / 2
    row_ptr = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    y = zs.zs_grouped_matmul(x.cuda(), w.cuda(), row_ptr).cpu()
    want = torch.full((M, N), 0.75 * top)
    want[11] = 0.375 * top
    keep = torch.ones(M, dtype=torch.bool)
    keep[[7, 9]] = False
    assert bool(((y - want)[keep].abs() <= 2.0 ** -22 * want[keep]).all())
    assert not bool(torch.isfinite(y[~keep]).any())


def spread(*shape, gen, dtype):
    """Values of one sign whose roundings go either way."""
    return (torch.rand(shape, generator=gen, device="cuda") * 0.1 + 0.05).to(dtype)


def low(got, want):
    """The mean relative error over as many elements as average their roundings out."""
    err = (got.double() - want) / want
    assert float(err.abs().max()) <= 2.0 ** -7
    return abs(float(err.mean()))


LOW = 1e-4   # each of 128 additions is up to an ulp of fp32 low, 2^-16 in all; and what is left of the roundings' mean


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,gathered", [(1024, 65536, 1024, False), (1024, 65528, 1024, True), (600, 40000, 100, True),
                                            (200, 32769, 136, True), (1024, 8200, 1024, False)])
def test_long_sums_over_columns(M, K, N, gathered, dtype):
    # sums of 16-bit products of one sign, much longer than the tensor cores' truncating additions bear
    gen = torch.Generator(device="cuda").manual_seed(K)
    x, w, dy = (spread(*s, gen=gen, dtype=TORCH[dtype]) for s in ((M, K), (1, N, K), (M, K)))
    w.mul_((torch.rand(1, N, 1, generator=gen, device="cuda") + 1).to(w.dtype))
    row_ptr = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    perm = torch.randperm(M, generator=gen, device="cuda").int() if gathered else None
    y = zs.zs_grouped_matmul(x, w, row_ptr, perm)
    wt = w.transpose(1, 2).contiguous()      # (1, K, N): dx of rows of K sums over K
    dx = zs.zs_grouped_matmul_dx(dy, wt, row_ptr, perm)
    torch.cuda.synchronize()
    zs.zs_check_timeouts()
    assert low(y, x.double() @ w[0].double().T) <= LOW
    assert low(dx, dy.double() @ w[0].double().T) <= LOW


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,gathered", [(65536, 2560, 2048, False), (100000, 2560, 2048, True), (70001, 1283, 2048, True)])
def test_long_sums_over_rows(M, K, N, gathered, dtype):
    # the weight gradient of one group of many rows, for as many tiles as SMs and more: a CTA sums a whole tile
    gen = torch.Generator(device="cuda").manual_seed(M)
    x, dy = (spread(*s, gen=gen, dtype=TORCH[dtype]) for s in ((M, K), (M, N)))
    dy.mul_((torch.rand(1, N, generator=gen, device="cuda") + 1).to(dy.dtype))
    row_ptr = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    perm = torch.randperm(M, generator=gen, device="cuda").int() if gathered else None
    dw = zs.zs_grouped_matmul_dw(dy, x, row_ptr, perm)[0]
    torch.cuda.synchronize()
    zs.zs_check_timeouts()
    assert low(dw[:, :200], dy.double().T @ x[:, :200].double()) <= LOW


@pytest.mark.gpu
@pytest.mark.parametrize("M", [8191, 8192, 8193, 16384, 16400, 24577])
def test_sums_about_the_long_ones(M):
    # several groups, whole and cut ones, their sums one chunk, one row more, or several chunks long
    rng = np.random.default_rng(M)
    group = np.concatenate([np.zeros(M, int), np.full(500, 1), np.full(9000, 2)])
    rows, K, N = len(group), 264, 1100
    x, xd = held(rng.standard_normal((rows, K)), "bf16")
    dy, dyd = held(rng.standard_normal((rows, N)), "bf16")
    row_ptr = torch.from_numpy(csr(group, 4)[0]).cuda()
    perm = rng.permutation(rows)
    for pm in (None, torch.from_numpy(perm.astype(np.int32)).cuda()):
        at = (lambda t: t.cuda()) if pm is None else (lambda t: t[torch.from_numpy(np.argsort(perm))].cuda())
        dw = zs.zs_grouped_matmul_dw(at(dy), at(x), row_ptr, pm)
        torch.cuda.synchronize()
        zs.zs_check_timeouts()
        for g in range(3):
            r = group == g
            close(dw[g], dyd[r].T @ xd[r], np.abs(dyd[r]).T @ np.abs(xd[r]), "bf16", f"dw[{g}]")
        assert not bool(dw[3].any())
