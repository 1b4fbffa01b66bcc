"""Grouped products on the paths that only certain sizes take: tiles formed by two
CTAs, and more groups than shared memory holds the starts of.  Tolerances as in
test_grouped.py."""
import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import zs
from test_grouped import check_all, close, draw, run
from train_refs import csr, grouped

SMS = 152


def pairs(M, summed, cols, G, gathered):
    """Whether a product of 16-bit rows takes the kernel of two CTAs a tile: the rule of
    launch_rows (zs_grouped_rows.cu) and of the rows put in order (zs_grouped.cu)."""
    tiles = (cols + 127) // 128
    if cols <= 64 or tiles % 2 or gathered and cols < 1280:
        return False
    rows = M // 128 + min(G, M)
    cost = lambda n: -(-rows * -(-cols // n) // SMS) * (n + 96)  # noqa: E731
    narrow = summed <= 512 and 4 * cost(64) <= 3 * cost(256)
    return not narrow and M >= 512 * G


# M, K, N, G, sizes, gathered, which of y and dx are formed by pairs
PAIRS = [
    (7000, 1000, 984, 2, "uniform", False, "y dx"),      # ragged columns in the second CTA's half, either way round
    (7000, 1000, 984, 2, "zipf", False, "y dx"),
    (3000, 528, 136, 1, "one", False, "y"),              # eight columns in the second half
    (3000, 136, 520, 3, "uniform", False, "dx"),
    (20000, 64, 256, 3, "uniform", False, "y"),          # a sum of one stage
    (20000, 232, 16, 3, "zipf", False, "dx"),            # of 16 elements
    (2000, 1416, 1432, 3, "zipf", True, "y dx"),         # gathered rows put in order first
    (2100, 1400, 1528, 4, "one", True, "y"),
    (2560, 3000, 2296, 5, "uniform", False, "y dx"),     # sums that leave the tensor cores in between
]


def test_which_sizes_are_formed_by_pairs():
    for M, K, N, G, _, gathered, which in PAIRS:
        got = [n for n, r, c in (("y", K, N), ("dx", N, K)) if pairs(M, r, c, G, gathered)]
        assert " ".join(got) == which, (M, K, N, G, got)


@pytest.mark.gpu
@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != SMS,
                    reason="the rule counts SMs")
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,G,sizes,gathered,which", PAIRS)
def test_tiles_of_pairs(M, K, N, G, sizes, gathered, which, dtype):
    group, t, d = draw(M, K, N, G, dtype, M + K, sizes, bad=0.03)
    if not gathered:
        group = np.sort(group)      # rows of no group last
    first = check_all(group, t, d, dtype, ordered=not gathered)
    again = run(group, G, *(a.cuda() for a in t), ordered=not gathered)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("M,K,N,G", [(9000, 64, 96, 1023), (9000, 40, 264, 2000), (9000, 33, 47, 1500), (70000, 72, 40, 1200)])
def test_more_groups_than_are_held(M, K, N, G, gathered, dtype):
    # their starts are searched in global memory; most groups are empty or of a few rows
    group, t, d = draw(M, K, N, G, dtype, M + G, "zipf", bad=0.02)
    if not gathered:
        group = np.sort(group)
    check_all(group, t, d, dtype, ordered=not gathered)


@pytest.mark.gpu
@pytest.mark.parametrize("K,N,M", [(64, 48, 500), (24, 16, 500), (64, 48, 20), (24, 16, 4)])
def test_infinities_of_fp32(K, N, M):
    """An infinity or a NaN among fp32 operands: a result that is not finite, NaN or the
    infinity that its sum is, wherever it meets a factor, and nothing elsewhere."""
    group, (x, w, dy), d = draw(M, K, N, 2, "f32", K + M)
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(group, 2))
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    y = zs.zs_grouped_matmul(x.cuda(), w.cuda(), row_ptr, perm)
    dw = zs.zs_grouped_matmul_dw(dy.cuda(), x.cuda(), row_ptr, perm)
    ry, ay, _, _, rdw, adw = grouped(d[0], d[1], group, d[2])
    keep = ~np.isin(np.arange(M), (1, 2))
    close(y[keep], ry[keep], ay[keep], "f32", "y")
    assert not bool(torch.isfinite(y[1]).any()) and bool(torch.isnan(y[2]).all())
    plus = (torch.from_numpy(d[1][group[1], :, 3]) > 0).cuda()
    assert bool((torch.isnan(y[1]) | ((y[1] > 0) == plus)).all())
    sick = np.zeros(dw.shape, bool)
    sick[group[1], :, 3] = sick[group[2], :, 5] = True
    assert not bool(torch.isfinite(dw.cpu()[torch.from_numpy(sick)]).any())
    bound = 1e-5 * adw + 2.0 ** -24 * np.abs(rdw)
    assert (np.abs(dw.double().cpu().numpy() - rdw) <= bound)[~sick].all()
